"""The Python binding of the long-context calls: the shapes that it takes, and whose memory."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import S  # noqa: F401  (the library)
from tests.test_long_contexts import Tokens, i32


def refused(S, status, fn, *a, **kw):  # noqa: F811
    with pytest.raises(S.SffnError) as e:
        fn(*a, **kw)
    assert e.value.status == status


def test_sizes_behind_the_first_are_exact(S):  # noqa: F811
    have = torch.empty(6, 2, 8)
    S._shaped(have, (6, 2, 8), "here")
    S._shaped(have, (5, 2, 8), "here")
    S._shaped(torch.empty(0, 2, 8), (0, 2, 8), "here")
    for shape in ((7, 2, 8), (6, 2, 4), (6, 1, 8), (6, 4, 4), (6, 16), (6, 2, 8, 1), (96,)):
        refused(S, S.ERR_SHAPE, S._shaped, have, shape, "here")


@pytest.mark.gpu
def test_lists_of_another_width_are_refused(S):  # noqa: F811
    """A fixed buffer wider than the lists would be filled with narrow rows and read with wide ones."""
    c = Tokens(S, [300, 90], [[299, 150], [89]], 8, 2, 64, 16, "bf16", 3, fill=0.0)
    for shape in ((3, 2, 8), (3, 2, 3), (3, 4, 4), (2, 2, 4), (3, 8), (24,), (3, 2, 4, 1)):
        refused(S, S.ERR_SHAPE, c.select, S, 4, sel=torch.zeros(shape, dtype=torch.int32, device="cuda"))
    refused(S, S.ERR_INVALID_ARG, c.select, S, 4, sel=torch.zeros(3, 2, 4, device="cuda"))
    good = c.select(S, 4)
    sel, n_sel = torch.full((5, 2, 4), 9, dtype=torch.int32, device="cuda"), i32([9] * 4)  # room for more tokens
    assert c.select(S, 4, sel=sel, n_sel=n_sel)[0] is sel
    assert torch.equal(sel[:3], good[0]) and (sel[3:] == 9).all()
    assert torch.equal(n_sel[:3], good[1]) and n_sel[3] == 9
    c.check_attention(c.attend(S, sel, n_sel), sel, n_sel)


@pytest.mark.gpu
def test_bounds_of_another_layout_are_refused(S):  # noqa: F811
    c = Tokens(S, [300], [[299]], 8, 2, 64, 16, "bf16", 3, fill=0.0)
    good, b = c.select(S, 4), c.bounds
    n = b.shape[0]
    for bad in (b.view(n, 2, 64, 2), b.view(n, 4, 1, 64), b.view(n, 2, 128), b.view(-1), b.view(n, 1, 2, 128), b[:-1]):
        c.bounds = bad
        refused(S, S.ERR_SHAPE, c.select, S, 4)
        refused(S, S.ERR_SHAPE, S.page_bounds, c.cache, i32([0]), bad)
    c.bounds = torch.cat([b, b[:1]])  # entries for pages that the cache does not have
    assert torch.equal(c.select(S, 4)[0], good[0])
    S.page_bounds(c.cache, i32([0]), c.bounds)
