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


class On:
    """A contiguous array of a device that need not be there."""

    is_cuda = True

    def __init__(self, device, shape, dtype):
        self.device, self.shape, self.dtype = torch.device("cuda", device), torch.Size(shape), dtype

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 4096


def test_every_tensor_has_to_be_on_the_device_of_the_call(S, monkeypatch):  # noqa: F811
    """Any one of them elsewhere is refused before the library is called."""
    called, S_lib = [], S.lib()

    class Library:
        def __getattr__(self, name):
            return S_lib.sffn_status_string if name == "sffn_status_string" else lambda *a: called.append(name) or 0

    monkeypatch.setattr(S, "lib", Library)
    monkeypatch.setattr(S, "_launch_stream", lambda stream: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    b, i = torch.bfloat16, torch.int32
    shapes = {"q": ((3, 8, 64), b), "k": ((5, 2, 16, 64), b), "v": ((5, 2, 16, 64), b), "table": ((2, 4), i), "ctx": ((2,), i),
              "cu": ((3,), i), "gs": ((2,), i), "pl": ((1,), i), "mask": ((3,), torch.int64), "out": ((3, 8, 64), b),
              "ws": ((4096,), torch.uint8), "pages": ((4,), i), "bounds": ((5, 2, 2, 64), b), "seqs": ((3,), i), "pos": ((3,), i),
              "sel": ((3, 2, 3), i), "n_sel": ((3,), i)}

    def call(name, elsewhere):
        x = {n: On(int(n == elsewhere), *s) for n, s in shapes.items()}
        cache = S.KVCache(x["k"], x["v"])
        if name == "attn_shared":
            S.attn_shared(x["q"], cache, x["table"], x["ctx"], x["cu"], x["gs"], x["pl"], x["mask"], out=x["out"], workspace=x["ws"])
        elif name == "page_bounds":
            S.page_bounds(cache, x["pages"], x["bounds"], workspace=x["ws"])
        elif name == "page_select":
            S.page_select(x["q"], cache, x["bounds"], x["table"], x["seqs"], x["pos"], 3, sel=x["sel"], n_sel=x["n_sel"],
                          workspace=x["ws"])
        else:
            S.attn_pages(x["q"], cache, x["table"], x["seqs"], x["pos"], x["sel"], x["n_sel"], out=x["out"], workspace=x["ws"])

    takes = {"attn_shared": "q k v table ctx cu gs pl mask out ws", "page_bounds": "k v pages bounds ws",
             "page_select": "q k v bounds table seqs pos sel n_sel ws", "attn_pages": "q k v table seqs pos sel n_sel out ws"}
    for name, tensors in takes.items():
        call(name, None)
        assert called == ["sffn_" + name]
        called.clear()
        for t in tensors.split():
            with pytest.raises(S.SffnError) as e:
                call(name, t)
            assert e.value.status == (S.ERR_WORKSPACE if t == "ws" else S.ERR_INVALID_ARG), (name, t)
            assert not called


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
