"""The serving example's draft-tree step against the definition in 64 bits, with the bound of
test_attention.py's docstring: each drafted token sees its context, itself and its ancestors and nothing
else.  The bound is tight enough to tell: the same outputs miss it for masks that swap the two siblings,
leave out a token itself or its ancestor, or let it see its sibling."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

from tests.test_attention import H, S  # noqa: F401  (S: the library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def bound(got, q, k, v):
    """Largest error of a token's heads, in units of its bound; q [hq, D], k and v [n, hkv, D] of the keys that it sees."""
    hkv, D, n = k.shape[1], k.shape[2], k.shape[0]
    q = q.double().view(hkv, -1, D)
    k, v = k.double().transpose(0, 1), v.double().transpose(0, 1)
    w = torch.softmax(q @ k.transpose(1, 2) * D ** -0.5, -1)
    ref, mag = w @ v, w @ v.abs()
    cond = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * D ** -0.5
    d = D * 2.0 ** -23 * cond + 2.0 ** -20
    tol = (2 * d + n * 2.0 ** -23 + H) * mag + H * ref.abs() + 1e-30
    return ((got.double().view(hkv, -1, D) - ref).abs() / tol).max().item()


@pytest.mark.gpu
def test_every_drafted_token_sees_its_branch_and_nothing_else(S, monkeypatch):  # noqa: F811
    spec = importlib.util.spec_from_file_location("serve_layer", os.path.join(ROOT, "examples", "serve_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    seen, attn_tree = {}, S.attn_tree

    def tree(q, cache, table, ctx, cu, mask):
        seen.update(q=q.clone(), k=cache.k.clone(), v=cache.v.clone(), table=table.cpu(), ctx=ctx.tolist(), cu=cu.tolist())
        return attn_tree(q, cache, table, ctx, cu, mask)

    monkeypatch.setattr(mod.sffn, "attn_tree", tree)
    r = mod.run()
    got, q = r["decode_attention"].cpu(), seen["q"].cpu()
    page = seen["k"].shape[2]

    def rows(c, s, at):  # logical positions of sequence s -> [n, hkv, D]
        at = torch.tensor(at)
        return c.cpu()[seen["table"][s][at // page].long(), :, at % page]

    def error(t, s, new):
        at = list(range(seen["ctx"][s])) + [seen["ctx"][s] + j for j in new]
        return bound(got[t], q[t], rows(seen["k"], s, at), rows(seen["v"], s, at))

    assert seen["ctx"] == [300, 77] and seen["cu"] == [0, 3, 4]
    for t, s, new in ((0, 0, [0]), (1, 0, [0, 1]), (2, 0, [0, 2]), (3, 1, [0])):
        assert error(t, s, new) <= 1.0, t
    for t, s, wrong in ((0, 0, []), (0, 0, [0, 1]), (1, 0, [0, 2]), (1, 0, [1]), (1, 0, [0]), (1, 0, [0, 1, 2]), (2, 0, [0, 1]),
                        (2, 0, [2]), (2, 0, [0, 1, 2]), (3, 1, [])):
        assert error(t, s, wrong) > 1.0, (t, wrong)
    # and the same tokens run as prompts: one bound each
    for i, (t, s, new) in enumerate(((1, 0, [0, 1]), (2, 0, [0, 2]), (3, 1, [0]))):
        at = list(range(seen["ctx"][s])) + [seen["ctx"][s] + j for j in new]
        assert bound(r["as_prompts"][i].cpu(), q[t], rows(seen["k"], s, at), rows(seen["v"], s, at)) <= 1.0
