"""What a row does not see has no influence on it, to the last bit: of the few-row kernels the partial results are
compared (fp32, in the workspace, where no rounding to bf16 hides a sum made in another order), with the same calls over caches
whose unseen places hold zeros, NaN, infinities or the largest finite values."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import Paged, S  # noqa: F401  (S: the library)
from tests.test_long_contexts import Tokens, call_shared, share

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), -float("inf"), 3e38]


def same_bits(ws, call):
    """The workspace (all zeros before) and the output that the call leaves."""
    ws.zero_()
    out = call()
    return ws.clone(), out


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens,at,hq,hkv,D,page", [
    ([1990], [[1989]], 8, 2, 128, 16),
    ([700, 77, 1031], [[699, 500], [76], [1030, 3]], 16, 8, 128, 8),
    ([900, 555], [[899, 20], [554]], 20, 2, 64, 32),
    ([1300], [[1291, 1292, 1283]], 48, 2, 64, 8),
])
def test_attn_pages_partial_results(S, lens, at, hq, hkv, D, page, dt, bad):  # noqa: F811
    kept = []
    for fill in (0.0, bad):
        c = Tokens(S, lens, at, hq, hkv, D, page, dt, sum(lens), fill=fill)
        if not kept:
            ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, len(c.pos), len(lens), hq, hkv, D)
            sel, n_sel = c.select(S, max(lens) // page + 1)
        kept.append(same_bits(ws, lambda: c.attend(S, sel, n_sel, workspace=ws)))
        c.check_attention(kept[-1][1], sel, n_sel)
    assert torch.equal(kept[0][1], kept[1][1])
    assert torch.equal(kept[0][0], kept[1][0])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("groups,prefix,own,n,hq,hkv,D,page", [
    ([3, 1], [500, 0], [10, 333, 0, 700], [1, 2, 1, 1], 8, 4, 128, 16),
    ([2, 2], [64, 129], [1001, 3, 60, 515], [3, 1, 2, 2], 4, 2, 64, 8),
    ([5], [900], [5, 1, 300, 2, 90], [1, 1, 1, 1, 1], 32, 2, 64, 64),
    ([30], [530], [(17 * i) % 90 for i in range(30)], [1] * 30, 16, 2, 128, 32),   # the prefix on the tensor cores
    ([2, 1], [640, 0], [7, 100, 900], [40, 33, 64], 8, 2, 64, 16),                 # all of it
    ([1], [300], [1700], [20], 7, 1, 128, 128),
])
def test_attn_shared_partial_results(S, groups, prefix, own, n, hq, hkv, D, page, dt, bad):  # noqa: F811
    of = [x for m, x in zip(groups, prefix) for _ in range(m)]
    ctx = [a + b for a, b in zip(of, own)]
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, sum(n), len(n), hq, hkv, D)
    kept = []
    for fill in (0.0, bad):
        p = Paged(S, ctx, n, hq, hkv, D, page, dt, sum(own), fill=fill)
        share(p, groups, prefix, page)
        kept.append(same_bits(ws, lambda: call_shared(S, p, groups, prefix, workspace=ws)))
        p.check(kept[-1][1])
    assert torch.equal(kept[0][1], kept[1][1])
    assert torch.equal(kept[0][0], kept[1][0])


@pytest.mark.parametrize("bad", BAD[:3])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D,page", [(8, 4, 128, 16), (4, 2, 64, 8), (12, 2, 64, 32)])
def test_a_value_that_some_rows_see_reaches_those_alone(S, hq, hkv, D, page, dt, bad):  # noqa: F811
    """One new token's values are non-finite: of the partial results whatever changes is non-finite, and the rows of
    the tokens that do not see it keep theirs."""
    n, ctx = [4, 2, 1], [777, 90, 300]
    p = Paged(S, ctx, n, hq, hkv, D, page, dt, 11, fill=0.0)
    masks = [0b0001, 0b0011, 0b0101, 0b1010, 0b01, 0b11, 0b1]  # tokens 1 and 3 of the first sequence see its token 1
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, 7, 3, hq, hkv, D)
    a, good = same_bits(ws, lambda: call_shared(S, p, [3], [0], masks, workspace=ws))
    p.check(good, masks)
    j = ctx[0] + 1
    p.cv[int(p.table[0, j // page]), :, j % page] = bad
    b, got = same_bits(ws, lambda: call_shared(S, p, [3], [0], masks, workspace=ws))
    keep = [0, 2, 4, 5, 6]
    assert torch.equal(got[keep], good[keep])
    want = bad if dt == "f32" or bad != bad else torch.tensor(bad).to(torch.bfloat16).item()
    assert torch.equal(got[[1, 3]].nan_to_num(nan=7.0), torch.full_like(got[[1, 3]], want).nan_to_num(nan=7.0))
    changed = a.view(torch.int32) != b.view(torch.int32)
    assert changed.any() and not torch.isfinite(b.view(torch.float32)[changed]).any()


@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (16, 2, 64)])
def test_half_a_tile_is_not_taken_from_what_shared_memory_held(S, hq, hkv, D):  # noqa: F811
    """Pages of 8, the last tile of 16 with 8 keys or fewer: its other half is what an earlier call left there."""
    full = Tokens(S, [512] * 160, [[511]] * 160, hq, hkv, D, 8, "bf16", 3, fill=0.0)
    lists = full.select(S, 64)
    c = Tokens(S, [1000, 300, 72, 20], [[963, 899, 515], [259, 131], [67, 71], [3]], hq, hkv, D, 8, "bf16", 5, fill=0.0)
    sel, n_sel = c.select(S, 125)
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, len(c.pos), 4, hq, hkv, D)
    w2 = S.alloc_attn_workspace(S.WS_ATTN_PAGES, 160, 160, hq, hkv, D)
    kept = []
    for value in (0.0, float("nan"), float("inf"), 1.0):
        full.p.cv.fill_(value)
        ws.zero_()
        torch.cuda.synchronize()
        full.attend(S, *lists, workspace=w2)
        out = c.attend(S, sel, n_sel, workspace=ws)
        c.check_attention(out, sel, n_sel)
        kept.append((ws.clone(), out))
    for w, out in kept[1:]:
        assert torch.equal(out, kept[0][1])
        assert torch.equal(w, kept[0][0])
