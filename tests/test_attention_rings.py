"""The attention calls where a CTA has much to do: several items one after the other, many key tiles of an
item, shared-memory rings that go round and hand over from one item to the next.  References, inputs'
layout and tolerances are test_attention.py's."""
from __future__ import annotations

import pytest
import torch

from tests import test_attention as A
from tests.test_attention import S, check_attention, gen  # noqa: F401  (S: the library)


def packed(lens, hq, hkv, D, seed, scale=1.5):
    qkv = (torch.randn(sum(lens), hq + 2 * hkv, D, generator=gen(seed)) * scale).bfloat16()
    return qkv, torch.tensor([0] + lens).cumsum(0).int()


def prompt_call(S, qkv, cu, hq, hkv, ws=None):
    dev = qkv.cuda()
    return S.attn_prompt(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], cu.cuda(), workspace=ws).cpu()


def check_prompt_rows(got, qkv, lens, hq, hkv, D, rows):
    """Every head of the packed rows `rows` against the definition in 64 bits."""
    starts = torch.tensor([0] + lens).cumsum(0).tolist()
    for t in rows:
        s = next(i for i in range(len(lens)) if starts[i] <= t < starts[i + 1])
        a, G = starts[s], hq // hkv
        q = qkv[t, :hq].double().view(hkv, G, D)
        k, v = (qkv[a:t + 1, hq + i * hkv:hq + (i + 1) * hkv].double().permute(1, 0, 2) for i in range(2))
        w = torch.softmax(q @ k.transpose(1, 2) * D ** -0.5, -1)
        cond = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * D ** -0.5
        check_attention(got[t].view(hkv, G, D), w @ v, w @ v.abs(), cond, D, t - a + 1, True)


# Prompts a little longer than a block of 2 * 128 / G tokens, many more than there are CTAs: a CTA first gets
# several short rests (one row tile, so nothing for the second softmax group), then whole first blocks.
SHORT = [(400, 33, 48, 16, 2, 128), (800, 33, 48, 16, 2, 64), (300, 37, 53, 28, 4, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,lo,hi,hq,hkv,D", SHORT)
def test_prompt_short_rests_before_whole_blocks(S, n, lo, hi, hq, hkv, D):
    """Infinite values in every prompt's last row: that row alone has them, in every call, and every
    other row is what it is without them."""
    lens = [lo + (7 * i * i + 3 * i) % (hi - lo + 1) for i in range(n)]
    qkv, cu = packed(lens, hq, hkv, D, n + D)
    good = prompt_call(S, qkv, cu, hq, hkv)
    last = (cu[1:] - 1).long()
    check_prompt_rows(good, qkv, lens, hq, hkv, D, last[::7].tolist() + cu[:-1][::11].tolist() + [5, 40, 100, 999])
    hurt, want = qkv.clone(), good.clone()
    for i, t in enumerate(last.tolist()):
        x = float("inf") if i & 1 else -float("inf")
        hurt[t, hq + hkv:, i % D] = x
        want[t, :, i % D] = x
    for _ in range(5):
        assert torch.equal(prompt_call(S, hurt, cu, hq, hkv), want)
        assert torch.equal(prompt_call(S, qkv, cu, hq, hkv), good)


# 28/4 heads of 128: a block is 36 tokens, so a CTA of 152 gets three or four whole blocks
RAGGED = [100, 383, 700, 257, 129, 640, 36, 512, 333, 501, 128, 611]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,D,copies", [(28, 4, 128, 1), (16, 16, 64, 4), (12, 12, 128, 4), (64, 8, 64, 2)])
def test_prompt_several_whole_items_a_cta(S, hq, hkv, D, copies):
    """The rings of one item going on into the next, whole row tiles written while the next item runs; then
    with infinite values in the middle and at the end of each prompt."""
    lens = RAGGED * copies
    qkv, cu = packed(lens, hq, hkv, D, 17 + D)
    good = prompt_call(S, qkv, cu, hq, hkv)
    check_prompt_rows(good, qkv, lens, hq, hkv, D, list(range(0, sum(lens), 97)) + (cu[1:] - 1).tolist()[:12])
    assert torch.equal(prompt_call(S, qkv, cu, hq, hkv), good)
    hurt, want = qkv.clone(), good.clone()
    G = hq // hkv
    for i, n in enumerate(lens):
        a = int(cu[i])
        for t, h, col, x in ((n // 2, 0, 3, float("inf")), (n - 1, hkv - 1, 5, -float("inf"))):
            hurt[a + t, hq + hkv + h, col] = x
            want[a + t:a + n, h * G:(h + 1) * G, col] = x
    assert torch.equal(prompt_call(S, hurt, cu, hq, hkv), want)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_scores_that_grow_along_the_keys(S, D):
    """Every key tile passes the running maximum, in all items of a CTA: key j is (j / n) of a direction
    that every query has, for scores up to about 60."""
    lens, hq, hkv = [700, 650, 333, 1100], 16, 16
    qkv, cu = packed(lens, hq, hkv, D, 23, 0.4)
    for i, n in enumerate(lens):
        a = int(cu[i])
        qkv[a:a + n, :hq, :8] = 4.0
        qkv[a:a + n, hq:hq + hkv, :8] = (torch.arange(n) / n * 60 * D ** 0.5 / 32)[:, None, None].bfloat16()
    good = prompt_call(S, qkv, cu, hq, hkv)
    check_prompt_rows(good, qkv, lens, hq, hkv, D, list(range(0, sum(lens), 61)))


@pytest.mark.gpu
@pytest.mark.parametrize("n,hq,hkv,D", [(3000, 4, 2, 64), (1700, 4, 4, 128)])
def test_prompt_thousands_of_sequences(S, n, hq, hkv, D):
    """Lengths from 0 to a few blocks in no order, a few long ones far apart: every row belongs to its sequence."""
    lens = [(13 * i * i + 7 * i) % 90 if i % 5 else 0 for i in range(n)]
    for i, m in ((3, 900), (n // 2, 2000), (n - 1, 1400), (n - 200, 515)):
        lens[i] = m
    qkv, cu = packed(lens, hq, hkv, D, n)
    ws = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, sum(lens), n, hq, hkv, D)
    out = prompt_call(S, qkv, cu, hq, hkv, ws)
    assert S.read_device_error(ws) == 0
    last = [int(b) - 1 for a, b in zip(cu[:-1], cu[1:]) if b > a]
    check_prompt_rows(out, qkv, lens, hq, hkv, D, last[::9] + last[-3:] + list(range(0, sum(lens), 331)))
    assert torch.isfinite(out.float()).all()


@pytest.mark.gpu
def test_prompt_time_grows_with_the_sequences_not_with_their_square(S):
    """Four times the prompts of 16 tokens take about four times as long; finding each item by a search
    from the first sequence took fifteen times as long.  Half way between in ratio: eight."""
    hq, hkv, D = 16, 8, 128

    def best(n):
        q = torch.randn(16 * n, hq, D, device="cuda").bfloat16()
        k = torch.randn(16 * n, hkv, D, device="cuda").bfloat16()
        cu = (torch.arange(n + 1, device="cuda") * 16).int()
        ws, out = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, 16 * n, n, hq, hkv, D), torch.empty_like(q)
        times = []
        for _ in range(6):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            S.attn_prompt(q, k, k, cu, out=out, workspace=ws)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times[1:])

    assert best(16384) < 8 * best(4096)


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

def check_tree_rows(p, got, tokens):
    """Every head of the packed new tokens `tokens` against the definition in 64 bits."""
    got, G = got.cpu(), p.hq // p.hkv
    for t in tokens:
        s = next(i for i in range(len(p.n)) if p.cu[i] <= t < p.cu[i + 1])
        c, n = p.ctx[s], p.n[s]
        sees = torch.ones(c + n, dtype=torch.bool)
        sees[c:] = torch.tensor([(p.masks[t] >> j) & 1 for j in range(n)], dtype=torch.bool)
        q = p.q[t].double().view(p.hkv, G, p.D)
        k, v = (x[s][sees].double().permute(1, 0, 2) for x in (p.k, p.v))
        w = torch.softmax(q @ k.transpose(1, 2) * p.D ** -0.5, -1)
        cond = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * p.D ** -0.5
        check_attention(got[t].view(p.hkv, G, p.D), w @ v, w @ v.abs(), cond, p.D, c + n, p.dt == "bf16")


# ctx, new tokens, hq, hkv, D, page, dtype, growing scores
LONG = [
    ([13000], [8], 64, 8, 64, 64, "bf16", False),
    ([13000], [8], 64, 8, 128, 64, "bf16", False),
    ([13003], [1], 8, 8, 128, 16, "bf16", True),
    ([12997], [3], 16, 8, 64, 128, "bf16", True),
    ([20000], [2], 4, 1, 128, 256, "bf16", True),       # one item in 152 pieces
    ([20000], [2], 4, 1, 64, 256, "f32", False),
    ([9000, 4001], [5, 2], 8, 8, 64, 64, "f32", True),
    ([6000], [8], 16, 8, 128, 64, "f32", True),
    # many items: several whole ones a CTA
    ([300, 517, 64, 449, 0, 601, 333, 128] * 5, [64, 40, 33, 64, 64, 1, 50, 64] * 5, 32, 8, 128, 32, "bf16", False),
    ([300, 517, 64, 449, 0, 601, 333, 128] * 5, [64, 40, 33, 64, 64, 1, 50, 64] * 5, 28, 4, 64, 16, "bf16", True),
    ([300, 517, 64, 449, 0, 601] * 4, [20, 40, 1, 64, 30, 1] * 4, 16, 8, 64, 32, "f32", True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,n,hq,hkv,D,page,dt,grow", LONG)
def test_tree_long_contexts_and_many_items(S, ctx, n, hq, hkv, D, page, dt, grow):
    """Unused places of the pages hold NaN.  With `grow`, key j is (j / n) of a direction that every query has:
    the running maximum moves at every tile."""
    p = A.Paged(S, ctx, n, hq, hkv, D, page, dt, sum(ctx) + hq + D)
    if grow:
        p.q[:, :, :8] = 4.0
        for s, (c, m) in enumerate(zip(ctx, n)):
            up = (torch.arange(c + m) / (c + m) * 60 * D ** 0.5 / 32)[:, None, None].expand(-1, hkv, 8).to(p.ck.dtype)
            p.k[s][:, :, :8] = up
            j = torch.arange(c + m)
            p.ck[p.table[s][j // page].long().cuda(), :, (j % page).cuda(), :8] = up.cuda()
    ws = S.alloc_attn_workspace(S.WS_ATTN_TREE, sum(n), len(n), hq, hkv, D)
    out = p.call(S, workspace=ws)
    assert S.read_device_error(ws) == 0
    T = sum(n)
    check_tree_rows(p, out, sorted({t for t in range(0, T, max(1, T // 40))} | {T - 1}))
    assert torch.equal(out, p.call(S, workspace=ws))


# ---------------------------------------------------------------------------
# norms and rotation of many rows: several rows a lane
# ---------------------------------------------------------------------------

MANY = [
    # T, hq, hkv, D, dtype, interleaved, rot, page, cache, k_out
    (300, 32, 2, 128, "bf16", False, 128, 64, True, True),
    (333, 28, 4, 128, "bf16", True, 64, 16, True, False),
    (301, 33, 3, 128, "bf16", True, 128, 32, True, True),
    (700, 16, 2, 64, "bf16", True, 64, 16, True, False),
    (310, 32, 2, 128, "f32", False, 64, 64, True, True),
    (333, 31, 1, 128, "f32", True, 128, 16, True, False),
    (640, 14, 2, 64, "f32", False, 64, 32, True, True),
    (640, 16, 4, 64, "f32", True, 32, 16, False, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,hq,hkv,D,dt,inter,rot,page,cached,k_out", MANY)
def test_rope_of_many_rows(S, T, hq, hkv, D, dt, inter, rot, page, cached, k_out):
    assert T * (hq + 2 * hkv) >= 64 * 152
    A.test_qk_norm_rope(S, T, hq, hkv, D, dt, True, inter, rot, page, cached, k_out)
