"""The attention half of the layer: head norms with rotation and the cache's new rows
(sffn_qk_norm_rope), attention over packed prompts (sffn_attn_prompt) and of drafted
tokens over the paged cache (sffn_attn_tree), against plain 64-bit implementations.

Tolerances, per output element, from the arithmetic (u = 2^-24, bf16, 8 significant bits, rounding h = 2^-8):
* norm + rotation: the sum of squares (8 terms a lane, then 4 levels) is good to 12 u, its
  root to half of that, and the root, the division, two products with the weight, the
  product with the cosine and the sum add an u or so each: 16 u of |y_a| + |y_b|, and
  h |out| for a bf16 output.
* attention: the score's D products accumulate to D 2^-23 of sum |q||k| scale; with the
  exponential's own 2^-20 that is d, a weight's relative error, and a ratio of sums of
  weights is off by 2 d at most; n keys add n 2^-23; bf16 weights and output add h each:
  (2 d + n 2^-23 + h) sum w|v| + h |out|  (no h for fp32)."""
from __future__ import annotations

import ctypes as C
import math

import pytest
import torch

U, H = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def S():
    from activation_sparse_ffn_gemv_gb300 import build as B
    B.build()
    from activation_sparse_ffn_gemv_gb300 import sffn
    sffn.lib()
    return sffn


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def dtype_of(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ---------------------------------------------------------------------------
# references, 64 bits, CPU
# ---------------------------------------------------------------------------

def ref_rope(x, w, table, pos, rot, interleaved, eps):
    """(out, |y_a| + |y_b| of each element's pair), [T, heads, D] double."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    out, mag = y.clone(), y.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, s = table[pos.long(), i].double()[:, None], table[pos.long(), rot // 2 + i].double()[:, None]
        ya, yb = y[..., a], y[..., b]
        out[..., a] = ya * c - yb * s
        out[..., b] = yb * c + ya * s
        mag[..., a] = mag[..., b] = ya.abs() + yb.abs()
    return out, mag


def ref_attention(q, k, v, sees, scale):
    """q [r, D], k, v [n, D], sees [r, n]: out, and the two factors of its error bound.  A key
    that is not seen takes no part; a row that sees nothing is zero."""
    q, k, v = q.double(), k.double(), v.double()
    out = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    cond = torch.zeros(q.shape[0], 1, dtype=torch.float64)
    for i in range(q.shape[0]):
        at = sees[i].nonzero()[:, 0]
        if at.numel() == 0:
            continue
        s = (k[at] @ q[i]) * scale
        w = torch.softmax(s, 0)
        out[i] = w @ v[at]
        mag[i] = w @ v[at].abs()
        cond[i] = (k[at].abs() @ q[i].abs()).max() * scale
    return out, mag, cond


def check_attention(got, ref, mag, cond, D, n, bf16):
    h = H if bf16 else 0.0
    d = D * 2.0 ** -23 * cond + 2.0 ** -20
    tol = (2 * d + n * 2.0 ** -23 + h) * mag + (h or U) * ref.abs() + 1e-30
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.float()).all()
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3f} of the bound"


# ---------------------------------------------------------------------------
# norms, rotation, cache rows
# ---------------------------------------------------------------------------

ROPE = [
    # T, hq, hkv, D, dtype, norm, interleaved, rot, page, cache, k_out
    (1, 32, 32, 128, "bf16", False, False, 128, 16, True, False),
    (1, 1, 1, 64, "f32", True, True, 64, 8, True, True),
    (7, 16, 2, 64, "f32", True, True, 32, 32, True, False),
    (61, 5, 1, 128, "bf16", True, False, 64, 16, True, True),
    (130, 28, 4, 128, "bf16", True, True, 128, 128, True, False),
    (33, 12, 12, 64, "bf16", True, False, 16, 64, False, True),
    (19, 8, 2, 128, "f32", True, False, 112, 16, True, True),
    (300, 64, 8, 64, "bf16", True, False, 64, 64, True, True),
    (5, 4, 2, 128, "f32", True, False, 0, 16, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,hq,hkv,D,dt,norm,inter,rot,page,cached,k_out", ROPE)
def test_qk_norm_rope(S, T, hq, hkv, D, dt, norm, inter, rot, page, cached, k_out):
    g, td, eps = gen(T * 31 + D), dtype_of(dt), 1e-5
    qkv = (torch.randn(T, hq + 2 * hkv + 1, D, generator=g) * 2).to(td)  # wider than the heads: a real stride
    if T > 2:
        qkv[1, 0] = 0  # a row of zeros
    wq = (1 + 0.3 * torch.randn(D, generator=g)).to(td) if norm else None
    wk = (1 + 0.3 * torch.randn(D, generator=g)).to(td) if norm and T != 61 else None
    max_pos = 5000
    table = S.rope_table(max_pos, rot, device="cpu") if rot else None
    pos = torch.randint(0, max_pos, (T,), generator=g).int()
    n_pages = (T + page - 1) // page + 2
    slots = torch.randperm(n_pages * page, generator=g)[:T].int()
    if T > 4:
        slots[3] = -1
    dev = qkv.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:hq + 2 * hkv]
    ck = torch.full((n_pages, hkv, page, D), 7.0, dtype=td, device="cuda")
    cv = torch.full_like(ck, -7.0)
    cache = S.KVCache(ck, cv) if cached else None
    ko = torch.empty(T, hkv, D, dtype=td, device="cuda") if k_out else None
    ws = S.alloc_attn_workspace(S.WS_QK_NORM_ROPE, T, 1, hq, hkv, D)
    qo, kk = S.qk_norm_rope(q, k, v, None if table is None else table.cuda(), pos.cuda(),
                            q_weight=None if wq is None else wq.cuda(), k_weight=None if wk is None else wk.cuda(),
                            eps=eps, style=S.ROPE_INTERLEAVED if inter else S.ROPE_HALF, cache=cache,
                            slots=slots.cuda() if cached else None, k_out=ko, workspace=ws)
    assert S.read_device_error(ws) == 0
    table = table if rot else torch.zeros(max_pos, 0)

    def check(got, x, w):
        ref, mag = ref_rope(x, w, table, pos, rot, inter, eps)
        tol = 16 * U * mag + (H if dt == "bf16" else U) * ref.abs() * 1.01 + 1e-30
        assert ((got.cpu().double() - ref).abs() <= tol).all()

    check(qo, qkv[:, :hq], wq)
    if kk is not None:
        check(kk, qkv[:, hq:hq + hkv], wk)
    if cached:
        flat_k = ck.transpose(1, 2).reshape(n_pages * page, hkv, D).cpu()
        flat_v = cv.transpose(1, 2).reshape(n_pages * page, hkv, D).cpu()
        put = slots >= 0
        if kk is not None:
            assert torch.equal(flat_k[slots[put].long()], kk.cpu()[put])
        else:
            ref, mag = ref_rope(qkv[:, hq:hq + hkv], wk, table, pos, rot, inter, eps)
            tol = 16 * U * mag + (H if dt == "bf16" else U) * ref.abs() * 1.01 + 1e-30
            assert ((flat_k[slots[put].long()].double() - ref[put]).abs() <= tol[put]).all()
        assert torch.equal(flat_v[slots[put].long()], qkv[:, hq + hkv:hq + 2 * hkv][put])
        rest = torch.ones(n_pages * page, dtype=torch.bool)
        rest[slots[put].long()] = False
        assert (flat_k[rest] == 7).all() and (flat_v[rest] == -7).all()  # nothing else was written


@pytest.mark.gpu
def test_qk_norm_rope_in_place_and_contract_errors(S):
    T, hq, hkv, D, page = 6, 4, 2, 64, 16
    g = gen(3)
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16().cuda() for h in (hq, hkv, hkv))
    table = S.rope_table(100, D)
    pos = torch.arange(T).int().cuda()
    qo, ko = S.qk_norm_rope(q, k, None, table, pos)
    q2, k2 = q.clone(), k.clone()
    S.qk_norm_rope(q2, k2, None, table, pos, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    # a position beyond the table: that token is skipped and recorded, the others are written
    ws = S.alloc_attn_workspace(S.WS_QK_NORM_ROPE, T, 1, hq, hkv, D)
    bad = pos.clone()
    bad[2] = 100
    mark = torch.full_like(q, 5.0)
    S.qk_norm_rope(q, k, None, table, bad, q_out=mark, workspace=ws)
    assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(mark[keep], qo[keep]) and (mark[2] == 5).all()
    # slots outside the cache: skipped and recorded
    ck = torch.zeros(2, hkv, page, D, dtype=torch.bfloat16, device="cuda")
    cv = torch.zeros_like(ck)
    slots = torch.tensor([0, 1, 32, -2, 31, -1], dtype=torch.int32, device="cuda")
    S.qk_norm_rope(q, k, v, table, pos, cache=S.KVCache(ck, cv), slots=slots, workspace=ws)
    assert S.read_device_error(ws) == S.ERR_DEVICE
    assert torch.equal(cv[0, :, 0], v[0]) and torch.equal(cv[0, :, 1], v[1]) and torch.equal(cv[1, :, 15], v[4])
    assert int((cv != 0).any(-1).sum()) == 3 * hkv


# ---------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------

PROMPT = [
    ([1], 1, 1, 64),
    ([1, 17, 130, 0, 44], 16, 2, 128),
    ([129, 127, 128, 257], 4, 4, 128),
    ([300, 0, 0, 5], 5, 1, 64),
    ([515], 14, 2, 64),
    ([64, 65, 63], 64, 1, 128),
    ([0, 700], 6, 2, 128),
    ([33] * 40, 8, 8, 64),
    ([1100], 3, 3, 128),
]


def prompt_inputs(lens, hq, hkv, D, seed, scale=1.5):
    T = sum(lens)
    qkv = (torch.randn(T, hq + 2 * hkv, D, generator=gen(seed)) * scale).bfloat16()
    cu = torch.tensor([0] + lens).cumsum(0).int()
    return qkv, cu


def ref_prompt(qkv, lens, hq, hkv, D, rows=None):
    outs = [torch.zeros(qkv.shape[0], hq, D, dtype=torch.float64) for _ in range(2)]
    cond = torch.zeros(qkv.shape[0], hq, 1, dtype=torch.float64)
    t0 = 0
    for n in lens:
        sees = torch.ones(n, n, dtype=torch.bool).tril()
        for h in range(hq):
            kv = hq + h // (hq // hkv)
            o, m, c = ref_attention(qkv[t0:t0 + n, h], qkv[t0:t0 + n, kv], qkv[t0:t0 + n, kv + hkv], sees, D ** -0.5)
            outs[0][t0:t0 + n, h], outs[1][t0:t0 + n, h], cond[t0:t0 + n, h] = o, m, c
        t0 += n
    return outs[0], outs[1], cond


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hq,hkv,D", PROMPT)
def test_attn_prompt(S, lens, hq, hkv, D):
    qkv, cu = prompt_inputs(lens, hq, hkv, D, sum(lens) + hq)
    dev = qkv.cuda()
    ws = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, dev.shape[0], len(lens), hq, hkv, D)
    args = (dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], cu.cuda())
    out = S.attn_prompt(*args, workspace=ws)
    assert S.read_device_error(ws) == 0
    check_attention(out.cpu(), *ref_prompt(qkv, lens, hq, hkv, D), D, max(lens), True)
    assert torch.equal(out, S.attn_prompt(*args, workspace=ws))  # equal calls, equal bits


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_attn_prompt_unseen_rows_have_no_influence(S, D, bad):
    """Row 200 of the second sequence holds `bad` in k and v: the rows before it and the other
    sequences are what they are without it."""
    lens, hq, hkv = [150, 290, 70], 4, 2
    qkv, cu = prompt_inputs(lens, hq, hkv, D, 11)
    hurt = qkv.clone()
    hurt[150 + 200, hq:] = bad
    good = S.attn_prompt(*(t.cuda() for t in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])), cu.cuda())
    got = S.attn_prompt(*(t.cuda() for t in (hurt[:, :hq], hurt[:, hq:hq + hkv], hurt[:, hq + hkv:])), cu.cuda())
    clear = [t for t in range(sum(lens)) if not 350 <= t < 440]
    assert torch.equal(got[clear], good[clear])
    if not math.isfinite(bad):
        assert not torch.isfinite(got[350].float()).all()  # the row that sees it shows it


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_attn_prompt_infinite_values_reach_the_rows_that_see_them(S, D):
    """An infinite value element: the rows from its own on have it in that column, and only there."""
    lens, hq, hkv = [400], 4, 2
    qkv, cu = prompt_inputs(lens, hq, hkv, D, 5, 0.5)
    hurt = qkv.clone()
    hurt[290, hq + hkv, 3] = float("inf")
    hurt[130, hq + hkv, 9] = -float("inf")
    good = S.attn_prompt(*(t.cuda() for t in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:])), cu.cuda()).cpu()
    got = S.attn_prompt(*(t.cuda() for t in (hurt[:, :hq], hurt[:, hq:hq + hkv], hurt[:, hq + hkv:])), cu.cuda()).cpu()
    want = good.clone()
    want[290:, :2, 3] = float("inf")
    want[130:, :2, 9] = -float("inf")
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_attn_prompt_peaked_and_flat_scores(S):
    """Scores of +-200 (weights of one key) in one head, all zero (the mean of the values) in another,
    and scores that grow along the keys, so that the running maximum moves at every step."""
    lens, hq, hkv, D = [700], 3, 3, 128
    qkv, cu = prompt_inputs(lens, hq, hkv, D, 8)
    qkv[:, 0] *= 12
    qkv[:, 1] = 0
    qkv[:, 2] = 1.0
    qkv[:, hq + 2] = (torch.arange(700)[:, None] * 0.01 * torch.ones(1, D)).bfloat16()
    dev = qkv.cuda()
    out = S.attn_prompt(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], cu.cuda())
    check_attention(out.cpu(), *ref_prompt(qkv, lens, hq, hkv, D), D, 700, True)


@pytest.mark.gpu
def test_attn_prompt_bad_offsets_are_skipped_and_recorded(S):
    hq, hkv, D = 4, 2, 64
    qkv, _ = prompt_inputs([100], hq, hkv, D, 2)
    dev = qkv.cuda()
    ws = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, 100, 3, hq, hkv, D)
    args = (dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:])
    for cu in ([0, 40, 101, 100], [0, 40, 30, 100], [-5, 40, 40, 100]):
        out = torch.full((100, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        S.attn_prompt(*args, torch.tensor(cu, dtype=torch.int32).cuda(), out=out, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0


# ---------------------------------------------------------------------------
# drafted tokens over the paged cache
# ---------------------------------------------------------------------------

def random_masks(n, g, full=False):
    u = torch.rand(n, generator=g).tolist()
    masks = []
    for i in range(n):
        parent = int(u[i] * (i + 1)) - 1
        masks.append((1 << i) | (masks[parent] if parent >= 0 else 0))
    return masks


def signed(m):
    return m - (1 << 64) if m >> 63 else m


class Paged:
    """Sequences in a shuffled paged cache whose unused places hold `fill`."""

    def __init__(self, S, ctx, n, hq, hkv, D, page, dt, seed, fill=float("nan"), first_page=0, extra=3):
        g, td = gen(seed), dtype_of(dt)
        self.ctx, self.n, self.hq, self.hkv, self.D, self.dt = ctx, n, hq, hkv, D, dt
        keys = [c + m for c, m in zip(ctx, n)]
        need = [(m + page - 1) // page for m in keys]
        n_pages = first_page + sum(need) + extra
        self.k = [torch.randn(m, hkv, D, generator=g).to(td) for m in keys]
        self.v = [torch.randn(m, hkv, D, generator=g).to(td) for m in keys]
        self.q = (torch.randn(sum(n), hq + 1, D, generator=g) * 1.5).to(td)[:, :hq]
        order = (torch.randperm(sum(need) + extra, generator=g) + first_page).tolist()
        self.ck = torch.empty(n_pages, hkv, page, D, dtype=td, device="cuda")
        self.cv = torch.empty_like(self.ck)
        self.ck[first_page:] = fill
        self.cv[first_page:] = fill
        self.table = torch.zeros(len(ctx), max(need) + 1, dtype=torch.int32)
        for s, m in enumerate(need):
            ids, order = order[:m], order[m:]
            self.table[s, :m] = torch.tensor(ids, dtype=torch.int32)
            for i, p in enumerate(ids):
                a, b = i * page, min(keys[s], (i + 1) * page)
                self.ck[p, :, : b - a] = self.k[s][a:b].transpose(0, 1).cuda()
                self.cv[p, :, : b - a] = self.v[s][a:b].transpose(0, 1).cuda()
        self.cache = S.KVCache(self.ck, self.cv)
        self.masks = sum((random_masks(m, g) for m in n), [])
        self.cu = torch.tensor([0] + n).cumsum(0).int()

    def call(self, S, masks="own", **kw):
        masks = self.masks if masks == "own" else masks
        dm = None if masks is None else torch.tensor([signed(m) for m in masks], dtype=torch.int64).cuda()
        q = torch.empty(self.q.shape[0], self.hq + 2, self.D, dtype=self.q.dtype, device="cuda")[:, :self.hq]
        q.copy_(self.q)
        return S.attn_tree(q, self.cache, self.table.cuda(), torch.tensor(self.ctx, dtype=torch.int32).cuda(),
                           self.cu.cuda(), dm, **kw)

    def check(self, got, masks="own"):
        masks = self.masks if masks == "own" else masks
        got, G = got.cpu(), self.hq // self.hkv
        for s, (c, n) in enumerate(zip(self.ctx, self.n)):
            t0 = int(self.cu[s])
            sees = torch.ones(n, c + n, dtype=torch.bool)
            for i in range(n):
                word = ((1 << (i + 1)) - 1) if masks is None else masks[t0 + i]
                sees[i, c:] = torch.tensor([(word >> j) & 1 for j in range(n)], dtype=torch.bool)
            for h in range(self.hq):
                ref = ref_attention(self.q[t0:t0 + n, h], self.k[s][:, h // G], self.v[s][:, h // G], sees,
                                    self.D ** -0.5)
                check_attention(got[t0:t0 + n, h], *ref, self.D, c + n, self.dt == "bf16")


TREE = [
    # ctx, new tokens, hq, hkv, D, page, dtype
    ([0], [1], 1, 1, 64, 8, "bf16"),
    ([300], [1], 32, 32, 128, 16, "bf16"),
    ([1999, 300, 700, 0], [8, 5, 1, 7], 16, 2, 64, 32, "f32"),
    ([0, 17, 64, 1095, 63, 65], [1, 1, 1, 1, 1, 1], 8, 2, 128, 16, "bf16"),
    ([777], [8], 64, 8, 128, 64, "bf16"),
    ([130, 0, 401, 63], [64, 25, 33, 60], 28, 4, 128, 128, "bf16"),
    ([250, 3], [64, 64], 20, 20, 64, 256, "bf16"),
    ([100], [3], 64, 1, 128, 8, "bf16"),
    ([511], [64], 64, 1, 64, 32, "bf16"),
    ([129] * 70, [1, 0, 2] * 23 + [5], 5, 1, 64, 16, "bf16"),
    ([40, 2100], [64, 3], 5, 1, 128, 64, "f32"),
    ([77], [2], 64, 1, 64, 16, "f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,n,hq,hkv,D,page,dt", TREE)
def test_attn_tree(S, ctx, n, hq, hkv, D, page, dt):
    p = Paged(S, ctx, n, hq, hkv, D, page, dt, sum(ctx) + hq)
    ws = S.alloc_attn_workspace(S.WS_ATTN_TREE, sum(n), len(n), hq, hkv, D)
    out = p.call(S, workspace=ws)
    assert S.read_device_error(ws) == 0
    p.check(out)
    assert torch.equal(out, p.call(S, workspace=ws))  # equal calls, equal bits
    p.check(p.call(S, masks=None, workspace=ws), masks=None)  # a chain


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_tree_rows_that_see_little_or_nothing(S, dt):
    """No committed position: a token that sees nothing is zero, one that sees only another token
    is that token's value row; bits beyond the new tokens are ignored."""
    p = Paged(S, [0, 0, 70], [4, 1, 3], 6, 2, 64, 16, dt, 4)
    masks = [0, 0b0001, 0b1010, (1 << 63) | 0b1000, 0b10, 0, 0b111, 0b100]
    out = p.call(S, masks)
    p.check(out, masks)
    assert not out[0].any() and not out[4].any()
    assert torch.equal(out[1].cpu(), p.v[0][0].repeat_interleave(3, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_tree_unseen_places_have_no_influence(S, dt, bad):
    """Stale contents of unused places and drafted tokens outside a token's mask may hold anything."""
    args = ([333, 0, 61], [9, 5, 64], 8, 2, 128, 32, dt, 6)
    good, hurt = Paged(S, *args, fill=0.0), Paged(S, *args, fill=bad)
    out = good.call(S)
    assert torch.equal(hurt.call(S), out)
    # new token 2 of sequence 0 holds `bad`: only the tokens that see it show it
    j = 333 + 2
    pg = int(hurt.table[0, j // 32])
    hurt.ck[pg, :, j % 32] = bad
    hurt.cv[pg, :, j % 32] = bad
    got = hurt.call(S)
    for t, m in enumerate(hurt.masks):
        if t < 9 and (m >> 2) & 1:
            assert not torch.isfinite(got[t].float()).any()
        else:
            assert torch.equal(got[t], out[t]), t


@pytest.mark.gpu
def test_attn_tree_infinite_values_reach_the_tokens_that_see_them(S):
    p = Paged(S, [100], [6], 8, 2, 64, 16, "bf16", 9)
    out = p.call(S)
    want = out.clone()
    for j, col, v in ((102, 5, float("inf")), (40, 7, -float("inf"))):
        p.cv[int(p.table[0, j // 16]), 0, j % 16, col] = v
        for t, m in enumerate(p.masks):
            if j < 100 or (m >> (j - 100)) & 1:
                want[t, :4, col] = v
    assert torch.equal(p.call(S), want)


@pytest.mark.gpu
def test_attn_tree_contract_errors_are_recorded(S):
    p = Paged(S, [50, 20], [3, 2], 4, 2, 64, 16, "bf16", 1)
    ws = S.alloc_attn_workspace(S.WS_ATTN_TREE, 5, 2, 4, 2, 64)
    good = p.call(S, workspace=ws)
    # a page outside the cache: recorded
    keep = p.table.clone()
    for bad in (p.cache.n_pages, -1):
        p.table = keep.clone()
        p.table[0, 1] = bad
        out = p.call(S, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE
        assert torch.equal(out[3:], good[3:]) and torch.isfinite(out.float()).all()
    p.table = keep
    # more positions than the table holds, a negative context, tokens past T: the sequence is skipped
    for ctx, cu in (([50, 10 ** 6], None), ([50, -1], None), ([50, 20], [0, 3, 6]), ([50, 20], [0, 3, 2])):
        out = torch.full_like(good, 9.0)
        c = p.cu if cu is None else torch.tensor(cu, dtype=torch.int32)
        S.attn_tree(p.q.cuda(), p.cache, p.table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), c.cuda(),
                    torch.tensor(p.masks, dtype=torch.int64).cuda(), out=out, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
        assert torch.equal(out[:3], good[:3]) and (out[3:] == 9).all()


@pytest.mark.gpu
def test_attn_tree_and_cache_rows_past_32_bit_offsets(S):
    """Pages whose elements lie past 2^32: written by the rotation call, read by the attention."""
    hkv, page, D = 8, 64, 128
    first = 2 ** 32 // (hkv * page * D) + 1
    p = Paged(S, [150], [2], 16, hkv, D, page, "bf16", 3, fill=0.0, first_page=first)
    j = 151
    slot = int(p.table[0, j // page]) * page + j % page
    k, v = p.k[0][j:j + 1].cuda(), p.v[0][j:j + 1].cuda()
    p.ck[slot // page, :, slot % page] = 0
    p.cv[slot // page, :, slot % page] = 0
    S.qk_norm_rope(p.q[:1].cuda(), k, v, None, None, cache=p.cache, slots=torch.tensor([slot], dtype=torch.int32).cuda())
    p.check(p.call(S))


@pytest.mark.gpu
def test_attention_on_another_stream_and_shared_workspace(S):
    """Calls on a side stream, one workspace for every entry point in turn."""
    p = Paged(S, [500, 31], [4, 9], 8, 2, 128, 16, "bf16", 12)
    lens = [90, 200]
    qkv, cu = prompt_inputs(lens, 8, 2, 128, 13)
    dev, cud = qkv.cuda(), cu.cuda()
    ws = torch.zeros(max(S.attn_workspace_size(w, 290, 2, 8, 2, 128) for w in (0, 1, 2)), dtype=torch.uint8, device="cuda")
    ws[256:] = 0xFF  # only the control block has to be zero
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = p.call(S, workspace=ws)
        b = S.attn_prompt(dev[:, :8], dev[:, 8:10], dev[:, 10:], cud, workspace=ws)
        c = p.call(S, workspace=ws)
    side.synchronize()
    p.check(a)
    assert torch.equal(a, c)
    check_attention(b.cpu(), *ref_prompt(qkv, lens, 8, 2, 128), 128, 200, True)


@pytest.mark.gpu
def test_attention_calls_in_a_cuda_graph(S):
    p = Paged(S, [500, 31], [4, 9], 8, 2, 128, 16, "bf16", 12)
    ws = S.alloc_attn_workspace(S.WS_ATTN_TREE, 13, 2, 8, 2, 128)
    q, table, ctx, cu = p.q.cuda().contiguous(), p.table.cuda(), torch.tensor(p.ctx, dtype=torch.int32).cuda(), p.cu.cuda()
    mask, out = torch.tensor(p.masks, dtype=torch.int64).cuda(), torch.zeros(13, 8, 128, dtype=torch.bfloat16).cuda()
    rot = S.rope_table(600, 128)
    pos = torch.arange(13).int().cuda()
    qr, kr = torch.empty_like(q), torch.empty(13, 2, 128, dtype=torch.bfloat16).cuda()

    def step():
        S.qk_norm_rope(q, kr0, None, rot, pos, q_out=qr, k_out=kr, workspace=ws)
        S.attn_tree(q, p.cache, table, ctx, cu, mask, out=out, workspace=ws)
        S.attn_prompt(qr, kr, kr, cu, out=pr, workspace=ws)

    kr0 = torch.randn(13, 2, 128).bfloat16().cuda()
    pr = torch.zeros_like(out)
    step()
    torch.cuda.synchronize()
    first, pfirst = out.clone(), pr.clone()
    out.zero_()
    pr.zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(pr, pfirst)
    p.check(out)


# ---------------------------------------------------------------------------
# refusals (before anything is launched)
# ---------------------------------------------------------------------------

def kv(S, **kw):
    f = dict(dtype=S.BF16, n_kv_heads=2, head_dim=128, page_size=16, n_pages=4, k=16, v=16)
    f.update(kw)
    return C.byref(S.KVCacheStruct(*[f[n] for n, _ in S.KVCacheStruct._fields_]))


def test_rope_refusals(S):
    L = S.lib()

    def call(dtype=S.BF16, q=16, qs=512, k=16, ks=256, v=16, vs=256, T=3, hq=4, hkv=2, D=128, wq=None, wk=None, eps=1e-6,
             table=16, rot=128, mp=10, style=0, pos=16, qo=16, ko=16, cache=None, slots=None, ws=256, wb=256):
        return L.sffn_qk_norm_rope(dtype, q, qs, k, ks, v, vs, T, hq, hkv, D, wq, wk, eps, table, rot, mp, style, pos,
                                   qo, ko, cache, slots, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(dtype=S.INT4_G64) == S.ERR_INVALID_ARG
    assert call(style=2) == S.ERR_INVALID_ARG
    assert call(eps=-1.0) == S.ERR_INVALID_ARG and call(eps=float("nan")) == S.ERR_INVALID_ARG
    assert call(hkv=3) == S.ERR_SHAPE and call(hkv=0) == S.ERR_SHAPE and call(hq=1026) == S.ERR_SHAPE
    assert call(D=96) == S.ERR_SHAPE and call(hq=130, hkv=2, qs=130 * 128) == S.ERR_SHAPE
    assert call(T=-1) == S.ERR_SHAPE and call(T=(1 << 20) + 1) == S.ERR_SHAPE
    assert call(rot=24) == S.ERR_SHAPE and call(rot=144) == S.ERR_SHAPE
    assert call(q=None) == S.ERR_INVALID_ARG and call(qo=None) == S.ERR_INVALID_ARG
    assert call(ko=None) == S.ERR_INVALID_ARG                      # no cache and nowhere to put the keys
    assert call(table=None) == S.ERR_INVALID_ARG and call(pos=None) == S.ERR_INVALID_ARG
    assert call(mp=0) == S.ERR_INVALID_ARG
    assert call(qs=511) == S.ERR_SHAPE and call(qs=516) == S.ERR_ALIGNMENT and call(k=24) == S.ERR_ALIGNMENT
    assert call(qo=8) == S.ERR_ALIGNMENT and call(wq=8) == S.ERR_ALIGNMENT
    assert call(cache=kv(S)) == S.ERR_INVALID_ARG                  # a cache without slots
    assert call(slots=16) == S.ERR_INVALID_ARG
    assert call(cache=kv(S), slots=16, v=None) == S.ERR_INVALID_ARG
    assert call(cache=kv(S, dtype=S.F32), slots=16) == S.ERR_INVALID_ARG
    assert call(cache=kv(S, page_size=24), slots=16) == S.ERR_SHAPE
    assert call(cache=kv(S, n_kv_heads=4), slots=16) == S.ERR_SHAPE
    assert call(cache=kv(S, n_pages=1 << 30), slots=16) == S.ERR_SHAPE
    assert call(ws=None) == S.ERR_WORKSPACE and call(wb=128) == S.ERR_WORKSPACE and call(ws=64) == S.ERR_WORKSPACE


def test_prompt_refusals(S):
    L = S.lib()

    def call(q=16, qs=512, k=16, ks=256, v=16, vs=256, T=3, hq=4, hkv=2, D=128, cu=16, n=1, scale=0.1, out=16, ws=256,
             wb=1 << 30):
        return L.sffn_attn_prompt(q, qs, k, ks, v, vs, T, hq, hkv, D, cu, n, scale, out, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(n=0) == S.ERR_SHAPE and call(n=65537) == S.ERR_SHAPE and call(T=(1 << 20) + 1) == S.ERR_SHAPE
    assert call(D=80) == S.ERR_SHAPE and call(hq=5) == S.ERR_SHAPE
    assert call(scale=0.0) == S.ERR_INVALID_ARG and call(scale=float("nan")) == S.ERR_INVALID_ARG
    assert call(scale=float("inf")) == S.ERR_INVALID_ARG
    for name in ("q", "k", "v", "cu", "out"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: 8}) == S.ERR_ALIGNMENT, name
    assert call(ks=255) == S.ERR_SHAPE and call(vs=260) == S.ERR_ALIGNMENT
    assert call(ws=None) == S.ERR_WORKSPACE and call(wb=16) == S.ERR_WORKSPACE
    assert S.attn_workspace_size(1, 10, 0, 4, 2, 128) == 0 and S.attn_workspace_size(1, 10, 1, 4, 2, 96) == 0
    assert S.attn_workspace_size(3, 10, 1, 4, 2, 128) == 0


def test_tree_refusals(S):
    L = S.lib()

    def call(q=16, qs=512, T=3, hq=4, cache="kv", table=16, width=4, ctx=16, cu=16, n=1, mask=16, scale=0.1, out=16,
             ws=256, wb=1 << 30):
        return L.sffn_attn_tree(q, qs, T, hq, kv(S) if cache == "kv" else cache, table, width, ctx, cu, n, mask, scale,
                                out, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(cache=None) == S.ERR_INVALID_ARG
    assert call(cache=kv(S, dtype=S.INT4_G64)) == S.ERR_INVALID_ARG
    assert call(cache=kv(S, head_dim=32)) == S.ERR_SHAPE and call(cache=kv(S, page_size=4)) == S.ERR_SHAPE
    assert call(cache=kv(S, k=None)) == S.ERR_INVALID_ARG and call(cache=kv(S, v=8)) == S.ERR_ALIGNMENT
    assert call(hq=5) == S.ERR_SHAPE and call(hq=256, qs=256 * 128) == S.ERR_SHAPE
    assert call(T=-1) == S.ERR_SHAPE and call(T=65537) == S.ERR_SHAPE
    assert call(n=0) == S.ERR_SHAPE and call(n=1025) == S.ERR_SHAPE and call(width=0) == S.ERR_SHAPE
    assert call(scale=-1.0) == S.ERR_INVALID_ARG
    for name in ("q", "table", "ctx", "cu", "out"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    assert call(q=8) == S.ERR_ALIGNMENT and call(out=8) == S.ERR_ALIGNMENT and call(mask=12) == S.ERR_ALIGNMENT
    assert call(qs=500) == S.ERR_SHAPE


@pytest.mark.gpu
def test_tree_workspace_refusals_and_binding_checks(S):
    p = Paged(S, [20], [2], 4, 2, 64, 16, "bf16", 1)
    need = S.attn_workspace_size(S.WS_ATTN_TREE, 2, 1, 4, 2, 64)
    assert need > 0
    with pytest.raises(S.SffnError) as e:
        p.call(S, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == S.ERR_WORKSPACE
    q = torch.zeros(3, 64, 4, dtype=torch.bfloat16, device="cuda").transpose(1, 2)  # heads not contiguous
    with pytest.raises(S.SffnError):
        S.attn_prompt(q, q, q, torch.tensor([0, 3], dtype=torch.int32).cuda())
    z = torch.zeros(3, 4, 64, dtype=torch.float32, device="cuda")
    with pytest.raises(S.SffnError) as e:
        S.attn_prompt(z, z, z, torch.tensor([0, 3], dtype=torch.int32).cuda())
    assert e.value.status == S.ERR_UNSUPPORTED
    with pytest.raises(S.SffnError):
        S.attn_prompt(z.bfloat16(), z.bfloat16(), z.bfloat16(), torch.tensor([0, 3]).cuda())  # 64-bit offsets
    with pytest.raises(S.SffnError):
        S.attn_tree(z, p.cache, p.table.cuda(), p.cu[:1].cuda(), p.cu.cuda())


@pytest.mark.gpu
def test_empty_calls_and_the_most_sequences(S):
    """No tokens at all; as many sequences as a call takes, most of them without new tokens."""
    e = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert S.attn_prompt(e, k, k, zero).shape == (0, 4, 64)
    q, kk = S.qk_norm_rope(e, k, None, S.rope_table(4, 64), zero[:0])
    assert q.shape == (0, 4, 64) and kk.shape == (0, 2, 64)
    p = Paged(S, [20], [2], 4, 2, 64, 16, "bf16", 1)
    assert S.attn_tree(e, p.cache, p.table.cuda(), zero[:1], zero).shape == (0, 4, 64)
    n = [0, 0, 1, 0] * 256
    p = Paged(S, [(7 * i) % 90 for i in range(1024)], n, 4, 2, 64, 16, "bf16", 2)
    p.check(p.call(S))
    lens = [0, 3, 1, 0, 20] * 60
    qkv, cu = prompt_inputs(lens, 4, 2, 64, 21)
    dev = qkv.cuda()
    out = S.attn_prompt(dev[:, :4], dev[:, 4:6], dev[:, 6:], cu.cuda())
    check_attention(out.cpu(), *ref_prompt(qkv, lens, 4, 2, 64), 64, 20, True)
