"""Long contexts in the paged cache: attention of sequences that share prefixes (sffn_attn_shared), key bounds of
pages (sffn_page_bounds), the choice of pages by a score against them (sffn_page_select) and attention
over the chosen pages (sffn_attn_pages), against plain 64-bit implementations.

Bounds and choices are exact: whole multiples of a power of two, and equal scores go to the lower page.
Attention is held to the bound derived in tests/test_attention.py: (2 d + n 2^-23 + h) sum w|v| + h |out| with
d = D 2^-23 sum |q||k| scale + 2^-20 and h = 2^-8 for bf16.  Joining the two halves of a shared row adds a
product, a factor and a sum for each half, an n of 8 more at the most."""
from __future__ import annotations

import ctypes as C
import math

import pytest
import torch

from tests.test_attention import Paged, S, check_attention, dtype_of, gen, kv, ref_attention, signed  # noqa: F401

TOP, LEAST = 2.0 ** 100, -100


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# references
# ---------------------------------------------------------------------------

def step_of(most):
    """Least 2^e, e >= -100, with most <= 127 * 2^e."""
    e = LEAST
    while most > 127.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def ref_bounds(page):
    """page [heads, page_size, D] -> [heads, 2, D], double."""
    x = page.double()
    hi = torch.where(x.isnan(), TOP, x).clamp(-TOP, TOP).amax(1)
    lo = torch.where(x.isnan(), -TOP, x).clamp(-TOP, TOP).amin(1)
    out = torch.empty(x.shape[0], 2, x.shape[2], dtype=torch.float64)
    for h in range(x.shape[0]):
        st = step_of(max(hi[h].abs().max().item(), lo[h].abs().max().item()))
        out[h, 0], out[h, 1] = torch.ceil(hi[h] / st) * st, torch.floor(lo[h] / st) * st
    return out


def ref_choice(q, bounds, mine, first, recent, keep):
    """q [G, D] of one key head, bounds [pages 0 .. mine, 2, D]: the chosen pages, ascending."""
    if mine + 1 <= keep:
        return list(range(mine + 1))
    q = torch.where(q.double().isnan(), 0.0, q.double()).clamp(-TOP, TOP)
    c = torch.round(q / step_of(q.abs().max().item()))
    b = bounds.double()
    score = (c.clamp(min=0) @ b[:, 0].T + c.clamp(max=0) @ b[:, 1].T).amax(0).tolist()
    always = [p for p in range(mine + 1) if p < first or p > mine - recent]
    rest = sorted((p for p in range(mine + 1) if p not in always), key=lambda p: (-score[p], p))
    return sorted(always + rest[:keep - len(always)])


# ---------------------------------------------------------------------------
# key bounds
# ---------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("page,hkv,D,dt,n_pages", [
    (8, 1, 64, "bf16", 3), (16, 8, 128, "bf16", 40), (32, 2, 64, "f32", 17), (64, 5, 128, "f32", 9),
    (128, 3, 64, "bf16", 11), (1024, 1, 128, "bf16", 3), (4096, 2, 64, "f32", 2),
])
def test_page_bounds(S, page, hkv, D, dt, n_pages):  # noqa: F811
    g = gen(page + D)
    k = torch.randn(n_pages, hkv, page, D, generator=g) * 2.0 ** torch.randint(-20, 20, (n_pages, hkv, 1, 1), generator=g)
    k[0, 0] = 0                     # nothing but zeros
    k[1, 0, :, 3] = -1e-38          # far below the step, on either side of zero
    k[1, 0, :, 4] = 1e-38
    k[-1, -1] = 127.0               # at the edge of a step, and just past it
    if n_pages > 4:
        k[2, 0] = 127.5
        k[3, 0] = k[3, 0].abs() * 1e-36
        k[4, 0, page // 2, 1] = float("nan")
        k[4, 0, 0, 2] = float("inf")
        k[4, 0, 0, 5] = -float("inf")
        k[4, 0, 0, 6] = 3e38
    k = k.to(dtype_of(dt)).cuda()
    cache = S.KVCache(k, torch.zeros_like(k))
    listed = torch.randperm(n_pages, generator=g).tolist()
    left = listed.pop() if n_pages > 4 else None
    pages = [-1] + listed + [-1, listed[0]]
    bounds = torch.full((n_pages, hkv, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = S.alloc_attn_workspace(S.WS_PAGE_BOUNDS, len(pages), 1, hkv, hkv, D)
    assert S.page_bounds(cache, i32(pages), bounds, workspace=ws) is bounds
    assert S.read_device_error(ws) == 0
    got, kc = bounds.double().cpu(), k.cpu()
    for p in range(n_pages):
        want = torch.full((hkv, 2, D), 9.0, dtype=torch.float64) if p == left else ref_bounds(kc[p])
        assert torch.equal(got[p], want), p
    # pages outside the cache: recorded, nothing else written
    S.page_bounds(cache, i32([n_pages, listed[0], -2]), bounds, workspace=ws)
    assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
    assert torch.equal(bounds.double().cpu(), got)
    assert torch.equal(S.page_bounds(cache, i32([])), torch.zeros_like(bounds))


# ---------------------------------------------------------------------------
# the choice
# ---------------------------------------------------------------------------

class Tokens:
    """Tokens of several sequences in a paged cache: sequence s has `lens[s]` positions, and tokens at `at[s]`."""

    def __init__(self, S, lens, at, hq, hkv, D, page, dt, seed, **kw):  # noqa: F811
        self.p = Paged(S, lens, [0] * len(lens), hq, hkv, D, page, dt, seed, **kw)
        self.hq, self.hkv, self.D, self.page, self.dt = hq, hkv, D, page, dt
        self.seqs = [s for s, row in enumerate(at) for _ in row]
        self.pos = [x for row in at for x in row]
        self.q = (torch.randn(len(self.pos), hq + 1, D, generator=gen(seed + 1)) * 1.5).to(dtype_of(dt))[:, :hq]
        self.cache, self.table = self.p.cache, self.p.table
        whole = sorted({int(self.table[s, i]) for s, n in enumerate(lens) for i in range(n // page)})
        self.bounds = S.page_bounds(self.cache, i32(whole))

    def queries(self):
        q = torch.empty(len(self.pos), self.hq + 2, self.D, dtype=self.q.dtype, device="cuda")[:, :self.hq]
        return q.copy_(self.q)

    def select(self, S, keep, first=1, recent=1, **kw):  # noqa: F811
        return S.page_select(self.queries(), self.cache, self.bounds, self.table.cuda(), i32(self.seqs), i32(self.pos),
                             keep, first, recent, **kw)

    def check_choice(self, sel, n_sel, keep, first, recent):
        sel, n_sel, b, G = sel.cpu().tolist(), n_sel.cpu().tolist(), self.bounds.cpu(), self.hq // self.hkv
        for t, (s, p) in enumerate(zip(self.seqs, self.pos)):
            mine = p // self.page
            assert n_sel[t] == min(mine + 1, keep)
            mine_b = b[self.table[s, :mine + 1].long()]
            for h in range(self.hkv):
                want = ref_choice(self.q[t, h * G:(h + 1) * G], mine_b[:, h], mine, first, recent, keep)
                assert sel[t][h] == want + [-1] * (keep - len(want)), (t, h)

    def attend(self, S, sel, n_sel, **kw):  # noqa: F811
        return S.attn_pages(self.queries(), self.cache, self.table.cuda(), i32(self.seqs), i32(self.pos), sel, n_sel, **kw)

    def check_attention(self, got, sel, n_sel):
        got, sel, n_sel, G = got.cpu(), sel.cpu().tolist(), n_sel.cpu().tolist(), self.hq // self.hkv
        for t, (s, p) in enumerate(zip(self.seqs, self.pos)):
            for h in range(self.hkv):
                at = [j for i in sel[t][h][:n_sel[t]] for j in range(i * self.page, (i + 1) * self.page) if j <= p]
                k, v = self.p.k[s][at, h], self.p.v[s][at, h]
                q = self.q[t, h * G:(h + 1) * G]
                ref = ref_attention(q, k, v, torch.ones(G, len(at), dtype=torch.bool), self.D ** -0.5)
                check_attention(got[t, h * G:(h + 1) * G], *ref, self.D, len(at) + 8, self.dt == "bf16")


SELECT = [
    # positions, tokens of each sequence, hq, hkv, D, page, dtype, first, recent, keep
    ([1], [[0]], 1, 1, 64, 8, "bf16", 0, 1, 1),
    ([900], [[899]], 64, 8, 128, 16, "bf16", 1, 2, 9),
    ([900, 40, 333], [[899, 500, 17], [39], [332]], 16, 2, 64, 32, "f32", 1, 1, 5),
    ([2000, 130, 8, 777], [[1999], [129], [0], [640]], 28, 4, 128, 8, "bf16", 2, 3, 33),
    ([600, 600], [list(range(560, 600)), list(range(0, 600, 37))], 5, 1, 128, 16, "bf16", 0, 1, 7),
    ([700], [list(range(100, 700, 11))], 20, 20, 64, 8, "bf16", 1, 4, 24),
    ([400], [[399, 398]], 64, 1, 64, 8, "bf16", 1, 1, 12),
    ([500], [[499, 3]], 48, 4, 128, 8, "f32", 3, 2, 5),                # no room beside the forced ones
    ([16400], [[16399, 9000]], 4, 2, 64, 8, "bf16", 1, 2, 100),        # 2050 pages
    ([40000], [[39999]], 2, 1, 64, 8, "bf16", 1, 1, 1500),             # 5000 pages
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,at,hq,hkv,D,page,dt,first,recent,keep", SELECT)
def test_page_select(S, lens, at, hq, hkv, D, page, dt, first, recent, keep):  # noqa: F811
    c = Tokens(S, lens, at, hq, hkv, D, page, dt, sum(lens) + hq, fill=0.0)
    T = len(c.pos)
    ws = S.alloc_page_select_workspace(T, hkv, c.table.shape[1])
    sel, n_sel = c.select(S, keep, first, recent, workspace=ws)
    assert S.read_device_error(ws) == 0
    c.check_choice(sel, n_sel, keep, first, recent)
    again = c.select(S, keep, first, recent, workspace=ws)
    assert torch.equal(again[0], sel) and torch.equal(again[1], n_sel)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_page_select_equal_scores_go_to_the_lower_page(S, dt):  # noqa: F811
    """Pages with the same keys (the same page of the cache, listed often), zero queries, and queries of extreme values."""
    c = Tokens(S, [800], [[799] * 6], 6, 2, 64, 16, dt, 5, fill=0.0)
    c.table[0, 3:40:2] = c.table[0, 3]
    c.table[0, 41:48] = c.table[0, 2]
    c.q[1] = 0
    c.q[2] *= 1e30
    c.q[3] *= 1e-36
    c.q[4, 0, 5] = float("inf")
    c.q[4, 1, 6] = float("nan")
    c.q[5] = float("nan")
    for keep, first, recent in ((2, 0, 1), (7, 1, 2), (20, 1, 1), (49, 3, 4)):
        c.check_choice(*c.select(S, keep, first, recent), keep, first, recent)
    sel, _ = c.select(S, 10, 0, 1)
    assert sel[1].tolist() == [list(range(9)) + [49]] * 2  # every score is zero


@pytest.mark.gpu
def test_page_select_extreme_bounds(S):  # noqa: F811
    """Keys that are infinite, NaN or huge put their page first; they disturb no other's score."""
    c = Tokens(S, [640], [[639, 630]], 8, 2, 128, 16, "bf16", 8, fill=0.0)
    c.p.ck[int(c.table[0, 7]), 0, 3, 9] = float("nan")
    c.p.ck[int(c.table[0, 9]), 1, 0, 0] = float("inf")
    c.p.ck[int(c.table[0, 20]), 1, 2, 1] = -3e38
    c.p.ck[int(c.table[0, 21]), 0] = 1e-38
    c.bounds = S.page_bounds(c.cache, c.table[0, :40].cuda())
    assert torch.isfinite(c.bounds.float()).all()
    for keep in (2, 5, 30):
        c.check_choice(*c.select(S, keep), keep, 1, 1)


@pytest.mark.gpu
def test_page_select_padding_and_contract_errors(S):  # noqa: F811
    c = Tokens(S, [300, 100], [[299, 10, 150], [99, 50]], 8, 2, 64, 16, "bf16", 3, fill=0.0)
    ws = S.alloc_page_select_workspace(5, 2, c.table.shape[1])
    good = c.select(S, 4, workspace=ws)
    pos, seqs = list(c.pos), list(c.seqs)

    def same_but(t, sel, n_sel):
        assert n_sel[t] == 0 and (sel[t] == -1).all()
        rest = [i for i in range(5) if i != t]
        assert torch.equal(sel[rest], good[0][rest]) and torch.equal(n_sel[rest], good[1][rest])

    c.pos[1] = -1
    same_but(1, *c.select(S, 4, workspace=ws))
    assert S.read_device_error(ws) == 0
    for what, bad in (("pos", c.table.shape[1] * 16), ("pos", 2 ** 31 - 1), ("seqs", 2), ("seqs", -1)):
        c.pos, c.seqs = list(pos), list(seqs)
        getattr(c, what)[2] = bad
        same_but(2, *c.select(S, 4, workspace=ws))
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
    c.pos, c.seqs = pos, seqs
    for bad in (c.cache.n_pages, -1):  # such a page's bounds count as zeros
        table = c.table.clone()
        c.table[0, 5] = bad
        sel, n_sel = c.select(S, 4, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
        assert torch.equal(sel[3:], good[0][3:]) and torch.equal(n_sel, good[1])
        b = c.bounds
        c.bounds = torch.cat([b, torch.zeros_like(b[:1])])
        c.table[0, 5] = b.shape[0]
        c.check_choice(sel, n_sel, 4, 1, 1)
        c.bounds, c.table = b, table


# ---------------------------------------------------------------------------
# attention over chosen pages
# ---------------------------------------------------------------------------

PAGES = [
    # positions, tokens of each sequence, hq, hkv, D, page, dtype, keep
    ([1], [[0]], 1, 1, 64, 8, "bf16", 1),
    ([900], [[899]], 64, 8, 128, 16, "bf16", 9),
    ([900, 40, 333], [[899, 500, 17], [39], [332]], 16, 2, 64, 32, "f32", 5),
    ([2000, 130, 8, 777], [[1999], [129], [0], [640]], 28, 4, 128, 8, "bf16", 100),
    ([600, 600], [list(range(560, 600)), list(range(0, 600, 37))], 5, 1, 128, 16, "bf16", 7),
    ([700], [list(range(100, 700, 11))], 20, 20, 64, 8, "bf16", 24),
    ([400, 129], [[399, 398], [128, 127]], 64, 1, 64, 64, "bf16", 3),
    ([500], [[499, 3]], 48, 4, 128, 128, "f32", 2),
    ([1500, 700], [[1499], [512]], 8, 2, 128, 512, "bf16", 3),
    ([300] * 40, [[299 - i] for i in range(40)], 4, 2, 64, 16, "bf16", 6),
    ([1000], [list(range(700, 1000))], 8, 1, 128, 32, "bf16", 8),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,at,hq,hkv,D,page,dt,keep", PAGES)
def test_attn_pages(S, lens, at, hq, hkv, D, page, dt, keep):  # noqa: F811
    """Unused places of the cache hold NaN; the pages are the score's."""
    c = Tokens(S, lens, at, hq, hkv, D, page, dt, sum(lens) + hq)
    T = len(c.pos)
    first = 1 if keep > 1 else 0
    sel, n_sel = c.select(S, keep, first)
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, T, len(lens), hq, hkv, D)
    out = c.attend(S, sel, n_sel, workspace=ws)
    assert S.read_device_error(ws) == 0
    c.check_attention(out, sel, n_sel)
    assert torch.equal(out, c.attend(S, sel, n_sel, workspace=ws))  # equal calls, equal bits


@pytest.mark.gpu
@pytest.mark.parametrize("lens,at,hq,hkv,D,page,keep", [
    ([900, 77], [[899], [76]], 3, 3, 128, 8, 40),
    ([900, 77], [[899, 3], [76, 75, 74]], 8, 4, 64, 16, 12),
    ([1300], [[1299, 1298]], 20, 5, 128, 32, 21),
    ([640, 64], [[500, 639], [63]], 64, 1, 64, 64, 3),
    ([1700], [list(range(1500, 1620))], 28, 4, 128, 16, 30),          # more units than warps
    ([3000] * 30, [[2999 - i] for i in range(30)], 32, 32, 64, 128, 7),
    ([4096], [[4095]], 2, 1, 128, 1024, 2),
])
def test_attn_pages_in_fp32(S, lens, at, hq, hkv, D, page, keep):  # noqa: F811
    test_attn_pages(S, lens, at, hq, hkv, D, page, "f32", keep)


MANY = [
    # positions, tokens of each sequence (many of one: they share what they read), hq, hkv, D, page, keep
    ([900, 700], [list(range(500, 640)), list(range(70))], 4, 4, 64, 8, 20),
    ([5000], [list(range(4000, 4100))], 7, 1, 128, 128, 6),
    ([6000], [list(range(5000, 5130))], 8, 2, 64, 512, 3),
    ([900], [list(range(790, 900))], 40, 8, 128, 64, 5),
    ([800, 300, 100], [list(range(700, 790)), [299], list(range(40, 100))], 16, 2, 64, 16, 11),
    ([300, 77], [list(range(300)), list(range(77))], 28, 4, 128, 32, 4),
    ([260], [[3 * i for i in range(80)]], 12, 12, 128, 16, 7),
    ([40], [list(range(40))], 128, 2, 64, 8, 2),
    ([50], [list(range(50))], 128, 2, 64, 8, 2),
]


def widen(sel, keep):
    """The lists in rows of `keep` entries (many, that may hold much: the tokens are taken together)."""
    return torch.nn.functional.pad(sel, (0, keep - sel.shape[2]), value=-1)


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 4096])
@pytest.mark.parametrize("lens,at,hq,hkv,D,page,keep", MANY)
def test_attn_pages_many_tokens_of_a_sequence(S, lens, at, hq, hkv, D, page, keep, room):  # noqa: F811
    c = Tokens(S, lens, at, hq, hkv, D, page, "bf16", sum(lens) + hq)
    sel, n_sel = c.select(S, keep, 1 if keep > 1 else 0)
    sel = widen(sel, max(room, keep))
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, len(c.pos), len(lens), hq, hkv, D)
    out = c.attend(S, sel, n_sel, workspace=ws)
    assert S.read_device_error(ws) == 0
    c.check_attention(out, sel, n_sel)
    assert torch.equal(out, c.attend(S, sel, n_sel, workspace=ws))  # equal calls, equal bits


@pytest.mark.gpu
@pytest.mark.parametrize("room", [6, 4096])
@pytest.mark.parametrize("hq,D", [(8, 128), (2, 64)])
def test_attn_pages_many_tokens_padding_and_contract_errors(S, hq, D, room):  # noqa: F811
    """Padding, tokens without pages, tokens and list entries out of range among many tokens of two sequences."""
    c = Tokens(S, [400, 200], [list(range(250, 380)), list(range(100, 190))], hq, 2, D, 16, "bf16", 9)
    sel, n_sel = c.select(S, 6)
    sel = widen(sel, room)
    T, pos, seqs, n = len(c.pos), list(c.pos), list(c.seqs), n_sel.tolist()
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, T, 2, hq, 2, D)

    def run(error, changed, n_new=n, lists=sel, zero=()):
        out = torch.full((T, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        c.attend(S, lists, i32(n_new), out=out, workspace=ws)
        assert S.read_device_error(ws) == error and S.read_device_error(ws) == 0
        assert torch.isfinite(out.float()).all()
        rows = [t for t in range(T) if t not in changed]
        d = Tokens.__new__(Tokens)
        d.__dict__.update(c.__dict__)
        d.pos, d.seqs, d.q = [pos[t] for t in rows], [seqs[t] for t in rows], c.q[rows]
        d.check_attention(out[rows], sel[rows], n_sel[rows])
        return out

    run(0, [])
    c.pos = [-1 if t in (0, 7, 60, 61, 140, T - 1) else p for t, p in enumerate(pos)]
    out = run(0, [0, 7, 60, 61, 140, T - 1])
    assert (out[[0, 7, 60, 61, 140, T - 1]] == 9).all()
    c.pos = list(pos)
    out = run(0, [3, 4, 131, T - 1], [0 if t in (3, 4, 131, T - 1) else x for t, x in enumerate(n)])
    assert not out[[3, 4, 131, T - 1]].any()
    for what, bad in (("pos", 10 ** 7), ("seqs", 2), ("seqs", -1)):
        c.pos, c.seqs = list(pos), list(seqs)
        getattr(c, what)[50] = bad
        assert (run(S.ERR_DEVICE, [50])[50] == 9).all()
    c.pos, c.seqs = pos, seqs
    assert (run(S.ERR_DEVICE, [33], [room + 1 if t == 33 else x for t, x in enumerate(n)])[33] == 9).all()
    for bad in (25, -1, 1 << 20, -(1 << 31)):  # list entries past the token's own page or outside the table
        hurt = sel.clone()
        hurt[20, 1, 0] = bad
        run(S.ERR_DEVICE, [20], lists=hurt)
    table = c.table.clone()
    for bad in (c.cache.n_pages, -1):  # a page of the second sequence outside the cache: its tokens' rows
        c.table[1, 5] = bad
        run(S.ERR_DEVICE, list(range(130, T)))
    c.table = table


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("D,page,room", [(128, 32, 4096), (64, 16, 4096), (64, 16, 3)])
def test_attn_pages_many_tokens_unseen_places_have_no_influence(S, bad, D, page, room):  # noqa: F811
    args = ([400], [list(range(200, 330))], 8, 2, D, page, "bf16", 6)
    c = Tokens(S, *args, fill=0.0)
    sel, n_sel = c.select(S, 3)
    sel = widen(sel, room)
    out = c.attend(S, sel, n_sel)
    c.check_attention(out, sel, n_sel)
    d = Tokens(S, *args, fill=bad)
    assert torch.equal(d.attend(S, sel, n_sel), out)
    # one position, as key and value or as value alone: only the tokens that see it show it
    for j, key in ((101, True), (250, True), (77, False), (310, False)):
        d = Tokens(S, *args, fill=0.0)
        pg = int(d.table[0, j // page])
        d.p.cv[pg, :, j % page] = bad
        if key:
            d.p.ck[pg, :, j % page] = bad
        got = d.attend(S, sel, n_sel)
        seen = 0
        for t, p in enumerate(d.pos):
            for h in range(2):
                rows = slice(h * 4, h * 4 + 4)
                if j <= p and j // page in sel[t, h, :n_sel[t]].tolist():
                    seen += 1
                    assert not torch.isfinite(got[t, rows].float()).any()
                else:
                    assert torch.equal(got[t, rows], out[t, rows]), (j, t, h)
        assert 0 < seen < 2 * len(d.pos)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_pages_lists_of_the_caller(S, dt):  # noqa: F811
    """Lists that leave the token's own page out, differ between heads, or are empty; padding keeps its row."""
    c = Tokens(S, [400, 90], [[399, 210, 33, 0], [89, 15]], 6, 2, 64, 32, dt, 9)
    lists = [[[0, 3, 7], [1, 2, 12]], [[5, 6], [0, 1]], [[0, 0], [0, 0]], [[0, 0], [0, 0]], [[2, 2], [0, 0]], [[0, 0], [0, 0]]]
    n = [3, 2, 0, 1, 1, 1]
    sel = torch.full((6, 2, 4), -1, dtype=torch.int32)
    for t, rows in enumerate(lists):
        for h, row in enumerate(rows):
            sel[t, h, :n[t]] = torch.tensor(row[:n[t]], dtype=torch.int32)
    sel, n_sel = sel.cuda(), i32(n)
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, 6, 2, 6, 2, 64)
    out = torch.full((6, 6, 64), 9.0, dtype=dtype_of(dt), device="cuda")
    c.attend(S, sel, n_sel, out=out, workspace=ws)
    assert S.read_device_error(ws) == 0
    assert not out[2].any()
    c.check_attention(out, sel, n_sel)
    good = out.clone()
    pos, seqs = list(c.pos), list(c.seqs)
    out.fill_(9.0)
    c.pos[1] = -7
    c.attend(S, sel, n_sel, out=out, workspace=ws)
    assert S.read_device_error(ws) == 0
    assert (out[1] == 9).all() and torch.equal(out[[0, 2, 3, 4, 5]], good[[0, 2, 3, 4, 5]])
    # tokens out of range: skipped and recorded
    for what, bad in (("pos", c.table.shape[1] * 32), ("seqs", 2), ("seqs", -1), ("n", 5), ("n", -1)):
        c.pos, c.seqs, m = list(pos), list(seqs), list(n)
        (m if what == "n" else getattr(c, what))[4] = bad
        out.fill_(9.0)
        c.attend(S, sel, i32(m), out=out, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
        assert (out[4] == 9).all() and torch.equal(out[[0, 1, 2, 3, 5]], good[[0, 1, 2, 3, 5]])
    c.pos, c.seqs = pos, seqs
    # entries past the token's own page or outside the table, pages outside the cache: zeros, recorded
    for bad in (13, -1, 1 << 20, -(1 << 31)):
        hurt = sel.clone()
        hurt[0, 1, 0] = bad
        got = c.attend(S, hurt, n_sel, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
        assert torch.equal(got[1:], good[1:]) and torch.equal(got[0, :3], good[0, :3])
        assert torch.isfinite(got.float()).all()
    table = c.table.clone()
    c.table[1, 2] = c.cache.n_pages
    got = c.attend(S, sel, n_sel, workspace=ws)
    assert S.read_device_error(ws) == S.ERR_DEVICE
    assert torch.equal(got[:4], good[:4]) and torch.isfinite(got.float()).all()
    c.table = table


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_pages_unseen_places_have_no_influence(S, dt, bad):  # noqa: F811
    """Positions behind a token's own in its page and pages that are not chosen may hold anything; a chosen
    position that holds it reaches the tokens that see it."""
    args = ([333, 61], [[332, 200, 120, 100, 99], [60, 3]], 8, 2, 128, 32, dt, 6)
    c = Tokens(S, *args, fill=0.0)
    sel, n_sel = c.select(S, 3)
    out = c.attend(S, sel, n_sel)
    c.check_attention(out, sel, n_sel)
    d = Tokens(S, *args, fill=bad)
    assert torch.equal(d.attend(S, sel, n_sel), out)
    j = 101  # of sequence 0: token 4 (position 99) has it in its page, token 3 (100) too, token 2 (120) sees it
    pg = int(d.table[0, j // 32])
    d.p.ck[pg, :, j % 32] = bad
    d.p.cv[pg, :, j % 32] = bad
    got = d.attend(S, sel, n_sel)
    for t in range(7):
        for h in range(2):
            sees = t < 3 and j // 32 in sel[t, h, :n_sel[t]].tolist()
            rows = slice(h * 4, h * 4 + 4)
            if sees:
                assert not torch.isfinite(got[t, rows].float()).any()
            else:
                assert torch.equal(got[t, rows], out[t, rows]), (t, h)


@pytest.mark.gpu
def test_attn_pages_with_every_page_is_plain_decode(S):  # noqa: F811
    """Enough room for all pages: the choice is every page, and the result the decode step's."""
    p = Paged(S, [700, 0, 33, 128], [1, 1, 1, 1], 28, 4, 128, 16, "bf16", 4)
    bounds = torch.zeros(p.cache.n_pages, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    q, table = p.q.cuda().contiguous(), p.table.cuda()
    sel, n_sel = S.page_select(q, p.cache, bounds, table, i32([0, 1, 2, 3]), i32(p.ctx), 44)
    assert n_sel.tolist() == [44, 1, 3, 9]
    out = S.attn_pages(q, p.cache, table, i32([0, 1, 2, 3]), i32(p.ctx), sel, n_sel)
    p.check(out)


# ---------------------------------------------------------------------------
# shared prefixes
# ---------------------------------------------------------------------------

def share(p, groups, prefix, page):
    """The whole pages of each group's prefix become those of its first sequence."""
    s = 0
    for m, n in zip(groups, prefix):
        w = n // page
        for r in range(s + 1, s + m):
            mine = p.table[r, :w].long()
            p.ck[mine] = float("nan")  # nobody's any more
            p.cv[mine] = float("nan")
            p.table[r, :w] = p.table[s, :w]
            p.k[r][:w * page] = p.k[s][:w * page]
            p.v[r][:w * page] = p.v[s][:w * page]
        s += m


def offsets(sizes):
    return i32([0] + torch.tensor(sizes).cumsum(0).tolist())


def call_shared(S, p, groups, prefix, masks="own", **kw):  # noqa: F811
    masks = p.masks if masks == "own" else masks
    dm = None if masks is None else torch.tensor([signed(m) for m in masks], dtype=torch.int64).cuda()
    q = torch.empty(p.q.shape[0], p.hq + 2, p.D, dtype=p.q.dtype, device="cuda")[:, :p.hq]
    q.copy_(p.q)
    return S.attn_shared(q, p.cache, p.table.cuda(), i32(p.ctx), p.cu.cuda(), offsets(groups), i32(prefix), dm, **kw)


SHARED = [
    # groups, prefix, positions behind the prefix, new tokens, hq, hkv, D, page, dtype
    ([1], [0], [0], [1], 1, 1, 64, 8, "bf16"),
    ([4], [256], [0, 7, 40, 13], [1, 1, 1, 1], 32, 32, 128, 16, "bf16"),
    ([3, 2], [100, 64], [10, 200, 0, 77, 31], [1, 5, 2, 1, 3], 16, 2, 64, 32, "f32"),
    ([5, 0, 1, 2], [700, 40, 0, 129], [0, 33, 120, 64, 1, 301, 8, 250], [8, 1, 25, 3, 8, 7, 64, 9], 28, 4, 128, 128, "bf16"),
    ([40], [333], [i % 19 for i in range(40)], [1] * 40, 64, 8, 128, 16, "bf16"),
    ([30, 1, 20], [530, 77, 128], [(7 * i) % 41 for i in range(51)], [1 + i % 3 for i in range(51)], 8, 1, 64, 64, "bf16"),
    ([2], [1500], [3, 0], [64, 64], 20, 20, 64, 8, "bf16"),
    ([2, 2], [0, 0], [50, 9, 70, 1], [2, 1, 0, 3], 4, 2, 128, 16, "bf16"),   # nothing in common
    ([6], [640], [0, 0, 0, 1, 2, 3], [0, 1, 2, 0, 3, 1], 64, 1, 64, 16, "bf16"),
    ([9], [90], [5] * 9, [7] * 9, 12, 4, 128, 8, "f32"),
    ([1] * 20, [64] * 20, [i for i in range(20)], [1] * 20, 8, 2, 64, 16, "bf16"),  # as many groups as sequences
    ([3], [4000], [0, 1, 100], [33, 40, 60], 5, 1, 128, 256, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("groups,prefix,own,n,hq,hkv,D,page,dt", SHARED)
def test_attn_shared(S, groups, prefix, own, n, hq, hkv, D, page, dt):  # noqa: F811
    of = [x for m, x in zip(groups, prefix) for _ in range(m)]
    p = Paged(S, [a + b for a, b in zip(of, own)], n, hq, hkv, D, page, dt, sum(own) + hq)
    share(p, groups, prefix, page)
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, sum(n), len(n), hq, hkv, D)
    out = call_shared(S, p, groups, prefix, workspace=ws)
    assert S.read_device_error(ws) == 0
    p.check(out)
    assert torch.equal(out, call_shared(S, p, groups, prefix, workspace=ws))  # equal calls, equal bits
    p.check(call_shared(S, p, groups, prefix, masks=None, workspace=ws), masks=None)  # a chain


@pytest.mark.gpu
@pytest.mark.parametrize("groups,prefix,own,n,hq,hkv,D,page", [
    ([3], [600], [1, 70, 200], [1, 1, 1], 3, 3, 64, 8),
    ([4, 4], [300, 129], [i * 31 for i in range(8)], [1] * 8, 8, 4, 128, 16),
    ([5], [77], [0, 1, 2, 130, 64], [2, 1, 1, 2, 1], 20, 5, 128, 32),
    ([7, 2], [900, 0], [11 * i for i in range(9)], [1] * 9, 14, 2, 64, 64),
    ([40], [1000], [3 * i for i in range(40)], [1 + i % 2 for i in range(40)], 10, 2, 128, 16),  # a group of many rows
    ([90, 1], [520, 8], [i % 70 for i in range(91)], [1] * 91, 4, 4, 64, 8),                     # and of single ones
    ([33], [2000], [50] * 33, [2] * 33, 8, 2, 64, 128),
])
def test_attn_shared_few_rows_in_fp32(S, groups, prefix, own, n, hq, hkv, D, page):  # noqa: F811
    of = [x for m, x in zip(groups, prefix) for _ in range(m)]
    args = ([a + b for a, b in zip(of, own)], n, hq, hkv, D, page, "f32", sum(own) + hq)
    p, hurt = Paged(S, *args), Paged(S, *args, fill=float("inf"))
    for x in (p, hurt):
        share(x, groups, prefix, page)
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, sum(n), len(n), hq, hkv, D)
    out = call_shared(S, p, groups, prefix, workspace=ws)
    assert S.read_device_error(ws) == 0
    p.check(out)
    assert torch.equal(out, call_shared(S, hurt, groups, prefix, workspace=ws))
    masks = [0 if t % 3 == 0 else m for t, m in enumerate(p.masks)]  # some see the prefix alone, or nothing
    p.check(call_shared(S, p, groups, prefix, masks, workspace=ws), masks)
    assert S.read_device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attn_shared_rows_that_see_little_or_nothing(S, dt):  # noqa: F811
    """A token whose mask is empty sees the prefix alone; without a prefix it is zero."""
    p = Paged(S, [0, 0, 64, 64], [4, 1, 3, 2], 6, 2, 64, 16, dt, 4)
    share(p, [2, 2], [0, 64], 16)
    masks = [0, 0b0001, 0b1010, (1 << 63) | 0b1000, 0b10, 0, 0b111, 0b100, 0, 0b10]
    out = call_shared(S, p, [2, 2], [0, 64], masks)
    p.check(out, masks)
    assert not out[0].any() and not out[4].any() and out[5].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attn_shared_unseen_places_have_no_influence(S, dt, bad):  # noqa: F811
    groups, prefix = [3, 1], [200, 0]
    args = ([333, 200, 261, 61], [9, 5, 33, 64], 8, 2, 128, 32, dt, 6)
    good, hurt = Paged(S, *args, fill=0.0), Paged(S, *args, fill=bad)
    share(good, groups, prefix, 32)
    share(hurt, groups, prefix, 32)
    out = call_shared(S, good, groups, prefix)
    assert torch.equal(call_shared(S, hurt, groups, prefix), out)
    j = 333 + 2  # a new token of sequence 0: only the tokens that see it show it
    pg = int(hurt.table[0, j // 32])
    hurt.ck[pg, :, j % 32] = bad
    hurt.cv[pg, :, j % 32] = bad
    got = call_shared(S, hurt, groups, prefix)
    for t, m in enumerate(hurt.masks):
        if t < 9 and (m >> 2) & 1:
            assert not torch.isfinite(got[t].float()).any()
        else:
            assert torch.equal(got[t], out[t]), t
    j = 40      # a prefix position: every token of its group, and no other
    pg = int(good.table[0, j // 32])
    good.cv[pg, 1, j % 32, 7] = bad
    got = call_shared(S, good, groups, prefix)
    want = out.clone()
    want[:47, 4:, 7] = bad
    assert torch.equal(got.nan_to_num(nan=5e4), want.nan_to_num(nan=5e4))


@pytest.mark.gpu
def test_attn_shared_contract_errors_are_recorded(S):  # noqa: F811
    p = Paged(S, [70, 64, 20], [3, 2, 2], 4, 2, 64, 16, "bf16", 1)
    groups, prefix = [2, 1], [64, 0]
    share(p, groups, prefix, 16)
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, 7, 3, 4, 2, 64)
    good = call_shared(S, p, groups, prefix, workspace=ws)
    q, table, mask = p.q.cuda(), p.table.cuda(), torch.tensor(p.masks, dtype=torch.int64).cuda()

    def check(skipped, ctx=(70, 64, 20), cu=(0, 3, 5, 7), gs=(0, 2, 3), pl=(64, 0), tab=table):
        out = torch.full_like(good, 9.0)
        S.attn_shared(q, p.cache, tab, i32(ctx), i32(cu), i32(gs), i32(pl), mask, out=out, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
        rows = [r for r in range(7) if r not in skipped]
        assert torch.equal(out[rows], good[rows])
        assert (out[skipped] == 9).all()

    check([5, 6], ctx=(70, 64, -1))
    check([5, 6], ctx=(70, 64, 10 ** 6))
    check([5, 6], cu=(0, 3, 5, 8))
    check([5, 6], pl=(64, 32))                     # more whole prefix pages than positions
    check([5, 6], pl=(64, -1))
    check([5, 6], pl=(64, 1 << 30))
    check([5, 6], gs=(0, 2, 2))                    # sequence 2 is in no group
    check([3, 4], ctx=(70, 63, 20))                # shorter than its group's prefix
    check([0, 1, 2, 3, 4], pl=(-5, 0))
    check([0, 1, 2, 3, 4], pl=(10 ** 6, 0))
    # a page outside the cache reads as zeros
    for row, col in ((0, 1), (1, 4), (2, 1)):
        tab = table.clone()
        tab[row, col] = p.cache.n_pages
        out = S.attn_shared(q, p.cache, tab, i32(p.ctx), p.cu.cuda(), i32([0, 2, 3]), i32(prefix), mask, workspace=ws)
        assert S.read_device_error(ws) == S.ERR_DEVICE
        assert torch.isfinite(out.float()).all()
        same = {0: [5, 6], 1: [0, 1, 2, 5, 6], 2: [0, 1, 2, 3, 4]}[row]
        assert torch.equal(out[same], good[same])
    # rows behind the last sequence are left alone
    out = torch.full((9, 4, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    q9 = torch.cat([q, q[:2]])
    S.attn_shared(q9, p.cache, table, i32(p.ctx), p.cu.cuda(), i32([0, 2, 3]), i32(prefix),
                  torch.cat([mask, mask[:2]]), out=out)
    p.check(out[:7])
    assert (out[7:] == 9).all()


# ---------------------------------------------------------------------------
# together; streams, graphs, large caches
# ---------------------------------------------------------------------------

@pytest.mark.gpu
def test_calls_together_in_a_cuda_graph_and_on_another_stream(S):  # noqa: F811
    """A decode loop's step: the new rows go to the cache, filled pages get their bounds, the tokens choose pages and
    attend; captured once, replayed while the sequences grow.  One workspace serves all the calls."""
    hq, hkv, D, page, n_seq = 8, 2, 128, 16, 3
    start = [95, 240, 31]
    p = Paged(S, [n + 40 for n in start], [0] * n_seq, hq, hkv, D, page, "bf16", 12, fill=0.0)
    keys, values = p.ck.clone(), p.cv.clone()
    table = p.table.cuda()
    width = table.shape[1]
    seqs, pos, slots, full = i32([0, 1, 2]), i32(start), i32([0, 0, 0]), i32([-1] * 3)
    q, k, v = (torch.zeros(n_seq, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    bounds = S.page_bounds(p.cache, i32([int(p.table[s, i]) for s, n in enumerate(start) for i in range(n // page)]))
    size = max([S.attn_workspace_size(w, n_seq, n_seq, hq, hkv, D) for w in (0, 2, 4, 5, 6)])
    size = max(size, S.lib().sffn_page_select_workspace_size(n_seq, hkv, width))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    ws[256:] = 0xFF  # only the control block has to be zero
    qo, out, dense, alike = (torch.empty_like(q) for _ in range(4))
    sel, n_sel = i32([[[0] * 6] * hkv] * n_seq), i32([0] * n_seq)
    cu, gs, pl = i32([0, 1, 2, 3]), i32([0, 3]), i32([0])

    def step():
        S.qk_norm_rope(q, k, v, None, None, cache=p.cache, slots=slots, q_out=qo, workspace=ws)
        S.page_bounds(p.cache, full, bounds, workspace=ws)
        S.page_select(qo, p.cache, bounds, table, seqs, pos, 6, 1, 2, sel=sel, n_sel=n_sel, workspace=ws)
        S.attn_pages(qo, p.cache, table, seqs, pos, sel, n_sel, out=out, workspace=ws)
        S.attn_shared(qo, p.cache, table, pos, cu, gs, pl, out=alike, workspace=ws)
        S.attn_tree(qo, p.cache, table, pos, cu, out=dense, workspace=ws)

    def feed(i):
        now = [n + i for n in start]
        pos.copy_(i32(now))
        at = [int(p.table[s, n // page]) * page + n % page for s, n in enumerate(now)]
        slots.copy_(i32(at))
        full.copy_(i32([int(p.table[s, n // page]) if n % page == page - 1 else -1 for s, n in enumerate(now)]))
        q.copy_(torch.randn(n_seq, hq, D, generator=gen(i)))
        for s, n in enumerate(now):
            k[s], v[s] = (c[int(p.table[s, n // page]), :, n % page] for c in (keys, values))
        return now

    side = torch.cuda.Stream()
    feed(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for i in range(0, 38, 3):
        for j in range(max(0, i - 2), i + 1):
            now = feed(j)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
        assert S.read_device_error(ws) == 0
        c = Tokens.__new__(Tokens)
        c.p, c.hq, c.hkv, c.D, c.page, c.dt, c.seqs, c.pos = p, hq, hkv, D, page, "bf16", [0, 1, 2], now
        c.q, c.table, c.bounds = q.cpu(), p.table, bounds
        c.check_choice(sel, n_sel, 6, 1, 2)
        c.check_attention(out, sel, n_sel)
        if i % 9 == 0:
            for s, n in enumerate(now):
                for h in range(hq):
                    ref = ref_attention(c.q[s:s + 1, h], p.k[s][:n + 1, h // 4], p.v[s][:n + 1, h // 4],
                                        torch.ones(1, n + 1, dtype=torch.bool), D ** -0.5)
                    check_attention(alike[s:s + 1, h].cpu(), *ref, D, n + 9, True)
                    check_attention(dense[s:s + 1, h].cpu(), *ref, D, n + 1, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_calls_at_once(S, dt):  # noqa: F811
    """On two streams, a workspace each: what each call gives alone, bit for bit."""
    groups, prefix, own = [40, 3], [700, 128], [9 * i % 250 for i in range(43)]
    of = [x for m, x in zip(groups, prefix) for _ in range(m)]
    p = Paged(S, [a + b for a, b in zip(of, own)], [2] * 43, 16, 4, 128, 32, dt, 8)
    share(p, groups, prefix, 32)
    c = Tokens(S, [900, 700], [list(range(500, 640)), list(range(70))], 16, 4, 128, 32, dt, 5)
    sel, n_sel = c.select(S, 9)
    sel = widen(sel, 1024)
    calls = [lambda ws, out: call_shared(S, p, groups, prefix, workspace=ws, out=out),
             lambda ws, out: c.attend(S, sel, n_sel, workspace=ws, out=out)]
    sizes = [(S.WS_ATTN_SHARED, 86, 43), (S.WS_ATTN_PAGES, len(c.pos), 2)]
    jobs = []
    for i in range(4):  # each call twice, on its own stream
        which, T, n_seq = sizes[i % 2]
        ws = S.alloc_attn_workspace(which, T, n_seq, 16, 4, 128)
        jobs.append((calls[i % 2], ws, torch.empty(T, 16, 128, dtype=dtype_of(dt), device="cuda"), torch.cuda.Stream()))
    alone = []
    for call, ws, out, _ in jobs:
        call(ws, out)
        torch.cuda.synchronize()
        alone.append(out.clone())
    p.check(alone[0])
    c.check_attention(alone[1], sel, n_sel)
    for _ in range(5):
        for call, ws, out, stream in jobs:
            with torch.cuda.stream(stream):
                out.zero_()
                call(ws, out)
        torch.cuda.synchronize()
        for (_, ws, out, _), want in zip(jobs, alone):
            assert torch.equal(out, want) and S.read_device_error(ws) == 0


@pytest.mark.gpu
def test_pages_past_32_bit_offsets(S):  # noqa: F811
    """Pages whose elements lie past 2^32, for every call."""
    hkv, page, D = 8, 64, 128
    first = 2 ** 32 // (hkv * page * D) + 1
    c = Tokens(S, [450, 390], [[449], [389]], 16, hkv, D, page, "bf16", 3, fill=0.0, first_page=first)
    sel, n_sel = c.select(S, 4)
    c.check_choice(sel, n_sel, 4, 1, 1)
    out = c.attend(S, sel, n_sel)
    c.check_attention(out, sel, n_sel)
    p = Paged(S, [300, 260], [1, 2], 16, hkv, D, page, "bf16", 3, fill=0.0, first_page=first)
    share(p, [2], [256], page)
    p.check(call_shared(S, p, [2], [256]))


@pytest.mark.gpu
def test_what_the_calls_make_belongs_to_their_launch_stream(S):  # noqa: F811
    from tests.test_attention_binding import stream_of
    c = Tokens(S, [450, 390], [[449], [389]], 8, 2, 64, 16, "bf16", 3, fill=0.0)
    p = Paged(S, [300, 260], [1, 2], 8, 2, 64, 16, "bf16", 3)
    q, table, seqs, pos = c.queries(), c.table.cuda(), i32(c.seqs), i32(c.pos)
    ids = c.table[0, :28].cuda()
    args = (p.q.cuda(), p.cache, p.table.cuda(), i32(p.ctx), p.cu.cuda(), i32([0, 2]), i32([0]))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = S.page_bounds(c.cache, ids, stream=side)
    sel, n_sel = S.page_select(q, c.cache, c.bounds, table, seqs, pos, 4, stream=side)
    out = S.attn_pages(q, c.cache, table, seqs, pos, sel, n_sel, stream=side.cuda_stream)
    alike = S.attn_shared(*args, stream=side)
    torch.cuda.synchronize()
    for t in (b, sel, n_sel, out, alike):
        assert stream_of(t) == side.cuda_stream
    c.check_choice(sel, n_sel, 4, 1, 1)
    c.check_attention(out, sel, n_sel)
    p.check(alike, masks=None)


@pytest.mark.gpu
def test_empty_calls_and_the_most_sequences(S):  # noqa: F811
    p = Paged(S, [20], [2], 4, 2, 64, 16, "bf16", 1)
    e, zero = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), i32([0, 0])
    bounds = torch.zeros(p.cache.n_pages, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = p.table.cuda()
    assert S.attn_shared(e, p.cache, table, zero[:1], zero, zero, zero[:1]).shape == (0, 4, 64)
    sel, n_sel = S.page_select(e, p.cache, bounds, table, zero[:0], zero[:0], 3)
    assert sel.shape == (0, 2, 3) and n_sel.shape == (0,)
    assert S.attn_pages(e, p.cache, table, zero[:0], zero[:0], sel, n_sel).shape == (0, 4, 64)
    # 1024 sequences in 256 groups, most without new tokens
    n, groups, prefix = [0, 0, 1, 0] * 256, [4] * 256, [(16 * i) % 96 for i in range(256)]
    own = [(7 * i) % 30 for i in range(1024)]
    p = Paged(S, [prefix[i // 4] + c for i, c in enumerate(own)], n, 4, 2, 64, 16, "bf16", 2)
    share(p, groups, prefix, 16)
    p.check(call_shared(S, p, groups, prefix))


# ---------------------------------------------------------------------------
# refusals (before anything is launched)
# ---------------------------------------------------------------------------

def test_shared_refusals(S):  # noqa: F811
    L = S.lib()

    def call(q=16, qs=512, T=3, hq=4, cache="kv", table=16, width=4, ctx=16, cu=16, n=1, gs=16, pl=16, ng=1, mask=16,
             scale=0.1, out=16, ws=256, wb=1 << 40):
        return L.sffn_attn_shared(q, qs, T, hq, kv(S) if cache == "kv" else cache, table, width, ctx, cu, n, gs, pl, ng,
                                  mask, scale, out, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(cache=None) == S.ERR_INVALID_ARG and call(cache=kv(S, dtype=S.INT4_G64)) == S.ERR_INVALID_ARG
    assert call(cache=kv(S, head_dim=32)) == S.ERR_SHAPE and call(cache=kv(S, page_size=4)) == S.ERR_SHAPE
    assert call(hq=5) == S.ERR_SHAPE and call(T=-1) == S.ERR_SHAPE and call(T=65537) == S.ERR_SHAPE
    assert call(n=0) == S.ERR_SHAPE and call(n=1025) == S.ERR_SHAPE and call(width=0) == S.ERR_SHAPE
    assert call(ng=0) == S.ERR_SHAPE and call(ng=257) == S.ERR_SHAPE
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(scale=scale) == S.ERR_INVALID_ARG
    for name in ("q", "table", "ctx", "cu", "gs", "pl", "out"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    assert call(q=8) == S.ERR_ALIGNMENT and call(out=8) == S.ERR_ALIGNMENT and call(mask=12) == S.ERR_ALIGNMENT
    assert call(qs=500) == S.ERR_SHAPE and call(qs=516) == S.ERR_ALIGNMENT
    for bad in ((65537, 1), (10, 0), (10, 1025), (-1, 1)):
        assert S.attn_workspace_size(S.WS_ATTN_SHARED, *bad, 4, 2, 128) == 0


def test_bounds_refusals(S):  # noqa: F811
    L = S.lib()

    def call(cache="kv", pages=16, n=3, bounds=16, ws=256, wb=256):
        return L.sffn_page_bounds(kv(S) if cache == "kv" else cache, pages, n, bounds, ws, wb, None)

    assert call(n=0) == S.OK
    assert call(cache=None) == S.ERR_INVALID_ARG and call(cache=kv(S, head_dim=96)) == S.ERR_SHAPE
    assert call(cache=kv(S, k=8)) == S.ERR_ALIGNMENT and call(cache=kv(S, n_kv_heads=0)) == S.ERR_SHAPE
    assert call(n=-1) == S.ERR_SHAPE and call(n=(1 << 20) + 1) == S.ERR_SHAPE
    assert call(pages=None) == S.ERR_INVALID_ARG and call(bounds=None) == S.ERR_INVALID_ARG
    assert call(bounds=8) == S.ERR_ALIGNMENT
    assert call(ws=None) == S.ERR_WORKSPACE and call(ws=64) == S.ERR_WORKSPACE and call(wb=128) == S.ERR_WORKSPACE
    assert S.attn_workspace_size(S.WS_PAGE_BOUNDS, 10, 1, 2, 2, 128) == 256


def test_select_refusals(S):  # noqa: F811
    L = S.lib()

    def call(q=16, qs=512, T=3, hq=4, cache="kv", bounds=16, table=16, width=4, n=1, seqs=16, pos=16, first=1, recent=1,
             keep=4, sel=16, n_sel=16, ws=256, wb=1 << 40):
        return L.sffn_page_select(q, qs, T, hq, kv(S) if cache == "kv" else cache, bounds, table, width, n, seqs, pos,
                                  first, recent, keep, sel, n_sel, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(cache=None) == S.ERR_INVALID_ARG and call(cache=kv(S, head_dim=32)) == S.ERR_SHAPE
    assert call(hq=5) == S.ERR_SHAPE and call(T=-1) == S.ERR_SHAPE and call(T=65537) == S.ERR_SHAPE
    assert call(width=0) == S.ERR_SHAPE and call(width=32769) == S.ERR_SHAPE and call(n=0) == S.ERR_SHAPE
    assert call(keep=0) == S.ERR_SHAPE and call(keep=4097) == S.ERR_SHAPE
    assert call(first=-1) == S.ERR_INVALID_ARG and call(recent=0) == S.ERR_INVALID_ARG
    assert call(first=3, recent=2) == S.ERR_INVALID_ARG and call(first=2 ** 31 - 1) == S.ERR_INVALID_ARG
    assert call(recent=2 ** 31 - 1) == S.ERR_INVALID_ARG
    for name in ("q", "bounds", "table", "seqs", "pos", "sel", "n_sel"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    assert call(q=8) == S.ERR_ALIGNMENT and call(bounds=8) == S.ERR_ALIGNMENT and call(qs=516) == S.ERR_ALIGNMENT
    assert call(ws=None) == S.ERR_WORKSPACE and call(wb=256) == S.ERR_WORKSPACE
    size = L.sffn_page_select_workspace_size
    assert size(3, 2, 4) >= 256 + 3 * 2 * 4 * 4
    assert size(65537, 2, 4) == 0 and size(3, 0, 4) == 0 and size(3, 2, 0) == 0 and size(3, 2, 32769) == 0


def test_pages_refusals(S):  # noqa: F811
    L = S.lib()

    def call(q=16, qs=512, T=3, hq=4, cache="kv", table=16, width=4, n=1, seqs=16, pos=16, sel=16, n_sel=16, keep=4,
             scale=0.1, out=16, ws=256, wb=1 << 40):
        return L.sffn_attn_pages(q, qs, T, hq, kv(S) if cache == "kv" else cache, table, width, n, seqs, pos, sel, n_sel,
                                 keep, scale, out, ws, wb, None)

    assert call(T=0) == S.OK
    assert call(cache=None) == S.ERR_INVALID_ARG and call(cache=kv(S, page_size=24)) == S.ERR_SHAPE
    assert call(hq=5) == S.ERR_SHAPE and call(T=-1) == S.ERR_SHAPE and call(T=65537) == S.ERR_SHAPE
    assert call(width=0) == S.ERR_SHAPE and call(n=0) == S.ERR_SHAPE
    assert call(keep=0) == S.ERR_SHAPE and call(keep=4097) == S.ERR_SHAPE
    assert call(scale=0.0) == S.ERR_INVALID_ARG and call(scale=math.inf) == S.ERR_INVALID_ARG
    for name in ("q", "table", "seqs", "pos", "sel", "n_sel", "out"):
        assert call(**{name: None}) == S.ERR_INVALID_ARG, name
    assert call(q=8) == S.ERR_ALIGNMENT and call(out=8) == S.ERR_ALIGNMENT and call(qs=500) == S.ERR_SHAPE
    assert S.attn_workspace_size(S.WS_ATTN_PAGES, 65537, 1, 4, 2, 128) == 0


def test_tensors_of_another_device_are_refused(S, monkeypatch):  # noqa: F811
    class Elsewhere:
        device = torch.device("cuda", 1)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(S.SffnError) as e:
        S._here(Elsewhere, "here")
    assert e.value.status == S.ERR_INVALID_ARG
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    S._here(Elsewhere, "here")


@pytest.mark.gpu
def test_binding_checks(S):  # noqa: F811
    p = Paged(S, [20], [2], 4, 2, 64, 16, "bf16", 1)
    q, table, one, cu = p.q.cuda().contiguous(), p.table.cuda(), i32([0, 0]), i32([0, 2])
    bounds = torch.zeros(p.cache.n_pages, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    sel, n_sel = S.page_select(q, p.cache, bounds, table, one, i32([20, 21]), 2)

    def refused(fn, *a, **kw):
        with pytest.raises(S.SffnError):
            fn(*a, **kw)

    refused(S.attn_shared, q.float(), p.cache, table, cu[:1], cu, i32([0, 1]), cu[:1])            # not the cache's type
    refused(S.attn_shared, q, p.cache, table, cu[:1].long(), cu, i32([0, 1]), cu[:1])             # 64-bit lengths
    refused(S.attn_shared, q, p.cache, table, cu[:1], cu, i32([0]), cu[:1])                       # too few offsets
    refused(S.page_bounds, p.cache, torch.zeros(2, dtype=torch.int32))                            # host memory
    refused(S.page_bounds, p.cache, one, bounds[:-1])
    refused(S.page_bounds, p.cache, one, bounds.float())
    refused(S.page_select, q, p.cache, bounds[:-1], table, one, one, 2)
    refused(S.page_select, q, p.cache, bounds, table, one[:1], one, 2)
    refused(S.page_select, q, p.cache, bounds, table, one, one, 2, sel=sel[:1].contiguous())
    refused(S.page_select, q, p.cache, bounds, table, one, one, 0)
    refused(S.page_select, q, p.cache, bounds, table.expand(2, -1), one, one, 2)              # rows not contiguous
    refused(S.attn_pages, q, p.cache, table, one, one, sel[:1].contiguous(), n_sel)
    refused(S.attn_pages, q, p.cache, table, one, one, sel[:, :1].contiguous(), n_sel)
    refused(S.attn_pages, q, p.cache, table, one, one, sel.transpose(0, 1), n_sel)
    refused(S.attn_pages, q, p.cache, table, one, one, sel, n_sel, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
