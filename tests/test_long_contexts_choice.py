"""The choice of pages (sffn_page_select) where its other kernels run: many lists (a warp each), tokens of many query heads taken
several at a time, batches of whole prompts' pieces.  Against 64 bits, exactly: scores are whole multiples of a power of two,
and equal ones go to the lower page."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import S, gen  # noqa: F401  (S: the library)
from tests.test_long_contexts import MANY, TOP, Tokens, step_of

pytestmark = pytest.mark.gpu


def check_lists(c, sel, n_sel, keep, first, recent):
    """As Tokens.check_choice, all tokens of a sequence at a time."""
    sel, n_sel, bounds, G = sel.cpu(), n_sel.cpu().tolist(), c.bounds.cpu().double(), c.hq // c.hkv
    for s in sorted(set(c.seqs)):
        rows = [t for t, (x, p) in enumerate(zip(c.seqs, c.pos)) if x == s and p >= 0]
        if not rows:
            continue
        mine = torch.tensor([c.pos[t] // c.page for t in rows])
        page = torch.arange(int(mine.max()) + 1)
        b = bounds[c.table[s, :len(page)].long()]
        for h in range(c.hkv):
            q = c.q[rows, h * G:(h + 1) * G].double()
            q = torch.where(q.isnan(), 0.0, q).clamp(-TOP, TOP)
            step = torch.tensor([step_of(x) for x in q.abs().amax((1, 2)).tolist()], dtype=torch.float64)
            code = torch.round(q / step[:, None, None])
            score = (code.clamp(min=0) @ b[:, h, 0].T + code.clamp(max=0) @ b[:, h, 1].T).amax(1)
            score = torch.where((page < first) | (page > mine[:, None] - recent), torch.inf, score)  # always
            score = torch.where(page > mine[:, None], -torch.inf, score)
            order = torch.sort(score, dim=1, descending=True, stable=True).indices
            for i, t in enumerate(rows):
                n = min(int(mine[i]) + 1, keep)
                want = order[i, :n].sort().values.tolist()
                assert n_sel[t] == n and sel[t, h].tolist() == want + [-1] * (keep - n), (t, h)


def pieces(S, lens, n, hq, hkv, D, page, dt, seed):  # noqa: F811
    """The last n[s] positions of each sequence."""
    return Tokens(S, lens, [list(range(a - b, a)) for a, b in zip(lens, n)], hq, hkv, D, page, dt, seed, fill=0.0)


# More lists than 16 an SM of up to 160 of them (2560): a warp takes a list; widths up to 512 and up to 1024; numbers of
# lists that are no multiple of four.
@pytest.mark.parametrize("lens,n,hq,hkv,D,page,dt,first,recent,keep", [
    ([2600, 300], [801, 61], 9, 3, 64, 8, "bf16", 1, 2, 24),        # 326 columns, 2586 lists
    ([4088], [2605], 2, 1, 64, 8, "bf16", 0, 1, 9),                 # 512 columns
    ([4100, 17], [641, 3], 8, 4, 128, 8, "bf16", 2, 3, 65),         # 514 columns
    ([8184], [865], 3, 3, 64, 8, "f32", 1, 1, 200),                 # 1024 columns
    ([5000, 5000], [430, 437], 12, 3, 128, 8, "bf16", 1, 4, 5),     # the forced ones alone
    ([3000], [2601], 1, 1, 64, 32, "f32", 0, 1, 2),
])
def test_many_lists(S, lens, n, hq, hkv, D, page, dt, first, recent, keep):  # noqa: F811
    assert sum(n) * hkv >= 2560
    c = pieces(S, lens, n, hq, hkv, D, page, dt, sum(lens))
    T = len(c.pos)
    g = gen(keep)
    some = sorted(torch.randperm(T, generator=g)[:9].tolist() + [0, T - 1])
    for t in some:  # padding
        c.pos[t] = -1
    ws = S.alloc_page_select_workspace(T, hkv, c.table.shape[1])
    sel, n_sel = c.select(S, keep, first, recent, workspace=ws)
    assert S.read_device_error(ws) == 0
    assert not n_sel[some].any() and (sel[some] == -1).all()
    check_lists(c, sel, n_sel, keep, first, recent)
    again = c.select(S, keep, first, recent, workspace=ws)
    assert torch.equal(again[0], sel) and torch.equal(again[1], n_sel)


@pytest.mark.parametrize("len_,n,hkv", [(2500, 1300, 2), (6000, 900, 3)])
def test_many_lists_with_ties_at_the_cut(S, len_, n, hkv):  # noqa: F811
    """Every third page is the same page of the cache, others come in pairs; some queries are zero."""
    c = pieces(S, [len_], [n], 2 * hkv, hkv, 64, 8, "bf16", 3)
    pages = len_ // 8
    c.table[0, 1:pages:3] = c.table[0, 1]
    c.table[0, 2:pages - 3:6] = c.table[0, 5:pages:6][:len(c.table[0, 2:pages - 3:6])]
    c.q[::50] = 0
    for keep, first, recent in ((2, 0, 1), (40, 1, 1), (pages // 3 + 5, 0, 2), (pages // 2, 2, 3)):
        sel, n_sel = c.select(S, keep, first, recent)
        check_lists(c, sel, n_sel, keep, first, recent)


# Query heads a key head: products of 8 rows, several a token, several tokens a CTA where they fit.
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,D", [
    (9, 1, 64), (12, 1, 128), (16, 1, 64), (20, 1, 128), (28, 1, 64), (32, 1, 128), (33, 1, 64), (48, 1, 128), (64, 1, 64),
    (24, 2, 128), (3, 1, 64), (5, 1, 128), (2, 1, 64), (6, 6, 128), (64, 2, 64),
])
def test_query_heads_of_several_tokens(S, hq, hkv, D, dt):  # noqa: F811
    c = Tokens(S, [700, 400, 650], [list(range(590, 700)), list(range(100, 400, 23)), [3, 649, 600, 599, 601]], hq, hkv, D, 16,
               dt, hq + D, fill=0.0)
    for keep, first, recent in ((11, 1, 2), (3, 0, 1)):
        check_lists(c, *c.select(S, keep, first, recent), keep, first, recent)


@pytest.mark.parametrize("lens,at,hq,hkv,D,page,keep", MANY)
def test_pieces_whose_attention_is_tested(S, lens, at, hq, hkv, D, page, keep):  # noqa: F811
    c = Tokens(S, lens, at, hq, hkv, D, page, "bf16", sum(lens) + hq)
    first = 1 if keep > 1 else 0
    check_lists(c, *c.select(S, keep, first), keep, first, 1)


def test_decode_tokens_beside_a_piece_of_a_prompt(S):  # noqa: F811
    """Runs of one token and of many in one call, the sequences in any order."""
    lens = [900] + [500 + 11 * i for i in range(30)]
    at = [list(range(700, 900))] + [[n - 1] for n in lens[1:]]
    c = Tokens(S, lens, at, 28, 4, 128, 16, "bf16", 9, fill=0.0)
    order = torch.randperm(len(c.pos), generator=gen(2)).tolist()
    for o in (list(range(len(c.pos))), order):
        d = Tokens.__new__(Tokens)
        d.__dict__.update(c.__dict__)
        d.seqs, d.pos, d.q = [c.seqs[t] for t in o], [c.pos[t] for t in o], c.q[o]
        sel, n_sel = d.select(S, 13, 1, 2)
        check_lists(d, sel, n_sel, 13, 1, 2)
        d.check_attention(d.attend(S, sel, n_sel), sel, n_sel)
