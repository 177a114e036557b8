"""Attention over long contexts in the paged cache: one prefix that many sequences share, read
once for all of them (``attn_shared``), and attention over the few pages that a cheap score picks
for each token: the pages' key bounds (``page_bounds``), the choice (``page_select``) and the
attention over the chosen pages (``attn_pages``).

Each case is run either in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or through the package's own calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
_TOP = 2.0 ** 100   # keys and queries beyond this count as this in bounds and scores
_LEAST = -100       # least exponent of their steps


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def listed():
    ragged = [0, 17, 640, 1999, 300, 1111, 64, 1500]
    return [
        # four answers begun after one system prompt, multi-head: the smallest call of a decode loop
        dict(name="shared-few", op="shared", groups="4", prefix="1024", own="0,7,40,13", n="1,1,1,1", hq=32,
             hkv=32, D=128, dtype="bf16", page=16),
        # a server's batch of questions on one long document
        dict(name="shared-batch", op="shared", groups="96", prefix="24576", own=_text(ragged * 12),
             n=_text([1] * 96), hq=64, hkv=8, D=128, dtype="bf16", page=64),
        # several prompts in one batch (one sequence shares nothing), drafted tokens, seven query heads for
        # each key head, a prefix that ends inside a page
        dict(name="shared-drafts", op="shared", groups="14,5,1,2", prefix="12032,4096,0,1000",
             own=_text([0, 333, 1200, 64, 90, 2047, 5] * 2 + [700, 0, 12, 150, 1] + [3001] + [80, 2500]),
             n=_text([8, 1, 25, 3, 8, 5, 16] * 2 + [8, 8, 2, 1, 4] + [7] + [33, 9]), hq=28, hkv=4, D=128,
             dtype="bf16", page=128),
        # the fp32 decode path, short heads
        dict(name="shared-f32", op="shared", groups="3,2", prefix="1504,640", own="10,200,0,77,31",
             n="1,5,2,1,3", hq=16, hkv=2, D=64, dtype="f32", page=32),
        # a decode step of the fp32 path: two of eight sequences have filled a page
        dict(name="bounds-step-f32", op="bounds", n=8, full=2, pool=512, hkv=2, D=64, dtype="f32", page=32),
        # every page of a long prompt, right after its prefill
        dict(name="bounds-prompt", op="bounds", n=1024, full=1024, pool=1100, hkv=8, D=128, dtype="bf16", page=64),
        # one decoded token over a long context
        dict(name="select-token", op="select", pos="65530", n="1", hq=64, hkv=8, D=128, dtype="bf16", page=64,
             first=1, recent=2, keep=64),
        # a decode step of a ragged batch, one sequence at its first token, small pages
        dict(name="select-batch", op="select", pos=_text([0, 1017, 16000, 4095, 9000, 2500, 13777, 801] * 6),
             n=_text([1] * 48), hq=32, hkv=8, D=128, dtype="bf16", page=16, first=1, recent=4, keep=128),
        # the next pieces of two prompts, seven query heads for each key head
        dict(name="select-chunk", op="select", pos="15000,3000", n="700,345", hq=28, hkv=4, D=128, dtype="bf16",
             page=32, first=1, recent=2, keep=48),
        # three tokens of the fp32 decode path, short heads
        dict(name="pages-token-f32", op="pages", pos="1999,300,4000", n="1,1,1", hq=16, hkv=2, D=64, dtype="f32",
             page=32, first=1, recent=1, keep=16),
        # the ragged batch's decode step: 2048 of up to 16000 positions
        dict(name="pages-batch", op="pages", pos=_text([0, 1017, 16000, 4095, 9000, 2500, 13777, 801] * 6),
             n=_text([1] * 48), hq=32, hkv=8, D=128, dtype="bf16", page=16, first=1, recent=4, keep=128),
        # the two prompts' next pieces: 1536 of up to 15700 positions for each token
        dict(name="pages-chunk", op="pages", pos="15000,3000", n="700,345", hq=28, hkv=4, D=128, dtype="bf16",
             page=32, first=1, recent=2, keep=48),
    ]


_HEADS = [(32, 32), (16, 2), (64, 8), (28, 4), (40, 8), (32, 8), (5, 1), (12, 12), (20, 20)]
_PAGES = [16, 32, 64, 128]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "bounds", "select", "pages"])
    hq, hkv = rng.choice(_HEADS)
    case = dict(op=op, hkv=hkv, D=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                page=rng.choice(_PAGES))
    D, page, f32 = case["D"], case["page"], case["dtype"] == "f32"
    if op == "bounds":
        pool = max(1, min(4096, (16_000_000 if f32 else 64_000_000) // (hkv * page * D)))
        n = _log(rng, 1, pool)
        return dict(case, n=n, full=rng.randint(1, n), pool=pool)
    case["hq"] = hq
    if op == "shared":
        n_seq = _log(rng, 1, 96)
        sizes = []
        while sum(sizes) < n_seq:
            sizes.append(rng.randint(1, n_seq - sum(sizes)))
        nmax = rng.choice([1, 1, 8, 64])
        # scores of the largest call, and the cache's elements
        top = max(64, min(32768, (8_000_000 if f32 else 100_000_000) // (n_seq * nmax * hq), 40_000_000 // (hkv * D)))
        prefix = [_log(rng, 1, top) - 1 for _ in sizes]
        top = max(2, min(4096, 20_000_000 // (n_seq * hkv * D)))
        return dict(case, groups=_text(sizes), prefix=_text(prefix),
                    own=_text([_log(rng, 1, top) - 1 for _ in range(n_seq)]),
                    n=_text([rng.randint(1, nmax) for _ in range(n_seq)]))
    n_seq = _log(rng, 1, 48)
    nmax = _log(rng, 1, max(1, min(512, (128 if f32 else 1024) // n_seq)))
    top = max(2, min(65536, 80_000_000 // (n_seq * hkv * D)))
    first, recent = rng.randint(0, 2), rng.randint(1, 4)
    keep = first + recent + _log(rng, 1, 2048 // page)
    return dict(case, pos=_text([_log(rng, 1, top) - 1 for _ in range(n_seq)]),
                n=_text([rng.randint(1, nmax) for _ in range(n_seq)]), first=first, recent=recent, keep=keep)


def work(case):
    hkv, D, page, es = case["hkv"], case["D"], case["page"], _ES[case["dtype"]]
    if case["op"] == "bounds":
        keys = case["full"] * hkv * page * D
        return {"bytes": keys * es + case["full"] * hkv * 4 * D + 4 * case["n"], "flops": 2 * keys}
    hq, new = case["hq"], _ints(case["n"])
    T = sum(new)
    if case["op"] == "shared":
        own_len, sizes = _ints(case["own"]), _ints(case["groups"])
        prefix = [p for p, m in zip(_ints(case["prefix"]), sizes) for _ in range(m)]
        keys = sum(_ints(case["prefix"])) + sum(own_len) + T
        pairs = sum((p + c + n) * n for p, c, n in zip(prefix, own_len, new))
        return {"bytes": es * (keys * hkv * D * 2 + 2 * T * hq * D), "flops": 4 * pairs * hq * D}
    pos, keep = _ints(case["pos"]), case["keep"]
    own_page = [[(p + i) // page for i in range(n)] for p, n in zip(pos, new)]  # each token's own page
    if case["op"] == "select":
        scored = sum(sum(p for p in row if p + 1 > keep) for row in own_page)  # with fewer pages all are taken
        read = sum(max([p for p in row if p + 1 > keep], default=0) for row in own_page)
        return {"bytes": read * hkv * 4 * D + T * hq * D * es + T * hkv * keep * 4,
                "flops": 4 * scored * hq * D}
    chosen = sum(min(keep * page, p + i + 1) for p, n in zip(pos, new) for i in range(n))
    read = sum(min(p + n, sum(min(keep * page, p + i + 1) for i in range(n))) for p, n in zip(pos, new))
    return {"bytes": es * (read * hkv * D * 2 + 2 * T * hq * D) + 4 * T * hkv * keep, "flops": 4 * chosen * hq * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(shape, g, dtype, scale=1.0):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    t.normal_(0.0, scale, generator=g)
    return t


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _tree_masks(n, g):
    """Ancestors-and-self masks (bit j: drafted token j) of a random tree of n drafted tokens."""
    u = torch.rand(n, generator=g).tolist()
    masks = []
    for i in range(n):
        parent = int(u[i] * (i + 1)) - 1  # -1: hangs on the context itself
        masks.append((1 << i) | (masks[parent] if parent >= 0 else 0))
    return [m - (1 << 64) if m >> 63 else m for m in masks]  # as signed 64-bit


def _cache(s, n_pages, g):
    """Keys that lie near one another within a page, as those of one passage do; and values."""
    dt = _DT[s["dtype"]]
    s["ck"] = _randn((n_pages, s["hkv"], s["page"], s["D"]), g, dt)
    s["ck"] += _randn((n_pages, s["hkv"], 1, s["D"]), g, dt, 0.7)
    s["cv"] = _randn((n_pages, s["hkv"], s["page"], s["D"]), g, dt)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "bounds":
        _cache(s, case["pool"], g)
        pages = torch.full((case["n"],), -1, dtype=torch.int32)
        gc = torch.Generator()
        gc.manual_seed(int(seed))
        pages[torch.randperm(case["n"], generator=gc)[:case["full"]]] = \
            torch.randperm(case["pool"], generator=gc)[:case["full"]].int()
        s["pages"] = pages.cuda()
        s["bounds"] = torch.zeros((case["pool"], case["hkv"], 2, case["D"]), dtype=torch.bfloat16, device="cuda")
    else:
        (_prepare_shared if case["op"] == "shared" else _prepare_pages)(s, g, seed)
    if own:
        _keep(s)
    return s


def _prepare_shared(s, g, seed):
    page = s["page"]
    for key in ("groups", "prefix", "own", "n"):
        s[key] = _ints(s[key])
    group = [i for i, m in enumerate(s["groups"]) for _ in range(m)]
    prefix = [s["prefix"][i] for i in group]
    ctx = [p + c for p, c in zip(prefix, s["own"])]
    common = [p // page for p in s["prefix"]]                                         # whole pages are shared
    alone = [(c + n + page - 1) // page - common[i] for c, n, i in zip(ctx, s["n"], group)]
    n_pages = sum(common) + sum(alone) + 3
    _cache(s, n_pages, g)
    T, dt = sum(s["n"]), _DT[s["dtype"]]
    s["q"] = _randn((T, s["hq"] + 2 * s["hkv"], s["D"]), g, dt, 1.25)[:, :s["hq"]]
    gc = torch.Generator()
    gc.manual_seed(int(seed))
    order = torch.randperm(n_pages, generator=gc).int()
    table = torch.zeros((len(ctx), max(common[i] + m for i, m in zip(group, alone)) + 1), dtype=torch.int32)
    first, after = _offsets(common), [sum(common) + o for o in _offsets(alone)]
    for r, (i, m) in enumerate(zip(group, alone)):
        table[r, :common[i]] = order[first[i]:first[i] + common[i]]
        table[r, common[i]:common[i] + m] = order[after[r]:after[r] + m]
    s["table"], s["ctx"], s["cu"] = table.cuda(), _i32(ctx), _i32(_offsets(s["n"]))
    s["group_seqs"], s["prefix_lens"] = _i32(_offsets(s["groups"])), _i32(s["prefix"])
    s["mask"] = None
    if max(s["n"]) > 1:
        s["mask"] = torch.tensor(sum((_tree_masks(n, gc) for n in s["n"]), []), dtype=torch.int64, device="cuda")
    # where each token stands: its sequence and its number among the new ones
    s["seq"] = torch.tensor([r for r, n in enumerate(s["n"]) for _ in range(n)], device="cuda")
    s["at"] = torch.tensor([i for n in s["n"] for i in range(n)], device="cuda")
    s["group_of"] = torch.tensor(group, device="cuda")


def _prepare_pages(s, g, seed):
    page, hkv = s["page"], s["hkv"]
    s["pos"], s["n"] = _ints(s["pos"]), _ints(s["n"])
    need = [(p + n + page - 1) // page for p, n in zip(s["pos"], s["n"])]
    n_pages, width = sum(need) + 3, max(need) + 1
    _cache(s, n_pages, g)
    T = sum(s["n"])
    s["q"] = _randn((T, s["hq"] + 2 * hkv, s["D"]), g, _DT[s["dtype"]], 1.25)[:, :s["hq"]]
    gc = torch.Generator()
    gc.manual_seed(int(seed))
    order = torch.randperm(n_pages, generator=gc).int()
    table = torch.zeros((len(need), width), dtype=torch.int32)
    for r, (a, m) in enumerate(zip(_offsets(need), need)):
        table[r, :m] = order[a:a + m]
    s["table"] = table.cuda()
    s["seqs"] = _i32([r for r, n in enumerate(s["n"]) for _ in range(n)])
    s["at"] = torch.tensor([i for n in s["n"] for i in range(n)], device="cuda")
    s["positions"] = _i32([p + i for p, n in zip(s["pos"], s["n"]) for i in range(n)])
    if s["op"] == "select":
        s["bounds"] = torch.zeros((n_pages, hkv, 2, s["D"]), dtype=torch.bfloat16, device="cuda")
        _plain_bounds(dict(s, pages=torch.arange(n_pages, device="cuda")))
        return
    # the chosen pages: neighbouring tokens want mostly the same ones
    like = torch.randn((len(need), hkv, width), generator=g, device="cuda")[s["seqs"].long()]
    like += 0.4 * torch.randn((T, hkv, width), generator=g, device="cuda")
    s["sel"], s["n_sel"] = _choose(s, like)


def _keep(s):
    """What a program of this package's calls keeps beside the inputs: cache handle, workspace, outputs."""
    from activation_sparse_ffn_gemv_gb300 import sffn
    s["cache"] = sffn.KVCache(s["ck"], s["cv"])
    hkv, D = s["hkv"], s["D"]
    if s["op"] == "bounds":
        s["ws"] = sffn.alloc_attn_workspace(sffn.WS_PAGE_BOUNDS, s["n"], 1, hkv, hkv, D)
        return
    T, hq, width = s["q"].shape[0], s["hq"], s["table"].shape[1]
    if s["op"] == "select":
        s["ws"] = sffn.alloc_page_select_workspace(T, hkv, width)
        s["sel"] = torch.empty((T, hkv, s["keep"]), dtype=torch.int32, device="cuda")
        s["n_sel"] = torch.empty(T, dtype=torch.int32, device="cuda")
        return
    which = sffn.WS_ATTN_SHARED if s["op"] == "shared" else sffn.WS_ATTN_PAGES
    s["ws"] = sffn.alloc_attn_workspace(which, T, s["table"].shape[0], hq, hkv, D)
    s["out"] = torch.empty((T, hq, D), dtype=s["q"].dtype, device="cuda")


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return {"shared": _own_shared, "bounds": _own_bounds, "select": _own_select, "pages": _own_pages}[s["op"]](s)
    return {"shared": _plain_shared, "bounds": _plain_bounds, "select": _plain_select, "pages": _plain_pages}[s["op"]](s)


def _own_shared(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.attn_shared(s["q"], s["cache"], s["table"], s["ctx"], s["cu"], s["group_seqs"], s["prefix_lens"],
                            s["mask"], out=s["out"], workspace=s["ws"])


def _own_bounds(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.page_bounds(s["cache"], s["pages"], s["bounds"], workspace=s["ws"])


def _own_select(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.page_select(s["q"], s["cache"], s["bounds"], s["table"], s["seqs"], s["positions"], s["keep"],
                            n_first=s["first"], n_recent=s["recent"], sel=s["sel"], n_sel=s["n_sel"],
                            workspace=s["ws"])


def _own_pages(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.attn_pages(s["q"], s["cache"], s["table"], s["seqs"], s["positions"], s["sel"], s["n_sel"],
                           out=s["out"], workspace=s["ws"])


def _softmax_av(scores, v):
    m = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - m)
    return torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)


def _paged(c, ids):
    """Rows of the pages ids [n, m] of a cache, one sequence after the other: fp32 [n, hkv, m * page, D]."""
    n, m = ids.shape
    return c[ids].permute(0, 2, 1, 3, 4).reshape(n, c.shape[1], m * c.shape[2], c.shape[3]).float()


def _plain_shared(s):
    """The scores of the prefixes, group by group (the groups' tokens padded to the largest), beside
    those of each sequence's own positions (padded likewise), under one softmax."""
    hq, hkv, D, page = s["hq"], s["hkv"], s["D"], s["page"]
    G, T, dev = hq // hkv, s["q"].shape[0], s["q"].device
    seq, at, ctx = s["seq"], s["at"], s["ctx"].long()
    group = s["group_of"][seq]
    whole = (s["prefix_lens"].long() // page) * page           # positions in shared pages
    start = s["cu"].long()[s["group_seqs"].long()]
    rank = torch.arange(T, device=dev) - start[group]           # a token's place in its group
    q = s["q"].float().view(T, hkv, G, D) / math.sqrt(D)

    def rows(ids, places, n, most):  # [n, hkv, most * G, D]: tokens dealt to padded batches
        x = torch.zeros((n, most, hkv, G, D), device=dev)
        x[ids, places] = q
        return x.permute(0, 2, 1, 3, 4).reshape(n, hkv, most * G, D)

    def back(x, ids, places, n, most):  # the tokens' rows again, [T, hkv, G, ...]
        return x.view(n, hkv, most, G, x.shape[-1])[ids, :, places]

    n_g, most_g = len(s["groups"]), max(sum(s["n"][a:b]) for a, b in zip(_offsets(s["groups"]), _offsets(s["groups"])[1:]))
    n_s, most_s = len(s["n"]), max(s["n"])
    pp = max(s["prefix"]) // page                               # pages of the longest prefix
    ids = s["table"].long()[s["group_seqs"].long()[:-1]][:, :pp]
    kp, vp = _paged(s["ck"], ids), _paged(s["cv"], ids)
    sc_p = back(torch.matmul(rows(group, rank, n_g, most_g), kp.transpose(2, 3)), group, rank, n_g, most_g)
    sc_p.masked_fill_((torch.arange(pp * page, device=dev) >= whole[group][:, None])[:, None, None], float("-inf"))
    lead = whole[s["group_of"]] // page                         # shared pages of each sequence
    mp = max(max((p % page + c + n + page - 1) // page for p, c, n in
                 zip([s["prefix"][i] for i, m in enumerate(s["groups"]) for _ in range(m)], s["own"], s["n"])), 1)
    col = (lead[:, None] + torch.arange(mp, device=dev)).clamp_(max=s["table"].shape[1] - 1)
    ids = torch.gather(s["table"].long(), 1, col)
    ko, vo = _paged(s["ck"], ids), _paged(s["cv"], ids)
    sc_o = back(torch.matmul(rows(seq, at, n_s, most_s), ko.transpose(2, 3)), seq, at, n_s, most_s)
    new = (lead * page)[seq][:, None] + torch.arange(mp * page, device=dev) - ctx[seq][:, None]  # new token's number
    sees = new < 0
    if s["mask"] is None:
        sees |= new <= at[:, None]
    else:
        sees |= ((s["mask"][:, None] >> new.clamp(0, 63)) & 1).bool() & (new < _new_counts(s)[seq][:, None])
    sc_o.masked_fill_(~sees[:, None, None], float("-inf"))
    m = torch.maximum(sc_p.amax(-1, keepdim=True), sc_o.amax(-1, keepdim=True)) if pp else sc_o.amax(-1, keepdim=True)
    p_p, p_o = torch.exp(sc_p - m), torch.exp(sc_o - m)
    total = p_p.sum(-1, keepdim=True) + p_o.sum(-1, keepdim=True)

    def weighed(p, v, ids, places, n, most):
        x = torch.zeros((n, most, hkv, G, p.shape[-1]), device=dev)
        x[ids, places] = p
        x = x.permute(0, 2, 1, 3, 4).reshape(n, hkv, most * G, p.shape[-1])
        return back(torch.matmul(x, v), ids, places, n, most)

    o = weighed(p_p, vp, group, rank, n_g, most_g) + weighed(p_o, vo, seq, at, n_s, most_s)
    return (o / total).reshape(T, hq, D).to(s["q"].dtype)


def _new_counts(s):
    return s["cu"][1:].long() - s["cu"][:-1].long()


def _step(most):
    """Least power of two 2^e, e >= -100, with most <= 127 * 2^e."""
    f, e = torch.frexp(most)                      # most = f 2^e, 1/2 <= f < 1
    e = (e - 7 + (f > 127.0 / 128.0)).clamp(min=_LEAST)
    return torch.ldexp(torch.ones_like(most), torch.where(most > 0, e, torch.full_like(e, _LEAST)))


def _plain_bounds(s):
    ids = s["pages"].long()
    ids = ids[ids >= 0]
    k = s["ck"][ids].float()                      # [n, hkv, page, D]
    hi = torch.nan_to_num(k, nan=_TOP).clamp_(-_TOP, _TOP).amax(2)
    lo = torch.nan_to_num(k, nan=-_TOP).clamp_(-_TOP, _TOP).amin(2)
    step = _step(torch.maximum(hi.abs(), lo.abs()).amax(-1))[..., None]
    s["bounds"][ids, :, 0] = (torch.ceil(hi / step) * step).bfloat16()
    s["bounds"][ids, :, 1] = (torch.floor(lo / step) * step).bfloat16()
    return s["bounds"]


def _choose(s, score):
    """Pages chosen by score [T, hkv, width], ascending, -1 behind them; how many."""
    keep = s["keep"]
    T, hkv, width = score.shape
    mine = s["positions"].long() // s["page"]
    page = torch.arange(width, device=score.device)
    always = (page < s["first"]) | (page > mine[:, None] - s["recent"])
    score = score.masked_fill(always[:, None], float("inf"))
    score = score.masked_fill((page > mine[:, None])[:, None], float("-inf"))
    count = (mine + 1).clamp(max=keep)
    by = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :keep]  # ties: the lower page first
    out = torch.full((T, hkv, keep), width, dtype=torch.int64, device=score.device)
    out[..., :by.shape[-1]] = by
    out = out.masked_fill((torch.arange(keep, device=score.device) >= count[:, None])[:, None], width)
    out = out.sort(dim=-1).values
    return out.masked_fill(out == width, -1).int(), count.int()


def _plain_select(s):
    hq, hkv, D = s["hq"], s["hkv"], s["D"]
    G, T, dev = hq // hkv, s["q"].shape[0], s["q"].device
    q = torch.nan_to_num(s["q"].float(), nan=0.0).clamp(-_TOP, _TOP).view(T, hkv, G * D)
    code = torch.round(q / _step(q.abs().amax(-1))[..., None]).view(T, hkv, G, D)
    both = torch.cat([code.clamp(min=0), code.clamp(max=0)], dim=-1)      # against upper and lower bounds
    n_s, most = len(s["n"]), max(s["n"])
    seq, at = s["seqs"].long(), s["at"]
    x = torch.zeros((n_s, most, hkv, G, 2 * D), device=dev)
    x[seq, at] = both
    x = x.permute(0, 2, 1, 3, 4).reshape(n_s, hkv, most * G, 2 * D)
    b = s["bounds"][s["table"].long()].permute(0, 2, 1, 3, 4).reshape(n_s, hkv, -1, 2 * D).float()
    # whole multiples, below 2^24, of a step: exact in 32 bits in any order
    sc = torch.matmul(x, b.transpose(2, 3)).view(n_s, hkv, most, G, -1).amax(3)
    return _choose(s, sc[seq, :, at])


def _plain_pages(s):
    hq, hkv, D, page = s["hq"], s["hkv"], s["D"], s["page"]
    G, T, dev = hq // hkv, s["q"].shape[0], s["q"].device
    sel = s["sel"].long()                                                 # [T, hkv, keep]
    there = torch.arange(sel.shape[-1], device=dev) < s["n_sel"].long()[:, None, None]
    ids = s["table"].long()[s["seqs"].long()[:, None, None], sel.clamp(min=0)]
    head = torch.arange(hkv, device=dev)[None, :, None]
    k = s["ck"][ids, head].reshape(T, hkv, -1, D).float()
    v = s["cv"][ids, head].reshape(T, hkv, -1, D).float()
    pos = sel[..., None] * page + torch.arange(page, device=dev)          # [T, hkv, keep, page]
    sees = (there[..., None] & (pos <= s["positions"].long()[:, None, None, None])).reshape(T, hkv, 1, -1)
    q = s["q"].float().view(T, hkv, G, D) / math.sqrt(D)
    sc = torch.matmul(q, k.transpose(2, 3)).masked_fill(~sees, float("-inf"))
    return _softmax_av(sc, v).reshape(T, hq, D).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_shared, "bounds": _exact_bounds, "select": _exact_select, "pages": _exact_pages}[case["op"]](s)


def _exact_rows(q, k, v, sees):
    """q [r, D], k and v [n, D] in 64 bits, sees [r, n]."""
    w = (q @ k.T).masked_fill(~sees, float("-inf"))
    return torch.exp(w - torch.logsumexp(w, dim=1, keepdim=True)) @ v


def _exact_shared(s):
    """Every sequence by itself over its own row of the table."""
    G, D, page = s["hq"] // s["hkv"], s["D"], s["page"]
    out = torch.empty((s["q"].shape[0], s["hq"], D), dtype=torch.float64, device="cuda")
    base = 0
    for i, (c, n) in enumerate(zip(s["ctx"].tolist(), s["n"])):
        at = torch.arange(c + n, device="cuda")
        ids, off = s["table"][i].long()[at // page], at % page
        sees = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        for r in range(n):
            word = s["mask"][base + r].item() if s["mask"] is not None else (1 << (r + 1)) - 1
            sees[r, c:] = torch.tensor([(word >> j) & 1 for j in range(n)], dtype=torch.bool)
        for h in range(s["hkv"]):
            k, v = s["ck"][ids, h, off].double(), s["cv"][ids, h, off].double()
            q = s["q"][base:base + n, h * G:(h + 1) * G].double().transpose(0, 1).reshape(G * n, D) / math.sqrt(D)
            o = _exact_rows(q, k, v, sees.repeat(G, 1))
            out[base:base + n, h * G:(h + 1) * G] = o.view(G, n, D).transpose(0, 1)
        base += n
    return out


def _exact_exponent(most):
    """Least e >= -100 with most <= 127 * 2^e, by halving from above."""
    e = torch.full_like(most, 100.0)
    for _ in range(200):
        e = torch.where((most <= 127.0 * torch.exp2(e - 1)) & (e > _LEAST), e - 1, e)
    return e


def _exact_bounds(s):
    out = s["bounds"].double()
    for p in s["pages"].tolist():
        if p < 0:
            continue
        k = s["ck"][p].double()
        step = torch.exp2(_exact_exponent(k.abs().flatten(1).max(1).values))[:, None]
        out[p, :, 0] = torch.ceil(k.max(1).values / step) * step
        out[p, :, 1] = torch.floor(k.min(1).values / step) * step
    return out


def _exact_select(s):
    """Token by token: pages above the cut, then as many of those at the cut as there is room for."""
    G, D, page, keep = s["hq"] // s["hkv"], s["D"], s["page"], s["keep"]
    T, hkv = s["q"].shape[0], s["hkv"]
    sel = torch.full((T, hkv, keep), -1, dtype=torch.int32, device="cuda")
    n_sel = torch.zeros(T, dtype=torch.int32, device="cuda")
    bounds = s["bounds"].double()
    for t, (r, p) in enumerate(zip(s["seqs"].tolist(), s["positions"].tolist())):
        mine = p // page
        n_sel[t] = min(mine + 1, keep)
        every = torch.arange(mine + 1, device="cuda")
        if mine + 1 <= keep:
            sel[t, :, :mine + 1] = every.int()
            continue
        q = s["q"][t].double().view(hkv, G, D)
        code = torch.round(q / torch.exp2(_exact_exponent(q.abs().amax((1, 2))))[:, None, None])
        b = bounds[s["table"][r, :mine + 1].long()].transpose(0, 1)       # [hkv, pages, 2, D]
        # the larger of the products with the two bounds
        sc = torch.where(code[:, :, None] > 0, code[:, :, None] * b[:, None, :, 0],
                         code[:, :, None] * b[:, None, :, 1]).sum(-1).amax(1)
        forced = (every < s["first"]) | (every > mine - s["recent"])
        room = keep - int(forced.sum())
        sc[:, forced] = -math.inf
        cut = torch.topk(sc, room, dim=1).values[:, -1:] if room else torch.full((hkv, 1), math.inf, device="cuda")
        above, equal = (sc > cut) & ~forced, (sc == cut) & ~forced
        spare = room - above.sum(1, keepdim=True)
        take = above | forced | (equal & (equal.cumsum(1) <= spare))
        sel[t] = take.nonzero()[:, 1].view(hkv, keep).int()
    return sel, n_sel


def _exact_pages(s):
    G, D, page = s["hq"] // s["hkv"], s["D"], s["page"]
    T, hkv = s["q"].shape[0], s["hkv"]
    out = torch.empty((T, s["hq"], D), dtype=torch.float64, device="cuda")
    for t, (r, p, c) in enumerate(zip(s["seqs"].tolist(), s["positions"].tolist(), s["n_sel"].tolist())):
        at = (s["sel"][t, :, :c].long()[..., None] * page + torch.arange(page, device="cuda")).flatten(1)
        ids, off = s["table"][r].long()[at // page], at % page
        h = torch.arange(hkv, device="cuda")[:, None]
        k, v = s["ck"][ids, h, off].double(), s["cv"][ids, h, off].double()
        w = (s["q"][t].double().view(hkv, G, D) / math.sqrt(D)) @ k.transpose(1, 2)
        w = w.masked_fill((at > p)[:, None], float("-inf"))
        out[t] = (torch.exp(w - torch.logsumexp(w, dim=-1, keepdim=True)) @ v).view(s["hq"], D)
    return out
