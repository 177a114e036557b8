"""The attention half of a layer whose FFN this package computes: per-head norms with the
position rotation (``qk_norm_rope``), attention over packed prompts (``attn_prompt``) and
attention of drafted tokens, or of the single next token, over a paged cache (``attn_tree``).

Each case is run either in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or through the package's own calls.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _text(values):
    return ",".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split(",")]


def listed():
    return [
        # one decoded token of a multi-head model (d_model 4096 = 32 x 128), keys and values go
        # straight to the cache; no head norms: the smallest call of a decode loop
        dict(name="rope-token", op="rope", T=1, hq=32, hkv=32, D=128, dtype="bf16", norm=False,
             style="half", rot=128, page=16, k_out=False),
        # a batch's drafted tokens in fp32 (the fp32 decode path), short heads, interleaved pairs
        # and only half of each head rotated; an odd number of tokens
        dict(name="rope-drafts-f32", op="rope", T=61, hq=16, hkv=2, D=64, dtype="f32", norm=True,
             style="interleaved", rot=32, page=32, k_out=False),
        # a whole prompt of the prefill length: rotated keys are needed packed (for the prompt's
        # attention) and in the cache (for the decode that follows)
        dict(name="rope-prompt", op="rope", T=16384, hq=64, hkv=8, D=128, dtype="bf16", norm=True,
             style="half", rot=128, page=64, k_out=True),
        # short chat turns packed together, one of them empty: latency counts
        dict(name="prompt-short", op="prompt", lens="1,17,130,0,44", hq=16, hkv=2, D=128),
        # ragged packed prompts of a server's batch, seven query heads for each key head
        dict(name="prompt-packed", op="prompt",
             lens="911,33,2047,128,640,1500,257,64,1201,5,777,129,383", hq=28, hkv=4, D=128),
        # one medium multi-head prompt with short heads next to an odd one
        dict(name="prompt-d64", op="prompt", lens="2048,1777,1", hq=32, hkv=32, D=64),
        # the prefill workload's length as one prompt
        dict(name="prompt-long", op="prompt", lens="16384", hq=64, hkv=8, D=128),
        # one token over a short multi-head context: the smallest decode call
        dict(name="tree-token", op="tree", ctx="300", n="1", hq=32, hkv=32, D=128, dtype="bf16", page=16),
        # a decode step of a batch of ragged sequences, one token each, one of them at its first token
        dict(name="tree-batch-token", op="tree", ctx=_text([0, 17, 64, 4095, 1000, 2500, 3777, 801] * 6),
             n=_text([1] * 48), hq=32, hkv=8, D=128, dtype="bf16", page=16),
        # eight drafted tokens (the most one FFN decode call takes) over a long context
        dict(name="tree-long", op="tree", ctx="65531", n="8", hq=64, hkv=8, D=128, dtype="bf16", page=64),
        # large draft trees of a batch, seven query heads for each key head, lengths that end inside a page
        dict(name="tree-batch-drafts", op="tree", ctx=_text([4001, 130, 7777, 5000, 12000, 63, 2222, 9001] * 4),
             n=_text([64, 25, 33, 60, 17, 64, 1, 48] * 4), hq=28, hkv=4, D=128, dtype="bf16", page=128),
        # the fp32 decode path: a few sequences with small trees
        dict(name="tree-f32", op="tree", ctx="1999,300,4000,0", n="8,5,1,7", hq=16, hkv=2, D=64,
             dtype="f32", page=32),
    ]


_HEADS = [(32, 32), (16, 2), (64, 8), (28, 4), (40, 8), (32, 8), (5, 1), (12, 12), (20, 20)]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "tree"])
    hq, hkv = rng.choice(_HEADS)
    D = rng.choice([64, 128])
    if op == "rope":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        T = _log(rng, 1, 16384 if dtype == "bf16" else 2048)
        return dict(op="rope", T=T, hq=hq, hkv=hkv, D=D, dtype=dtype, norm=rng.random() < 0.7,
                    style=rng.choice(["half", "interleaved"]), rot=rng.choice([D, D, D // 2]),
                    page=rng.choice([16, 32, 64, 128, 256]), k_out=rng.random() < 0.5)
    if op == "prompt":
        total = _log(rng, 2, 8192)
        n_seq = rng.randint(1, min(total, 16))
        cuts = sorted(rng.randint(0, total) for _ in range(n_seq - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return dict(op="prompt", lens=_text(lens), hq=hq, hkv=hkv, D=D)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    n_seq = _log(rng, 1, 48)
    nmax = rng.choice([1, 1, 8, 64])
    # cached positions x key heads x head size: within the large draft-tree case's
    budget = (80_000_000 if dtype == "bf16" else 16_000_000) // (hkv * D)
    top = max(2, min(65536, budget // n_seq))
    ctx = [_log(rng, 1, top) - 1 for _ in range(n_seq)]
    n = [rng.randint(1, nmax) for _ in range(n_seq)]
    return dict(op="tree", ctx=_text(ctx), n=_text(n), hq=hq, hkv=hkv, D=D, dtype=dtype,
                page=rng.choice([16, 32, 64, 128, 256]))


def work(case):
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    if case["op"] == "rope":
        T, es = case["T"], _ES[case["dtype"]]
        k_writes = 2 if case["k_out"] else 1
        elems = T * D * (2 * hq + (1 + k_writes) * hkv + 2 * hkv)  # q, k in and out; v into the cache
        small = T * (4 + 4 + 4 * case["rot"])                      # position, slot, table row
        return {"bytes": elems * es + small, "flops": 8 * T * D * (hq + hkv)}
    if case["op"] == "prompt":
        lens = _ints(case["lens"])
        T = sum(lens)
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * T * D * (2 * hq + 2 * hkv), "flops": 4 * pairs * hq * D}
    es = _ES[case["dtype"]]
    ctx, new = _ints(case["ctx"]), _ints(case["n"])
    T, keys = sum(new), sum(ctx) + sum(new)
    pairs = sum((c + n) * n for c, n in zip(ctx, new))
    return {"bytes": es * (keys * hkv * D * 2 + 2 * T * hq * D), "flops": 4 * pairs * hq * D}


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


def _table(max_pos, rot):
    """cos | sin of every position, made once in 64 bits and kept by the program."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv[None, :]
    return torch.cat([ang.cos(), ang.sin()], dim=1).float().cuda()


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


def prepare(case, seed):
    g = _gen(seed)
    hq, hkv, D = case["hq"], case["hkv"], case["D"]
    s = dict(case)
    s["scale"] = 1.0 / math.sqrt(D)
    for key in ("lens", "ctx", "n"):
        if key in case:
            s[key] = _ints(case[key])
    if case["op"] == "rope":
        T, dt, page = case["T"], _DT[case["dtype"]], case["page"]
        qkv = _randn((T, hq + 2 * hkv, D), g, dt, 1.7)  # one fused projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"] = (1.0 + 0.2 * _randn((D,), g, torch.float32)).to(dt)
            s["wk"] = (1.0 + 0.2 * _randn((D,), g, torch.float32)).to(dt)
        max_pos = max(T, 4096)
        s["table"] = _table(max_pos, case["rot"])
        s["pos"] = torch.randint(0, max_pos, (T,), generator=g, device="cuda").int()
        n_pages = (T + page - 1) // page + 3
        s["slots"] = torch.randperm(n_pages * page, generator=g, device="cuda")[:T].int()
        if T > 256:  # a prompt: its positions in order, its pages scattered, in order inside each
            s["pos"] = torch.arange(T, device="cuda").int()
            pages = torch.randperm(n_pages, generator=g, device="cuda")
            t = torch.arange(T, device="cuda")
            s["slots"] = (pages[t // page] * page + t % page).int()
        s["ck"] = torch.zeros((n_pages, hkv, page, D), dtype=dt, device="cuda")
        s["cv"] = torch.zeros_like(s["ck"])
    elif case["op"] == "prompt":
        T = sum(s["lens"])
        qkv = _randn((T, hq + 2 * hkv, D), g, torch.bfloat16, 1.25)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["cu"] = _i32(_offsets(s["lens"]))
    else:
        dt, page = _DT[case["dtype"]], case["page"]
        need = [(c + n + page - 1) // page for c, n in zip(s["ctx"], s["n"])]
        n_pages, width = sum(need) + 5, max(need) + 1
        s["ck"] = _randn((n_pages, hkv, page, D), g, dt, 1.25)
        s["cv"] = _randn((n_pages, hkv, page, D), g, dt)
        T = sum(s["n"])
        s["q"] = _randn((T, hq + 2 * hkv, D), g, dt, 1.25)[:, :hq]
        order = torch.randperm(n_pages, generator=g, device="cuda").int().cpu()
        s["pages"] = torch.zeros((len(need), width), dtype=torch.int32)
        for i, (a, m) in enumerate(zip(_offsets(need), need)):
            s["pages"][i, :m] = order[a:a + m]
        s["pages"] = s["pages"].cuda()
        s["ctx_d"] = _i32(s["ctx"])
        s["cu"] = _i32(_offsets(s["n"]))
        gc = torch.Generator()
        gc.manual_seed(int(seed))
        s["mask"] = torch.tensor(sum((_tree_masks(n, gc) for n in s["n"]), []), dtype=torch.int64,
                                 device="cuda")
    if own:
        from activation_sparse_ffn_gemv_gb300 import sffn
        T = s["q"].shape[0]
        which = {"rope": sffn.WS_QK_NORM_ROPE, "prompt": sffn.WS_ATTN_PROMPT, "tree": sffn.WS_ATTN_TREE}[case["op"]]
        n_seq = 1 if case["op"] == "rope" else s["cu"].numel() - 1
        s["ws"] = sffn.alloc_attn_workspace(which, T, n_seq, hq, hkv, D)
        if "ck" in s:
            s["cache"] = sffn.KVCache(s["ck"], s["cv"])
        s["out"] = torch.empty((T, hq, D), dtype=s["q"].dtype, device="cuda")
        if case["op"] == "rope" and case["k_out"]:
            s["kk"] = torch.empty((T, hkv, D), dtype=s["q"].dtype, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        return {"rope": _own_rope, "prompt": _own_prompt, "tree": _own_tree}[s["op"]](s)
    return {"rope": _plain_rope, "prompt": _plain_prompt, "tree": _plain_tree}[s["op"]](s)


def _own_rope(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    q, k = sffn.qk_norm_rope(s["q"], s["k"], s["v"], s["table"], s["pos"], q_weight=s["wq"], k_weight=s["wk"],
                             eps=EPS, style=sffn.ROPE_HALF if s["style"] == "half" else sffn.ROPE_INTERLEAVED,
                             cache=s["cache"], slots=s["slots"], q_out=s["out"], k_out=s.get("kk"),
                             workspace=s["ws"])
    return [q, s["ck"], s["cv"]] + ([k] if s["k_out"] else [])


def _own_prompt(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.attn_prompt(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], out=s["out"], workspace=s["ws"])


def _own_tree(s):
    from activation_sparse_ffn_gemv_gb300 import sffn
    return sffn.attn_tree(s["q"], s["cache"], s["pages"], s["ctx_d"], s["cu"], s["mask"], scale=s["scale"],
                          out=s["out"], workspace=s["ws"])


def _rotate(x, w, s):
    """RMS norm of each head (when there is a weight) and the rotation, in 32 bits."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()
    rot = s["rot"]
    row = s["table"][s["pos"].long()][:, None, :]
    cos, sin = row[..., : rot // 2], row[..., rot // 2:]
    if s["style"] == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(s):
    dt, page = s["q"].dtype, s["page"]
    q = _rotate(s["q"], s["wq"], s).to(dt)
    k = _rotate(s["k"], s["wk"], s).to(dt)
    at = s["slots"].long()
    s["ck"][at // page, :, at % page] = k
    s["cv"][at // page, :, at % page] = s["v"]
    return [q, s["ck"], s["cv"]] + ([k] if s["k_out"] else [])


def _softmax_av(scores, v):
    m = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - m)
    return torch.matmul(p, v) / p.sum(dim=-1, keepdim=True)


def _plain_prompt(s):
    hq, hkv, D = s["hq"], s["hkv"], s["D"]
    G = hq // hkv
    out = torch.empty((s["q"].shape[0], hq, D), dtype=s["q"].dtype, device="cuda")
    for t0, n in zip(_offsets(s["lens"]), s["lens"]):
        if n == 0:
            continue
        q = s["q"][t0:t0 + n].float() * s["scale"]
        k = s["k"][t0:t0 + n].float().permute(1, 2, 0)  # [hkv, D, n]
        v = s["v"][t0:t0 + n].float().permute(1, 0, 2)
        rows = max(64, min(n, (1 << 28) // (hq * n)))  # scores of a piece: at most 1 GB
        for a in range(0, n, rows):
            b = min(n, a + rows)
            qa = q[a:b].view(b - a, hkv, G, D).permute(1, 2, 0, 3).reshape(hkv, G * (b - a), D)
            sc = torch.matmul(qa, k[:, :, :b]).view(hkv, G, b - a, b)
            i = torch.arange(a, b, device="cuda")[:, None]
            j = torch.arange(b, device="cuda")[None, :]
            sc.masked_fill_(j > i, float("-inf"))
            o = _softmax_av(sc.view(hkv, G * (b - a), b), v[:, :b])
            out[t0 + a:t0 + b] = o.view(hkv, G, b - a, D).permute(2, 0, 1, 3).reshape(b - a, hq, D)
    return out


def _plain_tree(s):
    hq, hkv, D, page = s["hq"], s["hkv"], s["D"], s["page"]
    G = hq // hkv
    out = torch.empty((s["q"].shape[0], hq, D), dtype=s["q"].dtype, device="cuda")
    bit = torch.arange(64, device="cuda")
    for i, (t0, n, c) in enumerate(zip(_offsets(s["n"]), s["n"], s["ctx"])):
        m = (c + n + page - 1) // page
        ids = s["pages"][i, :m].long()
        k = s["ck"][ids].permute(1, 0, 2, 3).reshape(hkv, m * page, D)[:, :c + n].float()
        v = s["cv"][ids].permute(1, 0, 2, 3).reshape(hkv, m * page, D)[:, :c + n].float()
        q = s["q"][t0:t0 + n].float().view(n, hkv, G, D).permute(1, 2, 0, 3).reshape(hkv, G * n, D)
        sc = torch.matmul(q * s["scale"], k.transpose(1, 2)).view(hkv, G, n, c + n)
        sees = ((s["mask"][t0:t0 + n, None] >> bit[None, :n]) & 1).bool()
        sc[..., c:].masked_fill_(~sees, float("-inf"))
        o = _softmax_av(sc.view(hkv, G * n, c + n), v)
        out[t0:t0 + n] = o.view(hkv, G, n, D).permute(2, 0, 1, 3).reshape(n, hq, D)
    return out


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "tree": _exact_tree}[case["op"]](s)


def _exact_rotated(x, w, s):
    """Each rotated pair as a complex number times (cos + i sin) of its position."""
    y = x.double()
    if w is not None:
        rms = (y.pow(2).sum(-1) / s["D"] + EPS).sqrt()
        y = y / rms[..., None] * w.double()
    else:
        y = y.clone()
    half = s["rot"] // 2
    t = s["table"].double()[s["pos"].long()]
    turn = torch.complex(t[:, :half], t[:, half:])[:, None, :]
    if s["style"] == "half":
        z = torch.complex(y[..., :half].clone(), y[..., half:2 * half].clone()) * turn
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:2 * half:2].clone(), y[..., 1:2 * half:2].clone()) * turn
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    return y


def _exact_rope(s):
    q, k = _exact_rotated(s["q"], s["wq"], s), _exact_rotated(s["k"], s["wk"], s)
    n_pages, hkv, page, D = s["ck"].shape
    flat = s["slots"].long()
    ck = s["ck"].double().transpose(1, 2).reshape(n_pages * page, hkv, D)
    cv = s["cv"].double().transpose(1, 2).reshape(n_pages * page, hkv, D)
    ck[flat] = k
    cv[flat] = s["v"].double()

    def paged(c):
        return c.view(n_pages, page, hkv, D).transpose(1, 2).contiguous()

    return [q, paged(ck), paged(cv)] + ([k] if s["k_out"] else [])


def _exact_rows(q, k, v, sees):
    """q [r, D], k and v [n, D] in 64 bits, sees [r, n]."""
    w = (q @ k.T).masked_fill(~sees, float("-inf"))
    return torch.exp(w - torch.logsumexp(w, dim=1, keepdim=True)) @ v


def _exact_prompt(s):
    G, D = s["hq"] // s["hkv"], s["D"]
    out = torch.empty((s["q"].shape[0], s["hq"], D), dtype=torch.float64, device="cuda")
    base = 0
    for n in s["lens"]:
        for h in range(s["hq"]):
            q = s["q"][base:base + n, h].double() / math.sqrt(D)
            k = s["k"][base:base + n, h // G].double()
            v = s["v"][base:base + n, h // G].double()
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                sees = torch.ones((b - a, b), dtype=torch.bool, device="cuda").tril(a)
                out[base + a:base + b, h] = _exact_rows(q[a:b], k[:b], v[:b], sees)
        base += n
    return out


def _exact_tree(s):
    G, D, page = s["hq"] // s["hkv"], s["D"], s["page"]
    out = torch.empty((s["q"].shape[0], s["hq"], D), dtype=torch.float64, device="cuda")
    base = 0
    for i, (c, n) in enumerate(zip(s["ctx"], s["n"])):
        at = torch.arange(c + n, device="cuda")
        ids, off = s["pages"][i].long()[at // page], at % page
        sees = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        for r, word in enumerate(s["mask"][base:base + n].tolist()):
            sees[r, c:] = torch.tensor([(word >> j) & 1 for j in range(n)], dtype=torch.bool)
        for h in range(s["hkv"]):
            k, v = s["ck"][ids, h, off].double(), s["cv"][ids, h, off].double()
            q = s["q"][base:base + n, h * G:(h + 1) * G].double().transpose(0, 1).reshape(G * n, D) / math.sqrt(D)
            o = _exact_rows(q, k, v, sees.repeat(G, 1))
            out[base:base + n, h * G:(h + 1) * G] = o.view(G, n, D).transpose(0, 1)
        base += n
    return out
