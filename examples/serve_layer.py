"""One transformer layer served with this package: a packed prefill, then a step of drafted tokens.

Prefill (two prompts packed together): fused projection -> head norms, rotation and the cache's new
rows (qk_norm_rope) -> causal attention (attn_prompt) -> output projection -> the tokens whose
attention output carries the mass (token_select) -> the FFN on those (prefill).

Decode: three drafted tokens of the first prompt (a tree: two continuations of one token) and the next token of
the second -> qk_norm_rope into the cache -> attn_tree over the pages -> output projection ->
the sparse FFN (decode).

The plain products (projections) are torch matmuls; everything else runs in the library.  Run it on
a GPU with the library built:  python examples/serve_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from activation_sparse_ffn_gemv_gb300 import sffn  # noqa: E402
from activation_sparse_ffn_gemv_gb300 import workloads as W  # noqa: E402


class Layer:
    """Weights of a layer: d_model 1024, 8 query and 2 key heads of 128, SwiGLU FFN of 2816."""

    def __init__(self, seed: int = 0):
        self.d, self.hq, self.hkv, self.D, self.page = 1024, 8, 2, 128, 16
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()

        self.w_qkv = normal(self.d, (self.hq + 2 * self.hkv) * self.D, std=self.d ** -0.5)
        self.w_o = normal(self.hq * self.D, self.d, std=(self.hq * self.D) ** -0.5)
        self.q_norm, self.k_norm = (1 + normal(self.D, std=0.1) for _ in range(2))
        self.table = sffn.rope_table(4096, self.D)
        ffn = W.make_ffn_layer(5, seed=seed, device="cuda", d_model=self.d, d_ff=2816)
        self.ffn = sffn.Weights(ffn)
        self.ffn.set_down_norms(sffn.down_norms(self.ffn))

    def qkv(self, x):
        """Views of the fused projection's rows: q [T, hq, D], k and v [T, hkv, D]."""
        rows = (x @ self.w_qkv).view(x.shape[0], self.hq + 2 * self.hkv, self.D)
        return rows[:, :self.hq], rows[:, self.hq:self.hq + self.hkv], rows[:, self.hq + self.hkv:]


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def run(seed: int = 0) -> dict:
    layer = Layer(seed)
    page, D = layer.page, layer.D
    lens, n_pages, width = [300, 77], 40, 24
    T = sum(lens)
    shape = (n_pages, layer.hkv, page, D)
    cache = sffn.KVCache(torch.empty(shape, dtype=torch.bfloat16, device="cuda"),
                         torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
    # pages dealt to the two sequences alternately
    table = torch.zeros(2, width, dtype=torch.int32)
    for i in range(2):
        table[i, :20] = torch.arange(20, dtype=torch.int32) * 2 + i

    def slot(seq, pos):
        return int(table[seq, pos // page]) * page + pos % page

    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn(T, layer.d, generator=g, device="cuda").bfloat16()

    # ---- prefill ----
    pos = [p for n in lens for p in range(n)]
    slots = i32([slot(s, p) for s, n in enumerate(lens) for p in range(n)])
    q, k, v = layer.qkv(x)
    q, k = sffn.qk_norm_rope(q, k, v, layer.table, i32(pos), q_weight=layer.q_norm, k_weight=layer.k_norm, cache=cache,
                             slots=slots, k_out=torch.empty_like(k, memory_format=torch.contiguous_format))
    att = sffn.attn_prompt(q, k, v, i32([0, lens[0], T]))
    y_attn = att.view(T, -1) @ layer.w_o
    sel, n_sel = sffn.token_select(y_attn, 0.5, 16, 1)
    out = sffn.prefill(x, y_attn, layer.ffn, sel, n_sel)

    # ---- a decode step: tokens 0 and its two continuations 1, 2 for the first sequence, one for the second ----
    new, ctx = [3, 1], i32(lens)
    xd = torch.randn(4, layer.d, generator=g, device="cuda").bfloat16()
    depth = [0, 1, 1, 0]                       # position after the context: siblings share theirs
    place = [(0, 0), (0, 1), (0, 2), (1, 0)]   # where each token's key lies: its number among the new ones
    mask = torch.tensor([0b001, 0b011, 0b101, 0b1], dtype=torch.int64, device="cuda")
    q, k, v = layer.qkv(xd)
    q, _ = sffn.qk_norm_rope(q, k, v, layer.table, i32([lens[s] + d for (s, _), d in zip(place, depth)]),
                             q_weight=layer.q_norm, k_weight=layer.k_norm, cache=cache,
                             slots=i32([slot(s, lens[s] + j) for s, j in place]))
    datt = sffn.attn_tree(q, cache, table.cuda(), ctx, i32([0, new[0], sum(new)]), mask)
    yd = (xd + datt.view(4, -1) @ layer.w_o).contiguous()
    tau = float(sffn.gate_scores(yd, layer.ffn).flatten().quantile(0.8))
    ffn_out, _, n_active = sffn.decode(yd, layer.ffn, sffn.MODE_THRESHOLD, sffn.SCORE_GATE, tau)

    # the same four tokens as prompts of their own, for comparison: each branch after its context
    both = []
    for branch in ([0, 1], [0, 2], [3]):
        s = 0 if branch[0] == 0 else 1
        a = sum(lens[:s])
        xs = torch.cat([x[a:a + lens[s]], xd[branch]])
        qb, kb, vb = layer.qkv(xs)
        qb, kb = sffn.qk_norm_rope(qb, kb, None, layer.table, i32(list(range(len(xs)))), q_weight=layer.q_norm,
                                   k_weight=layer.k_norm)
        both.append(sffn.attn_prompt(qb, kb, vb, i32([0, len(xs)]))[-1])
    return dict(prefill=out, n_sel=int(n_sel.item()), tokens=T, decode_attention=datt, decode=ffn_out,
                n_active=n_active.tolist(), d_ff=layer.ffn.d_ff, as_prompts=torch.stack(both))


if __name__ == "__main__":
    r = run()
    print(f"prefill: FFN on {r['n_sel']} of {r['tokens']} tokens, output {tuple(r['prefill'].shape)}")
    print(f"decode: active neurons {r['n_active']} of {r['d_ff']}, output {tuple(r['decode'].shape)}")
    d = (r["decode_attention"][[1, 2, 3]].float() - r["as_prompts"].float()).abs().max().item()
    print(f"drafted tokens' attention against the same tokens as prompts: largest difference {d:.2e}")
