"""The attention calls where a CTA has much to do: several items one after the other, many key tiles of an
item, shared-memory rings that go round and hand over from one item to the next.  References, inputs'
layout and tolerances are test_attention.py's."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import S, gen, check_attention  # noqa: F401  (S: the library)


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
