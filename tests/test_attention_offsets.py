"""Packed prompts whose offsets break the contract: the sequence is skipped (its rows are not written) and
recorded, and every valid sequence is what it is in a call of its own."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import S, prompt_inputs  # noqa: F401  (S: the library)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cu,valid", [
    ([0, 40, 101, 100], [(0, 40)]),             # past the rows, then backwards
    ([-5, 40, 40, 100], [(40, 100)]),           # before the first row; an empty one
    ([0, 70, 60, 100], [(0, 70), (60, 100)]),   # backwards; the rows that two sequences claim are either's
    ([0, 1 << 30, 100, 100], [(0, 0)]),
    ([-(1 << 31), (1 << 31) - 1, 20, 100], [(20, 100)]),  # a length that does not fit 32 bits
])
def test_bad_offsets(S, D, cu, valid):  # noqa: F811
    hq, hkv, T = 4, 2, 100
    qkv, _ = prompt_inputs([T], hq, hkv, D, 2)
    q, k, v = (t.cuda() for t in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))
    ws = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, T, len(cu) - 1, hq, hkv, D)
    out = torch.full((T, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    S.attn_prompt(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda(), out=out, workspace=ws)
    assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0
    claimed = torch.zeros(T, dtype=torch.int32)
    for a, b in valid:
        claimed[a:b] += 1
    for a, b in valid:
        if a < b:
            own = S.attn_prompt(q[a:b], k[a:b], v[a:b], torch.tensor([0, b - a], dtype=torch.int32).cuda())
            sole = (claimed[a:b] == 1).cuda()
            assert torch.equal(out[a:b][sole], own[sole])
    assert (out[(claimed == 0).cuda()] == 9).all()
