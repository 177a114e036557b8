"""sffn_attn_shared with groups that are not ranges one after the other: every sequence is skipped and recorded."""
from __future__ import annotations

import pytest
import torch

from tests.test_attention import Paged, S  # noqa: F401  (S: the library)
from tests.test_long_contexts import call_shared, i32, share

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,hq", [([3, 2, 2, 1], 4), ([60, 64, 50, 64], 8)])
def test_groups_that_overlap(S, n, hq, dt):  # noqa: F811
    p = Paged(S, [70, 64, 66, 80], n, hq, 2, 64, 16, dt, 1)
    share(p, [4], [64], 16)
    T = sum(n)
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, T, 4, hq, 2, 64)
    good = call_shared(S, p, [4], [64], workspace=ws)
    p.check(good)
    q, table = p.q.cuda(), p.table.cuda()
    mask = torch.tensor([m - (1 << 64) if m >> 63 else m for m in p.masks], dtype=torch.int64).cuda()

    def call(groups, prefixes):
        out = torch.full_like(good, 9.0)
        S.attn_shared(q, p.cache, table, i32(p.ctx), p.cu.cuda(), i32(groups), i32(prefixes), mask, out=out, workspace=ws)
        return out

    for groups in ([0, 3, 1, 4], [0, 4, 0, 4], [0, 4, 2], [2, 0, 4], [4, 0], [0, 4, 4, 3, 4], [0, 2 ** 31 - 1, 0, 4],
                   [0, 2, -(2 ** 31), 2, 4]):
        out = call(groups, [64] * (len(groups) - 1))
        assert S.read_device_error(ws) == S.ERR_DEVICE and S.read_device_error(ws) == 0, groups
        assert (out == 9).all(), groups
    for groups in ([0, 0, 4, 4, 4], [0, 1, 1, 3, 4]):  # empty groups are fine
        p.check(call(groups, [64] * (len(groups) - 1)))
        assert S.read_device_error(ws) == 0
