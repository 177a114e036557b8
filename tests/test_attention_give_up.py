"""The tensor-core attention kernels when something that they wait for never comes: the loading warp leaves
out one load (attention_give_up.cu), the wait for it runs out after its two seconds, and the kernel records
SFFN_ERR_TIMEOUT and ends, wherever its other warps are: inside an item, between two items, or writing a
finished one.  Nothing is written outside the output, and the next call is correct."""
from __future__ import annotations

import ctypes as C
import os
import subprocess
import time

import pytest
import torch

from activation_sparse_ffn_gemv_gb300 import build as B
from tests.test_attention import Paged, S, prompt_inputs  # noqa: F401  (S: the library)

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", params=["packed", "paged"])
def lib(request, S, tmp_path_factory):  # noqa: F811
    out = str(tmp_path_factory.mktemp("give_up") / f"{request.param}.so")
    cmd = [B.nvcc(), *B.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-shared", "-Xcompiler", "-fPIC", "-I", B.CSRC, "-I",
           os.path.join(B.ROOT, "include"), os.path.join(HERE, "attention_give_up.cu"), "-o", out, S.LIB_PATH, "-Xlinker",
           "-rpath=" + B.OUT_DIR] + (["-DPAGED"] if request.param == "paged" else [])
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return request.param, C.CDLL(out).run_leaving_out


def stream():
    return C.c_void_p(torch.cuda.current_stream().cuda_stream)


def ptr(t):
    return C.c_void_p(t.data_ptr())


def timed_out(S, ws, call):  # noqa: F811
    torch.cuda.synchronize()
    t0 = time.monotonic()
    assert call() == 0
    torch.cuda.synchronize()
    took = time.monotonic() - t0
    assert S.read_device_error(ws) == S.ERR_TIMEOUT and S.read_device_error(ws) == 0
    assert 1.5 < took < 10.0, took  # two seconds of waiting, one more for the copies in flight, loading the module


# which load of each CTA: the first K, the first V, one inside an item, one of a later item, one that only
# the fullest CTAs get to
@pytest.mark.parametrize("skip", [0, 1, 4, 9, 17])
def test_a_load_that_never_comes_ends_the_kernel(S, lib, skip):  # noqa: F811
    kind, run = lib
    hq, hkv, D = 8, 4, 128
    if kind == "packed":
        lens = [300, 520, 77, 9] * 16
        qkv, cu = prompt_inputs(lens, hq, hkv, D, 3)
        q, k, v = (t.contiguous().cuda() for t in (qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]))
        cu, T = cu.cuda(), sum(lens)
        ws = S.alloc_attn_workspace(S.WS_ATTN_PROMPT, T, len(lens), hq, hkv, D)
        want = S.attn_prompt(q, k, v, cu, workspace=ws)
        out = torch.full((T + 512, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        timed_out(S, ws, lambda: run(ptr(q), ptr(k), ptr(v), T, hq, hkv, ptr(cu), len(lens), C.c_float(D ** -0.5),
                                     ptr(out[256:]), ptr(ws), skip, stream()))
        assert torch.equal(S.attn_prompt(q, k, v, cu, workspace=ws), want)
    else:
        ctx, n = [3000, 70, 1500, 4] * 8, [3, 1, 30, 40] * 8
        p = Paged(S, ctx, n, hq, hkv, D, 16, "bf16", 3, fill=0.0)
        T = sum(n)
        ws = S.alloc_attn_workspace(S.WS_ATTN_TREE, T, len(n), hq, hkv, D)
        want = p.call(S, masks=None, workspace=ws)
        q, table, c, cu = p.q.contiguous().cuda(), p.table.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), p.cu.cuda()
        out = torch.full((T + 512, hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
        timed_out(S, ws, lambda: run(ptr(q), ptr(p.ck), ptr(p.cv), T, hq, hkv, 4, p.cache.n_pages, ptr(table),
                                     table.shape[1], ptr(c), ptr(cu), len(n), C.c_float(D ** -0.5), ptr(out[256:]),
                                     ptr(ws[256:]), ptr(ws), skip, stream()))
        assert torch.equal(p.call(S, masks=None, workspace=ws), want)
    assert S.read_device_error(ws) == 0
    assert (out[:256] == 9).all() and (out[T + 256:] == 9).all()
