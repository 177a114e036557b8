"""The long-context attention kernels when something that they wait for never comes: the loads of one page's keys and values of a
key head are left out (long_contexts_give_up.cu), the waits for them run out, and the call records SFFN_ERR_TIMEOUT and ends.
Nothing is written outside the output, and the next call is correct.

A few-row warp waits one second, and one more for all copies that it has in flight; the tensor-core kernels' warps two and one."""
from __future__ import annotations

import concurrent.futures as cf
import ctypes as C
import os
import subprocess
import time

import pytest
import torch

from activation_sparse_ffn_gemv_gb300 import build as B
from tests.test_attention import Paged, S, dtype_of  # noqa: F401  (S: the library)
from tests.test_long_contexts import Tokens, call_shared, i32, share

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def hurt(S, tmp_path_factory):  # noqa: F811
    """The library with the two sources in their changed form, bound as the binding binds the library."""
    d = str(tmp_path_factory.mktemp("give_up"))
    changed = ["attn_shared", "attn_pages"]

    def compile_(name):
        out = os.path.join(d, name + ".o")
        cmd = [B.nvcc(), *B.ARCH, "-O3", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-I", B.CSRC, "-I",
               os.path.join(B.ROOT, "include"), "-c", os.path.join(HERE, "long_contexts_give_up.cu"), "-o", out]
        r = subprocess.run(cmd + (["-DSHARED"] if name == "attn_shared" else []), capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return out

    with cf.ThreadPoolExecutor() as ex:
        objs = list(ex.map(compile_, changed))
    others = [os.path.join(B.OUT_DIR, os.path.splitext(s)[0] + ".o") for s in B.SOURCES]
    objs += [o for o in others if os.path.splitext(os.path.basename(o))[0] not in changed]
    lib = os.path.join(d, "libhurt.so")
    r = subprocess.run([B.nvcc(), *B.ARCH, "-shared", "-o", lib, *objs, "-lcudart"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    mine, path, S._lib, S.LIB_PATH = S._lib, S.LIB_PATH, None, lib
    try:
        bound = S.lib()
    finally:
        S._lib, S.LIB_PATH = mine, path
    return bound


def check(S, hurt, monkeypatch, which, cache, pg, h, ws, T, hq, D, td, call, least, most):  # noqa: F811
    """call(out=...) by the library, by the changed one without the page's loads, and by the library again."""
    want = call(out=torch.empty(T, hq, D, dtype=td, device="cuda"))
    assert S.read_device_error(ws) == 0
    leave = getattr(hurt, "leave_out_" + which)

    def left(page):
        assert leave(C.c_void_p(cache.k.data_ptr()), C.c_void_p(cache.v.data_ptr()), page, h, cache.n_kv_heads, cache.page_size,
                     D * td.itemsize) == 0

    room = torch.full((T + 256, hq, D), 9.0, dtype=td, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(S, "_lib", hurt)
        left(-1)
        assert torch.equal(call(out=room[128:T + 128]), want)  # nothing left out: the library's result
        room.fill_(9.0)
        left(pg)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        call(out=room[128:T + 128])
        torch.cuda.synchronize()
        took = time.monotonic() - t0
        assert S.read_device_error(ws) == S.ERR_TIMEOUT and S.read_device_error(ws) == 0
        left(-1)
    assert least < took < most, took
    assert (room[:128] == 9).all() and (room[T + 128:] == 9).all()
    assert torch.equal(call(out=room[128:T + 128]), want) and S.read_device_error(ws) == 0


FEW, TENSOR = (0.8, 2.9), (1.8, 4.0)


@pytest.mark.parametrize("lens,at,hq,hkv,D,page,dt,room,seconds", [
    ([900, 300] * 8, [[899], [299]] * 8, 8, 2, 128, 64, "bf16", 0, FEW),
    ([900, 300] * 8, [[899], [299]] * 8, 16, 2, 64, 128, "bf16", 0, FEW),
    ([900, 300] * 8, [[899], [299]] * 8, 8, 2, 128, 8, "bf16", 0, FEW),
    ([900, 300] * 8, [[899], [299]] * 8, 8, 2, 128, 32, "f32", 0, FEW),
    ([900, 300] * 8, [[899], [299]] * 8, 4, 2, 64, 64, "f32", 0, FEW),
    ([900, 700], [list(range(600, 900)), list(range(640, 700))], 8, 2, 128, 32, "bf16", 4096, TENSOR),
    ([900, 700], [list(range(600, 900)), list(range(640, 700))], 8, 2, 64, 256, "bf16", 4096, TENSOR),
])
@pytest.mark.parametrize("late", [False, True])
def test_attn_pages(S, hurt, monkeypatch, lens, at, hq, hkv, D, page, dt, room, seconds, late):  # noqa: F811
    c = Tokens(S, lens, at, hq, hkv, D, page, dt, 3, fill=0.0)
    T, keep = len(c.pos), max(lens) // page + 1
    sel, n_sel = c.select(S, keep)  # every page
    sel = torch.nn.functional.pad(sel, (0, max(room, keep) - keep), value=-1)
    ws = S.alloc_attn_workspace(S.WS_ATTN_PAGES, T, len(lens), hq, hkv, D)
    pg = int(c.table[0, c.pos[0] // page - 1 if late else 0])
    check(S, hurt, monkeypatch, "pages", c.cache, pg, 1, ws, T, hq, D, dtype_of(dt),
          lambda out: c.attend(S, sel, n_sel, out=out, workspace=ws), *seconds)


@pytest.mark.parametrize("n,hq,hkv,D,page,dt,seconds", [
    ([1, 1, 1, 1], 8, 8, 128, 16, "bf16", FEW),                # few-row warps for all
    ([1, 1, 1, 1], 8, 8, 64, 64, "f32", FEW),
    ([1] * 20, 16, 2, 128, 64, "bf16", TENSOR),                # the prefix on the tensor cores beside them
    ([40, 64, 33, 50], 8, 2, 64, 32, "bf16", TENSOR),          # all on the tensor cores
    ([7, 9, 5, 3], 8, 2, 128, 16, "bf16", TENSOR),
])
@pytest.mark.parametrize("part", ["prefix", "own"])
def test_attn_shared(S, hurt, monkeypatch, n, hq, hkv, D, page, dt, seconds, part):  # noqa: F811
    prefix = 640
    p = Paged(S, [prefix + 150 + 31 * i for i in range(len(n))], n, hq, hkv, D, page, dt, 5, fill=0.0)
    share(p, [len(n)], [prefix], page)
    if part == "own" and hq // hkv * sum(n) <= 16 * len(n):
        seconds = FEW
    T = sum(n)
    ws = S.alloc_attn_workspace(S.WS_ATTN_SHARED, T, len(n), hq, hkv, D)
    pg = int(p.table[0, prefix // page + (1 if part == "own" else -2)])
    check(S, hurt, monkeypatch, "shared", p.cache, pg, 1, ws, T, hq, D, dtype_of(dt),
          lambda out: call_shared(S, p, [len(n)], [prefix], out=out, workspace=ws), *seconds)
