"""sffn_attn_shared's kernels have no tile size of sffn_attn_tree's to divide by (it is zero in such a call): the
arguments that both share hold none, and so does what checks a sequence's numbers for both."""
from __future__ import annotations

import os
import subprocess

from activation_sparse_ffn_gemv_gb300 import build as B

SOURCE = """
#include "attn.cuh"
#include <type_traits>
using namespace sffn;
template <typename A, typename = void> struct Has : std::false_type {};
template <typename A> struct Has<A, std::void_t<decltype(A::tile_tokens)>> : std::true_type {};
static_assert(Has<TreeArgs>::value && !Has<SeqArgs>::value && !Has<SharedArgs>::value);
__global__ void k(SharedArgs a, SeqTokens *q) { *q = seq_tokens(a, 0, true); }
"""


def test_shared_calls_have_no_tile_size_of_the_tree_calls(tmp_path):
    src = tmp_path / "arguments.cu"
    src.write_text(SOURCE)
    r = subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "--expt-relaxed-constexpr", "-I", B.CSRC, "-I",
                        os.path.join(B.ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "arguments.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
