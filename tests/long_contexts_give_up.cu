// The long-context attention kernels with a stretch of the cache whose loads are left out: the waits for them run out, and the
// kernels have to report that and end.  SHARED selects sffn_attn_shared's source.  Built together with the library's other
// objects, so that the calls are the library's own.
#include "tma_warp.cuh"

namespace sffn {
namespace {

// Loads of 8-row groups [first, end) of the cache (key head by key head of a page) are left out; in fp32 by addresses.
struct LeftOut {
    int first, end;
    const char *from[2], *to[2];
};
__device__ LeftOut g_left_out;

}  // namespace

SFFN_DEV void some_bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    const char *p = static_cast<const char *>(src);
    for (int i = 0; i < 2; ++i)
        if (p >= g_left_out.from[i] && p < g_left_out.to[i]) return;
    bulk_load(dst, src, bytes, bar, policy);
}

namespace tc {
SFFN_DEV bool left_out(int u) { return u >= g_left_out.first && u < g_left_out.end; }
SFFN_DEV void some_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int u, uint64_t *bar, uint64_t policy) {
    if (!left_out(u)) tma_load_4d(dst, map, x, y, z, u, bar, policy);
}
SFFN_DEV void some_load_rows_warp(uint32_t dst, const CUtensorMap *map, int u, uint32_t bar, uint64_t policy) {
    if (!left_out(__shfl_sync(0xffffffffu, u, 0))) tma_load_rows_warp(dst, map, u, bar, policy);
}
}  // namespace tc
}  // namespace sffn

#define bulk_load some_bulk_load
#define tma_load_4d some_load_4d
#define tma_load_rows_warp some_load_rows_warp
#ifdef SHARED
#include "attn_shared.cu"
#define LEAVE_OUT leave_out_shared
#else
#include "attn_pages.cu"
#define LEAVE_OUT leave_out_pages
#endif

// Of key head h of page pg, all positions (pg < 0: nothing is left out); sizes in bytes of a position and head.
extern "C" int LEAVE_OUT(const void *k, const void *v, int pg, int h, int n_kv_heads, int page, int row_bytes) {
    sffn::LeftOut l = {};
    if (pg >= 0) {
        const long long at = ((long long)pg * n_kv_heads + h) * page;
        l.first = (int)(at / 8), l.end = (int)((at + page) / 8);
        for (int i = 0; i < 2; ++i) {
            l.from[i] = static_cast<const char *>(i ? v : k) + at * row_bytes;
            l.to[i] = l.from[i] + (long long)page * row_bytes;
        }
    }
    return (int)cudaMemcpyToSymbol(sffn::g_left_out, &l, sizeof(l));
}
