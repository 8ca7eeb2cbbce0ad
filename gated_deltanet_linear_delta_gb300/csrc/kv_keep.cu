// kv_keep.cu -- the cache rows of a tree's accepted path, moved to the positions right after the context.
//
// With base = kv_lens[n] - T_n, row base + path[i] becomes row base + i. A path's nodes are in increasing order, so
// path[i] >= i, and a thread that takes one 16-byte column of all the path's rows, in order, reads each row before
// anything is stored over it: the move is in place, without a scratch copy and without a meeting of threads.
#include <algorithm>

#include "kv_pages.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kKeepThreads = 128;
constexpr int kKeepFlight = 8;  // rows in flight per thread

template <typename V>
__device__ __forceinline__ void move_column(V *pool, const long *to, const long *from, int count, long stride, long at) {
    for (int i0 = 0; i0 < count; i0 += kKeepFlight) {
        V x[kKeepFlight];
        bool go[kKeepFlight];
#pragma unroll
        for (int f = 0; f < kKeepFlight; ++f) {
            const int i = i0 + f;
            go[f] = i < count && to[i] >= 0 && from[i] >= 0 && to[i] != from[i];
            if (go[f]) x[f] = pool[from[i] * stride + at];
        }
#pragma unroll
        for (int f = 0; f < kKeepFlight; ++f)
            if (go[f]) pool[to[i0 + f] * stride + at] = x[f];
    }
}

__global__ void __launch_bounds__(kKeepThreads) kv_keep_kernel(const KeepArgs a, int row_pieces, bool scales) {
    __shared__ long to[kTreeMax], from[kTreeMax];  // pool rows of head 0
    KvPages p = a.pg;
    const int n = blockIdx.x, tid = threadIdx.x;
    next_may_begin();
    before_reading();
    if (p.cu) p.Ttot = p.cu[p.B];  // (the host does not say)
    SeqInfo s;
    if (!seq_info<true>(p, n, &s)) return;
    const int count = a.counts[n], base = s.len - s.T;
    bool bad = count < 0 || count > min(s.T, a.path_stride);
    if (!bad && tid < count && base >= 0) {
        const int32_t *path = a.path + (long)n * a.path_stride;
        const int u = path[tid];
        bad = u >= s.T || (tid == 0 ? u < 0 : u <= path[tid - 1]);
        if (!bad) {
            auto pool_row = [&](int pos) -> long {
                const long pg = pool_page(p, n, pos / p.page_size);
                return pg < 0 ? -1 : pg * p.Hkv * p.page_size + pos % p.page_size;
            };
            from[tid] = pool_row(base + u);
            to[tid] = u == tid ? from[tid] : pool_row(base + tid);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) flag_error(p.status);
        return;
    }
    if (base < 0) return;  // an idle row of the batch
    // columns of 16 bytes of all heads' keys, then values, then the scales
    const int c = blockIdx.y * kKeepThreads + tid, per = p.Hkv * row_pieces;
    if (c < 2 * per) {
        const int r = c % per, h = r / row_pieces;
        move_column((uint4 *)(c < per ? a.k_cache : a.v_cache), to, from, count, row_pieces,
                    (long)h * p.page_size * row_pieces + r % row_pieces);
    } else if (scales && c < 2 * per + 2 * p.Hkv) {
        const int r = c - 2 * per;
        move_column(r < p.Hkv ? a.k_scale : a.v_scale, to, from, count, 1, (long)(r % p.Hkv) * p.page_size);
    }
}

}  // namespace

cudaError_t launch_kv_keep(const KeepArgs &a, cudaStream_t s) {
    const int elem = a.pg.cache_dtype == GDN_BF16 ? 2 : a.pg.cache_dtype == GDN_F32 ? 4 : 1;
    const int pieces = a.pg.d * elem / 16;
    const bool scales = elem == 1;
    const long columns = 2L * a.pg.Hkv * (pieces + (scales ? 1 : 0));
    const dim3 grid((unsigned)a.pg.B, (unsigned)((columns + kKeepThreads - 1) / kKeepThreads));
    if (grid.y > 65535) return cudaErrorInvalidConfiguration;
    return launch_early(kv_keep_kernel, grid, kKeepThreads, 0, s, a, pieces, scales);
}

}  // namespace gdn
