// attn_simt.cu -- attention over a paged cache on the CUDA cores, in fp32 throughout.
//
// For fp32 inputs, whose results keep fp32's precision (bf16 inputs run on the tensor cores,
// attn_tc.cu). A CTA of 256 threads holds a row tile of Q and walks key tiles of 64 positions: scores by register
// tiles (each thread RT rows x 4 keys), softmax statistics per row by shuffles over the 16
// threads that share it, and the output tile (RT rows x D/16 columns a thread) in registers,
// rescaled when the running maximum grows. It is bound by shared-memory reads (5 to 8 16-byte reads
// per 16 to 64 multiply-adds): correct and steady, but no performance path. 2 x 100 tokens over 1000, 8
// heads on 2, d = 64: 28 us, about 3 key tiles per CTA after the plan and before the joining kernel (two
// CTAs per SM: 37 us).
#include <algorithm>

#include "attn_plan.cuh"
#include "attn_work.h"
#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int BN = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct SimtParams {
    AttnWork w;
    const float *q;
    const void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    float *out;
    int Hq;
    long q_stride;
    float scale2;  // softmax scale * log2 e
};

// 4 elements of a cached row as they are loaded, and dequantised; KIND is GDN_FP8, GDN_INT8 or GDN_F32
template <int KIND>
struct Raw4 {
    uint32_t code;
    float scale;
    template <int D>
    __device__ __forceinline__ void load(const void *cache, const float *scales, long at, int c) {
        code = *reinterpret_cast<const uint32_t *>((const uint8_t *)cache + at * D + c);
        scale = scales[at];
    }
    __device__ __forceinline__ void zero() { code = 0, scale = 0.f; }
    __device__ __forceinline__ float4 get() const {
        float x[4];
        if (KIND == GDN_FP8) decode4_e4m3(code, x);
        else decode4_int8(code, x);
        return make_float4(x[0] * scale, x[1] * scale, x[2] * scale, x[3] * scale);
    }
};
template <>
struct Raw4<GDN_F32> {
    float4 x;
    template <int D>
    __device__ __forceinline__ void load(const void *cache, const float *, long at, int c) {
        x = load4((const float *)cache + at * D + c);
    }
    __device__ __forceinline__ void zero() { x = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float4 get() const { return x; }
};

__device__ __forceinline__ float finite_or_zero(float x) { return fabsf(x) < INFINITY ? x : 0.f; }

template <int D, int R>
struct SimtSmem {
    float q[R][D + 4];
    float k[BN][D + 4];
    float v[BN][D];
    float p[R][BN + 4];
    long at[BN];  // pool row of each key of the tile, or -1
    PlanSmem plan;
};

template <int KIND, int D, int R, bool TREE>
__global__ void __launch_bounds__(kThreads) attn_simt_kernel(const SimtParams a) {
    constexpr int RT = R / 16, CT = D / 64;  // rows and groups of 4 columns per thread
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimtSmem<D, R> &sm = *reinterpret_cast<SimtSmem<D, R> *>(smem_raw);
    const AttnWork &w = a.w;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    next_may_begin();
    before_reading();
    plan_piece<BN, kThreads, TREE>(w, &sm.plan);
    if (sm.plan.padding) zero_padding<TREE>(w, a.out, a.Hq, D, tid, kThreads);
    Piece pc = sm.plan.piece;
    bool begun = pc.off == 0, careful = false;
    while (pc.left > 0) {
        const int t0 = pc.i * w.TPT, rows = min(w.TPT, pc.s.T - t0) * w.G;
        const int off = pc.off, take = (int)min((long)(pc.ntiles - off), pc.left);
        __syncthreads();
        for (int e = tid; e < R * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                x = load4(a.q + (pc.s.bos + t0 + r / w.G) * a.q_stride + (long)(pc.h * w.G + r % w.G) * D + c);
            *reinterpret_cast<float4 *>(&sm.q[r][c]) = x;
        }
        float m[RT], l[RT];
        float4 o[RT][CT];
        int limit[RT];  // last position the row sees
        // last position that every row of the unit sees; of a tree's: the context's last
        const int sure = pc.s.len - pc.s.T + (TREE ? -1 : t0);
        uint64_t path[RT];  // TREE: the rows' paths
        Paths paths;
        if constexpr (TREE) paths = tree_paths(w.parents + pc.s.bos, pc.s.T, w.pg.status);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            limit[r] = (TREE ? sure + 1 + t0 : sure) + (ty * RT + r) / w.G;
            if (ty * RT + r >= rows) limit[r] = -1;
            if constexpr (TREE) path[r] = paths.at(min(t0 + (ty * RT + r) / w.G, pc.s.T - 1));
#pragma unroll
            for (int c = 0; c < CT; ++c) o[r][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // While a tile is at work, the next one's rows are on their way to registers (they fit up to D = 128) and the
        // block table's entries of the one after it (4 x 300 tokens over 4000, 8 heads on 2, d = 128, e4m3: 515 us,
        // 622 with each tile loaded when it was due).
        auto pool_row = [&](int j) -> long {  // of key `tid` of tile j, or -1
            const int pos = j * BN + tid;
            if (tid >= BN || j >= off + take || pos >= pc.s.len) return -1;
            const long pg = pool_page(w.pg, pc.n, pos / w.pg.page_size);
            return pg < 0 ? -1 : (pg * w.pg.Hkv + pc.h) * w.pg.page_size + pos % w.pg.page_size;
        };
        constexpr bool kAhead = D <= 128;
        constexpr int NE = BN * (D / 4) / kThreads;
        Raw4<KIND> kr[kAhead ? NE : 1], vr[kAhead ? NE : 1];
        auto load_rows = [&](int e, Raw4<KIND> &k, Raw4<KIND> &v) {  // piece e of the tile whose pool rows are in sm.at
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            const long at = sm.at[r];
            if (at >= 0) {
                k.template load<D>(a.k_cache, a.k_scale, at, c);
                v.template load<D>(a.v_cache, a.v_scale, at, c);
            } else {  // a position past the end adds 0 * 0
                k.zero();
                v.zero();
            }
        };
        auto store_rows = [&](int e, const Raw4<KIND> &k, const Raw4<KIND> &v) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            *reinterpret_cast<float4 *>(&sm.k[r][c]) = k.get();
            *reinterpret_cast<float4 *>(&sm.v[r][c]) = v.get();
        };
        if (tid < BN) sm.at[tid] = pool_row(off);
        long at_next = pool_row(off + 1);
        if constexpr (kAhead) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NE; ++i) load_rows(tid + i * kThreads, kr[i], vr[i]);
        }
        for (int j = off; j < off + take; ++j) {
            __syncthreads();  // the tile before is used up
            if constexpr (kAhead) {
#pragma unroll
                for (int i = 0; i < NE; ++i) store_rows(tid + i * kThreads, kr[i], vr[i]);
                if (tid < BN) sm.at[tid] = at_next;
                __syncthreads();
                if (j + 1 < off + take)
#pragma unroll
                    for (int i = 0; i < NE; ++i) load_rows(tid + i * kThreads, kr[i], vr[i]);
            } else {
#pragma unroll 4
                for (int i = 0; i < NE; ++i) {
                    load_rows(tid + i * kThreads, kr[0], vr[0]);
                    store_rows(tid + i * kThreads, kr[0], vr[0]);
                }
                __syncthreads();
                if (tid < BN) sm.at[tid] = at_next;
            }
            at_next = pool_row(j + 2);
            if (__builtin_expect(careful, false)) {
#pragma unroll 1
                for (int e = tid; e < BN * D; e += kThreads)
                    if (j * BN + e / D > sure) sm.v[e / D][e % D] = finite_or_zero(sm.v[e / D][e % D]);
                __syncthreads();
            }
            float s[RT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 kk[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) kk[c] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * c][d]);
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float4 qq = *reinterpret_cast<const float4 *>(&sm.q[ty * RT + r][d]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[r][c] += dot4(qq, kk[c]);
                }
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if constexpr (TREE)
                        s[r][c] = limit[r] >= 0 && on_path(path[r], j * BN + tx + 16 * c - sure - 1) ? s[r][c] * a.scale2 : -INFINITY;
                    else
                        s[r][c] = j * BN + tx + 16 * c <= limit[r] ? s[r][c] * a.scale2 : -INFINITY;
                    top = fmaxf(top, s[r][c]);
                }
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float mn = fmaxf(m[r], top), ref = mn == -INFINITY ? 0.f : mn;
                const float f = exp2f(m[r] - ref);
                m[r] = mn;
                float add = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float e = exp2f(s[r][c] - ref);
                    add += e;
                    sm.p[ty * RT + r][tx + 16 * c] = e;
                }
                l[r] = l[r] * f + add;
#pragma unroll
                for (int c = 0; c < CT; ++c) { o[r][c].x *= f; o[r][c].y *= f; o[r][c].z *= f; o[r][c].w *= f; }
            }
            __syncwarp();  // a row's probabilities are written and read by the same half warp
#pragma unroll 2
            for (int k = 0; k < BN; k += 4) {
                float4 pp[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) pp[r] = *reinterpret_cast<const float4 *>(&sm.p[ty * RT + r][k]);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const float4 vv = *reinterpret_cast<const float4 *>(&sm.v[k + kk][64 * c + 4 * tx]);
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const float e = kk == 0 ? pp[r].x : kk == 1 ? pp[r].y : kk == 2 ? pp[r].z : pp[r].w;
                            o[r][c].x += e * vv.x; o[r][c].y += e * vv.y; o[r][c].z += e * vv.z; o[r][c].w += e * vv.w;
                        }
                    }
            }
            __syncwarp();
        }
        bool bad = false;  // a row's output is not finite
        const bool whole = begun && off + take == pc.ntiles;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float sum = l[r];
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            const int row = ty * RT + r;
            if (row >= rows) continue;
#pragma unroll
            for (int c = 0; c < CT; ++c)
                bad |= !(fabsf(o[r][c].x) + fabsf(o[r][c].y) + fabsf(o[r][c].z) + fabsf(o[r][c].w) < INFINITY);
            if (whole) {
                if (limit[r] < 0) continue;  // padding: already zeros
                const float inv = sum == 0.f ? 0.f : 1.f / sum;  // scores that are all -inf: zeros
                float *dst = a.out + ((pc.s.bos + t0 + row / w.G) * a.Hq + pc.h * w.G + row % w.G) * D;
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    *reinterpret_cast<float4 *>(dst + 64 * c + 4 * tx) =
                        make_float4(o[r][c].x * inv, o[r][c].y * inv, o[r][c].z * inv, o[r][c].w * inv);
            } else {
                const long at = part_index(w, blockIdx.x, begun ? 1 : 0, row);
                if (tx == 0) w.ml[at] = make_float2(m[r], sum);
#pragma unroll
                for (int c = 0; c < CT; ++c) *reinterpret_cast<float4 *>(w.part + at * D + 64 * c + 4 * tx) = o[r][c];
            }
        }
        if (__builtin_expect(careful, false)) {
#pragma unroll 1
            for (int r = 0; r < RT; ++r) {
                const int row = ty * RT + r, last = min((TREE ? sure + 1 + t0 : sure) + row / w.G, (off + take) * BN - 1);
                if (row >= rows) continue;
                float *dst = whole ? a.out + ((pc.s.bos + t0 + row / w.G) * a.Hq + pc.h * w.G + row % w.G) * D
                                   : w.part + part_index(w, blockIdx.x, begun ? 1 : 0, row) * D;
#pragma unroll 1
                for (int pos = max(max(sure + 1, off * BN), 0); pos <= last; ++pos) {
                    if (TREE && !on_path(path[r], pos - sure - 1)) continue;
                    const long pg = pool_page(w.pg, pc.n, pos / w.pg.page_size);
                    if (pg < 0) continue;
                    Raw4<KIND> v;
#pragma unroll 1
                    for (int c = 4 * tx; c < D; c += 64) {
                        v.template load<D>(a.v_cache, a.v_scale, (pg * w.pg.Hkv + pc.h) * w.pg.page_size + pos % w.pg.page_size, c);
                        const float4 x = v.get();
                        dst[c] += x.x - finite_or_zero(x.x); dst[c + 1] += x.y - finite_or_zero(x.y);
                        dst[c + 2] += x.z - finite_or_zero(x.z); dst[c + 3] += x.w - finite_or_zero(x.w);
                    }
                }
            }
        }
        // A value that is not finite makes rows that do not see it NaN (0 times it), so a unit whose output is not finite is
        // done again with care: without the values that some rows do not see and that are not finite, which the rows that
        // see them get added above. (Where every row sees all that any sees, there is no need.)
        careful = !careful && (TREE || rows > w.G) && __syncthreads_or(bad);
        if (!careful) {
            pc.left -= take;
            if (pc.left > 0) next_unit<BN, TREE>(w, &pc);
            begun = true;
        }
    }
}

template <int KIND, int D, int R, bool TREE>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
    const int G = a.Hq / a.pg.Hkv;
    SimtParams p{attn_work(a, R / G, 1), (const float *)a.q, a.k_cache, a.v_cache, a.k_scale, a.v_scale,
                 (float *)a.out, a.Hq, a.q_stride, a.scale * kLog2e};
    auto kernel = attn_simt_kernel<KIND, D, R, TREE>;
    constexpr int bytes = sizeof(SimtSmem<D, R>);
    static_assert(bytes <= 232448, "over the 227 KiB opt-in limit");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const int ctas = attn_ctas(a, p.w, BN);
    e = launch_early(kernel, dim3(ctas), kThreads, bytes, s, p);
    return e != cudaSuccess ? e : launch_attn_join(a, p.w, ctas, s);
}

template <int KIND, int D, bool TREE>
cudaError_t launch_rows(const AttnArgs &a, cudaStream_t s) {
    // a row tile of 16 or 32 where no sequence has more rows: a quarter or half of the products of the 64-row tile (8
    // tokens of 4 sequences over 4000, 32 rows, d = 128: 38 us, 47 in the 64-row tile)
    const long rows = (a.pg.cu ? a.pg.Ttot : a.pg.T) * (a.Hq / a.pg.Hkv);
    if (rows <= 16) return launch_t<KIND, D, 16, TREE>(a, s);
    return rows <= 32 ? launch_t<KIND, D, 32, TREE>(a, s) : launch_t<KIND, D, 64, TREE>(a, s);
}

template <int KIND>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.d) {
        case 64: return a.parents ? launch_rows<KIND, 64, true>(a, s) : launch_rows<KIND, 64, false>(a, s);
        case 128: return a.parents ? launch_rows<KIND, 128, true>(a, s) : launch_rows<KIND, 128, false>(a, s);
        case 256: return a.parents ? launch_rows<KIND, 256, true>(a, s) : launch_rows<KIND, 256, false>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.cache_dtype) {
        case GDN_FP8: return launch_d<GDN_FP8>(a, s);
        case GDN_INT8: return launch_d<GDN_INT8>(a, s);
        default: return launch_d<GDN_F32>(a, s);
    }
}

}  // namespace gdn
