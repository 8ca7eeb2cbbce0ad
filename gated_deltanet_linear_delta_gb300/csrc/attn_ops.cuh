// attn_ops.cuh -- what the two attention kernels of bf16 inputs share: constants, the exponential,
// 8-bit codes as fp16, the scaling of Q, and the tensor maps of the caches.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <cstdlib>

#include "attn_plan.cuh"
#include "attn_work.h"
#include "tc_ops.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;  // the softmax reference moves when the maximum has grown by 2^8
constexpr long long kWaitDefault = 2000000000LL;  // SM cycles (about 1 s) before a wait gives up
constexpr long long kDrainBudget = 200000000LL;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Wait for a phase, with a limit in SM cycles. The limit is looked at before the thread first sleeps
// inside try_wait, so that a limit of a few cycles makes every wait run out that is not over already.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t phase, long long budget) {
    if (tc::mbar_test_wait(bar, phase)) return true;
    const long long t0 = clock64();
    do {
        if (clock64() - t0 > budget) return false;
    } while (!tc::mbar_try_wait(bar, phase));
    return true;
}
// ... whose outcome the whole warp shares
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, long long budget) {
    return __all_sync(0xffffffffu, wait_for(bar, phase, budget));
}

// base-2 logarithm and reciprocal of a cached scale, to the hardware's 2^-22: their errors cancel in
// nothing but a relative 2^-21 of each probability
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The sum of an 8-bit cache's softmax is taken from P' = P vs as P' / vs. P' is flushed to zero below 2^-126, which
// matters where a key's scale is that much smaller than another's: a row of zeros (its scale is 2^-100) beside values of
// 2^30. Between these bounds it does not (a flushed term is then 2^-36 of the sum at most). A scale beyond them has NaN
// for its reciprocal, by which the sum shows that it has to be taken again, from P without vs.
constexpr float kPlainScaleMin = 9.3132257e-10f, kPlainScaleMax = 1.1258999e15f;  // 2^-30, 2^50
__device__ __forceinline__ float plain_reciprocal(float vs) {
    return vs >= kPlainScaleMin && vs <= kPlainScaleMax ? rcp(vs) : __int_as_float(0x7fffffff);
}

// 4 codes to fp16 (exact)
template <int KIND>
__device__ __forceinline__ void codes4_to_f16(uint32_t c, uint32_t &h0, uint32_t &h1) {
    if constexpr (KIND == GDN_FP8) {
        asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}"
            : "=r"(h0), "=r"(h1)
            : "r"(c));
    } else {
        // c + 128 as the low byte of an fp16 in [1024, 2048), whose unit is 1; minus 1152 gives c, exactly
        const uint32_t u = c ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
        const uint32_t w0 = __byte_perm(u, 0x64646464u, 0x4140), w1 = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&w0), bias);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&w1), bias);
        h0 = *reinterpret_cast<const uint32_t *>(&x);
        h1 = *reinterpret_cast<const uint32_t *>(&y);
    }
}

// Exponent e such that a row of largest magnitude amax, times 2^e, has it in [2^13, 2^14): in fp16
// the largest elements are far from overflow and all that count are normal.
__device__ __forceinline__ int f16_row_exponent(float amax) {
    if (!(amax > 0.f && amax < 3.4e38f)) return 0;
    return max(-100, min(100, 13 - ((int)(__float_as_uint(amax) >> 23) - 127)));
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

inline long long wait_budget() {
    if (const char *env = getenv("GDN_TEST_WAIT_CYCLES")) {  // test hook: a short limit makes the waits run out
        const long long x = atoll(env);
        if (x > 0) return x;
    }
    return kWaitDefault;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn tiled_encoder() {
    static EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}

// A cache as [page, head][lines of `line` bytes] -> 3-D map, box (128 bytes, `lines` lines, 1), 128B
// swizzle. A line is a position's row, or two positions' where a row has only 64 bytes.
inline bool page_map(CUtensorMap *m, const void *base, const KvPages &pg, int line, int lines) {
    EncodeTiledFn enc = tiled_encoder();
    if (!enc) return false;
    const int elem = pg.cache_dtype == GDN_BF16 ? 2 : 1;
    const cuuint64_t page = (cuuint64_t)pg.page_size * pg.d * elem;
    const cuuint64_t gdim[3] = {(cuuint64_t)(line / elem), page / line, (cuuint64_t)pg.num_pages * pg.Hkv};
    const cuuint64_t gstride[2] = {(cuuint64_t)line, page};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / elem), (cuuint32_t)lines, 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    return enc(m, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3,
               const_cast<void *>(base), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows q [tokens][heads][d] bf16 (token stride free) -> 3-D map, box (64 elements, G heads, TPT tokens),
// 128B swizzle: a unit's G * TPT rows, 128 bytes of each
inline bool rows_map(CUtensorMap *m, const void *base, int d, int heads, long tokens, long stride, int G, int TPT) {
    EncodeTiledFn enc = tiled_encoder();
    if (!enc) return false;
    const cuuint64_t gdim[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t gstride[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)TPT};
    const cuuint32_t estride[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Values at positions that some rows of a unit see and others do not. A masked probability is 0, and 0 times an
// infinity or a NaN is NaN, so in a product that the rows share such elements are taken as 0, and afterwards the rows
// that see them get them added to their output: any weight leaves them what they are. (What is rare is kept out of the
// kernels' code, which is fetched anew by every launch: the same inlined cost 8 prompts of 1024 tokens 7%.)
__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, false); }
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {  // the sign bits of a bf16 pair's that are not
    return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;  // (all ones in the exponent)
}
__device__ __forceinline__ bool any_not_finite(uint4 x) {
    return (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) != 0;
}
// Zeroes them in 16 bytes of shared memory.
static __device__ __noinline__ void drop_not_finite(uint4 *at) {
    uint32_t *w = reinterpret_cast<uint32_t *>(at);
    for (int i = 0; i < 4; ++i) w[i] &= ~((not_finite(w[i]) >> 15) * 0xffffu);
    tc::fence_async_smem();  // products and later copies see it
}
// Adds those of one key head's cached values, positions first .. last, columns c .. c + n - 1, to an output row.
// table: the sequence's pages; shift: log2 of their size.
template <typename T>
static __device__ __noinline__ void add_not_finite(const int32_t *table, int num_pages, int Hkv, int h, int shift,
                                                   const __nv_bfloat16 *v_cache, int d, int first, int last, int c, int n,
                                                   T *row) {
    for (int pos = first; pos <= last; ++pos) {
        const int page = table[pos >> shift];
        if ((unsigned)page >= (unsigned)num_pages) continue;  // (values of zero)
        const __nv_bfloat16 *v = v_cache + ((((long)page * Hkv + h) << shift) + (pos & ((1 << shift) - 1))) * d;
        for (int i = c; i < c + n; ++i) {
            const float x = __bfloat162float(v[i]);
            if (!(fabsf(x) < INFINITY)) row[i] = from_f32<T>((float)row[i] + x);
        }
    }
}

// A running softmax reference m of a row (log2 domain), given its maximum over more keys: moved when
// that has grown by more than 2^kGrow. l, the sum so far, is brought to it; f is the factor for what was summed otherwise.
// (In two halves: with an 8-bit cache the references of rows of zeros and of large values are further apart than a float's
// exponents reach, and l is as much larger.)
__device__ __forceinline__ bool above_reference(float m, float top) { return top > m + kGrow; }  // (-inf: any score)
template <bool CODES>
__device__ __forceinline__ bool grow_reference(float &m, float top, float &f, float &l) {
    const bool grow = above_reference(m, top);
    f = 1.f;
    if (grow) {
        f = ex2(m - top);  // m = -inf: 0
        if constexpr (CODES) {
            const float h = ex2(0.5f * (m - top));
            l = l * h * h;
        } else {
            l *= f;
        }
        m = top;
    }
    return grow;
}

}  // namespace gdn
