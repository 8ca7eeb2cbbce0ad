// kv_pages.cuh -- device helpers of the paged key/value cache: where a token's row lies, and the
// 8-bit codes of a cached row.
//
// Codes. A row x of d elements is stored as codes c and one fp32 scale s, x ~ c s:
//   e4m3: s = 2^k, the smallest with amax / s <= 448. Division and product by a power of two are
//         exact, so the only rounding is the code's own (relative 2^-4 at most); a scale between
//         two powers of two would not make it smaller, since the format's precision is relative.
//   int8: s = amax / 127, c = rint(x / s): the error is at most s / 2, relative to the row's
//         largest element, so here the scale is not rounded to a power of two.
// s is at least 2^-100, so that 1 / s and c s stay far from fp32's range; rows below that are
// stored as zeros or subnormal multiples of it. A row that holds an infinity or a NaN gets scale
// NaN and codes 0: it reads back as NaN throughout, never as something finite.
#pragma once

#include <cuda_fp8.h>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

constexpr float kMinKvScale = 7.8886090522101181e-31f;  // 2^-100

// ---- sequences -------------------------------------------------------------------
// A launch that may begin while the kernel before it in its stream still runs, so that the start of one hides
// behind the end of the other. A kernel so launched calls before_reading() before it touches any memory that other
// kernels use, with all its threads: that waits until everything before it in the stream is done. (One
// session's token 13.5 -> 11.6 us a call, a long read 67.6 -> 64.9.)
template <typename... P>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int block, size_t smem, cudaStream_t s, P... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void before_reading() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the kernel after this one may begin (and wait for this one's end)
__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct SeqInfo {
    long bos;  // first packed token
    int T;     // new tokens
    int len;   // cached tokens, the new ones among them
};

// Sequence n of the call. False (flagged) when cu is inconsistent or gives a tree too many nodes; a kv_len outside of the block
// table's row is flagged and counts as 0, which makes the sequence's tokens padding.
template <bool TREE = false>
__device__ __forceinline__ bool seq_info(const KvPages &p, int n, SeqInfo *s) {
    long eos;
    if (!seq_bounds(p.cu, n, p.B, p.cu ? p.Ttot : p.T, &s->bos, &eos, p.status)) {
        s->T = s->len = 0;
        return false;
    }
    if (TREE && eos - s->bos > kTreeMax) {
        flag_error(p.status);
        s->T = s->len = 0;
        return false;
    }
    s->T = (int)(eos - s->bos);
    int len = p.kv_lens[n];
    if (len < 0 || len > (long)p.max_pages * p.page_size) {
        flag_error(p.status);
        len = 0;
    }
    s->len = len;
    return true;
}

// The sequence of packed token i, found by a whole warp: the last n with cu[n] <= i (32 probes a
// step, so 2 dependent reads for up to 1024 sequences).
__device__ __forceinline__ int seq_of_token(const KvPages &p, long i) {
    if (p.cu == nullptr) return (int)((uint32_t)i / (uint32_t)p.T);  // (fewer than 2^31 tokens)
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lo + lane * step;
        const bool in = lane * step < n && (lane == 0 || p.cu[at] <= i);
        const unsigned m = __ballot_sync(0xffffffffu, in);
        const int k = 31 - __clz(m);  // for an increasing cu, lanes 0..k
        n = min(step, n - k * step);
        lo += k * step;
    }
    return lo;
}

// Flags offsets that are not increasing from 0 to Ttot. (A token's own sequence is checked where it
// is used; this finds the sequences that own no token because of their offsets.)
__device__ __forceinline__ void check_offsets(const KvPages &p) {
    if (p.cu == nullptr) return;
    const long all = (long)gridDim.x * blockDim.x;
    for (long n = (long)blockIdx.x * blockDim.x + threadIdx.x; n < p.B; n += all) {
        long bos, eos;
        seq_bounds(p.cu, (int)n, p.B, p.Ttot, &bos, &eos, p.status);
    }
}

// The index-th page of sequence n, or -1 (flagged) when the table names none of the pool's.
__device__ __forceinline__ long pool_page(const KvPages &p, int n, int index) {
    const int pg = p.table[(long)n * p.max_pages + index];
    if (pg < 0 || pg >= p.num_pages) {
        flag_error(p.status);
        return -1;
    }
    return pg;
}

// ---- codes -----------------------------------------------------------------------
__device__ __forceinline__ float scale_e4m3(float amax) {
    if (!(amax <= 3.4028234e38f)) return __int_as_float(0x7fffffff);
    const uint32_t u = __float_as_uint(amax);
    // amax = m 2^(e-127), m in [1, 2); 448 = 1.75 * 2^8 (a subnormal amax ends at the floor below)
    const int e = (int)(u >> 23), k = e - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(max(k, -100) + 127) << 23);
}
__device__ __forceinline__ float scale_int8(float amax) {
    if (!(amax <= 3.4028234e38f)) return __int_as_float(0x7fffffff);
    return fmaxf(__fdiv_rn(amax, 127.f), kMinKvScale);
}

// 1 / s: of a power of two of 2^-100 or more, exact; of any s, to 1 ulp
__device__ __forceinline__ float inverse_pow2(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }
__device__ __forceinline__ float rcp_near(float s) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    return y;
}

// 4 codes of x[0..3] (x / s rounded to nearest even), the first in the lowest byte
__device__ __forceinline__ uint32_t codes4_e4m3(const float *x, float inv) {  // inv = 1 / s, exact
    const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)a | ((uint32_t)b << 16);
}
// two fp32 operations in one instruction
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ void f2_get(F2 a, float &x, float &y) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}

// The code is the quotient x / s, correctly rounded to fp32, rounded to an integer. x (1 / s) is within
// 2^-15 of it (127 times 1 ulp of the reciprocal and two halves), so only where such a product comes
// that close to the middle between two integers are the four divided. (Adding 1.5 * 2^23 rounds to an integer, and leaves it in the low bits.)
__device__ __forceinline__ uint32_t codes4_int8(const float *x, float s, float inv) {
    constexpr float kRound = 12582912.f;
    float y[4], off = 0.f;
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const F2 t = f2_mul(f2(x[j], x[j + 1]), f2(inv, inv)), r = f2_add(t, f2(kRound, kRound));
        const F2 d = f2_fma(f2_add(r, f2(-kRound, -kRound)), f2(-1.f, -1.f), t);
        float d0, d1;
        f2_get(d, d0, d1);
        f2_get(r, y[j], y[j + 1]);
        off = fmaxf(off, fmaxf(fabsf(d0), fabsf(d1)));
    }
    if (off > 0.49995f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __fadd_rn(__fdiv_rn(x[j], s), kRound);
    }
    const uint32_t lo = __byte_perm(__float_as_uint(y[0]), __float_as_uint(y[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(y[2]), __float_as_uint(y[3]), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ void decode4_e4m3(uint32_t c, float *x) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> (16 * j)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
    }
}
__device__ __forceinline__ void decode4_int8(uint32_t c, float *x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = (float)(int8_t)(c >> (8 * j));
}

}  // namespace gdn
