// kv_cache.cu -- new keys and values into a paged cache (quantised on the way), and back.
//
// Both directions touch every byte once and are bound by memory: a token's row of one head is
// read, its largest magnitude is reduced across the lanes that hold it, and the codes and one
// scale are written; reading back is code times scale. (formulas: kv_pages.cuh)
//
// Work split: a warp takes one token and up to 4 passes over its rows (its Hkv keys, then its Hkv
// values; a pass is as many rows as fit the warp at one 16-byte piece of the narrower side a
// lane). Where the token lies (its sequence, kv_lens, the page) is found once per warp, and in
// the write the rows' loads are issued before it, since they do not depend on it.
#include "kv_pages.cuh"

namespace gdn {
namespace {

constexpr int kKvThreads = 256;
constexpr int kPasses = 4;

// E consecutive elements (E a multiple of 8) as fp32
template <int E>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *p, float *x) {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
        const uint4 r = __ldcs(reinterpret_cast<const uint4 *>(p) + j);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
            x[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <int E>
__device__ __forceinline__ void load_row(const float *p, float *x) {
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        const float4 r = __ldcs(reinterpret_cast<const float4 *>(p) + j);
        x[4 * j] = r.x; x[4 * j + 1] = r.y; x[4 * j + 2] = r.z; x[4 * j + 3] = r.w;
    }
}
template <int E>
__device__ __forceinline__ void store_row(__nv_bfloat16 *p, const float *x) {
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * j + 2 * i], x[8 * j + 2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        reinterpret_cast<uint4 *>(p)[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <int E>
__device__ __forceinline__ void store_row(float *p, const float *x) {
#pragma unroll
    for (int j = 0; j < E / 4; ++j)
        reinterpret_cast<float4 *>(p)[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}
// 8 or 16 code bytes
template <int E>
__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t *w) {
    if constexpr (E == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// KIND: GDN_BF16 / GDN_F32 here mean "as the inputs"
template <typename TIn, int KIND, int D>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvArgs a) {
    constexpr int E = 8, LPR = D / E, RPW = 32 / LPR;
    constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    const KvPages &p = a.pg;
    const int lane = threadIdx.x & 31, c = (lane % LPR) * E, sub = lane / LPR;
    const int chunks = (2 * p.Hkv + RPW * kPasses - 1) / (RPW * kPasses);
    const long w = (long)blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    const long i = w / chunks;
    const int j0 = (int)(w % chunks) * RPW * kPasses + sub;
    check_offsets(p);
    if (i >= p.Ttot) return;

    float x[kPasses][E];
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
        const int j = j0 + r * RPW;
        if (j < 2 * p.Hkv)
            load_row<E>(j < p.Hkv ? (const TIn *)a.k + i * a.k_stride + (long)j * D + c
                                  : (const TIn *)a.v + i * a.v_stride + (long)(j - p.Hkv) * D + c, x[r]);
    }
    const int n = seq_of_token(p, i);
    SeqInfo s;
    if (!seq_info(p, n, &s)) return;
    if (i < s.bos || i >= s.bos + s.T) {  // a token that cu gives to no sequence
        flag_error(p.status);
        return;
    }
    const int pos = s.len - s.T + (int)(i - s.bos);
    if (pos < 0) return;  // padding
    const long pg = pool_page(p, n, pos);
    if (pg < 0) return;
    const int row = pos % p.page_size;
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
        const int j = j0 + r * RPW;
        const bool live = j < 2 * p.Hkv;
        const int h = j < p.Hkv ? j : j - p.Hkv;
        const long at = (pg * p.Hkv + h) * p.page_size + row;
        uint8_t *cache = (uint8_t *)(j < p.Hkv ? a.k_cache : a.v_cache);
        if constexpr (!kCodes) {
            if (live) store_row<E>((TIn *)cache + at * D + c, x[r]);
        } else {
            float amax = 0.f;
            bool bad = false;
            if (live) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    amax = fmaxf(amax, fabsf(x[r][e]));
                    bad |= !(fabsf(x[r][e]) <= 3.4028234e38f);
                }
            }
            if (bad) amax = __int_as_float(0x7f800000);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            if (!live) continue;
            const float sc = KIND == GDN_FP8 ? scale_e4m3(amax) : scale_int8(amax);
            uint32_t code[E / 4];
#pragma unroll
            for (int e = 0; e < E / 4; ++e)
                code[e] = sc != sc ? 0u : KIND == GDN_FP8 ? codes4_e4m3(x[r] + 4 * e, 1.f / sc) : codes4_int8(x[r] + 4 * e, sc);
            store_codes<E>(cache + at * D + c, code);
            if (c == 0) (j < p.Hkv ? a.k_scale : a.v_scale)[at] = sc;
        }
    }
}

template <typename TOut, int KIND, int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvArgs a) {
    constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    constexpr int E = kCodes ? 16 : 8, LPR = D / E, RPW = 32 / LPR;
    const KvPages &p = a.pg;
    const int lane = threadIdx.x & 31, c = (lane % LPR) * E, sub = lane / LPR;
    const int chunks = (2 * p.Hkv + RPW * kPasses - 1) / (RPW * kPasses);
    const long w = (long)blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    const long i = w / chunks;
    const int j0 = (int)(w % chunks) * RPW * kPasses + sub;
    check_offsets(p);
    if (i >= p.Ttot) return;
    const int n = seq_of_token(p, i);
    SeqInfo s;
    if (!seq_info(p, n, &s)) return;
    if (i < s.bos || i >= s.bos + s.T) {
        flag_error(p.status);
        return;
    }
    const int pos = s.len - s.T + (int)(i - s.bos);
    const long pg = pos < 0 ? -1 : pool_page(p, n, pos);
    const int row = pos < 0 ? 0 : pos % p.page_size;
    float x[kPasses][E];
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
        const int j = j0 + r * RPW;
#pragma unroll
        for (int e = 0; e < E; ++e) x[r][e] = 0.f;  // padding reads as zeros
        if (j >= 2 * p.Hkv || pg < 0) continue;
        const int h = j < p.Hkv ? j : j - p.Hkv;
        const long at = (pg * p.Hkv + h) * p.page_size + row;
        const uint8_t *cache = (const uint8_t *)(j < p.Hkv ? a.k_cache : a.v_cache);
        if constexpr (!kCodes) {
            load_row<E>((const TOut *)cache + at * D + c, x[r]);
        } else {
            const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(cache + at * D + c));
            const float sc = (j < p.Hkv ? a.k_scale : a.v_scale)[at];
            const uint32_t code[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (KIND == GDN_FP8) decode4_e4m3(code[e], x[r] + 4 * e);
                else decode4_int8(code[e], x[r] + 4 * e);
#pragma unroll
                for (int m = 0; m < 4; ++m) x[r][4 * e + m] *= sc;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kPasses; ++r) {
        const int j = j0 + r * RPW;
        if (j < 2 * p.Hkv)
            store_row<E>(j < p.Hkv ? (TOut *)a.k + i * a.k_stride + (long)j * D + c
                                   : (TOut *)a.v + i * a.v_stride + (long)(j - p.Hkv) * D + c, x[r]);
    }
}

template <bool WRITE, typename T, int KIND, int D>
cudaError_t launch_kv(const KvArgs &a, cudaStream_t s) {
    constexpr int E = !WRITE && (KIND == GDN_FP8 || KIND == GDN_INT8) ? 16 : 8, RPW = 32 / (D / E);
    const long chunks = (2L * a.pg.Hkv + RPW * kPasses - 1) / (RPW * kPasses);
    const long blocks = (a.pg.Ttot * chunks + kKvThreads / 32 - 1) / (kKvThreads / 32);
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    if (WRITE) kv_write_kernel<T, KIND, D><<<(unsigned)blocks, kKvThreads, 0, s>>>(a);
    else kv_read_kernel<T, KIND, D><<<(unsigned)blocks, kKvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <bool WRITE, typename T, int KIND>
cudaError_t launch_d(const KvArgs &a, cudaStream_t s) {
    switch (a.pg.d) {
        case 64: return launch_kv<WRITE, T, KIND, 64>(a, s);
        case 128: return launch_kv<WRITE, T, KIND, 128>(a, s);
        case 256: return launch_kv<WRITE, T, KIND, 256>(a, s);
    }
    return cudaErrorInvalidValue;
}

template <bool WRITE, typename T>
cudaError_t launch_kind(const KvArgs &a, cudaStream_t s) {
    switch (a.pg.cache_dtype) {
        case GDN_FP8: return launch_d<WRITE, T, GDN_FP8>(a, s);
        case GDN_INT8: return launch_d<WRITE, T, GDN_INT8>(a, s);
        default: return launch_d<WRITE, T, GDN_BF16>(a, s);
    }
}

}  // namespace

cudaError_t launch_kv_write(const KvArgs &a, cudaStream_t s) {
    return a.pg.dtype == GDN_F32 ? launch_kind<true, float>(a, s) : launch_kind<true, __nv_bfloat16>(a, s);
}
cudaError_t launch_kv_read(const KvArgs &a, cudaStream_t s) {
    return a.pg.dtype == GDN_F32 ? launch_kind<false, float>(a, s) : launch_kind<false, __nv_bfloat16>(a, s);
}

}  // namespace gdn
