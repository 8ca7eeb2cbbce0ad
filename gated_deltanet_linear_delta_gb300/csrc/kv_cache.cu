// kv_cache.cu -- new keys and values into a paged cache (quantised on the way), and back.
//
// Both directions touch every byte once and are bound by memory: a token's row of one head is
// read, its largest magnitude is reduced across the lanes that hold it, and the codes and one
// scale are written; reading back is code times scale. (formulas: kv_pages.cuh)
//
// Work split: a CTA takes a run of tokens. Where each lies (its sequence, kv_lens, the page) is found
// first, by a warp per token, into shared memory; then the CTA's lanes stream over the run's rows
// (each token's Hkv keys, then its Hkv values), 2 or 4 rows' pieces in flight per lane before any is used.
// Runs get longer with the number of tokens: many small runs give a decode step's few tokens a CTA
// each, long ones spread the look-up over more bytes (with a token per warp, whose three dependent
// reads stood before every 1 KiB, a long session was read at 3.4 TB/s; with runs at 6.0).
//
// Measured: 131072 tokens of 2 heads, d = 256, e4m3 to bf16: 64.9 us, 93% of the measured copy rate; 24
// sessions of 8 heads, d = 128, int8 to fp32: 63.3 us, 96%; 16384 tokens of 8 heads, d = 128 stored as
// int8: 28.7 us, 3.5 TB/s, bound by the instructions that quantise (0.7 of 1 a cycle and scheduler).
#include <algorithm>

#include "kv_pages.cuh"

namespace gdn {
namespace {

constexpr int kKvThreads = 256;

// 16 bytes of rows as fp32
__device__ __forceinline__ void unpack16(uint4 r, float (&x)[8]) {  // bf16
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack16(uint4 r, float (&x)[4]) {  // fp32
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack16(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// The largest magnitude of a lane's pieces; infinity where one is not finite. bf16 by pairs (a maximum that keeps a NaN
// takes half an instruction an element, a comparison of each in fp32 four).
template <typename T, int NP>
__device__ __forceinline__ float largest(const uint4 (&x)[NP]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = 0;
#pragma unroll
        for (int g = 0; g < NP; ++g) {
            const uint32_t w[4] = {x[g].x, x[g].y, x[g].z, x[g].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm("{\n.reg .b32 t;\nabs.bf16x2 t, %1;\nmax.NaN.bf16x2 %0, %0, t;\n}" : "+r"(m) : "r"(w[i]));
        }
        const float a = __uint_as_float(m << 16), b = __uint_as_float(m & 0xffff0000u);
        return a == a && b == b ? fmaxf(a, b) : __int_as_float(0x7f800000);
    } else {
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int g = 0; g < NP; ++g) {
            float y[4];
            unpack16(x[g], y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                m = fmaxf(m, fabsf(y[e]));
                bad |= !(fabsf(y[e]) <= 3.4028234e38f);
            }
        }
        return bad ? __int_as_float(0x7f800000) : m;
    }
}

// Pool row (page, row in it, head 0) of packed token i, by a whole warp: -1 padding, -2 not to be touched
__device__ __forceinline__ long token_row(const KvPages &p, long i, int page_shift) {
    const int n = seq_of_token(p, i);
    SeqInfo s;
    if (!seq_info(p, n, &s)) return -2;
    if (i < s.bos || i >= s.bos + s.T) {  // a token that cu gives to no sequence
        flag_error(p.status);
        return -2;
    }
    const int pos = s.len - s.T + (int)(i - s.bos);
    if (pos < 0) return -1;
    const long pg = pool_page(p, n, pos >> page_shift);
    return pg < 0 ? -3 : ((pg * p.Hkv) << page_shift) + (pos & (p.page_size - 1));
}

constexpr int kMaxRun = 32;

// KIND: GDN_FP8, GDN_INT8, or anything else for a cache of the rows' type
template <bool WRITE, typename T, int KIND, int D>
__global__ void __launch_bounds__(kKvThreads, 4) kv_copy_kernel(const KvArgs a, int run, int page_shift) {
    constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    // A lane has 16 elements of a row, as pieces whose rows' side is 16 bytes: consecutive lanes' pieces are
    // consecutive, so that both sides' accesses are whole lines.
    constexpr int E = 16, PE = 16 / (int)sizeof(T), NP = E / PE, LPR = D / E, ROWS = kKvThreads / LPR;
    // rows in flight per lane, as many as fit its registers (fp32 copies of 16384 tokens, 8 heads, d = 128: 43 us with 2,
    // 50 with 4; bf16 rows stored as codes: with 4, the same tokens as int8 28 us instead of 29, but 131072 tokens of 2
    // heads, d = 256, as e4m3 83 instead of 78)
    constexpr int kFlight = (kCodes ? WRITE : sizeof(T) == 4) ? 2 : 4;
    __shared__ long where[kMaxRun];
    const KvPages &p = a.pg;
    const int tid = threadIdx.x, lane = tid & 31, c = (tid % LPR) * PE, sub = tid / LPR;
    const long first = (long)blockIdx.x * run;
    const int tokens = (int)min((long)run, p.Ttot - first), heads = 2 * p.Hkv;
    next_may_begin();
    before_reading();
    check_offsets(p);
    // This thread's rows, a pass at a time: whole tokens' rows side by side if a pass holds some, else a token's
    // rows in several passes.
    struct At {
        int t, j;
    };
    const int per_pass = ROWS / heads;
    At at0{per_pass ? sub / heads : 0, per_pass ? sub % heads : sub};
    if (per_pass && at0.t >= per_pass) at0.t = kMaxRun;  // no row of its own
    auto next = [&](At &r) {
        if (per_pass) {
            r.t += per_pass;
        } else if ((r.j += ROWS) >= heads) {
            r.j = sub;
            ++r.t;
        }
    };
    const int passes = per_pass ? (tokens + per_pass - 1) / per_pass : tokens * ((heads + ROWS - 1) / ROWS);
    auto live = [&](const At &r) { return r.t < tokens && r.j < heads; };
    auto outside = [&](const At &r) -> T * {  // the row in k or v
        const bool is_v = r.j >= p.Hkv;
        return (is_v ? (T *)a.v + (first + r.t) * a.v_stride : (T *)a.k + (first + r.t) * a.k_stride) +
               (long)(is_v ? r.j - p.Hkv : r.j) * D + c;
    };
    uint4 x[kFlight][NP];
    auto load_rows = [&](At r) {  // (a write's rows do not depend on where they go)
#pragma unroll
        for (int f = 0; f < kFlight; ++f, next(r)) {
            if (!live(r)) continue;
            const T *src = outside(r);
#pragma unroll
            for (int g = 0; g < NP; ++g) x[f][g] = __ldcs(reinterpret_cast<const uint4 *>(src + g * LPR * PE));
        }
    };
    if (WRITE) load_rows(at0);
    for (int t = tid >> 5; t < tokens; t += kKvThreads / 32) {
        const long w = token_row(p, first + t, page_shift);
        if (lane == 0) where[t] = w;
    }
    __syncthreads();
    At r0 = at0;
    for (int pass = 0; pass < passes; pass += kFlight) {
        if (WRITE && pass) load_rows(r0);
        At r = r0;
        if constexpr (WRITE) {
#pragma unroll
            for (int f = 0; f < kFlight; ++f, next(r)) {
                const long w = live(r) ? where[r.t] : -2;
                const bool is_v = r.j >= p.Hkv;
                const long at = w + ((long)(is_v ? r.j - p.Hkv : r.j) << page_shift);
                uint8_t *cache = (uint8_t *)(is_v ? a.v_cache : a.k_cache);
                if constexpr (!kCodes) {
                    if (w < 0) continue;
#pragma unroll
                    for (int g = 0; g < NP; ++g) *reinterpret_cast<uint4 *>((T *)cache + at * D + c + g * LPR * PE) = x[f][g];
                } else {
                    float amax = w >= 0 ? largest<T, NP>(x[f]) : 0.f;
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    if (w < 0) continue;
                    const float sc = KIND == GDN_FP8 ? scale_e4m3(amax) : scale_int8(amax);
                    const float inv = KIND == GDN_FP8 ? inverse_pow2(sc) : rcp_near(sc);
#pragma unroll
                    for (int g = 0; g < NP; ++g) {
                        float y[PE];
                        unpack16(x[f][g], y);
                        uint32_t code[PE / 4];
#pragma unroll
                        for (int e = 0; e < PE / 4; ++e)
                            code[e] = sc != sc ? 0u : KIND == GDN_FP8 ? codes4_e4m3(y + 4 * e, inv) : codes4_int8(y + 4 * e, sc, inv);
                        uint8_t *dst = cache + at * D + c + g * LPR * PE;
                        if constexpr (PE == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
                        else *reinterpret_cast<uint32_t *>(dst) = code[0];
                    }
                    if (c == 0) (is_v ? a.v_scale : a.k_scale)[at] = sc;
                }
            }
        } else {
            uint32_t code[kFlight][E / 4];
            float sc[kFlight];
            long w[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f, next(r)) {
                w[f] = live(r) ? where[r.t] : -2;
                if (w[f] < 0) continue;
                const bool is_v = r.j >= p.Hkv;
                const long at = w[f] + ((long)(is_v ? r.j - p.Hkv : r.j) << page_shift);
                const uint8_t *cache = (const uint8_t *)(is_v ? a.v_cache : a.k_cache);
#pragma unroll
                for (int g = 0; g < NP; ++g) {
                    if constexpr (!kCodes) {
                        x[f][g] = __ldcs(reinterpret_cast<const uint4 *>((const T *)cache + at * D + c + g * LPR * PE));
                    } else if constexpr (PE == 8) {
                        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(cache + at * D + c + g * LPR * PE));
                        code[f][2 * g] = v.x;
                        code[f][2 * g + 1] = v.y;
                    } else {
                        code[f][g] = __ldcs(reinterpret_cast<const uint32_t *>(cache + at * D + c + g * LPR * PE));
                    }
                }
                if constexpr (kCodes) sc[f] = __ldcs((is_v ? a.v_scale : a.k_scale) + at);
            }
            r = r0;
#pragma unroll
            for (int f = 0; f < kFlight; ++f, next(r)) {
                if (w[f] == -2) continue;
                T *dst = outside(r);
#pragma unroll
                for (int g = 0; g < NP; ++g) {
                    uint4 out = make_uint4(0, 0, 0, 0);  // padding, and pages outside of the pool
                    if (w[f] >= 0) {
                        if constexpr (kCodes) {
                            float y[PE];
#pragma unroll
                            for (int e = 0; e < PE / 4; ++e) {
                                if (KIND == GDN_FP8) decode4_e4m3(code[f][g * (PE / 4) + e], y + 4 * e);
                                else decode4_int8(code[f][g * (PE / 4) + e], y + 4 * e);
                            }
#pragma unroll
                            for (int e = 0; e < PE; ++e) y[e] *= sc[f];
                            out = pack16(y);
                        } else {
                            out = x[f][g];
                        }
                    }
                    __stcs(reinterpret_cast<uint4 *>(dst + g * LPR * PE), out);
                }
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) next(r0);
    }
}

template <bool WRITE, typename T, int KIND, int D>
cudaError_t launch_kv(const KvArgs &a, cudaStream_t s) {
    // A CTA per token until there are 8 per SM, then runs of up to 128 rows: of 2 key heads' tokens 32 (reading a
    // long session: 67 us, at 32 rows a run 129 us), of 8 key heads' 8 (a prompt's write 33 us, at 512 rows 37 us).
    const long per = a.pg.Ttot / (152 * 8), most = 128 / (2 * a.pg.Hkv);
    const int run = (int)std::max(1L, std::min(std::min(per, most), (long)kMaxRun));
    const long blocks = (a.pg.Ttot + run - 1) / run;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    int shift = 0;
    while ((1 << shift) < a.pg.page_size) ++shift;
    return launch_early(kv_copy_kernel<WRITE, T, KIND, D>, dim3((unsigned)blocks), kKvThreads, 0, s, a, run, shift);
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
