// attn_tc.cu -- attention over a paged cache on the sm_103a tensor cores (bf16 inputs).
//
// A unit of work (attn_plan.cuh) is up to 128 query rows -- the G query heads that share a key
// head, of consecutive new tokens -- against key tiles of BN positions. With q the rows, per tile j
//     S_j = Q K_j^T                     (tcgen05.mma, Q from TMEM, K_j from shared memory)
//     P_j = exp2(S_j scale log2 e - m)  (fp32, rounded once to 16 bits, stored over S_j in TMEM)
//     O  += P_j V_j                     (tcgen05.mma, P_j from TMEM, V_j from shared memory)
// and l = sum of P in fp32; m is a running reference within 2^8 of the row's maximum: it moves, and
// O is rescaled, only when the maximum has grown by more than that, which leaves P at most 2^8 and
// the result as precise (everything is relative to the same m).
//
// What bounds it. One token per sequence (G rows): the cache is read once, 2 G flops a byte in bf16,
// so HBM; the 128-row products that the G rows are padded to take a third of that time. A prompt's
// fragment (128 rows full): 4 BN D 128 flops a tile against 4 BN D bytes, so the tensor cores, if
// the softmax of one tile hides behind the products of its neighbours.
//
// Layout. TMEM holds O (D columns), two S buffers (P_j overlays S_j) and Q as the 16-bit A operand,
// 512 columns in all for D = 256; with Q in TMEM, shared memory is one ring of K and V tiles, and the
// S products read 64 bytes of it a cycle instead of 192. S_{j+1} is issued before O += P_j V_j, so
// the tensor cores work on it while the softmax of tile j runs.
// Warps: 0..7 softmax (two threads per row, half of the columns each), 8 loads, 9 issues the
// products; with an 8-bit cache 10..13 convert tiles. All CTAs are persistent over their piece of
// the work, and every wait has a limit, after which the CTA flags the status word and leaves.
//
// 8-bit caches. Codes are exact in fp16, so K and V tiles hold codes converted to fp16 (bf16 would
// take four times the conversion instructions for e4m3), Q is rounded to fp16 after an exact
// power-of-two scaling per row, and the cached rows' scales enter in fp32: with a_j = ks_j scale
// log2 e and b_j = log2 vs_j,   y_j = (q.c_j) a_j + b_j,   P'_j = exp2(y_j - m') = P_j vs_j,
//     O += P'_j C_j,   l += P'_j / vs_j.
// Taking vs_j into the exponent keeps P' near 1 for the keys that matter whatever the scales' range.
//
// Masks. A row sees positions up to its own; scores past it are replaced (not multiplied), so what
// K holds there has no effect. Rows of V past the sequence's end are zeroed in shared memory before
// the product, since 0 * NaN would reach the sum.
#include <cuda.h>
#include <cstdlib>
#include <cuda_fp16.h>

#include "attn_plan.cuh"
#include "attn_work.h"
#include "tc_ops.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGrow = 8.f;  // the reference moves when the maximum has grown by 2^8
constexpr long long kWaitDefault = 2000000000LL;  // SM cycles (about 1 s) before a wait gives up
constexpr long long kDrainBudget = 200000000LL;
constexpr int kSoftWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kConvWarp0 = 10, kConvWarps = 4;

template <int D, int KIND>
struct Cfg {
    static constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int HC = BN / 2;                      // columns of S per softmax thread
    static constexpr int NB = D / 64;                      // 128-byte wide blocks of a tile
    static constexpr uint32_t SLOT = BN * D * 2;           // a 16-bit K or V tile
    static constexpr uint32_t RAW = BN * D + 2 * BN * 4;   // a tile's codes, and K and V scales (K fills)
    static constexpr int NS = kCodes ? (D == 64 ? 4 : 3) : (D == 64 ? 12 : 6);
    static constexpr int NR = kCodes ? (D == 64 ? 12 : 7) : 0;
    // Column scales, a buffer per tile: tile j's are written once ring fill (K_j) - NS is used up. With NS = 3
    // that follows the softmax of tile j - 3, with NS = 4 that of tile j - 4.
    static constexpr int COLS = NS;
    static constexpr int THREADS = 32 * (kCodes ? kConvWarp0 + kConvWarps : kConvWarp0);
    static constexpr uint32_t TM_O = 0, TM_S = D == 256 ? 256 : 128, TM_Q = 384;
    // shared memory, from a 1 KiB aligned base
    static constexpr uint32_t SM_RAW = NS * SLOT;
    static constexpr uint32_t SM_COL = SM_RAW + NR * RAW;                    // [COLS][3][BN] a, b, 1 / vs
    static constexpr uint32_t SM_X = SM_COL + (kCodes ? COLS * 3 * BN * 4 : 0);  // [2][2][128] row exchange
    static constexpr uint32_t SM_BAR = SM_X + 2 * 2 * 128 * 4;
    static constexpr int B_FULL = 0, B_EMPTY = NS, B_RFULL = 2 * NS, B_REMPTY = B_RFULL + NR, B_COL = B_REMPTY + NR,
                         B_S = B_COL + COLS, B_P = B_S + 2, B_PV = B_P + 2, B_Q = B_PV + 2, B_FIN = B_Q + 1,
                         B_COUNT = B_FIN + 1;
    static constexpr uint32_t SM_INFO = SM_BAR + B_COUNT * 8;                // [NR] valid rows, page mask
    static constexpr uint32_t SM_TMEM = SM_INFO + (NR ? NR : 1) * 8;
    static constexpr uint32_t SM_PLAN = (SM_TMEM + 8 + 15) & ~15u;
    static constexpr uint32_t SM_BYTES = SM_PLAN + sizeof(PlanSmem) + 1024;
    static_assert(SM_BYTES <= 232448, "over the 227 KiB opt-in limit");
};

struct TcParams {
    AttnWork w;
    const __nv_bfloat16 *q;
    const uint8_t *k_cache, *v_cache;  // 8-bit caches
    const float *k_scale, *v_scale;
    __nv_bfloat16 *out;
    int Hq;
    long q_stride;
    float scale2;  // |softmax scale| * log2 e
    int negate;    // the scale is negative: Q is negated
    long long budget;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf2(float a, float b) { return bf2_bits(__floats2bfloat162_rn(a, b)); }

// A wait whose outcome the whole warp shares
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, long long budget) {
    return __all_sync(0xffffffffu, mbar_wait(bar, phase, budget));
}
__device__ __forceinline__ bool warp_wait_spin(uint64_t *bar, uint32_t phase, long long budget) {
    return __all_sync(0xffffffffu, mbar_wait_spin(bar, phase, budget));
}

// every thread's view of the walk over the piece's units
struct Walk {
    Piece pc;
    bool begun;  // the unit at hand started in this CTA
    __device__ __forceinline__ int take() const { return (int)min((long)(pc.ntiles - pc.off), pc.left); }
};
template <int BN>
__device__ __forceinline__ bool walk_next(const AttnWork &w, Walk *k) {
    k->pc.left -= k->take();
    if (k->pc.left <= 0) return false;
    next_unit<BN>(w, &k->pc);
    k->begun = true;
    return k->pc.left > 0;
}

// ---- loads ------------------------------------------------------------------------
// Fill order is the order of use: K_0, then K_{j+1}, V_j.
template <int D, int KIND>
__device__ void load_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k, const CUtensorMap *mk,
                          const CUtensorMap *mv) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN;
    const KvPages &pg = p.w.pg;
    const int lane = threadIdx.x & 31, P = pg.page_size;
    const int box = min(P, BN), per_tile = BN / box;       // rows of a page's piece, pieces of a tile
    constexpr int NP = C::kCodes ? 1 : C::NB;              // copies per piece
    const int piece = lane / NP, blk = lane % NP;
    constexpr int NSLOT = C::kCodes ? C::NR : C::NS;
    constexpr int FULL = C::kCodes ? C::B_RFULL : C::B_FULL, EMPTY = C::kCodes ? C::B_REMPTY : C::B_EMPTY;
    uint32_t fill = 0;
    bool ok = true;
    if (k.pc.left > 0) do {
        const int n = k.take(), len = k.pc.s.len;
        // page of this lane's piece of tile j: an index into the pool, -1 for none (past the end), -2 for a bad one
        auto page_of = [&](int j) -> int {
            const int pos = j * BN + piece * box;
            if (piece >= per_tile || pos >= len) return -1;
            const int x = pg.table[(long)k.pc.n * pg.max_pages + pos / P];
            if (x >= 0 && x < pg.num_pages) return x;
            flag_error(pg.status);
            return -2;
        };
        auto issue = [&](int j, int page, bool is_v) {
            const int s = fill % NSLOT;
            ok = warp_wait(bar + EMPTY + s, ((fill / NSLOT) & 1) ^ 1, p.budget);
            if (!ok) return;
            const int pos = j * BN + piece * box, row0 = pos & (P - 1);
            if constexpr (!C::kCodes) {
                const int pieces = __popc(__ballot_sync(0xffffffffu, page != -1 && blk == 0));
                if (lane == 0) mbar_expect_tx(bar + FULL + s, (uint32_t)pieces * box * D * 2);
                __syncwarp();
                // a bad page is read at a coordinate outside of the map: zeros
                if (page != -1)
                    tma_load_3d(sm + s * C::SLOT + blk * (BN * 128) + piece * (box * 128), is_v ? mv : mk, blk * 64, row0,
                                page == -2 ? -1 : page * pg.Hkv + k.pc.h, bar + FULL + s);
            } else {
                const bool live = page >= 0;
                const uint32_t rows = live ? (uint32_t)min(box, len - pos) : 0u;
                const uint32_t srows = (rows + 3) & ~3u;  // scales: whole 16-byte pieces, within the page
                uint32_t bytes = rows * D + (is_v ? 0 : 2 * srows * 4);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, d);
                const unsigned mask = __ballot_sync(0xffffffffu, live);
                uint8_t *raw = sm + C::SM_RAW + s * C::RAW;
                if (lane == 0) {
                    reinterpret_cast<int2 *>(sm + C::SM_INFO)[s] = make_int2(min(BN, len - j * BN), (int)mask);
                    mbar_expect_tx(bar + FULL + s, bytes);
                }
                __syncwarp();
                if (live) {
                    const long at = ((long)page * pg.Hkv + k.pc.h) * P + row0;
                    bulk_load(raw + piece * box * D, (is_v ? p.v_cache : p.k_cache) + at * D, rows * D, bar + FULL + s);
                    if (!is_v) {
                        bulk_load(raw + BN * D + piece * box * 4, p.k_scale + at, srows * 4, bar + FULL + s);
                        bulk_load(raw + BN * D + BN * 4 + piece * box * 4, p.v_scale + at, srows * 4, bar + FULL + s);
                    }
                }
            }
            ++fill;
        };
        int next = page_of(k.pc.off), cur = -1, prev = -1;
        for (int jj = 0; jj <= n && ok; ++jj) {
            if (jj < n) {
                cur = next;
                if (jj + 1 < n) next = page_of(k.pc.off + jj + 1);
                issue(k.pc.off + jj, cur, false);
            }
            if (jj > 0 && ok) issue(k.pc.off + jj - 1, prev, true);
            prev = cur;
        }
    } while (ok && walk_next<BN>(p.w, &k));
    if (!ok && lane == 0) flag_error(pg.status);
    // the copies in flight must land before the CTA leaves, also if another warp has given up
    for (uint32_t f = fill > NSLOT ? fill - NSLOT : 0; f < fill; ++f)
        mbar_wait(bar + FULL + f % NSLOT, (f / NSLOT) & 1, kDrainBudget);
    __syncwarp();
}

// ---- products ---------------------------------------------------------------------
template <int D, int KIND>
__device__ void mma_role(const TcParams &p, uint8_t *sm, uint32_t sb, uint64_t *bar, Walk k, uint32_t tmem) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN;
    constexpr uint32_t ID_S = C::kCodes ? idesc_f16(128, BN, 0, 0) : idesc_bf16(128, BN, 0, 0);
    constexpr uint32_t ID_O = C::kCodes ? idesc_f16(128, D, 0, 1) : idesc_bf16(128, D, 0, 1);
    const int lane = threadIdx.x & 31;
    uint32_t fill = 0, it = 0, unit = 0;
    bool ok = true;
    if (k.pc.left > 0) do {
        const int n = k.take();
        ok = warp_wait_spin(bar + C::B_Q, unit & 1, p.budget);
        ++unit;
        for (int jj = 0; jj <= n && ok; ++jj) {
            if (jj < n) {
                const uint32_t s = fill % C::NS, b = (it + jj) & 1;
                ok = warp_wait_spin(bar + C::B_FULL + s, (fill / C::NS) & 1, p.budget);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_f16_ts(tmem + C::TM_S + b * BN, tmem + C::TM_Q + 8 * ks,
                                   desc_sw128(sb + s * C::SLOT + (ks >> 2) * (BN * 128) + (ks & 3) * 32, 16, 1024), ID_S,
                                   ks > 0);
                    mma_commit(bar + C::B_EMPTY + s);
                    mma_commit(bar + C::B_S + b);
                }
                ++fill;
            }
            if (jj > 0) {
                const uint32_t s = fill % C::NS, b = (it + jj - 1) & 1;
                ok = warp_wait_spin(bar + C::B_FULL + s, (fill / C::NS) & 1, p.budget);
                if (!ok) break;
                if constexpr (!C::kCodes) {
                    const int valid = k.pc.s.len - (k.pc.off + jj - 1) * BN;
                    if (valid < BN) {  // rows of V past the end: zeros
                        const int dead = (BN - valid) * 8;
                        for (int e = lane; e < dead * C::NB; e += 32)
                            *reinterpret_cast<uint4 *>(sm + s * C::SLOT + (e / dead) * (BN * 128) + valid * 128 +
                                                       (e % dead) * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                }
                ok = warp_wait_spin(bar + C::B_P + b, ((it + jj - 1) >> 1) & 1, p.budget);
                if (!ok) break;
                tc_fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int ks = 0; ks < BN / 16; ++ks)
                        mma_f16_ts(tmem + C::TM_O, tmem + C::TM_S + b * BN + 8 * ks,
                                   desc_sw128(sb + s * C::SLOT + ks * 2048, BN * 128, 1024), ID_O, jj > 1 || ks > 0);
                    mma_commit(bar + C::B_EMPTY + s);
                    mma_commit(bar + C::B_PV + b);
                }
                ++fill;
            }
            __syncwarp();
        }
        it += n;
    } while (ok && walk_next<BN>(p.w, &k));
    if (!ok && lane == 0) flag_error(p.w.pg.status);
    if (lane == 0) {  // all products done before TMEM is given back
        mma_commit(bar + C::B_FIN);
        mbar_wait(bar + C::B_FIN, 0, kDrainBudget);
    }
    __syncwarp();
}

// ---- 8-bit tiles to fp16 --------------------------------------------------------------
template <int KIND>
__device__ __forceinline__ void codes4_to_f16(uint32_t c, uint32_t *h) {
    if constexpr (KIND == GDN_FP8) {
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
        h[0] = (uint32_t)a.x | ((uint32_t)a.y << 16);
        h[1] = (uint32_t)b.x | ((uint32_t)b.y << 16);
    } else {
        // c + 128 as the low byte of an fp16 in [1024, 2048), whose unit is 1; minus 1152 gives c, exactly
        const uint32_t u = c ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half((unsigned short)0x6480));
        uint32_t w0 = __byte_perm(u, 0x64646464u, 0x4140), w1 = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&w0), bias), y = __hsub2(*reinterpret_cast<__half2 *>(&w1), bias);
        h[0] = *reinterpret_cast<const uint32_t *>(&x);
        h[1] = *reinterpret_cast<const uint32_t *>(&y);
    }
}

template <int D, int KIND>
__device__ void convert_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, NT = kConvWarps * 32;
    const int tid = threadIdx.x - kConvWarp0 * 32, lane = tid & 31;
    const int P = p.w.pg.page_size, box_shift = 31 - __clz(min(P, BN));
    uint32_t fill = 0, tile = 0;
    bool ok = true;
    if (k.pc.left > 0) do {
        const int n = k.take();
        for (int jj = 0; jj <= n && ok; ++jj) {
#pragma unroll 1
            for (int is_v = 0; is_v < 2 && ok; ++is_v) {
                if (is_v ? jj == 0 : jj == n) continue;
                const uint32_t r = fill % C::NR, s = fill % C::NS;
                ok = warp_wait(bar + C::B_RFULL + r, (fill / C::NR) & 1, p.budget) &&
                     warp_wait(bar + C::B_EMPTY + s, ((fill / C::NS) & 1) ^ 1, p.budget);
                if (!ok) break;
                const uint8_t *raw = sm + C::SM_RAW + r * C::RAW;
                uint8_t *dst = sm + s * C::SLOT;
                const int2 info = reinterpret_cast<const int2 *>(sm + C::SM_INFO)[r];
                // 16 codes a step. Eight lanes take the halves (4 pieces) of two rows that lie in
                // different banks of both the codes and the swizzled tile.
#pragma unroll 4
                for (int e = tid; e < BN * D / 16; e += NT) {
                    const int i = e & 7, g = e >> 3;
                    const int row = 2 * (g / C::NB) + (i >> 2);
                    const int blk = C::NB == 1 ? 0 : (g % C::NB) ^ (i >> 2), c = i & 3;
                    uint4 q = *reinterpret_cast<const uint4 *>(raw + row * D + blk * 64 + c * 16);
                    if (row >= info.x || !((info.y >> (row >> box_shift)) & 1)) q = make_uint4(0, 0, 0, 0);
                    uint32_t h[8];
                    codes4_to_f16<KIND>(q.x, h);
                    codes4_to_f16<KIND>(q.y, h + 2);
                    codes4_to_f16<KIND>(q.z, h + 4);
                    codes4_to_f16<KIND>(q.w, h + 6);
                    uint8_t *d = dst + blk * (BN * 128);
                    *reinterpret_cast<uint4 *>(d + swz(row, 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(d + swz(row, 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
                if (!is_v) {
                    const uint32_t cb = tile % C::COLS;
                    if (tid < BN) {
                        const float *sc = reinterpret_cast<const float *>(raw + BN * D);
                        const bool live = tid < info.x && ((info.y >> (tid >> box_shift)) & 1);
                        const float ks = live ? sc[tid] : 0.f;
                        float vs = live ? sc[BN + tid] : kMinKvScale;
                        if (vs < kMinKvScale) vs = kMinKvScale;  // (a NaN stays)
                        float *col = reinterpret_cast<float *>(sm + C::SM_COL) + cb * 3 * BN;
                        col[tid] = ks * p.scale2;
                        col[BN + tid] = log2f(vs);
                        col[2 * BN + tid] = 1.f / vs;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar + C::B_COL + cb);
                    ++tile;
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar + C::B_FULL + s);
                    mbar_arrive(bar + C::B_REMPTY + r);
                }
                ++fill;
            }
        }
    } while (ok && walk_next<BN>(p.w, &k));
    if (!ok && lane == 0) flag_error(p.w.pg.status);
}

// ---- softmax, rescaling, output -----------------------------------------------------------
template <int D, int KIND>
__device__ void soft_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k, uint32_t tmem) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, HC = C::HC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = warp >> 2, pair = warp & 3, row = pair * 32 + lane;
    const int bar_id = 1 + pair;
    const uint32_t tl = tmem + ((uint32_t)(pair * 32) << 16);  // this warp's TMEM lanes
    float(*xch)[2][128] = reinterpret_cast<float(*)[2][128]>(sm + C::SM_X);
    uint32_t it = 0, turn = 0;
    // A wait that ran out is shared with the row's other warp at the next exchange, so that both leave there
    // (`failed` is the same for all their threads, `late` is a thread's own).
    bool failed = false, late = false;
    if (k.pc.left > 0) do {
        const int n = k.take(), t0 = k.pc.i * p.w.TPT;
        const int rows = min(p.w.TPT, k.pc.s.T - t0) * p.w.G;
        const bool live_warp = pair * 32 < rows;
        const int t = t0 + row / p.w.G, h = k.pc.h * p.w.G + row % p.w.G;
        const int limit = row < rows ? k.pc.s.len - k.pc.s.T + t : -1;  // last position the row sees
        const int sure = k.pc.s.len - k.pc.s.T + t0;                    // ... and every row of the unit
        float rs = 1.f;  // power of two that Q's row was divided by (8-bit caches)
        if (live_warp) {  // Q to TMEM: 16-bit pairs, D / 4 columns of this half
            constexpr int W = D / 4;
            uint32_t r[W];
#pragma unroll
            for (int c = 0; c < W; ++c) r[c] = 0;
            if (row < rows) {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (k.pc.s.bos + t) * p.q_stride + (long)h * D + g * (D / 2));
#pragma unroll
                for (int c = 0; c < W / 4; ++c) {
                    const uint4 x = __ldg(src + c);
                    r[4 * c] = x.x; r[4 * c + 1] = x.y; r[4 * c + 2] = x.z; r[4 * c + 3] = x.w;
                }
            }
            if constexpr (C::kCodes) {
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < W; ++c)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(r[c] << 16)), fabsf(__uint_as_float(r[c] & 0xffff0000u))));
                xch[turn & 1][g][row] = amax;
                bar_any(bar_id, 64, false);
                amax = fmaxf(amax, xch[turn & 1][g ^ 1][row]);
                ++turn;
                // amax 2^e in [2^13, 2^14): the largest elements far from overflow, the smallest normal
                int e = 13 - ((int)(__float_as_uint(amax) >> 23) - 127);
                if (!(amax > 0.f && amax < 3.4e38f)) e = 0;
                e = max(-100, min(100, e));
                const float f = __uint_as_float((uint32_t)(127 + e) << 23);
                rs = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                for (int c = 0; c < W; ++c)
                    r[c] = h2_bits(f * __uint_as_float(r[c] << 16), f * __uint_as_float(r[c] & 0xffff0000u));
            }
            if (p.negate)
#pragma unroll
                for (int c = 0; c < W; ++c) r[c] ^= 0x80008000u;
#pragma unroll
            for (int c = 0; c < W; c += 16) tmem_st16(tl + C::TM_Q + g * W + c, r + c);
            tmem_wait_st();
            tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::B_Q);
        float m = -INFINITY, l = 0.f;
        for (int jj = 0; jj < n && !failed; ++jj, ++it) {
            const uint32_t b = it & 1, ph = (it >> 1) & 1;
            late |= !mbar_wait(bar + C::B_S + b, ph, p.budget);
            if constexpr (C::kCodes) late = late || !mbar_wait(bar + C::B_COL + it % C::COLS, (it / C::COLS) & 1, p.budget);
            if (!live_warp) {
                failed = __any_sync(0xffffffffu, late);
                if (lane == 0 && !failed) mbar_arrive(bar + C::B_P + b);
                continue;
            }
            tc_fence_after();
            const int c0 = (k.pc.off + jj) * BN + g * HC;  // position of this thread's first column
            float x[HC];
            {
                uint32_t r[HC];
#pragma unroll
                for (int c = 0; c < HC; c += 32) tmem_ld32_nw(tl + C::TM_S + b * BN + g * HC + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < HC; ++c) x[c] = __uint_as_float(r[c]);
            }
            const float *col = reinterpret_cast<const float *>(sm + C::SM_COL) + (it % C::COLS) * 3 * BN + g * HC;
            if constexpr (C::kCodes) {
#pragma unroll
                for (int c = 0; c < HC; c += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(col + c), lv = *reinterpret_cast<const float4 *>(col + BN + c);
                    x[c] = fmaf(x[c] * rs, a.x, lv.x);
                    x[c + 1] = fmaf(x[c + 1] * rs, a.y, lv.y);
                    x[c + 2] = fmaf(x[c + 2] * rs, a.z, lv.z);
                    x[c + 3] = fmaf(x[c + 3] * rs, a.w, lv.w);
                }
            }
            if ((k.pc.off + jj + 1) * BN - 1 > sure) {
#pragma unroll
                for (int c = 0; c < HC; ++c)
                    if (c0 + c > limit) x[c] = -INFINITY;
            }
            float top = x[0];
#pragma unroll
            for (int c = 1; c < HC; ++c) top = fmaxf(top, x[c]);
            xch[turn & 1][g][row] = top;
            failed = bar_any(bar_id, 64, late);
            if (failed) break;
            top = fmaxf(top, xch[turn & 1][g ^ 1][row]);
            ++turn;
            const float sc = C::kCodes ? 1.f : p.scale2;
            const float mt = top * sc;
            const bool grow = mt > m + kGrow || (m == -INFINITY && mt > m);
            const float f = grow ? ex2(m - mt) : 1.f;  // m = -inf: 0
            if (grow) {
                m = mt;
                l *= f;
            }
            if (jj > 0 && __any_sync(0xffffffffu, grow)) {
                // O holds the tiles up to jj - 1
                late |= !mbar_wait(bar + C::B_PV + ((it - 1) & 1), ((it - 1) >> 1) & 1, p.budget);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    uint32_t r[32];
                    tmem_ld32_nw(tl + C::TM_O + g * (D / 2) + c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                    tmem_st32(tl + C::TM_O + g * (D / 2) + c, r);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            uint32_t pk[HC / 2];
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int c = 0; c < HC; c += 2) {
                const float e0 = ex2(C::kCodes ? x[c] - ref : fmaf(x[c], sc, -ref));
                const float e1 = ex2(C::kCodes ? x[c + 1] - ref : fmaf(x[c + 1], sc, -ref));
                if constexpr (C::kCodes) {
                    const float2 iv = *reinterpret_cast<const float2 *>(col + 2 * BN + c);
                    l0 = fmaf(e0, iv.x, l0);
                    l1 = fmaf(e1, iv.y, l1);
                    pk[c / 2] = h2_bits(e0, e1);
                } else {
                    l0 += e0;
                    l1 += e1;
                    pk[c / 2] = bf2(e0, e1);
                }
            }
            l += l0 + l1;
#pragma unroll
            for (int c = 0; c < HC / 2; c += 16) tmem_st16(tl + C::TM_S + b * BN + g * (HC / 2) + c, pk + c);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_P + b);
        }
        if (failed) break;
        // the unit's last product, then the row
        late |= !mbar_wait(bar + C::B_PV + ((it - 1) & 1), ((it - 1) >> 1) & 1, p.budget);
        if (live_warp) {
            tc_fence_after();
            xch[turn & 1][g][row] = l;
            failed = bar_any(bar_id, 64, late);
            if (failed) break;
            l += xch[turn & 1][g ^ 1][row];
            ++turn;
            const bool whole = k.begun && k.pc.off + n == k.pc.ntiles;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool store = row < rows && (!whole || limit >= 0);
            const long part = part_index(p.w, blockIdx.x, k.begun ? 1 : 0, row);
            if (!whole && row < rows && g == 0) p.w.ml[part] = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < D / 2; c += 32) {
                float o[32];
                tmem_ld32(tl + C::TM_O + g * (D / 2) + c, o);
                if (!store) continue;
                const int at = g * (D / 2) + c;
                if (whole) {
                    uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((k.pc.s.bos + t) * p.Hq + h) * D + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float *y = o + 8 * e;
                        dst[e] = make_uint4(bf2(y[0] * inv, y[1] * inv), bf2(y[2] * inv, y[3] * inv),
                                            bf2(y[4] * inv, y[5] * inv), bf2(y[6] * inv, y[7] * inv));
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.w.part + part * D + at);
#pragma unroll
                    for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            }
            tc_fence_before();
        } else {
            failed = __any_sync(0xffffffffu, late);
            if (failed) break;
        }
    } while (walk_next<BN>(p.w, &k));
    if (failed && lane == 0) flag_error(p.w.pg.status);
}

template <int D, int KIND>
__global__ void __launch_bounds__(Cfg<D, KIND>::THREADS, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const TcParams p) {
    using C = Cfg<D, KIND>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *sm = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::SM_BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + C::SM_TMEM);
    PlanSmem *plan = reinterpret_cast<PlanSmem *>(sm + C::SM_PLAN);
    const int tid = threadIdx.x, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(bar + C::B_FULL + s, C::kCodes ? kConvWarps : 1);
            mbar_init(bar + C::B_EMPTY + s, 1);
        }
        for (int s = 0; s < C::NR; ++s) {
            mbar_init(bar + C::B_RFULL + s, 1);
            mbar_init(bar + C::B_REMPTY + s, kConvWarps);
        }
        for (int s = 0; s < C::COLS; ++s) mbar_init(bar + C::B_COL + s, kConvWarps);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + C::B_S + s, 1);
            mbar_init(bar + C::B_P + s, kSoftWarps);
            mbar_init(bar + C::B_PV + s, 1);
        }
        mbar_init(bar + C::B_Q, kSoftWarps);
        mbar_init(bar + C::B_FIN, 1);
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc(slot, 512);
    tc_fence_before();
    plan_piece<C::BN, C::THREADS>(p.w, plan);  // (synchronises the CTA)
    tc_fence_after();
    const uint32_t tmem = *slot;
    Walk k{plan->piece, plan->piece.off == 0};
    if (warp < kSoftWarps) {
        soft_role<D, KIND>(p, sm, bar, k, tmem);
    } else if (warp == kLoadWarp) {
        load_role<D, KIND>(p, sm, bar, k, &mk, &mv);
    } else if (warp == kMmaWarp) {
        zero_padding(p.w, p.out, p.Hq, D, tid & 31, 32);  // while the first tiles are on their way
        mma_role<D, KIND>(p, sm, sb, bar, k, tmem);
    } else if constexpr (C::kCodes) {
        convert_role<D, KIND>(p, sm, bar, k);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---- host side ------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
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

// [page, head][page_size][d] bf16 -> 3-D map, box (64 elements, `rows` positions, 1), 128B swizzle
bool page_map(CUtensorMap *m, const void *base, const KvPages &pg, int rows) {
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    const cuuint64_t gdim[3] = {(cuuint64_t)pg.d, (cuuint64_t)pg.page_size, (cuuint64_t)pg.num_pages * pg.Hkv};
    const cuuint64_t gstride[2] = {(cuuint64_t)pg.d * 2, (cuuint64_t)pg.page_size * pg.d * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), gdim, gstride, box, estride,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
    using C = Cfg<D, KIND>;
    const int G = a.Hq / a.pg.Hkv;
    TcParams p{};
    p.w = attn_work(a, kAttnMaxRows / G, 2);
    p.q = (const __nv_bfloat16 *)a.q;
    p.k_cache = (const uint8_t *)a.k_cache;
    p.v_cache = (const uint8_t *)a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.out = (__nv_bfloat16 *)a.out;
    p.Hq = a.Hq;
    p.q_stride = a.q_stride;
    p.negate = a.scale < 0.f;
    // a scale of 0 must not meet the -inf of a masked score in a product: so small that no score counts
    p.scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
    p.budget = kWaitDefault;
    if (const char *env = getenv("GDN_TEST_WAIT_CYCLES")) {  // test hook: a short limit makes the waits run out
        const long long x = atoll(env);
        if (x > 0) p.budget = x;
    }
    CUtensorMap mk{}, mv{};
    if (!C::kCodes) {
        const int rows = a.pg.page_size < C::BN ? a.pg.page_size : C::BN;
        if (!page_map(&mk, a.k_cache, a.pg, rows) || !page_map(&mv, a.v_cache, a.pg, rows)) return cudaErrorInvalidValue;
    }
    auto kernel = attn_tc_kernel<D, KIND>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    kernel<<<kAttnCtas, C::THREADS, C::SM_BYTES, s>>>(mk, mv, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_join(a, p.w, s);
}

template <int KIND>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.d) {
        case 64: return launch_t<64, KIND>(a, s);
        case 128: return launch_t<128, KIND>(a, s);
        case 256: return launch_t<256, KIND>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.cache_dtype) {
        case GDN_FP8: return launch_d<GDN_FP8>(a, s);
        case GDN_INT8: return launch_d<GDN_INT8>(a, s);
        default: return launch_d<GDN_BF16>(a, s);
    }
}

}  // namespace gdn
