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
// What bounds it. A prompt's fragment (128 rows full): 4 BN D 128 flops a tile against 4 BN D bytes, so
// the tensor cores, if the softmax of one tile hides behind the products of its neighbours and L2 keeps
// up with 64 KB per SM and tile (D = 256: 13.4 TB/s without the softmax). With 8-bit caches it is shared
// memory: per tile of 128 positions at D = 128 the codes are read (256 cycles), written as fp16 (512),
// read by the products (480) and scaled by columns (770), 85% of its cycles.
//
// Measured, 2048 tokens over 32768, 16 query heads on 2: bf16 651, 355 and 328 us for D = 256, 128 and
// 64 (1.64 PFLOP/s for 256, of 1.92 measured; 712 us and 1.50 PFLOP/s in a run so long that power caps the
// clock), e4m3 875 us for 256 and 637 for 128 (int8 668). 8 prompts of 1024 tokens, 32 heads on 8, D = 128:
// bf16 101, e4m3 203 us: 14 units of 4 or 5 tiles per CTA, whose starts and ends (Q in, rows out) count for
// half of it. The kernels of 8-bit caches spill 76 to 118 bytes of stores a thread (for trees 104 to 132): 768 threads leave 80
// registers, and the softmax, which has 112 when it runs, is compiled within them.
//
// Layout. TMEM holds O (D columns), two S buffers (P_j overlays S_j) and Q as the 16-bit A operand,
// 512 columns in all for D = 256 (and for D = 128 with the next unit's Q beside it); with Q in TMEM,
// shared memory is two rings of K and V tiles, and the S products read 64 bytes of it a cycle instead
// of 192.
//
// Warps, in groups of four: two take the softmax, a thread per row and half of a tile's columns, which
// meet once per tile for the row's maximum; one brings the rows' Q into TMEM and takes finished rows
// out, beside the softmax of the neighbouring units; one has a warp each for the loads of K and V, for
// the products and, with a bf16 cache, for a look through V; with an 8-bit cache one converts K tiles
// and one V tiles. The products run S_0, S_1, O(0), S_2, O(1), .. across units, so that the tensor cores
// work on S_{j+1} while the softmax of tile j runs. All CTAs are persistent over their piece of the work,
// and every wait has a limit, after which the CTA flags the status word and leaves.
//
// 8-bit caches. Codes are exact in fp16, so K and V tiles hold codes converted to fp16 (bf16 would
// take four times the conversion instructions for e4m3), Q is rounded to fp16 after an exact
// power-of-two scaling per row, and the cached rows' scales enter in fp32: with a_j = ks_j scale
// log2 e and b_j = log2 vs_j,   y_j = (q.c_j) a_j + b_j,   P'_j = exp2(y_j - m') = P_j vs_j,
//     O += P'_j C_j,   l += P'_j / vs_j.
// Taking vs_j into the exponent keeps P' near 1 for the keys that matter whatever the scales' range. (l
// needs P_j itself of tiles whose scales are very small or large: plain_reciprocal.)
//
// Masks. A row sees positions up to its own; scores past it are replaced (not multiplied), so what
// K holds there has no effect. Of V, where 0 * NaN would reach the sum (bf16 caches; codes are finite):
// steps of 16 positions that no row of the unit sees are left out of the product, positions past the
// sequence's end are zeroed in shared memory, and from the first row's last position on elements that
// are not finite are taken as 0 and added to the rows that see them when these leave.
#include <type_traits>

#include "attn_ops.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kGroup = 4, kRowWarp0 = 8, kLoadWarp = 12 /* K, then V */, kMmaWarp = 14,
              kConvWarp0 = 16 /* K, then V */;
// With the converting groups the launch gives a thread 80 registers; the softmax groups, whose threads hold 64
// scores, take what the converting groups leave of theirs: 2 * 112 + 2 * 80 + 2 * 48 = 6 * 80.
constexpr int kSoftRegs = 112, kConvRegs = 48;

template <int D, int KIND>
struct Cfg {
    static constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    static constexpr int BN = D == 256 ? 64 : 128;
    static constexpr int NB = D / 64;                      // 128-byte wide blocks of a tile
    static constexpr uint32_t SLOT = BN * D * 2;           // a 16-bit K or V tile
    static constexpr uint32_t RAW_K = BN * D + 2 * BN * 4;  // a K tile's codes, and K and V scales
    static constexpr uint32_t RAW_V = BN * D;
    // ring slots: 16-bit tiles of K and of V, and with an 8-bit cache their codes
    static constexpr int NK = kCodes ? 2 : (D == 64 ? 6 : 3), NV = NK;
    static constexpr int NR = kCodes ? (D == 64 ? 6 : 2) : 0;
    static constexpr int COLS = 4;                         // column scales, a buffer per tile
    static constexpr int THREADS = 32 * (kCodes ? kConvWarp0 + 2 * kGroup : kConvWarp0);
    static constexpr uint32_t TM_O = 0, TM_S = D == 256 ? 256 : 128, TM_Q = 384;
    // Where there is room, the next unit's Q is put beside the one in use, so that its products follow without a gap.
    static constexpr int NQ = D == 256 ? 1 : 2;
    // shared memory, from a 1 KiB aligned base
    static constexpr uint32_t SM_V = NK * SLOT, SM_RK = SM_V + NV * SLOT, SM_RV = SM_RK + NR * RAW_K;
    static constexpr uint32_t SM_COL = SM_RV + NR * RAW_V;                   // [COLS][3][BN] a, b, 1 / vs
    static constexpr uint32_t SM_ODD = SM_COL + (kCodes ? COLS * 3 * BN * 4 : 0);  // [COLS][kGroup] bytes: scales out of bounds
    static constexpr uint32_t SM_X = SM_ODD + (kCodes ? COLS * kGroup : 0);  // [2][2][128] maxima of a tile's halves
    static constexpr uint32_t SM_STAT = SM_X + 2 * 2 * 128 * 4;              // [2][2][128] a unit's m, l by half
    static constexpr uint32_t SM_RS = SM_STAT + 2 * 2 * 128 * 8;             // [4][128] Q's row scales (8-bit caches)
    static constexpr uint32_t SM_Q = (SM_RS + (kCodes ? 4 * 128 * 4 : 0) + 1023) & ~1023u;  // [128 rows][128 B] of Q
    static constexpr uint32_t SM_BAR = SM_Q + 128 * 128;
    // S_j and O += P_j V_j done, by tile modulo 8: they also say that K_j's and V_j's slots are free. (Whoever fills
    // a slot looks back at most 6 tiles, so a barrier is never two phases ahead of its reader.)
    static constexpr int kTurns = 8;
    static constexpr int B_FK = 0, B_FV = B_FK + NK, B_RK = B_FV + NV, B_RV = B_RK + NR, B_REK = B_RV + NR,
                         B_REV = B_REK + NR, B_COL = B_REV + NR, B_S = B_COL + COLS, B_PV = B_S + kTurns,
                         B_P = B_PV + kTurns, B_ST = B_P + 2, B_SF = B_ST + 2,
                         B_Q = B_SF + 2, B_OF = B_Q + NQ, B_QF = B_OF + 1, B_QE = B_QF + 1,
                         B_US = B_QE + 1 /* all S of a unit */, B_UO = B_US + 1 /* all of its O */, B_FIN = B_UO + 1,
                         B_CV = B_FIN + 1 /* V looked through (bf16 caches) */, B_COUNT = B_CV + (kCodes ? 0 : NV);
    // [2][NR] valid rows, page mask; bf16 caches: [8], by unit, whether it has values that are not finite and hidden from
    // some of its rows
    static constexpr uint32_t SM_INFO = SM_BAR + B_COUNT * 8;
    static constexpr uint32_t SM_TMEM = SM_INFO + (NR ? 2 * NR : 4) * 8;
    static constexpr uint32_t SM_PLAN = (SM_TMEM + 8 + 15) & ~15u;
    static constexpr uint32_t SM_BYTES = SM_PLAN + sizeof(PlanSmem) + 1024;
    static_assert(SM_BYTES <= 232448, "over the 227 KiB opt-in limit");
};

struct TcParams {
    AttnWork w;
    const uint8_t *k_cache, *v_cache;  // 8-bit caches (and bf16 values that are not finite)
    const float *k_scale, *v_scale;
    __nv_bfloat16 *out;
    int Hq;
    float scale2;  // |softmax scale| * log2 e
    int negate;    // the scale is negative: Q is negated
    long long budget;
};

// 32 bytes to a 32-byte boundary. (A row's thread stores its own row, so a warp's store touches 32 lines whatever its
// width, and the number of stores is what a unit's rows cost.)
__device__ __forceinline__ void store32(void *to, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ uint32_t bf2(float a, float b) { return bf2_bits(__floats2bfloat162_rn(a, b)); }

// every thread's view of the walk over the piece's units
struct Walk {
    Piece pc;
    bool begun;  // the unit at hand started in this CTA
    __device__ __forceinline__ int take() const { return (int)min((long)(pc.ntiles - pc.off), pc.left); }
};
template <int BN, bool TREE>
__device__ __forceinline__ bool walk_next(const AttnWork &w, Walk *k) {
    k->pc.left -= k->take();
    if (k->pc.left <= 0) return false;
    next_unit<BN, TREE>(w, &k->pc);
    k->begun = true;
    return k->pc.left > 0;
}

// A ring's slot and phase, counted on instead of divided out of the tile's number.
template <int N>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
        }
    }
};
// Wait for tile t's S (or PV) product. The barrier's phases come round: only for a reader that follows the
// tiles closely (it knows that tile t - 8's is done, and tile t + 8's waits for itself).
template <int D, int KIND>
__device__ __forceinline__ bool product_done(uint64_t *bar, int which, uint32_t t, long long budget) {
    using C = Cfg<D, KIND>;
    return wait_for(bar + which + (t & (C::kTurns - 1)), (t / C::kTurns) & 1, budget);
}

// ---- loads ------------------------------------------------------------------------
// One warp loads K tiles, another V tiles.
template <int D, int KIND, bool TREE, bool IS_V>
__device__ void load_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k, const CUtensorMap *map) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN;
    const KvPages &pg = p.w.pg;
    const int lane = threadIdx.x & 31, P = pg.page_size, P_shift = 31 - __clz(P);
    const int box = min(P, BN), per_tile = BN / box;       // rows of a page's piece, pieces of a tile
    constexpr int NP = C::kCodes ? 1 : C::NB;              // copies per piece
    const int piece = lane / NP, blk = lane % NP;
    const bool issues = piece < per_tile;
    constexpr int N = C::kCodes ? C::NR : (IS_V ? C::NV : C::NK);
    constexpr int FULL = C::kCodes ? (IS_V ? C::B_RV : C::B_RK) : (IS_V ? C::B_FV : C::B_FK);
    const uint32_t dst0 = C::kCodes ? (uint32_t)(IS_V ? C::SM_RV : C::SM_RK) + piece * box * D
                                    : (IS_V ? C::SM_V : 0) + blk * (BN * 128) + piece * (box * 128);
    constexpr uint32_t STRIDE = C::kCodes ? (IS_V ? C::RAW_V : C::RAW_K) : C::SLOT;
    Ring<N> ring;
    uint32_t t = 0;  // tiles loaded
    bool ok = true;
    if (k.pc.left > 0) do {
        const int n = k.take(), len = k.pc.s.len;
        // The sequence's table entries, 32 pages at a time: a window in use and the next one on its way, so
        // that no tile waits for them.
        const int32_t *table = pg.table + (long)k.pc.n * pg.max_pages;
        const int used = (len + P - 1) >> P_shift;
        auto entries = [&](int window) -> int {
            const int i = window * 32 + lane;
            return i < used ? table[i] : -1;
        };
        int window = ((k.pc.off * BN) >> P_shift) >> 5, win = entries(window), win_next = entries(window + 1);
        int pos = k.pc.off * BN + piece * box;
        for (int jj = 0; jj < n; ++jj, ++t, pos += BN) {
            const int first = (pos - piece * box) >> P_shift;
            if ((first >> 5) != window) {  // (a tile's pages share a window)
                ++window;
                win = win_next;
                win_next = entries(window + 1);
            }
            const int page = __shfl_sync(0xffffffffu, win, (first + piece) & 31);
            const bool here = issues && pos < len;
            const bool good = (unsigned)page < (unsigned)pg.num_pages;
            if (here && !good) flag_error(pg.status);
            const int row0 = pos & (P - 1);
            if constexpr (C::kCodes) {
                ok = warp_wait(bar + (IS_V ? C::B_REV : C::B_REK) + ring.slot, ring.phase ^ 1, p.budget);
            } else if (t >= N) {
                ok = __all_sync(0xffffffffu, product_done<D, KIND>(bar, IS_V ? C::B_PV : C::B_S, t - N, p.budget));
            }
            if (!ok) break;
            if constexpr (!C::kCodes) {
                // pieces past the end are left out; a bad page is read outside of the map: zeros
                const int left = len - (pos - piece * box);
                const int pieces = left >= BN ? per_tile : (left + box - 1) / box;
                if (lane == 0) mbar_expect_tx(bar + FULL + ring.slot, (uint32_t)pieces * box * D * 2);
                __syncwarp();
                if (here)
                    tma_load_3d(sm + dst0 + ring.slot * STRIDE, map, blk * 64, row0, good ? page * pg.Hkv + k.pc.h : -1,
                                bar + FULL + ring.slot);
            } else {
                const bool live = here && good;
                const uint32_t rows = live ? (uint32_t)min(box, len - pos) : 0u;
                const uint32_t srows = (rows + 3) & ~3u;  // scales: whole 16-byte pieces, within the page
                uint32_t bytes = rows * D + (IS_V ? 0 : 2 * srows * 4);
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) bytes += __shfl_xor_sync(0xffffffffu, bytes, d);  // at most 8 pieces
                const unsigned mask = __ballot_sync(0xffffffffu, live);
                uint8_t *raw = sm + dst0 + ring.slot * STRIDE;
                if (lane == 0) {
                    reinterpret_cast<int2 *>(sm + C::SM_INFO)[(IS_V ? C::NR : 0) + ring.slot] = make_int2(min(BN, len - pos), (int)mask);
                    mbar_expect_tx(bar + FULL + ring.slot, bytes);
                }
                __syncwarp();
                if (live) {
                    const long at = ((long)page * pg.Hkv + k.pc.h) * P + row0;
                    bulk_load(raw, (IS_V ? p.v_cache : p.k_cache) + at * D, rows * D, bar + FULL + ring.slot);
                    if (!IS_V) {
                        uint8_t *sc = raw - piece * box * D + BN * D + piece * box * 4;
                        bulk_load(sc, p.k_scale + at, srows * 4, bar + FULL + ring.slot);
                        bulk_load(sc + BN * 4, p.v_scale + at, srows * 4, bar + FULL + ring.slot);
                    }
                }
            }
            ring.next();
        }
    } while (ok && walk_next<BN, TREE>(p.w, &k));
    if (!ok && lane == 0) flag_error(pg.status);
    // the copies in flight must land before the CTA leaves, also if another warp has given up
    for (uint32_t f = t > N ? t - N : 0; f < t; ++f) mbar_wait(bar + FULL + f % N, (f / N) & 1, kDrainBudget);
    __syncwarp();
}

// ---- products ---------------------------------------------------------------------
// One lane issues everything, in the order S_0, S_1, O(0), S_2, O(1), .. over all units: what stands
// between two products is time that the tensor cores may stand still, so the warp walks together
// (descriptors in uniform registers), slots and phases are counted on instead of divided out, and each
// product signals one barrier.
template <int D, int KIND, bool TREE>
__device__ void mma_role(const TcParams &p, uint8_t *sm, uint32_t sb, uint64_t *bar, Walk k, uint32_t tmem) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN;
    constexpr uint32_t ID_S = C::kCodes ? idesc_f16(128, BN, 0, 0) : idesc_bf16(128, BN, 0, 0);
    constexpr uint32_t ID_O = C::kCodes ? idesc_f16(128, D, 0, 1) : idesc_bf16(128, D, 0, 1);
    const int lane = threadIdx.x & 31;
    const uint32_t lead = elect_one();
    const uint64_t desc_k = desc_sw128(sb, 16, 1024), desc_v = desc_sw128(sb + C::SM_V, BN * 128, 1024);  // of slots 0
    Ring<C::NK> rk;
    Ring<C::NV> rv;
    Ring<C::NQ> rq;
    uint32_t t = 0, qslot = 0, o_free = 0;  // tiles whose S is issued, the unit's Q, phase of B_OF
    // The waits for tiles come before the one for P, which is the last to be met: what follows it is issued at once.
    auto k_ready = [&]() -> bool { return warp_wait(bar + C::B_FK + rk.slot, rk.phase, p.budget); };
    auto product_s = [&](bool last) {
        tc_fence_after();
        const uint64_t d = desc_k + (uint64_t)(rk.slot * (C::SLOT >> 4));
        const uint32_t to = tmem + C::TM_S + (t & 1) * BN, tq = tmem + C::TM_Q + qslot * (D / 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
            mma_f16_ts_by(lead, to, tq + 8 * ks, d + (uint64_t)(((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4),
                          ID_S, ks > 0);
        mma_commit_by(lead, bar + C::B_S + (t & (C::kTurns - 1)));
        if (C::NQ == 1 && last) mma_commit_by(lead, bar + C::B_US);
        rk.next();
        ++t;
    };
    // V of tile o, `first` of its unit, ready to be multiplied
    auto v_ready = [&](uint32_t o, bool first) -> bool {
        if (!warp_wait(bar + (C::kCodes ? C::B_FV : C::B_CV) + rv.slot, rv.phase, p.budget)) return false;
        if (first && o > 0) {  // the unit before has been taken out of O
            if (!warp_wait(bar + C::B_OF, o_free, p.budget)) return false;
            o_free ^= 1;
        }
        return true;
    };
    auto product_o = [&](uint32_t o, bool first, bool last, int seen) -> bool {
        if (!warp_wait(bar + C::B_P + (o & 1), (o >> 1) & 1, p.budget)) return false;
        tc_fence_after();
        const uint64_t d = desc_v + (uint64_t)(rv.slot * (C::SLOT >> 4));
        const uint32_t a = tmem + C::TM_S + (o & 1) * BN;
        auto step = [&](int ks) {
            mma_f16_ts_by(lead, tmem + C::TM_O, a + (ks < BN / 32 ? 8 * ks : BN / 2 + 8 * (ks - BN / 32)),
                          d + (uint64_t)(ks * 128), ID_O, !first || ks > 0);
        };
        if (C::kCodes || seen >= BN) {
#pragma unroll
            for (int ks = 0; ks < BN / 16; ++ks) step(ks);
        } else {
#pragma unroll 1
            for (int ks = 0; 16 * ks < seen; ++ks) step(ks);
        }
        mma_commit_by(lead, bar + C::B_PV + (o & (C::kTurns - 1)));
        if (last) {
            mma_commit_by(lead, bar + C::B_UO);
            if (!C::kCodes) {
                if (lane == 0) mbar_arrive(bar + C::B_UO);
                __syncwarp();
            }
        }
        rv.next();
        return true;
    };
    bool ok = true, prev_first = false, prev_last = false;
    int prev_seen = BN;
    if (k.pc.left > 0) {
        do {
            const int n = k.take();
            // positions that a row of the unit sees, from the piece's first on
            const int seen = k.pc.s.len - max(k.pc.s.T - (k.pc.i + 1) * p.w.TPT, 0) - k.pc.off * BN;
            ok = warp_wait(bar + C::B_Q + rq.slot, rq.phase, p.budget) && (t > 0 || k_ready());
            qslot = rq.slot;
            rq.next();
            for (int jj = 0; jj < n && ok; ++jj) {
                const bool more = jj + 1 < n || k.pc.left > n;  // another tile follows in the piece
                product_s(jj + 1 == n);
                if (t > 1) ok = v_ready(t - 2, prev_first) && product_o(t - 2, prev_first, prev_last, prev_seen);
                if (ok && more) ok = k_ready();
                prev_first = jj == 0;
                prev_last = jj + 1 == n;
                prev_seen = seen - jj * BN;
            }
        } while (ok && walk_next<BN, TREE>(p.w, &k));
        ok = ok && v_ready(t - 1, prev_first) && product_o(t - 1, prev_first, true, prev_seen);
    }
    if (!ok && lane == 0) flag_error(p.w.pg.status);
    mma_commit_by(lead, bar + C::B_FIN);  // all products done before TMEM is given back
    mbar_wait(bar + C::B_FIN, 0, kDrainBudget);
    __syncwarp();
}

// ---- V of bf16 caches, looked through ---------------------------------------------------
// One warp passes V tiles on to the products, and on its way looks through what not all of a unit's rows see: elements
// that are not finite become zeros (the rows group adds them to the rows that see them), and so do positions past the
// end. (8 prompts of 1024 tokens, 32 heads on 8, D = 128: 100 us without such a look, 102 by this warp, 117 by the one
// that issues the products.)
template <int D, int KIND, bool TREE>
__device__ void check_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, PR = 8 * C::NB;  // 16-byte pieces of a row
    const int lane = threadIdx.x & 31;
    int *flags = reinterpret_cast<int *>(sm + C::SM_INFO);
    Ring<C::NV> ring;
    uint32_t unit = 0;
    bool ok = true;
    if (k.pc.left > 0) do {
        const int n = k.take(), t0 = k.pc.i * p.w.TPT;
        // of the tile's positions: those before the end, those that every row sees, those that a row sees
        int valid = k.pc.s.len - k.pc.off * BN, sure = valid - k.pc.s.T + (TREE ? 0 : t0 + 1);
        int seen = valid - k.pc.s.T + t0 + min(p.w.TPT, k.pc.s.T - t0);
        bool dropped = false;
        for (int jj = 0; jj < n; ++jj, valid -= BN, sure -= BN, seen -= BN) {
            ok = warp_wait(bar + C::B_FV + ring.slot, ring.phase, p.budget);
            if (!ok) break;
            if (sure < BN) {
                uint8_t *v = sm + C::SM_V + ring.slot * C::SLOT;
                auto piece = [&](int row, int e) {
                    return reinterpret_cast<uint4 *>(v + (e % PR / 8) * (BN * 128) + (row + e / PR) * 128 + (e & 7) * 16);
                };
                const int from = max(sure, 0), end = (min(seen, BN) + 15) & ~15, to = min(end, valid);
                bool bad = false;
                const uint4 *at = piece(from, lane);
#pragma unroll 2
                for (int e = lane; e < (to - from) * PR; e += 32, at += 32 / PR * 8) bad |= any_not_finite(*at);
                if (rarely(__any_sync(0xffffffffu, bad))) {
                    for (int e = lane; e < (to - from) * PR; e += 32) drop_not_finite(piece(from, e));
                    dropped = true;
                }
                if (end > to) {
                    for (int e = lane; e < (end - to) * PR; e += 32) *piece(to, e) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                }
            }
            if (jj + 1 == n && lane == 0) flags[unit & 7] = dropped;  // (this warp is at most NV units ahead of the products)
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_CV + ring.slot);
            ring.next();
        }
        ++unit;
    } while (ok && walk_next<BN, TREE>(p.w, &k));
    if (!ok && lane == 0) flag_error(p.w.pg.status);
}

// ---- 8-bit tiles to fp16 --------------------------------------------------------------
// 16 codes a thread and step, from `raw` to the two swizzled 16-byte pieces. Eight lanes take the
// halves (4 pieces) of two rows that lie in different banks of both the codes and the tile; from
// one step to the next the row moves by a multiple of 8, which leaves the swizzle as it is.
template <int D, int KIND>
__device__ __forceinline__ void convert_tile(const uint8_t *raw, uint8_t *dst0, uint8_t *dst1, int row, int valid,
                                             int pages, int box_shift) {
    using C = Cfg<D, KIND>;
    constexpr int STEPS = C::BN * D / 16 / (kGroup * 32), ROWS = kGroup * 32 / (D / 16);
    static_assert(ROWS % 8 == 0 && STEPS % 4 == 0, "the swizzle must not change between steps");
#pragma unroll 1
    for (int st = 0; st < STEPS; st += 4) {
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = *reinterpret_cast<const uint4 *>(raw + (st + u) * ROWS * D);
        if (valid >= 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int r = row + (st + u) * ROWS;
                if (r >= valid || !((pages >> (r >> box_shift)) & 1)) q[u] = make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t h[8];
            codes4_to_f16<KIND>(q[u].x, h[0], h[1]);
            codes4_to_f16<KIND>(q[u].y, h[2], h[3]);
            codes4_to_f16<KIND>(q[u].z, h[4], h[5]);
            codes4_to_f16<KIND>(q[u].w, h[6], h[7]);
            *reinterpret_cast<uint4 *>(dst0 + (st + u) * ROWS * 128) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(dst1 + (st + u) * ROWS * 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
}

template <int D, int KIND, bool IS_V>
__device__ void convert_role(const TcParams &p, uint8_t *sm, uint64_t *bar, uint32_t tiles) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, N = IS_V ? C::NV : C::NK;
    const int tid = threadIdx.x & (kGroup * 32 - 1), lane = tid & 31;
    const int box = min(p.w.pg.page_size, BN), box_shift = 31 - __clz(box), all_pages = (1 << (BN / box)) - 1;
    const int e8 = tid & 7, g8 = tid >> 3, row0 = 2 * (g8 / C::NB) + (e8 >> 2);
    const int blk = C::NB == 1 ? 0 : (g8 % C::NB) ^ (e8 >> 2), c = e8 & 3;
    const uint8_t *src = sm + (IS_V ? C::SM_RV : C::SM_RK);
    const uint32_t src0 = row0 * D + blk * 64 + c * 16;
    uint8_t *dst = sm + (IS_V ? C::SM_V : 0) + blk * (BN * 128);
    const uint32_t dst0 = swz(row0, 2 * c), dst1 = swz(row0, 2 * c + 1);
    Ring<N> ring;
    Ring<C::NR> raw;
    bool ok = true, large = false;
    for (uint32_t t = 0; t < tiles; ++t) {  // all the piece's, whatever units they belong to
        bool got = wait_for(bar + (IS_V ? C::B_RV : C::B_RK) + raw.slot, raw.phase, p.budget);
        if (t >= N) got = got && product_done<D, KIND>(bar, IS_V ? C::B_PV : C::B_S, t - N, p.budget);
        ok = __all_sync(0xffffffffu, got);
        if (!ok) break;
        const uint8_t *from = src + raw.slot * (IS_V ? C::RAW_V : C::RAW_K);
        const int2 info = reinterpret_cast<const int2 *>(sm + C::SM_INFO)[(IS_V ? C::NR : 0) + raw.slot];
        if constexpr (!IS_V) {
            const uint32_t cb = t % C::COLS;
            bool odd = false;
            if (tid < BN) {
                const float *sc = reinterpret_cast<const float *>(from + BN * D);
                const bool live = tid < info.x && ((info.y >> (tid >> box_shift)) & 1);
                const float ks = live ? sc[tid] : 0.f;
                float vs = live ? sc[BN + tid] : 1.f;
                if (vs < kMinKvScale) vs = kMinKvScale;  // (a NaN stays)
                float *col = reinterpret_cast<float *>(sm + C::SM_COL) + cb * 3 * BN;
                col[tid] = ks * p.scale2;
                col[BN + tid] = lg2(vs);
                col[2 * BN + tid] = vs == vs ? rcp(vs) : 0.f;  // a NaN enters by b, and not where it is masked
                // (a large scale counts for the tiles after it too, whose references it may have moved)
                large |= vs > kPlainScaleMax;
                odd = large || vs < kPlainScaleMin;
            }
            odd = __any_sync(0xffffffffu, odd);
            if (lane == 0) sm[C::SM_ODD + cb * kGroup + (tid >> 5)] = odd;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_COL + cb);
        }
        // A tile that is whole takes no checks; rows past the end and bad pages become zeros.
        const bool whole = info.x == BN && info.y == all_pages;
        uint8_t *to = dst + ring.slot * C::SLOT;
        convert_tile<D, KIND>(from + src0, to + dst0, to + dst1, row0, whole ? -1 : info.x, info.y, box_shift);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(bar + (IS_V ? C::B_FV : C::B_FK) + ring.slot);
            mbar_arrive(bar + (IS_V ? C::B_REV : C::B_REK) + raw.slot);
        }
        ring.next();
        raw.next();
    }
    if (!ok && lane == 0) flag_error(p.w.pg.status);
}

// ---- softmax ----------------------------------------------------------------------------
// The sum of P over a row's half tile from its products in TMEM, without the value scales. (sees: whether the row sees a
// column)
template <int HC, typename F>
__device__ __forceinline__ float exact_sum(uint32_t ts, const float *key_scale, float rs, float ref, F sees) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < HC; ++c) {  // (few registers: this stands where the kernel has none to spare)
        const float s = __uint_as_float(tmem_ld1(ts + c)) * rs;
        if (sees(c)) sum += ex2(s * key_scale[c] - ref);
    }
    return sum;
}

template <int D, int KIND, bool TREE>
__device__ void soft_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k, uint32_t tmem) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, HC = BN / 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const int bar_id = 1 + quarter;                               // of the two warps that share these rows
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);  // this warp's TMEM lanes
    float *xch = reinterpret_cast<float *>(sm + C::SM_X) + row;
    float2 *stat = reinterpret_cast<float2 *>(sm + C::SM_STAT) + half * 128 + row;
    const float *rsq = reinterpret_cast<const float *>(sm + C::SM_RS) + row;
    const int tok = row / p.w.G;
    uint32_t t = 0, unit = 0;
    // A wait that ran out (`late`, a thread's own) is shared with the rows' other warp at the next meeting, so that
    // both leave there (`ok` is the same for all their threads).
    bool ok = true, late = false;
    if (k.pc.left > 0) do {
        const int n = k.take(), t0 = k.pc.i * p.w.TPT;
        const int rows = min(p.w.TPT, k.pc.s.T - t0) * p.w.G;
        const bool live_warp = quarter * 32 < rows;
        const int base = k.pc.s.len - k.pc.s.T;                    // position of the first new token
        const int sure = TREE ? base - 1 : base + t0;              // last position that every row of the unit sees
        const int limit = row < rows ? sure + tok : -1;            // ... that this row sees
        uint64_t path = 0;                                         // TREE: the nodes on the row's path
        if constexpr (TREE) {
            const Paths paths = tree_paths(p.w.parents + k.pc.s.bos, k.pc.s.T, p.w.pg.status);
            path = paths.at(min(t0 + tok, k.pc.s.T - 1));
        }
        float m = -INFINITY, l = 0.f;
        for (int jj = 0; jj < n; ++jj, ++t) {
            const uint32_t b = t & 1;
            if (!late) late = !product_done<D, KIND>(bar, C::B_S, t, p.budget);
            if (C::kCodes && !late) late = !wait_for(bar + C::B_COL + t % C::COLS, (t / C::COLS) & 1, p.budget);
            if (!live_warp) {
                if (lane == 0) mbar_arrive(bar + C::B_P + b);
                continue;
            }
            tc_fence_after();
            const uint32_t ts = tl + C::TM_S + b * BN + half * HC;
            const int pos0 = (k.pc.off + jj) * BN + half * HC;
            const bool masked = pos0 + HC - 1 > sure;
            const float *col = reinterpret_cast<const float *>(sm + C::SM_COL) + (t % C::COLS) * 3 * BN + half * HC;
            const float rs = C::kCodes ? rsq[(unit & 3) * 128] : 1.f;
            const bool odd = C::kCodes && *reinterpret_cast<const uint32_t *>(sm + C::SM_ODD + (t % C::COLS) * kGroup) != 0;
            float x[HC];  // the scores, in the log2 domain for 8-bit caches, masked
            {
                uint32_t r[HC];
#pragma unroll
                for (int e = 0; e < HC; e += 32) tmem_ld32_nw(ts + e, *reinterpret_cast<uint32_t(*)[32]>(r + e));
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < HC; ++e) x[e] = __uint_as_float(r[e]);
            }
            if constexpr (C::kCodes) {
                const F2 rs2 = f2(rs, rs);
#pragma unroll
                for (int e = 0; e < HC; e += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(col + e), lv = *reinterpret_cast<const float4 *>(col + BN + e);
                    f2_get(f2_fma(f2_mul(f2(x[e], x[e + 1]), rs2), f2(a.x, a.y), f2(lv.x, lv.y)), x[e], x[e + 1]);
                    f2_get(f2_fma(f2_mul(f2(x[e + 2], x[e + 3]), rs2), f2(a.z, a.w), f2(lv.z, lv.w)), x[e + 2], x[e + 3]);
                }
            }
            if constexpr (TREE) {
                if (masked) {
                    const uint64_t sees = path_window(path, pos0 - base);
                    const uint32_t w[2] = {(uint32_t)sees, (uint32_t)(sees >> 32)};
#pragma unroll
                    for (int e = 0; e < HC; ++e)
                        if (!(w[e >> 5] & (1u << (e & 31)))) x[e] = -INFINITY;
                }
            } else if (masked) {
                const int last = limit - pos0;
#pragma unroll
                for (int e = 0; e < HC; ++e)
                    if (e > last) x[e] = -INFINITY;
            }
            float t4[4] = {x[0], x[1], x[2], x[3]};  // four chains
#pragma unroll
            for (int e = 4; e < HC; e += 4)
#pragma unroll
                for (int y = 0; y < 4; ++y) t4[y] = fmaxf(t4[y], x[e + y]);
            const float sc = C::kCodes ? 1.f : p.scale2;
            float *xb = xch + (t & 1) * 256;
            xb[half * 128] = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            ok = !bar_any(bar_id, 64, late);
            if (!ok) break;
            float f;
            const bool grow = grow_reference<C::kCodes>(m, fmaxf(xb[0], xb[128]) * sc, f, l);
            if (jj > 0 && __any_sync(0xffffffffu, grow)) {  // O holds the unit's tiles up to the one before
                late = !product_done<D, KIND>(bar, C::B_PV, t - 1, p.budget);
                tc_fence_after();
#pragma unroll 1
                for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                    uint32_t r[16];
                    tmem_ld16_nw(tl + C::TM_O + c, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                    tmem_st16(tl + C::TM_O + c, r);
                }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            if constexpr (C::kCodes) {
                if (rarely(odd)) {
                    if constexpr (TREE)
                        l += exact_sum<HC>(ts, col, rs, ref, [&](int c) { return on_path(path, pos0 + c - base); });
                    else
                        l += exact_sum<HC>(ts, col, rs, ref, [last = limit - pos0](int c) { return c <= last; });
                }
            }
            F2 l2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
            const F2 sc2 = f2(sc, sc), ref2 = f2(-ref, -ref);
            uint32_t pk[HC / 2];
#pragma unroll
            for (int e = 0; e < HC; e += 2) {
                const F2 y = C::kCodes ? f2_add(f2(x[e], x[e + 1]), ref2) : f2_fma(f2(x[e], x[e + 1]), sc2, ref2);
                float e0, e1;
                f2_get(y, e0, e1);
                e0 = ex2(e0);
                e1 = ex2(e1);
                F2 &acc = l2[(e >> 1) & 1];
                if constexpr (C::kCodes) {
                    const float2 iv = *reinterpret_cast<const float2 *>(col + 2 * BN + e);
                    acc = f2_fma(f2(e0, e1), f2(iv.x, iv.y), acc);
                    pk[e / 2] = h2_bits(e0, e1);
                } else {
                    acc = f2_add(f2(e0, e1), acc);
                    pk[e / 2] = bf2(e0, e1);
                }
            }
            float a, d;
            f2_get(f2_add(l2[0], l2[1]), a, d);
            a += d;
            l += C::kCodes && odd ? 0.f : a;
#pragma unroll
            for (int e = 0; e < HC / 2; e += 16) tmem_st16(ts + e, pk + e);  // over the half's own scores
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_P + b);
        }
        if (!ok) break;
        if (unit >= 2 && !late) late = !wait_for(bar + C::B_SF + (unit & 1), ((unit >> 1) - 1) & 1, p.budget);
        ok = !bar_any(bar_id, 64, late);
        if (!ok) break;
        stat[(unit & 1) * 256] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::B_ST + (unit & 1));
        ++unit;
    } while (walk_next<BN, TREE>(p.w, &k));
    if (!ok && lane == 0) flag_error(p.w.pg.status);
}

// ---- rows: Q in, O out ----------------------------------------------------------------------
// A thread of this group stands for a row of TMEM. Q comes by TMA, 128 bytes of all the unit's rows at a
// time (box: 64 elements, the G heads of the key head, the unit's tokens, which lie in shared memory as
// rows), and goes on into TMEM from there; finished rows are stored straight from TMEM.
template <int D, int KIND, bool TREE>
__device__ void row_role(const TcParams &p, uint8_t *sm, uint64_t *bar, Walk k, uint32_t tmem, const CUtensorMap *mq) {
    using C = Cfg<D, KIND>;
    constexpr int BN = C::BN, PARTS = D / 64;
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, row = quarter * 32 + lane;
    const int tok = row / p.w.G, head = row % p.w.G;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const float2 *stat = reinterpret_cast<const float2 *>(sm + C::SM_STAT) + row;
    float *rsq = reinterpret_cast<float *>(sm + C::SM_RS) + row;
    const uint32_t bytes = (uint32_t)(p.w.TPT * p.w.G) * 128;
    uint32_t fills = 0;   // of the stage so far
    uint32_t issued = 0;  // copies that this warp has begun (fewer, after a wait that ran out)
    bool ok = true;      // the same for a warp's lanes: what follows a wait is done by all of them or by none
    auto unit_rows = [&](const Walk &w) { return min(p.w.TPT, w.pc.s.T - w.pc.i * p.w.TPT) * p.w.G; };
    // 128 bytes of the unit's rows into the stage, once the four warps have read what was there: one warp waits, a lane
    // of it issues the copy
    auto fetch = [&](const Walk &w, int part) {
        if (quarter == 0) {
            if (fills > 0) ok = ok && warp_wait(bar + C::B_QE, (fills - 1) & 1, p.budget);
            if (ok) {
                ++issued;
                if (lane == 0) {
                    mbar_expect_tx(bar + C::B_QF, bytes);
                    tma_load_3d(sm + C::SM_Q, mq, part * 64, w.pc.h * p.w.G, (int)(w.pc.s.bos + w.pc.i * p.w.TPT), bar + C::B_QF);
                }
            }
        }
        ++fills;
    };
    auto read = [&](uint32_t(&x)[32]) {  // this row's
        ok = __all_sync(0xffffffffu, ok && wait_for(bar + C::B_QF, (fills - 1) & 1, p.budget));
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const uint4 v = *reinterpret_cast<const uint4 *>(sm + C::SM_Q + swz(row, c));
            x[4 * c] = v.x; x[4 * c + 1] = v.y; x[4 * c + 2] = v.z; x[4 * c + 3] = v.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::B_QE);
    };
    // 16-bit pairs of Q as they go into TMEM: with an 8-bit cache in fp16, times the row's power of two
    auto pairs = [&](uint32_t(&x)[32], float f) {
        if constexpr (C::kCodes) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
                x[c] = h2_bits(f * __uint_as_float(x[c] << 16), f * __uint_as_float(x[c] & 0xffff0000u));
        }
        if (p.negate)
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] ^= 0x80008000u;
    };
    auto largest = [&](const uint32_t(&x)[32], float a) {
#pragma unroll
        for (int c = 0; c < 32; ++c)
            a = fmaxf(a, fmaxf(fabsf(__uint_as_float(x[c] << 16)), fabsf(__uint_as_float(x[c] & 0xffff0000u))));
        return a;
    };
    // Q of unit number `unit`, whose first part has been fetched, into TMEM. One Q: once the unit before, the one at
    // hand, has used it. Two: the unit before last, which used the same, is done.
    auto bring = [&](const Walk &w, uint32_t unit) {
        const uint32_t to = tl + C::TM_Q + (unit % C::NQ) * (D / 2);
        auto used = [&] {
            if (C::NQ == 1 && unit > 0) ok = ok && warp_wait(bar + C::B_US, (unit - 1) & 1, p.budget);
            tc_fence_after();
        };
        if constexpr (C::kCodes && C::NQ == 2) {  // the row waits for its exponent in TMEM
            float a = 0.f;
            used();
#pragma unroll 1
            for (int part = 0; part < PARTS && ok; ++part) {
                uint32_t x[32];
                read(x);
                if (part + 1 < PARTS) fetch(w, part + 1);
                a = largest(x, a);
                tmem_st32(to + part * 32, x);
            }
            tmem_wait_st();
            const int e = f16_row_exponent(a);
            rsq[(unit & 3) * 128] = pow2i(-e);
#pragma unroll 1
            for (int part = 0; part < PARTS; ++part) {
                uint32_t x[32];
                tmem_ld32_nw(to + part * 32, x);
                tmem_wait_ld();
                pairs(x, pow2i(e));
                tmem_st32(to + part * 32, x);
            }
        } else {
            int e = 0;
            if constexpr (C::kCodes) {
                float a = 0.f;
#pragma unroll 1
                for (int part = 1; part <= PARTS && ok; ++part) {
                    uint32_t x[32];
                    read(x);
                    fetch(w, part % PARTS);
                    a = largest(x, a);
                }
                e = f16_row_exponent(a);
                rsq[(unit & 3) * 128] = pow2i(-e);
            }
            used();
#pragma unroll 1
            for (int part = 0; part < PARTS && ok; ++part) {
                uint32_t x[32];
                read(x);
                if (part + 1 < PARTS) fetch(w, part + 1);
                pairs(x, pow2i(e));
                tmem_st32(to + part * 32, x);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar + C::B_Q + unit % C::NQ);
    };
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    if (k.pc.left > 0) {
        fetch(k, 0);
        bring(k, 0);
        Walk next = k;
        bool more = walk_next<BN, TREE>(p.w, &next);
        if (more) fetch(next, 0);
        for (uint32_t unit = 0; ok; ++unit) {
            if (more) bring(next, unit + 1);
            Walk after = next;
            const bool more2 = more && walk_next<BN, TREE>(p.w, &after);
            if (more2) fetch(after, 0);
            ok = ok && warp_wait(bar + C::B_ST + (unit & 1), (unit >> 1) & 1, p.budget);
            if (!ok) break;
            const float2 a = stat[(unit & 1) * 256], b = stat[(unit & 1) * 256 + 128];
            const float m = a.x, l = a.y + b.y;  // (both halves have the same reference)
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_SF + (unit & 1));
            ok = warp_wait(bar + C::B_UO, unit & 1, p.budget);
            if (!ok) break;
            const int n = k.take(), rows = unit_rows(k);
            if (quarter * 32 < rows) {
                tc_fence_after();
                const int t0 = k.pc.i * p.w.TPT;
                const bool whole = k.begun && k.pc.off + n == k.pc.ntiles;
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const bool repair = !C::kCodes && reinterpret_cast<const volatile int *>(sm + C::SM_INFO)[unit & 7];
                const bool store = row < rows && (!whole || k.pc.s.len - k.pc.s.T + t0 + tok >= 0);  // (padding: zeros already)
                const long part = part_index(p.w, blockIdx.x, k.begun ? 1 : 0, row);
                if (!whole && store) p.w.ml[part] = make_float2(m, l);
                __nv_bfloat16 *out = p.out + ((k.pc.s.bos + t0 + tok) * p.Hq + k.pc.h * p.w.G + head) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(tl + C::TM_O + c, o);
                    if (!store) continue;
                    if (whole) {
                        uint32_t y[16];
#pragma unroll
                        for (int x = 0; x < 16; ++x) y[x] = bf2(o[2 * x] * inv, o[2 * x + 1] * inv);
                        if (wide) {
                            store32(out + c, y);
                            store32(out + c + 16, y + 8);
                        } else {
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                reinterpret_cast<uint4 *>(out + c)[x] = make_uint4(y[4 * x], y[4 * x + 1], y[4 * x + 2], y[4 * x + 3]);
                        }
                    } else {
                        float *dst = p.w.part + part * D + c;
#pragma unroll
                        for (int x = 0; x < 32; x += 8) store32(dst + x, reinterpret_cast<const uint32_t *>(o) + x);
                    }
                }
                tc_fence_before();
                if (!C::kCodes && rarely(repair) && store) {  // what the products left out, for the row if it sees it
                    const KvPages &pg = p.w.pg;
                    const int base = k.pc.s.len - k.pc.s.T, shift = 31 - __clz(pg.page_size);
                    const int first = max(max(TREE ? base : base + t0 + 1, k.pc.off * BN), 0);
                    const int last = min(base + t0 + tok, (k.pc.off + n) * BN - 1);
                    const uint64_t on = TREE ? path_of(p.w.parents + k.pc.s.bos, t0 + tok) : 0;
                    const int32_t *table = pg.table + (long)k.pc.n * pg.max_pages;
                    const __nv_bfloat16 *v = reinterpret_cast<const __nv_bfloat16 *>(p.v_cache);
                    if (whole)
                        add_not_finite<__nv_bfloat16, TREE>(table, pg.num_pages, pg.Hkv, k.pc.h, shift, v, D, first, last, 0, D, out,
                                                            base, on);
                    else
                        add_not_finite<float, TREE>(table, pg.num_pages, pg.Hkv, k.pc.h, shift, v, D, first, last, 0, D,
                                                    p.w.part + part * D, base, on);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar + C::B_OF);
            if (!more) break;
            k = next;
            next = after;
            more = more2;
        }
    }
    if (!ok && lane == 0) flag_error(p.w.pg.status);
    // the copy in flight lands before the CTA leaves: the last one begun, which is not the last one asked for if a wait
    // ran out in between
    if (issued > 0) mbar_wait(bar + C::B_QF, (issued - 1) & 1, kDrainBudget);
    __syncwarp();
}

template <int D, int KIND, bool TREE>
__global__ void __launch_bounds__(Cfg<D, KIND>::THREADS, 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const TcParams p) {
    using C = Cfg<D, KIND>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *sm = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::SM_BAR);
    uint32_t *slot = reinterpret_cast<uint32_t *>(sm + C::SM_TMEM);
    PlanSmem *plan = reinterpret_cast<PlanSmem *>(sm + C::SM_PLAN);
    const int tid = threadIdx.x, warp = tid >> 5;
    next_may_begin();
    if (tid == 0) {
        prefetch_tmap(&mq);
        if (!C::kCodes) {
            prefetch_tmap(&mk);
            prefetch_tmap(&mv);
        }
    }
    if (tid == 0) {
        for (int s = 0; s < C::NK; ++s) mbar_init(bar + C::B_FK + s, C::kCodes ? kGroup : 1);
        for (int s = 0; s < C::NV; ++s) mbar_init(bar + C::B_FV + s, C::kCodes ? kGroup : 1);
        for (int s = 0; s < C::NR; ++s) {
            mbar_init(bar + C::B_RK + s, 1);
            mbar_init(bar + C::B_RV + s, 1);
            mbar_init(bar + C::B_REK + s, kGroup);
            mbar_init(bar + C::B_REV + s, kGroup);
        }
        for (int s = 0; s < C::COLS; ++s) mbar_init(bar + C::B_COL + s, kGroup);
        for (int s = 0; s < C::kTurns; ++s) {
            mbar_init(bar + C::B_S + s, 1);
            mbar_init(bar + C::B_PV + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar + C::B_P + s, 2 * kGroup);
            mbar_init(bar + C::B_ST + s, 2 * kGroup);
            mbar_init(bar + C::B_SF + s, kGroup);
        }
        for (int s = 0; s < C::NQ; ++s) mbar_init(bar + C::B_Q + s, kGroup);
        mbar_init(bar + C::B_OF, kGroup);
        mbar_init(bar + C::B_QF, 1);
        mbar_init(bar + C::B_US, 1);
        mbar_init(bar + C::B_UO, C::kCodes ? 1 : 2);  // (the products, and what SM_INFO says)
        mbar_init(bar + C::B_QE, kGroup);
        mbar_init(bar + C::B_FIN, 1);
        if (!C::kCodes)
            for (int s = 0; s < C::NV; ++s) mbar_init(bar + C::B_CV + s, 1);
        fence_mbar_init();
    }
    before_reading();  // (and before TMEM is asked for: a kernel that ends may still hold it)
    if (warp == 0) tmem_alloc(slot, 512);
    tc_fence_before();
    plan_piece<C::BN, C::THREADS, TREE>(p.w, plan);  // (synchronises the CTA)
    tc_fence_after();
    // All 512 columns are this CTA's, so the allocation starts at column 0, and addresses are constants (in uniform
    // registers; from a loaded value, the issue of each product took about 45 cycles).
    constexpr uint32_t tmem = 0;
    Walk k{plan->piece, plan->piece.off == 0};
    if (*slot != tmem) {
        if (tid == 0) flag_error(p.w.pg.status);
        k.pc.left = 0;
    }
    const int group = warp / kGroup;
    if (group < kRowWarp0 / kGroup) {
        if constexpr (C::kCodes) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        soft_role<D, KIND, TREE>(p, sm, bar, k, tmem);
    } else if (group == kRowWarp0 / kGroup) {
        row_role<D, KIND, TREE>(p, sm, bar, k, tmem, &mq);
    } else if (group == kLoadWarp / kGroup) {
        if (warp == kLoadWarp) {
            load_role<D, KIND, TREE, false>(p, sm, bar, k, &mk);
        } else if (warp == kLoadWarp + 1) {
            load_role<D, KIND, TREE, true>(p, sm, bar, k, &mv);
        } else if (warp == kMmaWarp) {
            mma_role<D, KIND, TREE>(p, sm, sb, bar, k, tmem);
        } else if constexpr (C::kCodes) {
            if (plan->padding) zero_padding<TREE>(p.w, p.out, p.Hq, D, tid & 31, 32);
        } else {
            check_role<D, KIND, TREE>(p, sm, bar, k);
        }
    } else if constexpr (C::kCodes) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
        if (group == kConvWarp0 / kGroup) convert_role<D, KIND, false>(p, sm, bar, (uint32_t)k.pc.left);
        else convert_role<D, KIND, true>(p, sm, bar, (uint32_t)k.pc.left);
    }
    if (!C::kCodes && plan->padding) zero_padding<TREE>(p.w, p.out, p.Hq, D, tid, C::THREADS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---- host side ------------------------------------------------------------------
template <int D, int KIND, bool TREE>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
    using C = Cfg<D, KIND>;
    const int G = a.Hq / a.pg.Hkv;
    TcParams p{};
    p.w = attn_work(a, kAttnMaxRows / G, 1);
    p.k_cache = (const uint8_t *)a.k_cache;
    p.v_cache = (const uint8_t *)a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.out = (__nv_bfloat16 *)a.out;
    p.Hq = a.Hq;
    p.negate = a.scale < 0.f;
    // a scale of 0 must not meet the -inf of a masked score in a product: so small that no score counts
    p.scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);
    p.budget = wait_budget();
    CUtensorMap mq, mk{}, mv{};
    if (!rows_map(&mq, a.q, D, a.Hq, a.pg.Ttot, a.q_stride, G, p.w.TPT)) return cudaErrorInvalidValue;
    if (!C::kCodes) {
        const int rows = a.pg.page_size < C::BN ? a.pg.page_size : C::BN;
        if (!page_map(&mk, a.k_cache, a.pg, D * 2, rows) || !page_map(&mv, a.v_cache, a.pg, D * 2, rows))
            return cudaErrorInvalidValue;
    }
    auto kernel = attn_tc_kernel<D, KIND, TREE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const int ctas = attn_ctas(a, p.w, C::BN);
    e = launch_early(kernel, dim3(ctas), C::THREADS, C::SM_BYTES, s, mq, mk, mv, p);
    return e != cudaSuccess ? e : launch_attn_join(a, p.w, ctas, s);
}

template <int KIND>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.d) {
        case 64: return a.parents ? launch_t<64, KIND, true>(a, s) : launch_t<64, KIND, false>(a, s);
        case 128: return a.parents ? launch_t<128, KIND, true>(a, s) : launch_t<128, KIND, false>(a, s);
        case 256: return a.parents ? launch_t<256, KIND, true>(a, s) : launch_t<256, KIND, false>(a, s);
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
