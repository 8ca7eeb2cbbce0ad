// attn_rows.cu -- attention over a paged cache for few query rows per key head (bf16 inputs): the
// decode step and the check of a few speculated tokens.
//
// With at most 16 rows (the G query heads of a key head, of few tokens) every cached row is read
// for 16 rows' worth of products at most, 16 to 32 flops a byte, so the kernel is bound by the bytes
// of the cache and, for short ones, by the length of its own dependent chain. It therefore keeps
// everything of a key chunk inside one warp: a CTA's warps take 16 or 32 positions each of a tile,
// every warp has its own ring of tiles in flight (TMA, one box per 128 bytes of row, 128B swizzle),
// its own running softmax and its own output in registers, and meets the others only once per unit of
// work, in shared memory. The products are m16n8k16 (mma.sync) with the cached rows as M,
//     S^T = K Q^T,   O^T = V^T P^T,
// so that N holds 8 query rows (R = 8) or twice 8 (R = 16) and nothing is padded to more;
// tcgen05's M of 128 would be padded 8 to 16 times and needs hand-overs between warps for each tile.
//
// Fragments without shuffles. The sums over d and over keys may run in any order, so both are
// permuted such that a thread's operands are 16-byte pieces of a row, free of bank conflicts:
//   S^T: of a piece of a row, each 4 elements in turn are the thread's k indexes of one product;
//        Q's fragments are laid out in the same order, once per unit;
//   O^T: rows n and n + 8 of product t are d = 8 n + 2 t and 8 n + 2 t + 1 of a 64-wide block (bf16;
//        16 n + 2 t of 128 for 8-bit codes), so that a thread ends with 8 (16) consecutive elements
//        of its rows;
//   slot c of 8 positions holds position r = g(c), g = 0 4 2 6 5 1 7 3.
// P^T leaves the softmax as S^T's layout has it (a position's rows side by side) and becomes the B
// operand by movmatrix, 8 x 8 at a time.
// 8-bit codes become fp16 in registers (attn_tc.cu says why fp16, and how the scales enter).
//
// Measured: 128 sessions of 4096, 2 key heads with 8 query heads each, D = 256: bf16 170 us (6.3 TB/s of
// 6.7 measured), e4m3 96 us (5.7); 32 of 8192, 8 key heads with 4, D = 128: bf16 168, int8 96, e4m3 94
// us (5.8 TB/s for codes), where the codes' conversion takes 0.55 instructions a cycle and scheduler; one
// session of 131072, e4m3, D = 256: 35 us, of which memory 20; one of 1000: 10.6 us from a graph, a chain
// of the plan, the table, the first tiles, the warps' meeting and the joining kernel.
#include <climits>

#include "attn_ops.cuh"

namespace gdn {
namespace {

using namespace tc;

template <int D, int KIND, int R>
struct RCfg {
    static constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    static constexpr int ROWB = D * (kCodes ? 1 : 2);           // bytes of a row
    static constexpr int NT = R / 8;                            // row tiles
    // Codes cost a warp 300 to 500 instructions per 16 positions, and two warps per scheduler issue one every two to
    // three cycles, so more warps help as long as registers and rings allow: int8, d = 128, 8 rows (32 sequences of
    // 8192 positions, 8 key heads): 113, 99 and 108 us with 8, 12 and 16 warps; fp8, d = 64 (twice the positions): 161,
    // 126 and 131. At d = 256 the output fills the registers (101, 102 and 106 us; 16 rows: 118 and 156 with 8 and 12
    // warps), and bf16 is bound by memory with any number.
    static constexpr int WARPS = kCodes && D < 256 ? 12 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr uint32_t RINGB = 196608 / WARPS;           // a warp's ring
    // Positions per chunk. 32 spread what a chunk costs beside its products (waits, loads, softmax steps: half of a
    // 16-position chunk's instructions at 128-byte rows); wider rows need 16 for at least two chunks in flight.
    static constexpr int CH = 4 * 32 * ROWB <= RINGB ? 32 : 16;
    static constexpr int U = CH / 16;                           // score tiles of a chunk
    static constexpr int BN = WARPS * CH;                       // positions per tile of work
    static constexpr int BOXES = ROWB >= 128 ? ROWB / 128 : 1;  // TMA boxes per 16 positions
    static constexpr int LINES = ROWB >= 128 ? CH : CH / 2;     // 128-byte lines of a chunk per 128 bytes of row
    static constexpr uint32_t SLOT = CH * ROWB;                 // K or V of a chunk
    // A chunk's K and V come as one stage of the ring, unless that leaves less than two stages (bf16, D = 256):
    // then K and V take turns in slots of their own.
    static constexpr bool kPair = RINGB / (2 * SLOT) >= 2;
    static constexpr uint32_t STAGE = kPair ? 2 * SLOT : SLOT;
    static constexpr int NSL = RINGB / STAGE;
    static_assert(NSL >= 2 && (kPair || (CH == 16 && !kCodes)), "ring");
    static constexpr int KS = D / 16;                           // products per score tile
    static constexpr int VE = kCodes ? (D == 64 ? 8 : 16) : 8;  // elements per piece of V
    static constexpr int MSTRIDE = D + 4;                       // floats per row where warps meet
    static constexpr uint32_t RING = WARPS * NSL * STAGE, MEET = WARPS * R * MSTRIDE * 4;
    static constexpr uint32_t SM_Q = RING > MEET ? RING : MEET;  // Q fragments [KS / 2][NT][32 lanes][16 bytes]
    static constexpr uint32_t SM_SC = SM_Q + KS * NT * 256;      // [warp][NSL][k, v][CH] scales
    static constexpr uint32_t SM_ML = SM_SC + (kCodes ? WARPS * NSL * 2 * CH * 4 : 0);  // [warp][R] m, l
    static constexpr uint32_t SM_RS = SM_ML + WARPS * R * 8;     // [R] Q row scales
    static constexpr uint32_t SM_BAR = SM_RS + R * 4;
    static constexpr uint32_t SM_PLAN = SM_BAR + WARPS * NSL * 8;
    static constexpr uint32_t SM_BYTES = SM_PLAN + sizeof(PlanSmem) + 1024;
    static_assert(SM_BYTES <= 232448, "over the 227 KiB opt-in limit");
};

struct RowParams {
    AttnWork w;
    const __nv_bfloat16 *q;
    const __nv_bfloat16 *v_cache;  // bf16 caches
    const float *k_scale, *v_scale;
    __nv_bfloat16 *out;
    int Hq;
    long q_stride;
    float scale2;  // |softmax scale| * log2 e
    int negate;
    long long budget;
};

// byte offset of 16-byte piece c of position r in a chunk
template <int ROWB, int CH>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    if (ROWB >= 128) return (uint32_t)((c >> 3) * (CH * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    const int line = r >> 1;
    return (uint32_t)(line * 128 + ((((r & 1) * 4 + c) ^ (line & 7)) << 4));
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {  // of 16-bit elements; every lane of the warp
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int KIND, int R>
__global__ void __launch_bounds__(RCfg<D, KIND, R>::THREADS, 1)
attn_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const RowParams p) {
    using C = RCfg<D, KIND, R>;
    constexpr int CH = C::CH, U = C::U, BN = C::BN, NT = C::NT, kThreads = C::THREADS, kWarps = C::WARPS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *sm = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const AttnWork &w = p.w;
    const KvPages &pg = w.pg;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = lane >> 2, q = lane & 3;
    const int g2 = 2 * q + (q >> 1);                        // g(2 q); g(2 q + 1) = g2 ^ 4
    const int gn = (2 * (n >> 1) + (n >> 2)) ^ ((n & 1) * 4);  // g(n)
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + C::SM_BAR) + warp * C::NSL;
    uint8_t *ring = sm + warp * (C::NSL * C::STAGE);
    float *scales = reinterpret_cast<float *>(sm + C::SM_SC) + warp * (C::NSL * 2 * CH);
    uint32_t *qf = reinterpret_cast<uint32_t *>(sm + C::SM_Q);
    float2 *ml = reinterpret_cast<float2 *>(sm + C::SM_ML);
    float *rs = reinterpret_cast<float *>(sm + C::SM_RS);
    PlanSmem *plan = reinterpret_cast<PlanSmem *>(sm + C::SM_PLAN);
    next_may_begin();
    if (tid == 0) {
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    if (lane == 0) {
        for (int s = 0; s < C::NSL; ++s) mbar_init(bar + s, 1);
        fence_mbar_init();
    }
    before_reading();
    plan_piece<BN, kThreads>(w, plan);  // (synchronises the CTA)
    Piece pc = plan->piece;
    const int P_shift = 31 - __clz(pg.page_size);
    uint32_t filled = 0, used_up = 0;  // ring slots of this warp
    uint32_t fslot = 0, uslot = 0, uphase = 0;
    bool failed = false;
    // 16 positions of a stage whose scales are not loaded: keys and values of zero
    auto clear_scales = [&](float *sc, int at) {
        sc[(lane < 16 ? 0 : CH) + at + (lane & 15)] = lane < 16 ? 0.f : 1.f;
        fence_async_smem();
    };
    auto bad_page = [&](float *sc, int at) {  // outside of the pool (the copies read zeros)
        if (lane == 0) flag_error(pg.status);
        if (C::kCodes) clear_scales(sc, at);
    };
    bool begun = pc.off == 0, repair = false;  // (repair: the unit is done a second time)
    while (pc.left > 0) {
        const int t0 = pc.i * w.TPT, rows = min(w.TPT, pc.s.T - t0) * w.G, len = pc.s.len;
        const int off = pc.off, take = (int)min((long)(pc.ntiles - off), pc.left);
        // this warp's chunks: positions start + BN i
        const int start = off * BN + warp * CH;
        const int chunks = start < len ? min(take, (len - start + BN - 1) / BN) : 0;
        const int32_t *table = pg.table + (long)pc.n * pg.max_pages;
        const int pages = (len + pg.page_size - 1) >> P_shift;
        auto entries = [&](int window) -> int {
            const int i = window * 32 + lane;
            return i < pages ? table[i] : -1;
        };
        int window = (start >> P_shift) >> 5, win = entries(window), win_next = entries(window + 1);
        int fill_pos = start, fills = C::kPair ? chunks : 2 * chunks, page = 0, page2 = 0;
        // The next stage: a chunk's K and V, or its K, then its V. Each box is issued by a lane of its own.
        auto issue = [&] {
            const bool is_v = !C::kPair && (filled & 1);
            if (!is_v) {
                const int idx = fill_pos >> P_shift;
                while ((idx >> 5) != window) {
                    ++window;
                    win = win_next;
                    win_next = entries(window + 1);
                }
                page = __shfl_sync(0xffffffffu, win, idx & 31);
                // the chunk's second page, where pages are shorter than it
                if constexpr (CH > 16) page2 = __shfl_sync(0xffffffffu, win, ((fill_pos + 16) >> P_shift) & 31);
            }
            const bool mine_v = C::kPair ? lane >= 16 : is_v;
            const int box = C::kPair ? lane & 15 : lane;
            uint8_t *to = ring + fslot * C::STAGE + (C::kPair && mine_v ? C::SLOT : 0);
            float *sc = scales + fslot * 2 * CH;
            const CUtensorMap *map = mine_v ? &mv : &mk;
            if constexpr (CH == 16) {
                const bool good = (unsigned)page < (unsigned)pg.num_pages;
                const int row0 = fill_pos & (pg.page_size - 1);
                const long at = ((long)page * pg.Hkv + pc.h) * pg.page_size + row0;
                if (!good && !is_v) bad_page(sc, 0);
                if (lane == 0) mbar_expect_tx(bar + fslot, C::STAGE + (C::kCodes && good && !is_v ? 2 * CH * 4 : 0));
                __syncwarp();
                if (box < C::BOXES)
                    tma_load_3d(to + box * (C::LINES * 128), map, box * (C::kCodes ? 128 : 64), row0,
                                good ? page * pg.Hkv + pc.h : -1, bar + fslot);
                if (C::kCodes && good && box == 15)
                    bulk_load(sc + (mine_v ? CH : 0), (mine_v ? p.v_scale : p.k_scale) + at, CH * 4, bar + fslot);
            } else {
                // two boxes of 16 positions each: they may lie on two pages, and the second may lie past the end
                const int half = box & 1, blk = box >> 1, pos = fill_pos + 16 * half;
                const int mine = half ? page2 : page;
                const bool there = pos < len, good = there && (unsigned)mine < (unsigned)pg.num_pages;
                const bool good0 = (unsigned)page < (unsigned)pg.num_pages;
                const bool there1 = fill_pos + 16 < len, good1 = there1 && (unsigned)page2 < (unsigned)pg.num_pages;
                if (!good0) bad_page(sc, 0);
                if (!good1) {
                    if (there1) bad_page(sc, 16);
                    else if (C::kCodes) clear_scales(sc, 16);
                }
                if (lane == 0)
                    mbar_expect_tx(bar + fslot, C::STAGE + (C::kCodes ? ((good0 ? 1 : 0) + (good1 ? 1 : 0)) * 2 * 16 * 4 : 0));
                __syncwarp();
                const int row0 = pos & (pg.page_size - 1);
                if (blk < C::BOXES)
                    tma_load_3d(to + blk * (C::LINES * 128) + half * (C::LINES * 64), map, blk * (C::kCodes ? 128 : 64),
                                C::ROWB >= 128 ? row0 : row0 >> 1, good ? mine * pg.Hkv + pc.h : -1, bar + fslot);
                if (C::kCodes && good && blk == 7)
                    bulk_load(sc + (mine_v ? CH : 0) + 16 * half,
                              (mine_v ? p.v_scale : p.k_scale) + ((long)mine * pg.Hkv + pc.h) * pg.page_size + row0, 64,
                              bar + fslot);
            }
            if (C::kPair || is_v) fill_pos += BN;
            if (++fslot == C::NSL) fslot = 0;
            ++filled;
            --fills;
        };
        auto wait_full = [&] {
            if (!failed) failed = !wait_for(bar + uslot, uphase, p.budget);
            failed = __any_sync(0xffffffffu, failed);
        };
        auto release = [&] {  // the slot at hand has been read
            __syncwarp();
            if (++uslot == C::NSL) {
                uslot = 0;
                uphase ^= 1;
            }
            ++used_up;
            if (fills > 0) issue();
        };
        while (fills > 0 && filled - used_up < (uint32_t)C::NSL) issue();

        // Q fragments, by the whole CTA: a row's 16 bytes to the lanes that hold its elements
        for (int e = tid; e < R * (D / 8); e += kThreads) {
            const int r = e / (D / 8), c = e % (D / 8);  // row, piece of 8 elements
            uint32_t x[4] = {0, 0, 0, 0};
            if (r < rows) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p.q + (pc.s.bos + t0 + r / w.G) * p.q_stride +
                                                                 (long)(pc.h * w.G + r % w.G) * D + 8 * c);
                x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
            }
            if constexpr (C::kCodes) {  // to fp16, by the row's power of two: its pieces sit in adjacent lanes
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
#pragma unroll
                for (int o = D / 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const int ex = f16_row_exponent(amax);
                const float f = pow2i(ex);
                if (c == 0) rs[r] = pow2i(-ex);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i] = h2_bits(f * __uint_as_float(x[i] << 16), f * __uint_as_float(x[i] & 0xffff0000u));
            }
            if (p.negate)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] ^= 0x80008000u;
            // elements 8 c + 4 s ..: of product ks, row tile r / 8, lane (r % 8, qq)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int ks = C::kCodes ? (c / 8) * 4 + (c & 1) * 2 + s : (c / 4) * 2 + s;
                const int qq = C::kCodes ? (c / 2) & 3 : c & 3;
                *reinterpret_cast<uint2 *>(qf + (((ks >> 1) * NT + (r >> 3)) * 32 + (r & 7) * 4 + qq) * 4 + (ks & 1) * 2) =
                    make_uint2(x[2 * s], x[2 * s + 1]);
            }
        }
        __syncthreads();

        // of row tile y: rows 8 y + 2 q + (i & 1), elements (tile t of 16) of n's piece, 2 t + (i >> 1)
        float o[D / 16][NT][4];
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][y][i] = 0.f;
        float m[NT][2], l[NT][2], rsc[NT][2];
        int limit[NT][2];  // last position that the thread's rows see
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * y + 2 * q + i;
                m[y][i] = -INFINITY;
                l[y][i] = 0.f;
                limit[y][i] = r < rows ? len - pc.s.T + t0 + r / w.G : INT_MAX;  // (rows past the last are not read)
                rsc[y][i] = C::kCodes ? rs[r] * p.scale2 : p.scale2;
            }
        const int sure = len - pc.s.T + t0;                      // every row sees up to here
        const int seen = sure + min(w.TPT, pc.s.T - t0);         // no row sees this position or one after it
        // What is rare shows in a unit's outcome, and the unit is done again with care. (To look for it beforehand made 2
        // tokens of 16 sessions 5% slower.) bf16: a value between the two that is not finite makes rows that do not see it
        // NaN (0 times it); it is left out then, and the rows that see it get it at the end. Codes: scales for which
        // P' / vs may not do (plain_reciprocal) make the sum NaN.
        const bool check = !repair && (C::kCodes || seen - sure > 1);
        for (int ch = 0; ch < chunks && !failed; ++ch) {
            const int pos0 = start + ch * BN;
            wait_full();
            if (failed) break;
            constexpr int SPLIT = 4 / (U * NT);  // chains of products per score tile
            float s[U][NT][SPLIT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int z = 0; z < SPLIT; ++z)
#pragma unroll
                        for (int i = 0; i < 4; ++i) s[u][y][z][i] = 0.f;
            const uint8_t *kc = ring + uslot * C::STAGE;
            constexpr int KP = C::kCodes ? 4 : 2;  // products per piece
#pragma unroll
            for (int i = 0; i < C::KS / KP; ++i) {
                uint4 b[KP / 2][NT];
#pragma unroll
                for (int x = 0; x < KP / 2; ++x)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
                        b[x][y] = *reinterpret_cast<const uint4 *>(qf + (((i * KP / 2 + x) * NT + y) * 32 + lane) * 4);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 k0 = *reinterpret_cast<const uint4 *>(kc + piece_at<C::ROWB, CH>(u * 16 + gn, 4 * i + q));
                    const uint4 k1 = *reinterpret_cast<const uint4 *>(kc + piece_at<C::ROWB, CH>(u * 16 + 8 + gn, 4 * i + q));
                    if constexpr (C::kCodes) {
                        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t a0, a1, a2, a3;
                            codes4_to_f16<KIND>(w0[x], a0, a2);
                            codes4_to_f16<KIND>(w1[x], a1, a3);
#pragma unroll
                            for (int y = 0; y < NT; ++y) {
                                const uint4 &c = b[x >> 1][y];
                                mma16816<true>(s[u][y][x & (SPLIT - 1)], a0, a1, a2, a3, x & 1 ? c.z : c.x, x & 1 ? c.w : c.y);
                            }
                        }
                    } else {
#pragma unroll
                        for (int y = 0; y < NT; ++y) {
                            mma16816<false>(s[u][y][2 * i & (SPLIT - 1)], k0.x, k1.x, k0.y, k1.y, b[0][y].x, b[0][y].y);
                            mma16816<false>(s[u][y][2 * i + 1 & (SPLIT - 1)], k0.z, k1.z, k0.w, k1.w, b[0][y].z, b[0][y].w);
                        }
                    }
                }
            }
            float iv[U][2];
            float x[U][NT][4];  // [score tile][row tile]: position 16 u + gn: 2 rows, then 16 u + 8 + gn: 2 rows
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[u][y][i] = s[u][y][0][i];
#pragma unroll
                        for (int z = 1; z < SPLIT; ++z) x[u][y][i] += s[u][y][z][i];
                    }
                if constexpr (C::kCodes) {
                    const float *sc = scales + uslot * 2 * CH + u * 16 + gn;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a = sc[8 * j];
                        float vs = sc[CH + 8 * j];
                        if (vs < kMinKvScale) vs = kMinKvScale;  // (a NaN stays)
                        const float lv = lg2(vs);
                        iv[u][j] = plain_reciprocal(vs);  // (a NaN enters by lv, and not where it is masked)
#pragma unroll
                        for (int y = 0; y < NT; ++y)
#pragma unroll
                            for (int i = 0; i < 2; ++i) x[u][y][2 * j + i] = fmaf(x[u][y][2 * j + i] * rsc[y][i], a, lv);
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[u][y][i] *= rsc[y][i & 1];
                }
            }
            if (!C::kPair) release();
            if (pos0 + CH - 1 > sure) {
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int lim = limit[y][i & 1] - pos0 - gn;
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (u * 16 + 8 * (i >> 1) > lim) x[u][y][i] = -INFINITY;
                    }
                if constexpr (C::kCodes)  // (whatever lies past the end must not show in the sum)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (pos0 + u * 16 + 8 * j + gn >= len) iv[u][j] = 0.f;
            }
            // The reference moves when a score is far above it (kGrow), so each lane looks at its own scores, and the
            // rows' maxima are brought together over the lanes only when one of them found such a score.
            float top[NT][2];
            bool grow = false;
#pragma unroll
            for (int y = 0; y < NT; ++y)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[y][i] = fmaxf(x[0][y][i], x[0][y][2 + i]);
#pragma unroll
                    for (int u = 1; u < U; ++u) top[y][i] = fmaxf(top[y][i], fmaxf(x[u][y][i], x[u][y][2 + i]));
                    grow |= above_reference(m[y][i], top[y][i]);
                }
            if (__any_sync(0xffffffffu, grow)) {
                float f[NT][2];
#pragma unroll
                for (int y = 0; y < NT; ++y)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
#pragma unroll
                        for (int d = 4; d < 32; d *= 2)
                            top[y][i] = fmaxf(top[y][i], __shfl_xor_sync(0xffffffffu, top[y][i], d));
                        grow_reference<C::kCodes>(m[y][i], top[y][i], f[y][i], l[y][i]);
                    }
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
#pragma unroll
                    for (int y = 0; y < NT; ++y)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[t][y][i] *= f[y][i & 1];
            }
            if constexpr (C::kCodes) {
                if (rarely(repair)) {  // P's sum from the scores without the scales
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float vs = scales[uslot * 2 * CH + CH + u * 16 + gn + 8 * j];
                            if (vs < kMinKvScale) vs = kMinKvScale;
                            const float lv = lg2(vs);
                            iv[u][j] = 0.f;
#pragma unroll
                            for (int y = 0; y < NT; ++y)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float s_lv = x[u][y][2 * j + i];
                                    if (s_lv != -INFINITY) l[y][i] += ex2((s_lv - lv) - m[y][i]);
                                }
                        }
                }
            }
            uint32_t pt[U][NT][2];  // P^T as the B operand
#pragma unroll
            for (int y = 0; y < NT; ++y) {
                const float ref0 = m[y][0] == -INFINITY ? 0.f : m[y][0], ref1 = m[y][1] == -INFINITY ? 0.f : m[y][1];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float e0 = ex2(x[u][y][2 * j] - ref0), e1 = ex2(x[u][y][2 * j + 1] - ref1);
                        uint32_t both;
                        if constexpr (C::kCodes) {
                            l[y][0] = fmaf(e0, iv[u][j], l[y][0]);
                            l[y][1] = fmaf(e1, iv[u][j], l[y][1]);
                            both = h2_bits(e0, e1);
                        } else {
                            l[y][0] += e0;
                            l[y][1] += e1;
                            both = bf2_bits(__floats2bfloat162_rn(e0, e1));
                        }
                        pt[u][y][j] = transpose8x8(both);
                    }
            }
            if constexpr (!C::kPair) {
                wait_full();
                if (failed) break;
            }
            const uint8_t *vc = ring + uslot * C::STAGE + (C::kPair ? C::SLOT : 0);
            const bool tail = pos0 + CH > seen;  // rows past the last that counts: zeros
            if (!C::kCodes && rarely(repair && pos0 + CH - 1 > sure)) {
                constexpr int PR = C::ROWB / 16;
                const int from = max(sure + 1 - pos0, 0), to = min(seen - pos0, CH);
                for (int e = lane; e < (to - from) * PR; e += 32)
                    drop_not_finite(reinterpret_cast<uint4 *>(const_cast<uint8_t *>(vc) + piece_at<C::ROWB, CH>(from + e / PR, e % PR)));
                __syncwarp();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int b = 0; b < D / (8 * C::VE); ++b) {
                    uint32_t v[4][4];  // positions g2, g2 ^ 4, 8 + g2, 8 + (g2 ^ 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = u * 16 + (j >> 1) * 8 + (g2 ^ (4 * (j & 1)));
                        if (C::VE * (C::kCodes ? 1 : 2) == 16) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(vc + piece_at<C::ROWB, CH>(r, b * 8 + n));
                            v[j][0] = y.x; v[j][1] = y.y; v[j][2] = y.z; v[j][3] = y.w;
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2 *>(vc + piece_at<C::ROWB, CH>(r, n >> 1) + (n & 1) * 8);
                            v[j][0] = y.x; v[j][1] = y.y; v[j][2] = v[j][3] = 0;
                        }
                        if (tail && pos0 + r >= seen) v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
                    }
#pragma unroll
                    for (int t = 0; t < C::VE / 2; ++t) {  // elements 2 t, 2 t + 1 of the pieces
                        uint32_t a0, a1, a2, a3;
                        if constexpr (C::kCodes) {
                            const int wd = t >> 1, sel = t & 1 ? 0x7362 : 0x5140;
                            codes4_to_f16<KIND>(__byte_perm(v[0][wd], v[1][wd], sel), a0, a1);
                            codes4_to_f16<KIND>(__byte_perm(v[2][wd], v[3][wd], sel), a2, a3);
                        } else {
                            a0 = __byte_perm(v[0][t], v[1][t], 0x5410);
                            a1 = __byte_perm(v[0][t], v[1][t], 0x7632);
                            a2 = __byte_perm(v[2][t], v[3][t], 0x5410);
                            a3 = __byte_perm(v[2][t], v[3][t], 0x7632);
                        }
#pragma unroll
                        for (int y = 0; y < NT; ++y)
                            mma16816<C::kCodes>(o[b * (C::VE / 2) + t][y], a0, a1, a2, a3, pt[u][y][0], pt[u][y][1]);
                    }
                }
            }
            release();
        }
        // the warps meet: O over the rings, which are empty now
        if (__syncthreads_or(failed)) break;
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * y + 2 * q + i;
#pragma unroll
                for (int d = 4; d < 32; d *= 2) l[y][i] += __shfl_xor_sync(0xffffffffu, l[y][i], d);
                if (n == 0) ml[warp * R + r] = make_float2(m[y][i], l[y][i]);
                if (r < rows && chunks > 0) {
                    float *dst = reinterpret_cast<float *>(sm) + (warp * R + r) * C::MSTRIDE + n * C::VE;
#pragma unroll
                    for (int b = 0; b < D / (8 * C::VE); ++b)
#pragma unroll
                        for (int t = 0; t < C::VE / 2; t += 2) {
                            const float(&lo)[4] = o[b * (C::VE / 2) + t][y], (&hi)[4] = o[b * (C::VE / 2) + t + 1][y];
                            *reinterpret_cast<float4 *>(dst + b * 8 * C::VE + 2 * t) = make_float4(lo[i], lo[2 + i], hi[i], hi[2 + i]);
                        }
                }
            }
        __syncthreads();
        bool bad = false;
        const bool whole = begun && off + take == pc.ntiles;
        for (int e = tid; e < rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) M = fmaxf(M, ml[x * R + r].x);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add_part = [&](int x, float f) {
                const float4 z = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(sm) + (x * R + r) * C::MSTRIDE + c);
                y.x = fmaf(f, z.x, y.x); y.y = fmaf(f, z.y, y.y); y.z = fmaf(f, z.z, y.z); y.w = fmaf(f, z.w, y.w);
            };
            if (C::kCodes && rarely(repair)) {
#pragma unroll 1
                for (int x = 0; x < kWarps; ++x) {
                    const float2 a = ml[x * R + r];
                    if (a.x == -INFINITY && a.y == 0.f) continue;
                    const float h = ex2(0.5f * (a.x - ref));  // (in two halves: grow_reference)
                    L = fmaf(h * a.y, h, L);
                    add_part(x, h * h);
                }
            } else {
#pragma unroll
                for (int x = 0; x < kWarps; ++x) {
                    const float2 a = ml[x * R + r];
                    if (a.x == -INFINITY && a.y == 0.f) continue;  // nothing seen
                    const float f = ex2(a.x - ref);
                    L = fmaf(f, a.y, L);
                    add_part(x, f);
                }
            }
            bad |= C::kCodes ? !(L == L) : !(fabsf(y.x) + fabsf(y.y) + fabsf(y.z) + fabsf(y.w) < INFINITY);
            if (whole) {
                const int t = t0 + r / w.G;
                if (len - pc.s.T + t < 0) continue;  // padding: written as zeros
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const __nv_bfloat162 a = __floats2bfloat162_rn(y.x * inv, y.y * inv), b = __floats2bfloat162_rn(y.z * inv, y.w * inv);
                *reinterpret_cast<uint2 *>(p.out + ((pc.s.bos + t) * p.Hq + pc.h * w.G + r % w.G) * D + c) =
                    make_uint2(bf2_bits(a), bf2_bits(b));
            } else {
                const long at = part_index(w, blockIdx.x, begun ? 1 : 0, r);
                *reinterpret_cast<float4 *>(w.part + at * D + c) = y;
                if (c == 0) w.ml[at] = make_float2(M, L);
            }
        }
        if (!C::kCodes && rarely(repair)) {  // what was dropped, for the rows that see it
            for (int e = tid; e < rows * (D / 4); e += kThreads) {
                const int r = e / (D / 4), c = (e % (D / 4)) * 4, t = t0 + r / w.G;
                const int first = max(max(sure + 1, off * BN), 0), last = min(len - pc.s.T + t, (off + take) * BN - 1);
                if (whole)
                    add_not_finite(table, pg.num_pages, pg.Hkv, pc.h, P_shift, p.v_cache, D, first, last, c, 4,
                                   p.out + ((pc.s.bos + t) * p.Hq + pc.h * w.G + r % w.G) * D);
                else
                    add_not_finite(table, pg.num_pages, pg.Hkv, pc.h, P_shift, p.v_cache, D, first, last, c, 4,
                                   w.part + part_index(w, blockIdx.x, begun ? 1 : 0, r) * D);
            }
        }
        fence_async_smem();  // the rings held O: before the next unit's copies
        repair = __syncthreads_or(check && bad);
        if (rarely(repair)) continue;
        pc.left -= take;
        if (pc.left > 0) next_unit<BN>(w, &pc);
        begun = true;
    }
    if (failed && lane == 0) flag_error(pg.status);
    // copies in flight (after a wait that ran out) must land before the CTA leaves
    for (; used_up < filled; ++used_up) {
        mbar_wait(bar + uslot, uphase, kDrainBudget);
        if (++uslot == C::NSL) {
            uslot = 0;
            uphase ^= 1;
        }
    }
    if (plan->padding) zero_padding(w, p.out, p.Hq, D, tid, kThreads);
}

template <int D, int KIND, int R>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
    using C = RCfg<D, KIND, R>;
    const int G = a.Hq / a.pg.Hkv;
    RowParams p{};
    p.w = attn_work(a, R / G, C::BN < 256 ? 1 : 0);
    p.q = (const __nv_bfloat16 *)a.q;
    p.v_cache = (const __nv_bfloat16 *)a.v_cache;
    p.k_scale = a.k_scale;
    p.v_scale = a.v_scale;
    p.out = (__nv_bfloat16 *)a.out;
    p.Hq = a.Hq;
    p.q_stride = a.q_stride;
    p.negate = a.scale < 0.f;
    p.scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);  // (0 must not meet -inf)
    p.budget = wait_budget();
    CUtensorMap mk, mv;
    const int line = C::ROWB >= 128 ? C::ROWB : 128;
    const int lines = C::LINES * 16 / C::CH;  // a box holds 16 positions, which always share a page
    if (!page_map(&mk, a.k_cache, a.pg, line, lines) || !page_map(&mv, a.v_cache, a.pg, line, lines))
        return cudaErrorInvalidValue;
    auto kernel = attn_rows_kernel<D, KIND, R>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const int ctas = attn_ctas(a, p.w, C::BN);
    e = launch_early(kernel, dim3(ctas), C::THREADS, C::SM_BYTES, s, mk, mv, p);
    return e != cudaSuccess ? e : launch_attn_join(a, p.w, ctas, s);
}

template <int KIND, int R>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.d) {
        case 64: return launch_t<64, KIND, R>(a, s);
        case 128: return launch_t<128, KIND, R>(a, s);
        case 256: return launch_t<256, KIND, R>(a, s);
    }
    return cudaErrorInvalidValue;
}

// on average at most `rows` query rows per sequence and key head, and no more of one token
bool rows_fit(const AttnArgs &a, int rows) {
    const int G = a.Hq / a.pg.Hkv;
    return G <= rows && a.pg.Ttot * G <= (long)rows * a.pg.B;
}

}  // namespace

// Few rows: at most 16 with an 8-bit cache, at most 8 with a bf16 one. Measured here and in attn_tc.cu: 128 sequences of
// 4096, 2 key heads, d = 256, e4m3: 95 and 133 us with 8 rows, 113 and 136 with 16, 205 and 139 with 32 (here two passes
// over the cache); 32 of 8192, 8 key heads, d = 128, int8: 118 and 190 us with 16, 216 and 201 with 32. A bf16 cache, 8
// rows: 172 and 172, 170 and 167 us, one session of 1000 10.6 and 11.2 (from a graph); 16 rows (two passes): 323 and 175,
// 324 and 169.
bool attn_rows_supported(const AttnArgs &a) { return rows_fit(a, a.pg.cache_dtype == GDN_BF16 ? 8 : 16); }

// Tiles of 8 rows where they do: half of the products, exponentials and accumulators (32 sequences of 8192, 8 key heads
// with 4 query heads each, d = 128, int8: 97 us, 112 us in tiles of 16; 128 of 4096, d = 256, e4m3: 100 and 108 us, both
// before later steps that made the tiles of 8 1 to 4 us faster).
cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t s) {
    const bool r8 = rows_fit(a, 8);
    switch (a.pg.cache_dtype) {
        case GDN_FP8: return r8 ? launch_d<GDN_FP8, 8>(a, s) : launch_d<GDN_FP8, 16>(a, s);
        case GDN_INT8: return r8 ? launch_d<GDN_INT8, 8>(a, s) : launch_d<GDN_INT8, 16>(a, s);
        default: return launch_d<GDN_BF16, 8>(a, s);
    }
}

}  // namespace gdn
