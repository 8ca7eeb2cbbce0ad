// attn_rows.cu -- attention over a paged cache for few query rows per key head (bf16 inputs): the
// decode step and the check of a few speculated tokens.
//
// With at most 16 rows (the G query heads of a key head, of a few tokens) every cached row is read
// for 16 rows' worth of products at most, 16 to 32 flops a byte, so the kernel is bound by the bytes
// of the cache and, for short ones, by the length of its own dependent chain. It therefore keeps
// everything of a key chunk inside one warp: a CTA's 8 warps take 16 positions each of a 128-position
// tile, every warp has its own ring of tiles in flight (TMA, one box per 128 bytes of row, 128B
// swizzle), its own running softmax and its own 16 x D output in registers, and meets the others
// only once per unit of work, in shared memory. The products are m16n8k16 (mma.sync): 16 rows fill
// its M, where tcgen05's M of 128 would be padded 8 to 16 times and needs hand-overs between warps
// for each tile.
//
// Fragments without shuffles. The sums over d and over keys may run in any order, so both are
// permuted such that a thread's operands are 16-byte pieces of a row, free of bank conflicts:
//   S = Q K^T : of a piece of row n, each 4 elements in turn are the thread's k indexes of one
//               product; Q's fragments are laid out in the same order, once per unit;
//   O += P V  : column n of product t is d = 8 n + t of a 64-wide block (bf16; 16 n + t of 128 for
//               8-bit codes), so that a thread ends with 16 (32) consecutive elements of its rows;
//   position r of a chunk stands at column c with r = g(c), g = 0 4 2 6 5 1 7 3.
// 8-bit codes become fp16 in registers (attn_tc.cu says why fp16, and how the scales enter).
#include <climits>

#include "attn_ops.cuh"

namespace gdn {
namespace {

using namespace tc;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr uint32_t kRingBytes = 24576;  // of each warp

template <int D, int KIND>
struct RCfg {
    static constexpr bool kCodes = KIND == GDN_FP8 || KIND == GDN_INT8;
    static constexpr int ROWB = D * (kCodes ? 1 : 2);           // bytes of a row
    // Positions per chunk. 32 spread what a chunk costs beside its products (waits, loads, softmax steps: half of a
    // 16-position chunk's instructions at 128-byte rows); wider rows need 16 for at least two chunks in flight.
    static constexpr int CH = ROWB <= 128 ? 32 : 16;
    static constexpr int U = CH / 8;                            // score tiles of a chunk
    static constexpr int BN = kWarps * CH;                      // positions per tile of work
    static constexpr int BOXES = ROWB >= 128 ? ROWB / 128 : 1;  // TMA boxes per 16 positions
    static constexpr int LINES = ROWB >= 128 ? CH : CH / 2;     // 128-byte lines of a chunk per 128 bytes of row
    static constexpr uint32_t SLOT = CH * ROWB;                 // K or V of a chunk
    // A chunk's K and V come as one stage of the ring, unless that leaves less than two stages (bf16, D = 256):
    // then K and V take turns in slots of their own.
    static constexpr bool kPair = kRingBytes / (2 * SLOT) >= 2;
    static constexpr uint32_t STAGE = kPair ? 2 * SLOT : SLOT;
    static constexpr int NSL = kRingBytes / STAGE;
    static constexpr int KS = D / 16;                           // products per score tile
    static constexpr int VE = kCodes ? (D == 64 ? 8 : 16) : 8;  // elements per piece of V
    static constexpr int MSTRIDE = D + 4;                       // floats per row where warps meet
    static constexpr uint32_t RING = kWarps * NSL * STAGE, MEET = kWarps * 16 * MSTRIDE * 4;
    static constexpr uint32_t SM_Q = RING > MEET ? RING : MEET;  // Q fragments [KS][32 lanes][16 bytes]
    static constexpr uint32_t SM_SC = SM_Q + KS * 512;           // [warp][NSL][k, v][CH] scales
    static constexpr uint32_t SM_ML = SM_SC + (kCodes ? kWarps * NSL * 2 * CH * 4 : 0);  // [warp][16] m, l
    static constexpr uint32_t SM_RS = SM_ML + kWarps * 16 * 8;   // [16] Q row scales, and factors
    static constexpr uint32_t SM_BAR = SM_RS + 16 * 4;
    static constexpr uint32_t SM_PLAN = SM_BAR + kWarps * NSL * 8;
    static constexpr uint32_t SM_BYTES = SM_PLAN + sizeof(PlanSmem) + 1024;
    static_assert(SM_BYTES <= 232448, "over the 227 KiB opt-in limit");
};

struct RowParams {
    AttnWork w;
    const __nv_bfloat16 *q;
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
attn_rows_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const RowParams p) {
    using C = RCfg<D, KIND>;
    constexpr int CH = C::CH, U = C::U, BN = C::BN;
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid == 0) {
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    if (lane == 0) {
        for (int s = 0; s < C::NSL; ++s) mbar_init(bar + s, 1);
        fence_mbar_init();
    }
    plan_piece<BN, kThreads>(w, plan);  // (synchronises the CTA)
    Piece pc = plan->piece;
    const int P_shift = 31 - __clz(pg.page_size);
    uint32_t filled = 0, used_up = 0;  // ring slots of this warp
    uint32_t fslot = 0, uslot = 0, uphase = 0;
    bool failed = false;
    // 16 positions of a stage whose scales are not loaded: keys and values of zero
    auto clear_scales = [&](float *sc, int at) {
        sc[(lane < 16 ? 0 : CH) + at + (lane & 15)] = lane < 16 ? 0.f : kMinKvScale;
        fence_async_smem();
    };
    auto bad_page = [&](float *sc, int at) {  // outside of the pool (the copies read zeros)
        if (lane == 0) flag_error(pg.status);
        if (C::kCodes) clear_scales(sc, at);
    };
    for (bool begun = pc.off == 0; pc.left > 0; begun = true) {
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
        for (int e = tid; e < 16 * (D / 8); e += kThreads) {
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
            // elements 8 c + 4 s ..: of product ks, lane (r % 8, qq); registers r / 8 and 2 + r / 8
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int ks = C::kCodes ? (c / 8) * 4 + (c & 1) * 2 + s : (c / 4) * 2 + s;
                const int qq = C::kCodes ? (c / 2) & 3 : c & 3;
                uint32_t *dst = qf + (ks * 32 + (r & 7) * 4 + qq) * 4 + (r >> 3);
                dst[0] = x[2 * s];
                dst[2] = x[2 * s + 1];
            }
        }
        __syncthreads();

        float o[D / 8][4];
#pragma unroll
        for (int t = 0; t < D / 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int limit[2];  // last position that rows n and n + 8 see
        float rsc[2] = {1.f, 1.f};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = n + 8 * i;
            limit[i] = r < rows ? len - pc.s.T + t0 + r / w.G : INT_MAX;  // (rows past the last are not read)
            if (C::kCodes) rsc[i] = rs[r];
        }
        const int sure = len - pc.s.T + t0;  // every row sees up to here
        for (int ch = 0; ch < chunks && !failed; ++ch) {
            const int pos0 = start + ch * BN;
            wait_full();
            if (failed) break;
            constexpr int SPLIT = U == 2 ? 2 : 1;  // chains of products per score tile
            float s[U][SPLIT][4];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int y = 0; y < SPLIT; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[u][y][i] = 0.f;
            const uint8_t *kc = ring + uslot * C::STAGE;
            constexpr int KP = C::kCodes ? 4 : 2;  // products per piece
#pragma unroll
            for (int i = 0; i < C::KS / KP; ++i) {
                uint4 a[KP];
#pragma unroll
                for (int x = 0; x < KP; ++x) a[x] = *reinterpret_cast<const uint4 *>(qf + ((i * KP + x) * 32 + lane) * 4);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(kc + piece_at<C::ROWB, CH>(u * 8 + gn, 4 * i + q));
                    if constexpr (C::kCodes) {
                        const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            uint32_t h0, h1;
                            codes4_to_f16<KIND>(bw[x], h0, h1);
                            mma16816<true>(s[u][x & (SPLIT - 1)], a[x], h0, h1);
                        }
                    } else {
                        mma16816<false>(s[u][0], a[0], b.x, b.y);
                        mma16816<false>(s[u][SPLIT - 1], a[1], b.z, b.w);
                    }
                }
            }
            float iv[U][2];
            float x[U][4];  // [score tile]: rows n, n, n + 8, n + 8; columns 2 q, 2 q + 1, ..
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = SPLIT == 2 ? s[u][0][i] + s[u][SPLIT - 1][i] : s[u][0][i];
                if constexpr (C::kCodes) {
                    const float *sc = scales + uslot * 2 * CH + u * 8;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float a = sc[g2 ^ (4 * j)] * p.scale2;
                        float vs = sc[CH + (g2 ^ (4 * j))];
                        if (vs < kMinKvScale) vs = kMinKvScale;  // (a NaN stays)
                        const float lv = lg2(vs);
                        iv[u][j] = vs == vs ? rcp(vs) : 0.f;  // a NaN enters by lv, and not where it is masked
                        x[u][j] = fmaf(x[u][j] * rsc[0], a, lv);
                        x[u][2 + j] = fmaf(x[u][2 + j] * rsc[1], a, lv);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[u][i] *= p.scale2;
                }
            }
            if (!C::kPair) release();
            if (pos0 + CH - 1 > sure) {
                const int lim[2] = {limit[0] - pos0 - g2, limit[1] - pos0 - g2}, lim4[2] = {limit[0] - pos0 - (g2 ^ 4), limit[1] - pos0 - (g2 ^ 4)};
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (u * 8 > ((i & 1) ? lim4[i >> 1] : lim[i >> 1])) x[u][i] = -INFINITY;
            }
            float f[2];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = fmaxf(x[0][2 * i], x[0][2 * i + 1]);
#pragma unroll
                for (int u = 1; u < U; ++u) top = fmaxf(top, fmaxf(x[u][2 * i], x[u][2 * i + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                grow |= grow_reference(m[i], top, f[i]);
                l[i] *= f[i];
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int t = 0; t < D / 8; ++t) {
                    o[t][0] *= f[0]; o[t][1] *= f[0];
                    o[t][2] *= f[1]; o[t][3] *= f[1];
                }
            }
            uint32_t pr[U / 2][4];  // P as the A operand of U / 2 products
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float e0 = ex2(x[u][2 * i] - ref), e1 = ex2(x[u][2 * i + 1] - ref);
                    if constexpr (C::kCodes) {
                        l[i] = fmaf(e0, iv[u][0], l[i]);
                        l[i] = fmaf(e1, iv[u][1], l[i]);
                        pr[u >> 1][2 * (u & 1) + i] = h2_bits(e0, e1);
                    } else {
                        l[i] += e0 + e1;
                        pr[u >> 1][2 * (u & 1) + i] = bf2_bits(__floats2bfloat162_rn(e0, e1));
                    }
                }
            }
            if constexpr (!C::kPair) {
                wait_full();
                if (failed) break;
            }
            const uint8_t *vc = ring + uslot * C::STAGE + (C::kPair ? C::SLOT : 0);
            const bool tail = pos0 + CH > len;  // rows past the end: zeros
#pragma unroll
            for (int hk = 0; hk < U / 2; ++hk) {
                const uint4 pa = make_uint4(pr[hk][0], pr[hk][1], pr[hk][2], pr[hk][3]);
#pragma unroll
                for (int b = 0; b < D / (8 * C::VE); ++b) {
                    uint32_t v[4][4];  // positions g2, g2 ^ 4, 8 + g2, 8 + (g2 ^ 4)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = hk * 16 + (j >> 1) * 8 + (g2 ^ (4 * (j & 1)));
                        if (C::VE * (C::kCodes ? 1 : 2) == 16) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(vc + piece_at<C::ROWB, CH>(r, b * 8 + n));
                            v[j][0] = y.x; v[j][1] = y.y; v[j][2] = y.z; v[j][3] = y.w;
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2 *>(vc + piece_at<C::ROWB, CH>(r, n >> 1) + (n & 1) * 8);
                            v[j][0] = y.x; v[j][1] = y.y; v[j][2] = v[j][3] = 0;
                        }
                        if (tail && pos0 + r >= len) v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0;
                    }
                    if constexpr (C::kCodes) {
#pragma unroll
                        for (int wd = 0; wd < C::VE / 4; ++wd) {
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {  // elements 4 wd + 2 hf, + 1
                                uint32_t b0[2], b1[2];
                                codes4_to_f16<KIND>(__byte_perm(v[0][wd], v[1][wd], hf ? 0x7362 : 0x5140), b0[0], b0[1]);
                                codes4_to_f16<KIND>(__byte_perm(v[2][wd], v[3][wd], hf ? 0x7362 : 0x5140), b1[0], b1[1]);
#pragma unroll
                                for (int y = 0; y < 2; ++y)
                                    mma16816<true>(o[b * C::VE + 4 * wd + 2 * hf + y], pa, b0[y], b1[y]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            const uint32_t sel = t & 1 ? 0x7632 : 0x5410;
                            mma16816<false>(o[b * 8 + t], pa, __byte_perm(v[0][t / 2], v[1][t / 2], sel),
                                            __byte_perm(v[2][t / 2], v[3][t / 2], sel));
                        }
                    }
                }
            }
            release();
        }
        // the warps meet: O over the rings, which are empty now
        if (__syncthreads_or(failed)) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = n + 8 * i;
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (q == 0) ml[warp * 16 + r] = make_float2(m[i], l[i]);
            if (r < rows && chunks > 0) {
                // columns 2 q and 2 q + 1 of products 0 .. VE - 1 of a block: 2 VE consecutive elements
                float *dst = reinterpret_cast<float *>(sm) + (warp * 16 + r) * C::MSTRIDE + q * 2 * C::VE;
#pragma unroll
                for (int b = 0; b < D / (8 * C::VE); ++b)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int t = 0; t < C::VE; t += 4)
                            *reinterpret_cast<float4 *>(dst + b * 8 * C::VE + j * C::VE + t) =
                                make_float4(o[b * C::VE + t][2 * i + j], o[b * C::VE + t + 1][2 * i + j],
                                            o[b * C::VE + t + 2][2 * i + j], o[b * C::VE + t + 3][2 * i + j]);
            }
        }
        __syncthreads();
        const bool whole = begun && off + take == pc.ntiles;
        for (int e = tid; e < rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) M = fmaxf(M, ml[x * 16 + r].x);
            const float ref = M == -INFINITY ? 0.f : M;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float2 a = ml[x * 16 + r];
                if (a.x == -INFINITY && a.y == 0.f) continue;  // nothing seen
                const float f = ex2(a.x - ref);
                const float4 z = *reinterpret_cast<const float4 *>(reinterpret_cast<float *>(sm) + (x * 16 + r) * C::MSTRIDE + c);
                L = fmaf(f, a.y, L);
                y.x = fmaf(f, z.x, y.x); y.y = fmaf(f, z.y, y.y); y.z = fmaf(f, z.z, y.z); y.w = fmaf(f, z.w, y.w);
            }
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
        pc.left -= take;
        if (pc.left > 0) next_unit<BN>(w, &pc);
        fence_async_smem();  // the rings held O: before the next unit's copies
        __syncthreads();
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

template <int D, int KIND>
cudaError_t launch_t(const AttnArgs &a, cudaStream_t s) {
    using C = RCfg<D, KIND>;
    const int G = a.Hq / a.pg.Hkv;
    RowParams p{};
    p.w = attn_work(a, 16 / G, C::CH == 16 ? 2 : 1);
    p.q = (const __nv_bfloat16 *)a.q;
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
    auto kernel = attn_rows_kernel<D, KIND>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const int ctas = attn_ctas(a, p.w, C::BN);
    kernel<<<ctas, kThreads, C::SM_BYTES, s>>>(mk, mv, p);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_attn_join(a, p.w, ctas, s);
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

// Few rows: on average at most 16 per sequence and key head, and 16 query heads per key head at most.
bool attn_rows_supported(const AttnArgs &a) {
    const int G = a.Hq / a.pg.Hkv;
    return G <= 16 && a.pg.Ttot * G <= 16L * a.pg.B;
}

cudaError_t launch_attn_rows(const AttnArgs &a, cudaStream_t s) {
    switch (a.pg.cache_dtype) {
        case GDN_FP8: return launch_d<GDN_FP8>(a, s);
        case GDN_INT8: return launch_d<GDN_INT8>(a, s);
        default: return launch_d<GDN_BF16>(a, s);
    }
}

}  // namespace gdn
