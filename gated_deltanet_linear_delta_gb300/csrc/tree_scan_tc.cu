// tree_scan_tc.cu -- the gated delta rule over trees for bf16 inputs, on the tensor cores (formulas: tree_scan.cu).
//
// Per (sequence, value head), with T nodes and S_0 (dv x dk fp32) read once:
//     X = S_0 [K; Q]^T          S_0 split into two bf16 terms (16 bits), k and q as they are (exact)
//     A_ts, P_ts                from K K^T and Q K^T (exact products), norms, gates and paths, for s on path(t)
//     (I + A) U^T = diag(beta) V - diag(beta e^G rk) X_k^T    in blocks of 16 nodes
//     O^T = diag(e^G rq) X_q^T + P U^T
// The products are m16n8k16 (mma.sync) with 16 rows of the state a warp: the accumulator of X, columns the nodes, is
// in the layout of the next products' operand, so U never leaves registers; a block's own 16 nodes are eliminated by
// shuffles within the 4 lanes that share rows. tcgen05's M of 128 would take S_0's terms through shared memory, 64 KiB
// more to write and read a head, and U through TMEM and back for each block.
//
// What bounds it: S_0's bytes, 64 KiB a head, up to about 16 nodes; beyond, the products and the elimination.
// CTAs are persistent, two to an SM, and S_0 comes as quarters (32 columns) through a ring of three, the next head's
// while this one's nodes are eliminated.
//
// Values that are not finite stay on their paths: a product with a coefficient of 0 would spread them, so a block
// whose U is not finite is eliminated again with those left out, and rows that have them on their path become NaN.
#include "kv_pages.cuh"
#include "tree_mma.cuh"

namespace gdn {
namespace {

template <int DK, int DV, int TP>
struct Cfg {
    static constexpr int WARPS = DV / 16, THREADS = 32 * WARPS;
    static constexpr int NB = TP / 16, NT = TP / 8;      // blocks and tiles of nodes
    static constexpr int NQ = DK / 32, RING = 3;         // parts of a state; slots
    static constexpr uint32_t SLOT = DV * 128;
    static constexpr int BLOCKS = NB * (NB + 1) / 2;
    // byte offsets
    static constexpr uint32_t SM_KQ = 0;                                      // [2 TP][DK] bf16: K, then Q
    static constexpr uint32_t SM_S = SM_KQ + 2 * TP * DK * 2;                  // [RING][DV][32] fp32
    static constexpr uint32_t SM_A = SM_S + RING * SLOT;                       // -A: upper terms, lower terms
    static constexpr uint32_t SM_P = SM_A + BLOCKS * 1024;                     // P
    static constexpr uint32_t SM_D = SM_P + BLOCKS * 1024;                     // -A of the blocks' own nodes [NB][s][t] fp32
    static constexpr uint32_t SM_SC = SM_D + NB * 1024;                        // per node: Scalars
    static constexpr uint32_t SM_PATH = SM_SC + TP * 32;                       // [TP] paths
    static constexpr uint32_t SM_G = SM_PATH + TP * 8;                         // [TP] g
    static constexpr uint32_t SM_R = SM_G + TP * 4;                            // [2 TP] inverse norms of K, Q
    static constexpr uint32_t SM_BYTES = SM_R + 2 * TP * 4;
    static constexpr int FIT = 233472 / (SM_BYTES + 1024), PER_SM = FIT < 3 ? FIT : 3;  // CTAs to an SM
    static_assert(PER_SM >= 2, "two CTAs to an SM");
};

struct __align__(16) Scalars {  // of a node
    float beta, x;      // beta;  beta e^G rk, the factor of X_k
    float z, rk;        // e^G rq, the factor of X_q;  1 / |k|
    float rq, g, g_lo;  // 1 / |q|;  G as a sum of two
    float pad;
};

struct Head {
    int n, h, nodes;
    long bos, slot;
};

template <int DK, int DV, int TP>
__global__ void __launch_bounds__(Cfg<DK, DV, TP>::THREADS, Cfg<DK, DV, TP>::PER_SM) tree_scan_tc_kernel(const TreeArgs a) {
    using C = Cfg<DK, DV, TP>;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t sb = tc::smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    Scalars *sc = reinterpret_cast<Scalars *>(sm + C::SM_SC);
    uint64_t *paths = reinterpret_cast<uint64_t *>(sm + C::SM_PATH);
    float *gs = reinterpret_cast<float *>(sm + C::SM_G), *norm = reinterpret_cast<float *>(sm + C::SM_R);
    const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q, *k = (const __nv_bfloat16 *)a.k, *v = (const __nv_bfloat16 *)a.v;
    const __nv_bfloat16 *ga = (const __nv_bfloat16 *)a.g, *be = (const __nv_bfloat16 *)a.b;
    __nv_bfloat16 *out = (__nv_bfloat16 *)a.out;
    const int heads = a.B * a.Hv, r = a.Hv / a.Hk;
    next_may_begin();
    before_reading();

    // The next head from `i` on that has nodes and a state; heads of padding sequences are written as zeros on the way.
    auto find = [&](int &i) -> Head {
        Head hd{0, 0, 0, 0, -1};
        for (; i < heads; i += gridDim.x) {
            hd.n = i / a.Hv;
            hd.h = i % a.Hv;
            if (!tree_bounds(a.cu, hd.n, a.B, a.cu ? a.Ttot : a.T, &hd.bos, &hd.nodes, a.status) || hd.nodes == 0) continue;
            hd.slot = state_slot(a, hd.n);
            if (hd.slot >= 0) break;
            for (int e = tid; e < hd.nodes * (DV / 8); e += C::THREADS)
                reinterpret_cast<uint4 *>(out + ((hd.bos + e / (DV / 8)) * a.Hv + hd.h) * DV)[e % (DV / 8)] = make_uint4(0, 0, 0, 0);
        }
        if (i >= heads) hd.slot = -1;
        return hd;
    };
    auto load_kq = [&](const Head &hd) {
        if (hd.slot >= 0) {
            constexpr int PR = DK / 8;
            const int hk = hd.h / r;
            for (int e = tid; e < hd.nodes * PR; e += C::THREADS) {
                const int t = e / PR, ch = e % PR;
                const long at = ((hd.bos + t) * a.Hk + hk) * DK + 8 * ch;
                copy16(sb + C::SM_KQ + row_piece<DK>(t, ch), k + at);
                copy16(sb + C::SM_KQ + row_piece<DK>(TP + t, ch), q + at);
            }
        }
        copies_commit();
    };
    auto load_state = [&](const Head &hd, int part, int slot) {
        if (hd.slot >= 0) {
            const float *src = a.state_in + (hd.slot * a.Hv + hd.h) * (long)(DV * DK) + part * 32;
            for (int e = tid; e < DV * 8; e += C::THREADS)
                copy16(sb + C::SM_S + slot * C::SLOT + state_piece(e >> 3, e & 7), src + (e >> 3) * DK + (e & 7) * 4);
        }
        copies_commit();
    };
    // this thread's node's gate and beta logit
    auto load_gates = [&](const Head &hd, float &gv, float &bv) {
        gv = bv = 0.f;
        if (hd.slot >= 0 && tid < hd.nodes) {
            gv = to_f32(ga[(hd.bos + tid) * a.Hv + hd.h]);
            bv = to_f32(be[(hd.bos + tid) * a.Hv + hd.h]);
        }
    };

    // Parts follow one another through the ring, head by head: after a part is used, the one three further on is asked
    // for; a head's keys and queries once those of the head before are, just before the part asked for at its last.
    int next_i = blockIdx.x;
    Head cur = find(next_i), next{0, 0, 0, 0, -1}, ahead{0, 0, 0, 0, -1};
    auto step_to = [&](const Head &from) -> Head {
        if (from.slot < 0) return from;
        next_i += gridDim.x;
        return find(next_i);
    };
    // with one or two parts to a head, three parts ahead is up to three heads ahead
    constexpr int AHEAD = (C::RING + C::NQ - 1) / C::NQ;  // heads to know of beside the one at hand
    static_assert(AHEAD <= 3, "heads ahead");
    Head more{0, 0, 0, 0, -1};
    next = step_to(cur);
    if (AHEAD > 1) ahead = step_to(next);
    if (AHEAD > 2) more = step_to(ahead);
    auto head_of = [&](int d) -> const Head & { return d == 0 ? cur : d == 1 ? next : d == 2 ? ahead : more; };
    int slot = 0;  // of the part at hand
#pragma unroll
    for (int i = -C::RING; i < 0; ++i) {
        if ((i + 1) % C::NQ == 0) {
            if (i == -1) load_kq(cur);
            else copies_commit();
        }
        load_state(head_of((i + C::RING) / C::NQ), (i + C::RING) % C::NQ, i + C::RING);
    }
    float gv, bv;
    load_gates(cur, gv, bv);
    while (cur.slot >= 0) {
        const int T = cur.nodes, nb = (T + 15) / 16;
        copies_wait<1>();  // keys and queries
        if (tid < TP) gs[tid] = gv;
        if (warp == 0) {
            const Paths p = tree_paths(a.parents + cur.bos, T, a.status);
            if (lane < TP) paths[lane] = p.of(0);
            if (TP > 32) paths[lane + 32] = p.of(1);
        }
        __syncthreads();
        // ---- norms, gates -----------------------------------------------------------
        for (int row = warp * 16 + (lane >> 1); row < 2 * TP; row += C::WARPS * 16) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 16; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(sm + C::SM_KQ + row_piece<DK>(row, (lane & 1) * (DK / 16) + i));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xffff0000u);
                    s = fmaf(lo, lo, s);
                    s = fmaf(hi, hi, s);
                }
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            if (!(lane & 1)) norm[row] = 1.f / sqrtf(s + kNormEps);
        }
        float hi = 0.f, lo = 0.f;
        if (tid < T)
            for (uint64_t m = paths[tid]; m; m &= m - 1) add_exact(hi, lo, gs[__ffsll((long long)m) - 1]);
        __syncthreads();
        if (tid < TP) {
            Scalars s;
            const float eg = expf(hi + lo);
            s.beta = sigmoidf_(bv);
            s.rk = norm[tid];
            s.rq = norm[TP + tid];
            s.x = s.beta * eg * s.rk;
            s.z = eg * s.rq;
            s.g = hi;
            s.g_lo = lo;
            s.pad = 0.f;
            sc[tid] = s;
        }
        __syncthreads();
        // ---- A and P: 16 rows of K or Q with all nodes before them, a warp each -----------------
        for (int mt = warp; mt < 2 * C::NB; mt += C::WARPS) {
            const bool is_p = mt >= C::NB;
            const int i = is_p ? mt - C::NB : mt;
            if (i >= nb) continue;
            float acc[C::NT][4];
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t x[4];
                load_matrices(x, sb + C::SM_KQ + row_piece<DK>((is_p ? TP : 0) + 16 * i + (lane & 15), 2 * ks + (lane >> 4)));
#pragma unroll
                for (int j = 0; j < C::NB; ++j)
                    if (j <= i) {
                        uint32_t y[4];
                        load_matrices(y, sb + C::SM_KQ + row_piece<DK>(16 * j + ((lane >> 4) << 3) + (lane & 7), 2 * ks + ((lane >> 3) & 1)));
                        mma_bf16_16816(acc[2 * j], x, y[0], y[1]);
                        mma_bf16_16816(acc[2 * j + 1], x, y[2], y[3]);
                    }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int tr = g + 8 * half, t = 16 * i + tr;
                const Scalars st = sc[t];
                uint64_t on = t < T ? paths[t] : 0;
                if (!is_p) on &= ~(1ull << t);
                const float f = is_p ? st.rq : -st.beta * st.rk;
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                    if (n > 2 * i + 1) continue;
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int s = 8 * n + 2 * c + e;
                        const Scalars ss = sc[s];
                        const float d = __expf((st.g - ss.g) + (st.g_lo - ss.g_lo));
                        w[e] = (on >> s) & 1 ? acc[n][2 * half + e] * (f * ss.rk) * d : 0.f;
                    }
                    if (!is_p && n >= 2 * i) {
                        float *dg = reinterpret_cast<float *>(sm + C::SM_D) + i * 256 + (8 * (n & 1) + 2 * c) * 16 + tr;
                        dg[0] = w[0];
                        dg[16] = w[1];
                    } else {
                        const uint32_t at = (is_p ? C::SM_P : C::SM_A) + coef_block(i, n >> 1) + coef_piece(tr, n & 1) + 4 * c;
                        *reinterpret_cast<uint32_t *>(sm + at) = split2(w[0], w[1]);
                        *reinterpret_cast<uint32_t *>(sm + at + C::BLOCKS * 512) = tc::bf2_bits(__floats2bfloat162_rn(w[0], w[1]));
                    }
                }
            }
        }
        // ---- X = S_0 [K; Q]^T, and the values on their way ---------------------------------------
        const int row0 = 16 * warp + 2 * g;  // this lane's rows of the state (the products' rows g and g + 8): row0, row0 + 1
        uint32_t vv[C::NT][2];  // rows row0, row0 + 1 of nodes 8 n + 2 c, + 1
        const long vat = (cur.bos * a.Hv + cur.h) * DV + row0;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * n + 2 * c + e;
                vv[n][e] = t < T ? *reinterpret_cast<const uint32_t *>(v + vat + (long)t * a.Hv * DV) : 0u;
            }
        float xk[C::NT][4], xq[C::NT][4];
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) xk[n][e] = xq[n][e] = 0.f;
#pragma unroll
        for (int part = 0; part < C::NQ; ++part) {
            constexpr int LATE0 = 2;  // groups after this part's: the two parts after it, and keys and queries in between
            if (C::NQ == 1) copies_wait<LATE0 + 2>();
            else if (C::NQ == 2 || part < 2) copies_wait<LATE0 + 1>();
            else copies_wait<LATE0>();
            __syncthreads();
            const uint8_t *s0 = sm + C::SM_S + slot * C::SLOT;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int ks = 2 * part + kk;
                uint32_t ah[4], al[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // rows row0, row0 + 1 (e & 1) of columns 2 c .., 2 c + 8 .. (e >> 1)
                    float2 x = *reinterpret_cast<const float2 *>(s0 + state_piece(row0 + (e & 1), 4 * kk + 2 * (e >> 1) + (c >> 1)) +
                                                                 8 * (c & 1));
                    ah[e] = split2(x.x, x.y);
                    al[e] = tc::bf2_bits(__floats2bfloat162_rn(x.x, x.y));
                }
#pragma unroll
                for (int j = 0; j < C::NB; ++j)
                    if (j < nb) {
                        const int rr = 16 * j + ((lane >> 4) << 3) + (lane & 7), ch = 2 * ks + ((lane >> 3) & 1);
                        uint32_t y[4];
                        load_matrices(y, sb + C::SM_KQ + row_piece<DK>(rr, ch));
                        mma_bf16_16816(xk[2 * j], ah, y[0], y[1]);
                        mma_bf16_16816(xk[2 * j + 1], ah, y[2], y[3]);
                        mma_bf16_16816(xk[2 * j], al, y[0], y[1]);
                        mma_bf16_16816(xk[2 * j + 1], al, y[2], y[3]);
                        load_matrices(y, sb + C::SM_KQ + row_piece<DK>(TP + rr, ch));
                        mma_bf16_16816(xq[2 * j], ah, y[0], y[1]);
                        mma_bf16_16816(xq[2 * j + 1], ah, y[2], y[3]);
                        mma_bf16_16816(xq[2 * j], al, y[0], y[1]);
                        mma_bf16_16816(xq[2 * j + 1], al, y[2], y[3]);
                    }
            }
            __syncthreads();  // the slot, and after the last part keys and queries, may be filled again
            if (part + 1 == C::NQ) {
                load_kq(next);
                load_gates(next, gv, bv);
            }
            load_state(head_of((part + C::RING) / C::NQ), (part + C::RING) % C::NQ, slot);
            if (++slot == C::RING) slot = 0;
        }
        // ---- U, and O block by block --------------------------------------------------------------
        uint64_t bad0 = 0, bad1 = 0;  // nodes whose U is not finite in this lane's rows
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * n + 2 * c + e;
                const Scalars st = sc[t];
                const bool live = t < T && paths[t] != 0;
                const float v0 = __uint_as_float(vv[n][e] << 16), v1 = __uint_as_float(vv[n][e] & 0xffff0000u);
                xk[n][e] = live ? st.beta * v0 - st.x * xk[n][e] : 0.f;
                xk[n][2 + e] = live ? st.beta * v1 - st.x * xk[n][2 + e] : 0.f;
                xq[n][e] *= st.z;
                xq[n][2 + e] *= st.z;
            }
#pragma unroll
        for (int j = 0; j < C::NB; ++j) {
            if (j >= nb) continue;
            const float *dg = reinterpret_cast<const float *>(sm + C::SM_D) + j * 256;
            float x[2][4], sure = 0.f;
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[y][e] = xk[2 * j + y][e];
            auto eliminate = [&](bool careful) {
#pragma unroll
                for (int s = 0; s < 16; ++s) {
                    const int owner = (lane & ~3) | ((s & 7) >> 1);
                    float u0 = __shfl_sync(0xffffffffu, x[s >> 3][s & 1], owner), u1 = __shfl_sync(0xffffffffu, x[s >> 3][2 + (s & 1)], owner);
                    if (careful) {
                        if (!(fabsf(u0) < INFINITY)) {
                            bad0 |= 1ull << (16 * j + s);
                            u0 = 0.f;
                        }
                        if (!(fabsf(u1) < INFINITY)) {
                            bad1 |= 1ull << (16 * j + s);
                            u1 = 0.f;
                        }
                        if (lane == owner) {
                            x[s >> 3][s & 1] = u0;
                            x[s >> 3][2 + (s & 1)] = u1;
                        }
                    }
#pragma unroll
                    for (int y = s >> 3; y < 2; ++y) {
                        const float2 w = *reinterpret_cast<const float2 *>(dg + s * 16 + 8 * y + 2 * c);
                        x[y][0] = fmaf(w.x, u0, x[y][0]);
                        x[y][1] = fmaf(w.y, u0, x[y][1]);
                        x[y][2] = fmaf(w.x, u1, x[y][2]);
                        x[y][3] = fmaf(w.y, u1, x[y][3]);
                    }
                }
            };
            eliminate(false);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) sure = fmaf(x[y][e], 0.f, sure);  // 0, or NaN
            if (__any_sync(0xffffffffu, sure != 0.f)) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[y][e] = xk[2 * j + y][e];
                eliminate(true);
            }
            uint32_t uh[4], ul[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo0 = x[e >> 1][2 * (e & 1)], lo1 = x[e >> 1][2 * (e & 1) + 1];
                uh[e] = split2(lo0, lo1);
                ul[e] = tc::bf2_bits(__floats2bfloat162_rn(lo0, lo1));
            }
            const uint32_t at = sb + coef_piece(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);
#pragma unroll
            for (int i = j; i < C::NB; ++i) {
                if (i >= nb) continue;
                uint32_t y[4];
                auto products = [&](float (&d0)[4], float (&d1)[4], uint32_t from) {
                    load_matrices(y, at + from + coef_block(i, j));
                    mma_bf16_16816(d0, uh, y[0], y[1]);
                    mma_bf16_16816(d1, uh, y[2], y[3]);
                    mma_bf16_16816(d0, ul, y[0], y[1]);
                    mma_bf16_16816(d1, ul, y[2], y[3]);
                    load_matrices(y, at + from + C::BLOCKS * 512 + coef_block(i, j));
                    mma_bf16_16816(d0, uh, y[0], y[1]);
                    mma_bf16_16816(d1, uh, y[2], y[3]);
                };
                if (i > j) products(xk[2 * i], xk[2 * i + 1], C::SM_A);
                products(xq[2 * i], xq[2 * i + 1], C::SM_P);
            }
        }
        // ---- rows out -----------------------------------------------------------------------------
        const bool any_bad = (bad0 | bad1) != 0;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * n + 2 * c + e;
                if (t >= T) continue;
                float o0 = xq[n][e], o1 = xq[n][2 + e];
                if (any_bad) {
                    if (bad0 & paths[t]) o0 = __int_as_float(0x7fffffff);
                    if (bad1 & paths[t]) o1 = __int_as_float(0x7fffffff);
                }
                *reinterpret_cast<uint32_t *>(out + vat + (long)t * a.Hv * DV) = tc::bf2_bits(__floats2bfloat162_rn(o0, o1));
            }
        __syncthreads();  // paths, scalars and coefficients have been read
        cur = next;
        next = ahead;
        if (AHEAD == 1) {
            next = step_to(cur);
        } else if (AHEAD == 2) {
            ahead = step_to(next);
        } else {
            ahead = more;
            more = step_to(ahead);
        }
    }
    copies_wait<0>();
}

template <int DK, int DV, int TP>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    using C = Cfg<DK, DV, TP>;
    auto kernel = tree_scan_tc_kernel<DK, DV, TP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const long heads = (long)a.B * a.Hv, most = 152L * C::PER_SM;
    return launch_early(kernel, dim3((unsigned)(heads < most ? heads : most)), C::THREADS, C::SM_BYTES, s, a);
}

template <int DK, int DV>
cudaError_t launch_tp(const TreeArgs &a, cudaStream_t s) {
    const long most = a.cu ? a.Ttot : a.T;  // nodes of a sequence
    if (most <= 16) return launch_t<DK, DV, 16>(a, s);
    return launch_t<DK, DV, 64>(a, s);
}

template <int DK>
cudaError_t launch_dv(const TreeArgs &a, cudaStream_t s) {
    switch (a.dv) {
        case 32: return launch_tp<DK, 32>(a, s);
        case 64: return launch_tp<DK, 64>(a, s);
        case 128: return launch_tp<DK, 128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree_scan_tc(const TreeArgs &a, cudaStream_t s) {
    switch (a.dk) {
        case 32: return launch_dv<32>(a, s);
        case 64: return launch_dv<64>(a, s);
        case 128: return launch_dv<128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
