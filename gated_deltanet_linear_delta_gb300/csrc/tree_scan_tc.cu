// tree_scan_tc.cu -- the gated delta rule over trees for bf16 inputs, on the tensor cores (formulas: tree_scan.cu).
//
// Per (sequence, value head), with T nodes, on(t) the nodes on path(t) and S_0 (dv x dk fp32) read once:
//     X = S_0 [K; Q]^T             S_0 split into two bf16 terms (16 bits), k and q as they are (exact)
//     R_s = beta_s v_s - beta_s e^{G_s} rk_s X_k,s          what u_s is without the nodes above it
//     O_t = e^{G_t} rq_t X_q,t + sum_{s in on(t)} W_ts R_s
// W is P (I + A)^-1: a node's sum over the corrections u of its path, put in terms of R. Its rows are independent of
// one another, and the decays and norms stand outside of them: W_ts = e^{G_t-G_s} rk_s w_s, where from t upwards
//     w_s = rq_t (q_t.k_s) - sum_{s' in on(t), s' > s} w_s' beta_s' rk_s'^2 (k_s'.k_s),
// with the raw products of K K^T and Q K^T. So a row costs L^2 / 2 multiply-adds for a path of L nodes, by four lanes,
// once per head; and the dv rows of the state, 16 to a warp, take no elimination of their own, just products.
//
// The products are m16n8k16 (mma.sync): their accumulator, rows of the state by nodes, is in the layout of the next
// product's operand, so that R goes from X to O within registers. tcgen05's M of 128 would take S_0's two terms through
// shared memory (64 KiB more to write and read a head) and R through TMEM and back.
//
// What bounds it: S_0's bytes, 64 KiB a head, for few nodes; for many the products, 2 dk (2 T) dv multiply-adds a head
// at mma.sync's 1024 a cycle and SM, and the instructions around them.
// CTAs are persistent, two or three to an SM, and S_0 comes in parts of 32 columns through a ring of three, the next
// head's during the end of this one's work.
//
// Values that are not finite stay on their paths: a product with a coefficient of 0 would spread them, so they are
// left out of the products, and the outputs that have them on their path become NaN.
#include "kv_pages.cuh"
#include "tree_mma.cuh"

namespace gdn {
namespace {

template <int DK, int DV, int TP>
struct Cfg {
    static constexpr int WARPS = DV / 16, THREADS = 32 * WARPS;
    static constexpr int NB = TP / 16, NT = TP / 8;      // blocks and tiles of nodes
    static constexpr int NQ = DK / 32, RING = TP == 16 ? 4 : 3;  // parts of a state; slots
    static constexpr uint32_t SLOT = DV * 128;
    static constexpr int BLOCKS = NB * (NB + 1) / 2;
    // byte offsets
    static constexpr uint32_t SM_KQ = 0;                                      // [2 TP][DK] bf16: K, then Q
    static constexpr uint32_t SM_S = SM_KQ + 2 * TP * DK * 2;                  // [RING][DV][32] fp32
    static constexpr uint32_t SM_A = SM_S + RING * SLOT;                       // K K^T, blocks of 16 x 16 fp32
    static constexpr uint32_t SM_W = SM_A + BLOCKS * 1024;                     // Q K^T, then W, fp32, then W as two terms
    static constexpr uint32_t SM_SC = SM_W + BLOCKS * 1024;                    // per node: Scalars
    static constexpr uint32_t SM_PATH = SM_SC + TP * 32;                       // [TP] paths
    static constexpr uint32_t SM_G = SM_PATH + TP * 8;                         // [TP] g
    static constexpr uint32_t SM_R = SM_G + TP * 4;                            // [TP] |q|^2
    static constexpr uint32_t SM_BYTES = SM_R + TP * 4;
    static constexpr int FIT = 233472 / (SM_BYTES + 1024), PER_SM = FIT < 3 ? FIT : 3;  // CTAs to an SM
    static_assert(PER_SM >= 2, "two CTAs to an SM");
};

struct __align__(16) Scalars {  // of a node
    float beta, x;   // beta;  beta e^G rk, the factor of X_k
    float z, rk;     // e^G rq, the factor of X_q;  1 / |k|
    float rq, b2;    // 1 / |q|;  beta rk^2
    float g, g_lo;   // G as a sum of two
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
    float *gs = reinterpret_cast<float *>(sm + C::SM_G), *qq = reinterpret_cast<float *>(sm + C::SM_R);
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
    auto state_of = [&](const Head &hd) { return hd.slot >= 0 ? a.state_in + (hd.slot * a.Hv + hd.h) * (long)(DV * DK) : nullptr; };
    auto load_state = [&](const float *state, int part, int slot) {
        if (state != nullptr) {
            const float *src = state + part * 32;
            for (int e = tid; e < DV * 8; e += C::THREADS)
                copy16(sb + C::SM_S + slot * C::SLOT + state_piece(e >> 3, e & 7), src + (e >> 3) * DK + (e & 7) * 4);
        }
        copies_commit();
    };
    // the node of a thread of the last warps, its gate and beta logit
    const int node = tid - (C::THREADS - TP);
    auto load_gates = [&](const Head &hd, float &gv, float &bv) {
        gv = bv = 0.f;
        if (hd.slot >= 0 && node >= 0 && node < hd.nodes) {
            gv = to_f32(ga[(hd.bos + node) * a.Hv + hd.h]);
            bv = to_f32(be[(hd.bos + node) * a.Hv + hd.h]);
        }
    };

    // Parts follow one another through the ring, head by head. When a head's products begin, as many parts as the ring
    // has slots are there or on their way; each slot is filled again once all warps are past it, the last one behind the
    // next head's keys and queries.
    int next_i = blockIdx.x;
    auto step_to = [&](const Head &from) -> Head {
        if (from.slot < 0) return from;
        next_i += gridDim.x;
        return find(next_i);
    };
    constexpr int AHEAD = (C::RING + C::NQ - 1) / C::NQ;  // heads to know of beside the one at hand
    static_assert(AHEAD <= 4, "heads ahead");
    Head hd[AHEAD + 1];
    hd[0] = find(next_i);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) hd[i + 1] = step_to(hd[i]);
#pragma unroll
    for (int i = 0; i < C::RING; ++i) {
        if (i == C::RING - 1) load_kq(hd[0]);
        load_state(state_of(hd[i / C::NQ]), i % C::NQ, i);
    }
    auto state_ahead = [&](int d) {  // of the head d ahead
        const float *s = state_of(hd[0]);
#pragma unroll
        for (int i = 1; i <= AHEAD; ++i)
            if (d == i) s = state_of(hd[i]);
        return s;
    };
    float gv, bv;
    load_gates(hd[0], gv, bv);
    int slot = 0;  // of the part at hand
    while (hd[0].slot >= 0) {
        const Head &cur = hd[0];
        const int T = cur.nodes, nb = (T + 15) / 16;
        copies_wait<1>();  // keys and queries, and the parts before the ring's last
        __syncthreads();
        // ---- paths, K K^T and Q K^T block by block of 16 x 16, |q|^2 --------------------------------
        if (warp == C::WARPS - 1) {
            const Paths p = tree_paths(a.parents + cur.bos, T, a.status);
            if (lane < TP) paths[lane] = p.of(0);
            if (TP > 32) paths[lane + 32] = p.of(1);
        }
        if (node >= 0) gs[node] = gv;
        for (int u = warp; u < nb * (nb + 2); u += C::WARPS) {
            const bool square = u >= nb * (nb + 1);  // Q Q^T of a block, for its diagonal
            const bool is_q = square || (u & 1);
            int i = 0, j = u >> 1;  // the block's rows and columns, j <= i
            while (j > i) j -= ++i;
            if (square) i = j = u - nb * (nb + 1);
            float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            const int ra = (is_q ? TP : 0) + 16 * i + (lane & 15), rb = (square ? TP : 0) + 16 * j + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t x[4], y[4];
                load_matrices(x, sb + C::SM_KQ + row_piece<DK>(ra, 2 * ks + (lane >> 4)));
                load_matrices(y, sb + C::SM_KQ + row_piece<DK>(rb, 2 * ks + ((lane >> 3) & 1)));
                mma_bf16_16816(acc[0], x, y[0], y[1]);
                mma_bf16_16816(acc[1], x, y[2], y[3]);
            }
            if (square) {
                if (c == g >> 1) {  // this lane's columns 2 c, 2 c + 1 hold the diagonal's of rows g and g + 8
                    qq[16 * i + g] = acc[0][g & 1];
                    qq[16 * i + 8 + g] = acc[1][2 + (g & 1)];
                }
                continue;
            }
            uint8_t *to = sm + (is_q ? C::SM_W : C::SM_A) + coef_block(i, j);
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int half = 0; half < 2; ++half)
                    *reinterpret_cast<float2 *>(to + coef_piece(g + 8 * half, 2 * n + (c >> 1)) + 8 * (c & 1)) =
                        make_float2(acc[n][2 * half], acc[n][2 * half + 1]);
        }
        __syncthreads();
        // ---- per node: norms, gates -------------------------------------------------------------
        if (node >= 0) {
            float hi = 0.f, lo = 0.f, kk = 0.f;
            if (node < T) {
                for (uint64_t m = paths[node]; m; m &= m - 1) add_exact(hi, lo, gs[__ffsll((long long)m) - 1]);
                kk = reinterpret_cast<const float *>(sm + C::SM_A + coef_block(node >> 4, node >> 4) +
                                                     coef_piece(node & 15, (node & 15) >> 2))[node & 3];
            }
            Scalars s;
            const float eg = expf(hi + lo);
            s.beta = sigmoidf_(bv);
            s.rk = 1.f / sqrtf(kk + kNormEps);
            s.rq = 1.f / sqrtf(qq[node] + kNormEps);
            s.x = s.beta * eg * s.rk;
            s.z = eg * s.rq;
            s.b2 = s.beta * s.rk * s.rk;
            s.g = hi;
            s.g_lo = lo;
            sc[node] = s;
        }
        __syncthreads();
        // ---- W, a row of it by four lanes: lane `sub` holds columns 16 j + 4 sub .. + 3 ---------------------
        for (int t = tid >> 2; t < 16 * nb; t += C::THREADS / 4) {
            const int sub = tid & 3;
            uint8_t *row = sm + C::SM_W + coef_block(t >> 4, 0);
            const uint64_t on = t < T ? paths[t] : 0;
            const Scalars st = sc[t];
            float w[C::NB][4];
#pragma unroll
            for (int j = 0; j < C::NB; ++j) {
                const float4 x = j <= t >> 4 ? *reinterpret_cast<const float4 *>(row + j * 1024 + coef_piece(t & 15, sub))
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                w[j][0] = st.rq * x.x; w[j][1] = st.rq * x.y; w[j][2] = st.rq * x.z; w[j][3] = st.rq * x.w;
            }
#pragma unroll
            for (int j = C::NB - 1; j >= 0; --j) {
                uint32_t left = (uint32_t)(on >> (16 * j)) & 0xffffu;
                // (the warp's eight rows step together, each along its own path: rows that part ways would run one by one)
                while (__any_sync(0xffffffffu, left != 0)) {
                    const int s = 31 - __clz(left | 1);  // of the block's nodes; w[s] is final: take it out of the columns before it
                    const int e = s & 3;
                    const float own = e == 0 ? w[j][0] : e == 1 ? w[j][1] : e == 2 ? w[j][2] : w[j][3];
                    const float ws = -__shfl_sync(0xffffffffu, own, (lane & ~3) | (s >> 2)) * sc[16 * j + s].b2;
                    if (left != 0) {
                        left &= ~(1u << s);
                        const uint8_t *kr = sm + C::SM_A + coef_block(j, 0) + coef_piece(s, sub);
                        const int before = s - 4 * sub;  // columns of this lane that stand before s, in s's own block
#pragma unroll
                        for (int i = 0; i < C::NB; ++i) {
                            if (i > j) continue;
                            const float4 x = *reinterpret_cast<const float4 *>(kr + i * 1024);
                            w[i][0] = fmaf(ws, i < j || before > 0 ? x.x : 0.f, w[i][0]);
                            w[i][1] = fmaf(ws, i < j || before > 1 ? x.y : 0.f, w[i][1]);
                            w[i][2] = fmaf(ws, i < j || before > 2 ? x.z : 0.f, w[i][2]);
                            w[i][3] = fmaf(ws, i < j || before > 3 ? x.w : 0.f, w[i][3]);
                        }
                    }
                }
            }
            // as two bf16 terms, in place: a row's 64 bytes of a block become 16 upper and 16 lower terms
            __syncwarp();
#pragma unroll
            for (int j = 0; j < C::NB; ++j) {
                if (j > t >> 4) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = 16 * j + 4 * sub + e;
                    const Scalars ss = sc[s];
                    const float d = __expf((st.g - ss.g) + (st.g_lo - ss.g_lo)) * ss.rk;
                    w[j][e] = (on >> s) & 1 ? w[j][e] * d : 0.f;
                }
                uint2 up, low;
                up.x = split2(w[j][0], w[j][1]);
                up.y = split2(w[j][2], w[j][3]);
                low.x = tc::bf2_bits(__floats2bfloat162_rn(w[j][0], w[j][1]));
                low.y = tc::bf2_bits(__floats2bfloat162_rn(w[j][2], w[j][3]));
                *reinterpret_cast<uint2 *>(row + j * 1024 + coef_piece(t & 15, sub >> 1) + 8 * (sub & 1)) = up;
                *reinterpret_cast<uint2 *>(row + j * 1024 + coef_piece(t & 15, 2 + (sub >> 1)) + 8 * (sub & 1)) = low;
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
#pragma unroll 1
        for (int part = 0; part < C::NQ; ++part) {
            if (part >= C::RING - 1) copies_wait<C::RING - 2>();
            if (part >= 1) {
                __syncthreads();
                const int p = part + C::RING - 1;
                load_state(state_ahead(p / C::NQ), p % C::NQ, slot == 0 ? C::RING - 1 : slot - 1);
            }
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
            if (++slot == C::RING) slot = 0;
        }
        __syncthreads();  // keys, queries and the last part's slot may be filled again
        load_kq(hd[1]);
        load_state(state_of(hd[(C::NQ + C::RING - 1) / C::NQ]), (C::NQ + C::RING - 1) % C::NQ, slot == 0 ? C::RING - 1 : slot - 1);
        load_gates(hd[1], gv, bv);
        // ---- R, and O ----------------------------------------------------------------------------------
        uint64_t bad0 = 0, bad1 = 0;  // nodes whose R is not finite in this lane's rows
        float sure = 0.f;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * n + 2 * c + e;
                const Scalars st = sc[t];
                const float v0 = __uint_as_float(vv[n][e] << 16), v1 = __uint_as_float(vv[n][e] & 0xffff0000u);
                xk[n][e] = t < T ? st.beta * v0 - st.x * xk[n][e] : 0.f;
                xk[n][2 + e] = t < T ? st.beta * v1 - st.x * xk[n][2 + e] : 0.f;
                xq[n][e] *= st.z;
                xq[n][2 + e] *= st.z;
                sure = fmaf(xk[n][e], 0.f, sure);  // 0, or NaN
                sure = fmaf(xk[n][2 + e], 0.f, sure);
            }
        if (__any_sync(0xffffffffu, sure != 0.f)) {
            uint32_t m[2][2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(fabsf(xk[n][e]) < INFINITY)) {
                        xk[n][e] = 0.f;
                        m[e >> 1][n >> 2] |= 1u << ((8 * n + 2 * c + (e & 1)) & 31);
                    }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e >> 1][e & 1] |= __shfl_xor_sync(0xffffffffu, m[e >> 1][e & 1], o);
            bad0 = (uint64_t)m[0][1] << 32 | m[0][0];
            bad1 = (uint64_t)m[1][1] << 32 | m[1][0];
        }
#pragma unroll
        for (int j = 0; j < C::NB; ++j) {
            if (j >= nb) continue;
            uint32_t uh[4], ul[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = xk[2 * j + (e >> 1)][2 * (e & 1)], y = xk[2 * j + (e >> 1)][2 * (e & 1) + 1];
                uh[e] = split2(x, y);
                ul[e] = tc::bf2_bits(__floats2bfloat162_rn(x, y));
            }
            const int tr = ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
            for (int i = j; i < C::NB; ++i) {
                if (i >= nb) continue;
                uint32_t y[4];
                load_matrices(y, sb + C::SM_W + coef_block(i, j) + coef_piece(tr, ch));
                mma_bf16_16816(xq[2 * i], uh, y[0], y[1]);
                mma_bf16_16816(xq[2 * i + 1], uh, y[2], y[3]);
                mma_bf16_16816(xq[2 * i], ul, y[0], y[1]);
                mma_bf16_16816(xq[2 * i + 1], ul, y[2], y[3]);
                load_matrices(y, sb + C::SM_W + coef_block(i, j) + coef_piece(tr, 2 + ch));
                mma_bf16_16816(xq[2 * i], uh, y[0], y[1]);
                mma_bf16_16816(xq[2 * i + 1], uh, y[2], y[3]);
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
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) hd[i] = hd[i + 1];
        hd[AHEAD] = step_to(hd[AHEAD - 1]);
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
