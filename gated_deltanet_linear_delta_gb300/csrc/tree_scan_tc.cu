// tree_scan_tc.cu -- the gated delta rule over trees for bf16 inputs, on the tensor cores (formulas: tree_scan.cu). This kernel
// serves head dimensions other than 128 x 128, for which tree_scan_umma.cu has the same products on tcgen05.
//
// Per (sequence, value head), with T nodes, on(t) the nodes on path(t) and S_0 (dv x dk fp32) read once:
//     X = S_0 [K; Q]^T             S_0 split into two bf16 terms (16 bits), k and q as they are (exact)
//     R_s = beta_s v_s - beta_s e^{G_s} rk_s X_k,s          what u_s is without the nodes above it
//     O_t = e^{G_t} rq_t X_q,t + sum_{s in on(t)} W_ts R_s
// W is P (I + A)^-1: a node's sum over the corrections u of its path, put in terms of R. Its rows are independent of
// one another, and the decays and norms stand outside of them: W_ts = e^{G_t-G_s} rk_s w_s, where from t upwards
//     w_s = rq_t (q_t.k_s) - sum_{s' in on(t), s' > s} w_s' beta_s' rk_s'^2 (k_s'.k_s),
// with the raw products of K K^T and Q K^T. So a row costs L^2 / 2 multiply-adds for a path of L nodes, by four lanes,
// once per head; and the dv rows of the state take no elimination of their own, just products. (With heads of 128 x 128,
// which ran here then, eliminating blocks of 16 nodes by shuffles in each warp for its own rows took 22% longer.)
//
// The products are m16n8k16 (mma.sync), 16 rows of the state to a warp: their accumulator, rows of the state by nodes, is
// in the layout of the next product's operand, so that R goes from X to O within registers.
//
// What bounds it: the dependent steps of a head and the instructions around the products (2930 a warp and head of 64 x 128 and 61
// nodes, one every 2 cycles and scheduler), with few nodes S_0's bytes beside them. 64 sequences, 32 heads, from a graph:
//     dk x dv             64 x 128    128 x 64    64 x 64    32 x 32
//     16 nodes, us              31          28         22         18    (bytes alone: 13, 13, 7, 2)
//     61 nodes, us              85          89         61         67    (22, 20, 12, 5)
// One session of 16 nodes and 64 x 128 takes 5.0 us. CTAs are persistent, two or three to an SM, and S_0 comes by TMA in parts of 32 columns through a ring, the next
// head's during the end of this one's work. Every wait has a limit, after which the call flags the status word.
//
// Values that are not finite stay on their paths: a product with a coefficient of 0 would spread them, so they are
// left out of the products, and the outputs that have them on their path become NaN.
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
    static constexpr uint32_t KQ_BYTES = TP * DK * 2, ROW = DK >= 64 ? 128 : 64;  // bytes of a row of a block of columns
    // byte offsets
    static constexpr uint32_t SM_KQ = 0;                                      // K, then Q [TP][DK] bf16
    static constexpr uint32_t SM_S = (2 * KQ_BYTES + 1023) & ~1023u;           // [RING][DV][32] fp32
    static constexpr uint32_t SM_A = SM_S + RING * SLOT;                       // K K^T, blocks of 16 x 16 fp32
    static constexpr uint32_t SM_W = SM_A + BLOCKS * 1024;                     // Q K^T, then W, fp32, then W as two terms
    static constexpr uint32_t SM_SC = SM_W + BLOCKS * 1024;                    // per node: Scalars
    static constexpr uint32_t SM_PATH = SM_SC + TP * 32;                       // [TP] paths
    static constexpr uint32_t SM_R = SM_PATH + TP * 8;                         // [TP] |q|^2
    static constexpr uint32_t SM_BAR = SM_R + TP * 4;                          // keys and queries; the slots
    static constexpr uint32_t SM_UNIT = SM_BAR + (1 + RING) * 8;               // the next block of products
    static constexpr uint32_t SM_BYTES = SM_UNIT + 8;
    static constexpr int FIT = 233472 / (SM_BYTES + 1024), PER_SM = FIT < 3 ? FIT : 3;  // CTAs to an SM
    static_assert(PER_SM >= 2, "two CTAs to an SM");
};

template <int DK, int DV, int TP>
__global__ void __launch_bounds__(Cfg<DK, DV, TP>::THREADS, Cfg<DK, DV, TP>::PER_SM)
tree_scan_tc_kernel(const __grid_constant__ CUtensorMap ms, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mq, const TreeArgs a, long long budget) {
    using C = Cfg<DK, DV, TP>;
    using namespace tc;
    // (on a 1 KiB boundary, as all of it is asked for at launch: checked, as room to align it would cost the third CTA)
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    Scalars<TP> &sc = *reinterpret_cast<Scalars<TP> *>(sm + C::SM_SC);
    uint64_t *paths = reinterpret_cast<uint64_t *>(sm + C::SM_PATH);
    float *qq = reinterpret_cast<float *>(sm + C::SM_R);
    uint64_t *bar_kq = reinterpret_cast<uint64_t *>(sm + C::SM_BAR), *bar_s = bar_kq + 1;
    int *unit = reinterpret_cast<int *>(sm + C::SM_UNIT);
    const __nv_bfloat16 *v = (const __nv_bfloat16 *)a.v;
    __nv_bfloat16 *out = (__nv_bfloat16 *)a.out;
    next_may_begin();
    if (tid == 0) {
        prefetch_tmap(&ms);
        prefetch_tmap(&mk);
        prefetch_tmap(&mq);
        for (int i = 0; i < 1 + C::RING; ++i) mbar_init(bar_kq + i, 1);
        fence_mbar_init();
        *unit = 0;
    }
    before_reading();
    __syncthreads();
    if (sb & 1023u) {
        flag_error(a.status);
        return;
    }

    Heads<DV, C::THREADS> heads(a);
    // Copies, by one thread. Keys and queries of TP tokens, whatever a sequence's number of nodes.
    uint32_t copies_kq = 0, copies_s = 0;  // begun
    auto load_kq = [&](const Head &hd) {
        if (hd.slot < 0) return;
        ++copies_kq;
        if (tid != 0) return;
        const int hk = hd.h / (a.Hv / a.Hk);
        mbar_expect_tx(bar_kq, 2 * C::KQ_BYTES);
#pragma unroll
        for (int b = 0; b < (DK >= 64 ? DK / 64 : 1); ++b) {
            tma_load_3d(sm + C::SM_KQ + b * (2 * TP * 128), &mk, 64 * b, hk, (int)hd.bos, bar_kq);
            tma_load_3d(sm + C::SM_KQ + b * (2 * TP * 128) + TP * C::ROW, &mq, 64 * b, hk, (int)hd.bos, bar_kq);
        }
    };
    auto load_state = [&](bool any, int state, int part, int slot) {
        if (!any) return;
        ++copies_s;
        if (tid != 0) return;
        mbar_expect_tx(bar_s + slot, C::SLOT);
        tma_load_3d(sm + C::SM_S + slot * C::SLOT, &ms, 32 * part, 0, state, bar_s + slot);
    };
    auto state_of = [&](const Head &hd) { return (int)(hd.slot * a.Hv + hd.h); };
    Nodes<TP, C::WARPS - 1, C::WARPS - 2> nodes;
    const CoefBlocks kk{sm + C::SM_A}, wt{sm + C::SM_W};

    // Parts follow one another through the ring, head by head. When a head's products begin, as many parts as the ring
    // has slots are there or on their way; each slot is filled again once all warps are past it, the last one behind the
    // next head's keys and queries.
    constexpr int AHEAD = (C::RING + C::NQ - 1) / C::NQ;  // heads to know of beside the one at hand
    static_assert(AHEAD <= 4, "heads ahead");
    Head hd[AHEAD + 1];
    hd[0] = heads.find(a);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) hd[i + 1] = heads.after(a, hd[i]);
    load_kq(hd[0]);
#pragma unroll
    for (int i = 0; i < C::RING; ++i) load_state(hd[i / C::NQ].slot >= 0, state_of(hd[i / C::NQ]), i % C::NQ, i);
    nodes.load(a, hd[0]);
    int slot = 0;                 // of the part at hand
    uint32_t phase_kq = 0, phase_s = 0;
    bool ok = true;
    while (hd[0].slot >= 0) {
        const Head &cur = hd[0];
        const int T = cur.nodes, nb = (T + 15) / 16;
        ok = wait_for(bar_kq, phase_kq, budget);
        phase_kq ^= 1;
        if (__syncthreads_or(!ok)) {  // (and what the nodes of the head before are known by has been read)
            ok = false;
            break;
        }
        // ---- the nodes: paths and gates, beside them the products; norms; W --------------------------------
        nodes.sums(paths, sc, a.status);
        node_products<DK, TP>(sb + C::SM_KQ, nb, unit, kk, wt, qq);
        __syncthreads();
        if (tid == 0) *unit = 0;
        nodes.finish(T, kk, qq, sc);
        __syncthreads();
        form_w<TP, C::THREADS>(T, paths, sc, kk, wt);
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
            if (part >= 1) {  // all warps are past the part before: its slot may be filled again
                if (__syncthreads_or(!ok)) break;
                const int p = part + C::RING - 1, d = p / C::NQ;
                bool any = cur.slot >= 0;
                int state = state_of(cur);
#pragma unroll
                for (int i = 1; i <= AHEAD; ++i)
                    if (d == i) {
                        any = hd[i].slot >= 0;
                        state = state_of(hd[i]);
                    }
                load_state(any, state, p % C::NQ, slot == 0 ? C::RING - 1 : slot - 1);
            }
            ok = wait_for(bar_s + slot, phase_s, budget);
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
                    al[e] = bf2_bits(__floats2bfloat162_rn(x.x, x.y));
                }
#pragma unroll
                for (int j = 0; j < C::NB; ++j)
                    if (j < nb) {
                        const int rr = 16 * j + ((lane >> 4) << 3) + (lane & 7), ch = 2 * ks + ((lane >> 3) & 1);
                        uint32_t y[4];
                        load_matrices(y, sb + C::SM_KQ + row_piece<DK, 2 * TP>(rr, ch));
                        mma_bf16_16816(xk[2 * j], ah, y[0], y[1]);
                        mma_bf16_16816(xk[2 * j + 1], ah, y[2], y[3]);
                        mma_bf16_16816(xk[2 * j], al, y[0], y[1]);
                        mma_bf16_16816(xk[2 * j + 1], al, y[2], y[3]);
                        load_matrices(y, sb + C::SM_KQ + row_piece<DK, 2 * TP>(TP + rr, ch));
                        mma_bf16_16816(xq[2 * j], ah, y[0], y[1]);
                        mma_bf16_16816(xq[2 * j + 1], ah, y[2], y[3]);
                        mma_bf16_16816(xq[2 * j], al, y[0], y[1]);
                        mma_bf16_16816(xq[2 * j + 1], al, y[2], y[3]);
                    }
            }
            if (++slot == C::RING) {
                slot = 0;
                phase_s ^= 1;
            }
        }
        if (__syncthreads_or(!ok)) {
            ok = false;
            break;
        }
        // keys, queries and the last part's slot may be filled again
        load_kq(hd[1]);
        {
            const Head &far = hd[(C::NQ + C::RING - 1) / C::NQ];
            load_state(far.slot >= 0, state_of(far), (C::NQ + C::RING - 1) % C::NQ, slot == 0 ? C::RING - 1 : slot - 1);
        }
        nodes.load(a, hd[1]);
        // ---- R, and O ----------------------------------------------------------------------------------
        uint64_t bad0 = 0, bad1 = 0;  // nodes whose R is not finite in this lane's rows
        float sure = 0.f;
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 8 * n + 2 * c + e;
                const float v0 = __uint_as_float(vv[n][e] << 16), v1 = __uint_as_float(vv[n][e] & 0xffff0000u);
                xk[n][e] = t < T ? sc.beta[t] * v0 - sc.x[t] * xk[n][e] : 0.f;
                xk[n][2 + e] = t < T ? sc.beta[t] * v1 - sc.x[t] * xk[n][2 + e] : 0.f;
                xq[n][e] *= sc.z[t];
                xq[n][2 + e] *= sc.z[t];
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
                ul[e] = bf2_bits(__floats2bfloat162_rn(x, y));
            }
            const int tr = ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
            for (int i = j; i < C::NB; ++i) {
                if (i >= nb) continue;
                uint32_t y[4];
                load_matrices(y, sb + C::SM_W + CoefBlocks::block(i, j) + CoefBlocks::piece(tr, ch));
                mma_bf16_16816(xq[2 * i], uh, y[0], y[1]);
                mma_bf16_16816(xq[2 * i + 1], uh, y[2], y[3]);
                mma_bf16_16816(xq[2 * i], ul, y[0], y[1]);
                mma_bf16_16816(xq[2 * i + 1], ul, y[2], y[3]);
                load_matrices(y, sb + C::SM_W + CoefBlocks::block(i, j) + CoefBlocks::piece(tr, 2 + ch));
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
                *reinterpret_cast<uint32_t *>(out + vat + (long)t * a.Hv * DV) = bf2_bits(__floats2bfloat162_rn(o0, o1));
            }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) hd[i] = hd[i + 1];
        hd[AHEAD] = heads.after(a, hd[AHEAD - 1]);
    }
    if (!ok) {
        flag_error(a.status);
        // copies in flight land before the CTA leaves
        if (tid == 0) {
            if (copies_kq > 0) mbar_wait(bar_kq, (copies_kq - 1) & 1, kDrainBudget);
            for (uint32_t i = copies_s > C::RING ? copies_s - C::RING : 0; i < copies_s; ++i)
                mbar_wait(bar_s + i % C::RING, (i / C::RING) & 1, kDrainBudget);
        }
        __syncthreads();
    }
}

template <int DK, int DV, int TP>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    using C = Cfg<DK, DV, TP>;
    CUtensorMap ms, mk, mq;
    const long states = (a.slots ? a.num_slots : (long)a.B) * a.Hv;
    // (without a state in the pool no sequence has one, and none is copied)
    if (!scan_map(&ms, states > 0 ? (const void *)a.state_in : a.k, true, DK, DV, states > 0 ? states : 1, 32, DV, 1) ||
        !scan_map(&mk, a.k, false, DK, a.Hk, a.Ttot, DK < 64 ? DK : 64, 1, TP) ||
        !scan_map(&mq, a.q, false, DK, a.Hk, a.Ttot, DK < 64 ? DK : 64, 1, TP))
        return cudaErrorInvalidValue;
    auto kernel = tree_scan_tc_kernel<DK, DV, TP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const long heads = (long)a.B * a.Hv, most = 152L * C::PER_SM;
    return launch_early(kernel, dim3((unsigned)(heads < most ? heads : most)), C::THREADS, C::SM_BYTES, s, ms, mk, mq, a,
                        wait_budget());
}

template <int DK, int DV>
cudaError_t launch_tp(const TreeArgs &a, cudaStream_t s) {
    // The most nodes that a sequence can have: of packed ones that is not known here, but their total is. Up to 16 take an
    // instance with a quarter of the accumulators: 64 sequences of 5 and of 16 nodes, heads of 64 x 128, take 29 and 31 us in it, and
    // 45 and 47 in that for 64 (128 x 64: 26, 27 and 43, 44; 64 x 64: 20, 22 and 29, 30; 32 x 32: 16, 18 and 25, 26). From 17 on it is
    // 55 (53, 36, 35) to 59 (56, 37, 37) at 32. With 128 rows of values the one for 64 spills 28 (dk = 64) and 56 bytes (32) a thread.
    const long most = a.cu ? a.Ttot : a.T;
    if (most <= 16) return launch_t<DK, DV, 16>(a, s);
    return launch_t<DK, DV, 64>(a, s);
}

}  // namespace

cudaError_t launch_tree_scan_tc(const TreeArgs &a, cudaStream_t s) {
    switch (a.dk * 1000 + a.dv) {
        case 32032: return launch_tp<32, 32>(a, s);
        case 32064: return launch_tp<32, 64>(a, s);
        case 32128: return launch_tp<32, 128>(a, s);
        case 64032: return launch_tp<64, 32>(a, s);
        case 64064: return launch_tp<64, 64>(a, s);
        case 64128: return launch_tp<64, 128>(a, s);
        case 128032: return launch_tp<128, 32>(a, s);
        case 128064: return launch_tp<128, 64>(a, s);
    }
    return cudaErrorInvalidValue;  // (128 x 128: tree_scan_umma.cu)
}

}  // namespace gdn
