// tree_scan_umma.cu -- the gated delta rule over trees for bf16 inputs and heads of 128 x 128, on tcgen05.
//
// The products of tree_scan_tc.cu (whose head says what X, R and W are), with all 128 rows of the state as M:
//     X = S_0 [K; Q]^T     A: S_0 split into two bf16 terms, in shared memory; B: keys and queries as they come by TMA
//     D = R W^T            A: R as two bf16 terms, in TMEM; B: W as two terms (upper times upper, lower times upper, upper
//                          times lower)
// and o_t = e^{G_t} rq_t X_q,t + D_t. A thread stands for a row of the state and half of the nodes: it takes X_k out of
// TMEM, forms R and puts it back, and takes X_q and D out at the end.
//
// Why this beside m16n8k16: there each warp feeds 16 rows with fragments of keys, queries and W, and its accumulators in
// registers leave room for 16 warps to an SM. Here the products are 36 instructions of one warp. m16n8k16 took 120 us for 64
// sequences of 61 nodes and 32 heads when this took 84 (32 nodes 61 and 53, 16 nodes 48 and 39, 8 nodes 46 and 36). This takes
// 62 now (from a graph), and with an L2 that holds other data 63, 44, 35 and 34; chains of 61 nodes 106.
//
// What bounds it: S_0's bytes are 20 us of those, and with few nodes all but 8 us of the time go with the bytes. With many
// it is the dependent steps of a head: about 14,500 cycles for 61 nodes, of which W's last rows 4,500, the paths and the
// products of nodes beside them 2,700, R 1,900, rows out 1,900; those of two CTAs run side by side on an SM. A warp issues
// an instruction every 9 cycles there, so that what counts is their number on the way of the slowest warp.
//
// A head's state comes to registers as two halves of 64 columns (the next head's first one early), and goes to shared
// memory as terms, one half at a time, so that two CTAs fit an SM, and three with up to 16 nodes (two: 43 us instead of 39;
// with up to 32, three leave 80 registers: 73 us instead of 53). Its loads are asked for where no other load is waited for
// soon: the paths' parents, asked for long before, were waited for together with a half of the state (68 us instead of 64).
// (All of a state asked for ahead into L2 by bulk prefetches: 41 us instead of 34 with 16 nodes.)
#include "tree_mma.cuh"

namespace gdn {
namespace {

using namespace tc;

template <int TP>
struct Cfg {
    static constexpr int THREADS = 256, NB = TP / 16, HALF = TP / 2;  // blocks of nodes; a thread's nodes
    static constexpr int BLOCKS = NB * (NB + 1) / 2;
    static constexpr int NODE_WARP = TP == 64 ? 4 : 7;                // (without products of nodes to take out of TMEM)
    static constexpr int CHUNK = HALF < 16 ? HALF : 16;               // nodes that a thread has in registers
    // TMEM columns: X of keys and of queries; [K; Q] [K; Q]^T, then R's terms (two nodes a column) and D
    static constexpr uint32_t TM_X = 0, TM_G = 2 * TP, TM_R = 2 * TP, TM_D = 3 * TP, COLS = 4 * TP;
    static constexpr uint32_t KQ_BLOCK = 2 * TP * 128, TERM = 128 * 128;
    // byte offsets
    static constexpr uint32_t SM_KQ = 0;                             // [2 blocks of 64 columns][K, Q: 2 TP rows] bf16
    static constexpr uint32_t SM_X = SM_KQ + 2 * KQ_BLOCK;            // half of a state: upper terms, lower terms
    static constexpr uint32_t SM_W = SM_X + 2 * TERM;                 // W: upper terms, lower terms (CoefRows)
    static constexpr uint32_t SM_A = SM_W + 2 * TP * 128;             // K K^T (CoefBlocks)
    static constexpr uint32_t SM_V = SM_A + BLOCKS * 1024;            // [TP][128] bf16
    static constexpr uint32_t SM_SC = SM_V + TP * 256;                // per node: Scalars
    static constexpr uint32_t SM_PATH = SM_SC + TP * 32;
    static constexpr uint32_t SM_BAD = SM_PATH + TP * 8;              // [2][128] nodes whose R is not finite, by row
    static constexpr uint32_t SM_R = SM_BAD + 1024;                  // |q|^2
    static constexpr uint32_t SM_BAR = SM_R + TP * 4;                 // keys and queries; values; [K; Q] [K; Q]^T; X; D; the end
    static constexpr uint32_t SM_TMEM = SM_BAR + 6 * 8;
    static constexpr uint32_t SM_BYTES = SM_TMEM + 16;
    static constexpr int PER_SM = TP >= 32 ? 2 : 3;
    static_assert(PER_SM * (SM_BYTES + 1024) <= 233472 && PER_SM * COLS <= 512, "CTAs to an SM");
};

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, float (&x)[N]) {
    uint32_t r[N];
    if constexpr (N == 16) tmem_ld16_nw(at, r);
    else tmem_ld8_nw(at, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
}

template <int TP>
__global__ void __launch_bounds__(Cfg<TP>::THREADS, Cfg<TP>::PER_SM)
tree_scan_umma_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mv, const TreeArgs a, long long budget) {
    using C = Cfg<TP>;
    // (on a 1 KiB boundary, as all of it is asked for at launch: checked, as room to align it may cost a CTA)
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Scalars<TP> &sc = *reinterpret_cast<Scalars<TP> *>(sm + C::SM_SC);
    uint64_t *paths = reinterpret_cast<uint64_t *>(sm + C::SM_PATH);
    uint32_t *bad = reinterpret_cast<uint32_t *>(sm + C::SM_BAD);
    float *qq = reinterpret_cast<float *>(sm + C::SM_R);
    uint64_t *bar_in = reinterpret_cast<uint64_t *>(sm + C::SM_BAR), *bar_g = bar_in + 1, *bar_x = bar_in + 2, *bar_d = bar_in + 3,
             *bar_v = bar_in + 4, *bar_end = bar_in + 5;
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(sm + C::SM_TMEM);
    __nv_bfloat16 *out = (__nv_bfloat16 *)a.out;
    next_may_begin();
    if (tid == 0) {
        prefetch_tmap(&mk);
        prefetch_tmap(&mq);
        prefetch_tmap(&mv);
        for (int i = 0; i < 6; ++i) mbar_init(bar_in + i, 1);
        fence_mbar_init();
    }
    before_reading();  // (and before TMEM is asked for: a kernel that ends may still hold it)
    if (warp == 0) tmem_alloc(tmem_at, C::COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    if (sb & 1023u) {
        flag_error(a.status);
        if (warp == 0) tmem_dealloc(tmem, C::COLS);
        return;
    }
    bool ok = true;  // the same for a warp's lanes
    const uint32_t lead = elect_one();

    Heads<128, C::THREADS> heads(a);
    Nodes<TP, C::NODE_WARP, 6> nodes;
    const CoefBlocks kk{sm + C::SM_A};
    const CoefRows<TP> wt{sm + C::SM_W};
    uint32_t loads = 0;  // begun: an odd number (bit 0) and any (1) of keys and queries, (2) and (3) of values
    auto load_in = [&](const Head &hd) {
        if (hd.slot < 0) return;
        loads = (loads ^ 1u) | 2u;
        if (tid != 0) return;
        const int hk = hd.h / (a.Hv / a.Hk);
        mbar_expect_tx(bar_in, 2 * C::KQ_BLOCK);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            tma_load_3d(sm + C::SM_KQ + b * C::KQ_BLOCK, &mk, 64 * b, hk, (int)hd.bos, bar_in);
            tma_load_3d(sm + C::SM_KQ + b * C::KQ_BLOCK + TP * 128, &mq, 64 * b, hk, (int)hd.bos, bar_in);
        }
    };
    auto load_v = [&](const Head &hd) {
        if (hd.slot < 0) return;
        loads = (loads ^ 4u) | 8u;
        if (tid != 0) return;
        mbar_expect_tx(bar_v, TP * 256);
        tma_load_3d(sm + C::SM_V, &mv, 0, hd.h, (int)hd.bos, bar_v);
    };
    // half of a state, 64 columns: this thread's 16 bytes (columns 4 ch ..) of 8 rows
    const int sr = tid >> 4, ch = tid & 15;
    float4 half[8];
    auto load_half = [&](const Head &hd, int h) {
        if (hd.slot < 0) return;
        const float *src = a.state_in + (hd.slot * a.Hv + hd.h) * 16384 + sr * 128 + h * 64 + ch * 4;
#pragma unroll
        for (int i = 0; i < 8; ++i) half[i] = __ldcs(reinterpret_cast<const float4 *>(src + i * 16 * 128));
    };
    auto split_half = [&] {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = sr + 16 * i;
            float4 x = half[i];
            uint2 up, low;
            up.x = split2(x.x, x.y);
            up.y = split2(x.z, x.w);
            low.x = bf2_bits(__floats2bfloat162_rn(x.x, x.y));
            low.y = bf2_bits(__floats2bfloat162_rn(x.z, x.w));
            uint8_t *at = sm + C::SM_X + swz(r, ch >> 1) + 8 * (ch & 1);
            *reinterpret_cast<uint2 *>(at) = up;
            *reinterpret_cast<uint2 *>(at + C::TERM) = low;
        }
        fence_async_smem();
    };
    // [K; Q] [K; Q]^T: rows of A past 2 TP are whatever follows in shared memory, and their results are not looked at
    auto product_g = [&] {  // by warp 0
        constexpr uint32_t ID = idesc_bf16(128, 2 * TP, 0, 0);
        const uint64_t x = desc_sw128(sb + C::SM_KQ, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint64_t at = x + (uint64_t)(((ks >> 2) * C::KQ_BLOCK + (ks & 3) * 32) >> 4);
            mma_f16_ss_by(lead, tmem + C::TM_G, at, at, ID, ks > 0);
        }
        mma_commit_by(lead, bar_g);
    };
    auto product_x = [&](int h) {  // by warp 0
        constexpr uint32_t ID = idesc_bf16(128, 2 * TP, 0, 0);
        const uint64_t x = desc_sw128(sb + C::SM_X, 16, 1024), y = desc_sw128(sb + C::SM_KQ + h * C::KQ_BLOCK, 16, 1024);
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_f16_ss_by(lead, tmem + C::TM_X, x + (uint64_t)((term * C::TERM + ks * 32) >> 4), y + (uint64_t)(ks * 2), ID,
                         h > 0 || term > 0 || ks > 0);
        mma_commit_by(lead, bar_x);
    };
    auto product_d = [&] {  // by warp 0
        constexpr uint32_t ID = idesc_bf16(128, TP, 0, 0);
        const uint64_t y = desc_sw128(sb + C::SM_W, 16, 1024);
#pragma unroll
        for (int term = 0; term < 3; ++term)  // R upper W upper, R lower W upper, R upper W lower
#pragma unroll
            for (int ks = 0; ks < TP / 16; ++ks)
                mma_f16_ts_by(lead, tmem + C::TM_D, tmem + C::TM_R + (term == 1 ? TP / 2 : 0) + 8 * ks,
                            y + (uint64_t)(((term == 2 ? TP * 128 : 0) + ks * 32) >> 4), ID, term > 0 || ks > 0);
        mma_commit_by(lead, bar_d);
    };
    const int part = warp >> 2, row = 32 * (warp & 3) + lane, t_first = part * C::HALF;  // this thread's row and nodes
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16);

    Head cur = heads.find(a), next = heads.after(a, cur);
    load_in(cur);
    load_v(cur);
    load_half(cur, 0);
    nodes.load(a, cur);
    uint32_t phase_in = 0, phase_v = 0, phase_g = 0, phase_x = 0, phase_d = 0;
    while (cur.slot >= 0) {
        const int T = cur.nodes;
        // ---- the state's first half; then the nodes beside its products ---------------------------
        split_half();
        ok = warp_wait(bar_in, phase_in, budget) && ok;
        phase_in ^= 1;
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;  // (and all that the head before has left has been read)
        if (warp == 0) {
            tc_fence_after();
            product_g();
            product_x(0);
        }
        __syncwarp();
        nodes.sums(paths, sc, a.status);
        load_half(cur, 1);  // (not before: the sums would wait for it)
        ok = warp_wait(bar_g, phase_g, budget);
        phase_g ^= 1;
        tc_fence_after();
        if (32 * (warp & 3) < 2 * TP) {  // rows of K, then of Q: the products up to the row's own block
            const bool is_q = row >= TP;
            const int t = is_q ? row - TP : row;
            const int first = (32 * (warp & 3)) & (TP - 1), t_last = TP < 32 ? TP - 1 : first + 31;  // of the warp's rows
#pragma unroll
            for (int c0 = 0; c0 < C::HALF; c0 += C::CHUNK) {
                if (t_first + c0 > t_last) continue;
                float x[C::CHUNK];
                tmem_load(tl + C::TM_G + t_first + c0, x);
#pragma unroll
                for (int i = 0; i < C::CHUNK; i += 4) {
                    const int s = t_first + c0 + i;
                    const bool past = !is_q && s > t;  // (zeros there: form_w)
                    if ((s >> 4) <= (t >> 4))
                        *reinterpret_cast<float4 *>(is_q ? wt.raw(t, s) : kk.raw(t, s)) =
                            past ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
            }
        }
        if (part == 1 && 32 * (warp & 3) < 2 * TP) {  // |q|^2: the diagonal of Q Q^T
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int t = 32 * (warp & 3) - TP + 16 * c;  // of 16 nodes
                if (t < 0) continue;
                float x[16];
                tmem_load(tl + C::TM_G + TP + t, x);
#pragma unroll
                for (int bit = 8; bit > 0; bit >>= 1)
#pragma unroll
                    for (int i = 0; i < bit; ++i) x[i] = lane & bit ? x[i + bit] : x[i];
                if ((lane >> 4) == c) qq[t + (lane & 15)] = x[0];
            }
        }
        tc_fence_before();  // (R is going to be where the products were)
        if (__syncthreads_or(!ok)) break;
        nodes.finish(T, kk, qq, sc);
        // ---- its second half; W beside its products -------------------------------------------------
        ok = warp_wait(bar_x, phase_x, budget);
        phase_x ^= 1;
        if (ok) split_half();
        if (__syncthreads_or(!ok)) break;
        if (warp == 0) {
            tc_fence_after();
            product_x(1);
        }
        __syncwarp();
        form_w<TP, C::THREADS>(T, paths, sc, kk, wt);
        fence_async_smem();
        load_half(next, 0);
        // ---- R ------------------------------------------------------------------------------------------
        ok = warp_wait(bar_x, phase_x, budget);
        phase_x ^= 1;
        if (ok) load_in(next);  // (none but the products read keys and queries)
        ok = warp_wait(bar_v, phase_v, budget) && ok;
        phase_v ^= 1;
        tc_fence_after();
        uint32_t not_finite = 0;  // of this thread's nodes
#pragma unroll
        for (int c0 = 0; c0 < C::HALF; c0 += C::CHUNK) {
            float x[C::CHUNK], sure = 0.f;
            tmem_load(tl + C::TM_X + t_first + c0, x);
#pragma unroll
            for (int i = 0; i < C::CHUNK; i += 4) {
                const int t = t_first + c0 + i;
                const float4 b4 = load4(sc.beta + t), x4 = load4(sc.x + t);
                const float be[4] = {b4.x, b4.y, b4.z, b4.w}, fx[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v =
                        __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(sm + C::SM_V + (t + e) * 256 + row * 2) << 16);
                    x[i + e] = t + e < T ? be[e] * v - fx[e] * x[i + e] : 0.f;
                    sure = fmaf(x[i + e], 0.f, sure);  // 0, or NaN
                }
            }
            if (sure != 0.f) {
#pragma unroll
                for (int i = 0; i < C::CHUNK; ++i)
                    if (!(fabsf(x[i]) < INFINITY)) {
                        x[i] = 0.f;
                        not_finite |= 1u << (c0 + i);
                    }
            }
            uint32_t up[C::CHUNK / 2], low[C::CHUNK / 2];
#pragma unroll
            for (int i = 0; i < C::CHUNK; i += 2) {
                up[i / 2] = split2(x[i], x[i + 1]);
                low[i / 2] = bf2_bits(__floats2bfloat162_rn(x[i], x[i + 1]));
            }
            const uint32_t to = tl + C::TM_R + (t_first + c0) / 2;
            if constexpr (C::CHUNK == 16) {
                tmem_st8(to, up);
                tmem_st8(to + TP / 2, low);
            } else {
                tmem_st4(to, up);
                tmem_st4(to + TP / 2, low);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        uint64_t off = 0;  // nodes whose R is not finite in this thread's row
        if (__syncthreads_or(!ok || not_finite != 0)) {
            bad[part * 128 + row] = not_finite;
            if (__syncthreads_or(!ok)) break;
            off = (uint64_t)bad[128 + row] << C::HALF | bad[row];
        }
        if (warp == 0) {
            tc_fence_after();
            product_d();
        }
        __syncwarp();
        load_v(next);
        nodes.load(a, next);
        // ---- rows out ------------------------------------------------------------------------------------
        ok = warp_wait(bar_d, phase_d, budget);
        phase_d ^= 1;
        tc_fence_after();
        if (ok) {
            const long token = (long)a.Hv * 128;
            __nv_bfloat16 *to = out + ((cur.bos + t_first) * a.Hv + cur.h) * 128 + row;
#pragma unroll
            for (int c0 = 0; c0 < C::HALF; c0 += C::CHUNK) {
                float x[C::CHUNK], d[C::CHUNK];
                tmem_load(tl + C::TM_X + TP + t_first + c0, x);
                tmem_load(tl + C::TM_D + t_first + c0, d);
                if (rarely(off != 0)) {
#pragma unroll
                    for (int i = 0; i < C::CHUNK; ++i)
                        if (off & paths[t_first + c0 + i]) d[i] = __int_as_float(0x7fffffff);
                }
#pragma unroll
                for (int i = 0; i < C::CHUNK; i += 4) {
                    const float4 z4 = load4(sc.z + t_first + c0 + i);
                    const float z[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e, to += token)
                        if (c0 + i + e < T - t_first) *to = __float2bfloat16_rn(fmaf(z[e], x[i + e], d[i + e]));
                }
            }
        }
        tc_fence_before();
        cur = next;
        next = heads.after(a, cur);
    }
    const bool failed = __syncthreads_or(!ok);
    if (failed) {
        if (tid == 0) {
            flag_error(a.status);
            // copies and products in flight end before the CTA leaves
            if (loads & 2u) mbar_wait(bar_in, ~loads & 1u, kDrainBudget);
            if (loads & 8u) mbar_wait(bar_v, ~(loads >> 2) & 1u, kDrainBudget);
        }
        if (warp == 0) {
            mma_commit_by(lead, bar_end);
            mbar_wait(bar_end, 0, kDrainBudget);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, C::COLS);
}

template <int TP>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    using C = Cfg<TP>;
    CUtensorMap mk, mq, mv;
    if (!scan_map(&mk, a.k, false, 128, a.Hk, a.Ttot, 64, 1, TP) || !scan_map(&mq, a.q, false, 128, a.Hk, a.Ttot, 64, 1, TP) ||
        !scan_map(&mv, a.v, false, 128, a.Hv, a.Ttot, 128, 1, TP))
        return cudaErrorInvalidValue;
    auto kernel = tree_scan_umma_kernel<TP>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SM_BYTES);
    if (e != cudaSuccess) return e;
    const long heads = (long)a.B * a.Hv, most = 152L * C::PER_SM;
    return launch_early(kernel, dim3((unsigned)(heads < most ? heads : most)), C::THREADS, C::SM_BYTES, s, mk, mq, mv, a,
                        wait_budget());
}

}  // namespace

cudaError_t launch_tree_scan_umma(const TreeArgs &a, cudaStream_t s) {
    // The most nodes that a sequence can have: of packed ones that is not known here, but their total is. 64 sequences of 8, 16
    // and 32 nodes each take 32, 33 and 41 us; packed, of up to as many, 52, 53 and 55, in the instance for 64. (That for 16 has 80
    // registers for three CTAs to an SM, and spills 24 bytes a thread.)
    const long most = a.cu ? a.Ttot : a.T;
    return most <= 16 ? launch_t<16>(a, s) : most <= 32 ? launch_t<32>(a, s) : launch_t<64>(a, s);
}

}  // namespace gdn
