// tree_scan.cu -- the gated delta rule over a tree of drafted tokens.
//
// Along the path of node t, with G_t the sum of g over it, S_t the state after it and S_0 the sequence's state,
//     S_t = e^{G_t} S_0 + sum_{s on path(t)} e^{G_t - G_s} u_s kh_s^T,
//     u_t = beta_t (v_t - e^{G_t} S_0 kh_t - sum_{s on path(t), s != t} e^{G_t - G_s} (kh_s . kh_t) u_s),
//     o_t = e^{G_t} S_0 qh_t + sum_{s on path(t)} e^{G_t - G_s} (kh_s . qh_t) u_s,
// so that no node's state is ever formed: S_0 is read once, and each node costs two products with it and two short
// sums over its path. u_t is the correction that the recurrence writes at t, the same for all that lie below t.
//
// The kernel here serves fp32 inputs, in fp32 throughout, on the CUDA cores; bf16 inputs run on the tensor cores
// (tree_scan_umma.cu, tree_scan_tc.cu, which says how the sum over u becomes one over R_s = beta_s (v_s - e^{G_s} S_0 kh_s)).
// A CTA takes a (sequence, value head): all products of nodes with nodes side by side, those of the state's rows with the
// nodes' vectors with a row in a thread's registers and the nodes dealt to groups of threads, W by four lanes a row,
// and the sums over paths by the threads of the rows again. It is bound by the length of that chain and by shared-memory
// reads; correct and steady, but no performance path.
#include "tree_mma.cuh"

namespace gdn {
namespace {

constexpr int kScanThreads = 256;

template <int DK, int DV>
struct ScanSmem {
    float kh[kTreeMax][DK + 4], qh[kTreeMax][DK + 4];  // unit vectors
    float kk[kTreeMax * CoefPlain::kRow], w[kTreeMax * CoefPlain::kRow];
    float r[kTreeMax][DV], xq[kTreeMax][DV];
    Scalars<kTreeMax> sc;
    uint64_t path[kTreeMax];
    float g[kTreeMax];
};

template <int DK, int DV>
__global__ void __launch_bounds__(kScanThreads) tree_scan_kernel(const TreeArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ScanSmem<DK, DV> &sm = *reinterpret_cast<ScanSmem<DK, DV> *>(smem_raw);
    const int n = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int WARPS = kScanThreads / 32;
    next_may_begin();
    before_reading();
    long bos;
    int nodes;
    if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &bos, &nodes, a.status)) return;
    const long slot = state_slot(a, n);
    const float *q = (const float *)a.q, *k = (const float *)a.k, *v = (const float *)a.v;
    float *out = (float *)a.out;
    if (slot < 0) {
        for (int e = tid; e < nodes * DV; e += kScanThreads) out[((bos + e / DV) * a.Hv + h) * DV + e % DV] = 0.f;
        return;
    }
    // the rows first: they come from memory. Thread: a row, and every NG-th node.
    constexpr int NG = kScanThreads / DV;
    const int mine = tid % DV, group = tid / DV;
    float row[DK];
    const float *src = a.state_in + ((slot * a.Hv + h) * DV + mine) * DK;
#pragma unroll
    for (int c = 0; c < DK; c += 4) {
        const float4 x = load4(src + c);
        row[c] = x.x; row[c + 1] = x.y; row[c + 2] = x.z; row[c + 3] = x.w;
    }
    if (warp == WARPS - 1) {
        const Paths p = tree_paths(a.parents + bos, nodes, a.status);
        sm.path[lane] = p.of(0);
        sm.path[lane + 32] = p.of(1);
    }
    if (tid < nodes) {
        const float g = ((const float *)a.g)[(bos + tid) * a.Hv + h];
        sm.g[tid] = g < kNoGate ? kNoGate : g;
    }
    for (int t = warp; t < nodes; t += WARPS) {
        const float *kr = k + ((bos + t) * a.Hk + hk) * DK, *qr = q + ((bos + t) * a.Hk + hk) * DK;
        float x[DK / 32], y[DK / 32], sk = 0.f, sq = 0.f;
#pragma unroll
        for (int e = 0; e < DK / 32; ++e) {
            x[e] = kr[lane + 32 * e];
            y[e] = qr[lane + 32 * e];
            sk = fmaf(x[e], x[e], sk);
            sq = fmaf(y[e], y[e], sq);
        }
        const float rk = 1.f / sqrtf(warp_sum(sk) + kNormEps), rq = 1.f / sqrtf(warp_sum(sq) + kNormEps);
#pragma unroll
        for (int e = 0; e < DK / 32; ++e) {
            sm.kh[t][lane + 32 * e] = x[e] * rk;
            sm.qh[t][lane + 32 * e] = y[e] * rq;
        }
    }
    __syncthreads();
    if (tid < kTreeMax) {
        float hi = 0.f, lo = 0.f;
        if (tid < nodes)
            for (uint64_t m = sm.path[tid]; m; m &= m - 1) add_exact(hi, lo, sm.g[__ffsll((long long)m) - 1]);
        const float eg = expf(hi + lo), beta = tid < nodes ? sigmoidf_(((const float *)a.b)[(bos + tid) * a.Hv + h]) : 0.f;
        sm.sc.beta[tid] = sm.sc.b2[tid] = beta;
        sm.sc.x[tid] = beta * eg;
        sm.sc.z[tid] = eg;
        sm.sc.rq[tid] = 1.f;
        sm.sc.g[tid] = hi;
        sm.sc.g_lo[tid] = sm.sc.gk[tid] = lo;
    }
    const CoefPlain kk{sm.kk}, w{sm.w};
    const int upto = (nodes + 15) & ~15;
    for (int e = tid; e < nodes * upto; e += kScanThreads) {  // (what is past a node's own block is not looked at)
        const int t = e / upto, s = e % upto;
        if (s >= nodes || s > t) {
            *kk.raw(t, s) = *w.raw(t, s) = 0.f;
            continue;
        }
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int c = 0; c < DK; c += 4) {
            const float4 ks = load4(&sm.kh[s][c]), kt = load4(&sm.kh[t][c]), qt = load4(&sm.qh[t][c]);
            x[0] = fmaf(ks.x, kt.x, x[0]); x[1] = fmaf(ks.y, kt.y, x[1]); x[2] = fmaf(ks.z, kt.z, x[2]); x[3] = fmaf(ks.w, kt.w, x[3]);
            y[0] = fmaf(ks.x, qt.x, y[0]); y[1] = fmaf(ks.y, qt.y, y[1]); y[2] = fmaf(ks.z, qt.z, y[2]); y[3] = fmaf(ks.w, qt.w, y[3]);
        }
        *kk.raw(t, s) = s < t ? (x[0] + x[1]) + (x[2] + x[3]) : 0.f;  // (form_w wants zeros from the diagonal on)
        *w.raw(t, s) = (y[0] + y[1]) + (y[2] + y[3]);
    }
    __syncthreads();
    for (int t = group; t < nodes; t += NG) {
        float xk[4] = {0.f, 0.f, 0.f, 0.f}, xq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < DK; c += 4) {
            const float4 kt = load4(&sm.kh[t][c]), qt = load4(&sm.qh[t][c]);
            xk[0] = fmaf(row[c], kt.x, xk[0]); xk[1] = fmaf(row[c + 1], kt.y, xk[1]);
            xk[2] = fmaf(row[c + 2], kt.z, xk[2]); xk[3] = fmaf(row[c + 3], kt.w, xk[3]);
            xq[0] = fmaf(row[c], qt.x, xq[0]); xq[1] = fmaf(row[c + 1], qt.y, xq[1]);
            xq[2] = fmaf(row[c + 2], qt.z, xq[2]); xq[3] = fmaf(row[c + 3], qt.w, xq[3]);
        }
        const float vt = v[((bos + t) * a.Hv + h) * DV + mine];
        sm.r[t][mine] = sm.sc.beta[t] * vt - sm.sc.x[t] * ((xk[0] + xk[1]) + (xk[2] + xk[3]));
        sm.xq[t][mine] = sm.sc.z[t] * ((xq[0] + xq[1]) + (xq[2] + xq[3]));
    }
    form_w<kTreeMax, kScanThreads>(nodes, sm.path, sm.sc, kk, w);
    __syncthreads();
    for (int t = group; t < nodes; t += NG) {
        float o = sm.xq[t][mine];
        for (uint64_t m = sm.path[t]; m; m &= m - 1) {  // (only these: what is not finite stays on its paths)
            const int s = __ffsll((long long)m) - 1;
            o = fmaf(*w.raw(t, s), sm.r[s][mine], o);
        }
        out[((bos + t) * a.Hv + h) * DV + mine] = o;
    }
}

template <int DK, int DV>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    auto kernel = tree_scan_kernel<DK, DV>;
    constexpr int bytes = sizeof(ScanSmem<DK, DV>);
    static_assert(bytes <= 232448, "over the 227 KiB opt-in limit");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3((unsigned)(a.B * a.Hv)), kScanThreads, bytes, s, a);
}

template <int DK>
cudaError_t launch_dv(const TreeArgs &a, cudaStream_t s) {
    switch (a.dv) {
        case 32: return launch_t<DK, 32>(a, s);
        case 64: return launch_t<DK, 64>(a, s);
        case 128: return launch_t<DK, 128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree_scan(const TreeArgs &a, cudaStream_t s) {
    if (a.dtype != GDN_F32) return a.dk == 128 && a.dv == 128 ? launch_tree_scan_umma(a, s) : launch_tree_scan_tc(a, s);
    switch (a.dk) {
        case 32: return launch_dv<32>(a, s);
        case 64: return launch_dv<64>(a, s);
        case 128: return launch_dv<128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
