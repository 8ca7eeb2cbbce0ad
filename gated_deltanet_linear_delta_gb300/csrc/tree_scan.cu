// tree_scan.cu -- the gated delta rule over a tree of drafted tokens.
//
// Along the path of node t, with G_t the sum of g over it, S_t the state after it and S_0 the sequence's state,
//     S_t = e^{G_t} S_0 + sum_{s on path(t)} e^{G_t - G_s} u_s kh_s^T,
//     u_t = beta_t (v_t - e^{G_t} S_0 kh_t - sum_{s on path(t), s != t} e^{G_t - G_s} (kh_s . kh_t) u_s),
//     o_t = e^{G_t} S_0 qh_t + sum_{s on path(t)} e^{G_t - G_s} (kh_s . qh_t) u_s,
// so that no node's state is ever formed: S_0 is read once, and each node costs two products with it and two short
// sums over its path. u_t is the correction that the recurrence writes at t, the same for all that lie below t.
#include "gdn_common.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

template <typename T, int DK, int DV>
struct ScanSmem {
    float kh[kTreeMax][DK], qh[kTreeMax][DK];
    float a[kTreeMax][kTreeMax], p[kTreeMax][kTreeMax];  // [t][s]: of u's and of o's sum
    float u[kTreeMax][DV];
    uint64_t path[kTreeMax];
    float g[kTreeMax], g_lo[kTreeMax], beta[kTreeMax];
};

// One (sequence, value head) a CTA, a row of the state a thread.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(128) tree_scan_kernel(const TreeArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    ScanSmem<T, DK, DV> &sm = *reinterpret_cast<ScanSmem<T, DK, DV> *>(smem_raw);
    const int n = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long bos;
    int nodes;
    if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &bos, &nodes, a.status)) return;
    const long slot = state_slot(a, n);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v, *g = (const T *)a.g, *b = (const T *)a.b;
    T *out = (T *)a.out;
    if (slot < 0) {
        for (int e = tid; e < nodes * DV; e += 128) out[((bos + e / DV) * a.Hv + h) * DV + e % DV] = from_f32<T>(0.f);
        return;
    }
    if (warp == 0) {
        const Paths p = tree_paths(a.parents + bos, nodes, a.status);
        sm.path[lane] = p.of(0);
        sm.path[lane + 32] = p.of(1);
    }
    for (int t = warp; t < nodes; t += 4) {
        const T *kr = k + ((bos + t) * a.Hk + hk) * DK, *qr = q + ((bos + t) * a.Hk + hk) * DK;
        float sk = 0.f, sq = 0.f;
        for (int c = lane; c < DK; c += 32) {
            const float x = to_f32(kr[c]), y = to_f32(qr[c]);
            sk += x * x;
            sq += y * y;
            sm.kh[t][c] = x;
            sm.qh[t][c] = y;
        }
        const float rk = 1.f / sqrtf(warp_sum(sk) + kNormEps), rq = 1.f / sqrtf(warp_sum(sq) + kNormEps);
        for (int c = lane; c < DK; c += 32) {
            sm.kh[t][c] *= rk;
            sm.qh[t][c] *= rq;
        }
    }
    __syncthreads();
    if (tid < nodes) {
        float hi = 0.f, lo = 0.f;
        for (uint64_t m = sm.path[tid]; m; m &= m - 1)
            add_exact(hi, lo, to_f32(g[(bos + __ffsll((long long)m) - 1) * a.Hv + h]));
        sm.g[tid] = hi;
        sm.g_lo[tid] = lo;
        sm.beta[tid] = sigmoidf_(to_f32(b[(bos + tid) * a.Hv + h]));
    }
    __syncthreads();
    for (int t = warp; t < nodes; t += 4)
        for (uint64_t m = sm.path[t]; m; m &= m - 1) {
            const int s = __ffsll((long long)m) - 1;
            float kk = 0.f, kq = 0.f;
            for (int c = lane; c < DK; c += 32) {
                kk += sm.kh[s][c] * sm.kh[t][c];
                kq += sm.kh[s][c] * sm.qh[t][c];
            }
            kk = warp_sum(kk);
            kq = warp_sum(kq);
            const float d = expf((sm.g[t] - sm.g[s]) + (sm.g_lo[t] - sm.g_lo[s]));
            if (lane == 0) {
                sm.a[t][s] = d * kk;
                sm.p[t][s] = d * kq;
            }
        }
    __syncthreads();
    if (tid >= DV) return;
    float row[DK];
    const float *src = a.state_in + ((slot * a.Hv + h) * DV + tid) * DK;
#pragma unroll
    for (int c = 0; c < DK; c += 4) {
        const float4 x = load4(src + c);
        row[c] = x.x; row[c + 1] = x.y; row[c + 2] = x.z; row[c + 3] = x.w;
    }
    for (int t = 0; t < nodes; ++t) {
        float xk[4] = {0.f, 0.f, 0.f, 0.f}, xq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < DK; c += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xk[e] = fmaf(row[c + e], sm.kh[t][c + e], xk[e]);
                xq[e] = fmaf(row[c + e], sm.qh[t][c + e], xq[e]);
            }
        const uint64_t path = sm.path[t];
        const float eg = path ? expf(sm.g[t] + sm.g_lo[t]) : 1.f;
        float sum = 0.f, o = eg * ((xq[0] + xq[1]) + (xq[2] + xq[3]));
        for (uint64_t m = path & ~(1ull << t); m; m &= m - 1) {
            const int s = __ffsll((long long)m) - 1;
            sum = fmaf(sm.a[t][s], sm.u[s][tid], sum);
            o = fmaf(sm.p[t][s], sm.u[s][tid], o);
        }
        const long at = ((bos + t) * a.Hv + h) * DV + tid;
        if (path) {
            const float u = sm.beta[t] * (to_f32(v[at]) - eg * ((xk[0] + xk[1]) + (xk[2] + xk[3])) - sum);
            sm.u[t][tid] = u;
            o = fmaf(sm.p[t][t], u, o);
        }
        out[at] = from_f32<T>(o);
    }
}

template <int DK, int DV>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    auto kernel = tree_scan_kernel<float, DK, DV>;
    constexpr int bytes = sizeof(ScanSmem<float, DK, DV>);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(a.B * a.Hv), 128, bytes, s>>>(a);
    return cudaGetLastError();
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
