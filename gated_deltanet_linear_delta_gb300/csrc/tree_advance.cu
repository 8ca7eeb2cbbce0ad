// tree_advance.cu -- the gated delta rule's states after the accepted path of a tree of drafted tokens.
//
// The recurrence, node by node (one read and one write of each state, whatever the path's length):
//     u_i = beta (v_i - alpha (S kh)_i),   S_i <- alpha S_i + u_i kh^T.
//
// Bound by the bytes of the states. A CTA takes one (sequence, value head): all of its state is asked for at once, and
// stands in registers while the path runs over it; two or three CTAs to an SM keep reads, work and writes of different
// heads side by side. A row lies in 8 lanes (16-byte pieces by turns, so that a warp's access is whole lines), 4 rows a
// warp and pass, up to 4 passes, whose reductions over the 8 lanes run side by side. What a node contributes to every
// row -- the unit key, v, alpha, beta -- is prepared once for all rows, eight nodes at a time, in shared memory.
// Measured: 128 sequences, up to 16 nodes and 4 accepted, 32 heads of 128 x 128: 88 us, 6.15 TB/s of 6.7 measured; one 5.1 us.
#include "kv_pages.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

// CTAs to an SM. Of the largest states (64 registers of a thread) two: 128 sequences of up to 16 nodes, 32 heads, 88 us;
// three leave 80 registers, spill, and take 106.
template <int DK, int DV>
constexpr int kAdvPerSm = DK * DV > 8192 ? 2 : 3;
constexpr int kAdvThreads = 256, kAdvWarps = kAdvThreads / 32, kAdvNodes = 8;

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kAdvThreads, kAdvPerSm<DK, DV>) tree_advance_kernel(const TreeArgs a) {
    constexpr int P = DK / 32;                                        // pieces of a row in a lane
    constexpr int ROWS = 4 * kAdvWarps, R = DV / ROWS;                // rows a pass; passes
    static_assert(DV % ROWS == 0, "every lane holds a piece of a row in every pass");
    __shared__ float kh[kAdvNodes][DK], vv[kAdvNodes][DV], alpha[kAdvNodes], beta[kAdvNodes];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c = lane & 7;
    const int n = blockIdx.x / a.Hv, h = blockIdx.x % a.Hv, hk = h / (a.Hv / a.Hk);
    next_may_begin();
    before_reading();
    long bos;
    int nodes;
    if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &bos, &nodes, a.status)) return;
    const long slot = state_slot(a, n);
    if (slot < 0) return;
    const long at = ((slot * a.Hv + h) * DV + warp * 4 + (lane >> 3)) * DK + 4 * c;
    float4 s[R][P];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int p = 0; p < P; ++p)
            s[r][p] = __ldcs(reinterpret_cast<const float4 *>(a.state_in + at + (long)r * ROWS * DK + 32 * p));
    int count = a.counts[n];
    bool bad = count < 0 || count > min(nodes, a.path_stride);
    const int32_t *path = a.path + (long)n * a.path_stride;
    if (!bad && tid < count) bad = path[tid] < 0 || path[tid] >= nodes;
    if (__syncthreads_or(bad)) {
        if (tid == 0) flag_error(a.status);
        count = 0;
    }
    for (int i0 = 0; i0 < count; i0 += kAdvNodes) {
        if (i0) __syncthreads();
        // a node a warp
        if (i0 + warp < count) {
            const long tok = bos + path[i0 + warp];
            const T *k = (const T *)a.k + (tok * a.Hk + hk) * DK, *v = (const T *)a.v + (tok * a.Hv + h) * DV;
            float x[DK / 32], sum = 0.f;
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) {
                x[e] = to_f32(k[lane + 32 * e]);
                sum = fmaf(x[e], x[e], sum);
            }
#pragma unroll
            for (int e = 0; e < DV / 32; ++e) vv[warp][lane + 32 * e] = to_f32(v[lane + 32 * e]);
            const float rk = 1.f / sqrtf(warp_sum(sum) + kNormEps);
#pragma unroll
            for (int e = 0; e < DK / 32; ++e) kh[warp][lane + 32 * e] = x[e] * rk;
            if (lane == 0) {
                alpha[warp] = expf(to_f32(((const T *)a.g)[tok * a.Hv + h]));
                beta[warp] = sigmoidf_(to_f32(((const T *)a.b)[tok * a.Hv + h]));
            }
        }
        __syncthreads();
        const int m = min(kAdvNodes, count - i0);
        for (int i = 0; i < m; ++i) {
            float4 x[P];
#pragma unroll
            for (int p = 0; p < P; ++p) x[p] = *reinterpret_cast<const float4 *>(&kh[i][4 * c + 32 * p]);
            const float al = alpha[i], be = beta[i];
            float dot[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                dot[r] = 0.f;
#pragma unroll
                for (int p = 0; p < P; ++p) dot[r] += dot4(s[r][p], x[p]);
            }
#pragma unroll
            for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                for (int r = 0; r < R; ++r) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], o);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float u = be * (vv[i][r * ROWS + warp * 4 + (lane >> 3)] - al * dot[r]);
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    s[r][p].x = fmaf(u, x[p].x, al * s[r][p].x);
                    s[r][p].y = fmaf(u, x[p].y, al * s[r][p].y);
                    s[r][p].z = fmaf(u, x[p].z, al * s[r][p].z);
                    s[r][p].w = fmaf(u, x[p].w, al * s[r][p].w);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int p = 0; p < P; ++p)
            __stcs(reinterpret_cast<float4 *>(a.state_out + at + (long)r * ROWS * DK + 32 * p), s[r][p]);
}

template <typename T, int DK, int DV>
cudaError_t launch_t(const TreeArgs &a, cudaStream_t s) {
    return launch_early(tree_advance_kernel<T, DK, DV>, dim3((unsigned)(a.B * a.Hv)), kAdvThreads, 0, s, a);
}

template <typename T, int DK>
cudaError_t launch_dv(const TreeArgs &a, cudaStream_t s) {
    switch (a.dv) {
        case 32: return launch_t<T, DK, 32>(a, s);
        case 64: return launch_t<T, DK, 64>(a, s);
        case 128: return launch_t<T, DK, 128>(a, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_dk(const TreeArgs &a, cudaStream_t s) {
    switch (a.dk) {
        case 32: return launch_dv<T, 32>(a, s);
        case 64: return launch_dv<T, 64>(a, s);
        case 128: return launch_dv<T, 128>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_tree_advance(const TreeArgs &a, cudaStream_t s) {
    return a.dtype == GDN_F32 ? launch_dk<float>(a, s) : launch_dk<__nv_bfloat16>(a, s);
}

}  // namespace gdn
