// tree_verify.cu -- drafted tokens of a tree against the target's probabilities, from given random numbers.
//
// A walk from node 0. At a node with target row p and draft row q, its children i in order: with w_1 = p, Z_1 = 1,
//     accepted if r_i Z_i q(x_i) < w_i(x_i),   else   w_{i+1} = max(w_i - Z_i q, 0),  Z_{i+1} = sum w_{i+1},
// which leaves the accepted token distributed as p. Unrolled, w_{i+1} = max(p - c q, 0) with c = Z_1 + .. + Z_i, so
// only one number is carried over the vocabulary, and a rejection followed by another child, or by the draw of the
// next token from what is left, costs one pass over the two rows. Without draft probabilities q is one at the child's
// token: a rejection takes that token out and needs no pass.
//
// What bounds it: a row or two of V fp32 per sequence. A cluster of CTAs takes a sequence, each a run of the row, each
// warp a part of that; what a pass finds is exchanged through distributed shared memory, and all CTAs take the same
// decisions. Everything that the walk itself looks at is fetched at once beforehand.
//
// Precision. A draw compares r times a sum with partial sums over V values that lie close to one another, so sums and
// weights are kept in two floats each (48 bits), which costs fp32 operations only; fp64 ones are few.
#include "kv_pages.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kVerFlight = 4;  // loads of 16 bytes of a row in flight per lane
constexpr int kVerThreads = 256, kVerWarps = kVerThreads / 32, kVerCluster = 8, kVerParts = kVerWarps * kVerCluster;
constexpr int kVerSteps = kVerMaxVocab / 4 / kVerParts / 32 + 2;  // of 32 groups of 4, per warp
static_assert(kVerParts == 64, "a lane holds two warps' sums");

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_meet() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(double *at, uint32_t rank, double x) {
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"((uint32_t)__cvta_generic_to_shared(at)), "r"(rank));
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(x) : "memory");
}
__device__ __forceinline__ double warp_sum_f64(double x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ double warp_scan_f64(double x) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)(threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// Values of two elements at a time, as hi + lo each: one packed operation serves both.
struct Two {
    F2 hi, lo;
};
__device__ __forceinline__ F2 less(F2 a, F2 b) { return f2_fma(b, f2(-1.f, -1.f), a); }  // a - b, rounded once
__device__ __forceinline__ void add(Two &a, const Two &b) {
    const F2 s = f2_add(a.hi, b.hi), y = less(s, a.hi);
    const F2 e = f2_add(less(a.hi, less(s, y)), less(b.hi, y));  // what the rounding of s lost
    a.lo = f2_add(a.lo, f2_add(e, b.lo));
    a.hi = s;
}

struct VerSmem {
    double part[2][kVerParts];  // a pass's sums by warp, two passes' by turns
    double step[kVerSteps];
    int up[kTreeMax], token[kTreeMax], gone[kTreeMax], path[kTreeMax];
    float p[kTreeMax], q[kTreeMax], r[kTreeMax];
};

// The weights of a node's row: max(p - c q, 0), or p without the tokens that are gone.
struct Row {
    const float *p, *q;
    int V, head;      // elements before p's first 16-byte boundary: group 0; group j > 0 has the 4 from head + 4 (j - 1)
    bool same;        // q's boundaries are p's
    float ch, cl;     // c
    const int *gone;
    int ngone;        // (as far as they concern the warp at hand)
    __device__ __forceinline__ int first(int j) const { return j == 0 ? 0 : head + 4 * (j - 1); }
    __device__ __forceinline__ void load(int j, float (&x)[4], float (&y)[4]) const {
        const int e = first(j), n = j == 0 ? head : V - e;
        if (j > 0 && n >= 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p + e));
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            if (ch != 0.f) {
                if (same) {
                    const float4 b = __ldg(reinterpret_cast<const float4 *>(q + e));
                    y[0] = b.x; y[1] = b.y; y[2] = b.z; y[3] = b.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = __ldg(q + e + i);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = i < n ? __ldg(p + e + i) : 0.f;
                y[i] = i < n && ch != 0.f ? __ldg(q + e + i) : 0.f;
            }
        }
    }
    // of elements e and e + 1
    __device__ __forceinline__ Two weights(float x0, float x1, float y0, float y1, int e) const {
        if (ch != 0.f) {
            const F2 x = f2(x0, x1), y = f2(y0, y1);
            const F2 mh = f2_mul(f2(-ch, -ch), y);  // -c y = mh + ml
            const F2 ml = f2_fma(f2(-cl, -cl), y, f2_fma(f2(-ch, -ch), y, f2_mul(mh, f2(-1.f, -1.f))));
            const F2 s = f2_add(x, mh), z = less(x, s);  // x + mh and what that lost
            const F2 lo = f2_add(f2_add(less(x, f2_add(s, z)), f2_add(z, mh)), ml);
            float h0, h1, l0, l1;
            f2_get(s, h0, h1);
            f2_get(lo, l0, l1);
            if (h0 + l0 <= 0.f) h0 = l0 = 0.f;
            if (h1 + l1 <= 0.f) h1 = l1 = 0.f;
            return Two{f2(h0, h1), f2(l0, l1)};
        }
        for (int i = 0; i < ngone; ++i) {
            if (gone[i] == e) x0 = 0.f;
            if (gone[i] == e + 1) x1 = 0.f;
        }
        return Two{f2(x0, x1), f2(0.f, 0.f)};
    }
};

__global__ void __launch_bounds__(kVerThreads) tree_verify_kernel(const VerifyArgs a) {
    __shared__ VerSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockIdx.x / kVerCluster;
    const uint32_t rank = cluster_rank();
    before_reading();
    long bos = 0;
    int nodes = 0;
    if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &bos, &nodes, a.status)) nodes = 0;
    if (nodes > a.path_stride) {
        flag_error(a.status);
        nodes = 0;
    }
    int32_t *path = a.path + (long)n * a.path_stride;
    const int root = nodes > 0 ? a.parents[bos] : -2;
    if (root != -1) {  // nothing to walk from: an idle row
        if (root >= 0) flag_error(a.status);
        if (rank == 0) {
            for (int i = tid; i < a.path_stride; i += kVerThreads) path[i] = -1;
            if (tid == 0) {
                a.counts[n] = 0;
                a.next[n] = -1;
            }
        }
        return;
    }
    if (tid < nodes) {
        const int up = tid == 0 ? -1 : a.parents[bos + tid], x = tid == 0 ? 0 : a.tokens[bos + tid];
        bool child = up >= 0;
        if (child && (up >= tid || x < 0 || x >= a.V)) {
            flag_error(a.status);
            child = false;
        }
        sm.up[tid] = child ? up : -2;
        sm.token[tid] = x;
        sm.r[tid] = child ? a.r[bos + tid] : 0.f;
        sm.p[tid] = child ? a.target[(bos + up) * a.target_stride + x] : 0.f;
        sm.q[tid] = child && a.draft ? a.draft[(bos + up) * a.draft_stride + x] : 1.f;
        if (tid == 0) sm.path[0] = 0;
    }
    cluster_meet();  // (and the CTA)
    int cur = 0, count = 1, ngone = 0, pass = 0;
    double c = 0., Z = 1.;
    Row row;
    row.p = row.q = nullptr;
    int g0 = 0, g1 = 0;         // this warp's groups
    double below0, below1;      // lane: the sums of warps 0 .. 2 lane, .. 2 lane + 1
    // Sums the current node's weights; the same result in every thread of the cluster.
    auto sum_row = [&]() -> double {
        row.p = a.target + (bos + cur) * a.target_stride;
        row.q = a.draft ? a.draft + (bos + cur) * a.draft_stride : nullptr;
        row.V = a.V;
        const int off = (int)((reinterpret_cast<uintptr_t>(row.p) >> 2) & 3);
        row.head = min((4 - off) & 3, a.V);
        row.same = (((reinterpret_cast<uintptr_t>(row.p) ^ reinterpret_cast<uintptr_t>(row.q)) & 15) == 0);
        row.ch = (float)c;
        row.cl = (float)(c - (double)row.ch);
        row.gone = sm.gone;
        const int groups = 1 + (a.V - row.head + 3) / 4, per = (groups + kVerParts - 1) / kVerParts;
        const int w = (int)rank * kVerWarps + warp;
        g0 = min(w * per, groups);
        g1 = min(g0 + per, groups);
        row.ngone = 0;
        if (ngone > 0) {
            const int e0 = row.first(g0), e1 = row.first(g1);
            for (int i = 0; i < ngone; ++i)
                if (sm.gone[i] >= e0 && sm.gone[i] < e1) row.ngone = ngone;
        }
        Two acc[2] = {{f2(0.f, 0.f), f2(0.f, 0.f)}, {f2(0.f, 0.f), f2(0.f, 0.f)}};
        for (int j = g0 + lane; j < g1; j += 32 * kVerFlight) {
            float x[kVerFlight][4], y[kVerFlight][4];
#pragma unroll
            for (int f = 0; f < kVerFlight; ++f) {
                if (j + 32 * f < g1) row.load(j + 32 * f, x[f], y[f]);
                else x[f][0] = x[f][1] = x[f][2] = x[f][3] = y[f][0] = y[f][1] = y[f][2] = y[f][3] = 0.f;
            }
#pragma unroll
            for (int f = 0; f < kVerFlight; ++f) {
                const int e = row.first(j + 32 * f);
                add(acc[0], row.weights(x[f][0], x[f][1], y[f][0], y[f][1], e));
                add(acc[1], row.weights(x[f][2], x[f][3], y[f][2], y[f][3], e + 2));
            }
        }
        float h[4], l[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f2_get(acc[i].hi, h[2 * i], h[2 * i + 1]);
            f2_get(acc[i].lo, l[2 * i], l[2 * i + 1]);
        }
        double mine = 0.;
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += (double)h[i] + (double)l[i];
        mine = warp_sum_f64(mine);
        double *part = sm.part[pass & 1];
        ++pass;
        if (lane < kVerCluster) store_remote(part + w, (uint32_t)lane, mine);
        cluster_meet();
        const double x0 = part[2 * lane], x1 = part[2 * lane + 1];
        below1 = warp_scan_f64(x0 + x1);
        below0 = below1 - x1;
        return __shfl_sync(0xffffffffu, below1, 31);
    };
    bool stale = false;  // Z is not yet known
    for (int t = 1; t < nodes; ++t) {  // children come after their parents, so one walk over the nodes meets them in turn
        if (sm.up[t] != cur) continue;
        if (stale) {
            Z = sum_row();
            stale = false;
        }
        const int x = sm.token[t];
        const double p = (double)sm.p[t], q = (double)sm.q[t];
        double w = p;
        if (a.draft) {
            w = p - c * q;
            if (w < 0.) w = 0.;
        } else {
            for (int i = 0; i < ngone; ++i)
                if (sm.gone[i] == x) w = 0.;
        }
        if ((double)sm.r[t] * Z * q < w) {
            cur = t;
            if (tid == 0) sm.path[count] = t;
            ++count;
            c = 0.;
            Z = 1.;
            __syncthreads();  // (gone is read until here)
            ngone = 0;
        } else if (a.draft) {
            c += Z;
            stale = true;
        } else {
            Z -= w;
            __syncthreads();
            if (tid == 0) sm.gone[ngone] = x;
            ++ngone;
            __syncthreads();
        }
    }
    double total = sum_row();
    if (!(total > 0.) && (c > 0. || ngone > 0)) {  // nothing is left of it: from p
        c = 0.;
        ngone = 0;
        total = sum_row();
    }
    if (rank == 0)
        for (int i = tid; i < a.path_stride; i += kVerThreads) path[i] = i < count ? sm.path[i] : -1;
    if (rank == 0 && tid == 0) a.counts[n] = count;
    if (!(total > 0. && total < (double)INFINITY)) {
        flag_error(a.status);
        if (rank == 0 && tid == 0) a.next[n] = -1;
        return;
    }
    // the part that holds the draw: the first whose end is above it, or else the last that has weight
    const double draw = (double)a.r_last[n] * total;
    const double below = __shfl_up_sync(0xffffffffu, below1, 1), start = lane == 0 ? 0. : below;
    unsigned at0 = __ballot_sync(0xffffffffu, below0 > draw && below0 > start);
    unsigned at1 = __ballot_sync(0xffffffffu, below1 > draw && below1 > below0);
    int owner;
    if (at0 | at1) {
        const int l0 = at0 ? __ffs(at0) - 1 : 64, l1 = at1 ? __ffs(at1) - 1 : 64;
        owner = l0 <= l1 ? 2 * l0 : 2 * l1 + 1;
    } else {
        at0 = __ballot_sync(0xffffffffu, below0 > start);
        at1 = __ballot_sync(0xffffffffu, below1 > below0);
        const int l0 = at0 ? 31 - __clz(at0) : -1, l1 = at1 ? 31 - __clz(at1) : -1;
        owner = l1 >= l0 ? 2 * l1 + 1 : 2 * l0;
    }
    if (owner / kVerWarps != (int)rank) return;
    const double s0 = __shfl_sync(0xffffffffu, start, owner >> 1), s1 = __shfl_sync(0xffffffffu, below0, owner >> 1);
    const double before = owner & 1 ? s1 : s0;
    // its steps of 128 elements, by all warps; then the step, by one
    const int groups = 1 + (a.V - row.head + 3) / 4, per = (groups + kVerParts - 1) / kVerParts;
    g0 = min(owner * per, groups);
    g1 = min(g0 + per, groups);
    row.ngone = ngone;
    const int steps = (g1 - g0 + 31) / 32;
    auto group_weights = [&](int j, double (&w)[4]) -> double {
        float x[4], y[4];
        if (j < g1) {
            row.load(j, x, y);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const Two v = row.weights(x[i], x[i + 1], y[i], y[i + 1], row.first(j) + i);
                float h0, h1, l0, l1;
                f2_get(v.hi, h0, h1);
                f2_get(v.lo, l0, l1);
                w[i] = (double)h0 + (double)l0;
                w[i + 1] = (double)h1 + (double)l1;
            }
        } else {
            w[0] = w[1] = w[2] = w[3] = 0.;
        }
        return (w[0] + w[1]) + (w[2] + w[3]);
    };
    for (int s = warp; s < steps; s += kVerWarps) {
        double w[4];
        const double x = warp_sum_f64(group_weights(g0 + 32 * s + lane, w));
        if (lane == 0) sm.step[s] = x;
    }
    __syncthreads();
    if (warp != 0) return;
    double base = before, step_base = before;
    int step = -1, fallback = -1;
    double fallback_base = before;
    for (int s = 0; s < steps && step < 0; s += 32) {
        const double x = s + lane < steps ? sm.step[s + lane] : 0.;
        const double end = base + warp_scan_f64(x);
        const unsigned hit = __ballot_sync(0xffffffffu, x > 0. && end > draw), some = __ballot_sync(0xffffffffu, x > 0.);
        if (hit) {
            step = s + __ffs(hit) - 1;
            step_base = __shfl_sync(0xffffffffu, end - x, __ffs(hit) - 1);
        } else if (some) {
            fallback = s + 31 - __clz(some);
            fallback_base = __shfl_sync(0xffffffffu, end - x, 31 - __clz(some));
        }
        base = __shfl_sync(0xffffffffu, end, 31);
    }
    if (step < 0) {
        step = fallback;
        step_base = fallback_base;
    }
    if (step < 0) {  // (weights below zero, which the caller must not pass)
        if (lane == 0) {
            flag_error(a.status);
            a.next[n] = -1;
        }
        return;
    }
    double w[4];
    const int j = g0 + 32 * step + lane;
    const double x = group_weights(j, w), end = step_base + warp_scan_f64(x);
    double sum = end - x;
    int pick = -1, last = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum += w[i];
        if (w[i] > 0.) {
            last = row.first(j) + i;
            if (pick < 0 && sum > draw) pick = last;
        }
    }
    const unsigned hit = __ballot_sync(0xffffffffu, pick >= 0), some = __ballot_sync(0xffffffffu, last >= 0);
    const int token = hit ? __shfl_sync(0xffffffffu, pick, __ffs(hit) - 1)
                          : __shfl_sync(0xffffffffu, last, some ? 31 - __clz(some) : 0);
    if (lane == 0) a.next[n] = token;
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kVerCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)a.B * kVerCluster);
    cfg.blockDim = dim3(kVerThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel, a);
}

}  // namespace gdn
