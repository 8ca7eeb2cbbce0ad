// tree_verify.cu -- drafted tokens of a tree against the target's probabilities, from given random numbers.
//
// A walk from node 0. At a node with target row p and draft row q, its children i in order: with w_1 = p, Z_1 = 1,
//     accepted if r_i Z_i q(x_i) < w_i(x_i),   else   w_{i+1} = max(w_i - Z_i q, 0),  Z_{i+1} = sum w_{i+1},
// which leaves the accepted token distributed as p. Unrolled, w_{i+1} = max(p - c q, 0) with c = Z_1 + .. + Z_i, so
// only one number is carried over the vocabulary, and a rejection followed by another child, or by the draw of the
// next token from what is left, costs one pass over the two rows. Without draft probabilities q is one at the child's
// token: a rejection takes that token out, Z_{i+1} = Z_i - w_i(x_i), and needs no pass. (That counts p's sum as 1. Where it
// is not, the children x_i still come with probability p(x_i), and all other tokens share 1 - p(x_1) - .. in p's
// proportions; by the sum of what is left it would be the children whose odds are off.)
//
// What bounds it: a row or two of V fp32 per sequence, and for few sequences the chain of dependent steps (the tree, the
// tokens' probabilities, a pass, the draw). A cluster of CTAs takes a sequence, each a run of the row, each warp a part
// of that; what a pass finds is sent to all CTAs of the cluster, which take the same decisions.
// Everything that the walk itself looks at is fetched at once beforehand. A lane's elements come through a ring of its own
// in shared memory, asked for ahead of their use: registers hold two groups a lane, the ring six (64 sequences of up to 13
// nodes with drafts, V = 131072: 38.5 us from registers, 33.5 so, 32.8 now; the first pass over them all takes 12 of those, 67 MB at
// 5.5 TB/s, the two later ones of the longest walks 4 to 5 each). What a warp finds goes to all CTAs by asynchronous stores
// that their barriers count, 0.4 us from the last one sent; by stores and a barrier of the cluster a pass took 1 us more.
// One session of 16 nodes, V = 150001, no draft probabilities: 7.0 us from a graph.
//
// Precision. A draw compares r times a sum with partial sums over V values that lie close to one another, so weights
// and sums are kept as two floats each (48 bits). In fp64, of which an SM does two operations a cycle, the sums over the
// warps alone kept its unit busy for a third of the time.
#include "attn_ops.cuh"
#include "kv_pages.cuh"
#include "tree.cuh"

namespace gdn {
namespace {

constexpr int kVerThreads = 256, kVerWarps = kVerThreads / 32;

// C: CTAs to a sequence. FLIGHT: pairs of groups of a row that a lane has on their way, in shared memory. PER_SM: CTAs that an SM
// has to hold.
template <bool DRAFT_, int C_, int FLIGHT_, int PER_SM_>
struct Cfg {
    static constexpr bool DRAFT = DRAFT_;
    static constexpr int C = C_, FLIGHT = FLIGHT_, PER_SM = PER_SM_;
    static constexpr int SLOT = (DRAFT ? 4 : 2) * kVerThreads * 16, RING_BYTES = FLIGHT * SLOT;  // [FLIGHT][2][p, q][thread]
    static constexpr int PARTS = kVerWarps * C, NP = PARTS / 32;                // warps of a sequence; ..' sums in a lane
    static constexpr int STEPS = kVerMaxVocab / 4 / PARTS / 32 + 2;             // of 32 groups of 4, per warp
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---- numbers of 48 bits: hi + lo, |lo| at most half a unit of hi -----------------------
// (By operations that round on their own whatever the compiler makes of their neighbours: a product drawn into the sum after it
// would leave lo beyond half a unit, and below() would compare the wrong hi.)
struct Wide {
    float hi, lo;
};
__device__ __forceinline__ Wide wide(float x) { return Wide{x, 0.f}; }
__device__ __forceinline__ Wide in_shape(float s, float e) {  // of s + e, e a unit or two of s at most
    const float h = __fadd_rn(s, e);
    return Wide{h, __fsub_rn(e, __fsub_rn(h, s))};
}
__device__ __forceinline__ Wide plus(Wide a, Wide b) {
    const float s = __fadd_rn(a.hi, b.hi), y = __fsub_rn(s, a.hi);
    const float lost = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, y)), __fsub_rn(b.hi, y));
    return in_shape(s, __fadd_rn(lost, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Wide minus(Wide a, Wide b) { return plus(a, Wide{-b.hi, -b.lo}); }
__device__ __forceinline__ Wide times(Wide a, float f) {
    const float p = __fmul_rn(a.hi, f);
    return in_shape(p, __fmaf_rn(a.lo, f, __fmaf_rn(a.hi, f, -p)));
}
__device__ __forceinline__ bool below(Wide a, Wide b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Wide shuffle(Wide a, int from) {
    return Wide{__shfl_sync(0xffffffffu, a.hi, from), __shfl_sync(0xffffffffu, a.lo, from)};
}
__device__ __forceinline__ Wide warp_total(Wide a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = plus(a, Wide{__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)});
    return a;
}
__device__ __forceinline__ Wide warp_scan(Wide a) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Wide b{__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        if ((int)(threadIdx.x & 31) >= o) a = plus(b, a);
    }
    return a;
}
// To `at` in the shared memory of CTA `rank`, whose `bar` counts the bytes
__device__ __forceinline__ void send(Wide *at, uint64_t *bar, uint32_t rank, Wide x) {
    uint32_t to, to_bar;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(at)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to_bar) : "r"(tc::smem_u32(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(x.hi), "f"(x.lo),
                 "r"(to_bar)
                 : "memory");
}
__device__ __forceinline__ void tell(int *at, uint32_t rank, int x) {  // (seen after the next barrier of the cluster)
    uint32_t to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(at)), "r"(rank));
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
}
__device__ __forceinline__ void count_off(uint64_t *bar, uint32_t bytes) {  // as if they had come
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(bytes) : "memory");
}
// Wait for what other CTAs send, with a limit in cycles, which is looked at before the thread first sleeps
__device__ __forceinline__ bool received(uint64_t *bar, uint32_t phase, long long budget) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(tc::smem_u32(bar)), "r"(phase)
                 : "memory");
    if (done) return true;
    const long long t0 = clock64();
    do {
        if (clock64() - t0 > budget) return false;
    } while (!tc::mbar_try_wait_cluster(bar, phase, 1000u));
    return true;
}

// Two such numbers side by side, without the last step that brings them into shape: one packed operation serves both.
struct Two {
    F2 hi, lo;
};
__device__ __forceinline__ float one_above_0(float x) {  // 1 if x > 0, else 0
    float k;
    asm("set.gt.f32.f32 %0, %1, 0f00000000;" : "=f"(k) : "f"(x));
    return k;
}
__device__ __forceinline__ F2 less(F2 a, F2 b) { return f2_fma(b, f2(-1.f, -1.f), a); }  // a - b, rounded once
__device__ __forceinline__ void add(Two &a, const Two &b) {
    const F2 s = f2_add(a.hi, b.hi), y = less(s, a.hi);
    const F2 e = f2_add(less(a.hi, less(s, y)), less(b.hi, y));  // what the rounding of s lost
    a.lo = f2_add(a.lo, f2_add(e, b.lo));
    a.hi = s;
}
__device__ __forceinline__ void get(const Two &a, Wide &x, Wide &y) {
    float h0, h1, l0, l1;
    f2_get(a.hi, h0, h1);
    f2_get(a.lo, l0, l1);
    x = plus(wide(h0), wide(l0));
    y = plus(wide(h1), wide(l1));
}

// Copies to shared memory that the asking thread alone waits for and reads
__device__ __forceinline__ void copy16(uint32_t to, const float *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const float *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // for all but the last N groups of copies
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void take16(uint32_t from, float (&x)[4]) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(from) : "memory");
}

template <typename C>
struct VerSmem {
    Wide part[2][C::PARTS];  // a pass's sums by warp, two passes' by turns
    uint64_t bar[2];         // .. arrivals
    int sent[C::C];          // of a CTA whose wait has run out: the passes whose sums it has sent; else 0
    Wide step[C::STEPS];
    int up[kTreeMax], token[kTreeMax], gone[kTreeMax], path[kTreeMax];
    float p[kTreeMax], q[kTreeMax], r[kTreeMax];
};

// The weights of a node's row: max(p - c q, 0) (DRAFT), or p, from which strike takes the tokens that are gone.
template <bool DRAFT>
struct Row {
    const float *p, *q;
    int V, shift;  // group j has the elements from shift + 4 j, 4 from a 16-byte boundary of p (the first and the last: those
                   // of them that there are)
    bool same;     // q's boundaries are p's
    Wide c;
    const int *gone;
    int ngone;     // (0 where none concerns the warp at hand)
    int mine[2];   // lane: entries lane and lane + 32 of the list
    __device__ __forceinline__ void place(const float *at, int n) {
        p = at;
        V = n;
        shift = -(int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
    }
    __device__ __forceinline__ int groups() const { return (V - shift + 3) / 4; }
    __device__ __forceinline__ int first(int j) const { return max(shift + 4 * j, 0); }
    __device__ __forceinline__ void load(int j, float (&x)[4], float (&y)[4]) const {
        const int e = first(j), n = min(shift + 4 * j + 4, V) - e;
        if (n == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(p + e));
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            if (DRAFT && c.hi != 0.f) {
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
                y[i] = DRAFT && i < n && c.hi != 0.f ? __ldg(q + e + i) : 0.f;
            }
        }
    }
    __device__ __forceinline__ Two weights(float x0, float x1, float y0, float y1) const {
        if constexpr (DRAFT) {
            if (c.hi != 0.f) {
                // Where p - c q is above 0, p >= fl(c q) >= 0, so that what the difference loses is found in two steps.
                const F2 x = f2(x0, x1), y = f2(y0, y1), m = f2_mul(f2(c.hi, c.hi), y), d = less(x, m);
                const F2 t = f2_fma(f2(-c.lo, -c.lo), y, f2_fma(f2(-c.hi, -c.hi), y, m));  // m - c y
                const F2 lo = f2_add(less(less(x, d), m), t);
                float h0, h1;
                f2_get(f2_add(d, lo), h0, h1);
                const F2 k = f2(one_above_0(h0), one_above_0(h1));  // (a NaN stays one: 0 times NaN)
                return Two{f2_mul(d, k), f2_mul(lo, k)};
            }
        }
        return Two{f2(x0, x1), f2(0.f, 0.f)};
    }
    // Of elements e .. e + 3, by one thread
    __device__ __forceinline__ void strike_alone(float (&x)[4], int e) const {
        if constexpr (!DRAFT)
            for (int i = 0; i < ngone; ++i)
#pragma unroll
                for (int f = 0; f < 4; ++f)
                    if (gone[i] == e + f) x[f] = 0.f;
    }
    // ... by a whole warp, whose lanes have 128 elements or less from `base` on. (Every token of the list compared with every
    // element made the warps that a token of the list concerns 2.3 us later than all others, for 14 tokens.)
    __device__ __forceinline__ void strike(float (&x)[4], int e, int base) const {
        if constexpr (!DRAFT) {
            if (ngone == 0) return;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                unsigned near = __ballot_sync(0xffffffffu, (unsigned)mine[i] - (unsigned)base < 128u);
                while (near) {
                    const int at = __shfl_sync(0xffffffffu, mine[i], __ffs(near) - 1) - e;
                    near &= near - 1;
#pragma unroll
                    for (int f = 0; f < 4; ++f)
                        if (at == f) x[f] = 0.f;
                }
            }
        }
    }
    // The list as far as it concerns the elements from e0 to e1
    __device__ __forceinline__ void list(int count, int e0, int e1) {
        if constexpr (!DRAFT) {
            const int lane = threadIdx.x & 31;
            bool any = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mine[i] = lane + 32 * i < count ? gone[lane + 32 * i] : -1;
                any |= mine[i] >= e0 && mine[i] < e1;
            }
            ngone = __any_sync(0xffffffffu, any) ? count : 0;
        }
    }
};

template <typename C>
__global__ void __launch_bounds__(kVerThreads, C::PER_SM) tree_verify_kernel(const VerifyArgs a, long long budget) {
    constexpr bool DRAFT = C::DRAFT;
    constexpr int kFlight = C::FLIGHT, NP = C::NP;
    __shared__ VerSmem<C> sm;
    extern __shared__ __align__(16) uint8_t ring[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockIdx.x / C::C;
    const uint32_t rank = cluster_rank();
    if (tid == 0) {
        tc::mbar_init(&sm.bar[0], 1);
        tc::mbar_init(&sm.bar[1], 1);
        tc::fence_mbar_init();
    }
    if (tid < C::C) sm.sent[tid] = 0;
    __syncwarp();
    cluster_arrive();  // (waited for before anything is sent to another CTA)
    next_may_begin();
    before_reading();
    long bos = 0;
    int nodes = 0;
    if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &bos, &nodes, a.status)) nodes = 0;
    if (nodes > a.path_stride) {
        flag_error(a.status);
        nodes = 0;
    }
    int32_t *path = a.path + (long)n * a.path_stride;
    // (all that a node's thread can fetch without knowing more)
    int up = -2, x = 0;
    float rn = 0.f;
    if (tid < nodes) {
        up = a.parents[bos + tid];
        if (tid > 0) {
            x = a.tokens[bos + tid];
            rn = a.r[bos + tid];
        }
    }
    const float r_last = a.r_last[n];
    if (tid < nodes) {
        bool child = tid > 0 && up >= 0;
        if (tid == 0 ? up >= 0 : child && (up >= tid || x < 0 || x >= a.V)) {
            flag_error(a.status);
            child = false;
        }
        sm.up[tid] = tid == 0 ? up : child ? up : -2;
        sm.token[tid] = x;
        sm.r[tid] = rn;
        sm.p[tid] = child ? a.target[(bos + up) * a.target_stride + x] : 0.f;
        sm.q[tid] = DRAFT && child ? a.draft[(bos + up) * a.draft_stride + x] : 1.f;
        if (tid == 0) sm.path[0] = 0;
    }
    __syncthreads();
    if (nodes == 0 || sm.up[0] != -1) {  // nothing to walk from: an idle row
        if (rank == 0) {
            for (int i = tid; i < a.path_stride; i += kVerThreads) path[i] = -1;
            if (tid == 0) {
                a.counts[n] = 0;
                a.next[n] = -1;
            }
        }
        cluster_wait();
        return;
    }
    int cur = 0, count = 1, ngone = 0, pass = 0;
    bool ok = true;  // the same in all threads of the CTA
    Wide c = wide(0.f), Z = wide(1.f);
    Row<DRAFT> row;
    int g0 = 0, g1 = 0;        // this warp's groups
    Wide ends[NP];             // lane: the sums of all parts up to NP lane + i
    const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(ring) + tid * 16;
    // Sums the current node's weights; the same result in every thread of the cluster.
    auto sum_row = [&]() -> Wide {
        row.place(a.target + (bos + cur) * a.target_stride, a.V);
        row.q = DRAFT ? a.draft + (bos + cur) * a.draft_stride : nullptr;
        row.same = ((reinterpret_cast<uintptr_t>(row.p) ^ reinterpret_cast<uintptr_t>(row.q)) & 15) == 0;
        row.c = c;
        row.gone = sm.gone;
        const int groups = row.groups(), per = (groups + C::PARTS - 1) / C::PARTS;
        const int w = (int)rank * kVerWarps + warp;
        g0 = min(w * per, groups);
        g1 = min(g0 + per, groups);
        row.list(ngone, row.first(g0), row.first(g1));
        Two acc[2] = {{f2(0.f, 0.f), f2(0.f, 0.f)}, {f2(0.f, 0.f), f2(0.f, 0.f)}};
        const bool with_q = DRAFT && c.hi != 0.f;
        const int whole0 = row.shift < 0, whole1 = (a.V - row.shift) / 4;  // groups of 4 elements
        const int j0 = max(g0, whole0) + lane, end = min(g1, whole1);
        const float *pp = row.p + row.first(j0), *pq = DRAFT ? row.q + row.first(j0) : nullptr;
        int asked = j0;
        uint32_t to = mine_at;
        auto ask = [&] {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (asked + 32 * u < end) {
                    const uint32_t at = to + u * (C::SLOT / 2);
                    copy16(at, pp + 128 * u);
                    if (with_q) {
                        if (row.same) copy16(at + kVerThreads * 16, pq + 128 * u);
                        else
#pragma unroll
                            for (int i = 0; i < 4; ++i) copy4(at + kVerThreads * 16 + 4 * i, pq + 128 * u + i);
                    }
                }
            copies_end();
            asked += 64;
            pp += 256;
            if (DRAFT) pq += 256;
            to = to == mine_at + (kFlight - 1) * C::SLOT ? mine_at : to + C::SLOT;
        };
#pragma unroll 1
        for (int f = 0; f < kFlight; ++f) ask();
        if ((g0 < whole0 && lane == 0) || (g1 > max(max(g0, whole0), whole1) && lane == 1)) {
            const int j = lane == 0 ? 0 : whole1;
            float x[4], y[4];
            row.load(j, x, y);
            row.strike_alone(x, row.first(j));
            add(acc[0], row.weights(x[0], x[1], y[0], y[1]));
            add(acc[1], row.weights(x[2], x[3], y[2], y[3]));
        }
        uint32_t at = mine_at;
#pragma unroll 1
        for (int j = j0; j - lane < end; j += 64) {
            copies_wait<kFlight - 1>();
            float x[2][4] = {}, y[2][4] = {};
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (j + 32 * u < end) {
                    take16(at + u * (C::SLOT / 2), x[u]);
                    if (with_q) take16(at + u * (C::SLOT / 2) + kVerThreads * 16, y[u]);
                }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                row.strike(x[u], row.first(j + 32 * u), row.first(j - lane + 32 * u));
                add(acc[0], row.weights(x[u][0], x[u][1], y[u][0], y[u][1]));
                add(acc[1], row.weights(x[u][2], x[u][3], y[u][2], y[u][3]));
            }
            ask();
            at = to;
        }
        Wide s0, s1, s2, s3;
        get(acc[0], s0, s1);
        get(acc[1], s2, s3);
        const Wide mine = warp_total(plus(plus(s0, s1), plus(s2, s3)));
        // A CTA's pass p + 2 comes after it has all sums of p + 1, and those after their warps are done with the sums of p.
        Wide *part = sm.part[pass & 1];
        uint64_t *bar = &sm.bar[pass & 1];
        const uint32_t phase = (pass >> 1) & 1;
        if (tid == 0) tc::mbar_expect_tx(bar, C::PARTS * (uint32_t)sizeof(Wide));
        if (pass++ == 0) cluster_wait();
        if (lane < C::C) send(part + w, bar, (uint32_t)lane, mine);
        if (__syncthreads_or(!received(bar, phase, budget))) {
            ok = false;
            return wide(0.f);
        }
        ends[0] = part[NP * lane];
#pragma unroll
        for (int i = 1; i < NP; ++i) ends[i] = plus(ends[i - 1], part[NP * lane + i]);
        const Wide all = ends[NP - 1], before = minus(warp_scan(all), all);
#pragma unroll
        for (int i = 0; i < NP; ++i) ends[i] = plus(before, ends[i]);
        return shuffle(ends[NP - 1], 31);
    };
    bool stale = false;  // Z is not yet known
    const int up0 = lane < nodes ? sm.up[lane] : -2, up1 = lane + 32 < nodes ? sm.up[lane + 32] : -2;
    auto children = [&]() -> uint64_t {
        return (uint64_t)__ballot_sync(0xffffffffu, up1 == cur) << 32 | __ballot_sync(0xffffffffu, up0 == cur);
    };
    uint64_t left = children();  // of the current node, in turn
    while (left != 0) {
        const int t = __ffsll((long long)left) - 1;
        left &= left - 1;
        if (stale) {
            Z = sum_row();
            if (!ok) break;
            stale = false;
        }
        const int x = sm.token[t];
        const float p = sm.p[t], q = sm.q[t];
        Wide w = wide(p);
        if (DRAFT) {
            w = minus(w, times(c, q));
            if (w.hi < 0.f) w = wide(0.f);
        } else {
            for (int i = 0; i < ngone; ++i)
                if (sm.gone[i] == x) w = wide(0.f);
        }
        if (below(times(times(Z, q), sm.r[t]), w)) {
            cur = t;
            if (tid == 0) sm.path[count] = t;
            ++count;
            c = wide(0.f);
            Z = wide(1.f);
            if (!DRAFT) __syncthreads();  // (gone is read until here)
            ngone = 0;
            left = children();
        } else if (DRAFT) {
            c = plus(c, Z);
            stale = true;
        } else {
            Z = minus(Z, w);
            __syncthreads();
            if (tid == 0) sm.gone[ngone] = x;
            ++ngone;
            __syncthreads();
        }
    }
    Wide total = wide(0.f);
    if (ok) total = sum_row();
    if (ok && !(total.hi > 0.f) && (c.hi > 0.f || ngone > 0)) {  // nothing is left of it: from p
        c = wide(0.f);
        ngone = 0;
        total = sum_row();
    }
    // No CTA leaves while others may send to it, and a sequence has the results of all of its CTAs or none: each says here
    // that it has every sum of the last pass, or that one of its waits has run out.
    if (ok) {
        cluster_arrive_relaxed();  // (nothing that it has written is for others: a release here took 0.4 us)
    } else {
        if (tid < C::C) tell(&sm.sent[rank], (uint32_t)tid, pass);
        __syncwarp();
        cluster_arrive();
    }
    constexpr int kNone = -2;
    // The next token, -1 if there is none (flagged), in one thread of the cluster; kNone in all others.
    auto draw_token = [&]() -> int {
        if (!(total.hi > 0.f && total.hi < INFINITY)) {
            flag_error(a.status);
            return rank == 0 && tid == 0 ? -1 : kNone;
        }
        // the part that holds the draw: the first whose end is above it, or else the last that has weight
        const Wide draw = times(total, r_last);
        int owner = kVerWarps * C::C, last_live = -1;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const bool live = sm.part[(pass - 1) & 1][NP * lane + i].hi > 0.f;
            const unsigned at = __ballot_sync(0xffffffffu, live && below(draw, ends[i])), some = __ballot_sync(0xffffffffu, live);
            if (at) owner = min(owner, NP * (__ffs(at) - 1) + i);
            if (some) last_live = max(last_live, NP * (31 - __clz(some)) + i);
        }
        if (owner == kVerWarps * C::C) owner = max(last_live, 0);
        if (owner / kVerWarps != (int)rank) return kNone;
        Wide base = wide(0.f);  // the sum of all parts before it
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const Wide e = shuffle(ends[i], (owner > 0 ? owner - 1 : 0) / NP);
            if (owner > 0 && (owner - 1) % NP == i) base = e;
        }
        // its steps of 128 elements, by all warps; then the step, by one
        const int groups = row.groups(), per = (groups + C::PARTS - 1) / C::PARTS;
        g0 = min(owner * per, groups);
        g1 = min(g0 + per, groups);
        row.list(ngone, row.first(g0), row.first(g1));
        const int steps = (g1 - g0 + 31) / 32;
        auto group_weights = [&](int j, Wide (&w)[4]) -> Wide {
            float x[4] = {}, y[4] = {};
            if (j < g1) row.load(j, x, y);
            row.strike(x, row.first(j), row.first(j - lane));
            get(row.weights(x[0], x[1], y[0], y[1]), w[0], w[1]);
            get(row.weights(x[2], x[3], y[2], y[3]), w[2], w[3]);
            return plus(plus(w[0], w[1]), plus(w[2], w[3]));
        };
        for (int s = warp; s < steps; s += kVerWarps) {
            Wide w[4];
            const Wide x = warp_total(group_weights(g0 + 32 * s + lane, w));
            if (lane == 0) sm.step[s] = x;
        }
        __syncthreads();
        if (warp != 0) return kNone;
        int step = -1, fallback = -1;
        Wide step_base = base, fallback_base = base;
        for (int s = 0; s < steps && step < 0; s += 32) {
            const Wide x = s + lane < steps ? sm.step[s + lane] : wide(0.f);
            const Wide end = plus(base, warp_scan(x));
            const unsigned hit = __ballot_sync(0xffffffffu, x.hi > 0.f && below(draw, end)), some = __ballot_sync(0xffffffffu, x.hi > 0.f);
            const Wide begin = minus(end, x);
            if (hit) {
                step = s + __ffs(hit) - 1;
                step_base = shuffle(begin, __ffs(hit) - 1);
            } else if (some) {
                fallback = s + 31 - __clz(some);
                fallback_base = shuffle(begin, 31 - __clz(some));
            }
            base = shuffle(end, 31);
        }
        if (step < 0) {
            step = fallback;
            step_base = fallback_base;
        }
        if (step < 0) {  // (weights below zero, which the caller must not pass)
            flag_error(a.status);
            return lane == 0 ? -1 : kNone;
        }
        Wide w[4];
        const int j = g0 + 32 * step + lane;
        const Wide x_all = group_weights(j, w);
        Wide sum = minus(plus(step_base, warp_scan(x_all)), x_all);
        int pick = -1, last = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sum = plus(sum, w[i]);
            if (w[i].hi > 0.f) {
                last = row.first(j) + i;
                if (pick < 0 && below(draw, sum)) pick = last;
            }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, pick >= 0), some = __ballot_sync(0xffffffffu, last >= 0);
        const int token = hit ? __shfl_sync(0xffffffffu, pick, __ffs(hit) - 1)
                              : __shfl_sync(0xffffffffu, last, some ? 31 - __clz(some) : 0);
        return lane == 0 ? token : kNone;
    };
    const int token = ok ? draw_token() : kNone;
    __syncwarp();
    cluster_wait();
    bool whole = true;
#pragma unroll
    for (int r = 0; r < C::C; ++r) whole &= sm.sent[r] == 0;
    if (!whole) count = 0;
    if (rank == 0) {
        for (int i = tid; i < a.path_stride; i += kVerThreads) path[i] = i < count ? sm.path[i] : -1;
        if (tid == 0) a.counts[n] = count;
        if (!whole && tid == 0) a.next[n] = -1;
    }
    if (whole && token != kNone) a.next[n] = token;
    if (!ok && tid == 0) {
        flag_error(a.status);
        // What others have sent lands before this CTA leaves. Every CTA sends its sums of a pass before it waits for those of the
        // others, so of the pass whose wait ran out all come but those of CTAs that gave up one pass before, which are counted
        // off; and CTAs that went on have sent those of one pass more, since it takes all CTAs' to go on again.
        int behind = 0, ahead = 0;
        for (int r = 0; r < C::C; ++r) {
            behind += sm.sent[r] != 0 && sm.sent[r] < pass;
            ahead += sm.sent[r] > pass;
        }
        constexpr uint32_t kBytes = kVerWarps * (uint32_t)sizeof(Wide);  // of a CTA
        uint64_t *bar = &sm.bar[(pass - 1) & 1], *next = &sm.bar[pass & 1];
        if (behind > 0) count_off(bar, behind * kBytes);
        received(bar, ((pass - 1) >> 1) & 1, kDrainBudget);
        if (ahead > 0) {
            tc::mbar_expect_tx(next, ahead * kBytes);
            received(next, (pass >> 1) & 1, kDrainBudget);
        }
    }
}

template <typename C>
cudaError_t launch_t(const VerifyArgs &a, cudaStream_t s) {
    auto kernel = tree_verify_kernel<C>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::RING_BYTES);
    if (e != cudaSuccess) return e;
    if (C::C > 8) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C::C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)a.B * C::C);
    cfg.blockDim = dim3(kVerThreads);
    cfg.dynamicSmemBytes = C::RING_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, wait_budget());
}

}  // namespace

cudaError_t launch_tree_verify(const VerifyArgs &a, cudaStream_t s) {
    // CTAs to a sequence: 16 against 8, us from a graph, sequences of 13 nodes.
    //     sequences                       1          4          8          9         12         16         32
    //     drafts, V = 131072       7.7  9.2  11.9 14.9  13.8 16.4  15.8 18.5  16.1 19.3  19.7 21.9  32.5 30.8
    //     drafts, V = 32000        8.4  8.6  10.0 10.4  11.7 11.8  10.6 10.7  12.4 12.8  13.2 13.5  22.2 15.9
    //     no drafts, V = 131072    6.3  7.4   6.7  7.9   7.5  7.9   7.4  8.2   8.8  8.7  10.2  9.5  13.5 11.8
    //     no drafts, V = 32000     5.7  5.6   6.1  6.0   6.5  6.1   6.5  6.2   7.6  6.2   8.7  6.9  11.1  8.4
    // (A cluster of 16 finds less room. Up to 16 sequences with drafts it would still be 10% ahead, without drafts behind.)
    // The kernel for drafts and 8 CTAs has 64 registers, so that four CTAs fit an SM, and spills 24 bytes a thread.
    if (a.B <= 8) return a.draft ? launch_t<Cfg<true, 16, 5, 1>>(a, s) : launch_t<Cfg<false, 16, 5, 1>>(a, s);
    return a.draft ? launch_t<Cfg<true, 8, 3, 4>>(a, s) : launch_t<Cfg<false, 8, 6, 4>>(a, s);
}

}  // namespace gdn
