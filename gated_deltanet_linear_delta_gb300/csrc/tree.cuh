// tree.cuh -- trees of drafted tokens: the nodes of a sequence, and the path from the root to each.
//
// A sequence's nodes are packed tokens; parents[t] < t is node t's parent, -1 the root's. Any other value below
// makes a padding node, whose path is empty, and so are its descendants'. A sequence has at most 64 nodes, so that
// a path is the set bits of one word.
#pragma once

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

// Bounds of sequence n and its nodes. False (flagged) where cu is inconsistent or there are too many nodes.
__device__ __forceinline__ bool tree_bounds(const int32_t *cu, int n, int B, long T, long *bos, int *nodes, int *status) {
    long eos;
    if (!seq_bounds(cu, n, B, T, bos, &eos, status)) return false;
    if (eos - *bos > kTreeMax) {
        flag_error(status);
        return false;
    }
    *nodes = (int)(eos - *bos);
    return true;
}

// hi + x as a rounded sum, and what that lost added to lo (no product that hi or x comes from may be drawn into it)
__device__ __forceinline__ void add_exact(float &hi, float &lo, float x) {
    const float s = __fadd_rn(hi, x), y = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, y)), __fsub_rn(x, y)));
    hi = s;
}

// The path of nodes `lane` and `lane + 32` (bit u: node u is on it), by a whole warp: each node knows the part of
// its path below some ancestor, and takes over what that one knows, so that the part doubles every step.
struct Paths {
    uint32_t lo[2], hi[2];  // of node lane: lo[0], hi[0] (nodes 0..31 and 32..63 on its path); of lane + 32: [1]
    __device__ __forceinline__ uint64_t of(int i) const { return (uint64_t)hi[i] << 32 | lo[i]; }
    // of any node, which may differ by lane (all lanes call)
    __device__ __forceinline__ uint64_t at(int node) const {
        const int src = node & 31;
        const uint32_t l0 = __shfl_sync(0xffffffffu, lo[0], src), l1 = __shfl_sync(0xffffffffu, lo[1], src);
        const uint32_t h1 = __shfl_sync(0xffffffffu, hi[1], src);
        return node & 32 ? (uint64_t)h1 << 32 | l1 : l0;  // (a node below 32 has none of 32.. on its path)
    }
};
// SUMS: hi + lo, at first a value of each of the two nodes, become the sums over the paths (0 over an empty one).
// SECOND: whether there are nodes from 32 on.
template <bool SUMS = false, bool SECOND = true>
__device__ __forceinline__ Paths tree_paths(int up0, int up1, int *status, float *hi = nullptr, float *lo = nullptr) {
    const int lane = threadIdx.x & 31;
    Paths p;
    int up[2] = {up0, SECOND ? up1 : -2};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = lane + 32 * i;
        if (up[i] >= t) {  // no parent of its own
            flag_error(status);
            up[i] = -2;
        }
        p.lo[i] = i == 0 ? 1u << lane : 0u;
        p.hi[i] = i == 0 ? 0u : 1u << lane;
    }
    while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
        const uint32_t was_lo[2] = {p.lo[0], p.lo[1]}, was_hi = p.hi[1];
        const int was_up[2] = {up[0], up[1]};
        float was[2][2];
        if constexpr (SUMS) was[0][0] = hi[0], was[0][1] = hi[1], was[1][0] = lo[0], was[1][1] = lo[1];
#pragma unroll
        for (int i = 0; i < (SECOND ? 2 : 1); ++i) {
            // what its ancestor knows: a node below 32, for those from 32 on of either half
            const int src = up[i] & 31;
            const bool second = i == 1 && (up[i] & 32);
            uint32_t l = __shfl_sync(0xffffffffu, was_lo[0], src), h = 0u;
            int next = __shfl_sync(0xffffffffu, was_up[0], src);
            float s = 0.f, r = 0.f;
            if constexpr (SUMS) {
                s = __shfl_sync(0xffffffffu, was[0][0], src);
                r = __shfl_sync(0xffffffffu, was[1][0], src);
            }
            if (i == 1) {
                const uint32_t l1 = __shfl_sync(0xffffffffu, was_lo[1], src), h1 = __shfl_sync(0xffffffffu, was_hi, src);
                const int next1 = __shfl_sync(0xffffffffu, was_up[1], src);
                l = second ? l1 : l;
                h = second ? h1 : 0u;
                next = second ? next1 : next;
                if constexpr (SUMS) {
                    const float s1 = __shfl_sync(0xffffffffu, was[0][1], src), r1 = __shfl_sync(0xffffffffu, was[1][1], src);
                    s = second ? s1 : s;
                    r = second ? r1 : r;
                }
            }
            if (up[i] >= 0) {
                p.lo[i] |= l;
                p.hi[i] |= h;
                up[i] = next;
                if constexpr (SUMS) {
                    add_exact(hi[i], lo[i], s);
                    lo[i] += r;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (up[i] != -1) {
            p.lo[i] = p.hi[i] = 0u;
            if constexpr (SUMS) hi[i] = lo[i] = 0.f;
        }
    return p;
}

__device__ __forceinline__ Paths tree_paths(const int32_t *parents, int nodes, int *status) {
    const int lane = threadIdx.x & 31;
    return tree_paths(lane < nodes ? parents[lane] : -2, lane + 32 < nodes ? parents[lane + 32] : -2, status);
}

// Whether a row with this path sees the position of node `i` of its sequence (below 0: the context, which all see)
__device__ __forceinline__ bool on_path(uint64_t path, int i) { return i < 0 || (i < kTreeMax && ((path >> i) & 1)); }

// ... of 64 positions at once, the first of which is that of node `first`
__device__ __forceinline__ uint64_t path_window(uint64_t path, int first) {
    if (first >= 0) return first < kTreeMax ? path >> first : 0;
    return first <= -kTreeMax ? ~0ull : path << -first | ((1ull << -first) - 1);
}

// The path of one node, by one thread (for what is rare)
static __device__ __noinline__ uint64_t path_of(const int32_t *parents, int t) {
    uint64_t path = 0;
    while (t >= 0) {
        path |= 1ull << t;
        const int up = parents[t];
        if (up >= t) return 0;
        t = up;
    }
    return t == -1 ? path : 0;
}

// Pool entry of sequence n; -1 for padding (flagged if it names none)
__device__ __forceinline__ long state_slot(const TreeArgs &a, int n) {
    if (a.slots == nullptr) return n;
    const long s = a.slots[n];
    if (s >= a.num_slots) flag_error(a.status);
    return s < 0 || s >= a.num_slots ? -1 : s;
}

}  // namespace gdn
