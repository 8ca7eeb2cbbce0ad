// tree_mma.cuh -- what the tensor-core kernels of the gated delta rule over trees share: m16n8k16 products of bf16
// (mma.sync), their operands from shared memory, and fp32 values split into bf16 terms.
#pragma once

#include "attn_ops.cuh"

namespace gdn {

// ---- products ----------------------------------------------------------------------
// Lane (g = lane / 4, c = lane % 4): D and C hold rows g and g + 8, columns 2 c and 2 c + 1, as {g 2c, g 2c+1, g+8 2c,
// g+8 2c+1}; A the same of both halves of its 16 columns; B rows 2 c .. and 2 c + 8 .. of column g.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// four 8 x 8 matrices whose rows are 16 bytes at the lanes' addresses (lanes 0..7 the first's, 8..15 the second's, ..)
__device__ __forceinline__ void load_matrices(uint32_t (&x)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}
// A pair of fp32 as bf16, and what that leaves of them
__device__ __forceinline__ uint32_t split2(float &x, float &y) {
    const uint32_t h = tc::bf2_bits(__floats2bfloat162_rn(x, y));
    x -= __uint_as_float(h << 16);
    y -= __uint_as_float(h & 0xffff0000u);
    return h;
}

// ---- layouts in shared memory: where the 16 bytes `ch` of row r lie (as the tensor maps' swizzles put them) ----
// rows of DK bf16, in blocks of 64 columns of ROWS rows; the 8 rows of a matrix lie in different banks
template <int DK, int ROWS>
__device__ __forceinline__ uint32_t row_piece(int r, int ch) {
    if (DK >= 64) return (uint32_t)((ch >> 3) * (ROWS * 128) + r * 128 + (((ch ^ r) & 7) << 4));
    return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4));
}
// 32 columns of a state, rows of 128 bytes: 32 bytes of 4 rows 2 apart lie in different banks
__device__ __forceinline__ uint32_t state_piece(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }
// ---- coefficients between nodes: row t, columns s (a multiple of 4: 16 bytes of fp32, or 8 bytes of each bf16 term) -------
// Blocks (i, j <= i) of 16 x 16, 64 bytes a row: for ldmatrix. Rows spread as above.
struct CoefBlocks {
    uint8_t *base;
    __device__ __forceinline__ static uint32_t piece(int r, int ch) { return (uint32_t)(r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)); }
    __device__ __forceinline__ static uint32_t block(int i, int j) { return (uint32_t)((i * (i + 1) / 2 + j) * 1024); }
    __device__ __forceinline__ float *raw(int t, int s) const {
        return reinterpret_cast<float *>(base + block(t >> 4, s >> 4) + piece(t & 15, (s & 15) >> 2));
    }
    // 4 upper and 4 lower terms, within the row's own 64 bytes of the block
    __device__ __forceinline__ void store(int t, int s, uint2 up, uint2 low) const {
        uint8_t *at = base + block(t >> 4, s >> 4);
        const int ch = (s & 15) >> 3, half = 8 * ((s >> 2) & 1);
        *reinterpret_cast<uint2 *>(at + piece(t & 15, ch) + half) = up;
        *reinterpret_cast<uint2 *>(at + piece(t & 15, 2 + ch) + half) = low;
    }
    static constexpr bool kWhole = false, kPlain = false;  // blocks above the diagonal do not exist
};
// Rows of 128 bytes, 128B swizzle: TP rows of upper terms, then TP of lower ones (a tcgen05 operand); as fp32 a row fills both.
template <int TP>
struct CoefRows {
    uint8_t *base;
    __device__ __forceinline__ static uint32_t piece(int r, int ch) { return (uint32_t)(r * 128 + ((ch ^ (r & 7)) << 4)); }
    __device__ __forceinline__ float *raw(int t, int s) const {
        return reinterpret_cast<float *>(base + (s >> 5) * (TP * 128) + piece(t, (s & 31) >> 2));
    }
    __device__ __forceinline__ void store(int t, int s, uint2 up, uint2 low) const {
        uint8_t *at = base + piece(t, s >> 3) + 8 * ((s >> 2) & 1);
        *reinterpret_cast<uint2 *>(at) = up;
        *reinterpret_cast<uint2 *>(at + TP * 128) = low;
    }
    static constexpr bool kWhole = true, kPlain = false;
};
// fp32 throughout, rows of 64 and 4 more, so that the same columns of 8 rows lie in different banks
struct CoefPlain {
    float *base;
    static constexpr int kRow = kTreeMax + 4;
    __device__ __forceinline__ float *raw(int t, int s) const { return base + t * kRow + s; }
    static constexpr bool kWhole = false, kPlain = true;
};

// ---- the nodes of a head ---------------------------------------------------------------------------
// A gate below this counts as it: nothing of what lies above the node is left either way, and what lies below takes its decays
// from differences of sums, which keep their precision (-infinity's would have none, nor those of a type's lowest value).
constexpr float kNoGate = -1e6f;

template <int TP>
struct __align__(16) Scalars {   // of each node (four nodes' are one access)
    float beta[TP], x[TP];       // beta;  beta e^G rk, the factor of X_k
    float z[TP];                 // e^G rq, the factor of X_q
    float rq[TP], b2[TP];        // 1 / |q|;  beta rk^2
    float g[TP], g_lo[TP];       // G as a sum of two (bf16 inputs: its log2 e fold)
    float gk[TP];                // g_lo less the logarithm of 1 / |k|, to the same base
};

struct Head {
    int n, h, nodes;
    long bos, slot;
};

// Heads by turns over the CTAs; those of padding sequences are written as zeros on the way.
template <int DV, int THREADS>
struct Heads {
    int n, h, dn, dh;
    __device__ __forceinline__ explicit Heads(const TreeArgs &a)
        : n((int)(blockIdx.x / a.Hv)), h((int)(blockIdx.x % a.Hv)), dn((int)(gridDim.x / a.Hv)), dh((int)(gridDim.x % a.Hv)) {}
    __device__ __forceinline__ void step(const TreeArgs &a) {
        n += dn;
        if ((h += dh) >= a.Hv) {
            h -= a.Hv;
            ++n;
        }
    }
    // the first from the one at hand on that has nodes and a state (slot < 0: none)
    __device__ __forceinline__ Head find(const TreeArgs &a) {
        Head hd{0, 0, 0, 0, -1};
        for (; n < a.B; step(a)) {
            hd.n = n;
            hd.h = h;
            if (!tree_bounds(a.cu, n, a.B, a.cu ? a.Ttot : a.T, &hd.bos, &hd.nodes, a.status) || hd.nodes == 0) continue;
            hd.slot = state_slot(a, n);
            if (hd.slot >= 0) return hd;
            __nv_bfloat16 *out = (__nv_bfloat16 *)a.out;
            for (int e = threadIdx.x; e < hd.nodes * (DV / 8); e += THREADS)
                reinterpret_cast<uint4 *>(out + ((hd.bos + e / (DV / 8)) * a.Hv + h) * DV)[e % (DV / 8)] = make_uint4(0, 0, 0, 0);
        }
        hd.slot = -1;
        return hd;
    }
    __device__ __forceinline__ Head after(const TreeArgs &a, const Head &from) {
        if (from.slot < 0) return from;
        step(a);
        return find(a);
    }
};

// What a node's thread knows of it, a head ahead: the threads of warp W0, and for nodes from 32 on of W1.
template <int TP, int W0, int W1>
struct Nodes {
    int up = -2;
    float g = 0.f, b = 0.f;
    __device__ __forceinline__ static int node() {  // -1: none
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        return warp == W0 && lane < TP ? lane : TP > 32 && warp == W1 ? lane + 32 : -1;
    }
    __device__ __forceinline__ void load(const TreeArgs &a, const Head &hd) {
        up = -2;
        g = b = 0.f;
        const int t = node();
        if (hd.slot < 0 || t < 0 || t >= hd.nodes) return;
        up = a.parents[hd.bos + t];
        g = to_f32(((const __nv_bfloat16 *)a.g)[(hd.bos + t) * a.Hv + hd.h]);
        b = to_f32(((const __nv_bfloat16 *)a.b)[(hd.bos + t) * a.Hv + hd.h]);
    }
    // Paths, and the sums of g over them, by those warps; b becomes beta.
    __device__ __forceinline__ void sums(uint64_t *paths, Scalars<TP> &sc, int *status) {
        const int warp = threadIdx.x >> 5, t = node();
        if (warp != W0 && !(TP > 32 && warp == W1)) return;
        b = sigmoidf_(b);
        // g log2 e, whose second float is 1.926e-8
        float hi = __fmul_rn(g, kLog2e), lo = fmaf(g, 1.92596303e-8f, fmaf(g, kLog2e, -hi));
        if (hi < kNoGate) {
            hi = kNoGate;
            lo = 0.f;
        }
        uint64_t path;
        if constexpr (TP <= 32) {
            float his[2] = {hi, 0.f}, los[2] = {lo, 0.f};
            path = tree_paths<true, false>(up, -2, status, his, los).of(0);
            hi = his[0];
            lo = los[0];
        } else {
            // as tree_paths does it, through shared memory: what is known of each node, where the scalars are going to be
            // (two nodes to a thread of one warp, and shuffles, is twice the instructions on the slowest warp's way)
            static_assert(TP == 64 && offsetof(Scalars<TP>, b2) == 1024, "room for what is known");
            uint4 *known = reinterpret_cast<uint4 *>(&sc);  // path, parent of its last node, hi
            float *known_lo = sc.b2;
            if (up >= t) {  // no parent of its own
                flag_error(status);
                up = -2;
            }
            path = 1ull << t;
            while (true) {
                known[t] = make_uint4((uint32_t)path, (uint32_t)(path >> 32), (uint32_t)up, __float_as_uint(hi));
                known_lo[t] = lo;
                if (!tc::bar_any(1, 64, up >= 0)) break;
                if (up >= 0) {
                    const uint4 k = known[up];
                    const float l = known_lo[up];
                    path |= (uint64_t)k.y << 32 | k.x;
                    up = (int)k.z;
                    add_exact(hi, lo, __uint_as_float(k.w));
                    lo += l;
                }
                tc::bar_sync(1, 64);
            }
            if (up != -1) {
                path = 0;
                hi = lo = 0.f;
            }
        }
        if (t < 0) return;
        paths[t] = path;
        sc.g[t] = hi;
        sc.g_lo[t] = lo;
        sc.z[t] = ex2(hi + lo);
    }
    // ... and with the products' diagonals at hand, the rest
    __device__ __forceinline__ void finish(int T, const CoefBlocks &kk, const float *qq, Scalars<TP> &sc) const {
        const int t = node();
        if (t < 0) return;
        float4 *row = reinterpret_cast<float4 *>(kk.raw(t, t & ~3));
        const float4 x = *row;
        const int e = t & 3;
        const float k2 = t >= T ? 0.f : e == 0 ? x.x : e == 1 ? x.y : e == 2 ? x.z : x.w;
        *row = make_float4(e > 0 ? x.x : 0.f, e > 1 ? x.y : 0.f, e > 2 ? x.z : 0.f, 0.f);  // (what follows in its block is 0)
        const float eg = sc.z[t], beta = b;
        const float rk = rsqrtf(k2 + kNormEps), rq = rsqrtf(qq[t] + kNormEps);
        sc.beta[t] = beta;
        sc.x[t] = beta * eg * rk;
        sc.z[t] = eg * rq;
        sc.gk[t] = sc.g_lo[t] - __log2f(rk);
        sc.rq[t] = rq;
        sc.b2[t] = beta * rk * rk;
    }
};

// K K^T into kk (zeros in the fours of a row past the diagonal's), Q K^T into w, block by block of 16 x 16, and |q|^2 into
// qq. K's rows are 0 .. of the tile at shared address kq, Q's TP .. . Warps take blocks from the counter `unit`, so that
// those which are late take fewer.
template <int DK, int TP, typename W>
__device__ __forceinline__ void node_products(uint32_t kq, int nb, int *unit, const CoefBlocks &kk, const W &w, float *qq) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    while (true) {
        int u = 0;
        if (lane == 0) u = atomicAdd(unit, 1);
        u = __shfl_sync(0xffffffffu, u, 0);
        if (u >= nb * (nb + 2)) break;
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
            load_matrices(x, kq + row_piece<DK, 2 * TP>(ra, 2 * ks + (lane >> 4)));
            load_matrices(y, kq + row_piece<DK, 2 * TP>(rb, 2 * ks + ((lane >> 3) & 1)));
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
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int t = 16 * i + g + 8 * half, s = 16 * j + 8 * n + 4 * (c >> 1);
                float *to = (is_q ? w.raw(t, s) : kk.raw(t, s)) + 2 * (c & 1);
                const bool past = !is_q && s > t;
                *reinterpret_cast<float2 *>(to) = past ? make_float2(0.f, 0.f) : make_float2(acc[n][2 * half], acc[n][2 * half + 1]);
            }
    }
}

// Q K^T in wt becomes W, as two bf16 terms. kk: K K^T, with zeros from the diagonal on in the blocks that it goes through. A
// row by four lanes: lane `sub` holds columns 16 j + 4 sub .. + 3.
// (kPlain: as fp32.)
template <int TP, int THREADS, typename KT, typename WT>
__device__ __forceinline__ void form_w(int T, const uint64_t *paths, const Scalars<TP> &sc, const KT &kk, const WT &wt) {
    constexpr int NB = TP / 16;
    const int lane = threadIdx.x & 31, sub = lane & 3, nb = (T + 15) / 16;
    for (int t = (int)threadIdx.x >> 2; t < 16 * nb; t += THREADS / 4) {
        const uint64_t on = t < T ? paths[t] : 0;
        const float rq = sc.rq[t], g = sc.g[t], g_lo = sc.g_lo[t];
        float w[NB][4];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const float4 x = j <= t >> 4 ? *reinterpret_cast<const float4 *>(wt.raw(t, 16 * j + 4 * sub))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
            w[j][0] = rq * x.x; w[j][1] = rq * x.y; w[j][2] = rq * x.z; w[j][3] = rq * x.w;
        }
#pragma unroll
        for (int j = NB - 1; j >= 0; --j) {
            uint32_t left = (uint32_t)(on >> (16 * j)) & 0xffffu;
            // (the warp's eight rows step together, each along its own path: rows that part ways would run one by one)
            const int steps = (int)__reduce_max_sync(0xffffffffu, (unsigned)__popc(left));
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                const int s = 31 - __clz(left | 1);  // of the block's nodes; w_s is final
                const float own = s & 2 ? (s & 1 ? w[j][3] : w[j][2]) : (s & 1 ? w[j][1] : w[j][0]);
                const float ws = -__shfl_sync(0xffffffffu, own, (lane & ~3) | (s >> 2)) * sc.b2[16 * j + s];
                if (left != 0) {
                    left ^= 1u << s;
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        if (i > j) continue;
                        const float4 x = *reinterpret_cast<const float4 *>(kk.raw(16 * j + s, 16 * i + 4 * sub));
                        w[i][0] = fmaf(ws, x.x, w[i][0]);  // (0 from s on)
                        w[i][1] = fmaf(ws, x.y, w[i][1]);
                        w[i][2] = fmaf(ws, x.z, w[i][2]);
                        w[i][3] = fmaf(ws, x.w, w[i][3]);
                    }
                }
            }
        }
        __syncwarp();  // the row has been read by all of its lanes
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            if (j > t >> 4) {  // (the same for the whole warp)
                if constexpr (WT::kWhole) wt.store(t, 16 * j + 4 * sub, make_uint2(0u, 0u), make_uint2(0u, 0u));
                continue;
            }
            const uint32_t mine = (uint32_t)(on >> (16 * j)) >> (4 * sub);
            const float4 sg = load4(sc.g + 16 * j + 4 * sub), sl = load4(sc.gk + 16 * j + 4 * sub);
            // (by masks: selects became branches, which took as long as all steps above)
            auto masked = [&](float x, float gs, float ls, int i) {
                const float d = (g - gs) + (g_lo - ls);
                return __uint_as_float(__float_as_uint(x * (WT::kPlain ? expf(d) : ex2(d))) & (0u - (mine >> i & 1u)));
            };
            w[j][0] = masked(w[j][0], sg.x, sl.x, 0);
            w[j][1] = masked(w[j][1], sg.y, sl.y, 1);
            w[j][2] = masked(w[j][2], sg.z, sl.z, 2);
            w[j][3] = masked(w[j][3], sg.w, sl.w, 3);
            if constexpr (WT::kPlain) {
                *reinterpret_cast<float4 *>(wt.raw(t, 16 * j + 4 * sub)) = make_float4(w[j][0], w[j][1], w[j][2], w[j][3]);
            } else {
                uint2 up, low;
                up.x = split2(w[j][0], w[j][1]);
                up.y = split2(w[j][2], w[j][3]);
                low.x = tc::bf2_bits(__floats2bfloat162_rn(w[j][0], w[j][1]));
                low.y = tc::bf2_bits(__floats2bfloat162_rn(w[j][2], w[j][3]));
                wt.store(t, 16 * j + 4 * sub, up, low);
            }
        }
    }
}

// x [outer][mid][inner] -> boxes of box_inner columns and rows along one of the other dimensions, swizzled over their bytes
inline bool scan_map(CUtensorMap *m, const void *base, bool f32, int inner, long mid, long outer, int box_inner, int box_mid,
                     int box_outer) {
    EncodeTiledFn enc = tiled_encoder();
    if (!enc) return false;
    const cuuint64_t elem = f32 ? 4 : 2, bytes = box_inner * elem;
    const cuuint64_t gdim[3] = {(cuuint64_t)inner, (cuuint64_t)mid, (cuuint64_t)outer};
    const cuuint64_t gstride[2] = {inner * elem, (cuuint64_t)mid * inner * elem};
    const cuuint32_t box[3] = {(cuuint32_t)box_inner, (cuuint32_t)box_mid, (cuuint32_t)box_outer};
    const cuuint32_t estride[3] = {1, 1, 1};
    return enc(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), gdim,
               gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
               bytes == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
               : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                             : CU_TENSOR_MAP_SWIZZLE_NONE,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace gdn
