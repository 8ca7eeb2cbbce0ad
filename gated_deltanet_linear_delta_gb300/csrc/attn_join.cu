// attn_join.cu -- the parts of units that were split between CTAs become output rows.
//
// Part p of a row holds O_p = sum_j exp2(s_j - m_p) v_j, m_p and l_p = sum_j exp2(s_j - m_p) over
// its keys; the row is (sum_p e^{m_p - m} O_p) / (sum_p e^{m_p - m} l_p), m = max_p m_p (base 2). (The
// factors of l_p are taken in two halves: with an 8-bit cache, whose value scales are in m_p and l_p, they
// may be smaller than a float and l_p as much larger.)
//
// A split unit is joined once, by the blocks of the first boundary between pieces that lies in
// it. Each row takes a team of 1, 2, 4 or 8 warps, as many as leave all of a unit's rows with the
// blocks at once and have two to four parts each, which a warp loads side by side. With few rows that is a block: its warps share the parts (one session's single
// token over a long cache has about 75 parts, and they should be in flight together) and add up
// through shared memory in a fixed order. With 128 rows it is one warp, without any meeting: prompts
// leave two or three parts a row, and a block for each took 37 us of their 143 us (8 prompts of 1024
// tokens, 32 heads, d = 128). Blocks whose boundary lies between units have nothing to do.
// The kernel is launched so that it may become resident while the attention kernel runs, and
// waits for it here, which hides its launch.
#include "attn_plan.cuh"
#include "attn_work.h"

namespace gdn {
namespace {

constexpr int kJoinThreads = 256;

__device__ __forceinline__ void store2(__nv_bfloat16 *to, float x, float y) {
    *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void store2(float *to, float x, float y) { *reinterpret_cast<float2 *>(to) = make_float2(x, y); }

// exp2(x) in two halves, for a factor of l; CODES: 8-bit caches of bf16 inputs
template <bool CODES>
struct Factor {
    float h;
    __device__ __forceinline__ explicit Factor(float x) : h(exp2f(CODES ? 0.5f * x : x)) {}
    __device__ __forceinline__ float of(float l) const { return CODES ? l * h * h : l * h; }
    __device__ __forceinline__ float whole() const { return CODES ? h * h : h; }
};

template <typename TOut, int D, bool CODES>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnWork w, TOut *out, int Hq) {
    constexpr int E = D / 32, NW = kJoinThreads / 32;
    __shared__ float acc[NW][D];
    __shared__ float2 ml[NW];
    before_reading();
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const AttnRec r = w.rec[c];
    if (c >= r.cut.active || r.off == 0) return;
    if (r.begin - r.off < r.cut.begin(c - 1)) return;  // an earlier boundary lies in this unit too
    const int last = r.cut.piece_of(r.begin - r.off + r.ntiles - 1);  // the piece that holds the unit's last key tile
    const int parts = last - c + 2, rows = r.tokens * w.G;
    int team = NW;
    while (team > 1 && (rows * team > (int)gridDim.y * NW || parts <= 2 * team)) team >>= 1;
    const int per_block = NW / team, sub = wid % team;
    for (int base = blockIdx.y * per_block; base < rows; base += gridDim.y * per_block) {
        const int row = base + wid / team, t = row / w.G;
        const bool live = row < rows && r.pos + t >= 0;  // the rows of padding tokens are written elsewhere
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int k0 = sub; live && k0 < parts; k0 += 4 * team) {
            float2 pm[4];
            float x[4][E];
#pragma unroll
            for (int u = 0; u < 4; ++u) {  // four parts' loads in flight
                const int k = k0 + u * team;
                pm[u] = make_float2(-INFINITY, 0.f);
                if (k >= parts) continue;
                const long at = part_index(w, c - 1 + k, k == 0 ? 1 : 0, row);
                pm[u] = w.ml[at];
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 f = *reinterpret_cast<const float2 *>(w.part + at * D + e * 32 + 2 * lane);
                    x[u][e] = f.x;
                    x[u][e + 1] = f.y;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (pm[u].x == -INFINITY && pm[u].y == 0.f) continue;  // no key of this part is seen by the row
                const float mn = fmaxf(m, pm[u].x);
                const Factor<CODES> fa(m - mn), fb(pm[u].x - mn);
                const float a = fa.whole(), b = fb.whole();
                m = mn;
                l = fa.of(l) + fb.of(pm[u].y);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = o[e] * a + x[u][e] * b;
            }
        }
        TOut *to = out + ((r.token + t) * Hq + r.h * w.G + row % w.G) * D;
        if (team == 1) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (live)
#pragma unroll
                for (int e = 0; e < E; e += 2) store2(to + e * 32 + 2 * lane, o[e] * inv, o[e + 1] * inv);
            continue;
        }
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<float2 *>(&acc[wid][e * 32 + 2 * lane]) = make_float2(o[e], o[e + 1]);
        if (lane == 0) ml[wid] = make_float2(m, l);
        __syncthreads();
        const int first = wid - sub;  // the team's warps
        float M = -INFINITY, L = 0.f, f[NW];
        for (int k = 0; k < team; ++k) M = fmaxf(M, ml[first + k].x);
        if (M == -INFINITY) M = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const Factor<CODES> fk(k < team ? ml[first + k].x - M : -INFINITY);
            f[k] = fk.whole();
            if (k < team) L += fk.of(ml[first + k].y);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        if (live)
            for (int e = sub * 32 + lane; e < D; e += team * 32) {
                float x = 0.f;
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    if (k < team) x += f[k] * acc[first + k][e];
                to[e] = from_f32<TOut>(x * inv);
            }
        __syncthreads();
    }
}

template <typename TOut, int D, bool CODES = false>
cudaError_t launch_t(const AttnWork &w, TOut *out, int Hq, int rows, int ctas, cudaStream_t s) {
    // (4 rows a block, one after another: one long session's 8 rows took 45 us instead of 41 us in all)
    const dim3 grid((unsigned)ctas - 1, (unsigned)(rows < 16 ? rows : 16), 1);
    return launch_early(attn_join_kernel<TOut, D, CODES>, grid, kJoinThreads, 0, s, w, out, Hq);
}

}  // namespace

cudaError_t launch_attn_join(const AttnArgs &a, const AttnWork &w, int ctas, cudaStream_t s) {
    if (ctas <= 1) return cudaSuccess;  // one piece: nothing is split
    const bool f32 = a.pg.dtype == GDN_F32, codes = a.pg.cache_dtype != a.pg.dtype;
    const int rows = w.rows < w.TPT * w.G ? w.rows : w.TPT * w.G;
#define GDN_JOIN_CASE(DV)                                                                      \
    case DV:                                                                                   \
        return f32     ? launch_t<float, DV>(w, (float *)a.out, a.Hq, rows, ctas, s)                 \
               : codes ? launch_t<__nv_bfloat16, DV, true>(w, (__nv_bfloat16 *)a.out, a.Hq, rows, ctas, s) \
                       : launch_t<__nv_bfloat16, DV>(w, (__nv_bfloat16 *)a.out, a.Hq, rows, ctas, s);
    switch (a.pg.d) { GDN_JOIN_CASE(64) GDN_JOIN_CASE(128) GDN_JOIN_CASE(256) }
#undef GDN_JOIN_CASE
    return cudaErrorInvalidValue;
}

namespace {
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

int attn_unit_rows(long tokens_per_seq, int G) {
    const long rows = tokens_per_seq * G;
    return (int)(rows < kAttnMaxRows ? rows : kAttnMaxRows / G * G);
}

size_t attn_workspace(long tokens_per_seq, int G, int d) {
    const size_t parts = (size_t)kAttnCtas * 2 * attn_unit_rows(tokens_per_seq, G);
    return up256(kAttnCtas * sizeof(AttnRec)) + up256(parts * sizeof(float2)) + parts * d * sizeof(float);
}

// CTAs that can have a piece at all, going by what the host knows (the block table's width)
int attn_ctas(const AttnArgs &a, const AttnWork &w, int BN) {
    const long positions = (long)a.pg.max_pages * a.pg.page_size;
    const long units = (a.pg.cu ? a.pg.B + a.pg.Ttot / w.TPT : (long)a.pg.B * ((a.pg.T + w.TPT - 1) / w.TPT)) * a.pg.Hkv;
    const long tiles = (positions + BN - 1) / BN;
    const long pieces = units > kAttnCtas || tiles > kAttnCtas ? (long)kAttnCtas << w.min_shift : units * tiles;
    const long ctas = (pieces + (1 << w.min_shift) - 1) >> w.min_shift;
    return (int)(ctas < kAttnCtas ? ctas : kAttnCtas);
}

AttnWork attn_work(const AttnArgs &a, int tokens_per_tile, int min_shift) {
    AttnWork w{};
    w.pg = a.pg;
    w.parents = a.parents;
    w.G = a.Hq / a.pg.Hkv;
    w.TPT = tokens_per_tile;
    w.rows = attn_unit_rows(a.pg.cu ? a.pg.Ttot : a.pg.T, w.G);
    w.min_shift = min_shift;
    const size_t parts = (size_t)kAttnCtas * 2 * w.rows;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    w.rec = reinterpret_cast<AttnRec *>(ws);
    ws += up256(kAttnCtas * sizeof(AttnRec));
    w.ml = reinterpret_cast<float2 *>(ws);
    ws += up256(parts * sizeof(float2));
    w.part = reinterpret_cast<float *>(ws);
    return w;
}

}  // namespace gdn
