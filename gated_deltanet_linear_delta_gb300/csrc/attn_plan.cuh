// attn_plan.cuh -- how the attention over a paged cache is cut into work, and the join of split
// rows' parts.
//
// A unit is (sequence n, key head h, row tile i): the query heads that share h of TPT consecutive
// new tokens, TPT * G rows, walked over key tiles of BN positions up to the last one any of its
// rows sees. Units have very different lengths (one token over 100 or over 100,000 positions), and
// the host does not know them (kv_lens is device data, and a captured graph replays with others),
// so the cut is made on the device: all units' key tiles form one line, in the order n, h, i, and
// each of at most kAttnCtas CTAs takes an equal piece of it. A CTA thus finishes some units alone
// and shares at most two with its neighbours; of those it leaves the unnormalised output, the
// running maximum and the sum in the workspace, and the joining kernel combines them. Every CTA
// finds its piece from kv_lens alone: no counters, no atomics, and the same order of sums each time.
#pragma once

#include "kv_pages.cuh"

namespace gdn {

// The line of `total` key tiles as `active` pieces whose sizes differ by one at most: piece c begins
// at c q + min(c, r).
struct Cut {
    long q;
    int r, active;
    __device__ __forceinline__ long begin(int c) const { return c * q + min(c, r); }
    __device__ __forceinline__ int piece_of(long tile) const {  // the piece that holds a tile
        const long wide = r * (q + 1);
        if (tile < wide) return (int)div(tile, q + 1);
        return r + (int)div(tile - wide, q);
    }
    // a 64-bit division takes hundreds of cycles; nearly all of these fit 32 bits
    __device__ __forceinline__ static long div(long a, long b) {
        if ((a | b) >> 31) return a / b;
        return (long)((uint32_t)a / (uint32_t)b);
    }
};

struct __align__(16) AttnRec {  // where CTA c's piece starts; read by the joining kernel
    Cut cut;       // the same in every record
    long begin;    // key tiles of all units before the piece
    int off;       // key tiles of the unit before the piece (0: the unit starts here)
    int ntiles;    // key tiles of the unit
    long token;    // packed token of the unit's first row
    int tokens;    // its new tokens
    int pos;       // position of the first (negative: padding)
    int h;         // key head of the unit
};

struct AttnWork {
    KvPages pg;
    const int32_t *parents;  // new tokens that form trees: their parents; else null
    int G;         // query heads per key head
    int TPT;       // tokens per row tile
    int rows;      // workspace rows per part
    int min_shift; // a piece is not cut below 2^min_shift tiles
    AttnRec *rec;  // [kAttnCtas]
    float2 *ml;    // [kAttnCtas][2][rows] running maximum (log2 domain) and sum
    float *part;   // [kAttnCtas][2][rows][d]
};

// part of CTA c: 0 = it continues a unit begun before, 1 = it begins a unit that goes on after it
__device__ __forceinline__ long part_index(const AttnWork &w, int c, int slot, int row) {
    return ((long)c * 2 + slot) * w.rows + row;
}

// key tiles of row tile i of a sequence
template <int BN>
__device__ __forceinline__ int unit_tiles(const AttnWork &w, const SeqInfo &s, int i) {
    const int t = min(s.T, (i + 1) * w.TPT);  // tokens up to the tile's last
    const int keys = s.len - s.T + t;
    return keys > 0 ? (keys + BN - 1) / BN : 0;
}
__device__ __forceinline__ int row_tiles(const AttnWork &w, const SeqInfo &s) { return (s.T + w.TPT - 1) / w.TPT; }

// Key tiles of all row tiles of one head, of the sequence that each thread holds; a warp works
// together on sequences of many row tiles.
template <int BN>
__device__ __forceinline__ long seq_tiles(const AttnWork &w, const SeqInfo &s) {
    const int lane = threadIdx.x & 31, nq = row_tiles(w, s);
    long sum = 0;
    const bool big = nq > 4;
    if (!big)
        for (int i = 0; i < nq; ++i) sum += unit_tiles<BN>(w, s, i);
    for (unsigned m = __ballot_sync(0xffffffffu, big); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        SeqInfo o;
        o.bos = 0;
        o.T = __shfl_sync(0xffffffffu, s.T, src);
        o.len = __shfl_sync(0xffffffffu, s.len, src);
        const int onq = __shfl_sync(0xffffffffu, nq, src);
        long x = 0;
        for (int i = lane; i < onq; i += 32) x += unit_tiles<BN>(w, o, i);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane == src) sum = x;
    }
    return sum;
}

// A CTA's piece and the unit it is at.
struct Piece {
    int n, h, i;     // unit
    int nq;          // row tiles of the sequence
    int off;         // its next key tile
    int ntiles;      // its key tiles
    long left;       // key tiles left in the piece
    SeqInfo s;
};

struct PlanSmem {
    long sum[32];
    int found;
    int padding;  // some sequence has more new tokens than positions
    Piece piece;
};

// Finds this CTA's piece; every thread of the CTA calls it (NT threads, a multiple of 32, at most
// 1024). The result is in sm->piece (left = 0: no work), and its record in the workspace. It stands
// before all other work of the call, so it is kept short: one pass over the sequences (a second
// where there are more than NT), two or three barriers, 32-bit divisions.
template <int BN, int NT, bool TREE = false>
__device__ void plan_piece(const AttnWork &w, PlanSmem *sm) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    constexpr int NW = NT / 32;
    const KvPages &p = w.pg;
    const bool one_pass = p.B <= NT;
    long mine = 0, per_head = 0;  // key tiles of this thread's sequences; of one head of the last of them
    SeqInfo s0{0, 0, 0};
    bool pad = false;
    for (int base = 0; base < p.B; base += NT) {
        SeqInfo s{0, 0, 0};
        if (base + tid < p.B) seq_info<TREE>(p, base + tid, &s);
        pad |= s.T > s.len;
        per_head = seq_tiles<BN>(w, s);
        mine += per_head * p.Hkv;
        s0 = s;
    }
    auto scan = [&](long y) {  // inclusive, over the warp
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long o = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += o;
        }
        return y;
    };
    long inc = scan(mine);
    if (lane == 31) sm->sum[wid] = inc;
    if (tid == 0) sm->found = -1;
    const int any_pad = __syncthreads_or(pad);
    if (tid == 0) sm->padding = any_pad;
    long total = 0, pre = inc - mine;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
        if (k < wid) pre += sm->sum[k];
        total += sm->sum[k];
    }
    const long want = (total + (1 << w.min_shift) - 1) >> w.min_shift;
    Cut cut;
    cut.active = (int)(want < (long)gridDim.x ? want : (long)gridDim.x);
    cut.q = cut.active ? Cut::div(total, cut.active) : 0;
    cut.r = (int)(total - cut.q * cut.active);
    const int c = blockIdx.x;
    const long begin = c < cut.active ? cut.begin(c) : total, end = c < cut.active ? cut.begin(c + 1) : total;
    auto own = [&](int n) {  // this thread's sequence holds `begin`: head, and row tile if there are few
        Piece pc;
        long rem = begin - pre;
        pc.n = n;
        pc.s = s0;
        pc.h = (int)Cut::div(rem, per_head);
        rem -= pc.h * per_head;
        pc.i = 0;
        pc.ntiles = unit_tiles<BN>(w, s0, 0);
        const int nq = row_tiles(w, s0);
        pc.nq = nq;
        if (nq <= 4) {
            while (rem >= pc.ntiles) {
                rem -= pc.ntiles;
                pc.ntiles = unit_tiles<BN>(w, s0, ++pc.i);
            }
        } else {
            pc.i = -1;
        }
        pc.off = (int)rem;  // (below 2^31: a head's tiles; checked below where there are many row tiles)
        pc.left = rem;
        sm->piece = pc;
        sm->found = n;
    };
    if (one_pass) {
        if (begin < end && begin >= pre && begin < pre + mine) own(tid);
        __syncthreads();
    } else {
        long before = 0;
        __syncthreads();
        for (int base = 0; base < p.B && begin < end; base += NT) {
            s0 = SeqInfo{0, 0, 0};
            if (base + tid < p.B) seq_info<TREE>(p, base + tid, &s0);
            per_head = seq_tiles<BN>(w, s0);
            const long y = per_head * p.Hkv;
            inc = scan(y);
            if (lane == 31) sm->sum[wid] = inc;
            __syncthreads();
            pre = before + inc - y;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                if (k < wid) pre += sm->sum[k];
                before += sm->sum[k];
            }
            if (begin >= pre && begin < pre + y) own(base + tid);
            __syncthreads();
            if (sm->found >= 0) break;
        }
    }
    const bool work = begin < end && sm->found >= 0;  // (not found: only if kv_lens changed under the call)
    if (work && sm->piece.i < 0) {  // many row tiles: a warp walks over them, 32 at a time
        __syncthreads();
        if (wid == 0) {
            Piece pc = sm->piece;
            const int nq = row_tiles(w, pc.s);
            long rem = pc.left;
            for (int i0 = 0; i0 < nq; i0 += 32) {
                const int t = i0 + lane < nq ? unit_tiles<BN>(w, pc.s, i0 + lane) : 0;
                long sum = scan(t);
                const long chunk = __shfl_sync(0xffffffffu, sum, 31);
                if (rem < chunk) {
                    const unsigned m = __ballot_sync(0xffffffffu, rem < sum);
                    const int src = __ffs(m) - 1;
                    pc.i = i0 + src;
                    pc.ntiles = __shfl_sync(0xffffffffu, t, src);
                    pc.off = (int)(rem - (__shfl_sync(0xffffffffu, sum, src) - pc.ntiles));
                    break;
                }
                rem -= chunk;
            }
            __syncwarp();
            if (lane == 0) sm->piece = pc;
        }
        __syncthreads();
    }
    if (tid == 0) {
        AttnRec r{cut, begin, 0, 0, 0, 0, 0, 0};
        if (work) {
            const Piece &pc = sm->piece;
            const int t0 = pc.i * w.TPT;
            r.off = pc.off;
            r.ntiles = pc.ntiles;
            r.token = pc.s.bos + t0;
            r.tokens = min(w.TPT, pc.s.T - t0);
            r.pos = pc.s.len - pc.s.T + t0;
            r.h = pc.h;
            sm->piece.left = end - begin;
        } else {
            sm->piece = Piece{};
        }
        w.rec[c] = r;
    }
    __syncthreads();
}

// The unit after the piece's current one that has any key tiles (left > 0 says there is one). All warps
// of a CTA take this step, between two units' work, so it divides only where the sequence changes (a
// division per step made it 1500 cycles).
template <int BN, bool TREE = false>
__device__ __forceinline__ void next_unit(const AttnWork &w, Piece *pc) {
    pc->off = 0;
    do {
        if (++pc->i >= pc->nq) {
            pc->i = 0;
            if (++pc->h >= w.pg.Hkv) {
                pc->h = 0;
                if (++pc->n >= w.pg.B) {  // kv_lens changed under the call: stop instead of running off
                    pc->left = 0;
                    return;
                }
                seq_info<TREE>(w.pg, pc->n, &pc->s);  // no tokens where cu is inconsistent
                pc->nq = row_tiles(w, pc->s);
            }
        }
        pc->ntiles = pc->i < pc->nq ? unit_tiles<BN>(w, pc->s, pc->i) : 0;
    } while (pc->ntiles == 0);
}

// Rows of padding tokens are zeros; no unit of work covers them. (`threads` threads of each CTA call
// it, if the plan has found any.)
template <bool TREE = false, typename TOut>
__device__ void zero_padding(const AttnWork &w, TOut *out, int Hq, int d, int thread, int threads) {
    for (int n = blockIdx.x; n < w.pg.B; n += gridDim.x) {
        SeqInfo s;
        if (!seq_info<TREE>(w.pg, n, &s)) continue;
        const long idle = (long)min(s.T, max(0, s.T - s.len)) * Hq * d;
        uint4 *p = reinterpret_cast<uint4 *>(out + s.bos * Hq * d);
        const long pieces = idle * (long)sizeof(TOut) / 16;
        for (long e = thread; e < pieces; e += threads) p[e] = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace gdn
