// What the attention kernels share: launch parameters, how the work is cut, and how the parts
// of a split sequence are joined.
//
// Work is counted in tiles of kTile consecutive visible positions of one (row, head group).
// A one-block prefix sum over the rows' lengths, which every block repeats (a row costs one
// word), numbers all tiles of the call; block c of C takes the tiles [T c / C, T (c + 1) / C).
// So ragged lengths balance without the host knowing them, and one long row spreads over every
// block.  A block's share is a run of segments, each a piece of one (row, head group).  A
// segment that is its (row, head group) whole is finished by its block; else the block leaves
// (max, sum, output) in its slot of the workspace, and the block that arrives last joins the
// parts in their order, so the result does not depend on timing.
//
// Visible positions are numbered 0 .. n-1 without gaps: the first `sinks`, then the window.
#pragma once

#include "decode_common.cuh"

namespace gs_decode {

constexpr int kTile = 64;                 // positions of a tile
constexpr int kWarps = 4;                 // warps of a block
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    CacheView c;
    int layer, batch;
    const int* seq;
    int q_heads, group;                   // query heads; of one kv head
    int parts, part;                      // head groups of a kv head; query heads of one
    const void* q;
    long long q_batch, q_head;
    const void* k_new;
    const void* v_new;
    long long new_batch, new_head;
    int new_aligned;
    float scale_log2;                     // scale * log2 e: scores are kept in powers of two
    int window, sinks;
    void* out;
    long long out_batch, out_head;
    float* lse;
    int* arrived;                         // [batch * heads * parts], 0 between calls
    float* slots;                         // [2 * blocks][part * (dim + 2)]
};

// A row's visible positions: j < sinks is position j, else position j + gap.
struct Row {
    int seq, n, sinks, gap, len;          // len: tokens of the sequence (0: nothing to read)
};

__device__ __forceinline__ Row row_of(const AttnParams& p, int b, unsigned* bad) {
    Row r;
    r.seq = p.seq != nullptr ? p.seq[b] : b;
    r.len = 0;
    if (r.seq < 0 || r.seq >= p.c.seqs) {
        *bad |= GS_DEV_BAD_SEQ;
        r.seq = 0;
    } else {
        r.len = p.c.lens[r.seq];
        const int most = p.c.cols * p.c.page;
        if (r.len < 0 || r.len > most) {
            *bad |= GS_DEV_BAD_SEQ;
            r.len = r.len < 0 ? 0 : most;
        }
    }
    r.n = r.len;
    r.sinks = 0;
    r.gap = 0;
    if (p.window > 0 && r.len > p.window) {
        const int first = r.len - p.window;
        r.sinks = p.sinks < first ? p.sinks : first;
        r.gap = first - r.sinks;
        r.n = r.sinks + p.window;
    }
    return r;
}

__device__ __forceinline__ int position(const Row& r, int j) {
    return j < r.sinks ? j : j + r.gap;
}

// at[b] = tiles of one head of the rows before b, for 0 <= b <= batch.  Ends with a barrier.
__device__ __forceinline__ void number_tiles(const AttnParams& p, int* at, int* tmp) {
    int carry = 0;
    unsigned bad = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        const int tiles = b < p.batch ? (row_of(p, b, &bad).n + kTile - 1) / kTile : 0;
        int total;
        const int ex = carry + block_scan<kThreads>(tiles, tmp, &total);
        if (b < p.batch) at[b] = ex;
        carry += total;
    }
    if (threadIdx.x == 0) at[p.batch] = carry;
    if (blockIdx.x == 0) flag(p.c.status, bad);
    __syncthreads();
}

// The block's walk over its segments.
struct Segment {
    Row row;
    int b, head, part;                    // row, kv head, head group of it
    int first, last;                      // positions [first, last) of 0 .. row.n
    int whole;                            // nothing of this (row, head group) is elsewhere
    int item;                             // (b * heads + head) * parts + part
    int slot;                             // where this segment leaves its part
    int lo_block, parts_n;                // the blocks that share the item, first and how many
    int lo_slot;                          // the slot of its first part (2 lo_block or + 1)
};

struct Walk {
    long long total, t, t1;               // all tiles; this block's next and end
    long long t0;
    int blocks;                           // blocks that have work

    __device__ __forceinline__ void begin(const AttnParams& p, const int* at) {
        total = static_cast<long long>(at[p.batch]) * p.c.heads * p.parts;
        blocks = static_cast<int>(total < gridDim.x ? total : gridDim.x);
        if (static_cast<int>(blockIdx.x) >= blocks) {
            t0 = t = t1 = 0;
            return;
        }
        t0 = t = total * blockIdx.x / blocks;
        t1 = total * (blockIdx.x + 1) / blocks;
    }
    __device__ __forceinline__ int block_of(long long tile) const {
        return static_cast<int>(((tile + 1) * blocks - 1) / total);
    }
    // The segment that begins at tile t; moves t past it.
    __device__ __forceinline__ Segment next(const AttnParams& p, const int* at) {
        const int hp = p.c.heads * p.parts;
        int lo = 0, hi = p.batch;         // the last row with at * hp <= t, tiles of its own
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (static_cast<long long>(at[mid]) * hp <= t) lo = mid; else hi = mid;
        }
        Segment s;
        unsigned bad = 0;
        s.b = lo;
        s.row = row_of(p, lo, &bad);
        const int tiles = at[lo + 1] - at[lo];
        const long long into = t - static_cast<long long>(at[lo]) * hp;
        const int hg = static_cast<int>(into / tiles);
        const int tile = static_cast<int>(into - static_cast<long long>(hg) * tiles);
        s.head = hg / p.parts;
        s.part = hg - s.head * p.parts;
        s.item = lo * hp + hg;
        const long long left = t1 - t;
        const int count = static_cast<int>(left < tiles - tile ? left : tiles - tile);
        s.first = tile * kTile;
        s.last = (tile + count) * kTile < s.row.n ? (tile + count) * kTile : s.row.n;
        s.whole = count == tiles ? 1 : 0;
        const long long a = t - tile;     // the item's first tile
        s.slot = 2 * blockIdx.x + (t == t0 ? 0 : 1);
        if (!s.whole) {
            s.lo_block = block_of(a);
            s.parts_n = block_of(a + tiles - 1) - s.lo_block + 1;
            s.lo_slot = 2 * s.lo_block + (a == total * s.lo_block / blocks ? 0 : 1);
        } else {
            s.lo_block = s.parts_n = s.lo_slot = 0;
        }
        t += count;
        return s;
    }
};

// The output of one head row: o[d] / sum, and its log-sum-exp (m in powers of two).
template <class T>
__device__ __forceinline__ void put_out(const AttnParams& p, int b, int head, int d, float o,
                                        float sum) {
    const float x = sum > 0.0f ? o / sum : (sum == 0.0f ? 0.0f : sum);   // a NaN sum stays NaN
    static_cast<T*>(p.out)[b * p.out_batch + head * p.out_head + d] = from_float<T>(x);
}
__device__ __forceinline__ void put_lse(const AttnParams& p, int b, int head, float m, float sum) {
    if (p.lse != nullptr)
        p.lse[static_cast<long long>(b) * p.q_heads + head] =
            sum == 0.0f ? kNegInf : (m + log2f(sum)) * kLn2;
}

// Rows with nothing to read: out 0, lse -inf.  at: from number_tiles.
template <class T>
__device__ __forceinline__ void put_empty_rows(const AttnParams& p, const int* at) {
    for (int b = blockIdx.x; b < p.batch; b += gridDim.x) {
        if (at[b + 1] != at[b]) continue;
        for (int x = threadIdx.x; x < p.q_heads * p.c.dim; x += kThreads) {
            const int h = x / p.c.dim, d = x - h * p.c.dim;
            put_out<T>(p, b, h, d, 0.0f, 0.0f);
            if (d == 0) put_lse(p, b, h, 0.0f, 0.0f);
        }
    }
}

// The segment's result is in shared memory: m[part], sum[part], o[part][dim] (o not divided).
// Whole: writes the output.  Else: leaves it in the workspace, and the last block of the item
// to arrive joins the parts.  `turn`: one int of shared memory.  Called by all threads, after a
// barrier; ends with one.
template <class T>
__device__ __forceinline__ void finish(const AttnParams& p, const Segment& s, const float* m,
                                       const float* sum, const float* o, int* turn) {
    const int dim = p.c.dim;
    const int first_head = s.head * p.group + s.part * p.part;
    const int heads = min(p.part, p.group - s.part * p.part);
    if (s.whole) {
        for (int x = threadIdx.x; x < heads * dim; x += kThreads) {
            const int g = x / dim, d = x - g * dim;
            put_out<T>(p, s.b, first_head + g, d, o[x], sum[g]);
            if (d == 0) put_lse(p, s.b, first_head + g, m[g], sum[g]);
        }
        __syncthreads();
        return;
    }
    const long long slot_size = static_cast<long long>(p.part) * (dim + 2);
    float* mine = p.slots + s.slot * slot_size;
    for (int x = threadIdx.x; x < heads * dim; x += kThreads) __stcg(mine + 2 * p.part + x, o[x]);
    if (static_cast<int>(threadIdx.x) < heads) {
        __stcg(mine + threadIdx.x, m[threadIdx.x]);
        __stcg(mine + p.part + threadIdx.x, sum[threadIdx.x]);
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int before = atomicAdd(p.arrived + s.item, 1);
        const int last = before == s.parts_n - 1 ? 1 : 0;
        if (last) p.arrived[s.item] = 0;                  // as the next call finds it
        *turn = last;
        __threadfence();
    }
    __syncthreads();
    if (*turn != 0) {
        for (int x = threadIdx.x; x < heads * dim; x += kThreads) {
            const int g = x / dim, d = x - g * dim;
            float top = kNegInf, all = 0.0f, acc = 0.0f;
            for (int i = 0; i < s.parts_n; ++i) {
                const int slot = i == 0 ? s.lo_slot : 2 * (s.lo_block + i);
                const float* part = p.slots + slot * slot_size;
                const float pm = __ldcg(part + g), ps = __ldcg(part + p.part + g);
                const float po = __ldcg(part + 2 * p.part + x);
                const float up = fmaxf(top, pm);
                const float base = up == kNegInf ? 0.0f : up;
                const float wa = exp2f(top - base), wb = exp2f(pm - base);
                all = fmaf(ps, wb, all * wa);
                acc = fmaf(po, wb, acc * wa);
                top = up;
            }
            put_out<T>(p, s.b, first_head + g, d, acc, all);
            if (d == 0) put_lse(p, s.b, first_head + g, top, all);
        }
    }
    __syncthreads();
}


}  // namespace gs_decode
