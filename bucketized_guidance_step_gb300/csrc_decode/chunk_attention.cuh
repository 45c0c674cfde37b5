// Attention of chunks of new tokens over a paged cache: how the work is cut and handed out, and how
// the parts of a cut row are joined.  The arithmetic is chunk_attention.cu's (fp32 multiply-adds, for
// fp32 caches) or chunk_attention_mma.cu's (the tensor cores, for 16-bit caches).
//
// An entry of the call is m new tokens of one sequence.  With one kv head it is m * group query rows
// (group: query heads of a kv head; row r is token r / group, head r % group of the group), which
// share the entry's keys and values: rows are taken ROWS at a time, a tile.  The positions that a tile
// sees are read in units of up to KT tokens: whole pages where a page has up to KT tokens, else a
// part of one page.
//
// Lengths and chunks are on the device, so the cut is found there: every block sums the entries'
// tiles and units, a pass over n entries that is a word or two a thread.  An item is a tile, or where
// there are few tiles a run of `each` units of one; blocks take items from a queue, the longest of an
// entry first.  The outputs of an item do not depend on who computes it or when, and the parts of a
// tile are joined in their order by further items of the queue: results do not depend on timing.
#pragma once

#include "decode_common.cuh"

namespace gs_decode {

constexpr float kChunkLog2e = 1.4426950408889634f;
constexpr float kChunkLn2 = 0.6931471805599453f;
constexpr int kChunkCounters = GS_CHUNK_COUNTERS;        // words of the workspace that are 0 between calls
constexpr int kChunkHead = 4;                            // of these, before the tiles' counts
constexpr int kChunkCut = kChunkCounters - kChunkHead;   // most tiles of a call whose tiles are cut
constexpr unsigned long long kChunkLimitNs = 200ull * 1000ull * 1000ull;   // of a wait

struct ChunkParams {
    CacheView c;                          // c.k and c.v are the layer's
    int n, tokens;
    const int* seq;
    const int* start;
    int q_heads, group;
    const void* q;
    long long q_token, q_head;
    int q_aligned, out_aligned;           // rows lie on 16 bytes
    int q_boxes;                          // TMA brings the queries
    float scale_log2;                     // |scale| * log2 e (1 where scale is 0)
    float q_sign;                         // what queries are multiplied with: 1, -1 or 0
    int window, sinks;
    void* out;
    long long out_token, out_head;
    float* lse;
    int* work;                            // [0] the queue, [1] blocks that are done, [kChunkHead ..]
                                          // parts of a tile that are done
    float* slots;                         // [slot_count][slot_words]
    int slot_count, slot_rows;            // slots; rows of one
};

// A slot: reference[rows], sum[rows], o[rows][dim].
__host__ __device__ inline long long chunk_slot_words(int rows, int dim) {
    return static_cast<long long>(rows) * (dim + 2);
}

struct ChunkEntry {
    int row, m, len, seq;                 // first row of q; new tokens; the sequence's length and number
};

// What does not hold is flagged: an entry whose rows are not within q's has none, a sequence outside
// the cache no tokens.
__device__ __forceinline__ ChunkEntry chunk_entry(const ChunkParams& p, int i, unsigned* bad) {
    ChunkEntry e;
    e.seq = p.seq[i];
    e.row = p.start[i];
    const long long m = static_cast<long long>(p.start[i + 1]) - e.row;
    e.m = static_cast<int>(m);
    if (e.row < 0 || m < 0 || e.row + m > p.tokens) {
        *bad |= GS_DEV_BAD_SEQ;
        e.row = e.m = 0;
    }
    e.len = 0;
    if (e.seq < 0 || e.seq >= p.c.seqs) {
        *bad |= GS_DEV_BAD_SEQ;
        e.seq = 0;
    } else {
        e.len = p.c.lens[e.seq];
        const int most = p.c.cols * p.c.page;
        if (e.len < 0 || e.len > most) {
            *bad |= GS_DEV_BAD_SEQ;
            e.len = e.len < 0 ? 0 : most;
        }
    }
    if (e.m > e.len) *bad |= GS_DEV_BAD_SEQ;             // rows before the sequence's first token
    return e;
}

// Units of a page table.
template <int KT>
struct ChunkUnits {
    int page, span, per;                  // tokens of a whole unit; page > KT: units of a page, else 0

    __device__ __forceinline__ explicit ChunkUnits(int page_tokens) : page(page_tokens) {
        per = page > KT ? (page + KT - 1) / KT : 0;
        span = per > 0 ? KT : KT / page * page;
    }
    __device__ __forceinline__ int of(int pos) const {
        if (per == 0) return pos / span;
        const int col = pos / page;
        return col * per + (pos - col * page) / KT;
    }
    // First position; *count: positions, *row: the first one's row in its page (page > KT).
    __device__ __forceinline__ int first(int unit, int* count, int* row) const {
        *row = 0;
        *count = span;
        if (per == 0) return unit * span;
        const int col = unit / per;
        *row = (unit - col * per) * KT;
        *count = min(KT, page - *row);
        return col * page + *row;
    }
};

// The units that a tile sees: number i is unit i for i < sinks, else i + skip.
struct ChunkSpan {
    int count, sinks, skip;

    __device__ __forceinline__ int unit(int i) const { return i < sinks ? i : i + skip; }
};

// first, last: positions of the tile's first and last row.
template <int KT>
__device__ __forceinline__ ChunkSpan chunk_span(const ChunkParams& p, const ChunkUnits<KT>& units,
                                                int first, int last) {
    ChunkSpan s = {0, 0, 0};
    if (last < 0) return s;
    const int end = units.of(last) + 1;
    s.count = end;
    if (p.window > 0) {
        const int from = first - p.window + 1;
        if (p.sinks > 0) s.sinks = units.of(min(p.sinks - 1, last)) + 1;
        if (from > 0) s.skip = max(0, units.of(from) - s.sinks);
        s.count = end - s.skip;
        if (s.skip == 0) s.sinks = 0;
    }
    return s;
}

struct ChunkItem {
    int kind;                             // 0: no more, 1: attend, 2: join
    ChunkEntry e;
    int head, row;                        // kv head; first row of the tile
    int rows;                             // rows of it (kind 2: of the piece)
    ChunkSpan span;
    int lo, hi;                           // units lo .. hi - 1 of the span
    int parts, slot;                      // parts of the tile; slot of this one (kind 2: of the first)
    int need;                             // its count once all parts are there
    int tile;                             // its count's number
    int at;                               // kind 2: first row of the piece in the tile
    int steps;                            // of the tensor cores' kernel
};

// The cut, found by every block alike: WIDTH of its THREADS threads take the entries.  A tile's
// parts count once for every HALF rows of it.
template <int ROWS, int HALF, int KT, int THREADS, int WIDTH>
struct ChunkCut {
    static constexpr int kMinUnits = 4;   // of a part
    struct Shared {
        int items[WIDTH], tiles[WIDTH];                  // before a thread's entries
        long long tmp[THREADS / 32 + 1];
        int each, total_items, total_tiles, pieces;
    };
    Shared* s;

    static __device__ __forceinline__ int tiles_of(const ChunkParams& p, const ChunkEntry& e) {
        return static_cast<int>((static_cast<long long>(e.m) * p.group + ROWS - 1) / ROWS);
    }
    // The most units that a tile of the entry sees, or a little more.
    static __device__ __forceinline__ int most_units(const ChunkParams& p, const ChunkUnits<KT>& u,
                                                     const ChunkEntry& e) {
        if (e.len == 0) return 0;
        const int all = u.of(e.len - 1) + 1;
        if (p.window == 0) return all;
        const long long seen = static_cast<long long>(p.window) + ROWS / p.group + 2;
        const long long sinks = p.sinks > 0 ? u.of(min(p.sinks, e.len) - 1) + 1 : 0;
        const long long few = sinks + (u.per == 0 ? seen / u.span + 2 : (seen / u.page + 2) * u.per);
        return static_cast<int>(min(static_cast<long long>(all), few));
    }
    static __device__ __forceinline__ int parts_of(int units, int each) {
        return units <= each ? 1 : (units + each - 1) / each;
    }

    // All threads; ends with a barrier.
    __device__ __forceinline__ void find(const ChunkParams& p) {
        const ChunkUnits<KT> u(p.c.page);
        const int per = (p.n + WIDTH - 1) / WIDTH, i0 = threadIdx.x * per, i1 = min(p.n, i0 + per);
        long long tiles = 0, units = 0;
        unsigned bad = 0;
        for (int i = i0; i < i1; ++i) {
            const ChunkEntry e = chunk_entry(p, i, &bad);
            const long long t = static_cast<long long>(tiles_of(p, e)) * p.c.heads;
            tiles += t;
            units += t * most_units(p, u, e);
        }
        if (blockIdx.x == 0) flag(p.c.status, bad);
        long long all_tiles, all_units;
        const long long before = block_scan<THREADS>(tiles, s->tmp, &all_tiles);
        block_scan<THREADS>(units, s->tmp, &all_units);
        const int blocks = gridDim.x;
        int each = 0x7fffffff;
        if (all_tiles < 4ll * blocks && all_tiles <= kChunkCut && p.slot_count > 0) {
            const long long want = (all_units + 2ll * blocks - 1) / (2ll * blocks);
            each = static_cast<int>(max(static_cast<long long>(kMinUnits), want));
        }
        long long items = 0, all_items = 0, items_before = 0;
        for (int turn = 0; turn < 2; ++turn) {
            items = 0;
            for (int i = i0; i < i1; ++i) {
                unsigned ignore = 0;
                const ChunkEntry e = chunk_entry(p, i, &ignore);
                items += static_cast<long long>(tiles_of(p, e)) * p.c.heads * parts_of(most_units(p, u, e), each);
            }
            items_before = block_scan<THREADS>(items, s->tmp, &all_items);
            if (each == 0x7fffffff || all_items <= p.slot_count) break;
            each = 0x7fffffff;            // (ranges that overlap, against the rules)
        }
        if (all_items > 0x3fffffffll) all_items = 0;     // (ranges that overlap)
        if (threadIdx.x < WIDTH) {
            s->items[threadIdx.x] = static_cast<int>(items_before);
            s->tiles[threadIdx.x] = static_cast<int>(before);
        }
        if (threadIdx.x == 0) {
            s->each = each;
            s->total_items = static_cast<int>(all_items);
            s->total_tiles = static_cast<int>(all_tiles);
            // Pieces of a tile for its join: about two a block in all.
            int pieces = each == 0x7fffffff || all_tiles == 0 ? 0 : static_cast<int>(2ll * blocks / all_tiles);
            if (pieces < 1 && each != 0x7fffffff) pieces = 1;
            s->pieces = min(pieces, ROWS / 8);
        }
        __syncthreads();
    }

    // Words of the workspace that the call counts in.
    __device__ __forceinline__ int used() const {
        return kChunkHead + (s->pieces > 0 ? s->total_tiles : 0);
    }

    // Item number j of the queue, by one thread.
    __device__ __forceinline__ ChunkItem item(const ChunkParams& p, int j) const {
        ChunkItem it;
        it.kind = 0;
        const bool join = j >= s->total_items;
        const int* before = join ? s->tiles : s->items;
        int x = j, piece = 0;
        if (join) {
            if (s->pieces == 0) return it;
            x = j - s->total_items;
            piece = x % s->pieces;
            x /= s->pieces;
            if (x >= s->total_tiles) return it;
        }
        int lo = 0, hi = WIDTH - 1;     // the last thread whose `before` is not above x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        const ChunkUnits<KT> u(p.c.page);
        const int per = (p.n + WIDTH - 1) / WIDTH, end = min(p.n, (lo + 1) * per);
        int items = s->items[lo], tiles = s->tiles[lo];
        unsigned ignore = 0;
        for (int i = lo * per; i < end; ++i) {
            const ChunkEntry e = chunk_entry(p, i, &ignore);
            const int mine = tiles_of(p, e) * p.c.heads;
            const int parts = parts_of(most_units(p, u, e), s->each);
            const int past = join ? tiles + mine : items + mine * parts;
            if (x >= past) {
                items += mine * parts;
                tiles += mine;
                continue;
            }
            it.kind = join ? 2 : 1;
            it.e = e;
            const int in = join ? x - tiles : (x - items) / parts;       // tile and head, the last tile first
            const int part = join ? 0 : x - items - in * parts;
            const int back = in / p.c.heads;
            it.head = in - back * p.c.heads;
            it.row = (tiles_of(p, e) - 1 - back) * ROWS;
            const int all = static_cast<int>(min(static_cast<long long>(ROWS),
                                                 static_cast<long long>(e.m) * p.group - it.row));
            it.rows = all;
            it.tile = tiles + in;
            const int first = e.len - e.m + it.row / p.group;
            const int last = e.len - e.m + (it.row + all - 1) / p.group;
            it.span = chunk_span<KT>(p, u, first, last);
            it.parts = parts_of(it.span.count, s->each);
            it.slot = items + in * parts + part;
            it.need = it.parts * ((all + HALF - 1) / HALF);
            it.lo = 0;
            it.hi = it.span.count;
            if (it.parts > 1) {
                // Equal parts: part k begins at unit count * k / parts.
                it.lo = static_cast<int>(static_cast<long long>(it.span.count) * part / it.parts);
                it.hi = static_cast<int>(static_cast<long long>(it.span.count) * (part + 1) / it.parts);
            }
            it.at = 0;
            if (join) {
                if (it.parts == 1) it.rows = 0;
                const int size = (ROWS + s->pieces - 1) / s->pieces;
                it.at = piece * size;
                it.rows = max(0, min(size, it.rows - it.at));
            } else if (part >= it.parts) {
                it.rows = 0;              // fewer parts than the entry's longest tile
            }
            return it;
        }
        return it;                        // (lengths that change during the call)
    }
};

// The last block of the call puts the `used` words of the workspace back to 0.  A warp, after its
// block's last use of them.
__device__ __forceinline__ void chunk_leave(const ChunkParams& p, int used) {
    const int lane = threadIdx.x & 31;
    int done = 0;
    if (lane == 0) {
        __threadfence();
        done = atomicAdd(p.work + 1, 1);
    }
    if (__shfl_sync(0xffffffffu, done, 0) != static_cast<int>(gridDim.x) - 1) return;
    for (int i = lane; i < used; i += 32) p.work[i] = 0;
}

// 2^x (results below 2^-126 are 0).
__device__ __forceinline__ float chunk_pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ unsigned long long chunk_clock() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits (200 ms at most) until all parts of a tile are in their slots.  One thread.
__device__ __forceinline__ bool chunk_wait_parts(const int* count, int parts) {
    const unsigned long long t0 = chunk_clock();
    for (;;) {
        int v;
        asm volatile("ld.acquire.gpu.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        if (v >= parts) return true;
        if (chunk_clock() - t0 > kChunkLimitNs) return false;
        __nanosleep(100);
    }
}

// Four neighbours of an output row.
template <class T>
__device__ __forceinline__ void chunk_put4(const ChunkParams& p, T* to, float4 o) {
    T r[4] = {from_float<T>(o.x), from_float<T>(o.y), from_float<T>(o.z), from_float<T>(o.w)};
    if (p.out_aligned) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<uint4*>(r);
        else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<uint2*>(r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = r[i];
    }
}

// The output row of row r of an entry's head, and its place in lse.
template <class T>
__device__ __forceinline__ T* chunk_out(const ChunkParams& p, const ChunkItem& it, int r, float** lse) {
    const int t = r / p.group, h = it.head * p.group + r - t * p.group;
    const long long token = it.e.row + t;
    *lse = p.lse != nullptr ? p.lse + token * p.q_heads + h : nullptr;
    return static_cast<T*>(p.out) + token * p.out_token + h * p.out_head;
}

// Joins a piece of a tile: the parts of a row are weighted to their common reference.  A warp a row: a
// lane looks at every 32nd part's reference and sum, then has four neighbouring dims of all parts, eight of
// them in flight (a thread that went through the parts one by one took 150 us for 38 parts of 132 rows).
// lift: what the sums are scaled by, in powers of two.
template <class T>
__device__ __forceinline__ void chunk_join(const ChunkParams& p, const ChunkItem& it, int warp, int warps,
                                           float lift) {
    const int dim = p.c.dim, lane = threadIdx.x & 31;
    const long long words = chunk_slot_words(p.slot_rows, dim);
    const float* const first = p.slots + it.slot * words;
    for (int x = warp; x < it.rows; x += warps) {
        const int r = it.at + x;
        float top = kNegInf;
        for (int k = lane; k < it.parts; k += 32) top = fmaxf(top, __ldcg(first + k * words + r));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float base = top == kNegInf ? 0.0f : top;
        float sum = 0.0f;
        float* lse;
        T* const to = chunk_out<T>(p, it, it.row + r, &lse);
        for (int d0 = 0; d0 < dim; d0 += 128) {
            const int d = d0 + 4 * lane;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k0 = 0; k0 < it.parts; k0 += 32) {
                float w = 0.0f;
                if (k0 + lane < it.parts) {
                    const float* const slot = first + (k0 + lane) * words + r;
                    w = chunk_pow2(__ldcg(slot) - base);
                    if (d0 == 0) sum = fmaf(__ldcg(slot + p.slot_rows), w, sum);
                }
                const int n = min(32, it.parts - k0);
                const float* from = first + k0 * words + 2 * p.slot_rows + static_cast<long long>(r) * dim + d;
                for (int k = 0; k < n; k += 8) {
                    float4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = k + i < n && d < dim ? __ldcg(reinterpret_cast<const float4*>(from + (k + i) * words))
                                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float f = __shfl_sync(0xffffffffu, w, k + i);
                        o.x = fmaf(v[i].x, f, o.x);
                        o.y = fmaf(v[i].y, f, o.y);
                        o.z = fmaf(v[i].z, f, o.z);
                        o.w = fmaf(v[i].w, f, o.w);
                    }
                }
            }
            if (d0 == 0) {
#pragma unroll
                for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
            }
            const float by = sum > 0.0f ? 1.0f / sum : sum;          // a NaN stays one
            if (d < dim) chunk_put4<T>(p, to + d, make_float4(o.x * by, o.y * by, o.z * by, o.w * by));
        }
        if (lane == 0 && lse != nullptr) *lse = sum == 0.0f ? kNegInf : (top + log2f(sum) - lift) * kChunkLn2;
    }
}

// What the two files' kernels take of a call, by the cache's type and head size.
struct ChunkShape {
    int rows, blocks;                     // rows of a tile; blocks of the grid
};
ChunkShape chunk_fp32_shape(int dim);
ChunkShape chunk_mma_shape(int dim);
gs_status launch_chunk_fp32(const ChunkParams& p, int blocks, gs_stream stream);
gs_status launch_chunk_mma(int dtype, ChunkParams& p, int blocks, gs_stream stream);

}  // namespace gs_decode
