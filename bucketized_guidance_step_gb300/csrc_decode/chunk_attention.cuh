// Attention of chunks of new tokens over a paged cache: how the work is cut and handed out, and how
// the parts of a cut row are joined.  The arithmetic is chunk_attention.cu's (split products, for fp32
// caches) or chunk_attention_mma.cuh's (tcgen05, for 16-bit caches).
//
// An entry of the call is m new tokens of one sequence.  With one kv head it is m * group query rows
// (group: query heads of a kv head; row r is token r / group, head r % group of the group), which
// share the entry's keys and values: rows are taken ROWS at a time, a tile.  The positions that a tile
// sees are read in units of up to KT tokens: whole pages where a page has up to KT tokens, else a
// part of one page.
//
// Lengths and chunks are on the device, so the cut is found there: every block sums up what the tiles of
// the call cost, a pass over n entries in closed form, and the sum is cut into as many equal shares as
// there are blocks, each a run of neighbouring tiles and parts of tiles.  So ragged chunks and lengths
// balance without the host knowing them, one long sequence spreads over every block, and there are two
// parts a share at most.  A share whose edge would leave less than two units of a tile, or lies in a tile
// of few, takes or leaves the tile whole.  Where tiles are more than the blocks and none is large, all stay whole:
// shares of falling size balance them without joins (16 chunks of up to 512 tokens, window 1024, 16 and 4 heads of 128:
// 105 us cut, 73 us whole; 8 prompts of up to 2048 tokens, 32 and 8 heads of 128: 164 us and 157 us).  The costs were fitted
// there; over heads of 64 to 256, groups of 4 and 7, bf16 and fp32 (48 calls) the rule is 2.8 % off the better way, at worst
// 1.4 times it (32 sequences, most with a few new tokens, 28 and 4 heads of 128: 272 us cut, 193 us whole).
//
// Blocks take shares from a queue, and once there are no more, the joins of the shares' parts: what waits
// for a part waits for a block that is running.  The outputs of a share do not depend on who computes it
// or when, and the parts of a tile are joined in a fixed order: results do not depend on timing.
//
// To find the first item takes a block 4 to 5 us of its 16 in the smallest calls (2 chunks of up to 7 tokens over
// up to 257), a chain of lookups and scans; later ones are found while the last one is computed (16-bit caches).
#pragma once

#include "chunk_limit.h"
#include "decode_common.cuh"

namespace gs_decode {

constexpr float kChunkLog2e = 1.4426950408889634f;
constexpr float kChunkLn2 = 0.6931471805599453f;
constexpr int kChunkCounters = GS_CHUNK_COUNTERS;        // words of the workspace that are 0 between calls
constexpr int kChunkHead = 4;                            // of these, before the shares' counts
constexpr int kChunkShares = kChunkCounters - kChunkHead;            // most shares

struct ChunkParams {
    CacheView c;                          // c.k and c.v are the layer's
    int n, tokens;
    const int* seq;
    const int* start;
    int q_heads, group;
    unsigned group_mul, group_shift;      // x / group = (mulhi(x, mul) + x) >> shift
    int tile_step;                        // 16ths of a position from one tile to the next
    const void* q;
    long long q_token, q_head;
    int q_aligned, out_aligned;           // rows lie on 16 bytes
    int q_boxes;                          // TMA brings the queries
    int out_wide, slots_wide;             // out's rows, and the slots', lie on 32 bytes
    float scale_log2;                     // |scale| * log2 e (1 where scale is 0)
    float q_sign;                         // what queries are multiplied with: 1, -1 or 0
    int window, sinks;
    void* out;
    long long out_token, out_head;
    float* lse;
    int* work;                            // [0] the queue, [1] blocks that are done, [kChunkHead ..] by
                                          // share: parts that are done of the tile it began and did not end
    float* slots;                         // two a share: for the tile it did not begin, the one it does not end
    int slot_rows;                        // rows of one
    int unit_page;                        // tokens that units are cut by: a page's, or a unit's (fp32: rows are copied one by one)
};

__device__ __forceinline__ unsigned long long chunk_clock() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// What ends a block's waits.
struct ChunkGuard {
    int dead;                             // one has run out
    unsigned long long limit;             // nanoseconds
    unsigned long long deadline;          // of all (16-bit caches): `limit` after the last item was found; 0: dead
};

// A slot: reference[rows], sum[rows], o[rows][dim].
__host__ __device__ inline long long chunk_slot_words(int rows, int dim) {
    return static_cast<long long>(rows) * (dim + 2);
}

__device__ __forceinline__ int chunk_token(const ChunkParams& p, int row) {
    return static_cast<int>((__umulhi(static_cast<unsigned>(row), p.group_mul) + static_cast<unsigned>(row)) >> p.group_shift);
}
// x / d for quotients that are small, x >= 0 and d > 0: a quotient in 24 bits and its remainder (a division
// of 64-bit numbers takes hundreds of cycles, and a block's first item waits for half a dozen).
__device__ __forceinline__ long long chunk_quotient(long long x, long long d) {
    long long q = static_cast<long long>(__fdividef(__ll2float_rn(x), __ll2float_rn(d)));
    long long r = x - q * d;
    while (r < 0) {
        --q;
        r += d;
    }
    while (r >= d) {
        ++q;
        r -= d;
    }
    return q;
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
    int parts, share;                     // parts of the tile; the share that has the first
    int slot;                             // of this part
    int need;                             // the tile's count once all parts are there
    int at;                               // kind 2: first row of the piece in the tile
};

// The slot of part k of a tile that begins in `share`.
__device__ __forceinline__ int chunk_slot(int share, int k) { return 2 * (share + k) + (k == 0); }

// The cut, found by every block alike: WIDTH of its THREADS threads take the entries.  A tile's parts
// count once for every HALF rows of it.  Costs are in 16ths of a position.
template <int ROWS, int HALF, int KT, int THREADS, int WIDTH>
struct ChunkCut {
    using ll = long long;
    static constexpr int kOver = 16 * 288;               // what a tile costs beside its positions
    static constexpr int kFew = 8;        // units of a tile that is not cut
    static constexpr int kLeast = 2;      // units of a part
    static constexpr int kCut = KT == 64 ? 16 * 1920 : 16 * 128;     // what cutting costs a block (about 25 us and 10 us)
    static constexpr int kLevels = 4;     // of sizes of shares, where tiles stay whole
    // Tiles are counted in one number with the rows, in its lowest bits, which all threads' together may not pass.
    static constexpr int kTileBits = 18;
    static constexpr ll kMostTiles = 1023;               // that a thread counts: more than decide anything below
    static_assert(WIDTH * kMostTiles < 1ll << kTileBits, "the tiles' count reaches into the rows'");
    struct Shared {
        ll before[WIDTH];                 // cost before a thread's entries
        ll tmp[THREADS / 32 + 1];
        ll each;                          // shares: the first `more` have each + 1, the others each
        int more, shares;
        int levels, per;                  // whole tiles: levels of shares, shares of a level, ...
        ll begin[kLevels + 1], step[kLevels];            // ... and where they begin
        unsigned most;                    // the largest tile's cost
        ChunkGuard guard;                 // (its limit)
    };

    // What the tiles of a head cost: a tile whose last row sees `a` positions kOver + a, a_t = from + (t + 1)
    // step up to `cap`.
    struct Cost {
        ll from, step, cap;
        int tiles, turn;                  // tiles; those below the cap
        __device__ __forceinline__ ll upto(int t) const {            // of the first t
            const ll y = t < turn ? t : turn;
            return t * static_cast<ll>(kOver) + y * from + step * (y * (y + 1) / 2) + (t - y) * cap;
        }
    };
    Shared* s;
    // The walk over a share's tiles (one thread's).
    ll x0, x1, entry_at;                  // the share; cost before the entry
    Cost cost;
    ChunkEntry e;
    int i, share, head, tile;
    bool walking, joining;
    int ticket;                           // taken from the queue ahead (its way to memory and back passes during find), or -1
    ll first_at;                          // joining: the share's first tile, until it is passed

    static __device__ __forceinline__ int tiles_of(const ChunkParams& p, const ChunkEntry& e) {
        return static_cast<int>((static_cast<ll>(e.m) * p.group + ROWS - 1) / ROWS);
    }
    static __device__ __forceinline__ Cost cost_of(const ChunkParams& p, const ChunkEntry& e) {
        Cost c;
        c.tiles = tiles_of(p, e);
        c.from = 16ll * max(0, e.len - e.m);
        c.step = p.tile_step;
        c.cap = 0x7fffffffffffll;
        c.turn = c.tiles;
        if (p.window > 0) {
            c.cap = 16 * (static_cast<ll>(p.window) + p.sinks + KT) + c.step;
            const ll below = c.cap - c.from;
            const ll t = below <= c.step ? 0 : below > c.step * c.tiles ? c.tiles : chunk_quotient(below - 1, c.step);
            if (t < c.tiles) c.turn = static_cast<int>(t);
        }
        return c;
    }

    // Where tiles are many and none is large, whole tiles balance as well as cut ones, and need no joins.
    __device__ __noinline__ void keep_whole(const ChunkParams& p, ll all, int tiles) {
        const int per = (p.n + WIDTH - 1) / WIDTH, i0 = threadIdx.x * per, i1 = min(p.n, i0 + per);
        unsigned mine = 0, ignore = 0;
        for (int k = i0; k < i1; ++k) {
            const Cost c = cost_of(p, chunk_entry(p, k, &ignore));
            if (c.tiles > 0) mine = max(mine, static_cast<unsigned>(min(c.upto(c.tiles) - c.upto(c.tiles - 1), 0x7fffffffll)));
        }
        __syncthreads();
        if (mine > 0) atomicMax(&s->most, mine);
        __syncthreads();
        if (threadIdx.x > 0) return;
        const int blocks = gridDim.x;
        const ll most = s->most;
        if (tiles >= 2 * blocks ? 3 * most > 4 * kCut : 2 * most > s->each + kCut) return;
        s->levels = tiles < 4 * blocks ? 2 : tiles < 8 * blocks ? 3 : kLevels;
        s->per = blocks;
        s->shares = s->levels * blocks;
        ll at = 0;
        for (int l = 0; l < s->levels; ++l) {
            const ll size = l + 1 < s->levels ? (all - at) / 2 : all - at;
            s->begin[l] = at;
            s->step[l] = size / blocks;
            at += size;
        }
        s->begin[s->levels] = all;
    }

    // All threads; ends with a barrier.
    __device__ __forceinline__ void find(const ChunkParams& p) {
        const int per = (p.n + WIDTH - 1) / WIDTH, i0 = threadIdx.x * per, i1 = min(p.n, i0 + per);
        ll mine = 0, counts = 0, all, all_counts;        // (counts: rows, and in the lowest bits tiles)
        int tiles = 0;
        unsigned bad = 0;
#pragma unroll 4
        for (int k = i0; k < i1; ++k) {
            const ChunkEntry e = chunk_entry(p, k, &bad);
            const Cost c = cost_of(p, e);
            tiles = static_cast<int>(min(kMostTiles, tiles + static_cast<ll>(c.tiles) * p.c.heads));
            mine += c.upto(c.tiles) * p.c.heads;
            counts += static_cast<ll>(e.m) << kTileBits;
        }
        counts += tiles;
        const ll before = block_scan<THREADS>(mine, s->tmp, &all);
        block_scan<THREADS>(counts, s->tmp, &all_counts);
        if (all_counts >> kTileBits > p.tokens) {        // entries share rows: there is no end to what they could ask for
            bad |= GS_DEV_BAD_SEQ;
            all = all_counts = 0;
        }
        const ll all_tiles = all_counts & ((1ll << kTileBits) - 1);
        if (blockIdx.x == 0) flag(p.c.status, bad);
        if (threadIdx.x < WIDTH) s->before[threadIdx.x] = before;
        if (threadIdx.x == 0) {
            // No more shares than blocks, than tiles, or than there are four units for.
            ll n = max(all_tiles, all / (16 * 4 * KT));
            n = min(n, static_cast<ll>(gridDim.x));
            s->shares = static_cast<int>(n);
            s->each = n > 0 ? all / n : 0;
            s->more = n > 0 ? static_cast<int>(all - s->each * n) : 0;
            s->levels = 0;
            s->most = 0;
            // (Tiles that stay whole cost `each` and kCut at most.)
            s->guard.limit = chunk_limit_ns(s->each + kCut, KT == 64 ? kChunkNs : kChunkNsFp32);
            s->guard.deadline = chunk_clock() + s->guard.limit;
        }
        if (all_tiles > gridDim.x) keep_whole(p, all, static_cast<int>(all_tiles));
        walking = false;
        __syncthreads();
    }

    // Words of the workspace that the call counts in.
    __device__ __forceinline__ int used() const { return kChunkHead + (s->levels == 0 ? s->shares : 0); }

    // Where share n begins.
    __device__ __forceinline__ ll first_of(int n) const { return n * s->each + min(n, s->more); }
    // The share's begin and end.  (Whole tiles: half of the work in shares of equal size, one a block, half of the
    // rest, ..., so that the last ones taken are small.)
    __device__ __forceinline__ void bound() {
        if (s->levels == 0) {
            x0 = first_of(share);
            x1 = first_of(share + 1);
            return;
        }
        int level = 0, i = share;
        for (; i >= s->per; i -= s->per) ++level;
        x0 = s->begin[level] + i * s->step[level];
        x1 = i + 1 < s->per ? x0 + s->step[level] : s->begin[level + 1];
    }
    __device__ __forceinline__ int share_of(ll x) const {
        const ll edge = s->more * (s->each + 1);
        return static_cast<int>(x < edge ? chunk_quotient(x, s->each + 1) : s->more + chunk_quotient(x - edge, s->each));
    }
    // The unit at which an edge `f` into a tile's cost cuts it.
    static __device__ __forceinline__ int cut(int units, ll all, ll f) {
        if (units < kFew) return 2 * f >= all ? units : 0;
        const int u = static_cast<int>(chunk_quotient(units * f + all / 2, all));
        return u < kLeast ? 0 : units - u < kLeast ? units : u;
    }

    __device__ __forceinline__ void enter(const ChunkParams& p, int entry) {
        unsigned ignore = 0;
        i = entry;
        e = chunk_entry(p, i, &ignore);
        cost = cost_of(p, e);
    }

    // To the tile at cost x.
    __device__ __forceinline__ void seek(const ChunkParams& p, ll x) {
        int lo = 0, hi = WIDTH - 1;       // the last thread whose entries begin at x or before
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s->before[mid] <= x) lo = mid;
            else hi = mid - 1;
        }
        entry_at = s->before[lo];
        enter(p, min(p.n - 1, lo * ((p.n + WIDTH - 1) / WIDTH)));
        ll all = cost.upto(cost.tiles);
        while (x >= entry_at + all * p.c.heads && i + 1 < p.n) {
            entry_at += all * p.c.heads;
            enter(p, i + 1);
            all = cost.upto(cost.tiles);
        }
        head = all > 0 ? static_cast<int>(min(chunk_quotient(x - entry_at, all), static_cast<ll>(p.c.heads))) : p.c.heads;
        walking = head < p.c.heads;       // (else lengths have changed during the call)
        const ll left = x - entry_at - head * all;
        int a = 0, b = cost.tiles - 1;    // the last tile that begins at x or before
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (cost.upto(mid) <= left) a = mid;
            else b = mid - 1;
        }
        tile = a;
    }
    __device__ __forceinline__ ll tile_at() const {
        return entry_at + head * cost.upto(cost.tiles) + cost.upto(tile);
    }
    __device__ __forceinline__ void step(const ChunkParams& p) {
        if (++tile < cost.tiles) return;
        tile = 0;
        if (++head < p.c.heads) return;
        head = 0;
        entry_at += cost.upto(cost.tiles) * p.c.heads;
        do {
            if (i + 1 >= p.n) {
                walking = false;
                return;
            }
            enter(p, i + 1);
        } while (cost.tiles == 0);
    }

    // This share's part of the tile it is at; false where it has none, or (join) nothing to join.
    __device__ __forceinline__ bool part(const ChunkParams& p, bool join, ChunkItem* it) const {
        const ChunkUnits<KT> u(p.unit_page);
        const ll at = tile_at(), all = cost.upto(tile + 1) - cost.upto(tile), end = at + all;
        it->kind = 1;
        it->e = e;
        it->head = head;
        it->row = tile * ROWS;
        const int rows = static_cast<int>(min(static_cast<ll>(ROWS), static_cast<ll>(e.m) * p.group - it->row));
        it->rows = rows;
        const int from = e.len - e.m;
        it->span = chunk_span<KT>(p, u, from + chunk_token(p, it->row), from + chunk_token(p, it->row + rows - 1));
        const int units = it->span.count;
        it->parts = 1;
        it->share = share;
        if (s->levels > 0) {              // who has the tile's middle has the tile
            it->lo = at >= x0 || 2 * (x0 - at) < all ? 0 : units;
            it->hi = end <= x1 || 2 * (x1 - at) >= all ? units : 0;
        } else {
            it->lo = at >= x0 ? 0 : cut(units, all, x0 - at);
            it->hi = end <= x1 ? units : cut(units, all, x1 - at);
        }
        if (s->levels == 0 && (it->lo > 0 || it->hi < units)) {
            // The edges that cut the tile: those in it but a first and a last one that leave too little.
            int j0 = share_of(at) + 1, j1 = share_of(end - 1);
            if (j0 <= j1 && cut(units, all, first_of(j0) - at) == 0) ++j0;
            if (j0 <= j1 && cut(units, all, first_of(j1) - at) == units) --j1;
            it->parts = j1 - j0 + 2;
            it->share = j0 - 1;
        }
        const int k = share - it->share;
        it->slot = chunk_slot(it->share, k);
        it->need = it->parts * ((rows + HALF - 1) / HALF);
        it->at = 0;
        if (it->lo >= it->hi && (units > 0 || at < x0)) return false;
        if (!join) return true;
        it->kind = 2;                     // a part's rows of the join
        it->at = static_cast<int>(static_cast<ll>(rows) * k / it->parts);
        it->rows = static_cast<int>(static_cast<ll>(rows) * (k + 1) / it->parts) - it->at;
        return it->parts > 1 && it->rows > 0;
    }

    // The block's next item, by one thread; kind 0 after the last.
    __device__ __forceinline__ ChunkItem item(const ChunkParams& p) {
        ChunkItem it;
        for (;;) {
            while (walking) {
                if (tile_at() >= x1) {
                    walking = false;
                    break;
                }
                const bool some = part(p, joining, &it);
                if (!joining) {
                    step(p);
                } else {                  // only a share's first and last tile have parts elsewhere
                    const ll was = tile_at();
                    if (was == first_at) seek(p, x1 - 1);
                    if (tile_at() == was) walking = false;
                }
                if (some) return it;
            }
            const int n = ticket >= 0 ? ticket : atomicAdd(p.work, 1);
            ticket = -1;
            if (n >= (s->levels == 0 ? 2 : 1) * s->shares) {
                it.kind = 0;
                return it;
            }
            joining = n >= s->shares;
            share = joining ? n - s->shares : n;
            bound();
            seek(p, x0);
            first_at = tile_at();
        }
    }
};

// The next item, apart from the kernel, whose registers are the products'.
template <class C>
__device__ __noinline__ void chunk_next_item(C* cut, const ChunkParams& p, ChunkItem* it) {
    C mine = *cut;
    *it = mine.item(p);
    *cut = mine;
}

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

// Waits (`limit` at most) until all parts of a tile are in their slots.  One thread.
__device__ __forceinline__ bool chunk_wait_parts(const int* count, int parts, unsigned long long limit) {
    const unsigned long long t0 = chunk_clock();
    for (;;) {
        int v;
        asm volatile("ld.acquire.gpu.s32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        if (v >= parts) return true;
        if (chunk_clock() - t0 > limit) return false;
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
    const int t = chunk_token(p, r), h = it.head * p.group + r - t * p.group;
    const long long token = it.e.row + t;
    *lse = p.lse != nullptr ? p.lse + token * p.q_heads + h : nullptr;
    return static_cast<T*>(p.out) + token * p.out_token + h * p.out_head;
}

// RR rows from x0 on of a join, PP parts at a time, by a warp: a lane has a part's reference and sum of a row,
// and four neighbouring dims of all of them.
template <class T, int PP, int RR>
__device__ __forceinline__ void chunk_join_rows(const ChunkParams& p, const ChunkItem& it, int x0, float lift) {
    const int dim = p.c.dim, lane = threadIdx.x & 31, rows = it.rows, parts = it.parts;
    const int part = lane & (PP - 1), mine = min(lane / PP, RR - 1);         // this lane's part and row
    const long long words = 2 * chunk_slot_words(p.slot_rows, dim);              // between the slots of two shares
    const float* const first = p.slots + it.share * words;
    const long long begin = words / 2;    // part 0 is in its share's second slot
    auto slot = [&](int k) { return first + k * words + (k == 0 ? begin : 0); };
    const int row = it.at + min(x0 + mine, rows - 1);
    for (int d0 = 0; d0 < dim; d0 += 128) {
        const int d = d0 + 4 * lane, at = d < dim ? d : 0;
        float4 o[RR];
#pragma unroll
        for (int r = 0; r < RR; ++r) o[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float top = kNegInf, sum = 0.0f;  // of this lane's row
        for (int k0 = 0; k0 < parts; k0 += PP) {
            const float* const from = slot(min(k0 + part, parts - 1)) + row;
            const float ref = __ldcg(from), weight = __ldcg(from + p.slot_rows);
            float4 v[RR][PP];
#pragma unroll
            for (int i = 0; i < PP; ++i)
#pragma unroll
                for (int r = 0; r < RR; ++r)
                    v[r][i] = __ldcg(reinterpret_cast<const float4*>(
                        slot(min(k0 + i, parts - 1)) + 2 * p.slot_rows +
                        static_cast<long long>(it.at + min(x0 + r, rows - 1)) * dim + at));
            float up = fmaxf(top, ref);
#pragma unroll
            for (int i = 1; i < PP; i <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, i));
            const float base = up == kNegInf ? 0.0f : up, fade = chunk_pow2(top - base);
            const float w = k0 + part < parts ? chunk_pow2(ref - base) : 0.0f;
            float all = weight * w;
#pragma unroll
            for (int i = 1; i < PP; i <<= 1) all += __shfl_xor_sync(0xffffffffu, all, i);
            sum = fmaf(sum, fade, all);
            top = up;
#pragma unroll
            for (int r = 0; r < RR; ++r) {
                const float f = __shfl_sync(0xffffffffu, fade, r * PP);
                o[r].x *= f;
                o[r].y *= f;
                o[r].z *= f;
                o[r].w *= f;
#pragma unroll
                for (int i = 0; i < PP; ++i) {
                    const float g = __shfl_sync(0xffffffffu, w, r * PP + i);
                    o[r].x = fmaf(v[r][i].x, g, o[r].x);
                    o[r].y = fmaf(v[r][i].y, g, o[r].y);
                    o[r].z = fmaf(v[r][i].z, g, o[r].z);
                    o[r].w = fmaf(v[r][i].w, g, o[r].w);
                }
            }
        }
        const float by = sum > 0.0f ? 1.0f / sum : sum;  // a NaN stays one
        float* lse;
#pragma unroll
        for (int r = 0; r < RR; ++r) {
            const float f = __shfl_sync(0xffffffffu, by, r * PP);
            if (x0 + r < rows && d < dim) {
                T* const to = chunk_out<T>(p, it, it.row + it.at + x0 + r, &lse);
                chunk_put4<T>(p, to + d, make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f));
            }
        }
        if (d0 == 0 && part == 0 && lane < RR * PP && x0 + mine < rows && p.lse != nullptr) {
            chunk_out<T>(p, it, it.row + row, &lse);
            *lse = sum == 0.0f ? kNegInf : (top + log2f(sum) - lift) * kChunkLn2;
        }
    }
}

// Joins a piece of a tile: the parts of a row are weighted to their common reference, in their order.
// What costs is latency, so a warp has 16 outputs a lane in flight, none under a condition (which would put
// them one after the other): what is past the parts, rows or dims reads the last one's and counts nothing.
// lift: what the sums are scaled by, in powers of two.
template <class T>
__device__ __noinline__ void chunk_join(const ChunkParams& p, const ChunkItem& it, int warp, int warps, float lift) {
    const int each = (it.rows + warps - 1) / warps;      // rows of a warp
    const int end = min(it.rows, (warp + 1) * each);
    for (int x = warp * each; x < end;) {
        if (it.parts <= 2) {
            chunk_join_rows<T, 2, 8>(p, it, x, lift);
            x += 8;
        } else if (it.parts <= 4) {
            chunk_join_rows<T, 4, 4>(p, it, x, lift);
            x += 4;
        } else {
            chunk_join_rows<T, 8, 2>(p, it, x, lift);
            x += 2;
        }
    }
}

// What the two files' kernels take of a call, by the cache's type and head size.
struct ChunkShape {
    int rows, blocks;                     // rows of a tile; blocks of the grid
};
int chunk_fp32_unit();                    // positions of a unit
ChunkShape chunk_fp32_shape(int dim);
ChunkShape chunk_mma_shape(int dim);
gs_status launch_chunk_fp32(const ChunkParams& p, int blocks, gs_stream stream);
gs_status launch_chunk_mma(int dtype, ChunkParams& p, int blocks, gs_stream stream);
gs_status launch_chunk_mma_split(int dtype, ChunkParams& p, int blocks, gs_stream stream);

}  // namespace gs_decode
