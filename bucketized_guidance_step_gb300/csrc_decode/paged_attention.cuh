// Attention of one new token over a paged cache: how the work is cut, the pipeline that reads
// K and V, and how the parts of a split sequence are joined.  The arithmetic on a run of
// positions is a policy: fp32 multiply-adds (paged_attention.cu) or the tensor cores
// (paged_attention_mma.cu).
//
// Work is counted in tiles of consecutive visible positions of one (row, head group).  Every
// block sums the rows' lengths (a word a row) and numbers all tiles of the call; with T tiles,
// each of the C blocks takes T / C neighbours.  So ragged lengths balance without the host
// knowing them, and one long row spreads over every block.  A block's share is a run of
// segments, each a piece of one (row, head group).  A segment that is its (row, head group)
// whole is finished by its block; else the block leaves (max, sum, output) in its slot of the
// workspace, and the block that arrives last joins the parts in their order, so the result
// does not depend on timing.
//
// Each of a block's four warps works alone: of every tile it takes one run of positions,
// copies their rows of K and V into a ring of its own in shared memory with 16-byte
// asynchronous copies (zeros past the end), and keeps its own maximum, sum and output.  There
// is no barrier but at a segment's end, where the four meet in shared memory.  Copies run
// STAGES - 1 tiles ahead, over the ends of segments, and the page numbers of a tile are looked
// up one tile before its copies: short sequences do not drain the pipeline.  The 16-byte
// pieces of a row are permuted by the row's number (piece c of row r lies at c ^ (r & 7)),
// which keeps the reads of 8 rows free of bank conflicts.
//
// Visible positions are numbered 0 .. n-1: the first `sinks`, then the window (struct Row).
//
// What bounds it, on a GB300 (graph replay, inputs not in L2; bf16, dim 128, 32 query and 8 kv
// heads unless said): HBM where rows are long: 2 rows of 200001 .. 262143 tokens (2.02 GB) take
// 301 us, 99 % of the measured copy rate, 32 rows of 8192 161 us (98 %).  Below that a call's
// fixed part shows, about 9 us: lengths, table and first rows are three DRAM latencies in a
// chain (4.5 us), the last segment's end, its count and the join 3 to 5 us.  32 rows of 2048
// tokens: 48 us (83 %), 32 ragged ones of 1 .. 4099 with new tokens: 52 us (79 %).  Where segments
// are a tile long, what beginning and ending one costs is not hidden any more: 1032 rows of 64
// tokens 75 us (57 %), 258 rows of 256 53 us (77 %).  The smallest calls (2 rows of 125 and 250
// tokens, with new tokens) take 6.9 us.  Looking where a new token may be stored is 2 to 4 % of a
// call with new tokens (49.7 us without it for the ragged rows).  Counters (ncu, the ragged rows): DRAM reads 277.7 MB of 277.7 required, tensor pipe
// 9.6 %, 8 warps an SM.
//
// Measured and not kept: finding the places of 32 tiles at once, a tile a lane (48 -> 51 us at 32
// rows of 2048: the work moves between the copies of two tiles); three blocks an SM with rings of
// two stages (48 -> 51); blocks of at least 2, 3 or 4 units for small calls (7.4 -> 8.1, 10.1,
// 10.9 us at the smallest: a tile more in a row costs more than a part more to join); joining in
// two passes, weights first (7.5 -> 9.7 us).
#pragma once

#include "decode_common.cuh"

namespace gs_decode {

constexpr int kWarps = 4;                 // warps of a block
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
    CacheView c;
    int batch;                            // c.k and c.v are the layer's
    const int* seq;
    int q_heads, group;                   // query heads; of one kv head
    int parts, part;                      // head groups of a kv head; query heads of one
    const void* q;
    long long q_batch, q_head;
    const void* k_new;
    const void* v_new;
    long long new_batch, new_head;
    int new_aligned;                      // k_new and v_new rows lie on 16 bytes
    int out_aligned;                      // out rows lie on 4 elements
    int q_aligned;                        // q rows lie on 2 elements
    unsigned page_mul, page_shift;        // position / page = (mulhi(position, mul) + position) >> shift
    int dumps;                            // places for a segment's end in shared memory: 1 or 2
    int page_runs;                        // a page holds whole runs: a run lies in one page
    unsigned dim_mul;                     // x / dim = x * mul >> 20, for x < 8 dim
    float scale_log2;                     // scale * log2 e: scores are kept in powers of two
    int window, sinks;
    void* out;
    long long out_batch, out_head;
    float* lse;
    int* arrived;                         // [batch * heads * parts], 0 between calls
    float* slots;                         // [2 * blocks][slot_size]
};

// A part in the workspace: m[part], sum[part], o[part][dim] on 16 bytes.
__host__ __device__ inline int slot_head(int part) { return (2 * part + 3) / 4 * 4; }
__host__ __device__ inline long long slot_size(int part, int dim) {
    return slot_head(part) + static_cast<long long>(part) * dim;
}

// A row's visible positions, numbered in runs that begin at multiples of RUN in the sequence
// too: the sinks are 0 .. sinks - 1, the window begins at number `turn` (a multiple of RUN)
// with position `from` (the multiple of RUN at or below its first).  Numbers in between, and
// positions from .. first - 1, are not visible.  Without a window all but n and len are 0.
struct Row {
    int seq, n, len;                      // n: numbers in all (0: nothing to read); len: tokens
    int sinks, turn, from, first;
};

// The row of sequence `seq` with what lens[seq] holds (0 for a sequence outside the cache).
template <int RUN>
__device__ __forceinline__ Row row_from(const AttnParams& p, int seq, int len, unsigned* bad) {
    Row r;
    r.seq = seq;
    r.len = len;
    if (seq < 0 || seq >= p.c.seqs) {
        *bad |= GS_DEV_BAD_SEQ;
        r.seq = r.len = 0;
    }
    const int most = p.c.cols * p.c.page;
    if (r.len < 0 || r.len > most) {
        *bad |= GS_DEV_BAD_SEQ;
        r.len = r.len < 0 ? 0 : most;
    }
    r.n = r.len;
    r.sinks = r.turn = r.from = r.first = 0;
    if (p.window > 0 && r.len - p.window > p.sinks) {
        r.first = r.len - p.window;
        r.from = r.first / RUN * RUN;
        r.sinks = p.sinks;
        r.turn = (p.sinks + RUN - 1) / RUN * RUN;
        r.n = r.turn + (r.len - r.from);
    }
    return r;
}
template <int RUN>
__device__ __forceinline__ Row row_of(const AttnParams& p, int b, unsigned* bad) {
    const int seq = p.seq != nullptr ? p.seq[b] : b;
    return row_from<RUN>(p, seq, seq >= 0 && seq < p.c.seqs ? p.c.lens[seq] : 0, bad);
}

// The split of all units: the first `more` blocks take each + 1, the others each.
struct Split {
    int blocks, each, more;

    __device__ __forceinline__ int first_of(int block) const {
        return block * each + min(block, more);
    }
    __device__ __forceinline__ int block_of(int unit) const {
        const int edge = more * (each + 1);
        return unit < edge ? unit / (each + 1) : more + (unit - edge) / each;
    }
};

// A place in the sequence of units: a tile is a unit, and every (row, head group) has one more
// after its tiles for what beginning and ending a segment costs (without it the blocks of short
// rows end late: 58 against 52 us for 32 rows of 1 .. 4099 tokens).
template <int RUN>
struct Cursor {
    static constexpr int TILE = kWarps * RUN;
    Row row;
    int b, tiles;                         // row; tiles of one head group of it
    int base;                             // number of its first unit
    int hg, tile;                         // head group (head * parts + part); tile of it

    __device__ __forceinline__ void take_row(const AttnParams& p, int row_number) {
        unsigned bad = 0;
        b = row_number;
        row = row_of<RUN>(p, b, &bad);
        tiles = (row.n + TILE - 1) / TILE;
    }
    __device__ __forceinline__ int item() const { return base + hg * (tiles + 1); }
    __device__ __forceinline__ int unit() const { return item() + tile; }
    // To the next tile; where that is not below `end` (the block's), unit() is not either.
    __device__ __forceinline__ void next(const AttnParams& p, int end) {
        if (++tile < tiles) return;
        tile = 0;
        const int hp = p.c.heads * p.parts;
        if (++hg < hp) return;
        hg = 0;
        base += (tiles + 1) * hp;
        if (base >= end || b + 1 >= p.batch) return;
        take_row(p, b + 1);
        while (tiles == 0) {              // empty rows: the next one that is not, 128 at a look
            const int lane = threadIdx.x & 31;
            unsigned live[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = b + 1 + i * 32 + lane;
                const int s = at < p.batch ? (p.seq != nullptr ? p.seq[at] : at) : -1;
                live[i] = __ballot_sync(0xffffffffu, s >= 0 && s < p.c.seqs && p.c.lens[s] > 0);
            }
            int past = 0;                 // rows before the live one
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (past == i * 32) past += live[i] != 0u ? __ffs(live[i]) - 1 : 32;
            if (b + 1 + past >= p.batch) return;         // (lengths that change during the call)
            if (past < 128) take_row(p, b + 1 + past);
            else b += 128;
        }
    }
};

template <int RUN>
__device__ __forceinline__ int units_in(const Row& r) {
    return r.n > 0 ? (r.n + kWarps * RUN - 1) / (kWarps * RUN) + 1 : 0;
}

// The end of this block's units and the cursor at its first tile; false where it has none.
// Every warp finds them by itself.
template <int RUN>
__device__ __forceinline__ bool find_work(const AttnParams& p, Split* split, int* end,
                                          Cursor<RUN>* at) {
    const int lane = threadIdx.x & 31;
    const int hp = p.c.heads * p.parts;
    const int groups = (p.batch + 31) / 32, per = (groups + 31) / 32;
    unsigned bad = 0;
    int mine = 0;
    if (groups == 1) {                                   // a row a lane
        if (lane < p.batch) mine = units_in<RUN>(row_of<RUN>(p, lane, &bad));
    } else {
        // 32 rows at a time, eight such loads in flight; lane i keeps the sum of `per` of them from
        // per * i on, then the lanes are summed up.
        constexpr int N = 8;
        for (int g0 = 0; g0 < groups; g0 += N) {
            int seq[N], len[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int b = (g0 + i) * 32 + lane;
                seq[i] = b < p.batch && p.seq != nullptr ? p.seq[b] : b;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int b = (g0 + i) * 32 + lane;
                len[i] = b < p.batch && seq[i] >= 0 && seq[i] < p.c.seqs ? p.c.lens[seq[i]] : 0;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (g0 + i >= groups) break;
                const int b = (g0 + i) * 32 + lane;
                const int sum = __reduce_add_sync(
                    0xffffffffu, b < p.batch ? units_in<RUN>(row_from<RUN>(p, seq[i], len[i], &bad)) : 0);
                if ((g0 + i) / per == lane) mine += sum;
            }
        }
    }
    if (blockIdx.x == 0 && threadIdx.x < 32) flag(p.c.status, bad);
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31) * hp;
    split->blocks = min(total, static_cast<int>(gridDim.x));
    if (static_cast<int>(blockIdx.x) >= split->blocks) return false;
    split->each = total / split->blocks;
    split->more = total - split->each * split->blocks;
    const int first = split->first_of(blockIdx.x);
    *end = split->first_of(blockIdx.x + 1);
    const int want = first / hp;          // unit of the rows' own count
    const int found = __ffs(__ballot_sync(0xffffffffu, upto > want)) - 1;
    int before = __shfl_sync(0xffffffffu, upto - mine, found);       // (groups == 1: found is the row)
    if (groups == 1) {
        at->take_row(p, found);
    } else {
        // The same for the found lane's rows, 32 at a time.
        for (int row = found * per * 32;; row += 32) {
            if (row >= p.batch) return false;                // (lengths that change during the call)
            const int units = row + lane < p.batch ? units_in<RUN>(row_of<RUN>(p, row + lane, &bad)) : 0;
            upto = units;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += o;
            }
            const unsigned past = __ballot_sync(0xffffffffu, before + upto > want);
            if (past != 0u) {
                const int i = __ffs(past) - 1;
                before += __shfl_sync(0xffffffffu, upto - units, i);
                at->take_row(p, row + i);
                break;
            }
            before += __shfl_sync(0xffffffffu, upto, 31);
        }
    }
    at->base = before * hp;
    const int into = first - at->base;
    at->hg = into / (at->tiles + 1);
    at->tile = into - at->hg * (at->tiles + 1);
    if (at->tile == at->tiles) {          // the unit after the tiles
        --at->tile;
        at->next(p, *end);
    }
    return at->unit() < *end;
}

// ---- asynchronous copies --------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_addr(const void* p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
// 16 bytes from global to shared memory; size 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy_async(unsigned dst, const void* src, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x (results below 2^-126 are 0).
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- outputs --------------------------------------------------------------------------------
// Four neighbours of an output row: o / sum (0 where nothing has weight; a NaN sum stays NaN).
template <class T>
__device__ __forceinline__ void put_out(const AttnParams& p, int b, int head, int d, float4 o,
                                        float sum) {
    const float by = sum > 0.0f ? 1.0f / sum : sum;
    T r[4] = {from_float<T>(o.x * by), from_float<T>(o.y * by), from_float<T>(o.z * by),
              from_float<T>(o.w * by)};
    T* to = static_cast<T*>(p.out) + b * p.out_batch + head * p.out_head + d;
    if (p.out_aligned) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(to) = *reinterpret_cast<uint4*>(r);
        else *reinterpret_cast<uint2*>(to) = *reinterpret_cast<uint2*>(r);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = r[i];
    }
}
// m in powers of two.
__device__ __forceinline__ void put_lse(const AttnParams& p, int b, int head, float m, float sum) {
    if (p.lse != nullptr)
        p.lse[static_cast<long long>(b) * p.q_heads + head] =
            sum == 0.0f ? kNegInf : (m + log2f(sum)) * kLn2;
}

// Rows with nothing to read: out 0, lse -inf.  A warp a row.
template <class T>
__device__ __forceinline__ void put_empty_rows(const AttnParams& p) {
    unsigned bad = 0;
    for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.batch; b += gridDim.x * kWarps) {
        if (row_of<8>(p, b, &bad).len > 0) continue;
        for (int x = 4 * (threadIdx.x & 31); x < p.q_heads * p.c.dim; x += 128) {
            const int h = x / p.c.dim, d = x - h * p.c.dim;
            put_out<T>(p, b, h, d, make_float4(0.0f, 0.0f, 0.0f, 0.0f), 0.0f);
            if (d == 0) put_lse(p, b, h, 0.0f, 0.0f);
        }
    }
}

// Joins `n` parts, values of one head: m[i], s[i], o[i].  `up` is the new reference.
template <int N>
__device__ __forceinline__ void join_parts(const float (&m)[N], const float (&s)[N],
                                           const float4 (&o)[N], float* top, float* sum,
                                           float4* acc) {
    float up = *top;
#pragma unroll
    for (int i = 0; i < N; ++i) up = fmaxf(up, m[i]);
    const float base = up == kNegInf ? 0.0f : up;
    const float w = pow2(*top - base);
    *sum *= w;
    acc->x *= w;
    acc->y *= w;
    acc->z *= w;
    acc->w *= w;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float f = pow2(m[i] - base);
        *sum = fmaf(s[i], f, *sum);
        acc->x = fmaf(o[i].x, f, acc->x);
        acc->y = fmaf(o[i].y, f, acc->y);
        acc->z = fmaf(o[i].z, f, acc->z);
        acc->w = fmaf(o[i].w, f, acc->w);
    }
    *top = up;
}

// ---- the kernel -----------------------------------------------------------------------------
// A policy P has
//   T, DP (dim rounded up), RUN (positions of a warp's share of a tile), STAGES, PER_SM (blocks
//   on an SM), HEADS (most query heads of a part), and registers of its own;
//   FULL, PARTIAL: runs of rows that fill DP, or do not, have copies of their own (48.1 us against
//     48.7 without for 32 rows of 2048 tokens with 32/8 heads of 128, and 49.3 where a run may cross
//     pages; 75.2, 78.2 and 81.6 for 1032 rows of 64 tokens);
//   AHEAD: fetch may be called during the segment before;
//   fetch(q, head_stride, heads, dim, aligned): reads the query heads of a segment;
//   begin(): takes them into use, empties max, sum and output;
//   step(stage, lo, hi, scale): the run in `stage` (K rows, then V rows), of which rows
//     lo .. hi - 1 are visible;
//   dump(o, pitch, first, heads, dim): leaves of heads first .. first + kRound - 1 (below heads)
//     the output (not divided), the reference and the sum in shared memory: a head's row of
//     pitch values is dim outputs, reference, sum.
constexpr int kRound = 8;                 // query heads that meet in shared memory at a time
template <class P>
struct Layout {
    static constexpr int kTile = kWarps * P::RUN;
    static constexpr int kRow = P::DP * static_cast<int>(sizeof(typename P::T));
    static constexpr int kHalf = P::RUN * kRow;          // bytes of a run's K, or V
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kWarp = P::STAGES * kStage;
    static constexpr int kRing = kWarps * kWarp;
    // Values between two heads of a dump: 4 more than dim (the reference, the sum, two unused), so
    // that the lanes of a store, which hold 8 dims of 4 even (or odd) heads, meet different banks.
    static __host__ __device__ constexpr int pitch(int dim) { return dim + 4; }
    static int dump(int part, int dim) {                 // bytes
        return 4 * kWarps * (part < kRound ? part : kRound) * pitch(dim);
    }
};

// What a warp's copies of one run need, found one tile ahead.
struct Pending {
    int page, row;                                       // of row 0 of the run (lane r: of row r,
                                                         // where runs cross pages)
    int lo, hi;                                          // visible rows
    int fresh;                                           // the row of the new token, or -1
    int b, hg, seq;
};

template <class P, bool APPEND>
__global__ void __launch_bounds__(kThreads, P::PER_SM)
attention_kernel(const __grid_constant__ AttnParams p) {
    using T = typename P::T;
    using L = Layout<P>;
    constexpr int V = 16 / static_cast<int>(sizeof(T));  // values of a 16-byte piece
    constexpr int CH = L::kRow / 16;                     // pieces of a row
    constexpr int STAGES = P::STAGES, RUN = P::RUN, TILE = L::kTile;
    static_assert(CH <= 64 && RUN % 8 == 0, "a lane copies one or two pieces of a row");
    extern __shared__ __align__(128) char smem[];
    float* so = reinterpret_cast<float*>(smem + L::kRing);           // [kWarps][kRound or part heads][pitch]
    __shared__ int turn;
    const int pitch = L::pitch(p.c.dim);
    const int gap = min(p.part, kRound) * pitch;         // between the warps' dumps
    int other = p.dumps == 2 ? kWarps * gap : 0;         // from this dump's place to the next one's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int dim = p.c.dim, hp = p.c.heads * p.parts;
    char* const ring = smem + warp * L::kWarp;
    const unsigned ring_at = smem_addr(ring);
    if (dim != P::DP) {                                  // the pieces that no copy writes
        for (int x = lane; x < L::kWarp / 16; x += 32)
            reinterpret_cast<uint4*>(ring)[x] = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
    }
    grid_wait();
    grid_trigger();
    Split split;
    Cursor<RUN> cur;
    int end;
    if (!find_work<RUN>(p, &split, &end, &cur)) {
        put_empty_rows<T>(p);
        return;
    }
    const int begin = cur.unit();

    // A lane copies piece c0 of every RPS-th row from r0 on (with rows of more than 32 pieces, two
    // pieces of every row).
    constexpr int RPS = CH < 32 ? 32 / CH : 1;
    const int r0 = CH < 32 ? lane / CH : 0, c0 = CH < 32 ? lane % CH : lane;
    const long long to_v = p.c.v - p.c.k;                // bytes from K to V
    const long long lane_at = (r0 * p.c.token_stride + c0 * V) * static_cast<int>(sizeof(T));
    const long long row_step = p.c.token_stride * RPS * static_cast<int>(sizeof(T));

    // The run of number j: its first position and visible rows.
    auto look_up = [&](const Cursor<RUN>& c) {
        Pending w;
        w.b = c.b;
        w.hg = c.hg;
        w.seq = c.row.seq;
        const int j = c.tile * TILE + warp * RUN;
        const bool sink = j < c.row.turn;
        const int pos = sink ? j : j - c.row.turn + c.row.from;
        w.lo = sink ? 0 : max(0, c.row.first - pos);
        w.hi = min(RUN, (sink ? c.row.sinks : c.row.len) - pos);
        w.fresh = APPEND && !sink && c.row.len - 1 - pos < RUN ? c.row.len - 1 - pos : -1;
        w.page = w.row = 0;
        const int r = p.page_runs ? 0 : lane & (RUN - 1);
        if (p.page_runs ? w.hi > 0 : r >= w.lo && r < w.hi) {
            const unsigned at = static_cast<unsigned>(pos + r);
            const unsigned col = (__umulhi(at, p.page_mul) + at) >> p.page_shift;
            w.row = static_cast<int>(at - col * static_cast<unsigned>(p.c.page));
            w.page = p.c.table[static_cast<long long>(c.row.seq) * p.c.cols + col];
        }
        return w;
    };
    auto load = [&](const Pending& w, int slot) {
        if (w.hi <= 0) return;                           // past the end
        const int head = p.parts == 1 ? w.hg : w.hg / p.parts;
        const bool ok = w.page >= 0 && w.page < p.c.pages;
        const char* const from = p.c.k + (head * p.c.head_stride +
                                          (ok ? w.page * p.c.page_stride + w.row * p.c.token_stride : 0)) *
                                             static_cast<int>(sizeof(T));
        const unsigned stage = ring_at + slot * L::kStage;
        const bool usual = p.page_runs && ok && w.lo == 0 && w.hi == RUN && w.fresh < 0;
        // The usual run: all rows, in one page.
        auto copy_rows = [&](bool mine) {
            const char* ks = from + lane_at;
            const char* vs = ks + to_v;
            const unsigned dst = stage + r0 * L::kRow;
#pragma unroll
            for (int x = 0; x < RUN / RPS; ++x) {
                const unsigned to = dst + x * RPS * L::kRow + (((c0 ^ r0) << 4) ^ (x * RPS & 7) << 4);
                if (mine) {
                    copy_async(to, ks, 16);
                    copy_async(to + L::kHalf, vs, 16);
                }
                ks += row_step;
                vs += row_step;
            }
        };
        if (P::FULL && usual && dim == P::DP) {
            copy_rows(true);
        } else if (P::PARTIAL && usual && dim != P::DP) {
            copy_rows(c0 * V < dim);
        } else if (p.page_runs) {
            if (!ok) flag(p.c.status, GS_DEV_BAD_SEQ);
            const char* src = from + lane_at;
            const unsigned dst = stage + r0 * L::kRow;
#pragma unroll
            for (int x = 0; x < RUN / RPS; ++x) {
                const int r = x * RPS + r0;
                // (c ^ (r & 7): r0 is below RPS, a power of two)
                const unsigned to = dst + x * RPS * L::kRow + (((c0 ^ r0) ^ (x * RPS & 7)) << 4);
                const int size = ok && r >= w.lo && r < w.hi ? 16 : 0;
                if (r != w.fresh) {
                    if (c0 * V < dim) {
                        copy_async(to, src, size);
                        copy_async(to + L::kHalf, src + to_v, size);
                    }
                    if (CH > 32 && (c0 + 32) * V < dim) {
                        copy_async(to + 512, src + 512, size);
                        copy_async(to + 512 + L::kHalf, src + 512 + to_v, size);
                    }
                }
                src += row_step;
            }
        } else {
            const bool mine = (lane & (RUN - 1)) >= w.lo && (lane & (RUN - 1)) < w.hi;
            if (mine && !ok) flag(p.c.status, GS_DEV_BAD_SEQ);
            const long long at = from - p.c.k;
            const int size = mine && ok ? 16 : 0;
#pragma unroll
            for (int x = 0; x < RUN * CH / 32; ++x) {
                const int r = (x * 32 + lane) / CH, c = (x * 32 + lane) % CH;
                const char* src = p.c.k + __shfl_sync(0xffffffffu, at, r) + 16 * c;
                const int sz = __shfl_sync(0xffffffffu, size, r);
                const unsigned to = stage + r * L::kRow + ((c ^ (r & 7)) << 4);
                if (c * V < dim && r != w.fresh) {
                    copy_async(to, src, sz);
                    copy_async(to + L::kHalf, src + to_v, sz);
                }
            }
        }
        if (APPEND && w.fresh >= 0) {                    // the new token's row comes from k_new, v_new
            const int r = w.fresh;
            const long long row = (from - p.c.k) + (p.page_runs ? r * p.c.token_stride * static_cast<int>(sizeof(T)) : 0);
            const int from_lane = p.page_runs ? 0 : r;
            const long long at = __shfl_sync(0xffffffffu, row, from_lane);
            const int page = __shfl_sync(0xffffffffu, ok ? w.page : -1, from_lane);
            // If the position is the token's own: the sequence got it by its last extension, its
            // length was not cut, and its page is in the pool and not shared.  Else the row is read
            // from the cache as any other.  (Asked for beside the row, so that it costs no latency
            // of its own.)
            const int len = p.c.lens[w.seq], mark = p.c.refused[w.seq];
            const int holders = page >= 0 ? p.c.refs[page] : 2;
            const bool own = holders <= 1 && len <= p.c.cols * p.c.page && !was_refused(mark, len);
            for (int c = lane; c * V < dim; c += 32) {
                const long long n = w.b * p.new_batch + head * p.new_head + c * V;
                const uint4 k = load16_any(static_cast<const T*>(p.k_new) + n, p.new_aligned != 0);
                const uint4 v = load16_any(static_cast<const T*>(p.v_new) + n, p.new_aligned != 0);
                const int off = slot * L::kStage + r * L::kRow + ((c ^ (r & 7)) << 4);
                if (own) {
                    *reinterpret_cast<uint4*>(ring + off) = k;
                    *reinterpret_cast<uint4*>(ring + off + L::kHalf) = v;
                    if (w.hg == head * p.parts) {
                        *reinterpret_cast<uint4*>(p.c.k + at + 16 * c) = k;
                        *reinterpret_cast<uint4*>(p.c.v + at + 16 * c) = v;
                    }
                } else {
                    const int size = page >= 0 ? 16 : 0;
                    copy_async(ring_at + off, p.c.k + at + 16 * c, size);
                    copy_async(ring_at + off + L::kHalf, p.c.v + at + 16 * c, size);
                    if (c == 0) flag(p.c.status, was_refused(mark, len) ? GS_DEV_NO_PAGE : GS_DEV_BAD_SEQ);
                }
            }
        }
    };

    Cursor<RUN> ahead = cur;
    Pending next[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        next[i].hi = 0;
        if (ahead.unit() < end) {
            next[i] = look_up(ahead);
            ahead.next(p, end);
        }
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        load(next[i], i);
        copy_commit();
    }
    Pending pending = next[STAGES - 1];
    put_empty_rows<T>(p);
    int slot = 0;
    P work;
    bool fresh = true, fetched = false;
    while (cur.unit() < end) {
        const int head = p.parts == 1 ? cur.hg : cur.hg / p.parts;
        const int part = cur.hg - head * p.parts;
        const int first_head = head * p.group + part * p.part;
        const int heads = min(p.part, p.group - part * p.part);
        if (fresh) {
            const T* const q = static_cast<const T*>(p.q) + cur.b * p.q_batch;
            if (!fetched) work.fetch(q + first_head * p.q_head, p.q_head, heads, dim, p.q_aligned != 0);
            work.begin();
            fresh = fetched = false;
            // The next segment's query heads, where it belongs to the same row.
            if (P::AHEAD && cur.hg + 1 < hp && cur.item() + cur.tiles + 1 < end) {
                const int next_head = p.parts == 1 ? cur.hg + 1 : (cur.hg + 1) / p.parts;
                const int next_part = cur.hg + 1 - next_head * p.parts;
                work.fetch(q + (next_head * p.group + next_part * p.part) * p.q_head, p.q_head,
                           min(p.part, p.group - next_part * p.part), dim, p.q_aligned != 0);
                fetched = true;
            }
        }
        copy_wait<STAGES - 2>();
        __syncwarp();
        load(pending, slot == 0 ? STAGES - 1 : slot - 1);
        copy_commit();
        pending.hi = 0;
        if (ahead.unit() < end) {
            pending = look_up(ahead);
            ahead.next(p, end);
        }
        const int j = cur.tile * TILE + warp * RUN;
        const bool sink = j < cur.row.turn;
        const int pos = sink ? j : j - cur.row.turn + cur.row.from;
        const int hi = min(RUN, (sink ? cur.row.sinks : cur.row.len) - pos);
        if (hi > 0)
            work.step(ring + slot * L::kStage, sink ? 0 : max(0, cur.row.first - pos), hi, p.scale_log2);
        slot = slot + 1 == STAGES ? 0 : slot + 1;

        if (cur.unit() + 1 == end || cur.tile + 1 == cur.tiles) {    // the segment's end
            const int a = cur.item();
            const bool whole = a >= begin && a + cur.tiles <= end;
            const int item = cur.b * hp + cur.hg;
            const long long size = slot_size(p.part, dim);
            // Slot 0 of a block for the segment it begins with, slot 1 for a later one.
            float* const mine = p.slots + (2 * blockIdx.x + (a <= begin ? 0 : 1)) * size;
#pragma unroll
            for (int h0 = 0; h0 < P::HEADS; h0 += kRound) {
                if (h0 >= heads) break;
                work.dump(so + warp * gap, pitch, h0, heads, dim);
                __syncthreads();
                for (int x = 4 * threadIdx.x; x < min(kRound, heads - h0) * dim; x += 4 * kThreads) {
                    const int h = static_cast<int>(x * p.dim_mul >> 20);
                    float m[kWarps], s[kWarps], top = kNegInf, sum = 0.0f;
                    float4 o[kWarps], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float* from = so + w * gap + h * pitch;
                        const float2 f = *reinterpret_cast<const float2*>(from + dim);
                        m[w] = f.x;
                        s[w] = f.y;
                        o[w] = *reinterpret_cast<const float4*>(from + (x - h * dim));
                    }
                    join_parts(m, s, o, &top, &sum, &acc);
                    if (whole) {
                        put_out<T>(p, cur.b, first_head + h0 + h, x - h * dim, acc, sum);
                        if (x == h * dim) put_lse(p, cur.b, first_head + h0 + h, top, sum);
                    } else {
                        __stcg(reinterpret_cast<float4*>(mine + slot_head(p.part) + h0 * dim + x), acc);
                        if (x == h * dim) {
                            __stcg(mine + h0 + h, top);
                            __stcg(mine + p.part + h0 + h, sum);
                        }
                    }
                }
                // The next dump overwrites this one, or (two places) the one before it, which every
                // thread was done with before the barrier above.
                if (other == 0) __syncthreads();
                so += other;
                other = -other;
            }
            if (!whole) {
                const int lo = split.block_of(a);
                const int n = split.block_of(a + cur.tiles - 1) - lo + 1;
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) {
                    const int last = atomicAdd(p.arrived + item, 1) == n - 1 ? 1 : 0;
                    if (last) p.arrived[item] = 0;       // as the next call finds it
                    __threadfence();
                    turn = last;
                }
                __syncthreads();
                if (turn != 0) {
                    // (block lo begins with this item where its first unit is the item's, or the one before it)
                    const float* first = p.slots + (2 * lo + (split.first_of(lo) >= a - 1 ? 0 : 1)) * size;
                    const float* rest = p.slots + 2 * static_cast<long long>(lo) * size;
                    for (int x = 4 * threadIdx.x; x < heads * dim; x += 4 * kThreads) {
                        const int h = x / dim;
                        float top = kNegInf, sum = 0.0f;
                        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        constexpr int N = 8;             // parts whose loads are in flight
                        for (int i0 = 0; i0 < n; i0 += N) {
                            float m[N], s[N];
                            float4 o[N];
#pragma unroll
                            for (int i = 0; i < N; ++i) {
                                const float* from = i0 + i == 0 ? first : rest + 2ll * (i0 + i) * size;
                                m[i] = kNegInf;
                                s[i] = 0.0f;
                                o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (i0 + i < n) {
                                    m[i] = __ldcg(from + h);
                                    s[i] = __ldcg(from + p.part + h);
                                    o[i] = __ldcg(reinterpret_cast<const float4*>(
                                        from + slot_head(p.part) + x));
                                }
                            }
                            join_parts(m, s, o, &top, &sum, &acc);
                        }
                        put_out<T>(p, cur.b, first_head + h, x - h * dim, acc, sum);
                        if (x == h * dim) put_lse(p, cur.b, first_head + h, top, sum);
                    }
                }
            }
            fresh = true;
        }
        cur.next(p, end);
    }
    copy_wait<0>();
}

template <class P>
gs_status launch_policy(const AttnParams& p, int blocks, gs_stream stream) {
    // Two places for a segment's end (which saves a barrier: 7.6 -> 7.5 us for the smallest calls,
    // 75.8 -> 75.1 for 1032 rows of 64 tokens) where PER_SM blocks then still share an SM (228 KB,
    // 1 KB a block for the system); else one.
    const int dump = Layout<P>::dump(p.part, p.c.dim);
    constexpr int most = 228 * 1024 / P::PER_SM - 1024 - 64;
    static_assert(Layout<P>::kRing < most, "the ring fits");
    AttnParams a = p;
    a.dumps = Layout<P>::kRing + 2 * dump <= most ? 2 : 1;
    const int smem = Layout<P>::kRing + a.dumps * dump;
    const dim3 grid(static_cast<unsigned>(blocks));
    // Calls without new tokens have an instance without their code (1032 rows of 64 tokens 74.9 us, and
    // 81.0 in one instance for both; 32 rows of 2048 in fp32, 32/8 heads of 64: 61.2 and 74.7; with new
    // tokens no difference: 51.7 us for 32 ragged rows).
    if (p.k_new == nullptr) {
        if (!allow_smem<attention_kernel<P, false>>(smem)) return GS_ERR_CUDA;
        return launch(attention_kernel<P, false>, grid, kThreads, smem, 1, stream, a);
    }
    if (!allow_smem<attention_kernel<P, true>>(smem)) return GS_ERR_CUDA;
    return launch(attention_kernel<P, true>, grid, kThreads, smem, 1, stream, a);
}

// How the query heads of a kv head (group) are served: positions of a tile, parts of the group
// and heads of a part, blocks resident on an SM.
struct Serves {
    int tile, parts, part, per_sm;
};
template <class P>
Serves serves_by(int group) {
    const int parts = (group + P::HEADS - 1) / P::HEADS;
    return {Layout<P>::kTile, parts, (group + parts - 1) / parts, P::PER_SM};
}
Serves fp32_serves(int dim, int group);
Serves mma_serves(int dim, int group);
gs_status launch_fp32(const AttnParams& p, int blocks, gs_stream stream);
gs_status launch_mma(int dtype, const AttnParams& p, int blocks, gs_stream stream);

}  // namespace gs_decode
