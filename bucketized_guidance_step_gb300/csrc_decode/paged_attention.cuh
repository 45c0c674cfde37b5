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
// Visible positions are numbered 0 .. n-1 without gaps: the first `sinks`, then the window.
#pragma once

#include "decode_common.cuh"

namespace gs_decode {

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
    int new_aligned;                      // k_new and v_new rows lie on 16 bytes
    int out_aligned;                      // out rows lie on 4 elements
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

// The split of all tiles: the first `more` blocks take each + 1, the others each.
struct Split {
    int blocks, each, more;

    __device__ __forceinline__ int first_of(int block) const {
        return block * each + min(block, more);
    }
    __device__ __forceinline__ int block_of(int tile) const {
        const int edge = more * (each + 1);
        return tile < edge ? tile / (each + 1) : more + (tile - edge) / each;
    }
};

// A place in the sequence of tiles.
template <int TILE>
struct Cursor {
    Row row;
    int b, tiles;                         // row; tiles of one head group of it
    int base;                             // number of its first tile
    int hg, tile;                         // head group (head * parts + part); tile of it

    __device__ __forceinline__ void take_row(const AttnParams& p, int row_number) {
        unsigned bad = 0;
        b = row_number;
        row = row_of(p, b, &bad);
        tiles = (row.n + TILE - 1) / TILE;
    }
    __device__ __forceinline__ void next(const AttnParams& p) {
        if (++tile < tiles) return;
        tile = 0;
        const int hp = p.c.heads * p.parts;
        if (++hg < hp) return;
        hg = 0;
        base += tiles * hp;
        do {
            if (b + 1 >= p.batch) return; // past the last tile: not used any more
            take_row(p, b + 1);
        } while (tiles == 0);
    }
};

// This block's tiles [t, t1) and the cursor at t.  Every warp finds them by itself.
template <int TILE>
__device__ __forceinline__ void find_work(const AttnParams& p, Split* split, int* t, int* t1,
                                          Cursor<TILE>* at) {
    const int lane = threadIdx.x & 31;
    const int hp = p.c.heads * p.parts;
    unsigned bad = 0;
    int all = 0;
    for (int b = lane; b < p.batch; b += 32) all += (row_of(p, b, &bad).n + TILE - 1) / TILE;
    all = __reduce_add_sync(0xffffffffu, all);
    if (blockIdx.x == 0 && threadIdx.x < 32) flag(p.c.status, bad);
    const int total = all * hp;
    split->blocks = min(total, static_cast<int>(gridDim.x));
    *t = *t1 = 0;
    if (static_cast<int>(blockIdx.x) >= split->blocks) return;
    split->each = total / split->blocks;
    split->more = total - split->each * split->blocks;
    *t = split->first_of(blockIdx.x);
    *t1 = split->first_of(blockIdx.x + 1);
    const int want = *t / hp;             // tile of the rows' own count
    int before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        const int b = b0 + lane;
        const int tiles = b < p.batch ? (row_of(p, b, &bad).n + TILE - 1) / TILE : 0;
        const int sum = __reduce_add_sync(0xffffffffu, tiles);
        if (before + sum <= want) {
            before += sum;
            continue;
        }
        int inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + inc > want);
        const int first = __ffs(past) - 1;
        before += __shfl_sync(0xffffffffu, inc - tiles, first);
        at->take_row(p, b0 + first);
        break;
    }
    at->base = before * hp;
    const int into = *t - at->base;
    at->hg = into / at->tiles;
    at->tile = into - at->hg * at->tiles;
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
        if (row_of(p, b, &bad).n > 0) continue;
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
    const float w = exp2f(*top - base);
    *sum *= w;
    acc->x *= w;
    acc->y *= w;
    acc->z *= w;
    acc->w *= w;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float f = exp2f(m[i] - base);
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
//   T, DP (dim rounded up), RUN (positions of a warp's share of a tile), STAGES, HEADS (most
//   query heads of a part), and registers of its own;
//   begin(q, head_stride, heads, dim): takes the query heads, empties max, sum and output;
//   step(stage, j, end, scale): the run in `stage` (K rows, then V rows), whose first row is
//     position j; rows from `end` on are not there;
//   dump(m, s, o, first, heads, dim): leaves reference, sum and output (not divided) of heads
//     first .. first + kRound - 1 (below heads) in shared memory.
constexpr int kRound = 8;                 // query heads that meet in shared memory at a time
template <class P>
struct Layout {
    static constexpr int kTile = kWarps * P::RUN;
    static constexpr int kRow = P::DP * static_cast<int>(sizeof(typename P::T));
    static constexpr int kHalf = P::RUN * kRow;          // bytes of a run's K, or V
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kWarp = P::STAGES * kStage;
    static constexpr int kRing = kWarps * kWarp;
    static int smem(int part, int dim) {
        return kRing + 4 * kWarps * (part < kRound ? part : kRound) * dim;
    }
};

// What a warp's copies of one tile need, found one tile ahead: of position j of its run (lane
// j), the page and the row in it.
struct Pending {
    int page, row;
    int kind;                                            // 0: zeros, 1: cached, 2: new token
    int b, hg;
};

template <class P>
__global__ void __launch_bounds__(kThreads)
attention_kernel(const __grid_constant__ AttnParams p) {
    using T = typename P::T;
    using L = Layout<P>;
    constexpr int V = 16 / static_cast<int>(sizeof(T));  // values of a 16-byte piece
    constexpr int CH = L::kRow / 16;                     // pieces of a row
    constexpr int STAGES = P::STAGES, RUN = P::RUN, TILE = L::kTile;
    extern __shared__ __align__(128) char smem[];
    float* const so = reinterpret_cast<float*>(smem + L::kRing);     // [kWarps][kRound or part heads][dim]
    __shared__ int turn;
    __shared__ float sm[kWarps][kRound], ss[kWarps][kRound];
    const int gap = min(p.part, kRound) * p.c.dim;       // between the warps' outputs
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
    put_empty_rows<T>(p);
    Split split;
    Cursor<TILE> cur;
    int t, t1;
    find_work<TILE>(p, &split, &t, &t1, &cur);
    if (t >= t1) return;
    const int t0 = t;

    auto look_up = [&](const Cursor<TILE>& c) {
        Pending w;
        w.b = c.b;
        w.hg = c.hg;
        w.page = w.row = w.kind = 0;
        const int j = c.tile * TILE + warp * RUN + (lane & (RUN - 1));
        if (j < c.row.n) {
            const int pos = position(c.row, j);
            const int col = pos / p.c.page;
            w.row = pos - col * p.c.page;
            w.page = p.c.table[static_cast<long long>(c.row.seq) * p.c.cols + col];
            w.kind = p.k_new != nullptr && pos == c.row.len - 1 ? 2 : 1;
        }
        return w;
    };
    auto load = [&](const Pending& w, int slot) {
        const int head = p.parts == 1 ? w.hg : w.hg / p.parts;
        const long long head_at = p.layer * p.c.layer_stride + head * p.c.head_stride;
        const bool ok = w.page >= 0 && w.page < p.c.pages;
        long long off = head_at;
        int size = 0;                                    // what the row's copies read of 16 bytes
        if (w.kind != 0) {
            if (ok) off += w.page * p.c.page_stride + w.row * p.c.token_stride;
            else if (lane < RUN) flag(p.c.status, GS_DEV_BAD_SEQ);
            size = w.kind == 2 ? -1 : ok ? 16 : 0;
        }
        const unsigned stage = ring_at + slot * L::kStage;
        const T* const kc = reinterpret_cast<const T*>(p.c.k);
        const T* const vc = reinterpret_cast<const T*>(p.c.v);
#pragma unroll
        for (int x = 0; x < RUN * CH / 32; ++x) {
            const int r = (x * 32 + lane) / CH, c = (x * 32 + lane) % CH;
            const long long o = __shfl_sync(0xffffffffu, off, r) + c * V;
            const int sz = __shfl_sync(0xffffffffu, size, r);
            const unsigned dst = stage + r * L::kRow + ((c ^ (r & 7)) << 4);
            if (c * V < dim && sz >= 0) {
                copy_async(dst, kc + o, sz);
                copy_async(dst + L::kHalf, vc + o, sz);
            }
        }
        const unsigned fresh = __ballot_sync(0xffffffffu, lane < RUN && w.kind == 2);
        if (fresh != 0u) {                               // the new token's row comes from k_new, v_new
            const int r = __ffs(fresh) - 1;
            const long long o = __shfl_sync(0xffffffffu, off, r);
            const bool store = __shfl_sync(0xffffffffu, ok ? 1 : 0, r) != 0 && w.hg == head * p.parts;
            for (int c = lane; c < CH; c += 32) {
                if (c * V >= dim) break;
                const long long n = w.b * p.new_batch + head * p.new_head + c * V;
                const uint4 k = load16_any(static_cast<const T*>(p.k_new) + n, p.new_aligned != 0);
                const uint4 v = load16_any(static_cast<const T*>(p.v_new) + n, p.new_aligned != 0);
                char* to = ring + slot * L::kStage + r * L::kRow + ((c ^ (r & 7)) << 4);
                *reinterpret_cast<uint4*>(to) = k;
                *reinterpret_cast<uint4*>(to + L::kHalf) = v;
                if (store) {
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.c.k) + o + c * V) = k;
                    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.c.v) + o + c * V) = v;
                }
            }
        }
    };

    Cursor<TILE> ahead = cur;
    Pending next[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        if (t + i < t1) {
            next[i] = look_up(ahead);
            ahead.next(p);
        }
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
        if (t + i < t1) load(next[i], i);
        copy_commit();
    }
    Pending pending = next[STAGES - 1];
    int slot = 0;
    P work;
    bool fresh = true;
    for (; t < t1; ++t) {
        const int head = p.parts == 1 ? cur.hg : cur.hg / p.parts;
        const int part = cur.hg - head * p.parts;
        const int first_head = head * p.group + part * p.part;
        const int heads = min(p.part, p.group - part * p.part);
        if (fresh) {
            work.begin(static_cast<const T*>(p.q) + cur.b * p.q_batch + first_head * p.q_head,
                       p.q_head, heads, dim);
            fresh = false;
        }
        copy_wait<STAGES - 2>();
        __syncwarp();
        if (t + STAGES - 1 < t1) load(pending, slot == 0 ? STAGES - 1 : slot - 1);
        copy_commit();
        if (t + STAGES < t1) {
            pending = look_up(ahead);
            ahead.next(p);
        }
        const int j = cur.tile * TILE + warp * RUN;
        if (j < cur.row.n) work.step(ring + slot * L::kStage, j, cur.row.n, p.scale_log2);
        slot = slot + 1 == STAGES ? 0 : slot + 1;

        if (t + 1 == t1 || cur.tile + 1 == cur.tiles) {  // the segment's end
            const int a = cur.base + cur.hg * cur.tiles; // the item's first tile
            const bool whole = a >= t0 && a + cur.tiles <= t1;
            const int item = cur.b * hp + cur.hg;
            const long long size = slot_size(p.part, dim);
            // Slot 0 of a block for the segment it begins with, slot 1 for a later one.
            float* const mine = p.slots + (2 * blockIdx.x + (a <= t0 ? 0 : 1)) * size;
#pragma unroll
            for (int h0 = 0; h0 < P::HEADS; h0 += kRound) {
                if (h0 >= heads) break;
                work.dump(sm[warp], ss[warp], so + warp * gap, h0, heads, dim);
                __syncthreads();
                for (int x = 4 * threadIdx.x; x < min(kRound, heads - h0) * dim; x += 4 * kThreads) {
                    const int h = x / dim;
                    float m[kWarps], s[kWarps], top = kNegInf, sum = 0.0f;
                    float4 o[kWarps], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        m[w] = sm[w][h];
                        s[w] = ss[w][h];
                        o[w] = *reinterpret_cast<const float4*>(so + w * gap + x);
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
                __syncthreads();                         // before the next dump
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
                    const float* first = p.slots + (2 * lo + (a == split.first_of(lo) ? 0 : 1)) * size;
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
        cur.next(p);
    }
    copy_wait<0>();
}

template <class P>
gs_status launch_policy(const AttnParams& p, int blocks, gs_stream stream) {
    const int smem = Layout<P>::smem(p.part, p.c.dim);
    if (!allow_smem<attention_kernel<P>>(smem)) return GS_ERR_CUDA;
    return launch(attention_kernel<P>, dim3(static_cast<unsigned>(blocks)), kThreads, smem, 1,
                  stream, p);
}

// How a policy's kernel serves a head dimension: positions of a tile, most query heads of a
// part, blocks resident on an SM.
struct Serves {
    int tile, heads, per_sm;
};
Serves fp32_serves(int dim);
Serves mma_serves(int dim);
gs_status launch_fp32(const AttnParams& p, int blocks, gs_stream stream);
gs_status launch_mma(int dtype, const AttnParams& p, int blocks, gs_stream stream);

}  // namespace gs_decode
