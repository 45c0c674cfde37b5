// Pages of a key-value cache: extend, fork, free, compact, and the copies they cause (sm_103a).
//
// The bookkeeping of one call (which pages are free, who gets which) is small: a few words
// a sequence and one word a page.  It runs in one block where both are few (one_block), else in
// one cluster of 8 blocks, so that the counts of the pages are read by eighths, without a
// grid-wide pass: each block counts the free pages of its eighth, the numbers are exchanged
// through distributed shared memory, and each block then hands out its own free pages by rank.
// The rank of a free page decides which entry of the list takes it, so the outcome does not
// depend on timing.  (A thread keeps what it read of its first 32 pages; pages beyond them are
// read a second time, and a compaction reads every count three times.)
//
// The copies (fork: the filled rows of a partly filled page; compact: whole pages) are a
// second kernel over a list that the first one leaves in the workspace, launched without the
// host knowing the list's length.  It is bound by HBM: each byte is read once and written once.
//
// Measured on a GB300 (graph replay): 64 forks of 32 layers of 8 heads of 64 x 128 bf16 pages, half
// filled (426 MB read and written), 76.3 us, of which the copies take 65 (97 % of the measured copy
// rate); compacting 1024 of 4096 pages of 4 layers (537 MB) 88 us (90 %); 24 prompts of 12.8k
// tokens in all freed, extended and written in 2 layers (210 MB) 48 us (64 %): 39 of them the two
// writes, of which looking whether a page is shared before storing into it is 1, 8 the
// bookkeeping.  That is a chain of DRAM latencies (list, lengths, tables, counts) and of cluster
// barriers: a fork or an extension of a few pages takes 4 to 6 us.
#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kCluster = 8;              // blocks of the bookkeeping's cluster, or one
constexpr int kMeta = 512;               // threads of a bookkeeping block
constexpr int kCopy = 256;               // threads of a copy block
constexpr int kNone = 0x7fffffff;
constexpr int kOnePages = 1024, kOneCells = 512;     // of a pool and a list that one block keeps

struct Copy {
    int from, to, tokens, pad;
};
__device__ __forceinline__ Copy* copies_of(int* work) { return reinterpret_cast<Copy*>(work + 4); }

__device__ __forceinline__ int pages_of(int len, int page) { return (len + page - 1) / page; }

// The bookkeeping's blocks as one.
template <int BLOCKS>
__device__ __forceinline__ int rank_in() {
    return BLOCKS == 1 ? 0 : static_cast<int>(cluster_rank());
}
template <int BLOCKS>
__device__ __forceinline__ void sync_all() {
    if (BLOCKS == 1) __syncthreads();
    else cluster_sync();
}

// Which pages of this block's eighth [lo, hi) are free.  A thread has every kMeta-th; it keeps the
// first 32 of them, so that they are read once.
struct Eighth {
    int lo, hi;
    unsigned kept;

    __device__ __forceinline__ bool read(const CacheView& c, int p) const {
        return p < hi && __ldcg(c.refs + p) == 0;
    }
    __device__ __forceinline__ int count(const CacheView& c) {
        int n = 0;
        kept = 0u;
#pragma unroll 4
        for (int k = 0; lo + k * kMeta < hi; ++k) {
            const bool f = read(c, lo + k * kMeta + static_cast<int>(threadIdx.x));
            if (k < 32 && f) kept |= 1u << k;
            n += f ? 1 : 0;
        }
        return n;
    }
    // Page k of this thread (before anything of the eighth beyond the pages already asked about
    // is handed out).
    __device__ __forceinline__ bool free_at(const CacheView& c, int k) const {
        return k < 32 ? (kept >> k & 1u) != 0u : read(c, lo + k * kMeta + static_cast<int>(threadIdx.x));
    }
};

// Counts the free pages: avail = of the whole cluster, before = of the lower blocks.  Contains
// two cluster barriers; `mine` is read by the other blocks until the second.
template <int BLOCKS>
__device__ __forceinline__ void count_free(const CacheView& c, Eighth* e, int* mine, int* tmp,
                                           int* avail, int* before) {
    const long long rank = BLOCKS == 1 ? 0 : cluster_rank();
    e->lo = static_cast<int>(c.pages * rank / BLOCKS);
    e->hi = static_cast<int>(c.pages * (rank + 1) / BLOCKS);
    int total;
    block_scan<kMeta>(e->count(c), tmp, &total);
    if (BLOCKS == 1) {
        *avail = total;
        *before = 0;
        return;
    }
    if (threadIdx.x == 0) *mine = total;
    cluster_sync();
    int a = 0, b = 0;
#pragma unroll
    for (int r = 0; r < BLOCKS; ++r) {
        const int v = cluster_read(mine, static_cast<unsigned>(r));
        a += v;
        if (r < rank) b += v;
    }
    *avail = a;
    *before = b;
    cluster_sync();
}

// The last i in [0, n) with at[i] <= r (at rises, at[0] = 0).
__device__ __forceinline__ int owner_of(const int* at, int n, int r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= r) lo = mid; else hi = mid;
    }
    return lo;
}

// at[i] = the sum of need(0) .. need(i - 1), held at `cap` at most; returns the sum of all, held
// likewise.  Ends with a barrier.
template <class F>
__device__ __forceinline__ int prefix_of(F need, int* at, int n, int cap, long long* tmp) {
    long long carry = 0;
    for (int i0 = 0; i0 < n; i0 += kMeta) {
        const int i = i0 + static_cast<int>(threadIdx.x);
        long long total;
        const long long ex =
            carry + block_scan<kMeta>(i < n ? static_cast<long long>(need(i)) : 0ll, tmp, &total);
        if (i < n) at[i] = static_cast<int>(ex < cap ? ex : cap);
        carry += total;
    }
    __syncthreads();
    return static_cast<int>(carry < cap ? carry : cap);
}

// Takes the list into shared memory and finds the first entry that names each sequence (kNone:
// none).  Ends with a barrier.
__device__ __forceinline__ void mark_first(int* mark, int seqs, const int* list, int* kept, int n) {
    for (int s = threadIdx.x; s < seqs; s += kMeta) mark[s] = kNone;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kMeta) {
        const int s = list[i];
        kept[i] = s;
        if (s >= 0 && s < seqs) atomicMin(mark + s, i);
    }
    __syncthreads();
}

template <int BLOCKS>
__global__ void __launch_bounds__(kMeta)
extend_kernel(CacheView c, const int* seq, const int* add, int n) {
    extern __shared__ int smem[];
    int* mark = smem;                    // [seqs]
    int* need = mark + c.seqs;           // [n] pages wanted
    int* held = need + n;                // [n] pages held, -1: not to be served
    int* at = held + n;                  // [n] pages wanted by the entries before
    int* ids = at + n;                   // [n] seq
    __shared__ long long tmp64[kMeta / 32 + 1];
    __shared__ int tmp[kMeta / 32 + 1];
    __shared__ int mine;
    grid_wait();
    grid_trigger();
    mark_first(mark, c.seqs, seq, ids, n);
    const bool first_block = rank_in<BLOCKS>() == 0;
    for (int i = threadIdx.x; i < n; i += kMeta) {
        const int s = ids[i];
        const int more = add != nullptr ? add[i] : 1;
        int want = 0, have = -1;
        if (s >= 0 && s < c.seqs && mark[s] == i && more >= 0) {
            const int len = __ldcg(c.lens + s);
            const long long total = static_cast<long long>(len) + more;
            if (len < 0 || len > c.cols * c.page) {
                if (first_block) flag(c.status, GS_DEV_BAD_SEQ);
            } else if (total > static_cast<long long>(c.cols) * c.page) {
                if (first_block) {
                    flag(c.status, GS_DEV_NO_PAGE);
                    c.refused[s] = len + 1;
                }
            } else {
                have = pages_of(len, c.page);
                want = pages_of(static_cast<int>(total), c.page) - have;
            }
        } else if (first_block) {
            flag(c.status, GS_DEV_BAD_SEQ);
        }
        need[i] = want;
        held[i] = have;
    }
    __syncthreads();
    const int total = prefix_of([&](int i) { return need[i]; }, at, n, c.pages + 1, tmp64);
    int avail = 0;
    if (total > 0) {
        int rank;
        Eighth e;
        count_free<BLOCKS>(c, &e, &mine, tmp, &avail, &rank);
        const int end = total < avail ? total : avail;
        for (int k = 0; e.lo + k * kMeta < e.hi && rank < end; ++k) {
            const int p = e.lo + k * kMeta + static_cast<int>(threadIdx.x);
            const int is_free = e.free_at(c, k) ? 1 : 0;
            int found;
            const int r = rank + block_scan<kMeta>(is_free, tmp, &found);
            rank += found;
            if (is_free && r < end) {
                const int i = owner_of(at, n, r);
                if (at[i] + need[i] <= avail) {
                    c.table[static_cast<long long>(ids[i]) * c.cols + held[i] + (r - at[i])] = p;
                    c.refs[p] = 1;
                }
            }
        }
    } else {
        sync_all<BLOCKS>();                  // every block has read the lengths
    }
    for (int i = rank_in<BLOCKS>() * kMeta + threadIdx.x; i < n; i += BLOCKS * kMeta) {
        if (held[i] < 0) continue;
        const int s = ids[i], more = add != nullptr ? add[i] : 1;
        if (need[i] == 0 || at[i] + need[i] <= avail) {
            c.lens[s] += more;
            if (more > 0) c.refused[s] = 0;
        } else {
            c.refused[s] = c.lens[s] + 1;
            flag(c.status, GS_DEV_NO_PAGE);
        }
    }
}

template <int BLOCKS>
__global__ void __launch_bounds__(kMeta)
fork_kernel(CacheView c, const int* src, const int* dst, int n) {
    extern __shared__ int smem[];
    int* mark = smem;                    // [seqs]
    int* from = mark + c.seqs;           // [n] length of src, -1: pair refused
    int* old = from + n;                 // [n] length of dst
    int* at = old + n;                   // [n] pairs before that need a page
    int* srcs = at + n;                  // [n]
    int* dsts = srcs + n;                // [n]
    __shared__ long long tmp64[kMeta / 32 + 1];
    __shared__ int tmp[kMeta / 32 + 1];
    __shared__ int mine;
    grid_wait();
    grid_trigger();
    mark_first(mark, c.seqs, dst, dsts, n);
    const bool first_block = rank_in<BLOCKS>() == 0;
    const int most = c.cols * c.page;
    for (int i = threadIdx.x; i < n; i += kMeta) {
        const int s = src[i], d = dsts[i];
        int len = -1, was = 0;
        if (s >= 0 && s < c.seqs && d >= 0 && d < c.seqs && mark[d] == i && mark[s] == kNone) {
            len = __ldcg(c.lens + s);
            was = __ldcg(c.lens + d);
            if (len < 0 || len > most || was < 0 || was > most) len = -1;
        }
        if (len < 0 && first_block) flag(c.status, GS_DEV_BAD_SEQ);
        from[i] = len;
        old[i] = was;
        srcs[i] = s;
    }
    __syncthreads();
    // A pair needs a page where src's last page is partly filled.
    auto need = [&](int i) { return from[i] > 0 && from[i] % c.page != 0 ? 1 : 0; };
    const int total = prefix_of(need, at, n, c.pages + 1, tmp64);
    // Release what the destinations hold, share the sources' full pages.
    const int self = rank_in<BLOCKS>() * kMeta + threadIdx.x;
    const long long cells = static_cast<long long>(n) * c.cols;
    for (long long q = self; q < cells; q += BLOCKS * kMeta) {
        const int i = static_cast<int>(q / c.cols), j = static_cast<int>(q % c.cols);
        if (from[i] < 0) continue;
        const bool release = j < pages_of(old[i], c.page), share = j < from[i] / c.page;
        int p = 0, r = 0;
        if (release) p = __ldcg(c.table + static_cast<long long>(dsts[i]) * c.cols + j);
        if (share) r = __ldcg(c.table + static_cast<long long>(srcs[i]) * c.cols + j);
        if (release) {
            if (p >= 0 && p < c.pages) atomicSub(c.refs + p, 1);
            else flag(c.status, GS_DEV_BAD_SEQ);
        }
        if (share) {
            if (r >= 0 && r < c.pages) atomicAdd(c.refs + r, 1);
            else flag(c.status, GS_DEV_BAD_SEQ);
        }
    }
    sync_all<BLOCKS>();
    int avail = 0;
    if (total > 0) {
        int rank;
        Eighth e;
        count_free<BLOCKS>(c, &e, &mine, tmp, &avail, &rank);
        const int end = total < avail ? total : avail;
        for (int k = 0; e.lo + k * kMeta < e.hi && rank < end; ++k) {
            const int p = e.lo + k * kMeta + static_cast<int>(threadIdx.x);
            const int is_free = e.free_at(c, k) ? 1 : 0;
            int found;
            const int r = rank + block_scan<kMeta>(is_free, tmp, &found);
            rank += found;
            if (is_free && r < end) {
                const int i = owner_of(at, n, r);
                const int col = from[i] / c.page;
                const int last = __ldcg(c.table + static_cast<long long>(srcs[i]) * c.cols + col);
                Copy w;
                w.from = last;
                w.to = p;
                w.tokens = last >= 0 && last < c.pages ? from[i] % c.page : 0;
                if (w.tokens == 0) flag(c.status, GS_DEV_BAD_SEQ);
                w.pad = 0;
                copies_of(c.work)[r] = w;
                c.table[static_cast<long long>(dsts[i]) * c.cols + col] = p;
                c.refs[p] = 1;
            }
        }
    }
    if (self == 0) c.work[0] = total < avail ? total : avail;
    for (long long q = self; q < cells; q += BLOCKS * kMeta) {
        const int i = static_cast<int>(q / c.cols), j = static_cast<int>(q % c.cols);
        if (from[i] < 0) continue;
        const int full = from[i] / c.page;
        const bool served = need(i) == 0 || at[i] < avail;
        if (j == 0) {
            c.lens[dsts[i]] = served ? from[i] : 0;
            c.refused[dsts[i]] = 0;
            if (!served) flag(c.status, GS_DEV_NO_PAGE);
        }
        int* to = c.table + static_cast<long long>(dsts[i]) * c.cols + j;
        int p = -1;
        if (j < full) {
            p = __ldcg(c.table + static_cast<long long>(srcs[i]) * c.cols + j);
            if (!served) {
                if (p >= 0 && p < c.pages) atomicSub(c.refs + p, 1);
                p = -1;
            }
        } else if (j == full && need(i) != 0 && served) {
            continue;                    // the page taken above
        }
        *to = p;
    }
    sync_all<BLOCKS>();                      // no block ends while another reads its count
}

// One warp a listed sequence.  Its length is taken once (atomicCAS), so that a second listing
// finds nothing to release; one outside its range stays.
__global__ void __launch_bounds__(128) free_kernel(CacheView c, const int* seq, int n) {
    grid_wait();
    grid_trigger();
    const int i = (blockIdx.x * 128 + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (i >= n) return;
    const int s = seq[i];
    if (s < 0 || s >= c.seqs) {
        if (lane == 0) flag(c.status, GS_DEV_BAD_SEQ);
        return;
    }
    int len = 0;
    if (lane == 0) {
        len = c.lens[s];
        if (len < 0 || len > c.cols * c.page) {
            flag(c.status, GS_DEV_BAD_SEQ);
            len = 0;
        } else if (c.refused != nullptr) {
            c.refused[s] = 0;
        }
        if (len > 0 && atomicCAS(c.lens + s, len, 0) != len) len = 0;
    }
    len = __shfl_sync(0xffffffffu, len, 0);
    const int held = pages_of(len, c.page);
    int* row = c.table + static_cast<long long>(s) * c.cols;
    for (int j = lane; j < held; j += 32) {
        const int p = row[j];
        if (p >= 0 && p < c.pages) atomicSub(c.refs + p, 1);
        else flag(c.status, GS_DEV_BAD_SEQ);
        row[j] = -1;
    }
}

// n = held pages.  The k-th lowest free page below n (rank among the free pages: k) takes the
// k-th highest held page (n - 1 - held pages before it = k).  The counts of the moved pages go
// through the list, so that refs_out may be refs.
template <int BLOCKS>
__global__ void __launch_bounds__(kMeta)
compact_kernel(CacheView c, int* refs_out, int* live_out) {
    __shared__ int tmp[kMeta / 32 + 1];
    __shared__ int mine;
    grid_wait();
    grid_trigger();
    int avail, before;
    Eighth e;
    count_free<BLOCKS>(c, &e, &mine, tmp, &avail, &before);
    const int lo = e.lo, hi = e.hi;
    const int live = c.pages - avail;
    Copy* copies = copies_of(c.work);
    int* rank_of = c.work + 4 + 4 * static_cast<long long>(c.pages > c.seqs ? c.pages : c.seqs);
    int moved = 0;
    for (int p0 = lo; p0 < hi; p0 += kMeta) {
        const int p = p0 + static_cast<int>(threadIdx.x);
        const int count = p < hi ? __ldcg(c.refs + p) : 1;
        int found;
        const int f = before + block_scan<kMeta>(count == 0 ? 1 : 0, tmp, &found);   // free before p
        before += found;
        if (p < hi) {
            if (count == 0 && p < live) {
                copies[f].to = p;                               // filled below
            } else if (count != 0 && p >= live) {
                const int k = live - 1 - (p - f);
                copies[k].from = p;
                copies[k].tokens = c.page;
                copies[k].pad = count;
                rank_of[p] = k;
                ++moved;
            } else if (p >= live) {
                rank_of[p] = -1;                                // free: no table should name it
            }
        }
    }
    int total;
    block_scan<kMeta>(moved, tmp, &total);
    if (threadIdx.x == 0) mine = total;
    sync_all<BLOCKS>();
    int all = BLOCKS == 1 ? total : 0;
    if (BLOCKS > 1) {
#pragma unroll
        for (unsigned r = 0; r < BLOCKS; ++r) all += cluster_read(&mine, r);
    }
    if (rank_in<BLOCKS>() == 0 && threadIdx.x == 0) {
        c.work[0] = all;
        c.work[1] = live;
        if (live_out != nullptr) *live_out = live;
    }
    // Counts: what stays is copied, what is above n is 0; then the moved pages' counts.
    for (int p = lo + static_cast<int>(threadIdx.x); p < hi; p += kMeta) {
        const int count = __ldcg(c.refs + p);
        if (p >= live) refs_out[p] = 0;
        else if (count != 0) refs_out[p] = count;
    }
    for (int k = rank_in<BLOCKS>() * kMeta + threadIdx.x; k < all; k += BLOCKS * kMeta) {
        const int4 w = __ldcg(reinterpret_cast<const int4*>(copies + k));
        refs_out[w.y] = w.w;
    }
    sync_all<BLOCKS>();
}

constexpr int kUnit = 512;               // vectors a copying warp takes at a time, at most: 8 KB (a
                                         // head's page whole: 33 us instead of 15 for a few of 128 KB)
__host__ __device__ inline int pieces_of(int vecs) { return (vecs + kUnit - 1) / kUnit; }

// The listed copies: a warp takes up to 512 vectors of 16 bytes (kUnit) of one head of one page of
// one layer of K or V at a time, 8 a lane in flight.  DENSE: a head's rows lie next to each other (64 forks
// 75.5 us, and 80.5 us by rows; compacting 86.9 and 91.8).  With REMAP
// the table's entries are renumbered too (compact).
template <bool REMAP, bool DENSE>
__global__ void __launch_bounds__(kCopy)
copy_kernel(CacheView c, int es, int* table_out) {
    grid_wait();
    grid_trigger();
    const int count = c.work[0];
    const int4* const copies = reinterpret_cast<const int4*>(copies_of(c.work));
    if constexpr (REMAP) {
        const int live = c.work[1];
        const int* rank_of = c.work + 4 + 4 * static_cast<long long>(c.pages > c.seqs ? c.pages : c.seqs);
        const long long cells = static_cast<long long>(c.seqs) * c.cols;
        for (long long q = static_cast<long long>(blockIdx.x) * kCopy + threadIdx.x; q < cells;
             q += static_cast<long long>(gridDim.x) * kCopy) {
            int p = c.table[q];
            // Entries past a sequence's pages may hold anything: only held pages are renumbered.
            const int s = static_cast<int>(q / c.cols), j = static_cast<int>(q % c.cols);
            if (p >= live && p < c.pages && j < pages_of(c.lens[s], c.page)) {
                const int k = rank_of[p];
                if (k >= 0) p = copies[k].y;
                else flag(c.status, GS_DEV_BAD_SEQ);
            }
            table_out[q] = p;
        }
    }
    const int lane = threadIdx.x & 31;
    const int per = c.dim * es / 16;                     // vectors of a row
    const int pieces = pieces_of(c.page * per);          // of a head's page
    const long long sides = 2ll * c.layers * c.heads * pieces;           // warps' units of a copy
    const long long units = count * sides;
    const long long warps = static_cast<long long>(gridDim.x) * (kCopy / 32);
    for (long long u = static_cast<long long>(blockIdx.x) * (kCopy / 32) + (threadIdx.x >> 5); u < units;
         u += warps) {
        const int i = static_cast<int>(u / sides);
        const long long side = u - i * sides;
        const int piece = static_cast<int>(side % pieces), row_of_heads = static_cast<int>(side / pieces);
        const int head = row_of_heads % c.heads, which = row_of_heads / c.heads;
        const int4 w = copies[i];                        // from, to, tokens
        char* const base = ((which & 1) != 0 ? c.v : c.k) +
                           ((which >> 1) * c.layer_stride + head * c.head_stride) * es;
        const char* const src = base + w.x * c.page_stride * es;
        char* const dst = base + w.y * c.page_stride * es;
        const int vecs = min(w.z * per, (piece + 1) * kUnit);
        constexpr int U = 8;
        for (int v0 = piece * kUnit + lane; v0 < vecs; v0 += 32 * U) {
            uint4 r[U];
            long long off[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int v = v0 + x * 32;
                if (v < vecs) {
                    if (DENSE) {
                        off[x] = 16ll * v;
                    } else {
                        const int row = v / per;
                        off[x] = row * c.token_stride * es + 16ll * (v - row * per);
                    }
                    r[x] = __ldcs(reinterpret_cast<const uint4*>(src + off[x]));
                }
            }
#pragma unroll
            for (int x = 0; x < U; ++x)
                if (v0 + x * 32 < vecs) __stcs(reinterpret_cast<uint4*>(dst + off[x]), r[x]);
        }
    }
}

// New tokens' K and V into one layer: a warp takes up to 128 vectors of K, and of V, of one token.
// They are asked for before the token's place is looked up.
template <class T>
__global__ void __launch_bounds__(kCopy)
write_kernel(CacheView c, int layer, const T* k, const T* v,
             long long token_stride, long long head_stride, int src_aligned, int tokens,
             const int* seq, const int* start, int n) {
    extern __shared__ int first[];                       // [n + 1]: start
    grid_wait();
    grid_trigger();
    const int lane = threadIdx.x & 31;
    constexpr int E = 16 / static_cast<int>(sizeof(T)), U = 4;
    const int per = c.dim / E, vecs = c.heads * per;     // vectors of a row; of a token's K
    const int parts = (vecs + 32 * U - 1) / (32 * U);
    const unsigned unit = blockIdx.x * (kCopy / 32) + (threadIdx.x >> 5);
    const int t = parts == 1 ? static_cast<int>(unit) : static_cast<int>(unit / parts);
    const int q0 = static_cast<int>(unit - static_cast<unsigned>(t * parts)) * 32 * U + lane;
    const T* const ks = k + t * token_stride;
    const T* const vs = v + t * token_stride;
    uint4 kr[U], vr[U];
    int head[U], x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int q = q0 + i * 32;
        if (q >= vecs || t >= tokens) continue;
        head[i] = q / per;
        x[i] = (q - head[i] * per) * E;
        kr[i] = load16_any(ks + head[i] * head_stride + x[i], src_aligned != 0);
        vr[i] = load16_any(vs + head[i] * head_stride + x[i], src_aligned != 0);
    }
    for (int i = threadIdx.x; i <= n; i += kCopy) first[i] = start[i];
    __syncthreads();
    if (unit == 0 && lane == 0 && (first[0] < 0 || first[n] > tokens)) flag(c.status, GS_DEV_BAD_SEQ);
    if (t >= tokens || t < first[0] || t >= first[n]) return;
    int lo = 0, hi = n;                                  // the last i with start[i] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid;
    }
    const int s = seq[lo];
    bool ok = s >= 0 && s < c.seqs;
    unsigned why = GS_DEV_BAD_SEQ;
    long long pos = -1;
    if (ok) {
        const int len = c.lens[s], mark = c.refused[s];
        pos = static_cast<long long>(len) - (first[lo + 1] - t);
        ok = pos >= 0 && pos < len && len <= c.cols * c.page;
        if (ok && was_refused(mark, len)) {              // these are tokens that it held before
            ok = false;
            why = GS_DEV_NO_PAGE;
        }
    }
    int p = -1;
    if (ok) {
        p = c.table[static_cast<long long>(s) * c.cols + pos / c.page];
        ok = p >= 0 && p < c.pages && __ldcg(c.refs + p) <= 1;      // never into a shared page
    }
    if (!ok) {
        if (lane == 0) flag(c.status, why);
        return;
    }
    const long long at = layer * c.layer_stride + p * c.page_stride + (pos % c.page) * c.token_stride;
    T* const kd = reinterpret_cast<T*>(c.k) + at;
    T* const vd = reinterpret_cast<T*>(c.v) + at;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        if (q0 + i * 32 >= vecs) continue;
        *reinterpret_cast<uint4*>(kd + head[i] * c.head_stride + x[i]) = kr[i];
        *reinterpret_cast<uint4*>(vd + head[i] * c.head_stride + x[i]) = vr[i];
    }
}

gs_status check_call(const gs_kv_cache* cache, int32_t n, CacheView* view) {
    const gs_status st = check_cache(cache, view);
    if (st != GS_OK) return st;
    if (n < 0) return GS_ERR_INVALID_ARG;
    if (n > GS_MAX_SEQS) return GS_ERR_UNSUPPORTED;
    return GS_OK;
}

// Small pools and short lists are kept by one block, which spares the cluster's barriers: 16 forks of
// 8 pages each 7.2 us against 8.8, compacting 1024 pages 6.6 against 7.4; but 16 forks of 64 pages
// 10.7 against 9.7, compacting 4096 pages 12.3 against 8.4.
bool one_block(const CacheView& c, long long n) { return c.pages <= kOnePages && n * c.cols <= kOneCells; }

// `most` copies at most; the list's length is on the device.
template <bool REMAP>
gs_status launch_copies(const CacheView& c, int dtype, long long most, int* table_out,
                        gs_stream stream) {
    const int es = static_cast<int>(elem_size(dtype));
    const long long units = most * 2 * c.layers * c.heads * pieces_of(c.page * (c.dim * es / 16));
    long long blocks = (units + kCopy / 32 - 1) / (kCopy / 32);
    // Fewer blocks an SM leave the last units to a few warps (64 forks of the case above: 77.8 us at
    // 8, 76.3 at 16, 75.5 at 32), more cost the call that has nothing to copy (compact: 6.7, 8.0, 10.4).
    const long long full = static_cast<long long>(sm_count()) * 16;
    if (blocks > full) blocks = full;
    const dim3 grid(static_cast<unsigned>(blocks));
    return c.token_stride == c.dim || c.page == 1
               ? launch(copy_kernel<REMAP, true>, grid, kCopy, 0, 1, stream, c, es, table_out)
               : launch(copy_kernel<REMAP, false>, grid, kCopy, 0, 1, stream, c, es, table_out);
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_pages_workspace(const gs_kv_cache* cache, int64_t* bytes) {
    if (bytes == nullptr) return GS_ERR_INVALID_ARG;
    const gs_status st = check_cache_sizes(cache);
    if (st != GS_OK) return st;
    *bytes = workspace_need(cache);
    return GS_OK;
}

extern "C" gs_status gs_pages_extend(const gs_kv_cache* cache, const int32_t* seq,
                                     const int32_t* add, int32_t n, gs_stream stream) {
    CacheView c;
    gs_status st = check_call(cache, n, &c);
    if (st != GS_OK) return st;
    if (n == 0) return GS_OK;
    if (seq == nullptr) return GS_ERR_INVALID_ARG;
    st = check_workspace(cache);
    if (st != GS_OK) return st;
    const int smem = 4 * (c.seqs + 4 * n);
    if (one_block(c, n)) {
        if (!allow_smem<extend_kernel<1>>(smem)) return GS_ERR_CUDA;
        return launch(extend_kernel<1>, dim3(1), kMeta, smem, 1, stream, c, seq, add, n);
    }
    if (!allow_smem<extend_kernel<kCluster>>(smem)) return GS_ERR_CUDA;
    return launch(extend_kernel<kCluster>, dim3(kCluster), kMeta, smem, kCluster, stream, c, seq, add, n);
}

extern "C" gs_status gs_pages_fork(const gs_kv_cache* cache, const int32_t* src,
                                   const int32_t* dst, int32_t n, gs_stream stream) {
    CacheView c;
    gs_status st = check_call(cache, n, &c);
    if (st != GS_OK) return st;
    if (n == 0) return GS_OK;
    if (src == nullptr || dst == nullptr) return GS_ERR_INVALID_ARG;
    st = check_workspace(cache);
    if (st != GS_OK) return st;
    const int smem = 4 * (c.seqs + 5 * n);
    if (!allow_smem<fork_kernel<1>>(smem) || !allow_smem<fork_kernel<kCluster>>(smem)) return GS_ERR_CUDA;
    st = one_block(c, n) ? launch(fork_kernel<1>, dim3(1), kMeta, smem, 1, stream, c, src, dst, n)
                         : launch(fork_kernel<kCluster>, dim3(kCluster), kMeta, smem, kCluster, stream, c, src, dst, n);
    if (st != GS_OK) return st;
    return launch_copies<false>(c, cache->dtype, n, nullptr, stream);
}

extern "C" gs_status gs_pages_free(const gs_kv_cache* cache, const int32_t* seq, int32_t n,
                                   gs_stream stream) {
    CacheView c;
    const gs_status st = check_call(cache, n, &c);
    if (st != GS_OK) return st;
    if (n == 0) return GS_OK;
    if (seq == nullptr) return GS_ERR_INVALID_ARG;
    return launch(free_kernel, dim3(static_cast<unsigned>((n + 3) / 4)), 128, 0, 1, stream, c, seq,
                  n);
}

extern "C" gs_status gs_pages_compact(const gs_kv_cache* cache, int32_t* table_out,
                                      int32_t* refs_out, int32_t* live_out, gs_stream stream) {
    CacheView c;
    gs_status st = check_call(cache, 0, &c);
    if (st != GS_OK) return st;
    if (table_out == nullptr || refs_out == nullptr) return GS_ERR_INVALID_ARG;
    st = check_workspace(cache);
    if (st != GS_OK) return st;
    st = one_block(c, 0) ? launch(compact_kernel<1>, dim3(1), kMeta, 0, 1, stream, c, refs_out, live_out)
                         : launch(compact_kernel<kCluster>, dim3(kCluster), kMeta, 0, kCluster, stream, c,
                                  refs_out, live_out);
    if (st != GS_OK) return st;
    return launch_copies<true>(c, cache->dtype, c.pages, table_out, stream);
}

extern "C" gs_status gs_kv_write(const gs_kv_cache* cache, int32_t layer, const void* k,
                                 const void* v, int64_t token_stride, int64_t head_stride,
                                 int32_t tokens, const int32_t* seq, const int32_t* start,
                                 int32_t n, gs_stream stream) {
    CacheView c;
    gs_status st = check_call(cache, n, &c);
    if (st != GS_OK) return st;
    if (layer < 0 || layer >= c.layers || tokens < 0) return GS_ERR_INVALID_ARG;
    if (n == 0 || tokens == 0) return GS_OK;
    st = check_workspace(cache);
    if (st != GS_OK) return st;
    const long long es = elem_size(cache->dtype);
    if (k == nullptr || v == nullptr || seq == nullptr || start == nullptr ||
        !aligned(k, es) || !aligned(v, es) || token_stride < 0 || head_stride < 0)
        return GS_ERR_INVALID_ARG;
    const int vec = aligned(k, 16) && aligned(v, 16) && (token_stride * es) % 16 == 0 &&
                    (head_stride * es) % 16 == 0;
    const long long parts = (c.heads * (c.dim * es / 16) + 127) / 128;   // warps a token
    const long long blocks = (32ll * tokens * parts + kCopy - 1) / kCopy;
    if (tokens * parts > 0x7ffffff0ll) return GS_ERR_UNSUPPORTED;
    const int smem = 4 * (n + 1);
    const dim3 grid(static_cast<unsigned>(blocks));
    switch (cache->dtype) {
        case GS_DTYPE_F32:
            return launch(write_kernel<float>, grid, kCopy, smem, 1, stream, c, layer,
                          static_cast<const float*>(k), static_cast<const float*>(v), token_stride,
                          head_stride, vec, tokens, seq, start, n);
        case GS_DTYPE_BF16:
            return launch(write_kernel<__nv_bfloat16>, grid, kCopy, smem, 1, stream, c, layer,
                          static_cast<const __nv_bfloat16*>(k),
                          static_cast<const __nv_bfloat16*>(v), token_stride, head_stride, vec,
                          tokens, seq, start, n);
        default:
            return launch(write_kernel<__half>, grid, kCopy, smem, 1, stream, c, layer,
                          static_cast<const __half*>(k), static_cast<const __half*>(v),
                          token_stride, head_stride, vec, tokens, seq, start, n);
    }
}
