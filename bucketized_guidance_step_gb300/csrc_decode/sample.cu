// Sampling (sm_103a): temperature, top-k, top-p, min-p and the token from given random numbers.
//
// What the filters keep is a beginning of the row's tokens in the order of falling z (ties: rising
// index), so it is known by its last token.  A row is a cluster's; each block streams its part once and
// keeps the largest key of every 16-byte vector (keys are 32-bit numbers in the order of z).  Then
//   with top-k: a histogram of these largest keys, over 2048 equal pieces of z's range, finds a z that at
//     least k vectors reach, so at least k tokens do, and hardly more.  Only vectors that reach it are read
//     again, and their tokens above it, a list of somewhat over k, go to the first block, which sorts them
//     and has all it needs: the k-th token, the weights' sum, where top-p ends, min-p, the token.
//   with top-p alone: a histogram of the weights finds the piece of z's range in which they reach p of
//     their sum, and the tokens of that piece alone are listed and sorted; a last pass takes what is kept.
//   with neither, the last pass alone.
// Where a list would be longer than its place (many tokens of one z; k over 1024), the last token is found
// digit by digit in the keys instead: histograms of 2048, 2048 and 1024 digits count the tokens or sum
// their weights from the largest down.
//
// Weights are summed as whole numbers (units of 2^-40 of the largest weight): sums do not depend on the
// order of the additions, nor does the sorted list on the order in which blocks fill it.
#include <cmath>

#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kDigits = 2048;
constexpr int kMaxCluster = 8;
constexpr int kGroups = 4096;             // groups of vectors of a block, of which the largest key is kept
constexpr int kList = 2048, kMostK = 1024;               // tokens of a list; largest top-k that goes by one
constexpr unsigned kNone = 0x007fffffu;   // the key of -inf: such tokens, and NaN, are not kept
constexpr float kLog2e = 1.4426950408889634f;

struct SampleParams {
    int batch, vocab, cluster;
    const void* logits;
    long long row_stride;
    const float* temperature;
    const int* top_k;
    const float* top_p;
    const float* min_p;
    const float* noise;
    long long noise_stride;
    int* token;
    float* logprob;
    unsigned* status;
};

// What a block shows to its cluster.
struct Shown {
    unsigned top, bottom;                 // largest and smallest key
    unsigned long long all;               // of its share of the digits: tokens, or weights
    unsigned long long above, above_weight, here;        // what lies above the found digit; its tokens
    int digit;
    unsigned listed;                      // tokens in the first block's list
    unsigned border;                      // the last token that is kept
    int limit;
    unsigned ties;                        // tokens at the border
    float pick, sum;                      // best token of the block, and the weights it keeps
    int best;
    unsigned best_key;
    unsigned long long weight;
};

struct alignas(16) Shared {
    union {
        unsigned long long list[kList];
        struct {
            unsigned low[kDigits], high[kDigits];
        };
    };
    unsigned most[kGroups];
    unsigned count[kDigits];
    unsigned long long scan[kWarps + 1];
    unsigned long long in[kMaxCluster];
    float f[kWarps], g[kWarps];
    int i[kWarps];
    unsigned u[kWarps], v[kWarps];
    int limit;
    Shown shown;
};

__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Keys rise with z; NaN is below everything.
__device__ __forceinline__ unsigned key_of(float z) {
    z += 0.0f;                            // -0 is 0
    const unsigned u = __float_as_uint(z);
    return z != z ? 0u : u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float(key ^ ((key >> 31) != 0u ? 0x80000000u : 0xffffffffu));
}

// The word at `local` (shared memory of this block) in the block of rank r.
template <class V>
__device__ __forceinline__ V far(const V* local, unsigned r) {
    const unsigned a = static_cast<unsigned>(__cvta_generic_to_shared(local));
    unsigned b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(r));
    if constexpr (sizeof(V) == 8) {
        unsigned long long v;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(b) : "memory");
        return static_cast<V>(v);
    } else {
        unsigned v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(b) : "memory");
        return *reinterpret_cast<V*>(&v);
    }
}

// A block's part of its row: vectors v0 .. v1 - 1, counted from the 16-byte vector that holds the row's
// first value.
template <class T>
struct Part {
    static constexpr int V = 16 / static_cast<int>(sizeof(T)), AHEAD = 4;    // values; vectors in flight
    const T* row;
    int shift, vocab, v0, v1;             // values of the first vector that are not the row's
    int whole0, whole1;                   // vectors that are the row's entirely: whole0 .. whole1
    float hot;

    __device__ __forceinline__ uint4 raw(int v) const {              // (any vector, read only if whole)
        const int at = min(max(v, whole0), whole1);
        return whole0 <= whole1 ? *reinterpret_cast<const uint4*>(row + static_cast<long long>(at) * V - shift)
                                : make_uint4(0u, 0u, 0u, 0u);
    }
    // The keys of vector v, of which `r` is raw(v); 0 for what is not the row's.
    __device__ __forceinline__ void keys(int v, const uint4& r, unsigned (&k)[V]) const {
        float f[V];
        if (v >= whole0 && v <= whole1) {
            unpack16<T>(r, f);
        } else {
            const int at = v * V - shift;
#pragma unroll
            for (int i = 0; i < V; ++i)
                f[i] = at + i >= 0 && at + i < vocab ? static_cast<float>(row[at + i]) : __int_as_float(0x7fffffff);
        }
        if (hot > 0.0f && hot != 1.0f) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = __fdiv_rn(f[i], hot);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) k[i] = key_of(f[i]);
    }
    __device__ __forceinline__ void fetch(int v, unsigned (&k)[V]) const { keys(v, raw(v), k); }
    // f(key, index in the row) for the thread's values.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads * AHEAD) {
            uint4 r[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) r[a] = raw(v + a * kThreads);
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int x = v + a * kThreads;
                if (x >= v1) break;
                unsigned k[V];
                keys(x, r[a], k);
#pragma unroll
                for (int i = 0; i < V; ++i) f(k[i], x * V + i - shift);
            }
        }
    }
};

// Weights relative to the largest.
struct Weigh {
    unsigned top;
    float ref;
    __device__ __forceinline__ float weight(unsigned key) const {
        return key == top ? 1.0f : pow2((value_of(key) - ref) * kLog2e);
    }
    // In units of 2^-40, rounded.
    __device__ __forceinline__ unsigned long long units(unsigned key) const {
        return __float2ull_rn(weight(key) * 1099511627776.0f);
    }
};

// The pieces of z's range, from the largest down: the first is the largest z, the last whatever is 32 and
// more below it.
struct Pieces {
    unsigned top;
    float ref, scale;
    __device__ __forceinline__ Pieces(unsigned most, unsigned least) : top(most), ref(value_of(most)) {
        const float range = fminf(ref - value_of(least), 32.0f);
        scale = static_cast<float>(kDigits - 2) / range;
    }
    __device__ __forceinline__ int of(unsigned key) const {
        if (key == top) return 0;
        return 1 + static_cast<int>(fminf((ref - value_of(key)) * scale, static_cast<float>(kDigits - 2)));
    }
};

__device__ __forceinline__ void clear(unsigned* x, int n) {
    for (int i = threadIdx.x; i < n; i += kThreads) x[i] = 0u;
}

// Adds a weight to digit d's sum.
__device__ __forceinline__ void add_weight(Shared& s, int d, unsigned long long w) {
    const unsigned lo = static_cast<unsigned>(w);
    unsigned hi = static_cast<unsigned>(w >> 32);
    if (lo != 0u) {
        const unsigned old = atomicAdd(&s.low[d], lo);
        if (old + lo < old) ++hi;
    }
    if (hi != 0u) atomicAdd(&s.high[d], hi);
}

struct Found {
    int digit;                            // -1: the target is not reached
    unsigned long long above, above_weight, here, all;   // (all: counts, or weights, of all digits)
};

// The digit at which the counts (BY_WEIGHT false) or weights of the cluster's histograms reach `target`,
// which reach(all) names.  Called once the histograms are whole (a cluster barrier); ends with one.  WITH:
// the other sum is there too.
template <bool BY_WEIGHT, bool WITH, class R>
__device__ Found locate(Shared& s, int digits, unsigned long long before_all, unsigned long long before_weight,
                        int cluster, unsigned rank, R reach) {
    // This block's share of the digits, over all blocks.
    const int share = digits / cluster, per = (share + kThreads - 1) / kThreads;
    constexpr int MOST = kDigits / kThreads;
    unsigned count[MOST];
    unsigned long long weight[MOST], counts = 0, weights = 0;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        count[j] = 0;
        weight[j] = 0;
        const int x = threadIdx.x * per + j;
        if (j >= per || x >= share) continue;
        const int d = rank * share + x;
        for (int r = 0; r < cluster; ++r) {
            if (!BY_WEIGHT || WITH) count[j] += far(&s.count[d], r);
            if (BY_WEIGHT || WITH)
                weight[j] += (static_cast<unsigned long long>(far(&s.high[d], r)) << 32) + far(&s.low[d], r);
        }
        counts += count[j];
        weights += weight[j];
    }
    unsigned long long all, ignored;
    unsigned long long w = 0, c = 0;      // before this thread's digits
    if (!BY_WEIGHT || WITH) c = block_scan<kThreads>(counts, s.scan, BY_WEIGHT ? &ignored : &all);
    if (BY_WEIGHT || WITH) w = block_scan<kThreads>(weights, s.scan, BY_WEIGHT ? &all : &ignored);
    if (threadIdx.x == 0) {
        s.shown.all = all;
        s.shown.weight = BY_WEIGHT ? all : ignored;
        s.shown.ties = static_cast<unsigned>(BY_WEIGHT ? ignored : all);
        s.shown.digit = -1;
    }
    cluster_sync();
    Found f = {-1, 0, 0, 0, 0};
    unsigned long long earlier_w = before_weight, earlier_c = before_all;
    for (int r = 0; r < cluster; ++r) {
        f.all += far(&s.shown.all, r);
        if (r < static_cast<int>(rank)) {
            if (BY_WEIGHT || WITH) earlier_w += far(&s.shown.weight, r);
            if (!BY_WEIGHT || WITH) earlier_c += far(&s.shown.ties, r);
        }
    }
    const unsigned long long target = reach(f.all);
    c += earlier_c;
    w += earlier_w;
#pragma unroll
    for (int j = 0; j < MOST; ++j) {
        const int x = threadIdx.x * per + j;
        if (j >= per || x >= share) continue;
        const unsigned long long at = BY_WEIGHT ? w : c, mine = BY_WEIGHT ? weight[j] : count[j];
        if (at < target && at + mine >= target) {
            s.shown.digit = static_cast<int>(rank) * share + x;
            s.shown.above = c;
            s.shown.above_weight = w;
            s.shown.here = count[j];
        }
        c += count[j];
        w += weight[j];
    }
    cluster_sync();
    for (int r = 0; r < cluster; ++r) {
        const int d = far(&s.shown.digit, r);
        if (d < 0) continue;
        f.digit = d;
        f.above = far(&s.shown.above, r);
        f.above_weight = far(&s.shown.above_weight, r);
        f.here = far(&s.shown.here, r);
    }
    cluster_sync();
    return f;
}

struct Border {
    unsigned key;                         // tokens above stay, and `need` of those at it (lowest indices)
    unsigned long long need;
    unsigned long long above;             // tokens above it
    unsigned long long weight;            // their weights
};

// The border by count (BY_WEIGHT false: the token number `target` from the top) or by weight (the token at
// which the sum reaches `target`), among keys >= floor.  All blocks of the cluster; ends with a cluster
// barrier.
template <bool BY_WEIGHT, class P>
__device__ __noinline__ Border find_border(Shared& s, const P& part, const Weigh& weigh, unsigned floor,
                                           unsigned long long target, int cluster, unsigned rank) {
    Border b = {0u, 0ull, 0ull, 0ull};
    int shift = 32;
    for (int level = 0; level < 3; ++level) {
        const int bits = level == 2 ? 10 : 11, digits = 1 << bits;
        const unsigned prefix = b.key;
        shift -= bits;
        clear(s.count, digits);
        clear(s.low, digits);
        clear(s.high, digits);
        __syncthreads();
        part.each([&](unsigned key, int) {
            if (key < floor || key <= kNone) return;
            if (level > 0 && key >> (shift + bits) != prefix) return;
            const int d = digits - 1 - static_cast<int>(key >> shift & static_cast<unsigned>(digits - 1));
            atomicAdd(&s.count[d], 1u);
            add_weight(s, d, weigh.units(key));
        });
        cluster_sync();
        const Found f = locate<BY_WEIGHT, true>(s, digits, b.above, b.weight, cluster, rank,
                                                [&](unsigned long long) { return target; });
        b.key = prefix << bits;
        b.need = 0;
        if (f.digit >= 0) {
            b.key |= static_cast<unsigned>(digits - 1 - f.digit);
            b.above = f.above;
            b.weight = f.above_weight;
            b.need = f.here;
        }
    }
    // b.need: all tokens at the border.
    if (BY_WEIGHT) {
        const unsigned long long one = weigh.units(b.key), left = target - b.weight;
        if (one > 0) b.need = min(b.need, (left + one - 1) / one);
    } else {
        b.need = min(b.need, target - b.above);
    }
    return b;
}

// Of the tokens at the border, those up to the index that this returns stay.  All blocks of the cluster.
template <class P>
__device__ __noinline__ int limit_of(Shared& s, const P& part, const Border& border, int cluster, unsigned rank) {
    constexpr int V = P::V;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned mine = 0;
    part.each([&](unsigned key, int) { mine += key == border.key; });
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s.u[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        unsigned n = 0;
        for (int i = 0; i < kWarps; ++i) n += s.u[i];
        s.shown.ties = n;
    }
    cluster_sync();
    unsigned long long before = 0, here = 0;
    for (int r = 0; r < cluster; ++r) {
        const unsigned n = far(&s.shown.ties, r);
        if (r < static_cast<int>(rank)) before += n;
        else if (r == static_cast<int>(rank)) here = n;
    }
    int limit = part.vocab;
    if (border.need <= before) {
        limit = -1;
    } else if (border.need < before + here) {
        // Its place in this block: in the order of the indices, kThreads vectors at a time.
        unsigned left = static_cast<unsigned>(border.need - before);
        __syncthreads();
        if (tid == 0) s.limit = part.vocab;
        for (int v = part.v0; v < part.v1; v += kThreads) {
            unsigned key[V];
            unsigned n = 0, all;
            const bool in = v + tid < part.v1;
            if (in) {
                part.fetch(v + tid, key);
#pragma unroll
                for (int i = 0; i < V; ++i) n += key[i] == border.key;
            }
            unsigned at = block_scan<kThreads>(n, reinterpret_cast<unsigned*>(s.scan), &all);
            if (in && at < left && at + n >= left) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] == border.key && ++at == left) s.limit = (v + tid) * V + i - part.shift;
            }
            if (all >= left) break;
            left -= all;
        }
        __syncthreads();
        limit = s.limit;
    }
    cluster_sync();
    return limit;
}

// ---- lists ---------------------------------------------------------------------------------------
// A listed token: key above, the index's complement below, so that falling numbers are falling z, then
// rising indices.
__device__ __forceinline__ unsigned long long entry_of(unsigned key, int at) {
    return static_cast<unsigned long long>(key) << 32 | ~static_cast<unsigned>(at);
}
// Into the block's list.  What does not fit is counted only.
__device__ __forceinline__ void put_in_list(Shared& s, unsigned key, int at) {
    const unsigned n = atomicAdd(&s.shown.listed, 1u);
    if (n < kList) s.list[n] = entry_of(key, at);
}
// The blocks' lists in the first one's, if they fit: their tokens in all.  Called behind a cluster barrier;
// the others' lists are read until the next.
__device__ __forceinline__ unsigned gather_lists(Shared& s, int cluster, unsigned rank) {
    unsigned all = 0;
    for (int r = 0; r < cluster; ++r) all += far(&s.shown.listed, r);
    if (rank == 0 && all <= kList) {
        unsigned at = s.shown.listed;
        for (int r = 1; r < cluster; ++r) {
            const unsigned n = far(&s.shown.listed, r);
            for (unsigned i = threadIdx.x; i < n; i += kThreads) s.list[at + i] = far(&s.list[i], r);
            at += n;
        }
        __syncthreads();
    }
    return all;
}
// Falling order of the list's n entries (a block; ends with a barrier): compare and exchange in powers of two.
__device__ __noinline__ void sort_list(unsigned long long* list, int n) {
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += kThreads) list[i] = 0;
    __syncthreads();
    for (int run = 2; run <= size; run <<= 1) {
        for (int step = run >> 1; step > 0; step >>= 1) {
            for (int t = threadIdx.x; t < size / 2; t += kThreads) {
                const int i = 2 * t - (t & (step - 1));
                const unsigned long long a = list[i], b = list[i + step];
                if ((a < b) == ((i & run) == 0)) {
                    list[i] = b;
                    list[i + step] = a;
                }
            }
            // (Up to 32 apart, both of a pair are in 64 entries that one warp has.)
            if (step > 32 || (step == 1 && run >= 64)) __syncthreads();
            else __syncwarp();
        }
    }
    __syncthreads();
}

// The best of two tokens.
__device__ __forceinline__ void better(float x, int i, unsigned key, float* pick, int* best, unsigned* best_key) {
    if (x > *pick || (x == *pick && i < *best)) {
        *pick = x;
        *best = i;
        *best_key = key;
    }
}
// The block's best token and sum, in thread 0.
__device__ __forceinline__ void join_block(Shared& s, float* pick, int* best, unsigned* best_key, float* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, *pick, d);
        const int i = __shfl_xor_sync(0xffffffffu, *best, d);
        const unsigned u = __shfl_xor_sync(0xffffffffu, *best_key, d);
        *sum += __shfl_xor_sync(0xffffffffu, *sum, d);
        better(x, i, u, pick, best, best_key);
    }
    __syncthreads();
    if (lane == 0) {
        s.f[warp] = *pick;
        s.g[warp] = *sum;
        s.i[warp] = *best;
        s.u[warp] = *best_key;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) {
            *sum += s.g[w];
            better(s.f[w], s.i[w], s.u[w], pick, best, best_key);
        }
    }
}
__device__ __forceinline__ void put_token(const SampleParams& p, int b, const Weigh& weigh, int best, unsigned best_key,
                                          float sum) {
    const bool none = best == 0x7fffffff;                // (noise of NaN everywhere)
    if (none) flag(p.status, GS_DEV_EMPTY_ROW);
    if (p.token != nullptr) p.token[b] = none ? -1 : best;
    if (p.logprob != nullptr)
        p.logprob[b] = none ? kNegInf : (best_key == weigh.top ? 0.0f : value_of(best_key) - weigh.ref) - logf(sum);
}

// A token stays where the sum before it is below p of all.
__device__ __forceinline__ unsigned long long reach_of(float top_p, unsigned long long all) {
    const double reach = ceil(static_cast<double>(fmaxf(top_p, 0.0f)) * static_cast<double>(all));
    return max(1ull, min(all, static_cast<unsigned long long>(reach)));
}

// The first block, with all tokens that may stay in its list: the filters and the token.
__device__ __noinline__ void finish_list(const SampleParams& p, Shared& s, const Weigh& weigh, int b, int n, int k,
                                         float top_p, float min_p, const float* noise) {
    sort_list(s.list, n);
    const int kept = k > 0 ? min(k, n) : n;
    constexpr int PER = kList / kThreads;
    const int per = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * per;
    unsigned long long mine = 0, all, units[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        units[j] = j < per && i0 + j < kept ? weigh.units(static_cast<unsigned>(s.list[i0 + j] >> 32)) : 0;
        mine += units[j];
    }
    unsigned long long before = block_scan<kThreads>(mine, s.scan, &all);
    const unsigned long long target = top_p < 1.0f ? reach_of(top_p, all) : ~0ull;
    float pick = kNegInf, sum = 0.0f, z[PER];
    int best = 0x7fffffff, at[PER];
    unsigned best_key = 0u, key[PER];
    bool stays[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        stays[j] = j < per && i0 + j < kept;
        const unsigned long long e = stays[j] ? s.list[i0 + j] : 0;
        key[j] = static_cast<unsigned>(e >> 32);
        at[j] = static_cast<int>(~static_cast<unsigned>(e));
        const float w = stays[j] ? weigh.weight(key[j]) : 0.0f;
        stays[j] = stays[j] && before < target && (!(w < min_p) || key[j] == weigh.top);
        before += units[j];
        if (stays[j]) sum += w;
        z[j] = stays[j] && noise != nullptr ? noise[at[j]] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (stays[j]) better(value_of(key[j]) + z[j], at[j], key[j], &pick, &best, &best_key);
    join_block(s, &pick, &best, &best_key, &sum);
    if (threadIdx.x == 0) put_token(p, b, weigh, best, best_key, sum);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = p.cluster > 1 ? cluster_rank() : 0u;
    const int b = blockIdx.x / p.cluster;
    if (tid == 0) s.shown.listed = 0u;
    clear(s.count, kDigits);
    grid_wait();
    grid_trigger();
    Part<T> part;
    constexpr int V = Part<T>::V;
    const T* const row = static_cast<const T*>(p.logits) + b * p.row_stride;
    part.shift = static_cast<int>((reinterpret_cast<unsigned long long>(row) & 15ull) / sizeof(T));
    part.row = row;
    part.vocab = p.vocab;
    part.hot = p.temperature != nullptr ? p.temperature[b] : 1.0f;
    const int k = p.top_k != nullptr ? p.top_k[b] : 0;
    const float top_p = p.top_p != nullptr ? p.top_p[b] : 1.0f, min_p = p.min_p != nullptr ? p.min_p[b] : 0.0f;
    const int vectors = (p.vocab + part.shift + V - 1) / V;
    part.v0 = static_cast<int>(static_cast<long long>(vectors) * rank / p.cluster);
    part.v1 = static_cast<int>(static_cast<long long>(vectors) * (rank + 1) / p.cluster);
    part.whole0 = part.shift > 0 ? 1 : 0;
    part.whole1 = (p.vocab + part.shift) / V - 1;
    int group = 0;                        // 2^group vectors make a group
    while ((part.v1 - part.v0 - 1) >> group >= kGroups) ++group;
    const int groups = part.v1 > part.v0 ? ((part.v1 - part.v0 - 1) >> group) + 1 : 0;
    // The largest key of every group, and of the row; the smallest.
    unsigned top = 0u, bottom = 0xffffffffu;
    constexpr int AHEAD = Part<T>::AHEAD;
    for (int g = tid; g < groups; g += kThreads * AHEAD) {
        unsigned most[AHEAD] = {0u, 0u, 0u, 0u};
        for (int x = 0; x < 1 << group; ++x) {
            uint4 r[AHEAD];
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) r[a] = part.raw(part.v0 + ((g + a * kThreads) << group) + x);
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int v = part.v0 + ((g + a * kThreads) << group) + x;
                if (v >= part.v1) break;
                unsigned key[V];
                part.keys(v, r[a], key);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    most[a] = max(most[a], key[i]);
                    bottom = min(bottom, key[i] > kNone ? key[i] : 0xffffffffu);
                }
            }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
            if (g + a * kThreads < groups) s.most[g + a * kThreads] = most[a];
            top = max(top, most[a]);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bottom = __reduce_min_sync(0xffffffffu, bottom);
    if (lane == 0) {
        s.u[warp] = top;
        s.v[warp] = bottom;
    }
    __syncthreads();
    if (warp == 0) {
        top = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.u[lane] : 0u);
        bottom = __reduce_min_sync(0xffffffffu, lane < kWarps ? s.v[lane] : 0xffffffffu);
        if (lane == 0) {
            s.shown.top = top;
            s.shown.bottom = bottom;
        }
    }
    cluster_sync();
    top = 0u;
    bottom = 0xffffffffu;
    for (int r = 0; r < p.cluster; ++r) {
        top = max(top, far(&s.shown.top, r));
        bottom = min(bottom, far(&s.shown.bottom, r));
    }
    if (top <= kNone) {                   // nothing to choose from
        if (rank == 0 && tid == 0) {
            if (p.token != nullptr) p.token[b] = -1;
            if (p.logprob != nullptr) p.logprob[b] = kNegInf;
            flag(p.status, GS_DEV_EMPTY_ROW);
        }
        cluster_sync();
        return;
    }
    const Weigh weigh = {top, value_of(top)};
    const Pieces pieces(top, bottom);
    const float* const noise = p.noise != nullptr && part.hot > 0.0f ? p.noise + b * p.noise_stride : nullptr;
    const bool by_k = k > 0 && k < p.vocab, by_p = top_p < 1.0f;
    unsigned border = kNone + 1u;         // the last token that stays: everything
    int limit = p.vocab;
    bool known = !by_k && !by_p;
    if (!known && (p.vocab <= kList || (by_k && k <= kMostK))) {
        // All tokens from a z on that k tokens reach (of a short row all) to the first block.
        int last = kDigits - 1;
        bool some = true;
        if (p.vocab > kList) {
            for (int g = tid; g < groups; g += kThreads)
                if (s.most[g] > kNone) atomicAdd(&s.count[pieces.of(s.most[g])], 1u);
            cluster_sync();
            const Found f = locate<false, false>(s, kDigits, 0, 0, p.cluster, rank,
                                                 [&](unsigned long long) { return static_cast<unsigned long long>(k); });
            if (f.digit >= 0) last = f.digit;
            some = f.above + f.here <= kList;            // (else there are too many tokens for certain)
        }
        for (int g = tid; g < groups; g += kThreads) {
            if (!some || s.most[g] <= kNone || pieces.of(s.most[g]) > last) continue;
            for (int x = 0; x < 1 << group; ++x) {
                const int v = part.v0 + (g << group) + x;
                if (v >= part.v1) break;
                unsigned key[V];
                part.fetch(v, key);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i] > kNone && pieces.of(key[i]) <= last) put_in_list(s, key[i], v * V + i - part.shift);
            }
        }
        cluster_sync();
        const unsigned n = gather_lists(s, p.cluster, rank);
        if (some && n <= kList) {
            if (rank == 0) finish_list(p, s, weigh, b, static_cast<int>(n), by_k ? k : 0, top_p, min_p, noise);
            cluster_sync();               // (lists stay until they are read)
            return;
        }
        cluster_sync();
        if (tid == 0) s.shown.listed = 0u;
    }
    if (!known && !by_k) {
        // The piece in which the weights reach top_p of their sum; its tokens to the first block.
        clear(s.low, kDigits);
        clear(s.high, kDigits);
        __syncthreads();
        part.each([&](unsigned key, int) {
            if (key > kNone) add_weight(s, pieces.of(key), weigh.units(key));
        });
        cluster_sync();
        unsigned long long target = 0;
        const Found f = locate<true, false>(s, kDigits, 0, 0, p.cluster, rank, [&](unsigned long long all) {
            return target = reach_of(top_p, all);
        });
        part.each([&](unsigned key, int at) {
            if (key > kNone && pieces.of(key) == f.digit) put_in_list(s, key, at);
        });
        cluster_sync();
        const unsigned n = gather_lists(s, p.cluster, rank);
        if (n <= kList) {
            known = true;
            if (rank == 0) {
                sort_list(s.list, n);
                constexpr int PER = kList / kThreads;
                const int per = (static_cast<int>(n) + kThreads - 1) / kThreads, i0 = tid * per;
                unsigned long long mine = 0, all, units[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    units[j] = j < per && i0 + j < static_cast<int>(n) ? weigh.units(static_cast<unsigned>(s.list[i0 + j] >> 32)) : 0;
                    mine += units[j];
                }
                unsigned long long before = f.above_weight + block_scan<kThreads>(mine, s.scan, &all);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (units[j] > 0 && before < target && before + units[j] >= target) {
                        s.shown.border = static_cast<unsigned>(s.list[i0 + j] >> 32);
                        s.shown.limit = static_cast<int>(~static_cast<unsigned>(s.list[i0 + j]));
                    }
                    before += units[j];
                }
            }
            cluster_sync();
            border = far(&s.shown.border, 0);
            limit = far(&s.shown.limit, 0);
        }
        cluster_sync();
    }
    if (!known) {
        Border last = {border, ~0ull, 0ull, 0ull};
        if (by_k) {
            const Border found = find_border<false>(s, part, weigh, 0u, static_cast<unsigned long long>(k), p.cluster, rank);
            if (found.need > 0) last = found;            // (else fewer than k tokens can be chosen)
        }
        if (by_p) {
            // The sum over what top-k left.
            unsigned long long mine = 0, all;
            part.each([&](unsigned key, int) {
                if (key > last.key || (key == last.key && last.need == ~0ull)) mine += weigh.units(key);
            });
            block_scan<kThreads>(mine, s.scan, &all);
            if (tid == 0) s.shown.weight = all;
            cluster_sync();
            all = 0;
            for (int r = 0; r < p.cluster; ++r) all += far(&s.shown.weight, r);
            cluster_sync();
            if (last.need != ~0ull) all += last.need * weigh.units(last.key);
            const Border found = find_border<true>(s, part, weigh, last.key, reach_of(top_p, all), p.cluster, rank);
            if (found.key > last.key || (found.key == last.key && found.need < last.need)) last = found;
        }
        border = last.key;
        if (last.need != ~0ull) limit = limit_of(s, part, last, p.cluster, rank);
    }
    // The token, and the weights of what stays.
    float pick = kNegInf, sum = 0.0f, rest = 0.0f;       // (sum - rest: what rounding left out is kept)
    int best = 0x7fffffff;
    unsigned best_key = 0u;
    part.each([&](unsigned key, int at) {
        if (key < border || key <= kNone || (key == border && at > limit)) return;
        const float w = weigh.weight(key);
        if (w < min_p && key != top) return;
        const float y = w - rest, t = sum + y;
        rest = (t - sum) - y;
        sum = t;
        better(noise != nullptr ? value_of(key) + noise[at] : value_of(key), at, key, &pick, &best, &best_key);
    });
    join_block(s, &pick, &best, &best_key, &sum);
    if (tid == 0) {
        s.shown.pick = pick;
        s.shown.sum = sum;
        s.shown.best = best;
        s.shown.best_key = best_key;
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
        for (int r = 1; r < p.cluster; ++r) {
            sum += far(&s.shown.sum, r);
            better(far(&s.shown.pick, r), far(&s.shown.best, r), far(&s.shown.best_key, r), &pick, &best, &best_key);
        }
        put_token(p, b, weigh, best, best_key, sum);
    }
    cluster_sync();                       // (what rank 0 read stays until it is read)
}

// Blocks of a row: enough of them for every SM, but no part below 4096 tokens.
int cluster_of(const gs_sample_args* a) {
    int n = 1;
    while (n < kMaxCluster && a->vocab / n >= 8192 && static_cast<long long>(a->batch) * n < 4ll * sm_count()) n *= 2;
    return n;
}

template <class T>
gs_status launch_type(const SampleParams& p, gs_stream stream) {
    const dim3 grid(static_cast<unsigned>(p.batch) * p.cluster);
    constexpr int bytes = static_cast<int>(sizeof(Shared));
    if (!allow_smem<sample_kernel<T>>(bytes)) return GS_ERR_CUDA;
    return launch(sample_kernel<T>, grid, kThreads, bytes, p.cluster, stream, p);
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_sample(const gs_sample_args* a, gs_stream stream) {
    if (a == nullptr || a->batch < 0 || a->vocab < 1 || !known_dtype(a->dtype)) return GS_ERR_INVALID_ARG;
    if (a->batch > GS_MAX_SEQS || a->vocab > (1 << 28)) return GS_ERR_UNSUPPORTED;
    if (a->token == nullptr && a->logprob == nullptr) return GS_ERR_INVALID_ARG;
    if (a->batch == 0) return GS_OK;
    const long long es = elem_size(a->dtype);
    if (a->logits == nullptr || !aligned(a->logits, es) || (a->batch > 1 && a->row_stride < a->vocab) ||
        a->noise_stride < 0 || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) || !aligned(a->top_p, 4) ||
        !aligned(a->min_p, 4) || !aligned(a->noise, 4) || !aligned(a->token, 4) || !aligned(a->logprob, 4))
        return GS_ERR_INVALID_ARG;
    SampleParams p = {};
    p.batch = a->batch;
    p.vocab = a->vocab;
    p.cluster = cluster_of(a);
    p.logits = a->logits;
    p.row_stride = a->batch > 1 ? a->row_stride : 0;
    p.temperature = a->temperature;
    p.top_k = a->top_k;
    p.top_p = a->top_p;
    p.min_p = a->min_p;
    p.noise = a->noise;
    p.noise_stride = a->noise_stride;
    p.token = a->token;
    p.logprob = a->logprob;
    p.status = a->dev_status;
    if (a->dtype == GS_DTYPE_F32) return launch_type<float>(p, stream);
    if (a->dtype == GS_DTYPE_BF16) return launch_type<__nv_bfloat16>(p, stream);
    return launch_type<__half>(p, stream);
}
