// Sampling (sm_103a): temperature, top-k, top-p, min-p and the token from given random numbers.
//
// What the filters keep is a beginning of the row's tokens in the order of falling z (ties: rising
// index), so it is known by its last token.  A row is a cluster's; each block brings its part into shared
// memory once (a part too large is read again for each pass).  Then
//   with top-k: a histogram of the largest z of every 16-byte vector, over 2048 equal pieces of z's range,
//     finds a z that at least k vectors reach, so at least k tokens do, and hardly more.  The tokens above
//     it, a list of somewhat over k, go to the first block, which sorts them and has all it needs: the k-th
//     token, the weights' sum, where top-p ends, min-p, the token.
//   with top-p alone: a histogram of the weights finds the piece of z's range in which they reach p of
//     their sum, and the tokens of that piece alone are listed and sorted; a last pass takes what is kept.
//     (To list the first 1024 tokens as with top-k, and look whether they reach p, took longer: 28 us
//     against 26 for a row of 16384 where they do, 74 against 53 for 128 rows of 32000 where not.)
//   with neither, the last pass alone.
// Where a list would be longer than its place (many tokens of one z; k over 1024), the last token is found
// digit by digit in the keys instead: histograms of 2048, 2048 and 1024 digits count the tokens or sum
// their weights from the largest down.
//
// Weights are summed as whole numbers (units of 2^-40 of the largest weight): sums do not depend on the
// order of the additions, nor does the sorted list on the order in which blocks fill it.
//
// Measured: one row of 16384 bf16 logits 12 us with top-k 50, 22 us with top-p 0.9; 64 rows of 131072 fp32 logits 47 us
// with top-k 500, 87 us with top-p 0.9 (inputs in turn, more than L2 holds).  HBM would take 5 us of the last two: what bounds the kernel are the cluster's
// barriers and lookups in other blocks (a fifth of the issue slots are used), with top-p the shared atomics of the
// histogram, and with more rows than the GPU holds at a time (32 of 8 blocks) the last of them.
#include <cmath>

#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kDigits = 2048;
constexpr int kMaxCluster = 8;
constexpr int kHeld = 66 * 1024;          // bytes of a row that a block holds: two blocks an SM
constexpr int kList = 2048, kMostK = 1024;               // tokens of a list; largest top-k that goes by one
constexpr int kMostVocab = 1 << 23;       // (their weights' sum stays below 2^64 units)
constexpr unsigned kNone = 0x007fffffu;   // the key of -inf: such tokens are not kept
constexpr float kLog2e = 1.4426950408889634f;

struct SampleParams {
    int batch, vocab, cluster, held;      // held: the blocks hold their parts
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
    unsigned long long border;            // the last token that is kept (an entry)
    unsigned ties;                        // tokens at the border
    float pick, sum;                      // best token of the block, and the weights it keeps
    int best;
    float best_z;
    unsigned long long weight;
};

struct alignas(16) Shared {
    union {
        unsigned long long list[kList];
        struct {
            unsigned low[kDigits], high[kDigits];
        };
    };
    unsigned count[kDigits];
    unsigned long long weights[kDigits];  // of the whole row, a digit
    unsigned long long scan[kWarps + 1];
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

// Keys rise with z (which is not NaN).
__device__ __forceinline__ unsigned key_of(float z) {
    z += 0.0f;                            // -0 is 0
    const unsigned u = __float_as_uint(z);
    return u ^ (static_cast<unsigned>(static_cast<int>(u) >> 31) | 0x80000000u);
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

template <class V>
__device__ __forceinline__ void put_far(V* local, unsigned r, V v) {
    const unsigned a = static_cast<unsigned>(__cvta_generic_to_shared(local));
    unsigned b;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(r));
    if constexpr (sizeof(V) == 8) asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(b), "l"(v) : "memory");
    else asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(b), "r"(v) : "memory");
}

// A row's divisor.  Where it is usual, a product with the rounded reciprocal and one correction by its
// remainder is the correctly rounded quotient of numbers that are neither huge nor tiny (P. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor, 1990); infinities and NaN stay.
struct Divisor {
    float by, inverse;
    bool one, usual, endless;
    __device__ __forceinline__ explicit Divisor(float t) : by(t > 0.0f ? t : 1.0f), inverse(1.0f / by) {
        one = by == 1.0f;
        endless = by == __builtin_huge_valf();
        usual = by >= 0x1p-30f && by <= 0x1p30f;
    }
    template <int V>
    __device__ __forceinline__ void divide(float (&z)[V], bool any_size) const {
        if (one) return;
        bool odd = !usual;
        if (any_size) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const unsigned size = __float_as_uint(z[i]) & 0x7fffffffu;           // not 0, below 2^-60; from 2^96 on
                odd = odd || size - 1u < 0x217fffffu || (size >= 0x6f800000u && size < 0x7f800000u);
            }
        }
        if (!odd) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float q = z[i] * inverse, r = fmaf(fmaf(-q, by, z[i]), inverse, q);
                z[i] = fabsf(q) < __builtin_huge_valf() ? r : q;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = __fdiv_rn(z[i], by);
        }
    }
    __device__ __forceinline__ float of(float z) const {             // (-inf for NaN)
        float x[1] = {z};
        divide<1>(x, true);
        return fmaxf(x[0], kNegInf);
    }
};

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<unsigned>(__cvta_generic_to_shared(to))),
                 "l"(from)
                 : "memory");
}

// A block's part of its row: vectors v0 .. v1 - 1, counted from the 16-byte vector that holds the row's
// first value.  A thread has every kThreads-th.
template <class T>
struct Part {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));       // values of a vector
    const T* row;
    const uint4* from;                    // vector 0: in shared memory (held) or the row's
    int shift, vocab, v0, v1;             // values of the first vector that are not the row's
    int whole0, whole1;                   // vectors that are the row's entirely: whole0 .. whole1
    Divisor cool;

    __device__ __forceinline__ void hold(uint4* place) {
        const uint4* const far = reinterpret_cast<const uint4*>(row - shift);
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads)
            if (v >= whole0 && v <= whole1) copy16(place + (v - v0), far + v);
        asm volatile("cp.async.wait_all;" ::: "memory");
        from = place - v0;                // (a thread reads what it has copied itself)
    }
    // The largest logit of vector v as it is (a quotient's order is that of the logits); -inf for none.
    __device__ __forceinline__ float most(int v) const {
        if (cool.endless) {               // infinities become NaN: 0 where there is a finite logit
            float z[V], m = kNegInf;
            values(v, z);
#pragma unroll
            for (int i = 0; i < V; ++i) m = fmaxf(m, z[i]);
            return m;
        }
        if (v < whole0 || v > whole1) {
            float m = kNegInf;
#pragma unroll 1
            for (int i = max(0, v * V - shift); i < min(vocab, (v + 1) * V - shift); ++i) m = fmaxf(m, static_cast<float>(row[i]));
            return m;
        }
        const uint4 r = from[v];
        if constexpr (sizeof(T) == 4) {
            return fmaxf(fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)),
                               fmaxf(__uint_as_float(r.z), __uint_as_float(r.w))), kNegInf);
        } else {
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const T2 m = __hmax2(__hmax2(*reinterpret_cast<const T2*>(&r.x), *reinterpret_cast<const T2*>(&r.y)),
                                 __hmax2(*reinterpret_cast<const T2*>(&r.z), *reinterpret_cast<const T2*>(&r.w)));
            return fmaxf(fmaxf(static_cast<float>(m.x), static_cast<float>(m.y)), kNegInf);
        }
    }
    __device__ __forceinline__ float most_z(int v) const { return cool.of(most(v)); }
    // z of vector v; -inf for NaN and what is not the row's.
    __device__ __forceinline__ void values(int v, float (&z)[V]) const {
        if (v >= whole0 && v <= whole1) {
            unpack16<T>(from[v], z);
        } else {
            const int at = v * V - shift;
#pragma unroll
            for (int i = 0; i < V; ++i)
                z[i] = at + i >= 0 && at + i < vocab ? static_cast<float>(row[at + i]) : kNegInf;
        }
        cool.divide<V>(z, !std::is_same<T, __half>::value);          // (fp16 has no numbers of odd size)
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = fmaxf(z[i], kNegInf);
    }
    // f(z, index in the row of the first) for the thread's vectors that are wanted.
    template <class W, class F>
    __device__ __forceinline__ void vectors(W wanted, F f) const {
#pragma unroll 1
        for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
            if (!wanted(v)) continue;
            float z[V];
            values(v, z);
            f(z, v * V - shift);
        }
    }
    // f(z, index in the row) for the thread's values.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        vectors([](int) { return true; }, [&](const float (&z)[V], int at) {
#pragma unroll
            for (int i = 0; i < V; ++i) f(z[i], at + i);
        });
    }
};

// Weights relative to the largest: e^-d off by 2^-24 d each for d, log2 e (a quarter of that) and their product, and by
// the exponential's 2^-22.
struct Weigh {
    float ref;
    __device__ __forceinline__ float weight(float z) const { return z == ref ? 1.0f : pow2((z - ref) * kLog2e); }
    // In units of 2^-40, cut: 2^-8 in the upper word (two conversions to 32 bits, cheaper than one to 64).
    static __device__ __forceinline__ void words_of(float w, unsigned* low, unsigned* high) {
        const float a = w * 256.0f;
        *high = static_cast<unsigned>(a);
        *low = static_cast<unsigned>((a - static_cast<float>(*high)) * 4294967296.0f);
    }
    __device__ __forceinline__ unsigned long long units(float z) const {
        unsigned low, high;
        words_of(weight(z), &low, &high);
        return static_cast<unsigned long long>(high) << 32 | low;
    }
};

// The pieces of z's range, from the largest down: the first is the largest z, the last whatever is `range`
// and more below it.
struct Pieces {
    float ref, scale;
    __device__ __forceinline__ Pieces(float top, float range)
        : ref(top), scale(static_cast<float>(kDigits - 2) / range) {}
    __device__ __forceinline__ int of(float z) const {
        // (The sum's last bits are the nearest whole number.)
        const float x = fminf((ref - z) * scale, static_cast<float>(kDigits - 2)) + 8388608.0f;
        return z == ref ? 0 : 1 + (__float_as_int(x) & (kDigits - 1));
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

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

struct Found {
    int digit;                            // -1: the target is not reached
    unsigned long long above, above_weight, here, all;   // (all: counts, or weights, of all digits)
};

// The digit at which the counts (BY_WEIGHT false) or weights of the cluster's histograms reach `target`,
// which reach(all) names.  Called once the histograms are whole (a cluster barrier); nobody reads them
// afterwards, and what the blocks show stays until the next barrier.
template <bool BY_WEIGHT, class R>
__device__ Found locate(Shared& s, int digits, unsigned long long before_all, unsigned long long before_weight,
                        int cluster, unsigned rank, R reach) {
    // This block's share of the digits, over all blocks.
    const int share = digits / cluster, per = (share + kThreads - 1) / kThreads, lane = threadIdx.x & 31;
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
        unsigned n[kMaxCluster], lo[kMaxCluster], hi[kMaxCluster];   // (asked for together)
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            n[r] = r < cluster ? far(&s.count[d], r) : 0u;
            lo[r] = r < cluster ? far(&s.low[d], r) : 0u;
            hi[r] = r < cluster ? far(&s.high[d], r) : 0u;
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
            count[j] += n[r];
            weight[j] += (static_cast<unsigned long long>(hi[r]) << 32) + lo[r];
        }
        counts += count[j];
        weights += weight[j];
    }
    unsigned long long all, ignored;
    unsigned long long w = 0, c = 0;      // before this thread's digits
    c = block_scan<kThreads>(counts, s.scan, BY_WEIGHT ? &ignored : &all);
    w = block_scan<kThreads>(weights, s.scan, BY_WEIGHT ? &all : &ignored);
    if (threadIdx.x == 0) {
        s.shown.all = all;
        s.shown.weight = BY_WEIGHT ? all : ignored;
        s.shown.ties = static_cast<unsigned>(BY_WEIGHT ? ignored : all);
        s.shown.digit = -1;
    }
    cluster_sync();
    Found f = {-1, 0, 0, 0, 0};
    const bool other = lane < cluster, earlier = lane < static_cast<int>(rank);
    const unsigned long long theirs = other ? far(&s.shown.all, lane) : 0ull;
    const unsigned long long their_w = other ? far(&s.shown.weight, lane) : 0ull;
    const unsigned long long their_c = other ? far(&s.shown.ties, lane) : 0ull;
    f.all = warp_sum(theirs);
    const unsigned long long earlier_w = before_weight + warp_sum(earlier ? their_w : 0ull);
    const unsigned long long earlier_c = before_all + warp_sum(earlier ? their_c : 0ull);
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
    const int d = other ? far(&s.shown.digit, lane) : -1;
    const unsigned has = __ballot_sync(0xffffffffu, d >= 0);
    if (has != 0u) {
        const unsigned r = __ffs(has) - 1;
        f.digit = __shfl_sync(0xffffffffu, d, r);
        f.above = far(&s.shown.above, r);
        f.above_weight = far(&s.shown.above_weight, r);
        f.here = far(&s.shown.here, r);
    }
    return f;
}

// The same for kDigits digits and one of the sums: each block adds up its share of the digits and writes the
// sums to all blocks, each of which then looks by itself (one way to other SMs and back fewer than above).
// Sums of counts lie where s.low does.
template <bool BY_WEIGHT, class R>
__device__ __noinline__ Found locate_one(Shared& s, int cluster, unsigned rank, R reach) {
    using Sum = typename std::conditional<BY_WEIGHT, unsigned long long, unsigned>::type;
    constexpr int PER = kDigits / kThreads;
    Sum* sums;
    if constexpr (BY_WEIGHT) sums = s.weights;
    else sums = cluster > 1 ? s.low : s.count;
    if (cluster > 1 || BY_WEIGHT) {
        const int share = kDigits / cluster;
        for (int x = threadIdx.x; x < share; x += kThreads) {
            const int d = rank * share + x;
            Sum sum = 0;
            if (cluster > 1) {
                unsigned n[kMaxCluster], hi[kMaxCluster];            // (asked for together)
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) {
                    n[r] = r < cluster ? far(BY_WEIGHT ? &s.low[d] : &s.count[d], r) : 0u;
                    hi[r] = BY_WEIGHT && r < cluster ? far(&s.high[d], r) : 0u;
                }
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) sum += static_cast<Sum>((static_cast<unsigned long long>(hi[r]) << 32) + n[r]);
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r)
                    if (r < cluster) put_far(&sums[d], r, sum);
            } else {
                sums[d] = static_cast<Sum>((static_cast<unsigned long long>(s.high[d]) << 32) + s.low[d]);
            }
        }
        if (cluster > 1) cluster_sync();
        else __syncthreads();
    }
    Sum mine[PER], total = 0, all;
#pragma unroll
    for (int j = 0; j < PER; ++j) total += mine[j] = sums[threadIdx.x * PER + j];
    if (threadIdx.x == 0) s.shown.digit = -1;
    Sum at = block_scan<kThreads>(total, reinterpret_cast<Sum*>(s.scan), &all);
    const unsigned long long target = reach(all);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (at < target && at + mine[j] >= target) {
            s.shown.digit = static_cast<int>(threadIdx.x) * PER + j;
            s.shown.above = at;
            s.shown.here = mine[j];
        }
        at += mine[j];
    }
    __syncthreads();
    Found f = {s.shown.digit, 0, 0, 0, all};
    if (f.digit >= 0) {
        f.above = BY_WEIGHT ? 0 : s.shown.above;
        f.above_weight = BY_WEIGHT ? s.shown.above : 0;
        f.here = BY_WEIGHT ? 0 : s.shown.here;
    }
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
        part.each([&](float z, int) {
            const unsigned key = key_of(z);
            if (key < floor || key <= kNone) return;
            if (level > 0 && key >> (shift + bits) != prefix) return;
            const int d = digits - 1 - static_cast<int>(key >> shift & static_cast<unsigned>(digits - 1));
            atomicAdd(&s.count[d], 1u);
            add_weight(s, d, weigh.units(z));
        });
        cluster_sync();                   // (also: what the last level has shown is read)
        const Found f = locate<BY_WEIGHT>(s, digits, b.above, b.weight, cluster, rank,
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
    cluster_sync();
    // b.need: all tokens at the border.
    if (BY_WEIGHT) {
        const unsigned long long one = weigh.units(value_of(b.key)), left = target - b.weight;
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
    const float edge = value_of(border.key);
    part.each([&](float z, int) { mine += z == edge; });
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s.u[warp] = mine;
    __syncthreads();
    if (tid == 0) {
        unsigned n = 0;
        for (int i = 0; i < kWarps; ++i) n += s.u[i];
        s.shown.ties = n;
    }
    cluster_sync();
    const unsigned ties = lane < cluster ? far(&s.shown.ties, lane) : 0u;
    const unsigned long long before = __reduce_add_sync(0xffffffffu, lane < static_cast<int>(rank) ? ties : 0u);
    const unsigned long long here = __shfl_sync(0xffffffffu, ties, rank);
    int limit = part.vocab;
    if (border.need <= before) {
        limit = -1;
    } else if (border.need < before + here) {
        // Its place in this block: in the order of the indices, kThreads vectors at a time.
        unsigned left = static_cast<unsigned>(border.need - before);
        __syncthreads();
        if (tid == 0) s.limit = part.vocab;
        for (int v = part.v0; v < part.v1; v += kThreads) {
            float z[V];
            unsigned n = 0, all;
            const bool in = v + tid < part.v1;
            if (in) {
                part.values(v + tid, z);
#pragma unroll
                for (int i = 0; i < V; ++i) n += z[i] == edge;
            }
            unsigned at = block_scan<kThreads>(n, reinterpret_cast<unsigned*>(s.scan), &all);
            if (in && at < left && at + n >= left) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (z[i] == edge && ++at == left) s.limit = (v + tid) * V + i - part.shift;
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
__device__ __forceinline__ void put_in_list(Shared& s, float z, int at) {
    const unsigned n = atomicAdd(&s.shown.listed, 1u);
    if (n < kList) s.list[n] = entry_of(key_of(z), at);
}
// The blocks' lists in the first one's, if they fit: their tokens in all.  Called behind a cluster barrier;
// the others' lists are read until the next.
__device__ __forceinline__ unsigned gather_lists(Shared& s, int cluster, unsigned rank) {
    if (cluster == 1) return s.shown.listed;
    const int lane = threadIdx.x & 31;
    const unsigned mine = lane < cluster ? far(&s.shown.listed, lane) : 0u;
    unsigned upto = mine;
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
        const unsigned o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    const unsigned all = __shfl_sync(0xffffffffu, upto, kMaxCluster - 1);
    if (rank == 0 && all <= kList) {
        const unsigned own = __shfl_sync(0xffffffffu, mine, 0);
        for (unsigned base = own; base < all; base += kThreads) {
            const unsigned i = base + threadIdx.x;
            unsigned r = 0, at = 0;       // entry i's block, and the entries before that block's
#pragma unroll
            for (int x = 0; x < kMaxCluster; ++x) {
                const unsigned to = __shfl_sync(0xffffffffu, upto, x);
                if (i >= to) {
                    r = x + 1;
                    at = to;
                }
            }
            if (i < all) s.list[i] = far(&s.list[i - at], r);
        }
        __syncthreads();
    }
    return all;
}
// One exchange of a sort in falling order: entry number i keeps the larger of the pair where its run falls and
// it is the pair's first, or neither.
__device__ __forceinline__ unsigned long long exchange(unsigned long long mine, unsigned long long other, int i,
                                                       int run, int step) {
    const bool larger = ((i & run) == 0) == ((i & step) == 0);
    return (mine < other) == larger ? other : mine;
}
// Falling order of the list's n entries (a block; ends with a barrier): compare and exchange in powers of two,
// four neighbours a thread, by as many warps as that takes.  Steps within a thread are in registers, within a
// warp by shuffles, further ones through the list's place.
__device__ __noinline__ void sort_list(unsigned long long* list, int n) {
    constexpr int E = 4;
    const int tid = threadIdx.x;
    int size = 32 * E;
    while (size < n) size <<= 1;
    const bool active = tid * E < size;
    __syncthreads();
    unsigned long long x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = tid * E + j < n ? list[tid * E + j] : 0ull;
#pragma unroll 1
    for (int run = 2; run <= size; run <<= 1) {
#pragma unroll 1
        for (int step = run >> 1; step >= 32 * E; step >>= 1) {
            __syncthreads();
            if (active) {
#pragma unroll
                for (int j = 0; j < E; ++j) list[tid * E + j] = x[j];
            }
            __syncthreads();
            if (active) {
#pragma unroll
                for (int j = 0; j < E; ++j) x[j] = exchange(x[j], list[(tid * E + j) ^ step], tid * E + j, run, step);
            }
        }
        if (!active) continue;            // (whole warps)
#pragma unroll 1
        for (int step = min(run >> 1, 16 * E); step >= E; step >>= 1) {
#pragma unroll
            for (int j = 0; j < E; ++j)
                x[j] = exchange(x[j], __shfl_xor_sync(0xffffffffu, x[j], step / E), tid * E + j, run, step);
        }
#pragma unroll
        for (int step = E / 2; step > 0; step >>= 1) {
            if (step >= run) continue;
#pragma unroll
            for (int j = 0; j < E; ++j) {
                if ((j & step) != 0) continue;
                const unsigned long long a = x[j], b = x[j | step];
                x[j] = exchange(a, b, tid * E + j, run, step);
                x[j | step] = exchange(b, a, tid * E + (j | step), run, step);
            }
        }
    }
    __syncthreads();
    if (active) {
#pragma unroll
        for (int j = 0; j < E; ++j) list[tid * E + j] = x[j];
    }
    __syncthreads();
}
static_assert(kList == 4 * kThreads, "lists that are sorted");

// The same, by 2048 pieces of the list's range of z, where hardly any share one: an entry's place is that of
// its piece and the number of larger ones in it.  (From 128 entries on; below, one warp exchanges them.)
constexpr int kCrowd = 64;                // entries of a piece that are compared with each other
__device__ __noinline__ void order_list(Shared& s, int n) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int E = kList / kThreads;
    if (n <= 128) {
        sort_list(s.list, n);
        return;
    }
    __syncthreads();
    unsigned long long x[E];
    unsigned top = 0u, bottom = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        const int i = tid + j * kThreads;
        x[j] = i < n ? s.list[i] : 0ull;
        const unsigned key = static_cast<unsigned>(x[j] >> 32);
        if (i < n) {
            top = max(top, key);
            bottom = min(bottom, key);
        }
        s.count[i] = 0u;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    bottom = __reduce_min_sync(0xffffffffu, bottom);
    if (lane == 0) {
        s.u[warp] = top;
        s.v[warp] = bottom;
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, s.u[lane & (kWarps - 1)]);
    bottom = __reduce_min_sync(0xffffffffu, s.v[lane & (kWarps - 1)]);
    const Pieces pieces(value_of(top), value_of(top) - value_of(bottom));
    int piece[E];
    unsigned nth[E];
    bool crowded = false;
#pragma unroll
    for (int j = 0; j < E; ++j) {
        piece[j] = pieces.of(value_of(static_cast<unsigned>(x[j] >> 32)));
        nth[j] = tid + j * kThreads < n ? atomicAdd(&s.count[piece[j]], 1u) : 0u;
        crowded = crowded || nth[j] >= kCrowd;
    }
    if (__syncthreads_or(crowded)) {
        sort_list(s.list, n);
        return;
    }
    unsigned c[E], mine = 0, all;
#pragma unroll
    for (int j = 0; j < E; ++j) mine += c[j] = s.count[tid * E + j];
    unsigned before = block_scan<kThreads>(mine, reinterpret_cast<unsigned*>(s.scan), &all);
#pragma unroll
    for (int j = 0; j < E; ++j) {
        s.count[tid * E + j] = before;
        before += c[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (tid + j * kThreads < n) s.list[s.count[piece[j]] + nth[j]] = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) {
        if (tid + j * kThreads >= n) continue;
        const unsigned first = s.count[piece[j]], end = piece[j] + 1 < kDigits ? s.count[piece[j] + 1] : n;
        nth[j] = first;
        for (unsigned i = first; i < end; ++i) nth[j] += s.list[i] > x[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j)
        if (tid + j * kThreads < n) s.list[nth[j]] = x[j];
    __syncthreads();
}
static_assert(kList == kDigits, "a piece an entry");

// The best token so far: what it is chosen by, its index, its z.
struct Best {
    float pick, z;
    int at;
    __device__ __forceinline__ void take(float x, int i, float value) {
        if (x > pick || (x == pick && i < at)) {
            pick = x;
            at = i;
            z = value;
        }
    }
};
constexpr int kNobody = 0x7fffffff;
// The block's best token and sum, in thread 0.
__device__ __forceinline__ void join_block(Shared& s, Best* best, float* sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto join_warp = [&](int from) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            if (d > from) continue;
            const float x = __shfl_xor_sync(0xffffffffu, best->pick, d), z = __shfl_xor_sync(0xffffffffu, best->z, d);
            const int i = __shfl_xor_sync(0xffffffffu, best->at, d);
            *sum += __shfl_xor_sync(0xffffffffu, *sum, d);
            best->take(x, i, z);
        }
    };
    join_warp(16);
    __syncthreads();
    if (lane == 0) {
        s.f[warp] = best->pick;
        s.g[warp] = *sum;
        s.i[warp] = best->at;
        s.u[warp] = __float_as_uint(best->z);
    }
    __syncthreads();
    if (warp == 0) {
        const bool has = lane < kWarps;
        best->pick = has ? s.f[lane] : kNegInf;
        best->at = has ? s.i[lane] : kNobody;
        best->z = has ? __uint_as_float(s.u[lane]) : 0.0f;
        *sum = has ? s.g[lane] : 0.0f;
        join_warp(kWarps / 2);
    }
}
__device__ __forceinline__ void put_token(const SampleParams& p, int b, const Weigh& weigh, const Best& best, float sum) {
    const bool none = best.at == kNobody;                // (noise of NaN everywhere)
    if (none) flag(p.status, GS_DEV_EMPTY_ROW);
    if (p.token != nullptr) p.token[b] = none ? -1 : best.at;
    if (p.logprob != nullptr)
        p.logprob[b] = none ? kNegInf : (best.z == weigh.ref ? 0.0f : best.z - weigh.ref) - logf(sum);
}

// A token stays where the sum before it is below p of all.
__device__ __forceinline__ unsigned long long reach_of(float top_p, unsigned long long all) {
    const double reach = ceil(static_cast<double>(fmaxf(top_p, 0.0f)) * static_cast<double>(all));
    return max(1ull, min(all, static_cast<unsigned long long>(reach)));
}

// The first block, with all tokens that may stay in its list: the filters and the token.
__device__ __noinline__ void finish_list(const SampleParams& p, Shared& s, const Weigh& weigh, int b, int n, int k,
                                         float top_p, float min_p, const float* noise) {
    order_list(s, n);
    const int kept = k > 0 ? min(k, n) : n;
    constexpr int PER = kList / kThreads;
    const int per = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * per;
    unsigned long long mine = 0, all, units[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        units[j] = j < per && i0 + j < kept ? weigh.units(value_of(static_cast<unsigned>(s.list[i0 + j] >> 32))) : 0;
        mine += units[j];
    }
    unsigned long long before = block_scan<kThreads>(mine, s.scan, &all);
    const unsigned long long target = top_p < 1.0f ? reach_of(top_p, all) : ~0ull;
    float sum = 0.0f, z[PER], add[PER];
    int at[PER];
    bool stays[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        stays[j] = j < per && i0 + j < kept;
        const unsigned long long e = stays[j] ? s.list[i0 + j] : 0;
        z[j] = value_of(static_cast<unsigned>(e >> 32));
        at[j] = static_cast<int>(~static_cast<unsigned>(e));
        const float w = stays[j] ? weigh.weight(z[j]) : 0.0f;
        stays[j] = stays[j] && before < target && (!(w < min_p) || z[j] == weigh.ref);
        before += units[j];
        if (stays[j]) sum += w;
        add[j] = stays[j] && noise != nullptr ? noise[at[j]] : 0.0f;
    }
    Best best = {kNegInf, 0.0f, kNobody};
#pragma unroll
    for (int j = 0; j < PER; ++j)
        if (stays[j]) best.take(z[j] + add[j], at[j], z[j]);
    join_block(s, &best, &sum);
    if (threadIdx.x == 0) put_token(p, b, weigh, best, sum);
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = p.cluster > 1 ? cluster_rank() : 0u;
    const int b = blockIdx.x / p.cluster;
    if (tid == 0) s.shown.listed = 0u;
    clear(s.count, kDigits);
    grid_wait();
    grid_trigger();
    const float hot = p.temperature != nullptr ? p.temperature[b] : 1.0f;
    Part<T> part = {nullptr, nullptr, 0, 0, 0, 0, 0, 0, Divisor(hot)};
    constexpr int V = Part<T>::V;
    const T* const row = static_cast<const T*>(p.logits) + b * p.row_stride;
    part.shift = static_cast<int>((reinterpret_cast<unsigned long long>(row) & 15ull) / sizeof(T));
    part.row = row;
    part.vocab = p.vocab;
    const int k = p.top_k != nullptr ? p.top_k[b] : 0;
    const float top_p = p.top_p != nullptr ? p.top_p[b] : 1.0f, min_p = p.min_p != nullptr ? p.min_p[b] : 0.0f;
    const int vectors = (p.vocab + part.shift + V - 1) / V;
    part.v0 = static_cast<int>(static_cast<long long>(vectors) * rank / p.cluster);
    part.v1 = static_cast<int>(static_cast<long long>(vectors) * (rank + 1) / p.cluster);
    part.whole0 = part.shift > 0 ? 1 : 0;
    part.whole1 = (p.vocab + part.shift) / V - 1;
    part.from = reinterpret_cast<const uint4*>(row - part.shift);
    if (p.held != 0) part.hold(reinterpret_cast<uint4*>(raw + sizeof(Shared)));
    // The largest key, and the smallest of the vectors' largest.
    float largest = kNegInf, smallest = __builtin_huge_valf();
#pragma unroll 4
    for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
        const float m = part.most(v);
        largest = fmaxf(largest, m);
        smallest = fminf(smallest, m > kNegInf ? m : __builtin_huge_valf());
    }
    unsigned top = key_of(part.cool.of(largest)), bottom = key_of(part.cool.of(smallest));
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
    // (What other blocks show is read a block a lane: one after the other each costs a way to its SM and back.)
    top = __reduce_max_sync(0xffffffffu, lane < p.cluster ? far(&s.shown.top, lane) : 0u);
    bottom = __reduce_min_sync(0xffffffffu, lane < p.cluster ? far(&s.shown.bottom, lane) : 0xffffffffu);
    if (top <= kNone) {                   // nothing to choose from
        if (rank == 0 && tid == 0) {
            if (p.token != nullptr) p.token[b] = -1;
            if (p.logprob != nullptr) p.logprob[b] = kNegInf;
            flag(p.status, GS_DEV_EMPTY_ROW);
        }
        cluster_sync();
        return;
    }
    const Weigh weigh = {value_of(top)};
    Pieces pieces(weigh.ref, fminf(weigh.ref - value_of(bottom), 32.0f));
    const float* const noise = p.noise != nullptr && hot > 0.0f ? p.noise + b * p.noise_stride : nullptr;
    const bool by_k = k > 0 && k < p.vocab, by_p = top_p < 1.0f;
    float edge = kNegInf;                 // what is above stays, and at it up to index limit: everything
    int limit = -1;
    bool known = !by_k && !by_p;
    // The block's sum of a value a thread, in thread 0.
    auto block_sum = [&](float x) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        __syncthreads();
        if (lane == 0) s.f[warp] = x;
        __syncthreads();
        x = lane < kWarps ? s.f[lane] : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        return x;
    };
    // The sum of the values that the cluster's blocks show.
    auto cluster_sum = [&] {
        float x = lane < p.cluster ? far(&s.shown.sum, lane) : 0.0f;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        return x;
    };
    if (!known && (p.vocab <= kList || (by_k && k <= kMostK))) {
        // All tokens from a z on that k tokens reach (of a short row all) to the first block.
        int last = kDigits - 1;
        bool some = true;
        if (p.vocab > kList) {
#pragma unroll 2
            for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
                const float most = part.most_z(v);
                if (most > kNegInf) atomicAdd(&s.count[pieces.of(most)], 1u);
            }
            cluster_sync();
            const Found f = locate_one<false>(s, p.cluster, rank,
                                              [&](unsigned long long) { return static_cast<unsigned long long>(k); });
            if (f.digit >= 0) last = f.digit;
            some = f.above + f.here <= kList;            // (else there are too many tokens for certain)
        }
        if (some)
            part.vectors([&](int v) {
                const float most = part.most_z(v);
                return most > kNegInf && pieces.of(most) <= last;
            }, [&](const float (&z)[V], int at) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (z[i] > kNegInf && pieces.of(z[i]) <= last) put_in_list(s, z[i], at + i);
            });
        cluster_sync();
        const unsigned n = gather_lists(s, p.cluster, rank);
        if (some && n <= kList) {
            cluster_sync();               // (lists stay until they are read; the others' SMs take the next row)
            if (rank == 0) finish_list(p, s, weigh, b, static_cast<int>(n), by_k ? k : 0, top_p, min_p, noise);
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
        // A token of less than (1 - p) / vocab of the sum is not kept: all such together are less than 1 - p of
        // it.  The sum is at least that of the vectors' largest weights.  Of the tokens below, the sum alone
        // counts (in fp32: it is 1 - p of all at most), and the pieces need not reach them.
        float least = 0.0f;
#pragma unroll 2
        for (int v = part.v0 + tid; v < part.v1; v += kThreads) {
            least += weigh.weight(part.most_z(v));       // (0 for -inf)
        }
        least = block_sum(least);
        if (tid == 0) s.shown.sum = least;
        cluster_sync();
        least = cluster_sum();
        const float little = fminf(0.5f, (1.0f - fmaxf(top_p, 0.0f)) * least / static_cast<float>(p.vocab) * 0.99f);
        pieces = Pieces(weigh.ref, fminf(logf(1.0f / little) + 0.01f, 32.0f));
        float rest = 0.0f;
        part.vectors([](int) { return true; }, [&](const float (&z)[V], int) {
            unsigned lo[V], old[V], hi[V];
            int d[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = weigh.weight(z[i]);
                const bool counts = w > little;
                rest += counts ? 0.0f : w;
                lo[i] = hi[i] = 0u;
                d[i] = 0;
                if (counts) {
                    Weigh::words_of(w, &lo[i], &hi[i]);
                    d[i] = pieces.of(z[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) old[i] = lo[i] != 0u ? atomicAdd(&s.low[d[i]], lo[i]) : 0u;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                hi[i] += old[i] + lo[i] < old[i];
                if (hi[i] != 0u) atomicAdd(&s.high[d[i]], hi[i]);
            }
        });
        // (The rest goes to the last piece: it lies behind all that may be kept.)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, d);
        if (lane == 0) add_weight(s, kDigits - 1, __float2ull_rz(rest * 1099511627776.0f));
        cluster_sync();
        unsigned long long target = 0;
        const Found f = locate_one<true>(s, p.cluster, rank, [&](unsigned long long all) {
            return target = reach_of(top_p, all);
        });
        part.vectors([&](int v) {
            const float most = part.most_z(v);
            return most > kNegInf && pieces.of(most) <= f.digit;
        }, [&](const float (&z)[V], int at) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (z[i] > kNegInf && pieces.of(z[i]) == f.digit) put_in_list(s, z[i], at + i);
        });
        cluster_sync();
        const unsigned n = gather_lists(s, p.cluster, rank);
        if (n <= kList) {
            known = true;
            if (rank == 0) {
                order_list(s, static_cast<int>(n));
                constexpr int PER = kList / kThreads;
                const int per = (static_cast<int>(n) + kThreads - 1) / kThreads, i0 = tid * per;
                unsigned long long mine = 0, all, units[PER];
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    units[j] = j < per && i0 + j < static_cast<int>(n) ? weigh.units(value_of(static_cast<unsigned>(s.list[i0 + j] >> 32))) : 0;
                    mine += units[j];
                }
                unsigned long long before = f.above_weight + block_scan<kThreads>(mine, s.scan, &all);
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    if (units[j] > 0 && before < target && before + units[j] >= target) {
                        const unsigned long long e = s.list[i0 + j];
                        if (p.cluster == 1) s.shown.border = e;
                        for (int r = 0; p.cluster > 1 && r < p.cluster; ++r) put_far(&s.shown.border, r, e);
                    }
                    before += units[j];
                }
            }
            cluster_sync();
            edge = value_of(static_cast<unsigned>(s.shown.border >> 32));
            limit = static_cast<int>(~static_cast<unsigned>(s.shown.border));
        } else {
            cluster_sync();               // (what follows takes the lists' place)
        }
    }
    if (!known) {
        Border last = {kNone + 1u, ~0ull, 0ull, 0ull};   // everything
        if (by_k) {
            const Border found = find_border<false>(s, part, weigh, 0u, static_cast<unsigned long long>(k), p.cluster, rank);
            if (found.need > 0) last = found;            // (else fewer than k tokens can be chosen)
        }
        if (by_p) {
            // The sum over what top-k left.
            unsigned long long mine = 0, all;
            const float over = last.need == ~0ull ? kNegInf : value_of(last.key);
            part.each([&](float z, int) {
                if (z > over) mine += weigh.units(z);
            });
            block_scan<kThreads>(mine, s.scan, &all);
            if (tid == 0) s.shown.weight = all;
            cluster_sync();
            all = warp_sum(lane < p.cluster ? far(&s.shown.weight, lane) : 0ull);
            cluster_sync();
            if (last.need != ~0ull) all += last.need * weigh.units(value_of(last.key));
            const Border found = find_border<true>(s, part, weigh, last.key, reach_of(top_p, all), p.cluster, rank);
            if (found.key > last.key || (found.key == last.key && found.need < last.need)) last = found;
        }
        if (last.need != ~0ull) {
            edge = value_of(last.key);
            limit = limit_of(s, part, last, p.cluster, rank);
        }
    }
    // The token, and the weights of what stays.
    Best best = {kNegInf, 0.0f, kNobody};
    float sum = 0.0f, rest = 0.0f;        // (sum - rest: what rounding left out is kept)
    const float least = min_p * 0.99f;    // (weights of neighbouring z are not compared with min_p itself)
    const bool all = edge == kNegInf && !(least > 0.0f);
    // What stays has z >= from, or in vectors up to the limit z >= edge, and no weight below `light`.
    const float from = min_p > 1.0f && edge < weigh.ref ? weigh.ref : value_of(key_of(edge) + 1u);       // (NaN above +inf)
    const float tied = edge == kNegInf ? from : min_p > 1.0f ? weigh.ref : edge, light = min_p > 1.0f ? 0.0f : min_p;
    const bool by4 = noise != nullptr && part.shift == 0 && (reinterpret_cast<unsigned long long>(noise) & 15ull) == 0;
    bool some = false;
    auto pass = [&](auto take) {
        part.vectors([&](int v) {
            if (all) return true;
            const float most = part.most_z(v);
            return most >= edge && (!(least > 0.0f) || weigh.weight(most) >= least || most == weigh.ref);
        }, [&](float (&z)[V], int at) {
            float add[V], here = 0.0f;
            const bool vector = by4 && at + V <= p.vocab;
            if (vector) {
#pragma unroll
                for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(add + i) = *reinterpret_cast<const float4*>(noise + at + i);
            }
            const float low = at > limit ? from : tied;
            if (at <= limit && at + V - 1 > limit) {     // (one vector of the row)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (z[i] == edge && at + i > limit) z[i] = kNegInf;
            }
            bool stays[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float w = weigh.weight(z[i]);
                stays[i] = z[i] >= low && !(w < light);
                here += stays[i] ? w : 0.0f;
                some = some || stays[i];
            }
            if (!vector) {
#pragma unroll
                for (int i = 0; i < V; ++i) add[i] = stays[i] && noise != nullptr ? noise[at + i] : 0.0f;
            }
            const float y = here - rest, t = sum + y;
            rest = (t - sum) - y;
            sum = t;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (stays[i]) take(z[i] + add[i], at + i, z[i]);
        });
    };
    // (A thread's indices rise: of equal ones the first stays.)
    pass([&](float x, int at, float z) {
        if (x > best.pick) best = {x, z, at};
    });
    if (best.at == kNobody && some) {     // noise of -inf or NaN alone
        sum = rest = 0.0f;
        pass([&](float x, int at, float z) { best.take(x, at, z); });
    }
    join_block(s, &best, &sum);
    if (tid == 0) {
        s.shown.pick = best.pick;
        s.shown.best = best.at;
        s.shown.best_z = best.z;
        s.shown.sum = sum;
    }
    cluster_sync();
    if (rank == 0 && warp == 0) {
        const bool other = lane < p.cluster;
        best.pick = other ? far(&s.shown.pick, lane) : kNegInf;
        best.at = other ? far(&s.shown.best, lane) : kNobody;
        best.z = other ? far(&s.shown.best_z, lane) : 0.0f;
        sum = other ? far(&s.shown.sum, lane) : 0.0f;
#pragma unroll
        for (int d = kMaxCluster / 2; d > 0; d >>= 1) {
            const float x = __shfl_xor_sync(0xffffffffu, best.pick, d), z = __shfl_xor_sync(0xffffffffu, best.z, d);
            const int i = __shfl_xor_sync(0xffffffffu, best.at, d);
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
            best.take(x, i, z);
        }
        if (lane == 0) put_token(p, b, weigh, best, sum);
    }
    cluster_sync();                       // (what rank 0 read stays until it is read)
}

// Blocks of a row: as many as it takes to hold the row, and more where they find SMs (two blocks each) and
// have more than two vectors a thread: a barrier of a cluster costs more than one of a block.
int cluster_of(const gs_sample_args* a) {
    const long long bytes = a->vocab * elem_size(a->dtype);
    int n = 1;
    while (n < kMaxCluster &&
           (bytes / n > kHeld - 64 ||
            (bytes / n > 16 * 2 * kThreads && 2ll * a->batch * n <= 2ll * sm_count())))
        n *= 2;
    return n;
}

template <class T>
gs_status launch_type(const SampleParams& p, gs_stream stream) {
    const dim3 grid(static_cast<unsigned>(p.batch) * p.cluster);
    const int bytes = static_cast<int>(sizeof(Shared)) + p.held;
    if (!allow_smem<sample_kernel<T>>(bytes)) return GS_ERR_CUDA;
    return launch(sample_kernel<T>, grid, kThreads, bytes, p.cluster, stream, p);
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_sample(const gs_sample_args* a, gs_stream stream) {
    if (a == nullptr || a->batch < 0 || a->vocab < 1 || !known_dtype(a->dtype)) return GS_ERR_INVALID_ARG;
    if (a->batch > GS_MAX_SEQS || a->vocab > kMostVocab) return GS_ERR_UNSUPPORTED;
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
    // (A part has a vector or two more than its share.)
    const long long part = (a->vocab * es + 16) / p.cluster + 32;
    p.held = part <= kHeld ? static_cast<int>(part / 16 * 16) : 0;
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
