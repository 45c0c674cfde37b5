// Sampling (sm_103a): temperature, top-k, top-p, min-p and the token from given random numbers.
//
// What the filters keep is a beginning of the row's tokens in the order of falling z (ties: rising
// index), so it is known by its last token: a border (a value of z) and how many of the tokens with
// just that value stay.  The border is found digit by digit in the 32-bit keys whose order is that of z:
// a histogram of 2048, 2048 and 1024 digits counts the tokens and sums their weights e^(z - max), the
// digits are scanned from the largest down, and the one that holds the border is looked into.  For top-k
// the border is the k-th token, for top-p the token at which the weights reach p of their sum over what
// top-k left.  min-p is a bound on a token's own weight, looked at last.
//
// Weights are summed as whole numbers (units of 2^-40 of the largest weight): sums do not depend on the
// order of the additions.  A row is a cluster's; its blocks keep a part of it each in shared memory, as
// keys, and read it once.
#include <cmath>

#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kDigits = 2048;
constexpr int kMaxCluster = 8;
constexpr unsigned kNone = 0x007fffffu;   // the key of -inf: such tokens, and NaN, are not kept
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct SampleParams {
    int batch, vocab, cluster, held;      // held: places of a block's keys in shared memory (0: not kept)
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
    unsigned top;                         // largest key
    unsigned long long count, weight;     // of its share of the digits
    unsigned long long above_count, above_weight, here;  // of what lies above the found digit; its tokens
    int digit;
    unsigned ties;                        // tokens at the border
    float pick, sum;                      // best token of the block, and the weights it keeps
    int best;
    unsigned best_key;
};

struct alignas(16) Shared {
    unsigned count[kDigits], low[kDigits], high[kDigits];
    unsigned long long scan[kWarps + 1];
    unsigned long long in[kMaxCluster][2];
    float f[kWarps], g[kWarps];
    int i[kWarps];
    unsigned u[kWarps];
    int limit;
    Shown shown;
};

__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

static_assert(sizeof(Shared) % 16 == 0, "the keys follow it in 16-byte vectors");

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

// A block's part of its row.  Places count from the 16-byte vector that holds the row's first value.
template <class T, bool HELD>
struct Part {
    static constexpr int V = 16 / static_cast<int>(sizeof(T));
    const T* row;
    unsigned* keys;
    int shift, vocab, v0, v1;             // values of the first vector that are not the row's; vectors
    float hot;

    __device__ __forceinline__ float settle(float z) const { return hot > 0.0f ? __fdiv_rn(z, hot) : z; }
    // The keys of vector v (0 for what is not the row's).
    __device__ __forceinline__ void fetch(int v, unsigned (&k)[V]) const {
        const int at = v * V - shift;
        float f[V];
        if (at >= 0 && at + V <= vocab) {
            unpack16<T>(*reinterpret_cast<const uint4*>(row + at), f);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = at + i >= 0 && at + i < vocab ? static_cast<float>(row[at + i]) : __int_as_float(0x7fffffff);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) k[i] = key_of(settle(f[i]));
    }
    __device__ __forceinline__ void load() const {
        if constexpr (HELD) {
            for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
                unsigned k[V];
                fetch(v, k);
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    *reinterpret_cast<uint4*>(keys + (v - v0) * V + i) = make_uint4(k[i], k[i + 1], k[i + 2], k[i + 3]);
            }
        }
    }
    // f(key, index in the row) for the thread's values.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        if constexpr (HELD) {
            const int n = (v1 - v0) * V / 4;
            for (int x = threadIdx.x; x < n; x += kThreads) {
                const uint4 k = reinterpret_cast<const uint4*>(keys)[x];
                const int at = v0 * V + 4 * x - shift;
                f(k.x, at);
                f(k.y, at + 1);
                f(k.z, at + 2);
                f(k.w, at + 3);
            }
        } else {
            for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
                unsigned k[V];
                fetch(v, k);
#pragma unroll
                for (int i = 0; i < V; ++i) f(k[i], v * V + i - shift);
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
__device__ Border find_border(Shared& s, const P& part, const Weigh& weigh, unsigned floor,
                              unsigned long long target, int cluster, unsigned rank) {
    Border b = {0u, 0ull, 0ull, 0ull};
    int shift = 32;
    for (int level = 0; level < 3; ++level) {
        const int bits = level == 2 ? 10 : 11, digits = 1 << bits;
        const unsigned prefix = b.key;
        shift -= bits;
        for (int x = threadIdx.x; x < digits; x += kThreads) s.count[x] = s.low[x] = s.high[x] = 0u;
        __syncthreads();
        part.each([&](unsigned key, int) {
            if (key < floor || key <= kNone) return;
            if (level > 0 && key >> (shift + bits) != prefix) return;
            const int d = digits - 1 - static_cast<int>(key >> shift & static_cast<unsigned>(digits - 1));
            const unsigned long long w = weigh.units(key);
            atomicAdd(&s.count[d], 1u);
            const unsigned lo = static_cast<unsigned>(w);
            unsigned hi = static_cast<unsigned>(w >> 32);
            if (lo != 0u) {
                const unsigned old = atomicAdd(&s.low[d], lo);
                if (old + lo < old) ++hi;
            }
            if (hi != 0u) atomicAdd(&s.high[d], hi);
        });
        cluster_sync();
        // This block's share of the digits, over all blocks.
        const int share = digits / cluster, per = (share + kThreads - 1) / kThreads;
        unsigned long long count[4], weight[4], counts = 0, weights = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            count[j] = weight[j] = 0;
            const int x = threadIdx.x * per + j;
            if (j >= per || x >= share) continue;
            const int d = rank * share + x;
            for (int r = 0; r < cluster; ++r) {
                count[j] += far(&s.count[d], r);
                weight[j] += (static_cast<unsigned long long>(far(&s.high[d], r)) << 32) + far(&s.low[d], r);
            }
            counts += count[j];
            weights += weight[j];
        }
        unsigned long long all_count, all_weight;
        const unsigned long long before_count = block_scan<kThreads>(counts, s.scan, &all_count);
        const unsigned long long before_weight = block_scan<kThreads>(weights, s.scan, &all_weight);
        if (threadIdx.x == 0) {
            s.shown.count = all_count;
            s.shown.weight = all_weight;
            s.shown.digit = -1;
        }
        cluster_sync();
        if (threadIdx.x < cluster) {
            s.in[threadIdx.x][0] = far(&s.shown.count, threadIdx.x);
            s.in[threadIdx.x][1] = far(&s.shown.weight, threadIdx.x);
        }
        __syncthreads();
        unsigned long long c = b.above, w = b.weight;
        for (unsigned r = 0; r < rank; ++r) {
            c += s.in[r][0];
            w += s.in[r][1];
        }
        c += before_count;
        w += before_weight;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = threadIdx.x * per + j;
            if (j >= per || x >= share) continue;
            const unsigned long long at = BY_WEIGHT ? w : c, mine = BY_WEIGHT ? weight[j] : count[j];
            if (at < target && at + mine >= target) {
                s.shown.digit = static_cast<int>(rank) * share + x;
                s.shown.above_count = c;
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
            b.key = prefix << bits | static_cast<unsigned>(digits - 1 - d);
            b.above = far(&s.shown.above_count, r);
            b.weight = far(&s.shown.above_weight, r);
            b.need = far(&s.shown.here, r);
        }
        cluster_sync();
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

template <class T, bool HELD>
__global__ void __launch_bounds__(kThreads) sample_kernel(const __grid_constant__ SampleParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared& s = *reinterpret_cast<Shared*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rank = p.cluster > 1 ? cluster_rank() : 0u;
    const int b = blockIdx.x / p.cluster;
    grid_wait();
    grid_trigger();
    Part<T, HELD> part;
    constexpr int V = Part<T, HELD>::V;
    const T* const row = static_cast<const T*>(p.logits) + b * p.row_stride;
    part.shift = static_cast<int>((reinterpret_cast<unsigned long long>(row) & 15ull) / sizeof(T));
    part.row = row;
    part.vocab = p.vocab;
    part.keys = reinterpret_cast<unsigned*>(raw + sizeof(Shared));
    part.hot = p.temperature != nullptr ? p.temperature[b] : 1.0f;
    const int vectors = (p.vocab + part.shift + V - 1) / V;
    part.v0 = static_cast<int>(static_cast<long long>(vectors) * rank / p.cluster);
    part.v1 = static_cast<int>(static_cast<long long>(vectors) * (rank + 1) / p.cluster);
    part.load();
    __syncthreads();
    // The largest key.
    unsigned top = 0u;
    part.each([&](unsigned key, int) { top = max(top, key); });
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s.u[warp] = top;
    __syncthreads();
    if (warp == 0) {
        const unsigned most = __reduce_max_sync(0xffffffffu, lane < kWarps ? s.u[lane] : 0u);
        if (lane == 0) s.shown.top = most;
    }
    cluster_sync();
    top = 0u;
    for (int r = 0; r < p.cluster; ++r) top = max(top, far(&s.shown.top, r));
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
    const int k = p.top_k != nullptr ? p.top_k[b] : 0;
    const float top_p = p.top_p != nullptr ? p.top_p[b] : 1.0f, min_p = p.min_p != nullptr ? p.min_p[b] : 0.0f;
    Border border = {kNone + 1u, ~0ull, 0ull, 0ull};     // everything stays
    if (k > 0 && k < p.vocab) {
        const Border found = find_border<false>(s, part, weigh, 0u, static_cast<unsigned long long>(k), p.cluster, rank);
        if (found.need > 0) border = found;              // (else fewer than k tokens can be chosen)
    }
    if (top_p < 1.0f) {
        // The sum over what top-k left.
        unsigned long long mine = 0, all;
        part.each([&](unsigned key, int) {
            if (key > border.key || (key == border.key && border.need == ~0ull)) mine += weigh.units(key);
        });
        block_scan<kThreads>(mine, s.scan, &all);
        if (tid == 0) s.shown.weight = all;
        cluster_sync();
        all = 0;
        for (int r = 0; r < p.cluster; ++r) all += far(&s.shown.weight, r);
        cluster_sync();
        if (border.need != ~0ull) all += border.need * weigh.units(border.key);
        // A token stays where the sum before it is below p of all.
        const double reach = ceil(static_cast<double>(fmaxf(top_p, 0.0f)) * static_cast<double>(all));
        const unsigned long long target = max(1ull, min(all, static_cast<unsigned long long>(reach)));
        const Border found = find_border<true>(s, part, weigh, border.key, target, p.cluster, rank);
        if (found.key > border.key || (found.key == border.key && found.need < border.need)) border = found;
    }
    // Of the tokens at the border, those up to index `limit`.
    int limit = p.vocab;
    if (border.need != ~0ull) {
        unsigned mine = 0, ties;
        part.each([&](unsigned key, int) { mine += key == border.key; });
        ties = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) s.u[warp] = ties;
        __syncthreads();
        if (tid == 0) {
            unsigned n = 0;
            for (int i = 0; i < kWarps; ++i) n += s.u[i];
            s.shown.ties = n;
        }
        cluster_sync();
        unsigned long long before = 0, here = 0;
        for (int r = 0; r < p.cluster; ++r) {
            const unsigned n = far(&s.shown.ties, r);
            if (r < static_cast<int>(rank)) before += n;
            else if (r == static_cast<int>(rank)) here = n;
        }
        if (border.need <= before) {
            limit = -1;
        } else if (border.need < before + here) {
            // Its place in this block: in the order of the indices, kThreads vectors at a time.
            unsigned left = static_cast<unsigned>(border.need - before);
            __syncthreads();
            if (tid == 0) s.limit = p.vocab;
            for (int v = part.v0; v < part.v1; v += kThreads) {
                unsigned key[V];
                unsigned n = 0;
                const bool in = v + tid < part.v1;
                if (in) {
                    if constexpr (HELD) {
#pragma unroll
                        for (int i = 0; i < V; ++i) key[i] = part.keys[(v + tid - part.v0) * V + i];
                    } else {
                        part.fetch(v + tid, key);
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) n += key[i] == border.key;
                }
                unsigned all;
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
    }
    // The token, and the weights of what stays.
    const float* const noise = p.noise != nullptr && part.hot > 0.0f ? p.noise + b * p.noise_stride : nullptr;
    float pick = kNegInf, sum = 0.0f, rest = 0.0f;       // (sum - rest: what rounding left out is kept)
    int best = 0x7fffffff;
    unsigned best_key = 0u;
    part.each([&](unsigned key, int at) {
        if (key < border.key || key <= kNone || (key == border.key && at > limit)) return;
        const float w = weigh.weight(key);
        if (w < min_p && key != top) return;
        const float y = w - rest, t = sum + y;
        rest = (t - sum) - y;
        sum = t;
        const float x = noise != nullptr ? value_of(key) + noise[at] : value_of(key);
        if (x > pick || (x == pick && at < best)) {
            pick = x;
            best = at;
            best_key = key;
        }
    });
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, pick, d);
        const int i = __shfl_xor_sync(0xffffffffu, best, d);
        const unsigned u = __shfl_xor_sync(0xffffffffu, best_key, d);
        sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (x > pick || (x == pick && i < best)) {
            pick = x;
            best = i;
            best_key = u;
        }
    }
    if (lane == 0) {
        s.f[warp] = pick;
        s.g[warp] = sum;
        s.i[warp] = best;
        s.u[warp] = best_key;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) {
            sum += s.g[w];
            if (s.f[w] > pick || (s.f[w] == pick && s.i[w] < best)) {
                pick = s.f[w];
                best = s.i[w];
                best_key = s.u[w];
            }
        }
        s.shown.pick = pick;
        s.shown.sum = sum;
        s.shown.best = best;
        s.shown.best_key = best_key;
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
        for (int r = 1; r < p.cluster; ++r) {
            const float x = far(&s.shown.pick, r);
            const int i = far(&s.shown.best, r);
            sum += far(&s.shown.sum, r);
            if (x > pick || (x == pick && i < best)) {
                pick = x;
                best = i;
                best_key = far(&s.shown.best_key, r);
            }
        }
        const bool none = best == 0x7fffffff;            // (noise of NaN everywhere)
        if (none) flag(p.status, GS_DEV_EMPTY_ROW);
        if (p.token != nullptr) p.token[b] = none ? -1 : best;
        if (p.logprob != nullptr)
            p.logprob[b] = none ? kNegInf : (best_key == top ? 0.0f : value_of(best_key) - weigh.ref) - logf(sum);
    }
    cluster_sync();                       // (what rank 0 read stays until it is read)
}

struct Plan {
    int cluster, held;
};

// Blocks of a row: enough of them for every SM, but no part below 2048 tokens; more where a part would not
// fit in shared memory, and where it does not fit with eight, parts are read again for each pass.
Plan plan_of(const gs_sample_args* a) {
    const long long most = (227 * 1024 - static_cast<long long>(sizeof(Shared))) / 4 - 64;
    Plan plan = {1, 0};
    while (plan.cluster < kMaxCluster &&
           (a->vocab / plan.cluster > most ||
            (a->vocab / plan.cluster >= 4096 && static_cast<long long>(a->batch) * plan.cluster < 2ll * sm_count())))
        plan.cluster *= 2;
    const long long part = (a->vocab + 16ll) / plan.cluster + 32;
    plan.held = part <= most ? static_cast<int>(part / 8 * 8) : 0;
    return plan;
}

template <class T>
gs_status launch_type(const SampleParams& p, gs_stream stream) {
    const dim3 grid(static_cast<unsigned>(p.batch) * p.cluster);
    const int bytes = static_cast<int>(sizeof(Shared)) + 4 * p.held;
    if (p.held > 0) {
        if (!allow_smem<sample_kernel<T, true>>(bytes)) return GS_ERR_CUDA;
        return launch(sample_kernel<T, true>, grid, kThreads, bytes, p.cluster, stream, p);
    }
    return launch(sample_kernel<T, false>, grid, kThreads, bytes, p.cluster, stream, p);
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
    const Plan plan = plan_of(a);
    SampleParams p = {};
    p.batch = a->batch;
    p.vocab = a->vocab;
    p.cluster = plan.cluster;
    p.held = plan.held;
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
