// Guided logits (sm_103a): the two branches' logits, bias, penalties for repeated tokens,
// temperature and a grammar mask to the final logits, and from them the token and its
// log-probability, in one pass over the vocabulary.
//
// A block takes one chunk of one row; chunks are cut so that all blocks of the call are
// resident at once where a chunk then holds 16384 logits at most (what a block does once -
// settings, history, joining - costs about 4 us and is then paid once an SM's slot).  Larger
// calls have several waves of such blocks (67 rows of 131072 25.8 us, 68 27.5, 128 47.9, 256 83.3).
// Each warp streams 256 logits at a time through a buffer of its own in shared memory, by 16-byte
// asynchronous copies: once a piece is in registers the next one's copies are issued, and then
// the piece is worked on.
//
// Rows need no alignment: groups of 8 logits are laid so that the output is written in 16-byte
// vectors, the inputs are copied as the aligned vectors that cover them, and a lane shifts its
// 8 values out of its vectors by the row's offset (the same for the whole row).  Only bytes of
// the row itself are read: the vector that holds a row's first value is read value by value
// where it begins before the row, and a copy ends with the row.
//
// The penalties need which tokens of the chunk were said, and how often.  The block marks the
// history's tokens in a bitmap (a bit a logit) and counts them in a dense array indexed by a
// token's rank among the marked ones, so that no table of counts of the vocabulary's size is
// kept or read, and a group of 8 logits looks at one byte.
//
// Each thread carries a running maximum and sum of the softmax and the best token so far; a
// block's five numbers go to the workspace, and the block of a row that arrives last joins
// them in the order of the chunks.
//
// What bounds it, on a GB300 (graph replay, inputs not in L2): 64 rows of 131072 fp32 logits
// without extras (67 MB) take 16.3 us, 61 % of the measured copy rate; bf16 with guidance, histories
// of up to 2048 tokens, mask, bias and noise (102 MB) 26 us, 58 %: 67 instructions a logit at half
// of the issue slots, 5 us of settings, counting and joining, and as the blocks are cut evenly
// some SMs have four and some three.  Histories cost 4.5 us at 2048 tokens, 10 at 8192 and 36 at
// 32768 (every block of a row counts its whole history, and the counts' shared memory costs
// blocks on an SM, which the cut does not look at).  The instances for rows off 16 bytes are held
// to 64 registers for four blocks an SM and spill 12 to 64 bytes.  One row of 16384 takes 6.0 us:
// five latencies in a chain.
//
// Measured and not kept: logits held in registers instead of a buffer (45 us, and 29 us at four
// blocks an SM, for the 64 rows above), a count a logit instead of a bitmap (32 KB a block), two
// buffers a warp (51 us), shorter chunks (8192: 30 us).
#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kLogitThreads = 256;
constexpr int kLogitWarps = kLogitThreads / 32;
constexpr int kPer = 8;                                  // logits a lane takes at a time
constexpr int kPiece = 32 * kPer;                        // a warp
constexpr int kStride = kLogitWarps * kPiece;            // a block
constexpr int kPerSm = 4;                                // blocks wanted on an SM
constexpr int kMaxChunk = 16384;
constexpr float kLog2e = 1.4426950408889634f;

struct LogitParams {
    int batch, vocab, chunk, chunks;
    const void* uncond;
    const void* cond;
    long long row_stride;
    const int* step_idx;
    int step;
    const float* lut;
    int n_lut;
    float cfg;
    const float* bias;
    long long bias_stride;
    const int* tokens;
    long long tokens_stride;
    const int* tokens_len;
    const int* prompt_len;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const float* temperature;
    const unsigned* mask;
    long long mask_stride;
    const unsigned char* mask_present;
    const float* noise;
    long long noise_stride;
    float* out;
    long long out_stride;
    int* token;
    float* logprob;
    unsigned* status;
    int* arrived;                                        // [batch], 0 between calls
    struct Part* parts;                                  // [batch][chunks]
    int stage;                                           // bytes of a warp's buffer
    int off_uncond, off_bias, off_noise;                 // in it (cond lies at 0)
};

// What is known of a piece of a row: max and sum of the softmax, the best token.
struct __align__(16) Part {
    float top, sum;                                      // sum of e^(z - top)
    float best, z;                                       // largest z (+ noise), its z
    int token;                                           // kNoToken: none above -inf
    int pad[3];
};
constexpr int kNoToken = 0x7fffffff;

__device__ __forceinline__ Part no_part() {
    Part a;
    a.top = a.best = a.z = kNegInf;
    a.sum = 0.0f;
    a.token = kNoToken;
    a.pad[0] = a.pad[1] = a.pad[2] = 0;
    return a;
}
// e^x (results below 2^-126 are 0; e^0 is 1 exactly).
__device__ __forceinline__ float exp_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * kLog2e));
    return y;
}
// A row's divisor.
struct Divisor {
    float by, inverse;
    bool usual;                                          // by is neither tiny nor huge
};
__device__ __forceinline__ Divisor divisor(float by) {
    return {by, 1.0f / by, fabsf(by) >= 0x1p-40f && fabsf(by) <= 0x1p40f};
}
// f(value, its number) for each of the 8 values, one after the other: for what is rare, so that its
// code is there once.
template <class F>
__device__ __forceinline__ void in_turn(float (&z)[kPer], F f) {
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
        const float x = f(z[0], i);
#pragma unroll
        for (int e = 0; e + 1 < kPer; ++e) z[e] = z[e + 1];
        z[kPer - 1] = x;
    }
}
// z / by, correctly rounded.  A product with the rounded reciprocal and one correction by its
// remainder is the correctly rounded quotient where nothing overflows or loses bits below the
// normal numbers (P. Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990); other values are divided.  (64 rows of 131072: 17.4 us, 17.1 with the product
// alone, 18.2 with divisions.)
__device__ __forceinline__ void divide(float (&z)[kPer], const Divisor& d) {
    float least = fabsf(z[0]), most = least;
#pragma unroll
    for (int e = 1; e < kPer; ++e) {
        least = fminf(least, fabsf(z[e]));
        most = fmaxf(most, fabsf(z[e]));
    }
    if (d.usual && least >= 0x1p-60f && most <= 0x1p60f) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float q = z[e] * d.inverse;
            z[e] = fmaf(fmaf(-q, d.by, z[e]), d.inverse, q);
        }
    } else {
        in_turn(z, [&](float x, int) { return x / d.by; });
    }
}
// Unsigned numbers in the order of the floats (-0 counts as 0; no NaN).
__device__ __forceinline__ unsigned order_of(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return (u >> 31) != 0u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(unsigned o) {
    return __uint_as_float((o >> 31) != 0u ? o & 0x7fffffffu : ~o);
}

// The parts of a warp's lanes as one, in every lane.
__device__ __forceinline__ Part join_warp(Part a) {
    const float top = float_of(__reduce_max_sync(0xffffffffu, order_of(a.top)));
    a.sum *= exp_of(a.top - (top == kNegInf ? 0.0f : top));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) a.sum += __shfl_xor_sync(0xffffffffu, a.sum, d);
    a.top = top;
    const unsigned mine = order_of(a.best);
    const unsigned best = __reduce_max_sync(0xffffffffu, mine);
    const int token = __reduce_min_sync(0xffffffffu, mine == best ? a.token : kNoToken);
    const unsigned who = __ballot_sync(0xffffffffu, a.token == token);
    a.z = __shfl_sync(0xffffffffu, a.z, __ffs(who) - 1);
    a.best = float_of(best);
    a.token = token;
    return a;
}

// The parts of the block's warps as one, in every lane of warp 0.
__device__ __forceinline__ Part join_block(Part a, Part* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = join_warp(a);
    if (lane == 0) tmp[warp] = a;
    __syncthreads();
    if (warp == 0) a = join_warp(lane < kLogitThreads / 32 ? tmp[lane] : no_part());
    return a;
}

// ---- streams: rows of T that pass through a warp's buffer -----------------------------------
__device__ __forceinline__ void copy_async(unsigned dst, const void* src, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size)
                 : "memory");
}

// MIS: the row may lie off 16 bytes.
template <class T, bool MIS>
struct Stream {
    static constexpr int kSize = static_cast<int>(sizeof(T));
    static constexpr int N = kPer * kSize / 16;          // vectors of 8 values
    const char* row;                                     // null: there is none
    const char* next;                                    // this lane's first vector of the next piece
    int mis;                                             // (row - lead) mod 16, bytes
    char* buffer;                                        // this stream's, of this warp

    // r: the row; at: the first value of the warp's first piece, which with its lead is the
    // place of a group of 8.
    __device__ __forceinline__ void begin(const T* r, int at, int lead, char* to, int lane) {
        row = reinterpret_cast<const char*>(r);
        mis = MIS ? static_cast<int>((reinterpret_cast<uintptr_t>(r) - lead * kSize) & 15) : 0;
        next = row + (static_cast<long long>(at) * kSize - mis + lane * 16);
        buffer = to;
    }
    // Copies the vectors that cover values at .. at + 255 of a row of `vocab`.  Successive calls
    // are kStride values apart.
    __device__ __forceinline__ void copy(int at, int vocab, int lane) {
        if (row == nullptr) return;
        char* const to = buffer + lane * 16;
        const unsigned dst = static_cast<unsigned>(__cvta_generic_to_shared(to));
        if ((!MIS || at * kSize >= mis) && (at + kPiece + (MIS ? 16 / kSize : 0)) <= vocab) {    // all inside the row
#pragma unroll
            for (int i = 0; i < N; ++i) copy_async(dst + i * 512, next + i * 512, 16);
            if (MIS && mis != 0 && lane == 0) copy_async(dst + N * 512, next + N * 512, 16);
        } else {
            const int b = static_cast<int>(next - row);  // of the row
#pragma unroll
            for (int i = 0; i < N; ++i) put(to + i * 512, b + i * 512, vocab * kSize);
            if (MIS && mis != 0 && lane == 0) put(to + N * 512, b + N * 512, vocab * kSize);
        }
        next += kStride * kSize;
    }
    // The vector at byte b of a row of so many bytes, what of it lies in the row.
    __device__ __forceinline__ void put(char* to, int b, int bytes) const {
        if (!MIS || b >= 0) {
            if (b < bytes)
                copy_async(static_cast<unsigned>(__cvta_generic_to_shared(to)), row + b, min(16, bytes - b));
        } else if (b > -16) {
            for (int i = 0; i < 16; i += kSize)
                if (b + i >= 0 && b + i < bytes)
                    *reinterpret_cast<T*>(to + i) = *reinterpret_cast<const T*>(row + b + i);
        }
    }
    // This lane's 8 values.
    __device__ __forceinline__ void get(float* f, int lane) const {
        const uint4* from = reinterpret_cast<const uint4*>(buffer) + lane * N;
        unsigned w[4 * N + 4];
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<uint4*>(w + 4 * i) = from[i];
        if (MIS && mis != 0) {
            *reinterpret_cast<uint4*>(w + 4 * N) = from[N];
            if ((mis & 8) != 0) {
#pragma unroll
                for (int i = 0; i < 4 * N + 2; ++i) w[i] = w[i + 2];
            }
            if ((mis & 4) != 0) {
#pragma unroll
                for (int i = 0; i < 4 * N + 1; ++i) w[i] = w[i + 1];
            }
            if (kSize == 2 && (mis & 2) != 0) {
#pragma unroll
                for (int i = 0; i < 4 * N; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            unpack16<T>(make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]), f + i * (16 / kSize));
    }
    // Bytes of it in a buffer: a piece, and a vector where the rows are not aligned.
    static constexpr int size() { return N * 512 + 16; }
};

template <class T, bool MIS>
__global__ void __launch_bounds__(kLogitThreads, kPerSm)
logits_kernel(const __grid_constant__ LogitParams p) {
    extern __shared__ __align__(16) char smem[];
    __shared__ Part tmp[kLogitWarps];
    __shared__ int scan[kLogitWarps + 1];
    const int row = blockIdx.y, chunk = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* const out = p.out != nullptr ? p.out + row * p.out_stride : nullptr;
    // The chunk's groups of 8 logits begin at origin, origin + 8, ..: where out is on 16 bytes.
    const int lead = MIS ? static_cast<int>(reinterpret_cast<uintptr_t>(out) >> 2 & 3) : 0;
    const int origin = chunk * p.chunk - lead;
    const int end = min(origin + p.chunk, p.vocab);
    char* const buffer = smem + warp * p.stage;
    unsigned* const bits = reinterpret_cast<unsigned*>(smem + kLogitWarps * p.stage);
    int* const rank = reinterpret_cast<int*>(bits) + p.chunk / 32;
    unsigned* const count = reinterpret_cast<unsigned*>(rank + p.chunk / 32);

    grid_wait();
    grid_trigger();
    // The first logits are asked for before the row's settings are known.
    Stream<T, MIS> cond, uncond;
    Stream<float, MIS> bias, noise;
    const int start = origin + warp * kPiece;            // this warp's pieces: start + 2048 i
    cond.begin(static_cast<const T*>(p.cond) + row * p.row_stride, start, lead, buffer, lane);
    if (start < end) cond.copy(start, p.vocab, lane);

    // So is the history's beginning, whatever its length: HELD tokens a thread.
    constexpr int HELD = 8;
    const int* const tokens = p.tokens + (p.tokens != nullptr ? row * p.tokens_stride : 0);
    const int room = p.tokens != nullptr ? static_cast<int>(min(p.tokens_stride, 0x7fffffffll)) : 0;
    int held[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int t = i * kLogitThreads + static_cast<int>(threadIdx.x);
        held[i] = t < room ? tokens[t] : -1;
    }

    // The row's settings.
    const int step = p.step_idx != nullptr ? p.step_idx[row] : p.step;
    const float hot = p.temperature != nullptr ? p.temperature[row] : 1.0f;
    const float rep = p.repetition != nullptr ? p.repetition[row] : 1.0f;
    const float freq = p.frequency != nullptr ? p.frequency[row] : 0.0f;
    const float pres = p.presence != nullptr ? p.presence[row] : 0.0f;
    int known = p.tokens != nullptr ? p.tokens_len[row] : 0;
    const int prompt = p.prompt_len != nullptr ? p.prompt_len[row] : 0;
    const bool masked = p.mask != nullptr && (p.mask_present == nullptr || p.mask_present[row] != 0);
    float s = p.cfg;
    unsigned bad = 0;
    if (p.lut != nullptr) {
        if (step < 0 || step >= p.n_lut) bad = GS_DEV_STEP_RANGE;
        else s = p.lut[step];
    }
    const bool guided = s != 1.0f;
    if (bad == 0 && guided && p.uncond == nullptr) bad = GS_DEV_NEED_UNCOND;
    if (bad != 0) {
        if (chunk == 0 && threadIdx.x == 0) {
            flag(p.status, bad);
            if (p.token != nullptr) p.token[row] = -1;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    const float rest = 1.0f - s;
    const Divisor cool = divisor(hot), milder = divisor(rep);
    const float fewer = milder.usual ? milder.inverse : 1.0f, more = milder.usual ? rep : 1.0f;
    const unsigned* const mask = masked ? p.mask + row * p.mask_stride : nullptr;
    uncond.begin(guided ? static_cast<const T*>(p.uncond) + row * p.row_stride : nullptr, start, lead,
                 buffer + p.off_uncond, lane);
    bias.begin(p.bias != nullptr ? p.bias + row * p.bias_stride : nullptr, start, lead,
               buffer + p.off_bias, lane);
    noise.begin(p.noise != nullptr && hot > 0.0f ? p.noise + row * p.noise_stride : nullptr, start, lead,
                buffer + p.off_noise, lane);
    if (start < end) {
        uncond.copy(start, p.vocab, lane);
        bias.copy(start, p.vocab, lane);
        noise.copy(start, p.vocab, lane);
    }

    // Which tokens of the chunk were said, and how often.
    if (rep == 1.0f && freq == 0.0f && pres == 0.0f) known = 0;
    known = min(max(known, 0), room);
    bool said = false;
    if (known > 0) {
        const int words = p.chunk / 32;
        for (int i = threadIdx.x; i < words; i += kLogitThreads) bits[i] = 0u;
        __syncthreads();
        const int low = max(origin, 0);
        // Of the tokens held, the place in the chunk; -1 elsewhere.
        bool any = false;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int t = i * kLogitThreads + static_cast<int>(threadIdx.x);
            held[i] = t < known && held[i] >= low && held[i] < end ? held[i] - origin : -1;
            if (held[i] >= 0) {
                atomicOr(bits + (held[i] >> 5), 1u << (held[i] & 31));
                any = true;
            }
        }
        // Calls f(t, token - origin) for the other tokens in the chunk.
        auto each_other = [&](auto f) {
            for (int t0 = HELD * kLogitThreads + threadIdx.x; t0 < known; t0 += HELD * kLogitThreads) {
                int v[HELD];
#pragma unroll
                for (int i = 0; i < HELD; ++i) {
                    const int t = t0 + i * kLogitThreads;
                    v[i] = t < known ? tokens[t] : -1;
                }
#pragma unroll
                for (int i = 0; i < HELD; ++i)
                    if (v[i] >= low && v[i] < end) f(t0 + i * kLogitThreads, v[i] - origin);
            }
        };
        each_other([&](int, int b) {
            atomicOr(bits + (b >> 5), 1u << (b & 31));
            any = true;
        });
        said = __syncthreads_or(any ? 1 : 0) != 0;
        if (said) {
            // The words' ranks, two words a thread; the counts from 0.
            static_assert(kMaxChunk / 32 <= 2 * kLogitThreads, "two words a thread");
            const int i = 2 * static_cast<int>(threadIdx.x);
            const int n0 = i < words ? __popc(bits[i]) : 0, n1 = i + 1 < words ? __popc(bits[i + 1]) : 0;
            int total;
            const int r = block_scan<kLogitThreads>(n0 + n1, scan, &total);
            if (i < words) rank[i] = r;
            if (i + 1 < words) rank[i + 1] = r + n0;
            for (int x = threadIdx.x; x < total; x += kLogitThreads) count[x] = 0u;
            __syncthreads();
            auto add = [&](int t, int b) {
                if (t >= prompt)
                    atomicAdd(count + rank[b >> 5] + __popc(bits[b >> 5] & ((1u << (b & 31)) - 1u)), 1u);
            };
            if (any) {
#pragma unroll
                for (int k = 0; k < HELD; ++k)
                    if (held[k] >= 0) add(k * kLogitThreads + static_cast<int>(threadIdx.x), held[k]);
                each_other(add);
            }
            __syncthreads();
        }
    }

    // The mask's word(s) for the lane's 8 logits from v on; asked for one piece ahead.
    unsigned allow_lo = 0u, allow_hi = 0u;
    auto fetch_mask = [&](int v) {
        if (mask == nullptr || v >= end) return;
        const int w = max(v, 0) >> 5;
        allow_lo = mask[w];
        if (MIS && v >= 0 && (v & 31) > 24 && (w + 1) * 32 < p.vocab) allow_hi = mask[w + 1];
    };
    fetch_mask(start + lane * kPer);

    const bool choose = p.token != nullptr || p.logprob != nullptr;
    Part mine = no_part();
    for (int at = start; at < end; at += kStride) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        const int v0 = at + lane * kPer;                 // this lane's logits: v0 .. v0 + 7
        const bool full = (!MIS || v0 >= 0) && v0 + kPer <= end;
        float z[kPer], add[kPer];
        cond.get(z, lane);
        if (uncond.row != nullptr) {
            float odd = 0.0f;                            // NaN where a value is not finite
            uncond.get(add, lane);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                z[e] = fmaf(s, z[e], rest * add[e]);
                odd = fmaf(z[e], 0.0f, odd);
            }
            if (odd != 0.0f) {                           // cond where either is -inf
                float c[kPer];
                cond.get(c, lane);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (c[e] == kNegInf || add[e] == kNegInf) z[e] = c[e];
            }
        }
        if (bias.row != nullptr) {
            bias.get(add, lane);
#pragma unroll
            for (int e = 0; e < kPer; ++e) z[e] += add[e];
        }
        if (noise.row != nullptr) noise.get(add, lane);
        __syncwarp();                                    // the buffer has been read
        const unsigned allow = MIS && v0 < 0 ? allow_lo << -v0 : __funnelshift_r(allow_lo, allow_hi, v0 & 31);
        if (at + kStride < end) {
            fetch_mask(v0 + kStride);
            cond.copy(at + kStride, p.vocab, lane);
            uncond.copy(at + kStride, p.vocab, lane);
            bias.copy(at + kStride, p.vocab, lane);
            noise.copy(at + kStride, p.vocab, lane);
        }
        if (said && v0 < end) {
            const int b = v0 - origin;                   // (a multiple of 8)
            const unsigned word = bits[b >> 5], these = word >> (b & 31) & 0xffu;
            if (these != 0u) {
                const unsigned* n = count + rank[b >> 5] + __popc(word & ((1u << (b & 31)) - 1u));
                // (The product with the rounded reciprocal has one rounding more than a quotient, but this
                // is done for nearly every piece where histories are long: 25.6 us for the 64 rows
                // above, 29.1 with quotients.)
                if (!milder.usual)
                    in_turn(z, [&](float x, int e) {
                        return (these >> e & 1u) == 0u ? x : x > 0.0f ? x / rep : x * rep;
                    });
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    const bool hit = (these >> e & 1u) != 0u;
                    const unsigned times = hit ? *n : 0u;
                    n += hit ? 1 : 0;
                    const float by = z[e] > 0.0f ? fewer : more;
                    z[e] = hit ? z[e] * by : z[e];
                    z[e] = times != 0u ? z[e] - fmaf(freq, static_cast<float>(times), pres) : z[e];
                }
            }
        }
        if (hot > 0.0f) {
            if (!full) {                                 // what lies outside the row may be anything
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((MIS && v0 + e < 0) || v0 + e >= end) z[e] = 1.0f;
            }
            divide(z, cool);
        }
        if (mask != nullptr) {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if ((allow >> e & 1u) == 0u) z[e] = kNegInf;
        }
        if (out != nullptr) {
            if (full) {
                __stcs(reinterpret_cast<float4*>(out + v0), make_float4(z[0], z[1], z[2], z[3]));
                __stcs(reinterpret_cast<float4*>(out + v0 + 4), make_float4(z[4], z[5], z[6], z[7]));
            } else {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((!MIS || v0 + e >= 0) && v0 + e < end) out[v0 + e] = z[e];
            }
        }
        if (choose) {
            if (!full) {
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if ((MIS && v0 + e < 0) || v0 + e >= end) z[e] = kNegInf;
            }
            float top = kNegInf;
#pragma unroll
            for (int e = 0; e < kPer; ++e) top = fmaxf(top, z[e]);
            // The best of the group, the lowest of equals last.
            if (noise.row != nullptr) {
                float best = kNegInf;
#pragma unroll
                for (int e = 0; e < kPer; ++e) {
                    add[e] += z[e];
                    best = fmaxf(best, add[e]);
                }
                if (best > mine.best) {
                    mine.best = best;
#pragma unroll
                    for (int e = kPer - 1; e >= 0; --e)
                        if (add[e] == best) {
                            mine.z = z[e];
                            mine.token = v0 + e;
                        }
                }
            } else if (top > mine.best) {
                mine.best = mine.z = top;
#pragma unroll
                for (int e = kPer - 1; e >= 0; --e)
                    if (z[e] == top) mine.token = v0 + e;
            }
            if (top > mine.top) {
                mine.sum *= exp_of(mine.top - top);
                mine.top = top;
            }
            const float from = mine.top == kNegInf ? 0.0f : mine.top;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) sum += exp_of(z[e] - from);
            mine.sum += sum;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!choose) return;

    mine = join_block(mine, tmp);
    if (threadIdx.x >= 32) return;
    Part* parts = p.parts + static_cast<long long>(row) * p.chunks;
    if (p.chunks > 1) {
        int last = 0;
        if (threadIdx.x == 0) {
            int4* to = reinterpret_cast<int4*>(parts + chunk);
            __stcg(to, make_int4(__float_as_int(mine.top), __float_as_int(mine.sum),
                                 __float_as_int(mine.best), __float_as_int(mine.z)));
            __stcg(to + 1, make_int4(mine.token, 0, 0, 0));
            __threadfence();
            last = atomicAdd(p.arrived + row, 1) == p.chunks - 1 ? 1 : 0;
            if (last) p.arrived[row] = 0;                // as the next call finds it
            __threadfence();
        }
        if (__shfl_sync(0xffffffffu, last, 0) == 0) return;
        __syncwarp();                                    // thread 0's fence holds for all lanes
        Part all = no_part();
        for (int c0 = 0; c0 < p.chunks; c0 += 32) {      // in the order of the chunks
            const int c = c0 + static_cast<int>(threadIdx.x);
            Part b = no_part();
            if (c < p.chunks) {
                const int4 a = __ldcg(reinterpret_cast<const int4*>(parts + c));
                b.top = __int_as_float(a.x);
                b.sum = __int_as_float(a.y);
                b.best = __int_as_float(a.z);
                b.z = __int_as_float(a.w);
                b.token = __ldcg(reinterpret_cast<const int*>(parts + c) + 4);
            }
            const float up = fmaxf(all.top, b.top);
            const float from = up == kNegInf ? 0.0f : up;
            all.sum = fmaf(all.sum, exp_of(all.top - from), b.sum * exp_of(b.top - from));
            all.top = up;
            if (b.best > all.best) {                     // (a lane's later chunks hold later tokens)
                all.best = b.best;
                all.z = b.z;
                all.token = b.token;
            }
        }
        mine = join_warp(all);
    }
    if (threadIdx.x == 0) {
        const bool none = mine.token == kNoToken;
        if (none) flag(p.status, GS_DEV_EMPTY_ROW);
        if (p.token != nullptr) p.token[row] = none ? -1 : mine.token;
        if (p.logprob != nullptr)
            p.logprob[row] = none ? kNegInf : (mine.z - mine.top) - logf(mine.sum);
    }
}

struct Cut {
    int chunk, chunks, stage, off_uncond, off_bias, off_noise, counts, smem;
    long long counters, bytes;
};

// The streams' buffers, the cut of the rows and the workspace.
gs_status cut_of(const gs_guided_logits_args* a, Cut* cut) {
    if (a == nullptr || a->batch < 0 || a->vocab < 1 || a->tokens_stride < 0 || !known_dtype(a->dtype))
        return GS_ERR_INVALID_ARG;
    if (a->batch > GS_MAX_SEQS || a->vocab > (1 << 28)) return GS_ERR_UNSUPPORTED;
    if (a->tokens != nullptr && a->tokens_stride > (1ll << 30)) return GS_ERR_UNSUPPORTED;   // (t0 + 2048 is an int)
    const int in = a->dtype == GS_DTYPE_F32 ? Stream<float, true>::size() : Stream<__half, true>::size();
    int stage = in;
    cut->off_uncond = stage;
    if (a->uncond != nullptr) stage += in;
    cut->off_bias = stage;
    if (a->bias != nullptr) stage += Stream<float, true>::size();
    cut->off_noise = stage;
    if (a->noise != nullptr) stage += Stream<float, true>::size();
    cut->stage = stage;
    const long long history = a->tokens != nullptr ? a->tokens_stride : 0;
    // As many chunks of a row as make the call's blocks resident at once; chunks are whole pieces
    // of a warp, and of a block at least.  kMaxChunk bounds the counts a block may hold (64 KB).
    const long long slots = static_cast<long long>(kPerSm) * sm_count();
    long long chunks = a->batch > 0 ? slots / a->batch : 1;
    if (chunks < 1) chunks = 1;
    long long chunk = (a->vocab + 3 + chunks - 1) / chunks;
    if (chunk < kStride) chunk = kStride;
    if (chunk > kMaxChunk) chunk = kMaxChunk;
    chunk = (chunk + kPiece - 1) / kPiece * kPiece;
    cut->chunk = static_cast<int>(chunk);
    cut->chunks = static_cast<int>((a->vocab + 3 + chunk - 1) / chunk);      // (a row may begin 3 early)
    cut->counts = static_cast<int>(history < chunk ? history : chunk);
    cut->smem = kLogitWarps * stage + (history > 0 ? cut->chunk / 4 + 4 * cut->counts : 0);
    cut->counters = (static_cast<long long>(a->batch) + 3) / 4 * 4;
    cut->bytes = 4 * cut->counters + static_cast<long long>(sizeof(Part)) * a->batch * cut->chunks;
    return GS_OK;
}

template <class T, bool MIS>
gs_status launch_logits(const LogitParams& p, int smem, gs_stream stream) {
    if (!allow_smem<logits_kernel<T, MIS>>(smem)) return GS_ERR_CUDA;
    return launch(logits_kernel<T, MIS>, dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(p.batch)),
                  kLogitThreads, smem, 1, stream, p);
}
template <class T>
gs_status launch_type(const LogitParams& p, bool mis, int smem, gs_stream stream) {
    return mis ? launch_logits<T, true>(p, smem, stream) : launch_logits<T, false>(p, smem, stream);
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_guided_logits_workspace(const gs_guided_logits_args* args,
                                                int64_t* bytes) {
    if (bytes == nullptr) return GS_ERR_INVALID_ARG;
    Cut cut;
    const gs_status st = cut_of(args, &cut);
    if (st != GS_OK) return st;
    *bytes = cut.bytes;
    return GS_OK;
}

extern "C" gs_status gs_guided_logits(const gs_guided_logits_args* a, gs_stream stream) {
    Cut cut;
    const gs_status st = cut_of(a, &cut);
    if (st != GS_OK) return st;
    if (a->batch == 0) return GS_OK;
    const long long es = elem_size(a->dtype);
    if (a->cond == nullptr || !aligned(a->cond, es) || !aligned(a->uncond, es) ||
        (a->batch > 1 && a->row_stride < a->vocab) || a->row_stride < 0)
        return GS_ERR_INVALID_ARG;
    if (a->scale_lut != nullptr &&
        (a->n_lut < 1 || (a->step_idx == nullptr && (a->step < 0 || a->step >= a->n_lut))))
        return GS_ERR_INVALID_ARG;
    if (a->bias_stride < 0 || a->noise_stride < 0 || a->mask_stride < 0 || a->tokens_stride < 0)
        return GS_ERR_INVALID_ARG;
    if (a->tokens != nullptr && a->tokens_len == nullptr) return GS_ERR_INVALID_ARG;
    if (a->out == nullptr && a->token == nullptr && a->logprob == nullptr) return GS_ERR_INVALID_ARG;
    if (a->out != nullptr && a->batch > 1 && a->out_stride < a->vocab) return GS_ERR_INVALID_ARG;
    if (!aligned(a->out, 4) || !aligned(a->bias, 4) || !aligned(a->noise, 4) ||
        !aligned(a->mask, 4) || !aligned(a->tokens, 4))
        return GS_ERR_INVALID_ARG;
    if (a->workspace == nullptr || !aligned(a->workspace, 16) || a->workspace_bytes < cut.bytes)
        return GS_ERR_INVALID_ARG;
    LogitParams p = {};
    p.batch = a->batch;
    p.vocab = a->vocab;
    p.chunk = cut.chunk;
    p.chunks = cut.chunks;
    p.uncond = a->uncond;
    p.cond = a->cond;
    p.row_stride = a->row_stride;
    p.step_idx = a->step_idx;
    p.step = a->step;
    p.lut = a->scale_lut;
    p.n_lut = a->n_lut;
    p.cfg = a->cfg;
    p.bias = a->bias;
    p.bias_stride = a->bias_stride;
    p.tokens = a->tokens;
    p.tokens_stride = a->tokens_stride;
    p.tokens_len = a->tokens_len;
    p.prompt_len = a->prompt_len;
    p.repetition = a->repetition;
    p.frequency = a->frequency;
    p.presence = a->presence;
    p.temperature = a->temperature;
    p.mask = a->mask;
    p.mask_stride = a->mask_stride;
    p.mask_present = a->mask_present;
    p.noise = a->noise;
    p.noise_stride = a->noise_stride;
    p.out = a->out;
    p.out_stride = a->out_stride;
    p.token = a->token;
    p.logprob = a->logprob;
    p.status = a->dev_status;
    p.arrived = static_cast<int*>(a->workspace);
    p.parts = reinterpret_cast<Part*>(static_cast<int*>(a->workspace) + cut.counters);
    p.stage = cut.stage;
    p.off_uncond = cut.off_uncond;
    p.off_bias = cut.off_bias;
    p.off_noise = cut.off_noise;
    // Rows on 16 bytes need no shifts (the 64 rows above: 25.9 us, and 29.5 us with them).
    const bool one = a->batch == 1;
    const bool mis = !(aligned(a->cond, 16) && aligned(a->uncond, 16) && aligned(a->out, 16) &&
                       aligned(a->bias, 16) && aligned(a->noise, 16) &&
                       (one || ((a->row_stride * es) % 16 == 0 && a->out_stride % 4 == 0 &&
                                a->bias_stride % 4 == 0 && a->noise_stride % 4 == 0)));
    switch (a->dtype) {
        case GS_DTYPE_F32: return launch_type<float>(p, mis, cut.smem, stream);
        case GS_DTYPE_BF16: return launch_type<__nv_bfloat16>(p, mis, cut.smem, stream);
        default: return launch_type<__half>(p, mis, cut.smem, stream);
    }
}
