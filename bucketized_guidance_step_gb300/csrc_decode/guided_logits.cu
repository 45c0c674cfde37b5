// Guided logits (sm_103a): the two branches' logits, bias, penalties for repeated tokens,
// temperature and a grammar mask to the final logits, and from them the token and its
// log-probability, in one pass over the vocabulary.
//
// A block takes one chunk of one row.  The penalties need how often each token of the chunk
// was said: the block counts the row's history into shared memory (one word a token of the
// chunk: bit 31 = in the prompt, the rest = times said), so no table of counts of the size of
// the vocabulary is kept or read.  Each thread carries a running maximum and sum of the
// softmax and the best token so far; a block's five numbers go to the workspace, and the block
// of a row that arrives last joins them in the order of the chunks.
#include "decode_common.cuh"

namespace gs_decode {
namespace {

constexpr int kLogitThreads = 256;
constexpr int kPer = 8;                                  // logits a thread takes at a time
constexpr int kStride = kLogitThreads * kPer;
constexpr unsigned kPrompt = 0x80000000u;
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
__device__ __forceinline__ float exp_of(float x) { return exp2f(x * kLog2e); }

__device__ __forceinline__ Part join(const Part& a, const Part& b) {
    Part r = a;
    r.top = fmaxf(a.top, b.top);
    const float base = r.top == kNegInf ? 0.0f : r.top;
    r.sum = fmaf(a.sum, exp_of(a.top - base), b.sum * exp_of(b.top - base));
    if (b.best > a.best || (b.best == a.best && b.token < a.token)) {
        r.best = b.best;
        r.z = b.z;
        r.token = b.token;
    }
    return r;
}

// All threads' parts; the result is in thread 0.  Ends with a barrier.
__device__ __forceinline__ Part join_block(Part a, Part* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        Part b = a;
        b.top = __shfl_xor_sync(0xffffffffu, a.top, d);
        b.sum = __shfl_xor_sync(0xffffffffu, a.sum, d);
        b.best = __shfl_xor_sync(0xffffffffu, a.best, d);
        b.z = __shfl_xor_sync(0xffffffffu, a.z, d);
        b.token = __shfl_xor_sync(0xffffffffu, a.token, d);
        a = (lane & d) == 0 ? join(a, b) : join(b, a);
    }
    if (lane == 0) tmp[warp] = a;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kLogitThreads / 32; ++w) a = join(a, tmp[w]);
    }
    __syncthreads();
    return a;
}

template <class T, bool VEC>
__device__ __forceinline__ void load_logits(const T* row, int at, int stride, int end, bool full,
                                            float* f) {
    if constexpr (VEC) {
        if (full) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < kPer; i += V)
                unpack16<T>(__ldcs(reinterpret_cast<const uint4*>(row + at + i)), f + i);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int v = at + i * stride;
        f[i] = v < end ? to_float(row[v]) : kNegInf;
    }
}

// VEC: rows start on 16 bytes and a thread takes 8 neighbours; else every 256th.
template <class T, bool VEC>
__global__ void __launch_bounds__(kLogitThreads)
logits_kernel(const __grid_constant__ LogitParams p) {
    extern __shared__ unsigned said[];                   // [chunk]
    __shared__ Part tmp[kLogitThreads / 32];
    __shared__ int turn;
    grid_wait();
    grid_trigger();
    const int row = blockIdx.y, chunk = blockIdx.x;
    const int begin = chunk * p.chunk;
    const int end = min(begin + p.chunk, p.vocab);

    // The row's scale.
    float s = p.cfg;
    unsigned bad = 0;
    if (p.lut != nullptr) {
        const int i = p.step_idx != nullptr ? p.step_idx[row] : p.step;
        if (i < 0 || i >= p.n_lut) bad = GS_DEV_STEP_RANGE;
        else s = p.lut[i];
    }
    const bool guided = s != 1.0f;
    if (bad == 0 && guided && p.uncond == nullptr)
        bad = GS_DEV_NEED_UNCOND;
    if (bad != 0) {
        if (chunk == 0 && threadIdx.x == 0) {
            flag(p.status, bad);
            if (p.token != nullptr) p.token[row] = -1;
        }
        return;
    }
    const float rest = 1.0f - s;
    const float hot = p.temperature != nullptr ? p.temperature[row] : 1.0f;
    const float cool = hot > 0.0f ? 1.0f / hot : 1.0f;
    const float* noise = p.noise != nullptr && hot > 0.0f ? p.noise + row * p.noise_stride : nullptr;
    const float* bias = p.bias != nullptr ? p.bias + row * p.bias_stride : nullptr;
    const unsigned* mask =
        p.mask != nullptr && (p.mask_present == nullptr || p.mask_present[row] != 0)
            ? p.mask + row * p.mask_stride : nullptr;

    // How often each token of the chunk was said.
    const float rep = p.repetition != nullptr ? p.repetition[row] : 1.0f;
    const float freq = p.frequency != nullptr ? p.frequency[row] : 0.0f;
    const float pres = p.presence != nullptr ? p.presence[row] : 0.0f;
    int known = 0;
    if (p.tokens != nullptr && (rep != 1.0f || freq != 0.0f || pres != 0.0f)) {
        known = p.tokens_len[row];
        known = known < 0 ? 0 : known;
        if (known > p.tokens_stride) known = static_cast<int>(p.tokens_stride);
    }
    if (known > 0) {
        for (int v = threadIdx.x; v < p.chunk; v += kLogitThreads) said[v] = 0u;
        __syncthreads();
        const int prompt = p.prompt_len != nullptr ? p.prompt_len[row] : 0;
        const int* tokens = p.tokens + row * p.tokens_stride;
        for (int t = threadIdx.x; t < known; t += kLogitThreads) {
            const int v = tokens[t];
            if (v >= begin && v < end) {
                if (t < prompt) atomicOr(said + (v - begin), kPrompt);
                else atomicAdd(said + (v - begin), 1u);
            }
        }
        __syncthreads();
    }

    const T* cond = static_cast<const T*>(p.cond) + row * p.row_stride;
    const T* uncond = guided && p.uncond != nullptr
                          ? static_cast<const T*>(p.uncond) + row * p.row_stride : nullptr;
    float* out = p.out != nullptr ? p.out + row * p.out_stride : nullptr;
    const bool choose = p.token != nullptr || p.logprob != nullptr;
    Part mine = no_part();
    constexpr int kStep = VEC ? 1 : kLogitThreads;       // between a thread's logits
    for (int base = begin; base < end; base += kStride) {
        const int at = base + static_cast<int>(threadIdx.x) * (VEC ? kPer : 1);
        const bool full = VEC && at + kPer <= end;
        float z[kPer], add[kPer];
        load_logits<T, VEC>(cond, at, kStep, end, full, z);
        if (uncond != nullptr) {
            float u[kPer];
            load_logits<T, VEC>(uncond, at, kStep, end, full, u);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (z[i] != kNegInf && u[i] != kNegInf) z[i] = fmaf(s, z[i], rest * u[i]);
        }
        if (bias != nullptr) {
            load_logits<float, VEC>(bias, at, kStep, end, full, add);
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[i] += add[i];
        }
        if (known > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = at + i * kStep;
                const unsigned w = v < end ? said[v - begin] : 0u;
                if (w != 0u) {
                    z[i] = z[i] > 0.0f ? z[i] / rep : z[i] * rep;
                    const unsigned n = w & ~kPrompt;
                    if (n != 0u) z[i] -= fmaf(freq, static_cast<float>(n), pres);
                }
            }
        }
        if (hot > 0.0f) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) z[i] *= cool;
        }
        if (mask != nullptr) {
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int v = at + i * kStep;
                if (v < end && ((__ldg(mask + (v >> 5)) >> (v & 31)) & 1u) == 0u) z[i] = kNegInf;
            }
        }
        if (out != nullptr) {
            if (full) {
                __stcs(reinterpret_cast<float4*>(out + at), make_float4(z[0], z[1], z[2], z[3]));
                __stcs(reinterpret_cast<float4*>(out + at + 4), make_float4(z[4], z[5], z[6], z[7]));
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (at + i * kStep < end) out[at + i * kStep] = z[i];
            }
        }
        if (choose) {
            float top = mine.top;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (at + i * kStep >= end) z[i] = kNegInf;
                top = fmaxf(top, z[i]);
            }
            const float from = top == kNegInf ? 0.0f : top;
            mine.sum *= exp_of(mine.top - from);
            mine.top = top;
#pragma unroll
            for (int i = 0; i < kPer; ++i) mine.sum += exp_of(z[i] - from);
            if (noise != nullptr) {
                load_logits<float, VEC>(noise, at, kStep, end, full, add);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float x = noise != nullptr ? z[i] + add[i] : z[i];
                if (x > mine.best && z[i] > kNegInf) {
                    mine.best = x;
                    mine.z = z[i];
                    mine.token = at + i * kStep;
                }
            }
        }
    }
    if (!choose) return;

    mine = join_block(mine, tmp);
    Part* parts = p.parts + static_cast<long long>(row) * p.chunks;
    if (threadIdx.x == 0) {
        int4* to = reinterpret_cast<int4*>(parts + chunk);
        __stcg(to, make_int4(__float_as_int(mine.top), __float_as_int(mine.sum),
                             __float_as_int(mine.best), __float_as_int(mine.z)));
        __stcg(to + 1, make_int4(mine.token, 0, 0, 0));
        __threadfence();
        const int last = atomicAdd(p.arrived + row, 1) == p.chunks - 1 ? 1 : 0;
        if (last) p.arrived[row] = 0;                    // as the next call finds it
        __threadfence();
        turn = last;
    }
    __syncthreads();
    if (turn == 0) return;
    Part all = no_part();
    for (int c = threadIdx.x; c < p.chunks; c += kLogitThreads) {
        const int4 a = __ldcg(reinterpret_cast<const int4*>(parts + c));
        Part b = no_part();
        b.top = __int_as_float(a.x);
        b.sum = __int_as_float(a.y);
        b.best = __int_as_float(a.z);
        b.z = __int_as_float(a.w);
        b.token = __ldcg(reinterpret_cast<const int*>(parts + c) + 4);
        all = join(all, b);
    }
    all = join_block(all, tmp);
    if (threadIdx.x == 0) {
        const bool none = all.token == kNoToken;
        if (none) flag(p.status, GS_DEV_EMPTY_ROW);
        if (p.token != nullptr) p.token[row] = none ? -1 : all.token;
        if (p.logprob != nullptr)
            p.logprob[row] = none ? kNegInf : (all.z - all.top) - logf(all.sum);
    }
}

struct Cut {
    int chunk, chunks;
    long long counters, bytes;
};

// Chunks of 8192 logits (32 KB of counts, four or more blocks an SM) where the batch fills the
// device, shorter ones where it does not.
gs_status cut_of(const gs_guided_logits_args* a, Cut* cut) {
    if (a == nullptr || a->batch < 0 || a->vocab < 1) return GS_ERR_INVALID_ARG;
    if (a->batch > GS_MAX_SEQS || a->vocab > (1 << 30)) return GS_ERR_UNSUPPORTED;
    int chunk = 8192;
    while (chunk > kStride &&
           static_cast<long long>(a->batch) * ((a->vocab + chunk - 1) / chunk) < 4ll * sm_count())
        chunk >>= 1;
    cut->chunk = chunk;
    cut->chunks = (a->vocab + chunk - 1) / chunk;
    cut->counters = (static_cast<long long>(a->batch) + 3) / 4 * 4;
    cut->bytes = 4 * cut->counters + static_cast<long long>(sizeof(Part)) * a->batch * cut->chunks;
    return GS_OK;
}

template <class T, bool VEC>
gs_status launch_logits(const LogitParams& p, gs_stream stream) {
    return launch(logits_kernel<T, VEC>, dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(p.batch)),
                  kLogitThreads, 4 * p.chunk, 1, stream, p);
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
    if (!known_dtype(a->dtype)) return GS_ERR_INVALID_ARG;
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
    const bool one = a->batch == 1;
    const bool vec =
        aligned(a->cond, 16) && aligned(a->uncond, 16) && aligned(a->out, 16) &&
        aligned(a->bias, 16) && aligned(a->noise, 16) &&
        (one || ((a->row_stride * es) % 16 == 0 && a->out_stride % 4 == 0 &&
                 a->bias_stride % 4 == 0 && a->noise_stride % 4 == 0));
    switch (a->dtype) {
        case GS_DTYPE_F32:
            return vec ? launch_logits<float, true>(p, stream) : launch_logits<float, false>(p, stream);
        case GS_DTYPE_BF16:
            return vec ? launch_logits<__nv_bfloat16, true>(p, stream)
                       : launch_logits<__nv_bfloat16, false>(p, stream);
        default:
            return vec ? launch_logits<__half, true>(p, stream) : launch_logits<__half, false>(p, stream);
    }
}
