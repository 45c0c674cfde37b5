// Attention of one new token over a paged cache (sm_103a): the argument checks, and the policy
// that computes with fp32 multiply-adds, for fp32 caches.
//
// For each query head and position: s = q . k, the running maximum and sum of a softmax in
// powers of two, and o += 2^(s - m) v, all in fp32.  Eight lanes hold a row (a 16-byte piece
// every eighth), so a warp works on four positions at a time; each group of eight lanes keeps
// a maximum, sum and output of its own, and they meet at the segment's end.
//
// What bounds it: 16 rows of 4096 tokens with 32 query and 8 kv heads of dim 128 (537 MB) take
// 92 us, 86 % of the measured copy rate; 8 rows of 333 .. 3001 with 8 and 4 heads of 96 (45 MB)
// 17.1 us, 39 %: the call's fixed part, and five or six tiles a block in a row, whose multiply-adds
// two warps a scheduler do not hide.
#include <cmath>

#include "paged_attention.cuh"

namespace gs_decode {
namespace {

// NV: 16-byte pieces of a row that a lane holds; H: query heads of a part, for whose values and
// output a lane has 4 NV H registers each.
template <int NV, int H>
struct Fp32 {
    using T = float;
    static constexpr int DP = 32 * NV, RUN = 8, HEADS = H;
    // Blocks on an SM as registers allow; rings of 64, 96 or 192 KB.
    static constexpr int PER_SM = NV > 4 ? 1 : NV > 2 || H > 4 ? 2 : 3;
    static constexpr int STAGES = NV > 2 ? 3 : PER_SM == 3 ? 4 : 6;
    static constexpr int E = 4 * NV, U = RUN / 4;
    static_assert(HEADS <= kRound, "one dump");
    float q[HEADS][E], o[HEADS][E], top[HEADS], sum[HEADS];

    static constexpr bool AHEAD = false, FULL = NV <= 4, PARTIAL = NV <= 4;

    __device__ __forceinline__ void fetch(const float* query, long long head_stride, int heads,
                                          int dim, bool) {
        const int sub = threadIdx.x & 7;
#pragma unroll
        for (int h = 0; h < HEADS; ++h)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = (sub + 8 * (e / 4)) * 4 + e % 4;
                q[h][e] = h < heads && d < dim ? query[h * head_stride + d] : 0.0f;
            }
    }

    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            top[h] = kNegInf;
            sum[h] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = 0.0f;
        }
    }

    __device__ __forceinline__ void step(const char* stage, int lo, int hi, float scale) {
        const int sub = threadIdx.x & 7, group = (threadIdx.x >> 3) & 3;
        float s[U][HEADS];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = u * 4 + group;
#pragma unroll
            for (int h = 0; h < HEADS; ++h) s[u][h] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 k = *reinterpret_cast<const float4*>(
                    stage + r * DP * 4 + (((sub + 8 * i) ^ (r & 7)) << 4));
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    s[u][h] = fmaf(q[h][4 * i], k.x, s[u][h]);
                    s[u][h] = fmaf(q[h][4 * i + 1], k.y, s[u][h]);
                    s[u][h] = fmaf(q[h][4 * i + 2], k.z, s[u][h]);
                    s[u][h] = fmaf(q[h][4 * i + 3], k.w, s[u][h]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            float up = top[h];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int d = 1; d < 8; d <<= 1) s[u][h] += __shfl_xor_sync(0xffffffffu, s[u][h], d);
                s[u][h] = u * 4 + group >= lo && u * 4 + group < hi ? s[u][h] * scale : kNegInf;
                up = fmaxf(up, s[u][h]);
            }
            if (up > top[h]) {
                const float w = pow2(top[h] - up);      // 0 at the first position
                sum[h] *= w;
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] *= w;
                top[h] = up;
            }
            const float base = up == kNegInf ? 0.0f : up;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][h] = pow2(s[u][h] - base);
                sum[h] += s[u][h];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = u * 4 + group;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(
                    stage + (RUN + r) * DP * 4 + (((sub + 8 * i) ^ (r & 7)) << 4));
#pragma unroll
                for (int h = 0; h < HEADS; ++h) {
                    o[h][4 * i] = fmaf(s[u][h], v.x, o[h][4 * i]);
                    o[h][4 * i + 1] = fmaf(s[u][h], v.y, o[h][4 * i + 1]);
                    o[h][4 * i + 2] = fmaf(s[u][h], v.z, o[h][4 * i + 2]);
                    o[h][4 * i + 3] = fmaf(s[u][h], v.w, o[h][4 * i + 3]);
                }
            }
        }
    }

    __device__ __forceinline__ void dump(float* out, int pitch, int, int heads, int dim) {
        const int lane = threadIdx.x & 31, sub = lane & 7, group = lane >> 3;
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            float up = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 8));
            up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
            const float w = pow2(top[h] - (up == kNegInf ? 0.0f : up));
            float all = sum[h] * w;
            all += __shfl_xor_sync(0xffffffffu, all, 8);
            all += __shfl_xor_sync(0xffffffffu, all, 16);
            if (lane == 0 && h < heads) {
                out[h * pitch + dim] = up;
                out[h * pitch + dim + 1] = all;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = o[h][4 * i + e] * w;
                    x[e] += __shfl_xor_sync(0xffffffffu, x[e], 8);
                    x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
                }
                const int d = (sub + 8 * i) * 4;
                if (group == 0 && h < heads && d < dim)
                    *reinterpret_cast<float4*>(out + h * pitch + d) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
    }
};


// An instance computes for all its heads, so small groups have instances of their own: groups of 2
// with dim 96 (8 rows of 333 .. 3001 tokens) took 18.9 us, and 22.0 us in the instance of 4; groups
// of 4 with dim 64 (32 rows of 2048) 61 us, and 107 us in the instance of 8, whose registers allow
// two blocks an SM instead of three (the instance of 4 is held to 168 registers for the third
// and spills 40 to 64 bytes); groups of 8 107 us, and 127 us in two parts of 4.
template <class F>
auto with_instance(int dim, int group, F f) {
    if (dim <= 64) return group <= 2 ? f(Fp32<2, 2>()) : group <= 4 ? f(Fp32<2, 4>()) : f(Fp32<2, 8>());
    if (dim <= 128) return group <= 2 ? f(Fp32<4, 2>()) : f(Fp32<4, 4>());
    return f(Fp32<8, 2>());
}

}  // namespace

Serves fp32_serves(int dim, int group) {
    return with_instance(dim, group, [&](auto policy) { return serves_by<decltype(policy)>(group); });
}

gs_status launch_fp32(const AttnParams& p, int blocks, gs_stream stream) {
    return with_instance(p.c.dim, p.group, [&](auto policy) {
        return launch_policy<decltype(policy)>(p, blocks, stream);
    });
}

namespace {

struct Plan {
    int part, parts, blocks, run;
    long long counters, slots;            // words of the workspace
};

// Sizes, and what follows from them: the head groups, the grid and the workspace.
gs_status plan_of(const gs_paged_attention_args* a, Plan* plan) {
    if (a == nullptr) return GS_ERR_INVALID_ARG;
    const gs_status st = check_cache_sizes(a->cache);
    if (st != GS_OK) return st;
    const gs_kv_cache* c = a->cache;
    if (a->batch < 0 || a->q_heads < 1 || a->q_heads % c->kv_heads != 0 || a->window < 0 ||
        a->sinks < 0 || (a->sinks > 0 && a->window == 0))
        return GS_ERR_INVALID_ARG;
    if (a->batch > GS_MAX_SEQS || a->q_heads > (1 << 16)) return GS_ERR_UNSUPPORTED;
    const int group = a->q_heads / c->kv_heads;
    const Serves by = c->dtype == GS_DTYPE_F32 ? fp32_serves(c->dim, group) : mma_serves(c->dim, group);
    plan->run = by.tile / kWarps;
    plan->parts = by.parts;
    plan->part = by.part;
    long long most = static_cast<long long>(c->cols) * c->page;
    const long long visible = static_cast<long long>(a->window) + a->sinks + 2 * by.tile;   // whole runs
    if (a->window > 0 && visible < most) most = visible;
    const long long items = static_cast<long long>(a->batch) * c->kv_heads * plan->parts;
    const long long tiles = items * ((most + by.tile - 1) / by.tile + 1);         // units
    if (tiles > 0x7fffffffll || items > 0x3fffffffll) return GS_ERR_UNSUPPORTED;
    // What is resident at once, no more blocks than tiles.
    const long long full = static_cast<long long>(by.per_sm) * sm_count();
    plan->blocks = static_cast<int>(tiles < full ? (tiles > 0 ? tiles : 1) : full);
    plan->counters = (items + 3) / 4 * 4;
    plan->slots = 2ll * plan->blocks * slot_size(plan->part, c->dim);
    return GS_OK;
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_paged_attention_workspace(const gs_paged_attention_args* args,
                                                  int64_t* bytes) {
    if (bytes == nullptr) return GS_ERR_INVALID_ARG;
    Plan plan;
    const gs_status st = plan_of(args, &plan);
    if (st != GS_OK) return st;
    *bytes = 4 * (plan.counters + plan.slots);
    return GS_OK;
}

extern "C" gs_status gs_paged_attention(const gs_paged_attention_args* args, gs_stream stream) {
    Plan plan;
    gs_status st = plan_of(args, &plan);
    if (st != GS_OK) return st;
    AttnParams p = {};
    st = check_cache(args->cache, &p.c);
    if (st != GS_OK) return st;
    const long long es = elem_size(args->cache->dtype);
    if (args->layer < 0 || args->layer >= p.c.layers) return GS_ERR_INVALID_ARG;
    if (args->seq == nullptr && args->batch > p.c.seqs) return GS_ERR_INVALID_ARG;
    if ((args->k_new == nullptr) != (args->v_new == nullptr)) return GS_ERR_INVALID_ARG;
    if (args->k_new != nullptr && check_workspace(args->cache) != GS_OK) return GS_ERR_INVALID_ARG;
    if (!std::isfinite(args->scale)) return GS_ERR_INVALID_ARG;
    if (args->batch == 0) return GS_OK;
    if (args->q == nullptr || args->out == nullptr || !aligned(args->q, es) ||
        !aligned(args->out, es) || !aligned(args->k_new, es) || !aligned(args->v_new, es) ||
        !aligned(args->lse, 4))
        return GS_ERR_INVALID_ARG;
    if (args->q_batch_stride < 0 || args->q_head_stride < 0 || args->new_batch_stride < 0 ||
        args->new_head_stride < 0)
        return GS_ERR_INVALID_ARG;
    if ((args->batch > 1 && args->out_batch_stride < p.c.dim) ||
        (args->q_heads > 1 && args->out_head_stride < p.c.dim))
        return GS_ERR_INVALID_ARG;                        // output rows overlap
    if (args->workspace == nullptr || !aligned(args->workspace, 16) ||
        args->workspace_bytes < 4 * (plan.counters + plan.slots))
        return GS_ERR_INVALID_ARG;
    p.c.k += args->layer * p.c.layer_stride * es;
    p.c.v += args->layer * p.c.layer_stride * es;
    p.batch = args->batch;
    p.seq = args->seq;
    p.q_heads = args->q_heads;
    p.group = args->q_heads / p.c.heads;
    p.parts = plan.parts;
    p.part = plan.part;
    p.q = args->q;
    p.q_batch = args->q_batch_stride;
    p.q_head = args->q_head_stride;
    p.k_new = args->k_new;
    p.v_new = args->v_new;
    p.new_batch = args->new_batch_stride;
    p.new_head = args->new_head_stride;
    p.new_aligned = aligned(args->k_new, 16) && aligned(args->v_new, 16) &&
                    (args->new_batch_stride * es) % 16 == 0 && (args->new_head_stride * es) % 16 == 0;
    p.out_aligned = aligned(args->out, 4 * es) && args->out_batch_stride % 4 == 0 &&
                    args->out_head_stride % 4 == 0;
    p.q_aligned = aligned(args->q, 2 * es) && args->q_batch_stride % 2 == 0 && args->q_head_stride % 2 == 0;
    // Division by the page size: with s = ceil(log2 page), mul = 2^32 (2^s - page) / page + 1.
    p.page_shift = 0;
    while ((1u << p.page_shift) < static_cast<unsigned>(p.c.page)) ++p.page_shift;
    p.page_mul = static_cast<unsigned>(
        (((1ull << p.page_shift) - static_cast<unsigned>(p.c.page)) << 32) / static_cast<unsigned>(p.c.page) + 1);
    p.page_runs = p.c.page % plan.run == 0;
    p.dim_mul = (1u << 20) / static_cast<unsigned>(p.c.dim) + 1;
    p.scale_log2 = args->scale * kLog2e;
    p.window = args->window;
    p.sinks = args->sinks;
    p.out = args->out;
    p.out_batch = args->out_batch_stride;
    p.out_head = args->out_head_stride;
    p.lse = args->lse;
    p.arrived = static_cast<int*>(args->workspace);
    p.slots = static_cast<float*>(args->workspace) + plan.counters;
    if (args->cache->dtype == GS_DTYPE_F32) return launch_fp32(p, plan.blocks, stream);
    return launch_mma(args->cache->dtype, p, plan.blocks, stream);
}
