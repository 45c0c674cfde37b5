// Attention of chunks of new tokens over a paged cache (sm_103a): the argument checks, and the kernel
// that computes with fp32 multiply-adds, for fp32 caches.
#include <cmath>

#include "chunk_attention.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 256, kRows = 64;

// Rows of 64 queries against units of KT positions: 16 x 16 threads, of which one has 4 rows and
// KT / 16 positions of the scores, then 4 rows and DP / 16 dims of the output.
template <class T, int DP, int KT>
struct Tile {
    static constexpr int kPitch = DP + 4, kScore = KT + 4;
    struct Smem {
        float q[kRows][kPitch], k[KT][kPitch], v[KT][kPitch], s[kRows][kScore];
        float top[kRows], sum[kRows], fade[kRows];
    };
};

template <class T, int DP, int KT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using S = typename Tile<T, DP, KT>::Smem;
    using Cut = ChunkCut<kRows, kRows, KT, kThreads, kThreads>;
    constexpr int V = 16 / static_cast<int>(sizeof(T)), CH = DP / V, CPT = KT / 16, NV = DP / 64;
    extern __shared__ __align__(16) char smem[];
    S& s = *reinterpret_cast<S*>(smem);
    __shared__ typename Cut::Shared plan;
    __shared__ ChunkItem item;
    __shared__ int ok;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, dim = p.c.dim;
    grid_wait();
    grid_trigger();
    Cut cut;
    cut.s = &plan;
    cut.find(p);
    const ChunkUnits<KT> units(p.c.page);
    for (;;) {
        if (tid == 0) item = cut.item(p);
        __syncthreads();
        const ChunkItem it = item;
        __syncthreads();
        if (it.kind == 0) break;
        if (it.kind == 2) {
            if (tid == 0) ok = chunk_wait_parts(p.work + kChunkHead + it.share, it.need);
            __syncthreads();
            if (ok) chunk_join<T>(p, it, tid >> 5, kThreads / 32, 0.0f);
            else if (tid == 0) flag(p.c.status, GS_DEV_TIMEOUT);
            __syncthreads();
            continue;
        }
        // The queries, with the scale's sign; zeros past the tile's rows and past dim.
        for (int x = tid; x < kRows * CH; x += kThreads) {
            const int r = x / CH, c = x - r * CH, row = it.row + r;
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.0f;
            if (r < it.rows && c * V < dim) {
                const int t = chunk_token(p, row), h = it.head * p.group + row - t * p.group;
                const T* from = static_cast<const T*>(p.q) + (it.e.row + t) * p.q_token + h * p.q_head + c * V;
                unpack16<T>(load16_any(from, p.q_aligned != 0), f);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) s.q[r][c * V + i] = f[i] * p.q_sign;
        }
        for (int r = tid; r < kRows; r += kThreads) {
            s.top[r] = kNegInf;
            s.sum[r] = 0.0f;
        }
        float o[4][NV * 4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 0; d < NV * 4; ++d) o[i][d] = 0.0f;
        const int from = it.e.len - it.e.m;              // position of the entry's first row
        const int first_row = from + chunk_token(p, it.row), last_row = from + chunk_token(p, it.row + it.rows - 1);
        for (int n = it.lo; n < it.hi; ++n) {
            int count, in_page;
            const int at = units.first(it.span.unit(n), &count, &in_page);
            const int valid = min(count, it.e.len - at);
            __syncthreads();                             // (the last unit's rows are not read any more)
            for (int x = tid; x < KT * CH; x += kThreads) {
                const int r = x / CH, c = x - r * CH;
                uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
                if (r < valid && c * V < dim) {
                    const int col = (at + r) / p.c.page, row = at + r - col * p.c.page;
                    const int page = p.c.table[static_cast<long long>(it.e.seq) * p.c.cols + col];
                    if (page >= 0 && page < p.c.pages) {
                        const long long off = (page * p.c.page_stride + it.head * p.c.head_stride +
                                               row * p.c.token_stride + c * V) * static_cast<int>(sizeof(T));
                        k = *reinterpret_cast<const uint4*>(p.c.k + off);
                        v = *reinterpret_cast<const uint4*>(p.c.v + off);
                    } else {
                        flag(p.c.status, GS_DEV_BAD_SEQ);
                    }
                }
                unpack16<T>(k, &s.k[r][c * V]);
                unpack16<T>(v, &s.v[r][c * V]);
            }
            __syncthreads();
            float a[4][CPT];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < CPT; ++c) a[i][c] = 0.0f;
#pragma unroll 4
            for (int d = 0; d < DP; d += 4) {
                float4 q[4], k[CPT];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4*>(&s.q[ty * 4 + i][d]);
#pragma unroll
                for (int c = 0; c < CPT; ++c) k[c] = *reinterpret_cast<const float4*>(&s.k[tx + 16 * c][d]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < CPT; ++c) {
                        a[i][c] = fmaf(q[i].x, k[c].x, a[i][c]);
                        a[i][c] = fmaf(q[i].y, k[c].y, a[i][c]);
                        a[i][c] = fmaf(q[i].z, k[c].z, a[i][c]);
                        a[i][c] = fmaf(q[i].w, k[c].w, a[i][c]);
                    }
            }
            // Whether some row does not see the whole unit.
            const bool masked = valid < KT || at + KT - 1 > first_row ||
                                (p.window > 0 && at <= last_row - p.window && at + KT > p.sinks);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = it.row + ty * 4 + i, pos = from + chunk_token(p, row);
                float up = kNegInf;
                bool seen[CPT];
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const int j = at + tx + 16 * c;
                    seen[c] = !masked || (tx + 16 * c < valid && j <= pos &&
                                          (p.window == 0 || j > pos - p.window || j < p.sinks));
                    a[i][c] = seen[c] ? a[i][c] * p.scale_log2 : kNegInf;
                    up = fmaxf(up, a[i][c]);
                }
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
                const float old = s.top[ty * 4 + i];
                up = fmaxf(up, old);
                const float base = up == kNegInf ? 0.0f : up;
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const float w = chunk_pow2(a[i][c] - base);
                    if (seen[c]) sum += w;
                    s.s[ty * 4 + i][tx + 16 * c] = seen[c] ? w : -1.0f;      // -1: not to be multiplied
                }
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (tx == 0) {
                    const float fade = chunk_pow2(old - base);
                    s.top[ty * 4 + i] = up;
                    s.sum[ty * 4 + i] = fmaf(s.sum[ty * 4 + i], fade, sum);
                    s.fade[ty * 4 + i] = fade;
                }
            }
            __syncwarp();                                // a warp's rows are its own
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float fade = s.fade[ty * 4 + i];
#pragma unroll
                for (int d = 0; d < NV * 4; ++d) o[i][d] *= fade;
            }
            for (int k = 0; k < valid; ++k) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = s.s[ty * 4 + i][k];
#pragma unroll
                for (int x = 0; x < NV; ++x) {
                    const float4 v = *reinterpret_cast<const float4*>(&s.v[k][x * 64 + tx * 4]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (!masked || w[i] >= 0.0f || w[i] != w[i]) {
                            o[i][4 * x] = fmaf(w[i], v.x, o[i][4 * x]);
                            o[i][4 * x + 1] = fmaf(w[i], v.y, o[i][4 * x + 1]);
                            o[i][4 * x + 2] = fmaf(w[i], v.z, o[i][4 * x + 2]);
                            o[i][4 * x + 3] = fmaf(w[i], v.w, o[i][4 * x + 3]);
                        }
                    }
                }
            }
        }
        __syncthreads();                                 // (the first values of top and sum, where no unit came)
        float* const slot = p.slots + it.slot * chunk_slot_words(p.slot_rows, dim);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= it.rows) continue;
            const float sum = s.sum[r], top = s.top[r];
            if (it.parts == 1) {
                const float by = sum > 0.0f ? 1.0f / sum : sum;      // a NaN stays one
                float* lse;
                T* const to = chunk_out<T>(p, it, it.row + r, &lse);
#pragma unroll
                for (int x = 0; x < NV; ++x)
                    if (x * 64 + tx * 4 < dim)
                        chunk_put4<T>(p, to + x * 64 + tx * 4,
                                      make_float4(o[i][4 * x] * by, o[i][4 * x + 1] * by, o[i][4 * x + 2] * by,
                                                  o[i][4 * x + 3] * by));
                if (tx == 0 && lse != nullptr) *lse = sum == 0.0f ? kNegInf : (top + log2f(sum)) * kChunkLn2;
            } else {
#pragma unroll
                for (int x = 0; x < NV; ++x)
                    if (x * 64 + tx * 4 < dim)
                        *reinterpret_cast<float4*>(slot + 2 * p.slot_rows + static_cast<long long>(r) * dim +
                                                   x * 64 + tx * 4) =
                            make_float4(o[i][4 * x], o[i][4 * x + 1], o[i][4 * x + 2], o[i][4 * x + 3]);
                if (tx == 0) {
                    slot[r] = top;
                    slot[p.slot_rows + r] = sum;
                }
            }
        }
        if (it.parts > 1) {
            __threadfence();
            __syncthreads();
            if (tid == 0) atomicAdd(p.work + kChunkHead + it.share, 1);
        }
    }
    if (tid < 32) chunk_leave(p, cut.used());
}

template <class T, int DP, int KT>
gs_status launch_as(const ChunkParams& p, int blocks, gs_stream stream) {
    const int bytes = static_cast<int>(sizeof(typename Tile<T, DP, KT>::Smem));
    if (!allow_smem<chunk_kernel<T, DP, KT>>(bytes)) return GS_ERR_CUDA;
    return launch(chunk_kernel<T, DP, KT>, dim3(blocks), kThreads, bytes, 1, stream, p);
}

}  // namespace

ChunkShape chunk_fp32_shape(int) { return {kRows, sm_count()}; }

gs_status launch_chunk_fp32(const ChunkParams& p, int blocks, gs_stream stream) {
    if (p.c.dim <= 64) return launch_as<float, 64, 64>(p, blocks, stream);
    if (p.c.dim <= 128) return launch_as<float, 128, 64>(p, blocks, stream);
    return launch_as<float, 256, 32>(p, blocks, stream);
}

namespace {

struct Plan {
    ChunkShape shape;
    int slots, rows;
};

gs_status plan_of(const gs_chunk_attention_args* a, Plan* plan) {
    if (a == nullptr) return GS_ERR_INVALID_ARG;
    const gs_status st = check_cache_sizes(a->cache);
    if (st != GS_OK) return st;
    const gs_kv_cache* c = a->cache;
    if (a->n < 0 || a->tokens < 0 || a->q_heads < 1 || a->q_heads % c->kv_heads != 0 || a->window < 0 ||
        a->sinks < 0 || (a->sinks > 0 && a->window == 0))
        return GS_ERR_INVALID_ARG;
    if (a->n > GS_MAX_SEQS || a->q_heads > (1 << 16)) return GS_ERR_UNSUPPORTED;
    // Rows of an entry, and items of the call, count in 32 bits.
    const long long group = a->q_heads / c->kv_heads;
    if (a->tokens * group > (1ll << 30) || static_cast<long long>(a->tokens) * a->q_heads > (1ll << 30) ||
        static_cast<long long>(a->n) * c->kv_heads > (1ll << 28))
        return GS_ERR_UNSUPPORTED;
    plan->shape = c->dtype == GS_DTYPE_F32 ? chunk_fp32_shape(c->dim) : chunk_mma_shape(c->dim);
    const long long rows = (a->tokens * group + 7) / 8 * 8;
    plan->rows = static_cast<int>(rows < plan->shape.rows ? rows : plan->shape.rows);
    if (plan->shape.blocks > kChunkShares) plan->shape.blocks = kChunkShares;
    plan->slots = a->tokens == 0 || a->n == 0 ? 0 : 2 * plan->shape.blocks;
    return GS_OK;
}

long long need_of(const gs_chunk_attention_args* a, const Plan& plan) {
    return 4ll * (kChunkCounters + plan.slots * chunk_slot_words(plan.rows, a->cache->dim));
}

}  // namespace
}  // namespace gs_decode

using namespace gs_decode;

extern "C" gs_status gs_chunk_attention_workspace(const gs_chunk_attention_args* args, int64_t* bytes) {
    if (bytes == nullptr) return GS_ERR_INVALID_ARG;
    Plan plan;
    const gs_status st = plan_of(args, &plan);
    if (st != GS_OK) return st;
    *bytes = need_of(args, plan);
    return GS_OK;
}

extern "C" gs_status gs_chunk_attention(const gs_chunk_attention_args* args, gs_stream stream) {
    Plan plan;
    gs_status st = plan_of(args, &plan);
    if (st != GS_OK) return st;
    ChunkParams p = {};
    st = check_cache(args->cache, &p.c);
    if (st != GS_OK) return st;
    const long long es = elem_size(args->cache->dtype);
    if (args->layer < 0 || args->layer >= p.c.layers || !std::isfinite(args->scale)) return GS_ERR_INVALID_ARG;
    if (args->tokens == 0 || args->n == 0) return GS_OK;
    if (args->q == nullptr || args->out == nullptr || args->seq == nullptr || args->start == nullptr ||
        !aligned(args->q, es) || !aligned(args->out, es) || !aligned(args->lse, 4) ||
        !aligned(args->seq, 4) || !aligned(args->start, 4))
        return GS_ERR_INVALID_ARG;
    if (args->q_token_stride < 0 || args->q_head_stride < 0) return GS_ERR_INVALID_ARG;
    if ((args->tokens > 1 && args->out_token_stride < p.c.dim) ||
        (args->q_heads > 1 && args->out_head_stride < p.c.dim))
        return GS_ERR_INVALID_ARG;                        // output rows overlap
    if (args->workspace == nullptr || !aligned(args->workspace, 16) ||
        args->workspace_bytes < need_of(args, plan))
        return GS_ERR_INVALID_ARG;
    p.c.k += args->layer * p.c.layer_stride * es;
    p.c.v += args->layer * p.c.layer_stride * es;
    p.n = args->n;
    p.tokens = args->tokens;
    p.seq = args->seq;
    p.start = args->start;
    p.q_heads = args->q_heads;
    p.group = args->q_heads / p.c.heads;
    // Division by the group: with s = ceil(log2 group), mul = 2^32 (2^s - group) / group + 1.
    while ((1u << p.group_shift) < static_cast<unsigned>(p.group)) ++p.group_shift;
    p.group_mul = static_cast<unsigned>(
        (((1ull << p.group_shift) - static_cast<unsigned>(p.group)) << 32) / static_cast<unsigned>(p.group) + 1);
    p.tile_step = 16 * plan.shape.rows / p.group;
    p.q = args->q;
    p.q_token = args->q_token_stride;
    p.q_head = args->q_head_stride;
    p.q_aligned = aligned(args->q, 16) && (args->q_token_stride * es) % 16 == 0 && (args->q_head_stride * es) % 16 == 0;
    p.out_aligned = aligned(args->out, 16) && (args->out_token_stride * es) % 16 == 0 &&
                    (args->out_head_stride * es) % 16 == 0;
    p.out_wide = aligned(args->out, 32) && (args->out_token_stride * es) % 32 == 0 && (args->out_head_stride * es) % 32 == 0;
    p.slots_wide = aligned(args->workspace, 32);
    // Scores are kept in powers of two, the largest first: a negative scale turns the queries' signs,
    // and scale 0 makes them 0.
    p.scale_log2 = args->scale == 0.0f ? 1.0f : std::fabs(args->scale) * kChunkLog2e;
    p.q_sign = args->scale > 0.0f ? 1.0f : args->scale < 0.0f ? -1.0f : 0.0f;
    p.window = args->window;
    p.sinks = args->sinks;
    p.out = args->out;
    p.out_token = args->out_token_stride;
    p.out_head = args->out_head_stride;
    p.lse = args->lse;
    p.work = static_cast<int*>(args->workspace);
    p.slots = static_cast<float*>(args->workspace) + kChunkCounters;
    p.slot_rows = plan.rows;
    if (args->cache->dtype == GS_DTYPE_F32) return launch_chunk_fp32(p, plan.shape.blocks, stream);
    return launch_chunk_mma(args->cache->dtype, p, plan.shape.blocks, stream);
}
