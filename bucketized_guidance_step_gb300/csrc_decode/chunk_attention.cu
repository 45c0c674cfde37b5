// Attention of chunks of new tokens over a paged cache (sm_103a): the argument checks, and the kernel
// that computes with fp32 multiply-adds, for fp32 caches.
//
// A block has a tile of 64 query rows and reads units of 64 positions (32 for heads of over 128 dims) by
// 16-byte asynchronous copies, one unit ahead; where a unit's rows lie is looked up a unit before that.  Its
// 16 x 16 threads have 4 rows and 4 positions (2) of the scores each, then 4 rows and every 16th group of 4
// dims of the output.  Multiply-adds are two at a time (fma.rn.f32x2): over pairs of dims in the scores,
// whose two sums are added at the end, and over pairs of outputs.
#include <cmath>

#include "chunk_attention.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 256, kRows = 64;

template <int DP, int KT>
struct Tile {
    static constexpr int kPitch = DP + 4, kScore = KT + 4;
    struct Smem {
        float q[kRows][kPitch], k[2][KT][kPitch], v[2][KT][kPitch], s[kRows][kScore];
        float top[kRows], sum[kRows], fade[kRows];
        long long at[3][KT];              // bytes of a position's row in K and V; -1: read as zeros
    };
};

using Pair = unsigned long long;
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair twice(float x) {
    Pair r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float2 halves(Pair p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
// 16 bytes from global to shared memory; size 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(void* to, const void* from, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<unsigned>(__cvta_generic_to_shared(to))),
                 "l"(from), "r"(size)
                 : "memory");
}

template <int DP, int KT>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using S = typename Tile<DP, KT>::Smem;
    using Cut = ChunkCut<kRows, kRows, KT, kThreads, kThreads>;
    constexpr int CPT = KT / 16, NV = DP / 64;
    extern __shared__ __align__(16) char smem[];
    S& s = *reinterpret_cast<S*>(smem);
    __shared__ typename Cut::Shared plan;
    __shared__ ChunkItem item;
    __shared__ int ok;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, dim = p.c.dim, pieces = dim / 4;
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
            if (ok) chunk_join<float>(p, it, tid >> 5, kThreads / 32, 0.0f);
            else if (tid == 0) flag(p.c.status, GS_DEV_TIMEOUT);
            __syncthreads();
            continue;
        }
        const int count = it.hi - it.lo;
        // Where unit u's rows lie (KT threads); its copies (all).
        auto look_up = [&](int u) {
            if (u >= count || tid >= KT) return;
            int here, in_page;
            const int at = units.first(it.span.unit(it.lo + u), &here, &in_page);
            long long off = -1;
            if (tid < min(here, it.e.len - at)) {
                const int col = (at + tid) / p.c.page, row = at + tid - col * p.c.page;
                const int page = p.c.table[static_cast<long long>(it.e.seq) * p.c.cols + col];
                if (page >= 0 && page < p.c.pages)
                    off = 4 * (page * p.c.page_stride + it.head * p.c.head_stride + row * p.c.token_stride);
                else
                    flag(p.c.status, GS_DEV_BAD_SEQ);
            }
            s.at[u % 3][tid] = off;
        };
        auto load = [&](int u) {
            if (u < count) {
                for (int x = tid; x < KT * pieces; x += kThreads) {
                    const int r = x / pieces, c = x - r * pieces;
                    const long long off = s.at[u % 3][r];
                    const int size = off >= 0 ? 16 : 0;
                    const long long from = off >= 0 ? off + 16 * c : 0;
                    copy16(&s.k[u & 1][r][4 * c], p.c.k + from, size);
                    copy16(&s.v[u & 1][r][4 * c], p.c.v + from, size);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look_up(0);
        look_up(1);
        // The queries, with the scale's sign; zeros past the tile's rows.
        for (int x = tid; x < kRows * pieces; x += kThreads) {
            const int r = x / pieces, c = x - r * pieces, row = it.row + r;
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < it.rows) {
                const int t = chunk_token(p, row), h = it.head * p.group + row - t * p.group;
                const float* from = static_cast<const float*>(p.q) + (it.e.row + static_cast<long long>(t)) * p.q_token +
                                    h * p.q_head + c * 4;
                unpack16<float>(load16_any(from, p.q_aligned != 0), &f.x);
            }
            *reinterpret_cast<float4*>(&s.q[r][c * 4]) =
                make_float4(f.x * p.q_sign, f.y * p.q_sign, f.z * p.q_sign, f.w * p.q_sign);
        }
        for (int r = tid; r < kRows; r += kThreads) {
            s.top[r] = kNegInf;
            s.sum[r] = 0.0f;
        }
        Pair o[4][NV][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < NV; ++x) o[i][x][0] = o[i][x][1] = 0ull;
        const int from = it.e.len - it.e.m;              // position of the entry's first row
        const int first_row = from + chunk_token(p, it.row), last_row = from + chunk_token(p, it.row + it.rows - 1);
        int pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pos[i] = from + chunk_token(p, it.row + ty * 4 + i);
        __syncthreads();
        load(0);
        for (int u = 0; u < count; ++u) {
            int here, in_page;
            const int at = units.first(it.span.unit(it.lo + u), &here, &in_page);
            const int valid = min(here, it.e.len - at), now = u & 1;
            load(u + 1);
            look_up(u + 2);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads();
            Pair a[4][CPT];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < CPT; ++c) a[i][c] = 0ull;
#pragma unroll 2
            for (int d = 0; d < dim; d += 4) {
                ulonglong2 q[4], k[CPT];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const ulonglong2*>(&s.q[ty * 4 + i][d]);
#pragma unroll
                for (int c = 0; c < CPT; ++c) k[c] = *reinterpret_cast<const ulonglong2*>(&s.k[now][tx + 16 * c][d]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < CPT; ++c) a[i][c] = fma2(q[i].y, k[c].y, fma2(q[i].x, k[c].x, a[i][c]));
            }
            // Whether some row does not see the whole unit.
            const bool masked = valid < KT || at + KT - 1 > first_row ||
                                (p.window > 0 && at <= last_row - p.window && at + KT > p.sinks);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float up = kNegInf, x[CPT];
                bool seen[CPT];
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const int j = at + tx + 16 * c;
                    const float2 h = halves(a[i][c]);
                    seen[c] = !masked || (tx + 16 * c < valid && j <= pos[i] &&
                                          (p.window == 0 || j > pos[i] - p.window || j < p.sinks));
                    x[c] = seen[c] ? (h.x + h.y) * p.scale_log2 : kNegInf;
                    up = fmaxf(up, x[c]);
                }
#pragma unroll
                for (int d = 1; d < 16; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
                const float old = s.top[ty * 4 + i];
                up = fmaxf(up, old);
                const float base = up == kNegInf ? 0.0f : up;
                float sum = 0.0f;
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const float w = chunk_pow2(x[c] - base);
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
                const Pair fade = twice(s.fade[ty * 4 + i]);
#pragma unroll
                for (int x = 0; x < NV; ++x) {
                    o[i][x][0] = mul2(o[i][x][0], fade);
                    o[i][x][1] = mul2(o[i][x][1], fade);
                }
            }
            // O += P V, V's infinities and NaN only to rows that see them.
            auto add = [&](auto only_seen) {
#pragma unroll 4
                for (int k = 0; k < valid; ++k) {
                    float w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = s.s[ty * 4 + i][k];
#pragma unroll
                    for (int x = 0; x < NV; ++x) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&s.v[now][k][x * 64 + tx * 4]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (!decltype(only_seen)::value || !(w[i] < 0.0f)) {
                                o[i][x][0] = fma2(twice(w[i]), v.x, o[i][x][0]);
                                o[i][x][1] = fma2(twice(w[i]), v.y, o[i][x][1]);
                            }
                        }
                    }
                }
            };
            if (masked) add(std::true_type());
            else add(std::false_type());
            __syncthreads();                             // (the unit's place is filled again)
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                                 // (the first values of top and sum, where no unit came)
        float* const slot = p.slots + it.slot * chunk_slot_words(p.slot_rows, dim);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= it.rows) continue;
            const float sum = s.sum[r], top = s.top[r];
            const bool whole = it.parts == 1;
            const float by = !whole ? 1.0f : sum > 0.0f ? 1.0f / sum : sum;          // a NaN stays one
            float* lse = nullptr;
            float* const to = whole ? chunk_out<float>(p, it, it.row + r, &lse)
                                    : slot + 2 * p.slot_rows + static_cast<long long>(r) * dim;
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                if (x * 64 + tx * 4 >= dim) continue;
                const float2 lo = halves(o[i][x][0]), hi = halves(o[i][x][1]);
                const float4 f = make_float4(lo.x * by, lo.y * by, hi.x * by, hi.y * by);
                if (whole) chunk_put4<float>(p, to + x * 64 + tx * 4, f);
                else *reinterpret_cast<float4*>(to + x * 64 + tx * 4) = f;
            }
            if (tx == 0 && whole && lse != nullptr) *lse = sum == 0.0f ? kNegInf : (top + log2f(sum)) * kChunkLn2;
            if (tx == 0 && !whole) {
                slot[r] = top;
                slot[p.slot_rows + r] = sum;
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

template <int DP, int KT>
gs_status launch_as(const ChunkParams& p, int blocks, gs_stream stream) {
    const int bytes = static_cast<int>(sizeof(typename Tile<DP, KT>::Smem));
    if (!allow_smem<chunk_kernel<DP, KT>>(bytes)) return GS_ERR_CUDA;
    return launch(chunk_kernel<DP, KT>, dim3(blocks), kThreads, bytes, 1, stream, p);
}

}  // namespace

ChunkShape chunk_fp32_shape(int) { return {kRows, sm_count()}; }

gs_status launch_chunk_fp32(const ChunkParams& p, int blocks, gs_stream stream) {
    if (p.c.dim <= 64) return launch_as<64, 64>(p, blocks, stream);
    if (p.c.dim <= 128) return launch_as<128, 64>(p, blocks, stream);
    return launch_as<256, 32>(p, blocks, stream);
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
