// Attention of one new token over a paged cache: the argument checks, and the kernel that
// computes with fp32 multiply-adds (sm_103a).
//
// For each query head and visible position: s = q . k (fp32), the running maximum and sum of a
// softmax in powers of two, and o += 2^(s - m) v.  K and V are read once for `part` query heads
// that share them.  Eight lanes hold a row of K (16 bytes a lane and vector, so a warp reads
// four rows at a time, coalesced); each group of eight lanes keeps a maximum, sum and output of
// its own, and they meet once a segment, by shuffles and then through shared memory.
#include <cmath>

#include "paged_attention.cuh"

namespace gs_decode {
namespace {

// Values of a row that a lane holds, for rows of up to 8 * E values; query heads of a part: the
// output takes PART * E = 64 registers.
template <class T, int NV>
struct Shape {
    static constexpr int V = 16 / sizeof(T);
    static constexpr int E = NV * V;
    static constexpr int PART = 64 / E;
    static constexpr int DIM = 8 * E;
};

template <class T, int NV>
__global__ void __launch_bounds__(kThreads)
attention_kernel(const __grid_constant__ AttnParams p) {
    using S = Shape<T, NV>;
    constexpr int V = S::V, E = S::E, PART = S::PART, DIM = S::DIM, U = 2;
    extern __shared__ int at[];                          // [batch + 1]
    __shared__ int tmp[kWarps + 1];
    __shared__ int turn;
    __shared__ __align__(16) float sq[PART * DIM];       // the query heads, scaled
    __shared__ float sm[kWarps][PART], ss[kWarps][PART];
    __shared__ float so[kWarps][PART * DIM];
    __shared__ float rm[PART], rs[PART];
    grid_wait();
    grid_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & 7, group = lane >> 3;
    const int dim = p.c.dim;
    number_tiles(p, at, tmp);
    put_empty_rows<T>(p, at);
    Walk walk;
    walk.begin(p, at);
    while (walk.t < walk.t1) {
        const Segment seg = walk.next(p, at);
        const int first_head = seg.head * p.group + seg.part * PART;
        const int heads = min(PART, p.group - seg.part * PART);
        for (int x = threadIdx.x; x < PART * DIM; x += kThreads) {
            const int g = x / DIM, d = x - g * DIM;
            float f = 0.0f;
            if (g < heads && d < dim)
                f = to_float(static_cast<const T*>(p.q)[seg.b * p.q_batch +
                                                        (first_head + g) * p.q_head + d]);
            sq[x] = f * p.scale_log2;
        }
        __syncthreads();
        const int* table = p.c.table + static_cast<long long>(seg.row.seq) * p.c.cols;
        const long long head_at = p.layer * p.c.layer_stride + seg.head * p.c.head_stride;
        T* const kc = reinterpret_cast<T*>(p.c.k) + head_at;
        T* const vc = reinterpret_cast<T*>(p.c.v) + head_at;
        const T* const kn = static_cast<const T*>(p.k_new) + (p.k_new != nullptr ? seg.b * p.new_batch + seg.head * p.new_head : 0);
        const T* const vn = static_cast<const T*>(p.v_new) + (p.k_new != nullptr ? seg.b * p.new_batch + seg.head * p.new_head : 0);
        float m[PART], sum[PART], o[PART][E];
#pragma unroll
        for (int g = 0; g < PART; ++g) {
            m[g] = kNegInf;
            sum[g] = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[g][e] = 0.0f;
        }
        for (int j0 = seg.first + warp * 4 * U; j0 < seg.last; j0 += kWarps * 4 * U) {
            uint4 k[U][NV], v[U][NV];
            bool seen[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * 4 + group;
                seen[u] = j < seg.last;
                const int pos = position(seg.row, seen[u] ? j : seg.first);
                const int col = pos / p.c.page;
                const int pg = table[col];
                const bool ok = pg >= 0 && pg < p.c.pages;
                const long long off = (ok ? pg : 0) * p.c.page_stride +
                                      (pos - col * p.c.page) * p.c.token_stride;
                const bool fresh = seen[u] && p.k_new != nullptr && pos == seg.row.len - 1;
                if (!ok && sub == 0) flag(p.c.status, GS_DEV_BAD_SEQ);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int d = (sub + 8 * i) * V;
                    k[u][i] = v[u][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (d >= dim || !seen[u]) continue;
                    if (fresh) {
                        k[u][i] = load16_any(kn + d, p.new_aligned != 0);
                        v[u][i] = load16_any(vn + d, p.new_aligned != 0);
                        if (ok && seg.part == 0) {
                            *reinterpret_cast<uint4*>(kc + off + d) = k[u][i];
                            *reinterpret_cast<uint4*>(vc + off + d) = v[u][i];
                        }
                    } else if (ok) {
                        k[u][i] = *reinterpret_cast<const uint4*>(kc + off + d);
                        v[u][i] = *reinterpret_cast<const uint4*>(vc + off + d);
                    }
                }
            }
            float s[U][PART];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int g = 0; g < PART; ++g) s[u][g] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float kf[U][V];
#pragma unroll
                for (int u = 0; u < U; ++u) unpack16<T>(k[u][i], kf[u]);
#pragma unroll
                for (int g = 0; g < PART; ++g) {
                    const float* qp = sq + g * DIM + (sub + 8 * i) * V;
#pragma unroll
                    for (int e = 0; e < V; e += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(qp + e);
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            s[u][g] = fmaf(f.x, kf[u][e], s[u][g]);
                            s[u][g] = fmaf(f.y, kf[u][e + 1], s[u][g]);
                            s[u][g] = fmaf(f.z, kf[u][e + 2], s[u][g]);
                            s[u][g] = fmaf(f.w, kf[u][e + 3], s[u][g]);
                        }
                    }
                }
            }
#pragma unroll
            for (int g = 0; g < PART; ++g) {
                float top = m[g];
#pragma unroll
                for (int u = 0; u < U; ++u) {
#pragma unroll
                    for (int d = 1; d < 8; d <<= 1) s[u][g] += __shfl_xor_sync(0xffffffffu, s[u][g], d);
                    if (!seen[u]) s[u][g] = kNegInf;
                    top = fmaxf(top, s[u][g]);
                }
                if (top > m[g]) {
                    const float w = exp2f(m[g] - top);           // 0 at the first position
                    sum[g] *= w;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[g][e] *= w;
                    m[g] = top;
                }
                const float base = top == kNegInf ? 0.0f : top;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u][g] = exp2f(s[u][g] - base);
                    sum[g] += s[u][g];
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float vf[V];
                    unpack16<T>(v[u][i], vf);
#pragma unroll
                    for (int g = 0; g < PART; ++g)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            o[g][i * V + e] = fmaf(s[u][g], vf[e], o[g][i * V + e]);
                }
        }
        // The four groups of the warp, then the warps.
#pragma unroll
        for (int g = 0; g < PART; ++g) {
            float top = m[g];
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float w = exp2f(m[g] - (top == kNegInf ? 0.0f : top));
            sum[g] *= w;
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 8);
            sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 16);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                float x = o[g][e] * w;
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (group == 0) so[warp][g * DIM + (sub + 8 * (e / V)) * V + e % V] = x;
            }
            if (lane == 0) {
                sm[warp][g] = top;
                ss[warp][g] = sum[g];
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < PART * dim; x += kThreads) {
            const int g = x / dim, d = x - g * dim;
            float top = kNegInf;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w][g]);
            const float base = top == kNegInf ? 0.0f : top;
            float acc = 0.0f, all = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2f(sm[w][g] - base);
                acc = fmaf(so[w][g * DIM + d], f, acc);
                all = fmaf(ss[w][g], f, all);
            }
            sq[x] = acc;                                  // the queries are not needed any more
            if (d == 0) {
                rm[g] = top;
                rs[g] = all;
            }
        }
        __syncthreads();
        finish<T>(p, seg, rm, rs, sq, &turn);
    }
}

template <class T, int NV>
gs_status launch_one(const AttnParams& p, int blocks, gs_stream stream) {
    const int smem = 4 * (p.batch + 1);
    if (!allow_smem<attention_kernel<T, NV>>(smem + 24 * 1024)) return GS_ERR_CUDA;
    return launch(attention_kernel<T, NV>, dim3(static_cast<unsigned>(blocks)), kThreads, smem, 1,
                  stream, p);
}

// 16-byte vectors a lane holds of a row: 1, 2, 4 or 8.
int vectors_of(int dtype, int dim) {
    const int v = static_cast<int>((dim * elem_size(dtype) / 16 + 7) / 8);
    return v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8;
}
int part_of(int dtype, int dim) {
    return 64 / static_cast<int>(vectors_of(dtype, dim) * 16 / elem_size(dtype));
}

template <class T>
gs_status launch_simple(int dtype, const AttnParams& p, int blocks, gs_stream stream) {
    switch (vectors_of(dtype, p.c.dim)) {
        case 1: return launch_one<T, 1>(p, blocks, stream);
        case 2: return launch_one<T, 2>(p, blocks, stream);
        case 4: return launch_one<T, 4>(p, blocks, stream);
        default:
            if constexpr (sizeof(T) == 4) return launch_one<T, 8>(p, blocks, stream);
            return GS_ERR_UNSUPPORTED;
    }
}

struct Plan {
    int part, parts, blocks;
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
    plan->part = part_of(c->dtype, c->dim);
    if (plan->part > group) plan->part = group;
    plan->parts = (group + plan->part - 1) / plan->part;
    long long most = static_cast<long long>(c->cols) * c->page;
    const long long visible = static_cast<long long>(a->window) + a->sinks;
    if (a->window > 0 && visible < most) most = visible;
    const long long tiles = a->batch * ((most + kTile - 1) / kTile);
    const long long items = static_cast<long long>(a->batch) * c->kv_heads * plan->parts;
    if (tiles > 0x7fffffffll || items > 0x3fffffffll) return GS_ERR_UNSUPPORTED;
    // Two blocks an SM (registers), no more blocks than tiles.
    const long long full = 2ll * sm_count();
    const long long all = tiles * c->kv_heads * plan->parts;
    plan->blocks = static_cast<int>(all < full ? (all > 0 ? all : 1) : full);
    plan->counters = (items + 3) / 4 * 4;
    plan->slots = 2ll * plan->blocks * plan->part * (c->dim + 2);
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
    p.layer = args->layer;
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
    p.scale_log2 = args->scale * kLog2e;
    p.window = args->window;
    p.sinks = args->sinks;
    p.out = args->out;
    p.out_batch = args->out_batch_stride;
    p.out_head = args->out_head_stride;
    p.lse = args->lse;
    p.arrived = static_cast<int*>(args->workspace);
    p.slots = static_cast<float*>(args->workspace) + plan.counters;
    switch (args->cache->dtype) {
        case GS_DTYPE_F32: return launch_simple<float>(args->cache->dtype, p, plan.blocks, stream);
        case GS_DTYPE_BF16:
            return launch_simple<__nv_bfloat16>(args->cache->dtype, p, plan.blocks, stream);
        default: return launch_simple<__half>(args->cache->dtype, p, plan.blocks, stream);
    }
}
