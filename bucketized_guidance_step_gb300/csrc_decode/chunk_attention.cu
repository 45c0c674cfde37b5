// Attention of chunks of new tokens over a paged cache (sm_103a): the argument checks, and the kernel
// for fp32 caches.
//
// Its products run on the tensor cores with numbers split in two: x = hi + lo, hi 11 bits of it, and
// x y = hi hi' + hi lo' + lo hi' up to about 2^-21 of it, sums in fp32 (mma.sync m16n8k8).  8 chunks of up to
// 129 tokens over up to 1001, 8 and 4 heads of 96, take 90 us; a 64 x 64 tile of fp32 multiply-adds from
// shared memory, whose reads bound it, took 123 us.  Now the warps wait for each other: two barriers a unit,
// and the next item, which one thread finds (issue slots 26 % busy, tensor pipe 19 %, HBM 2 %); a warp of its own for
// that would take the registers that two blocks an SM leave.
//
// A block has a tile of 64 query rows and reads units of 32 positions by 16-byte asynchronous copies, one
// unit ahead; where a unit's rows lie is looked up a unit before that.  Of its 8 warps, each has 16 rows and
// half of every unit's positions, with a softmax and an output of its own; the two halves meet at the item's
// end.  The scores' fragments are the second product's operands as they are: a step takes positions 2 t and
// 2 t + 1 where the instruction numbers them t and t + 4, and reads V's rows likewise.
#include <cmath>
#include <limits>

#include "chunk_attention.cuh"

namespace gs_decode {
namespace {

constexpr int kThreads = 256, kRows = 64;
constexpr int KT = 32;                    // positions of a unit

template <int DP>
struct Tile {
    static constexpr int kPitch = DP + 4; // (8 rows' neighbours in 32 banks)
    struct Smem {
        float q[kRows][kPitch], k[2][KT][kPitch], v[2][KT][kPitch];
        long long at[3][KT];              // bytes of a position's row in K and V; -1: read as zeros
        float top[kRows], sum[kRows];
    };
};

// 16 bytes from global to shared memory; size 0 fills with zeros and reads nothing.
__device__ __forceinline__ void copy16(void* to, const void* from, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<unsigned>(__cvta_generic_to_shared(to))),
                 "l"(from), "r"(size)
                 : "memory");
}
// x = hi + lo: hi rounded to 11 bits (a), or cut to them (b: one operation less).
__device__ __forceinline__ void split_a(float x, unsigned* hi, unsigned* lo) {
    *hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    *lo = __float_as_uint(x - __uint_as_float(*hi));
}
__device__ __forceinline__ void split_b(float x, unsigned* hi, unsigned* lo) {
    *hi = __float_as_uint(x) & 0xffffe000u;
    *lo = __float_as_uint(x - __uint_as_float(*hi));
}
__device__ __forceinline__ void mma(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// big + small += a b, a split already.  The tensor cores cut their sums instead of rounding them: sums stay short,
// the small products have one of their own, and are added up by rounded additions.
__device__ __forceinline__ void mma_split(float (&big)[4], float (&small)[4], const unsigned (&hi)[4], const unsigned (&lo)[4],
                                          float b0, float b1) {
    unsigned h0, l0, h1, l1;
    split_b(b0, &h0, &l0);
    split_b(b1, &h1, &l1);
    mma(small, lo, h0, h1);
    mma(small, hi, l0, l1);
    mma(big, hi, h0, h1);
}

template <int DP>
__global__ void __launch_bounds__(kThreads, DP > 128 ? 1 : 2) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using S = typename Tile<DP>::Smem;
    using Cut = ChunkCut<kRows, kRows, KT, kThreads, kThreads>;
    constexpr int NT = DP / 8;            // groups of 8 dims
    extern __shared__ __align__(16) char smem[];
    S& s = *reinterpret_cast<S*>(smem);
    __shared__ typename Cut::Shared plan;
    __shared__ ChunkItem item;
    __shared__ int ok;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, dim = p.c.dim, pieces = dim / 4;
    const int r0 = warp / 2 * 16, half = warp & 1, g = lane >> 2, t = lane & 3;      // rows r0 + g, r0 + g + 8
    const int steps = (dim + 7) / 8;
    // (Dims from dim on, up to the next multiple of 8.)
    for (int x = tid; x < (kRows + 4 * KT) * 4; x += kThreads) s.q[x / 4][dim + x % 4] = 0.0f;
    grid_wait();
    grid_trigger();
    Cut cut;
    cut.s = &plan;
    cut.ticket = tid == 0 ? atomicAdd(p.work, 1) : -1;
    cut.find(p);
    const ChunkUnits<KT> units(p.unit_page);
    for (;;) {
        if (tid == 0) chunk_next_item(&cut, p, &item);
        __syncthreads();
        const ChunkItem it = item;
        __syncthreads();
        if (it.kind == 0) break;
        if (it.kind == 2) {
            if (tid == 0) ok = chunk_wait_parts(p.work + kChunkHead + it.share, it.need, plan.guard.limit);
            __syncthreads();
            if (ok) chunk_join<float>(p, it, warp, kThreads / 32, 0.0f);
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
                // A warp has every 8th row, a lane every 32nd piece of it.
                for (int r = warp; r < KT; r += kThreads / 32) {
                    const long long off = s.at[u % 3][r];
                    const int size = off >= 0 ? 16 : 0;
                    for (int c = lane; c < pieces; c += 32) {
                        const long long from = off >= 0 ? off + 16 * c : 0;
                        copy16(&s.k[u & 1][r][4 * c], p.c.k + from, size);
                        copy16(&s.v[u & 1][r][4 * c], p.c.v + from, size);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        look_up(0);
        look_up(1);
        // The queries, with the scale's sign; zeros past the tile's rows.
        for (int r = warp; r < kRows; r += kThreads / 32) {
            const int row = it.row + r, token = chunk_token(p, row), h = it.head * p.group + row - token * p.group;
            const float* const from = static_cast<const float*>(p.q) + (it.e.row + static_cast<long long>(token)) * p.q_token +
                                      h * p.q_head;
            for (int c = lane; c < pieces; c += 32) {
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (r < it.rows) unpack16<float>(load16_any(from + 4 * c, p.q_aligned != 0), &f.x);
                *reinterpret_cast<float4*>(&s.q[r][c * 4]) =
                    make_float4(f.x * p.q_sign, f.y * p.q_sign, f.z * p.q_sign, f.w * p.q_sign);
            }
        }
        float o[NT][4], top[2] = {kNegInf, kNegInf}, sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.0f;
        const int from = it.e.len - it.e.m;              // position of the entry's first row
        const int first_row = from + chunk_token(p, it.row), last_row = from + chunk_token(p, it.row + it.rows - 1);
        const int pos[2] = {from + chunk_token(p, it.row + r0 + g), from + chunk_token(p, it.row + r0 + g + 8)};
        __syncthreads();
        load(0);
        for (int u = 0; u < count; ++u) {
            int here, in_page;
            const int at = units.first(it.span.unit(it.lo + u), &here, &in_page);
            const int valid = min(here, it.e.len - at), now = u & 1;
            load(u + 1);
            look_up(u + 2);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            // Whether V has an infinity or NaN here: each thread looks at what it copied.
            float zero = 0.0f;
            for (int r = warp; r < KT; r += kThreads / 32)
                for (int c = lane; c < pieces; c += 32) {
                    const float4 f = *reinterpret_cast<const float4*>(&s.v[now][r][4 * c]);
                    zero = fmaf(f.x, 0.0f, fmaf(f.y, 0.0f, fmaf(f.z, 0.0f, fmaf(f.w, 0.0f, zero))));
                }
            const bool odd = __syncthreads_or(zero != 0.0f) != 0;
            // The scores of 16 rows and this half's 16 positions.
            float x[2][4], small[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] = small[n][i] = 0.0f;
            const float(*const kk)[Tile<DP>::kPitch] = s.k[now] + half * 16;
            const float(*const vv)[Tile<DP>::kPitch] = s.v[now] + half * 16;
            for (int d0 = 0; d0 < steps; d0 += 2) {
                float big[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) big[n][i] = 0.0f;
#pragma unroll
                for (int d = d0; d < d0 + 2; ++d) {
                    if (d >= steps) break;
                    unsigned hi[4], lo[4];
                    split_a(s.q[r0 + g][8 * d + t], &hi[0], &lo[0]);
                    split_a(s.q[r0 + g + 8][8 * d + t], &hi[1], &lo[1]);
                    split_a(s.q[r0 + g][8 * d + t + 4], &hi[2], &lo[2]);
                    split_a(s.q[r0 + g + 8][8 * d + t + 4], &hi[3], &lo[3]);
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        mma_split(big[n], small[n], hi, lo, kk[8 * n + g][8 * d + t], kk[8 * n + g][8 * d + t + 4]);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[n][i] += big[n][i];
            }
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[n][i] += small[n][i];
            // Infinities and NaNs (of queries or K) do not pass through split products.
            float bad = 0.0f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) bad = fmaf(x[n][i], 0.0f, bad);
            if (__any_sync(0xffffffffu, bad != 0.0f)) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (fabsf(x[n][i]) < __builtin_huge_valf()) continue;
                        x[n][i] = 0.0f;
                        for (int d = 0; d < dim; ++d)
                            x[n][i] = fmaf(s.q[r0 + g + 4 * (i & 2)][d], kk[8 * n + 2 * t + (i & 1)][d], x[n][i]);
                    }
            }
            // Whether some row does not see the whole unit.
            const bool masked = valid < KT || at + KT - 1 > first_row ||
                                (p.window > 0 && at <= last_row - p.window && at + KT > p.sinks);
            float w[2][4];
            unsigned seen = 0xffu;                       // bit 4 n + i
            float fade[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {                // rows r0 + g + 8 r
                float up = kNegInf;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 2 * r; i < 2 * r + 2; ++i) {
                        const int c = half * 16 + 8 * n + 2 * t + (i & 1), j = at + c;
                        const bool yes = !masked || (c < valid && j <= pos[r] &&
                                                     (p.window == 0 || j > pos[r] - p.window || j < p.sinks));
                        if (!yes) seen &= ~(1u << (4 * n + i));
                        x[n][i] = yes ? x[n][i] : kNegInf;
                        up = fmaxf(up, x[n][i]);
                    }
                up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 1));
                up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2));
                up = fmaxf(up * p.scale_log2, top[r]);
                const float base = up == kNegInf ? 0.0f : up;
                fade[r] = chunk_pow2(top[r] - base);
                top[r] = up;
                sum[r] *= fade[r];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 2 * r; i < 2 * r + 2; ++i) {
                        w[n][i] = chunk_pow2(fmaf(x[n][i], p.scale_log2, -base));    // (one rounding)
                        if (seen >> (4 * n + i) & 1u) sum[r] += w[n][i];
                        else w[n][i] = 0.0f;
                    }
            }
            // V's infinities and NaNs are added to the rows that see them (a weight of 0 would carry them on to
            // the others), and zeros take their places.
            if (odd) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][i] *= fade[i >> 1];
                fade[0] = fade[1] = 1.0f;
                for (int k = 0; k < 16; ++k) {           // (lane 4 g + k / 2 % 4 has the weights of position k)
                    const int lane_of = 4 * g + (k >> 1 & 3), i = k & 1;
                    const unsigned bits = __shfl_sync(0xffffffffu, seen, lane_of) >> (4 * (k >> 3) + i);
                    const float a = k < 8 ? (i ? w[0][1] : w[0][0]) : (i ? w[1][1] : w[1][0]);
                    const float b = k < 8 ? (i ? w[0][3] : w[0][2]) : (i ? w[1][3] : w[1][2]);
                    const float wk[2] = {__shfl_sync(0xffffffffu, a, lane_of), __shfl_sync(0xffffffffu, b, lane_of)};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float y = vv[k][8 * n + 2 * t + (j & 1)];
                            if (n < steps && (bits >> (j & 2) & 1u) != 0u && !(fabsf(y) < __builtin_huge_valf()))
                                o[n][j] = fmaf(wk[j >> 1], y, o[n][j]);
                        }
                }
                __syncthreads();
                for (int r = warp; r < KT; r += kThreads / 32)
                    for (int d = lane; d < dim; d += 32) {
                        float* const y = &s.v[now][r][d];
                        if (!(fabsf(*y) < __builtin_huge_valf())) *y = 0.0f;
                    }
                __syncthreads();
            }
            // 8 positions each: numbers t and t + 4 of a product are 2 t and 2 t + 1.
            unsigned hi[2][4], lo[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                split_a(w[k][0], &hi[k][0], &lo[k][0]);
                split_a(w[k][2], &hi[k][1], &lo[k][1]);
                split_a(w[k][1], &hi[k][2], &lo[k][2]);
                split_a(w[k][3], &hi[k][3], &lo[k][3]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= steps) continue;
                float big[4] = {0.0f, 0.0f, 0.0f, 0.0f}, rest[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    mma_split(big, rest, hi[k], lo[k], vv[8 * k + 2 * t][8 * n + g], vv[8 * k + 2 * t + 1][8 * n + g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] = o[n][i] * fade[i >> 1] + (big[i] + rest[i]);
            }
            __syncthreads();                             // (the unit's place is filled again)
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
            sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        }
        // The second halves' outputs go through the place of K.
        float(*const other)[Tile<DP>::kPitch] = reinterpret_cast<float(*)[Tile<DP>::kPitch]>(&s.k[0][0][0]);
        __syncthreads();
        if (half == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r0 + g + 8 * r;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    *reinterpret_cast<float2*>(&other[row][8 * n + 2 * t]) = make_float2(o[n][2 * r], o[n][2 * r + 1]);
                if (t == 0) {
                    s.top[row] = top[r];
                    s.sum[row] = sum[r];
                }
            }
        }
        __syncthreads();
        if (half == 0) {
            float* const slot = p.slots + it.slot * chunk_slot_words(p.slot_rows, dim);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r0 + g + 8 * r;
                if (row >= it.rows) continue;
                const float up = fmaxf(top[r], s.top[row]), base = up == kNegInf ? 0.0f : up;
                const float mine = chunk_pow2(top[r] - base), theirs = chunk_pow2(s.top[row] - base);
                const float all = fmaf(s.sum[row], theirs, sum[r] * mine);
                const bool whole = it.parts == 1;
                const float by = !whole ? 1.0f : all > 0.0f ? 1.0f / all : all;        // a NaN stays one
                float* lse = nullptr;
                float* const to = whole ? chunk_out<float>(p, it, it.row + row, &lse)
                                        : slot + 2 * p.slot_rows + static_cast<long long>(row) * dim;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int d = 8 * n + 2 * t;
                    if (d >= dim) break;
                    const float2 y = *reinterpret_cast<const float2*>(&other[row][d]);
                    const float2 f = make_float2(fmaf(y.x, theirs, o[n][2 * r] * mine) * by,
                                                 fmaf(y.y, theirs, o[n][2 * r + 1] * mine) * by);
                    if (!whole || p.out_aligned != 0) {
                        *reinterpret_cast<float2*>(to + d) = f;
                    } else {
                        to[d] = f.x;
                        to[d + 1] = f.y;
                    }
                }
                if (t == 0 && whole && lse != nullptr) *lse = all == 0.0f ? kNegInf : (up + log2f(all)) * kChunkLn2;
                if (t == 0 && !whole) {
                    slot[row] = up;
                    slot[p.slot_rows + row] = all;
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

template <int DP>
gs_status launch_as(const ChunkParams& p, int blocks, gs_stream stream) {
    const int bytes = static_cast<int>(sizeof(typename Tile<DP>::Smem));
    if (!allow_smem<chunk_kernel<DP>>(bytes)) return GS_ERR_CUDA;
    return launch(chunk_kernel<DP>, dim3(blocks), kThreads, bytes, 1, stream, p);
}

}  // namespace

int chunk_fp32_unit() { return KT; }

ChunkShape chunk_fp32_shape(int dim) { return {kRows, dim > 128 ? sm_count() : 2 * sm_count()}; }

gs_status launch_chunk_fp32(const ChunkParams& p, int blocks, gs_stream stream) {
    if (p.c.dim <= 64) return launch_as<64>(p, blocks, stream);
    if (p.c.dim <= 128) return launch_as<128>(p, blocks, stream);
    return launch_as<256>(p, blocks, stream);
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
    if (args->split_weights != 0 && args->split_weights != 1) return GS_ERR_INVALID_ARG;
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
    // (The largest scales would become infinite, and scores of 0 with them NaN.)
    p.scale_log2 = args->scale == 0.0f ? 1.0f : std::fmin(std::fabs(args->scale) * kChunkLog2e, std::numeric_limits<float>::max());
    p.q_sign = args->scale > 0.0f ? 1.0f : args->scale < 0.0f ? -1.0f : 0.0f;
    // No position is past 2^30, so more leave none out; and a row 2^30 before its sequence less a window stays in 32 bits.
    constexpr int kMostWindow = 1 << 30;
    p.window = args->window < kMostWindow ? args->window : kMostWindow;
    p.sinks = args->sinks < kMostWindow ? args->sinks : kMostWindow;
    p.out = args->out;
    p.out_token = args->out_token_stride;
    p.out_head = args->out_head_stride;
    p.lse = args->lse;
    p.work = static_cast<int*>(args->workspace);
    p.slots = static_cast<float*>(args->workspace) + kChunkCounters;
    p.slot_rows = plan.rows;
    p.unit_page = args->cache->dtype == GS_DTYPE_F32 ? chunk_fp32_unit() : p.c.page;
    if (args->cache->dtype == GS_DTYPE_F32) return launch_chunk_fp32(p, plan.shape.blocks, stream);
    if (args->split_weights != 0) return launch_chunk_mma_split(args->cache->dtype, p, plan.shape.blocks, stream);
    return launch_chunk_mma(args->cache->dtype, p, plan.shape.blocks, stream);
}
