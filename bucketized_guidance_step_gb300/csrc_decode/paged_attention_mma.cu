// Attention of one new token over a paged cache: the tensor-core policy, for 16-bit caches
// (sm_103a).
//
// The query heads that share a kv head are the columns of two matrix products with that
// head's K and V: S^T = K Q^T (positions x heads) and O^T = V^T P^T (dim x heads).  Positions
// and dim take the rows of the instruction (m16n8k16) and heads its 8 columns, so groups of
// 1 to 8 heads cost one instruction and 9 to 16 two; K and V pass once for all of them.
// The warp-wide mma.sync is used rather than tcgen05: a tile has 8 or 16 columns, each byte of
// K and V is used for a few operations only, and the time goes to reading them from HBM.
//
// Heads that fill one column of 8 take the instance of one (48 us against 50.5 us in the instance
// of two, 32 rows of 2048 tokens, groups of 4), more the instance of two, which reads K and V once
// (36.9 us against 42.7 us in two parts of 8, groups of 16 and 4 kv heads).
//
// The weights 2^(s - m) enter the second product as two 16-bit numbers, hi + lo: with hi alone
// the rounding of the weights would add as much error as the rounding of the output.  The sum
// of the weights is taken before they are rounded.  For fp16 the weights are scaled by 2^11
// (the reference of the softmax is m - 11), so that small ones stay clear of fp16's subnormals.
#include "paged_attention.cuh"

namespace gs_decode {
namespace {

__device__ __forceinline__ void load_matrix(unsigned a, unsigned (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void load_matrix_t(unsigned a, unsigned (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ unsigned transpose8(unsigned x) {
    unsigned y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <class T>
__device__ __forceinline__ void mma(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values rounded and packed (x low), and what the rounding left, rounded and packed.
template <class T>
__device__ __forceinline__ void split2(float x, float y, unsigned* hi, unsigned* lo) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
        *hi = *reinterpret_cast<const unsigned*>(&h);
        *lo = *reinterpret_cast<const unsigned*>(&l);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        *hi = *reinterpret_cast<const unsigned*>(&h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(x - __uint_as_float(*hi << 16),
                                                       y - __uint_as_float(*hi & 0xffff0000u));
        *lo = *reinterpret_cast<const unsigned*>(&l);
    }
}
__device__ __forceinline__ float max_rows(float x) {     // over the lanes of one column
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_rows(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// NH: columns of 8 query heads; STEPS: of 16 dims.  Of a warp's 32 lanes, lane = 4 g + t.
template <class Type, int DIM, int NH, int STEPS = DIM / 16>
struct Mma {
    using T = Type;
    static constexpr int DP = DIM, RUN = 16, HEADS = 8 * NH;
    static constexpr int STAGES = DIM == 64 ? 4 : 3, PER_SM = DIM == 64 ? 3 : DIM == 128 ? 2 : 1;
    static_assert(kRound == 8, "a dump is one column of heads");
    static constexpr int KS = STEPS;                     // steps of 16 over dim
    static constexpr bool FULL = KS * 16 == DP, PARTIAL = !FULL;
    static constexpr float kShift = std::is_same<T, __half>::value ? 11.0f : 0.0f;
    static constexpr float kSlack = std::is_same<T, __half>::value ? 4.0f : 8.0f;    // 2^(11 + 4) fits fp16
    unsigned q[NH][KS][2];                               // head g (+ 8), dims 2t, 2t+1; 2t+8, 2t+9
    float o[NH][KS][4];                                  // dims g (0, 1), g+8 (2, 3), heads 2t, 2t+1
    float top[NH][2], sum[NH][2];                        // heads 2t, 2t+1
    bool empty;                                          // no run yet: o and sum are 0

    // The next segment's query heads wait in registers where there is room for them.
    static constexpr bool AHEAD = NH == 1 && DP <= 128;
    unsigned next[AHEAD ? KS : 1][2];

    __device__ __forceinline__ void fetch(const T* query, long long head_stride, int heads, int dim,
                                          bool aligned) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const bool usual = aligned && dim == 16 * KS;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const unsigned short* const qp =
                reinterpret_cast<const unsigned short*>(query + (h * 8 + g) * head_stride + 2 * t);
            const bool here = h * 8 + g < heads;
            if (usual) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
                        keep(h, s, half, here ? *reinterpret_cast<const unsigned*>(qp + s * 16 + half * 8) : 0u);
            } else {
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int d = s * 16 + half * 8;
                        const bool in = here && d < dim;
                        const unsigned low = in ? qp[d] : 0u, high = in ? qp[d + 1] : 0u;
                        keep(h, s, half, low | high << 16);
                    }
            }
        }
    }
    __device__ __forceinline__ void keep(int h, int s, int half, unsigned two) {
        if constexpr (AHEAD) next[s][half] = two;
        else q[h][s][half] = two;
    }

    __device__ __forceinline__ void begin() {
        empty = true;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            top[h][0] = top[h][1] = kNegInf;
            sum[h][0] = sum[h][1] = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                if constexpr (AHEAD) {
                    q[h][s][0] = next[s][0];
                    q[h][s][1] = next[s][1];
                }
                o[h][s][0] = o[h][s][1] = o[h][s][2] = o[h][s][3] = 0.0f;
            }
        }
    }

    __device__ __forceinline__ void step(const char* stage, int lo, int hi, float scale) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        float s[NH][4], odd[NH][4];                      // positions g (0, 1), g+8 (2, 3)
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][e] = odd[h][e] = 0.0f;
        {
            const int r = lane & 15;
            const unsigned row = smem_addr(stage) + r * DP * 2;
#pragma unroll
            for (int x = 0; x < KS; x += 2) {            // two sums, for shorter chains
                unsigned a[4], b[4];
                load_matrix(row + (((2 * x + (lane >> 4)) ^ (r & 7)) << 4), a);
                load_matrix(row + (((2 * x + 2 + (lane >> 4)) ^ (r & 7)) << 4), b);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    mma<T>(s[h], a, q[h][x][0], q[h][x][1]);
                    mma<T>(odd[h], b, q[h][x + 1][0], q[h][x + 1][1]);
                }
            }
        }
        // The reference `top` is the largest score so far, or up to 2^kSlack below it: it moves only
        // when a score passes it by more, so that most runs need no maximum over the lanes.
        bool over = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][e] = (s[h][e] + odd[h][e]) * scale;
            if (lo > 0 || hi < RUN) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (g + (e >> 1) * 8 < lo || g + (e >> 1) * 8 >= hi) s[h][e] = kNegInf;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) over = over || s[h][e] > top[h][e & 1] + kSlack;
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float up = fmaxf(top[h][e], max_rows(fmaxf(s[h][e], s[h][e + 2])));
                    if (!empty) {
                        const float w = up > top[h][e] ? pow2(top[h][e] - up) : 1.0f;
                        sum[h][e] *= w;
#pragma unroll
                        for (int x = 0; x < KS; ++x) {
                            o[h][x][e] *= w;
                            o[h][x][e + 2] *= w;
                        }
                    }
                    top[h][e] = up;
                }
        }
        empty = false;
        unsigned wh[NH][2], wl[NH][2];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float base = top[h][e] == kNegInf ? 0.0f : top[h][e] - kShift;
                s[h][e] = pow2(s[h][e] - base);
                s[h][e + 2] = pow2(s[h][e + 2] - base);
                sum[h][e] += s[h][e] + s[h][e + 2];
            }
            split2<T>(s[h][0], s[h][1], &wh[h][0], &wl[h][0]);
            split2<T>(s[h][2], s[h][3], &wh[h][1], &wl[h][1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                wh[h][e] = transpose8(wh[h][e]);
                wl[h][e] = transpose8(wl[h][e]);
            }
        }
        {
            const int r = (lane & 7) + ((lane >> 4) << 3);
            const unsigned row = smem_addr(stage) + (RUN + r) * DP * 2;
#pragma unroll
            for (int x = 0; x < KS; ++x) {
                unsigned a[4];
                load_matrix_t(row + (((2 * x + ((lane >> 3) & 1)) ^ (r & 7)) << 4), a);
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    mma<T>(o[h][x], a, wh[h][0], wh[h][1]);
                    mma<T>(o[h][x], a, wl[h][0], wl[h][1]);
                }
            }
        }
    }

    __device__ __forceinline__ void dump(float* out, int pitch, int first, int heads, int dim) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            if (h * 8 != first) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int head = 2 * t + e;              // of this dump
                const float all = sum_rows(sum[h][e]);
                if (first + head >= heads) continue;
                if (g == 0) {
                    out[head * pitch + dim] = top[h][e] - kShift;
                    out[head * pitch + dim + 1] = all;
                }
                float* const to = out + head * pitch + g;
                if (dim == 16 * KS) {
#pragma unroll
                    for (int x = 0; x < 2 * KS; ++x) to[x * 8] = o[h][x / 2][e + 2 * (x & 1)];
                } else {
#pragma unroll
                    for (int x = 0; x < 2 * KS; ++x)
                        if (x * 8 < dim) to[x * 8] = o[h][x / 2][e + 2 * (x & 1)];
                }
            }
        }
    }
};

// The instance for a head dimension and a group of query heads.  As many blocks on an SM as
// registers and rings allow: rows of up to 128 bytes take three with rings of four stages (2 rows
// of 200000 tokens, 32/8 heads of 64: 129 us, and 143 us with two blocks and six stages, 153 us
// with four and three), rows of up to 256 bytes two with three.  Dims of up to 96 lie in rows of
// 256 bytes, but for their products (32 rows of 2048 tokens, 32/8 heads of 96: 39.3 us, and 42.4 us
// with the products of 128).  Rows over that take 8 query heads
// at a time: the output of 16 would not fit the registers.
template <class T, class F>
auto with_instance(int dim, int group, F f) {
    if (dim <= 64) return group <= 8 ? f(Mma<T, 64, 1>()) : f(Mma<T, 64, 2>());
    if (dim <= 96) return group <= 8 ? f(Mma<T, 128, 1, 6>()) : f(Mma<T, 128, 2, 6>());
    if (dim <= 128) return group <= 8 ? f(Mma<T, 128, 1>()) : f(Mma<T, 128, 2>());
    return f(Mma<T, 256, 1>());
}

}  // namespace

Serves mma_serves(int dim, int group) {
    return with_instance<__half>(dim, group, [&](auto policy) { return serves_by<decltype(policy)>(group); });
}

gs_status launch_mma(int dtype, const AttnParams& p, int blocks, gs_stream stream) {
    const auto run = [&](auto policy) { return launch_policy<decltype(policy)>(p, blocks, stream); };
    return dtype == GS_DTYPE_BF16 ? with_instance<__nv_bfloat16>(p.c.dim, p.group, run)
                                  : with_instance<__half>(p.c.dim, p.group, run);
}

}  // namespace gs_decode
