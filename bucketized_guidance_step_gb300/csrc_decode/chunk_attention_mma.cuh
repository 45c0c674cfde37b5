// Attention of chunks of new tokens over a paged cache (sm_103a), for 16-bit caches: both products on
// the tensor cores (tcgen05), sums in tensor memory, keys and values brought by TMA, a box a page.
//
// A block works on two tiles of 128 query rows at a time (one for heads of over 128 dims), which share
// every unit of keys and values.  Of its warps
//   one takes items from the queue and brings their queries and K by TMA, another brings V: units of 64
//     positions through a ring of stages in shared memory each, as far ahead as the ring has room, over the
//     ends of items;
//   one a tile issues its products: S = Q K^T into one of the tile's two places in tensor memory, and O += P V
//     from there (the tensor cores have hardly a product waiting: while one warp waits, the other issues);
//   four a tile have a row a thread: they read S, keep the softmax's reference and sum, write the
//     weights P over S as 16-bit numbers, and at the item's end read O and store it.
// The scores of a step are there before the weights of the last one are done: the rows' threads never
// wait for the tensor cores, but where those are what bounds the kernel.
//
// With s the scores in powers of two (times scale log2 e), the weights are 2^(s - m + kLift) with a
// reference m that is the row's largest score so far, or up to kSlack below: O and the sum are
// rescaled only when a score passes m by more, which few units after the first do.  Weights are
// rounded once to 16 bits, off by half a step, as the output is; their sums, not rounded, are fp32.  A caller
// who asks for it gets them as sums of two 16-bit numbers, with which the output's own rounding is all that is
// left, for a second product with V (below).
//
// Measured (bf16, 32 and 8 heads of 128): a chunk of 2048 tokens over 16384 takes 400 us, 1290 TFLOP/s or 68 % of
// what a plain matrix product reaches; a unit of two tiles is 1940 cycles, of which the tensor cores need 1280
// (S with N = 64 takes 48 cycles a product of 16 dims, not 32; of N = 128 one place a tile fits beside O, not two) and
// the exponentials 1024.  32 sequences of up to 8200 tokens with 1 to 8 new ones: 127 us, HBM at 65 %.
// With weights as two numbers a unit's products take 1792 cycles, and the two calls 481 and 137 us.
//
// Positions that a row does not see get the weight 0.  So that 0 times an infinity or NaN reaches no
// row, V is looked through in units that some row sees in part: what is not finite there is added to
// the rows that see it and then taken out of the unit (give_out).
#pragma once

#include <cuda.h>

#include "chunk_attention.cuh"

namespace gs_decode {
namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
    static EncodeTiled fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return static_cast<EncodeTiled>(nullptr);
        }
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

// ---- instructions -----------------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_at(const void* p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0u;
}
// Waits, to the block's deadline at most, for the phase of this parity; once one wait of the block has run out, all of
// them end.  (A deadline, not a time for each: there are two dozen copies of this, and the smallest calls wait for
// instructions; reading a limit beside the clock cost them 0.9 us of 16.  The clock is not read before the second look,
// which waits for some time itself: the clock's own latency was 5 % of a long prompt.)
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity, ChunkGuard* guard) {
    if (bar_try(bar, parity)) return true;
    while (!bar_try(bar, parity)) {
        volatile unsigned long long* const deadline = &guard->deadline;
        if (chunk_clock() > *deadline) {
            *static_cast<volatile int*>(&guard->dead) = 1;
            *deadline = 0;
            return false;
        }
    }
    return true;
}
// The time to the next item begins.  One thread.
__device__ __forceinline__ void start_clock(ChunkGuard* guard) {
    volatile unsigned long long* const deadline = &guard->deadline;
    if (*static_cast<volatile int*>(&guard->dead) == 0) *deadline = chunk_clock() + guard->limit;
}
// The same for a warp: whether all its lanes saw the phase.
__device__ __forceinline__ bool warp_wait(unsigned bar, unsigned parity, ChunkGuard* guard) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, guard));
}
// A barrier of the threads that a barrier in shared memory counts, whole warps (one that waits with a
// limit, as every wait here).
__device__ __forceinline__ bool meet(unsigned bar, unsigned* turn, ChunkGuard* guard) {
    bar_arrive(bar);
    const bool ok = warp_wait(bar, *turn, guard);
    *turn ^= 1;
    return ok;
}
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void load_box(unsigned dst, const CUtensorMap* map, int x, int row, int head,
                                         int page, unsigned bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(row), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void load_box3(unsigned dst, const CUtensorMap* map, int x, int head, int token,
                                          unsigned bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(head), "r"(token), "r"(bar)
        : "memory");
}

// Two fp32 numbers in a register pair.
__device__ __forceinline__ unsigned long long pair_of(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_pair(unsigned long long p, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(p));
}
__device__ __forceinline__ unsigned long long fma_pair(unsigned long long a, unsigned long long b,
                                                       unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add_pair(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void mma_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mma_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// A matrix in shared memory in columns of 64 values (128 bytes a row, rows permuted in groups of 8 as
// TMA's 128-byte swizzle leaves them).  K-major: groups of 8 rows follow each other.  MN-major: `next`
// bytes lead to the next 64 values.
__host__ __device__ constexpr unsigned long long matrix_at(unsigned at, unsigned next) {
    return static_cast<unsigned long long>((at & 0x3ffffu) >> 4) |
           static_cast<unsigned long long>(next >> 4) << 16 | 64ull << 32 | 1ull << 46 | 2ull << 61;
}

// Both operands in shared memory.
__device__ __forceinline__ void mma_ss(unsigned d, unsigned long long a, unsigned long long b, unsigned what,
                                       unsigned add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(what), "r"(add)
        : "memory");
}
// Four neighbouring steps of 16 of a product, their descriptors made from the first one's low words within
// one block of instructions: what is given to an instruction goes through registers of the warp, and asked
// for one by one that takes as long as a product of 128 by 128.
__device__ __forceinline__ void mma_ss4(unsigned d, unsigned a, unsigned b, unsigned high, unsigned what, unsigned add) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 a1, a2, a3, b1, b2, b3;\n\t.reg .b64 x0, x1, x2, x3, y0, y1, y2, y3;\n\t"
        "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 2;\n\tadd.u32 a2, %1, 4;\n\tadd.u32 a3, %1, 6;\n\t"
        "add.u32 b1, %2, 2;\n\tadd.u32 b2, %2, 4;\n\tadd.u32 b3, %2, 6;\n\t"
        "mov.b64 x0, {%1, %3};\n\tmov.b64 x1, {a1, %3};\n\tmov.b64 x2, {a2, %3};\n\tmov.b64 x3, {a3, %3};\n\t"
        "mov.b64 y0, {%2, %3};\n\tmov.b64 y1, {b1, %3};\n\tmov.b64 y2, {b2, %3};\n\tmov.b64 y3, {b3, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x0, y0, %4, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x1, y1, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x2, y2, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x3, y3, %4, t;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(what), "r"(add)
        : "memory");
}
// A in tensor memory, 8 columns a step; B 2048 bytes a step.
__device__ __forceinline__ void mma_ts4(unsigned d, unsigned a, unsigned b, unsigned high, unsigned what, unsigned add) {
    asm volatile(
        "{\n\t.reg .pred p, t;\n\t.reg .b32 a1, a2, a3, b1, b2, b3;\n\t.reg .b64 y0, y1, y2, y3;\n\t"
        "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u32 a2, %1, 16;\n\tadd.u32 a3, %1, 24;\n\t"
        "add.u32 b1, %2, 128;\n\tadd.u32 b2, %2, 256;\n\tadd.u32 b3, %2, 384;\n\t"
        "mov.b64 y0, {%2, %3};\n\tmov.b64 y1, {b1, %3};\n\tmov.b64 y2, {b2, %3};\n\tmov.b64 y3, {b3, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y0, %4, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], y1, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], y2, %4, t;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], y3, %4, t;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(what), "r"(add)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    unsigned yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0u;
}
// The barrier gets an arrival once all products issued so far are done.
__device__ __forceinline__ void mma_commit(unsigned bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"l"(
                     static_cast<unsigned long long>(bar))
                 : "memory");
}

// 32 columns of a lane's row of tensor memory.
__device__ __forceinline__ void tmem_load(unsigned at, float* f) {
    unsigned* r = reinterpret_cast<unsigned*>(f);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
        "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// Waits for the loads into x: what uses x comes after it (the loads' outputs alone would not tell the
// compiler so).
template <int N>
__device__ __forceinline__ void tmem_wait_load(float (&x)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(x[i]));
}
__device__ __forceinline__ void tmem_store32(unsigned at, const float* f) {
    const unsigned* r = reinterpret_cast<const unsigned*>(f);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
        "%23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_store16(unsigned at, const unsigned* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes at once: a whole sector (with two halves of it one after the other the rows' stores took twice
// the time).
__device__ __forceinline__ void store32(void* to, const unsigned* r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <class T>
struct Weights;                           // of type T: kept below 2^(kLift + kSlack)
template <>
struct Weights<__nv_bfloat16> {
    static constexpr float kLift = 0.0f, kSlack = 8.0f;
    static constexpr unsigned kExponent = 0x7f807f80u, kOne = 0x00800080u, kType = 1u;
    static constexpr unsigned kHigh = 0xffff0000u;       // of an fp32 number: what the type holds
    static __device__ __forceinline__ unsigned pack(float lo, float hi) {
        unsigned r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
template <>
struct Weights<__half> {
    static constexpr float kLift = 9.0f, kSlack = 6.0f;
    static constexpr unsigned kExponent = 0x7c007c00u, kOne = 0x04000400u, kType = 0u;
    static constexpr unsigned kHigh = 0xffffe000u;
    static __device__ __forceinline__ unsigned pack(float lo, float hi) {
        unsigned r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// Two weights as sums of two 16-bit numbers each: what the type holds of them, cut, and the rest, rounded.  Off by
// 2^-15 (bf16) and 2^-21 (fp16) of a weight at most, and in fp16, where numbers are not normal, 2^-24.
template <class T>
__device__ __forceinline__ void split_weights(float a, float b, unsigned* high, unsigned* low) {
    using W = Weights<T>;
    const float ah = __uint_as_float(__float_as_uint(a) & W::kHigh), bh = __uint_as_float(__float_as_uint(b) & W::kHigh);
    if constexpr (std::is_same<T, __nv_bfloat16>::value) *high = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    else *high = W::pack(ah, bh);
    float x, y;
    split_pair(fma_pair(pair_of(ah, bh), pair_of(-1.0f, -1.0f), pair_of(a, b)), &x, &y);
    *low = W::pack(x, y);
}

// ---- shapes -----------------------------------------------------------------------------------
constexpr int kUnit = 64;                 // positions of a unit
template <int DP>
struct Shape {
    static constexpr int TILES = DP > 128 ? 1 : 2;       // tiles of 128 rows
    static constexpr int Q = 128 * DP * 2, STAGE = kUnit * DP * 2;   // bytes
    static constexpr int K_STAGES = DP == 64 ? 10 : DP == 128 ? 5 : 3, V_STAGES = DP == 256 ? 2 : K_STAGES;
    static constexpr int GROUP = 128 * TILES;            // threads with a row
    static constexpr int THREADS = GROUP + 64 + 32 * TILES, WIDTH = 128;
    // Tensor memory: two places of S for each tile (P in the last half of the place, what is left of weights that are
    // split in the first), then O of each.
    static constexpr int P = kUnit / 2, O = 256;
    static_assert(TILES * 2 * kUnit <= O && O + TILES * DP <= 512, "tensor memory");
    using Cut = ChunkCut<128 * TILES, 128, kUnit, THREADS, WIDTH>;
};

constexpr int kItems = 2;                 // items under way
template <int DP>
struct alignas(1024) Smem {
    using S = Shape<DP>;
    unsigned char q[S::TILES][S::Q];
    unsigned char k[S::K_STAGES][S::STAGE], v[S::V_STAGES][S::STAGE];
    unsigned long long k_full[S::K_STAGES], k_empty[S::K_STAGES], v_full[S::V_STAGES], v_empty[S::V_STAGES];
    unsigned long long item_full[kItems], item_empty[kItems];
    unsigned long long q_full[2], q_empty[2], s_full[2][2], p_full[2][2], o_full[2][2];
    unsigned long long tile_meet[2], both_meet, tail, drain[2];
    ChunkItem items[kItems];
    int seeded[2], hot[2][2];
    unsigned tmem;
    typename S::Cut::Shared plan;
};
static_assert(sizeof(Smem<128>) <= 227 * 1024 && sizeof(Smem<256>) <= 227 * 1024, "shared memory of a block");

// What is not finite in a unit's V: added to the rows that see it, then 0.  A warp calls it together;
// a thread's row sees positions lo .. hi - 1 and those below sinks.  `first`: O holds nothing yet.
template <class T, int DP>
__device__ __noinline__ bool give_out(unsigned char* v, unsigned o_at, int dim, int lo, int hi, int sinks,
                                      int valid, bool first, int threads, unsigned bar, unsigned* turn,
                                      ChunkGuard* guard) {
    using S = Shape<DP>;
    for (int d0 = 0; d0 < dim; d0 += 32) {
        float o[32];
        if (first) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        } else {
            tmem_load(o_at + d0, o);
            tmem_wait_load(o);
        }
        for (int r = 0; r < valid; ++r) {
            if (!((r >= lo || r < sinks) && r < hi)) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int d = d0 + i, c = d & 63;
                const T x = *reinterpret_cast<const T*>(v + (d >> 6) * (kUnit * 128) + r * 128 +
                                                        (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
                const float f = static_cast<float>(x);
                if (!(fabsf(f) <= 3.4e38f)) o[i] += f;
            }
        }
        __syncwarp();
        tmem_store32(o_at + d0, o);
        tmem_wait_store();
    }
    if (!meet(bar, turn, guard)) return false;           // every row has what it sees
    using W = Weights<T>;
    unsigned* const words = reinterpret_cast<unsigned*>(v);
    for (int x = threadIdx.x; x < S::STAGE / 4; x += threads) {
        const unsigned w = words[x], hot = ((w & W::kExponent) + W::kOne) & 0x80008000u;
        if (hot != 0u) words[x] = w & ~((hot >> 15) * 0xffffu);
    }
    async_fence();
    return meet(bar, turn, guard);
}

// SPLIT: weights enter the product with V as sums of two 16-bit numbers, a second product with the same V.
template <class T, int DP, bool SPLIT>
__global__ void __launch_bounds__(Shape<DP>::THREADS, 1)
chunk_mma_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map) {
    using S = Shape<DP>;
    using W = Weights<T>;
    constexpr int TILES = S::TILES;
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<DP>& s = *reinterpret_cast<Smem<DP>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dim = p.c.dim;
    const ChunkUnits<kUnit> units(p.c.page);
    const int role = warp - S::GROUP / 32;               // below 0: rows; 0, 1: bring K, V; 2, 3: issue a tile's products

    if (tid == 0) {
        for (int i = 0; i < S::K_STAGES; ++i) {
            bar_init(smem_at(&s.k_full[i]), 1);
            bar_init(smem_at(&s.k_empty[i]), TILES);
        }
        for (int i = 0; i < S::V_STAGES; ++i) {
            bar_init(smem_at(&s.v_full[i]), 1);
            bar_init(smem_at(&s.v_empty[i]), TILES);
        }
        for (int i = 0; i < kItems; ++i) {
            bar_init(smem_at(&s.item_full[i]), 1);
            bar_init(smem_at(&s.item_empty[i]), S::GROUP + 1 + TILES);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_at(&s.q_full[i]), 1);
            bar_init(smem_at(&s.q_empty[i]), 1);
            bar_init(smem_at(&s.s_full[i][0]), 1);
            bar_init(smem_at(&s.s_full[i][1]), 1);
            bar_init(smem_at(&s.p_full[i][0]), 128);
            bar_init(smem_at(&s.p_full[i][1]), 128);
            bar_init(smem_at(&s.o_full[i][0]), 1);
            bar_init(smem_at(&s.o_full[i][1]), 1);
            bar_init(smem_at(&s.tile_meet[i]), 128);
            s.hot[i][0] = s.hot[i][1] = 0;
        }
        bar_init(smem_at(&s.both_meet), S::GROUP);
        bar_init(smem_at(&s.tail), 1);
        for (int i = 0; i < 2; ++i) bar_init(smem_at(&s.drain[i]), 1);
        s.plan.guard.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (role == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&s.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (units.span < kUnit) {             // rows of a stage that no box reaches
        for (int x = tid; x < S::V_STAGES * S::STAGE / 16; x += S::THREADS)
            reinterpret_cast<uint4*>(s.v)[x] = make_uint4(0u, 0u, 0u, 0u);
        async_fence();
    }
    grid_wait();
    grid_trigger();
    typename S::Cut cut;
    cut.s = &s.plan;
    cut.ticket = role == 0 && lane == 0 ? atomicAdd(p.work, 1) : -1;
    mma_fence_before();
    cut.find(p);                          // (ends with a barrier)
    mma_fence_after();
    const unsigned tmem = s.tmem;
    if (role == 0 || role == 1) {
        const bool is_v = role == 1, one = elect_one();
        const int halves = (dim + 63) / 64;
        const int box = min(p.c.page, kUnit) * 128;      // bytes
        const int pages = units.per > 0 ? 1 : kUnit / p.c.page;      // of a unit
        const unsigned stages = is_v ? S::V_STAGES : S::K_STAGES;
        unsigned char* const stage0 = is_v ? s.v[0] : s.k[0];
        const unsigned full0 = smem_at(is_v ? s.v_full : s.k_full), empty0 = smem_at(is_v ? s.v_empty : s.k_empty);
        const CUtensorMap* const map = is_v ? &v_map : &k_map;
        // Page numbers are looked up 32 at a time, a page a lane, and a batch ahead: of `batch` units, or where
        // pages have one token of half a unit a word.
        const int batch = pages < 32 ? 32 / pages : 1;
        const int my_unit = pages < 32 ? lane / pages : 0, my_page = pages < 32 ? lane - my_unit * pages : lane;
        unsigned stage = 0, turn = 1;     // of the ring; the parity of the stage's last use
        unsigned tails = 0, bad = 0, q_turn = 3u;        // (q_turn: a bit a tile)
        bool go = true;
        for (int n = 0; go; ++n) {
            const int slot = n & 1;
            int kind = 0;
            if (is_v) {
                if (!warp_wait(smem_at(&s.item_full[slot]), (n >> 1) & 1, &s.plan.guard)) break;
                kind = s.items[slot].kind;
            } else {
                if (lane == 0) {
                    ChunkItem it;
                    chunk_next_item(&cut, p, &it);
                    if (bar_wait(smem_at(&s.item_empty[slot]), ((n >> 1) & 1) ^ 1, &s.plan.guard)) {
                        s.items[slot] = it;
                        kind = it.kind;
                        start_clock(&s.plan.guard);
                        bar_arrive(smem_at(&s.item_full[slot]));
                    } else {
                        kind = -1;
                    }
                }
                kind = __shfl_sync(0xffffffffu, kind, 0);
                __syncwarp();
            }
            if (kind <= 0) break;
            const ChunkItem& it = s.items[slot];
            const int head = it.head, len = it.e.len, lo = it.lo, hi = it.hi;
            const ChunkSpan span = it.span;
            const int tiles = TILES == 2 && it.rows > 128 ? 2 : 1;
            const int q_token = it.e.row + chunk_token(p, it.row);
            const int* const table = p.c.table + static_cast<long long>(it.e.seq) * p.c.cols;
            __syncwarp();
            if (is_v && one) bar_arrive(smem_at(&s.item_empty[slot]));
            if (kind == 2) continue;
            // This lane's page (>= 0; c.pages: outside the pool), and the unit's first row in it.
            struct Known {
                int page, more, row;
            };
            auto look_up = [&](int from) {
                Known k = {0, 0, 0};
                const int u = from + my_unit;
                if (u >= hi || my_unit >= batch) return k;
                const int unit = span.unit(u);
                int col = unit * pages + my_page;
                if (units.per > 0) {
                    col = unit / units.per;
                    k.row = (unit - col * units.per) * kUnit;
                }
                auto page_at = [&](int c) {
                    if (c * p.c.page >= len) return 0;
                    const int id = table[c];
                    if (id >= 0 && id < p.c.pages) return id;
                    bad |= GS_DEV_BAD_SEQ;
                    return p.c.pages;
                };
                k.page = page_at(col);
                if (pages > 32) k.more = page_at(col + 32);
                return k;
            };
            // The last unit may end inside.
            int count = 0, row_ignored, valid = 0, live_last = 1;
            if (lo < hi) {
                const int at = units.first(span.unit(hi - 1), &count, &row_ignored);
                valid = min(count, len - at);
                if (units.per == 0) live_last = (valid + p.c.page - 1) / p.c.page;
            }
            Known now = {0, 0, 0}, next = look_up(lo);
            int in_batch = batch;
            for (int u = lo; u < hi; ++u) {
                if (++in_batch >= batch) {
                    in_batch = 0;
                    now = next;
                    if (u + batch < hi) next = look_up(u + batch);
                }
                const int live = u + 1 < hi ? pages : live_last;
                if (!(go = warp_wait(empty0 + 8 * stage, turn, &s.plan.guard))) break;
                unsigned char* const here = stage0 + stage * S::STAGE;
                const unsigned full = full0 + 8 * stage;
                if (++stage == stages) {
                    stage = 0;
                    turn ^= 1;
                }
                // Rows past the sequence's end hold anything: of V they are taken out.
                const bool tail = is_v && u + 1 == hi && valid < count;
                const unsigned bar = tail ? smem_at(&s.tail) : full;
                if (one) bar_expect(bar, live * halves * box);
                const int row = __shfl_sync(0xffffffffu, now.row, in_batch * pages & 31);
                // (One lane issues: boxes that lanes give one each take turns, 66 cycles a box of 16 rows against 33.)
                unsigned to = smem_at(here);
                for (int x = 0; x < live; ++x, to += box) {
                    const int page = __shfl_sync(0xffffffffu, x < 32 ? now.page : now.more, in_batch * pages + x & 31);
                    if (one) {
#pragma unroll
                        for (int col = 0; col < DP / 64; ++col)
                            if (col < halves) load_box(to + col * (kUnit * 128), map, col * 64, row, head, page, bar);
                    }
                }
                if (!is_v && u == lo && p.q_boxes != 0) {            // the queries, once the last item's are done with
                    for (int w = 0; w < tiles && go; ++w) {
                        go = warp_wait(smem_at(&s.q_empty[w]), q_turn >> w & 1, &s.plan.guard);
                        q_turn ^= 1u << w;
                        if (!go) break;
                        const unsigned q_bar = smem_at(&s.q_full[w]);
                        if (one) {
                            bar_expect(q_bar, halves * 128 * 128);
                            for (int col = 0; col < halves; ++col)
                                load_box3(smem_at(s.q[w]) + col * (128 * 128), &q_map, col * 64, head * p.group,
                                          q_token + w * (128 / p.group), q_bar);
                        }
                        __syncwarp();
                    }
                    if (!go) break;
                }
                if (tail) {
                    if (!(go = warp_wait(bar, tails & 1, &s.plan.guard))) break;
                    ++tails;
                    for (int x = lane; x < (kUnit - valid) * 8 * halves; x += 32) {
                        const int col = x / ((kUnit - valid) * 8), y = x - col * ((kUnit - valid) * 8);
                        *reinterpret_cast<uint4*>(here + col * (kUnit * 128) + valid * 128 + y * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    async_fence();
                    __syncwarp();
                    if (one) bar_arrive(full);
                }
            }
        }
        flag(p.c.status, bad);
        // Where a wait has run out, the boxes under way land before the block ends.
        __syncwarp();
        if (s.plan.guard.dead != 0) {
            const unsigned long long t0 = chunk_clock();
            while (chunk_clock() - t0 < 10ull * 1000ull * 1000ull) __nanosleep(10000);
        }
    } else if (role >= 2) {
        const int w = role - 2;
        if (elect_one()) {
            const unsigned kind = 1u << 4 | W::kType << 7 | W::kType << 10 | (128u >> 4) << 24;
            const unsigned what_s = kind | static_cast<unsigned>(kUnit >> 3) << 17;
            const unsigned what_o = kind | 1u << 16 | static_cast<unsigned>((dim + 15) / 16 * 2) << 17;
            const int steps = (dim + 15) / 16;
            const unsigned q = static_cast<unsigned>(matrix_at(smem_at(s.q[w]), 16));
            const unsigned k_low = static_cast<unsigned>(matrix_at(smem_at(s.k[0]), 16));
            const unsigned v_low = static_cast<unsigned>(matrix_at(smem_at(s.v[0]), kUnit * 128));
            constexpr unsigned high = static_cast<unsigned>(matrix_at(0, 0) >> 32);      // (the same of all)
            const unsigned o_at = tmem + S::O + w * DP, s_at = tmem + w * 2 * kUnit;
            unsigned q_turn = 0, done = 0;               // items and units of the tile so far
            unsigned k_stage = 0, k_turn = 0, v_stage = 0, v_turn = 0;
            bool go = true;
            for (int n = 0; go; ++n) {
                const int slot = n & 1;
                if (!bar_wait(smem_at(&s.item_full[slot]), (n >> 1) & 1, &s.plan.guard)) break;
                const int item = s.items[slot].kind, rows = s.items[slot].rows;
                const unsigned count = s.items[slot].hi - s.items[slot].lo;
                bar_arrive(smem_at(&s.item_empty[slot]));
                if (item == 0) break;
                if (item == 2 || count == 0) continue;
                const bool alone = TILES == 2 && rows <= 128;        // the tile of the two that has rows
                // Every thread that waits for a unit of the rings has waited for all before it: a wait by parity
                // takes an older phase for its own where the one before is not over.  So the second tile's
                // thread goes through the units of an item that has no second tile, and frees them for its part.
                // (Rows wait for a unit of V behind its scores, which this thread has issued behind the units of
                // V before the last one.)
                if (alone && w == 1) {
                    for (unsigned u = 0; u < count + 2 && go; ++u) {
                        if (u >= 2) {     // (in the order in which the first tile's thread takes them)
                            if (!(go = bar_wait(smem_at(&s.v_full[v_stage]), v_turn, &s.plan.guard))) break;
                            bar_arrive(smem_at(&s.v_empty[v_stage]));
                            if (++v_stage == S::V_STAGES) {
                                v_stage = 0;
                                v_turn ^= 1;
                            }
                        }
                        if (u < count) {
                            if (!(go = bar_wait(smem_at(&s.k_full[k_stage]), k_turn, &s.plan.guard))) break;
                            bar_arrive(smem_at(&s.k_empty[k_stage]));
                            if (++k_stage == S::K_STAGES) {
                                k_stage = 0;
                                k_turn ^= 1;
                            }
                        }
                    }
                    continue;
                }
                // Unit u's scores; the first ones wait for the queries.
                auto scores = [&](unsigned u) {
                    if (!(go = bar_wait(smem_at(&s.k_full[k_stage]), k_turn, &s.plan.guard))) return;
                    if (u == 0) {
                        go = bar_wait(smem_at(&s.q_full[w]), q_turn, &s.plan.guard);
                        q_turn ^= 1;
                        if (!go) return;
                        mma_fence_after();
                    }
                    const unsigned place = done + u & 1, to = s_at + place * kUnit;
                    const unsigned k = k_low + k_stage * (S::STAGE / 16);
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c) {
                        if (steps >= 4 * (c + 1)) {
                            mma_ss4(to, q + c * (128 * 128 / 16), k + c * (kUnit * 128 / 16), high, what_s, c > 0);
                        } else {
                            for (int i = 4 * c; i < steps; ++i)
                                mma_ss(to, (static_cast<unsigned long long>(high) << 32) + q + c * (128 * 128 / 16) + (i & 3) * 2,
                                       (static_cast<unsigned long long>(high) << 32) + k + c * (kUnit * 128 / 16) + (i & 3) * 2,
                                       what_s, i > 0);
                            break;
                        }
                    }
                    mma_commit(smem_at(&s.s_full[w][place]));
                    mma_commit(smem_at(&s.k_empty[k_stage]));
                    if (u + 1 == count) mma_commit(smem_at(&s.q_empty[w]));
                    if (++k_stage == S::K_STAGES) {
                        k_stage = 0;
                        k_turn ^= 1;
                    }
                };
                scores(0);
                if (go && count > 1) scores(1);
                for (unsigned u = 0; u < count && go; ++u) {
                    // (A place has a barrier of its own: a warp may be a unit ahead of another.)
                    const unsigned place = done + u & 1;
                    if (!(go = bar_wait(smem_at(&s.v_full[v_stage]), v_turn, &s.plan.guard))) break;
                    if (!(go = bar_wait(smem_at(&s.p_full[w][place]), done + u >> 1 & 1, &s.plan.guard))) break;
                    mma_fence_after();
                    const unsigned add = u > 0 || *static_cast<volatile int*>(&s.seeded[w]) != 0;
                    mma_ts4(o_at, s_at + place * kUnit + S::P, v_low + v_stage * (S::STAGE / 16), high, what_o, add);
                    if constexpr (SPLIT)
                        mma_ts4(o_at, s_at + place * kUnit, v_low + v_stage * (S::STAGE / 16), high, what_o, 1u);
                    mma_commit(smem_at(&s.o_full[w][place]));
                    mma_commit(smem_at(&s.v_empty[v_stage]));
                    if (++v_stage == S::V_STAGES) {
                        v_stage = 0;
                        v_turn ^= 1;
                    }
                    if (u + 2 < count) scores(u + 2);
                }
                done += count;
            }
            if (s.plan.guard.dead != 0) {  // products under way end before the block does
                mma_commit(smem_at(&s.drain[w]));
                const unsigned long long t0 = chunk_clock();
                while (!bar_try(smem_at(&s.drain[w]), 0) && chunk_clock() - t0 < 10ull * 1000ull * 1000ull) {}
            }
        }
        __syncwarp();
    } else {
        const int w = TILES == 2 ? warp >> 2 : 0, mine = tid & 127;
        const unsigned lanes = static_cast<unsigned>((warp & 3) * 32) << 16;
        const unsigned s_at = tmem + lanes + w * 2 * kUnit, o_at = tmem + lanes + S::O + w * DP;
        const float scale = p.scale_log2;
        unsigned meet_turn = 0, both_turn = 0;                               // parities of the next phases
        unsigned done = 0;                // units
        int looked = 0;                   // units looked through
        unsigned ring = 0;                // units gone through of the block
        // Unit number `step`'s products with V are in O.  (The two barriers take turns with the places of
        // S: the one before last is known to be done, so that a phase is never taken for an older one.)
        auto added = [&](unsigned unit) {
            const bool ok = warp_wait(smem_at(&s.o_full[w][unit & 1]), unit >> 1 & 1, &s.plan.guard);
            mma_fence_after();
            return ok;
        };
        bool go = true;
        for (int n = 0; go; ++n) {
            const int slot = n & 1;
            if (!warp_wait(smem_at(&s.item_full[slot]), (n >> 1) & 1, &s.plan.guard)) break;
            const ChunkItem& it = s.items[slot];
            if (it.kind == 0) break;
            if (it.kind == 2) {
                if (mine == 0 && !chunk_wait_parts(p.work + kChunkHead + it.share, it.need, s.plan.guard.limit))
                    *static_cast<volatile int*>(&s.plan.guard.dead) = 1;
                if (!meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.plan.guard)) break;
                chunk_join<T>(p, it, warp, S::GROUP / 32, W::kLift);
                bar_arrive(smem_at(&s.item_empty[slot]));
                continue;
            }
            const int count = it.hi - it.lo, tiles = TILES == 2 && it.rows > 128 ? 2 : 1;
            if (w >= tiles) {
                ring += count;
                bar_arrive(smem_at(&s.item_empty[slot]));
                continue;
            }
            const int r = w * 128 + mine, row = it.row + r;         // of the tile, of the entry
            const bool real = r < it.rows;
            const int from = it.e.len - it.e.m;
            const int token = chunk_token(p, row), pos = from + token;
            if (count > 0 && p.q_boxes == 0) {
                // The row of Q, with the scale's sign, where TMA cannot bring it.
                const T* const q = static_cast<const T*>(p.q) + (it.e.row + static_cast<long long>(token)) * p.q_token +
                                   (it.head * p.group + row - token * p.group) * p.q_head;
                unsigned char* const to = s.q[w] + mine * 128;
                const unsigned flip = p.q_sign < 0.0f ? 0x80008000u : 0u;
                const bool zero = p.q_sign == 0.0f;
#pragma unroll
                for (int c = 0; c < DP / 8; ++c) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (real && c * 8 < dim && !zero) {
                        x = load16_any(q + c * 8, p.q_aligned != 0);
                        x.x ^= flip;
                        x.y ^= flip;
                        x.z ^= flip;
                        x.w ^= flip;
                    }
                    *reinterpret_cast<uint4*>(to + (c >> 3) * (128 * 128) + (((c & 7) ^ (mine & 7)) << 4)) = x;
                }
                async_fence();
                if (!(go = meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.plan.guard))) break;
                if (mine == 0) bar_arrive(smem_at(&s.q_full[w]));
            }
            float top = kNegInf, sum = 0.0f;
            const int first_pos = from + chunk_token(p, it.row), last_pos = from + chunk_token(p, it.row + it.rows - 1);
            const bool idle = w * 128 + (warp & 3) * 32 >= it.rows;      // none of the warp's rows is the tile's
            for (int u = 0; u < count; ++u) {
                int here, in_page;
                const int at = units.first(it.span.unit(it.lo + u), &here, &in_page);
                const int valid = min(here, it.e.len - at);
                // What this row sees of the unit: lo .. hi - 1, and those below sink.
                const int hi = min(valid, pos - at + 1);
                const int lo = p.window > 0 ? pos - p.window + 1 - at : 0;
                const int sink = p.window > 0 ? p.sinks - at : 0;
                // Whether some row of the block's tiles sees the unit in part (all threads alike).
                const bool part = at + valid - 1 > first_pos ||
                                  (p.window > 0 && at <= last_pos - p.window && at + valid > p.sinks);
                const unsigned place = done + u & 1;
                if (!(go = warp_wait(smem_at(&s.s_full[w][place]), done + u >> 1 & 1, &s.plan.guard))) break;
                mma_fence_after();
                bool odd = false;
                if (part) {
                    const unsigned v_stage = (ring + u) % S::V_STAGES;
                    if (!(go = warp_wait(smem_at(&s.v_full[v_stage]), (ring + u) / S::V_STAGES & 1, &s.plan.guard))) break;
                    unsigned hot = 0;
                    const uint4* const v = reinterpret_cast<const uint4*>(s.v[v_stage]);
#pragma unroll 8
                    for (int x = mine; x < S::STAGE / 16; x += 128) {
                        const uint4 y = v[x];
                        hot |= ((y.x & W::kExponent) + W::kOne) | ((y.y & W::kExponent) + W::kOne) |
                               ((y.z & W::kExponent) + W::kOne) | ((y.w & W::kExponent) + W::kOne);
                    }
                    // (All of a tile's threads look at all of it.)
                    ++looked;
                    if (__any_sync(0xffffffffu, (hot & 0x80008000u) != 0u) && lane == 0)
                        *static_cast<volatile int*>(&s.hot[w][looked & 1]) = looked;
                    if (!(go = meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.plan.guard))) break;
                    odd = *static_cast<volatile int*>(&s.hot[w][looked & 1]) == looked;
                    if (odd) {
                        if (u > 0 && !(go = added(done + u - 1))) break;
                        if (!(go = give_out<T, DP>(s.v[v_stage], o_at, dim, lo, hi, sink, valid, u == 0, 128 * tiles,
                                                   smem_at(tiles == 2 ? &s.both_meet : &s.tile_meet[w]),
                                                   tiles == 2 ? &both_turn : &meet_turn, &s.plan.guard)))
                            break;
                    }
                }
                if (u == 0 && mine == 0) s.seeded[w] = odd;
                if (!idle) {
                    float x[kUnit];
                    const unsigned from_at = s_at + place * kUnit;
                    tmem_load(from_at, x);
                    tmem_load(from_at + 32, x + 32);
                    tmem_wait_load(x);
                    if (!__all_sync(0xffffffffu, hi >= kUnit && lo <= 0)) {
#pragma unroll
                        for (int c = 0; c < kUnit; ++c)
                            if (!(c < hi && (c >= lo || c < sink))) x[c] = kNegInf;
                    }
                    float up0 = x[0], up1 = x[1];
#pragma unroll
                    for (int c = 2; c < kUnit - 2; c += 4) {
                        up0 = max3(up0, x[c], x[c + 1]);
                        up1 = max3(up1, x[c + 2], x[c + 3]);
                    }
                    const float up = max3(max3(up0, x[kUnit - 2], x[kUnit - 1]), up1, kNegInf) * scale;
                    const bool move = up > top + W::kSlack || (top == kNegInf && up > kNegInf);
                    if (__any_sync(0xffffffffu, move)) {
                        const float by = move ? chunk_pow2(top - up) : 1.0f;         // 0 at the first position
                        if (move) top = up;
                        sum *= by;
                        if (u > 0) {
                            if (!(go = added(done + u - 1))) break;
                            for (int d = 0; d < dim; d += 32) {
                                float o[32];
                                tmem_load(o_at + d, o);
                                tmem_wait_load(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= by;
                                tmem_store32(o_at + d, o);
                            }
                            tmem_wait_store();
                        }
                    }
                    const float base = W::kLift - (top == kNegInf ? 0.0f : top);
                    const unsigned long long scale2 = pair_of(scale, scale), base2 = pair_of(base, base);
                    unsigned long long sums = 0ull, more = 0ull;
#pragma unroll
                    for (int h = 0; h < kUnit; h += 32) {
                        unsigned r16[16], rest16[SPLIT ? 16 : 1];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            float a, b, e, f;
                            split_pair(fma_pair(pair_of(x[h + i], x[h + i + 1]), scale2, base2), &a, &b);
                            split_pair(fma_pair(pair_of(x[h + i + 2], x[h + i + 3]), scale2, base2), &e, &f);
                            a = chunk_pow2(a);
                            b = chunk_pow2(b);
                            e = chunk_pow2(e);
                            f = chunk_pow2(f);
                            sums = add_pair(sums, pair_of(a, b));
                            more = add_pair(more, pair_of(e, f));
                            if constexpr (SPLIT) {
                                split_weights<T>(a, b, &r16[i / 2], &rest16[i / 2]);
                                split_weights<T>(e, f, &r16[i / 2 + 1], &rest16[i / 2 + 1]);
                            } else {
                                r16[i / 2] = W::pack(a, b);
                                r16[i / 2 + 1] = W::pack(e, f);
                            }
                        }
                        tmem_store16(from_at + S::P + h / 2, r16);
                        if constexpr (SPLIT) tmem_store16(from_at + h / 2, rest16);
                    }
                    float a, b;
                    split_pair(add_pair(sums, more), &a, &b);
                    sum += a + b;
                    tmem_wait_store();
                }
                mma_fence_before();
                bar_arrive(smem_at(&s.p_full[w][place]));
            }
            ring += count;
            done += count;
            if (!go) break;
            if (count > 0 && !(go = added(done - 1))) break;
            float* lse = nullptr;
            T* const to = real ? chunk_out<T>(p, it, row, &lse) : nullptr;
            float* const part = p.slots + it.slot * chunk_slot_words(p.slot_rows, dim);
            const float by = sum > 0.0f ? 1.0f / sum : sum;         // a NaN stays one
            for (int d = 0; d < dim; d += 32) {
                float o[32];
                if (count > 0) {
                    tmem_load(o_at + d, o);
                    tmem_wait_load(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
                }
                if (!real) continue;
                if (it.parts > 1) {
                    float* const keep = part + 2 * p.slot_rows + static_cast<long long>(r) * dim + d;
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (d + i >= dim) break;
                        if (p.slots_wide != 0) {
                            store32(keep + i, reinterpret_cast<const unsigned*>(o + i));
                        } else {
                            *reinterpret_cast<float4*>(keep + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            *reinterpret_cast<float4*>(keep + i + 4) = make_float4(o[i + 4], o[i + 5], o[i + 6], o[i + 7]);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        unsigned y[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = W::pack(o[i + 2 * k] * by, o[i + 2 * k + 1] * by);
                        if (p.out_wide != 0 && d + i + 16 <= dim) {
                            store32(to + d + i, y);
                            continue;
                        }
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
                            if (d + i + h >= dim) break;
                            if (p.out_aligned != 0) {
                                *reinterpret_cast<uint4*>(to + d + i + h) = make_uint4(y[h / 2], y[h / 2 + 1], y[h / 2 + 2], y[h / 2 + 3]);
                            } else {
                                const T* const e = reinterpret_cast<const T*>(y + h / 2);
#pragma unroll
                                for (int k = 0; k < 8; ++k) to[d + i + h + k] = e[k];
                            }
                        }
                    }
                }
            }
            mma_fence_before();
            if (it.parts > 1) {
                if (real) {
                    part[r] = top;
                    part[p.slot_rows + r] = sum;
                }
                __threadfence();
                if (!(go = meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.plan.guard))) break;
                if (mine == 0) atomicAdd(p.work + kChunkHead + it.share, 1);
            } else if (real && lse != nullptr) {
                *lse = sum == 0.0f ? kNegInf : (top + log2f(sum) - W::kLift) * kChunkLn2;
            }
            bar_arrive(smem_at(&s.item_empty[slot]));
        }
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    if (role == 2) {
        if (s.plan.guard.dead != 0 && lane == 0) flag(p.c.status, GS_DEV_TIMEOUT);
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    }
    if (warp == 0) chunk_leave(p, cut.used());
}

// K or V of a layer as boxes of 64 values of the rows of a page.
bool encode(CUtensorMap* map, int dtype, const CacheView& c, const char* base, int rows) {
    const auto type = dtype == GS_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.dim), static_cast<cuuint64_t>(c.page),
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    // (A dimension of one entry is never stepped: its stride may be 0 in the cache, not here.)
    const long long row = 2ll * ((c.dim + 7) / 8 * 8);
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.page > 1 ? 2 * c.token_stride : row),
                                   static_cast<cuuint64_t>(c.heads > 1 ? 2 * c.head_stride : row),
                                   static_cast<cuuint64_t>(c.pages > 1 ? 2 * c.page_stride : row)};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
    const cuuint32_t step[4] = {1, 1, 1, 1};
    return encoder() != nullptr &&
           encoder()(map, type, 4, const_cast<char*>(base), dims, strides, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries as boxes of 64 values of a tile's rows: token after token, the heads of a group.
bool encode_q(CUtensorMap* map, int dtype, const ChunkParams& p) {
    const auto type = dtype == GS_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.c.dim), static_cast<cuuint64_t>(p.q_heads),
                                static_cast<cuuint64_t>(p.tokens)};
    const long long row = 2ll * p.c.dim;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.q_heads > 1 ? 2 * p.q_head : row),
                                   static_cast<cuuint64_t>(p.tokens > 1 ? 2 * p.q_token : row)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
    const cuuint32_t step[3] = {1, 1, 1};
    return encoder() != nullptr &&
           encoder()(map, type, 3, const_cast<void*>(p.q), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap k, v, q;
};

template <class T, int DP, bool SPLIT>
gs_status launch_as(const ChunkParams& p, const Maps& m, int blocks, gs_stream stream) {
    constexpr int bytes = static_cast<int>(sizeof(Smem<DP>));
    if (!allow_smem<chunk_mma_kernel<T, DP, SPLIT>>(bytes)) return GS_ERR_CUDA;
    return launch(chunk_mma_kernel<T, DP, SPLIT>, dim3(blocks), Shape<DP>::THREADS, bytes, 1, stream, p, m.k, m.v, m.q);
}

template <class T, bool SPLIT>
gs_status launch_type(const ChunkParams& p, const Maps& m, int blocks, gs_stream stream) {
    if (p.c.dim <= 64) return launch_as<T, 64, SPLIT>(p, m, blocks, stream);
    if (p.c.dim <= 128) return launch_as<T, 128, SPLIT>(p, m, blocks, stream);
    return launch_as<T, 256, SPLIT>(p, m, blocks, stream);
}

template <bool SPLIT>
gs_status launch_mma(int dtype, ChunkParams& p, int blocks, gs_stream stream) {
    Maps m = {};
    const int rows = p.c.page < kUnit ? p.c.page : kUnit;
    if (!encode(&m.k, dtype, p.c, p.c.k, rows) || !encode(&m.v, dtype, p.c, p.c.v, rows)) return GS_ERR_CUDA;
    // TMA brings the queries as they are, in boxes that hold whole tokens of a group, from rows on 16 bytes.
    p.q_boxes = p.q_aligned != 0 && p.q_sign > 0.0f && 128 % p.group == 0 && (p.tokens == 1 || p.q_token > 0) &&
                (p.q_heads == 1 || p.q_head > 0);
    if (p.q_boxes != 0 && !encode_q(&m.q, dtype, p)) p.q_boxes = 0;  // (strides that no map holds)
    if (dtype == GS_DTYPE_BF16) return launch_type<__nv_bfloat16, SPLIT>(p, m, blocks, stream);
    return launch_type<__half, SPLIT>(p, m, blocks, stream);
}

}  // namespace
}  // namespace gs_decode
