// Attention of chunks of new tokens over a paged cache (sm_103a), for 16-bit caches: both products on
// the tensor cores (tcgen05), sums in tensor memory, keys and values brought by TMA, a box a page.
//
// A block works on two tiles of 128 query rows at a time (one for heads of over 128 dims), which share
// every unit of keys and values.  Of its warps
//   one takes items from the queue and brings units: K and V in turn through a ring of stages in
//     shared memory, as many units ahead as the ring has room, over the ends of items;
//   one issues the products: S = Q K^T of 128 rows and the unit's positions into tensor memory, and
//     O += P V from there;
//   four a tile have a row a thread: they read S, keep the softmax's reference and sum, write the
//     weights P over S as 16-bit numbers, and at the item's end read O and store it.
// While one tile's rows take their softmax, the tensor cores work for the other.
//
// With s the scores in powers of two (times scale log2 e), the weights are 2^(s - m + kLift) with a
// reference m that is the row's largest score so far, or up to kSlack below: O and the sum are
// rescaled only when a score passes m by more, which few units after the first do.  Weights are
// rounded once to 16 bits, off by half a step, as the output is; their sums, not rounded, are fp32.
//
// Positions that a row does not see get the weight 0.  So that 0 times an infinity or NaN reaches no
// row, V is looked through in units that some row sees in part: what is not finite there is added to
// the rows that see it and then taken out of the unit (give_out).
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
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0u;
}
// Waits (kChunkLimitNs at most) for the phase of this parity; once one wait of the block has run out,
// all of them end.
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity, volatile int* dead) {
    if (bar_try(bar, parity)) return true;
    const unsigned long long t0 = chunk_clock();
    while (!bar_try(bar, parity)) {
        if (*dead != 0) return false;
        if (chunk_clock() - t0 > kChunkLimitNs) {
            *dead = 1;
            return false;
        }
    }
    return true;
}
// The same for a warp: whether all its lanes saw the phase.
__device__ __forceinline__ bool warp_wait(unsigned bar, unsigned parity, volatile int* dead) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, dead));
}
// A barrier of the threads that a barrier in shared memory counts, whole warps (one that waits with a
// limit, as every wait here).
__device__ __forceinline__ bool meet(unsigned bar, unsigned* turn, volatile int* dead) {
    bar_arrive(bar);
    const bool ok = warp_wait(bar, *turn, dead);
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

__device__ __forceinline__ void mma_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mma_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
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
// A in tensor memory.
__device__ __forceinline__ void mma_ts(unsigned d, unsigned a, unsigned long long b, unsigned what, unsigned add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(what), "r"(add)
        : "memory");
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
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
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

// A matrix in shared memory in columns of 64 values (128 bytes a row, rows permuted in groups of 8 as
// TMA's 128-byte swizzle leaves them).  K-major: groups of 8 rows follow each other.  MN-major: `next`
// bytes lead to the next 64 values.
__device__ __forceinline__ unsigned long long matrix_at(unsigned at, unsigned next) {
    return static_cast<unsigned long long>((at & 0x3ffffu) >> 4) |
           static_cast<unsigned long long>(next >> 4) << 16 | 64ull << 32 | 1ull << 46 | 2ull << 61;
}

template <class T>
struct Weights;                           // of type T: kept below 2^(kLift + kSlack)
template <>
struct Weights<__nv_bfloat16> {
    static constexpr float kLift = 0.0f, kSlack = 8.0f;
    static constexpr unsigned kExponent = 0x7f807f80u, kOne = 0x00800080u, kType = 1u;
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
    static __device__ __forceinline__ unsigned pack(float lo, float hi) {
        unsigned r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
};

// ---- shapes -----------------------------------------------------------------------------------
template <int DP>
struct Shape {
    static constexpr int TILES = DP > 128 ? 1 : 2;       // tiles of 128 rows
    static constexpr int KT = DP > 128 ? 64 : 128;       // positions of a unit
    static constexpr int Q = 128 * DP * 2, STAGE = KT * DP * 2;      // bytes
    static constexpr int STAGES = DP == 64 ? 8 : 5;
    static constexpr int GROUP = 128 * TILES;            // threads with a row
    static constexpr int THREADS = GROUP + 64, WIDTH = 128;
    // Tensor memory: S of each tile (later P, in the last half of S), then O of each.
    static constexpr int P = KT / 2, O = 256;
    static_assert(TILES * KT <= O && O + TILES * DP <= 512, "tensor memory");
    using Cut = ChunkCut<128 * TILES, 128, KT, THREADS, WIDTH>;
};

constexpr int kItems = 2;                 // items under way
template <int DP>
struct alignas(1024) Smem {
    using S = Shape<DP>;
    unsigned char q[S::TILES][S::Q];
    unsigned char ring[S::STAGES][S::STAGE];
    unsigned long long full[S::STAGES], empty[S::STAGES];
    unsigned long long item_full[kItems], item_empty[kItems];
    unsigned long long q_full[2], s_full[2], p_full[2], o_full[2], tile_meet[2], both_meet, tail, drain;
    ChunkItem items[kItems];
    int dead, seeded[2], hot[2];
    unsigned tmem;
    typename S::Cut::Shared plan;
};
static_assert(sizeof(Smem<128>) <= 227 * 1024 && sizeof(Smem<256>) <= 227 * 1024, "shared memory of a block");

// What is not finite in a unit's V: added to the rows that see it, then 0.  A warp calls it together;
// a thread's row sees positions lo .. hi - 1 and those below sinks.  `first`: O holds nothing yet.
template <class T, int DP>
__device__ __noinline__ bool give_out(unsigned char* v, unsigned o_at, int dim, int lo, int hi, int sinks,
                                      int valid, bool first, int threads, unsigned bar, unsigned* turn,
                                      volatile int* dead) {
    using S = Shape<DP>;
    for (int d0 = 0; d0 < dim; d0 += 32) {
        float o[32];
        if (first) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        } else {
            tmem_load(o_at + d0, o);
            tmem_wait_load();
        }
        for (int r = 0; r < valid; ++r) {
            if (!((r >= lo || r < sinks) && r < hi)) continue;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int d = d0 + i, c = d & 63;
                const T x = *reinterpret_cast<const T*>(v + (d >> 6) * (S::KT * 128) + r * 128 +
                                                        (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2);
                const float f = static_cast<float>(x);
                if (!(fabsf(f) <= 3.4e38f)) o[i] += f;
            }
        }
        __syncwarp();
        tmem_store32(o_at + d0, o);
        tmem_wait_store();
    }
    if (!meet(bar, turn, dead)) return false;            // every row has what it sees
    using W = Weights<T>;
    unsigned* const words = reinterpret_cast<unsigned*>(v);
    for (int x = threadIdx.x; x < S::STAGE / 4; x += threads) {
        const unsigned w = words[x], hot = ((w & W::kExponent) + W::kOne) & 0x80008000u;
        if (hot != 0u) words[x] = w & ~((hot >> 15) * 0xffffu);
    }
    async_fence();
    return meet(bar, turn, dead);
}

template <class T, int DP>
__global__ void __launch_bounds__(Shape<DP>::THREADS, 1)
chunk_mma_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
    using S = Shape<DP>;
    using W = Weights<T>;
    constexpr int KT = S::KT, TILES = S::TILES;
    extern __shared__ __align__(1024) unsigned char raw[];
    Smem<DP>& s = *reinterpret_cast<Smem<DP>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dim = p.c.dim;
    const ChunkUnits<KT> units(p.c.page);
    const bool loader = warp == S::GROUP / 32, issuer = warp == S::GROUP / 32 + 1;

    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            bar_init(smem_at(&s.full[i]), 1);
            bar_init(smem_at(&s.empty[i]), 1);
        }
        for (int i = 0; i < kItems; ++i) {
            bar_init(smem_at(&s.item_full[i]), 1);
            bar_init(smem_at(&s.item_empty[i]), S::GROUP + 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_at(&s.q_full[i]), 128);
            bar_init(smem_at(&s.s_full[i]), 1);
            bar_init(smem_at(&s.p_full[i]), 128);
            bar_init(smem_at(&s.o_full[i]), 1);
            bar_init(smem_at(&s.tile_meet[i]), 128);
            s.hot[i] = 0;
        }
        bar_init(smem_at(&s.both_meet), S::GROUP);
        bar_init(smem_at(&s.tail), 1);
        bar_init(smem_at(&s.drain), 1);
        s.dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (issuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&s.tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (units.span < KT) {                // rows of a stage that no box reaches
        for (int x = tid; x < S::STAGES * S::STAGE / 16; x += S::THREADS)
            reinterpret_cast<uint4*>(s.ring)[x] = make_uint4(0u, 0u, 0u, 0u);
        async_fence();
    }
    grid_wait();
    grid_trigger();
    typename S::Cut cut = {&s.plan};
    mma_fence_before();
    cut.find(p);                          // (ends with a barrier)
    mma_fence_after();
    const unsigned tmem = s.tmem;
    int stage = 0;                        // the ring: stage, and the parity of its use
    unsigned turn = 0;
    unsigned loads = 0;                   // loader: stages filled

    if (loader) {
        const int halves = (dim + 63) / 64;
        const int page_rows = min(p.c.page, KT);
        const unsigned box = page_rows * 128;
        const int pages = units.per > 0 ? 1 : KT / p.c.page, boxes = pages * halves;
        unsigned tails = 0, bad = 0;
        bool go = true;
        for (int n = 0; go;) {
            const int slot = n & 1;
            int kind = 0;
            if (lane == 0) {
                ChunkItem it;
                do {
                    it = cut.item(p, atomicAdd(p.work, 1));
                } while (it.kind != 0 && it.rows == 0);
                if (bar_wait(smem_at(&s.item_empty[slot]), ((n >> 1) & 1) ^ 1, &s.dead)) {
                    s.items[slot] = it;
                    kind = it.kind;
                    bar_arrive(smem_at(&s.item_full[slot]));
                } else {
                    kind = -1;
                }
            }
            kind = __shfl_sync(0xffffffffu, kind, 0);
            __syncwarp();
            ++n;
            if (kind <= 0) break;
            if (kind == 2) continue;
            const ChunkItem& it = s.items[slot];
            const int head = it.head, len = it.e.len, lo = it.lo, hi = it.hi;
            const ChunkSpan span = it.span;
            const int* const table = p.c.table + static_cast<long long>(it.e.seq) * p.c.cols;
            // Box `lane` of a unit, its page one unit ahead.
            auto page_of = [&](int at, int x) {
                const int pos = at + x / halves * p.c.page;          // page <= KT: the box's first position
                return pos < len ? table[pos / p.c.page] : -2;
            };
            int count, row;
            int at = lo < hi ? units.first(span.unit(lo), &count, &row) : 0;
            int next = lo < hi && lane < boxes ? page_of(at, lane) : -2;
            for (int u = lo; u < hi && go; ++u) {
                at = units.first(span.unit(u), &count, &row);
                int page = next;
                if (u + 1 < hi) {
                    int c, r;
                    const int then = units.first(span.unit(u + 1), &c, &r);
                    next = lane < boxes ? page_of(then, lane) : -2;
                }
                const int valid = min(count, len - at);
                const int live = (units.per > 0 ? 1 : (valid + p.c.page - 1) / p.c.page) * halves;
                for (int kv = 0; kv < 2; ++kv) {
                    const CUtensorMap* const map = kv == 0 ? &k_map : &v_map;
                    if (!warp_wait(smem_at(&s.empty[stage]), turn ^ 1, &s.dead)) {
                        go = false;
                        break;
                    }
                    // Rows past the sequence's end hold anything: of V they are taken out.
                    const bool tail = kv == 1 && valid < count;
                    const unsigned bar = smem_at(tail ? &s.tail : &s.full[stage]);
                    if (lane == 0) bar_expect(bar, live * box);
                    __syncwarp();
                    for (int x = lane; x < live; x += 32) {
                        if (x != lane) page = page_of(at, x);
                        const bool ok = page >= 0 && page < p.c.pages;
                        if (!ok) bad |= GS_DEV_BAD_SEQ;
                        const int in = x / halves, col = x - in * halves;
                        load_box(smem_at(s.ring[stage]) + col * (KT * 128) + in * box, map, col * 64, row, head,
                                 ok ? page : p.c.pages, bar);
                    }
                    if (live > 32) page = lane < boxes ? page_of(at, lane) : -2;
                    ++loads;
                    if (tail) {
                        if (!warp_wait(bar, tails & 1, &s.dead)) {
                            go = false;
                            break;
                        }
                        ++tails;
                        for (int x = lane; x < (KT - valid) * 8 * halves; x += 32) {
                            const int col = x / ((KT - valid) * 8), y = x - col * ((KT - valid) * 8);
                            *reinterpret_cast<uint4*>(s.ring[stage] + col * (KT * 128) + valid * 128 + y * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        async_fence();
                        __syncwarp();
                        if (lane == 0) bar_arrive(smem_at(&s.full[stage]));
                    }
                    if (++stage == S::STAGES) {
                        stage = 0;
                        turn ^= 1;
                    }
                }
            }
        }
        flag(p.c.status, bad);
        // Where a wait has run out, the boxes under way land before the block ends.
        __syncwarp();
        if (s.dead != 0) {
            const unsigned long long t0 = chunk_clock();
            while (chunk_clock() - t0 < 10ull * 1000ull * 1000ull) __nanosleep(10000);
        }
    } else if (issuer) {
        if (lane == 0) {
            const unsigned kind = 1u << 4 | W::kType << 7 | W::kType << 10 | (128u >> 4) << 24;
            const unsigned what_s = kind | static_cast<unsigned>(KT >> 3) << 17;
            const unsigned what_o = kind | 1u << 16 | static_cast<unsigned>((dim + 15) / 16 * 2) << 17;
            const int steps = (dim + 15) / 16;
            unsigned q_turn = 0, p_turn = 0;
            bool go = true;
            for (int n = 0; go; ++n) {
                const int slot = n & 1;
                if (!bar_wait(smem_at(&s.item_full[slot]), (n >> 1) & 1, &s.dead)) break;
                const int item = s.items[slot].kind, rows = s.items[slot].rows;
                const int count = s.items[slot].hi - s.items[slot].lo;
                bar_arrive(smem_at(&s.item_empty[slot]));
                if (item == 0) break;
                if (item == 2 || count == 0) continue;
                const int tiles = TILES == 2 && rows > 128 ? 2 : 1;
                auto scores = [&](int w, unsigned k) {
                    const unsigned q = smem_at(s.q[w]);
                    for (int i = 0; i < steps; ++i)
                        mma_ss(tmem + w * KT, matrix_at(q + (i >> 2) * (128 * 128) + (i & 3) * 32, 16),
                               matrix_at(k + (i >> 2) * (KT * 128) + (i & 3) * 32, 16), what_s, i > 0);
                };
                if (!(go = bar_wait(smem_at(&s.full[stage]), turn, &s.dead))) break;
                for (int w = 0; w < tiles && go; ++w) {
                    go = bar_wait(smem_at(&s.q_full[w]), q_turn >> w & 1, &s.dead);
                    q_turn ^= 1u << w;
                    if (!go) break;
                    mma_fence_after();
                    scores(w, smem_at(s.ring[stage]));
                    mma_commit(smem_at(&s.s_full[w]));
                }
                if (!go) break;
                mma_commit(smem_at(&s.empty[stage]));
                for (int u = 0; u < count && go; ++u) {
                    if (++stage == S::STAGES) {
                        stage = 0;
                        turn ^= 1;
                    }
                    const int v_stage = stage;
                    if (!(go = bar_wait(smem_at(&s.full[stage]), turn, &s.dead))) break;
                    const bool more = u + 1 < count;
                    if (more) {
                        if (++stage == S::STAGES) {
                            stage = 0;
                            turn ^= 1;
                        }
                    }
                    for (int w = 0; w < tiles && go; ++w) {
                        go = bar_wait(smem_at(&s.p_full[w]), p_turn >> w & 1, &s.dead);
                        p_turn ^= 1u << w;
                        if (!go) break;
                        mma_fence_after();
                        const unsigned v = smem_at(s.ring[v_stage]);
                        const unsigned add = u > 0 || *static_cast<volatile int*>(&s.seeded[w]) != 0;
                        for (int i = 0; i < KT / 16; ++i)
                            mma_ts(tmem + S::O + w * DP, tmem + w * KT + S::P + i * 8, matrix_at(v + i * 2048, KT * 128),
                                   what_o, add | (i > 0));
                        mma_commit(smem_at(&s.o_full[w]));
                        if (w == tiles - 1) mma_commit(smem_at(&s.empty[v_stage]));
                        if (more) {
                            if (w == 0 && !(go = bar_wait(smem_at(&s.full[stage]), turn, &s.dead))) break;
                            scores(w, smem_at(s.ring[stage]));
                            mma_commit(smem_at(&s.s_full[w]));
                            if (w == tiles - 1) mma_commit(smem_at(&s.empty[stage]));
                        }
                    }
                }
                if (++stage == S::STAGES) {
                    stage = 0;
                    turn ^= 1;
                }
            }
            if (s.dead != 0) {            // products under way end before the block does
                mma_commit(smem_at(&s.drain));
                const unsigned long long t0 = chunk_clock();
                while (!bar_try(smem_at(&s.drain), 0) && chunk_clock() - t0 < 10ull * 1000ull * 1000ull) {}
            }
        }
        __syncwarp();
    } else if (warp < S::GROUP / 32) {
        const int w = TILES == 2 ? warp >> 2 : 0, mine = tid & 127;
        const unsigned lanes = static_cast<unsigned>((warp & 3) * 32) << 16;
        const unsigned s_at = tmem + lanes + w * KT, o_at = tmem + lanes + S::O + w * DP;
        const float scale = p.scale_log2;
        unsigned s_turn = 0, o_turn = 0, meet_turn = 0, both_turn = 0;       // parities of the next phases
        int looked = 0;                   // units looked through
        int v_stage = 0;                  // the ring as the issuer goes through it
        unsigned v_turn = 0;
        auto next_stage = [&] {
            if (++v_stage == S::STAGES) {
                v_stage = 0;
                v_turn ^= 1;
            }
        };
        bool go = true;
        for (int n = 0; go; ++n) {
            const int slot = n & 1;
            if (!warp_wait(smem_at(&s.item_full[slot]), (n >> 1) & 1, &s.dead)) break;
            const ChunkItem& it = s.items[slot];
            if (it.kind == 0) break;
            if (it.kind == 2) {
                if (mine == 0 && !chunk_wait_parts(p.work + kChunkHead + it.tile, it.need))
                    *static_cast<volatile int*>(&s.dead) = 1;
                if (!meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.dead)) break;
                chunk_join<T>(p, it, tid, S::GROUP, W::kLift);
                bar_arrive(smem_at(&s.item_empty[slot]));
                continue;
            }
            const int count = it.hi - it.lo, tiles = TILES == 2 && it.rows > 128 ? 2 : 1;
            if (w >= tiles) {
                for (int u = 0; u < 2 * count; ++u) next_stage();
                bar_arrive(smem_at(&s.item_empty[slot]));
                continue;
            }
            const int r = w * 128 + mine, row = it.row + r;         // of the tile, of the entry
            const bool real = r < it.rows;
            const int from = it.e.len - it.e.m;
            const int token = row / p.group, pos = from + token;
            if (count > 0) {
                // The row of Q, with the scale's sign.
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
                bar_arrive(smem_at(&s.q_full[w]));
            }
            float top = kNegInf, sum = 0.0f;
            const int first_pos = from + it.row / p.group, last_pos = from + (it.row + it.rows - 1) / p.group;
            for (int u = 0; u < count; ++u) {
                int here, in_page;
                const int at = units.first(it.span.unit(it.lo + u), &here, &in_page);
                const int valid = min(here, it.e.len - at);
                // What this row sees of the unit: lo .. hi - 1, and those below sink.
                const int hi = min(valid, pos - at + 1);
                const int lo = p.window > 0 ? pos - p.window + 1 - at : 0;
                const int sink = p.window > 0 ? p.sinks - at : 0;
                next_stage();                            // to V's
                // Whether some row of the block's tiles sees the unit in part (all threads alike).
                const bool part = at + valid - 1 > first_pos ||
                                  (p.window > 0 && at <= last_pos - p.window && at + valid > p.sinks);
                if (!(go = warp_wait(smem_at(&s.s_full[w]), s_turn, &s.dead))) break;
                s_turn ^= 1;
                mma_fence_after();
                bool odd = false;
                if (part) {
                    if (!(go = warp_wait(smem_at(&s.full[v_stage]), v_turn, &s.dead))) break;
                    unsigned hot = 0;
                    const uint4* const v = reinterpret_cast<const uint4*>(s.ring[v_stage]);
#pragma unroll 4
                    for (int x = mine; x < S::STAGE / 16; x += 128) {
                        const uint4 y = v[x];
                        hot |= ((y.x & W::kExponent) + W::kOne) | ((y.y & W::kExponent) + W::kOne) |
                               ((y.z & W::kExponent) + W::kOne) | ((y.w & W::kExponent) + W::kOne);
                    }
                    // (All of a tile's threads look at all of it.)
                    ++looked;
                    if (__any_sync(0xffffffffu, (hot & 0x80008000u) != 0u) && lane == 0)
                        *static_cast<volatile int*>(&s.hot[w]) = looked;
                    if (!(go = meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.dead))) break;
                    odd = *static_cast<volatile int*>(&s.hot[w]) == looked;
                }
                if (odd) {
                    if (u > 0 && !(go = warp_wait(smem_at(&s.o_full[w]), o_turn ^ 1, &s.dead))) break;
                    mma_fence_after();
                    if (!(go = give_out<T, DP>(s.ring[v_stage], o_at, dim, lo, hi, sink, valid, u == 0, 128 * tiles,
                                               smem_at(tiles == 2 ? &s.both_meet : &s.tile_meet[w]),
                                               tiles == 2 ? &both_turn : &meet_turn, &s.dead)))
                        break;
                }
                if (u == 0 && mine == 0) s.seeded[w] = odd;
                next_stage();                            // to the next K's
                // S 64 columns at a time, the last ones last: they stay in registers for the weights, the
                // others are read again (a thread with all 128 would have to spill).
                float x[64];
                const bool whole = __all_sync(0xffffffffu, hi >= KT && lo <= 0);
                auto read = [&](int c0) {
                    tmem_load(s_at + c0, x);
                    tmem_load(s_at + c0 + 32, x + 32);
                    tmem_wait_load();
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (!(c < hi - c0 && (c >= lo - c0 || c < sink - c0))) x[c] = kNegInf;
                    }
                };
                float up = kNegInf;
#pragma unroll
                for (int c0 = 0; c0 < KT; c0 += 64) {
                    read(c0);
                    float up0 = up, up1 = x[1], up2 = x[2], up3 = x[3];
                    up0 = fmaxf(up0, x[0]);
#pragma unroll
                    for (int c = 4; c < 64; c += 4) {
                        up0 = fmaxf(up0, x[c]);
                        up1 = fmaxf(up1, x[c + 1]);
                        up2 = fmaxf(up2, x[c + 2]);
                        up3 = fmaxf(up3, x[c + 3]);
                    }
                    up = fmaxf(fmaxf(up0, up1), fmaxf(up2, up3));
                }
                up *= scale;
                const bool move = up > top + W::kSlack || (top == kNegInf && up > kNegInf);
                if (__any_sync(0xffffffffu, move)) {
                    const float by = move ? chunk_pow2(top - up) : 1.0f;     // 0 at the first position
                    if (move) top = up;
                    sum *= by;
                    if (u > 0) {
                        if (!(go = warp_wait(smem_at(&s.o_full[w]), o_turn ^ 1, &s.dead))) break;
                        mma_fence_after();
                        for (int d = 0; d < dim; d += 32) {
                            float o[32];
                            tmem_load(o_at + d, o);
                            tmem_wait_load();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] *= by;
                            tmem_store32(o_at + d, o);
                        }
                        tmem_wait_store();
                    }
                }
                const float base = W::kLift - (top == kNegInf ? 0.0f : top);
                float sum1 = 0.0f, sum2 = 0.0f, sum3 = 0.0f;
#pragma unroll
                for (int c0 = KT - 64; c0 >= 0; c0 -= 64) {
                    if (c0 != KT - 64) read(c0);
#pragma unroll
                    for (int h = 0; h < 64; h += 32) {
                        unsigned r16[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float a = chunk_pow2(fmaf(x[h + i], scale, base));
                            const float b = chunk_pow2(fmaf(x[h + i + 1], scale, base));
                            const float e = chunk_pow2(fmaf(x[h + i + 2], scale, base));
                            const float f = chunk_pow2(fmaf(x[h + i + 3], scale, base));
                            sum += a;
                            sum1 += b;
                            sum2 += e;
                            sum3 += f;
                            r16[i / 2] = W::pack(a, b);
                            r16[i / 2 + 1] = W::pack(e, f);
                        }
                        // (over columns of S that have been read)
                        tmem_store16(s_at + S::P + (c0 + h) / 2, r16);
                    }
                }
                sum = (sum + sum1) + (sum2 + sum3);
                tmem_wait_store();
                mma_fence_before();
                bar_arrive(smem_at(&s.p_full[w]));
                o_turn ^= 1;
            }
            if (!go) break;
            // (o_turn has changed count times: the last phase's parity is its opposite.)
            if (count > 0) {
                if (!(go = warp_wait(smem_at(&s.o_full[w]), o_turn ^ 1, &s.dead))) break;
                mma_fence_after();
            }
            float* lse = nullptr;
            T* const to = real ? chunk_out<T>(p, it, row, &lse) : nullptr;
            float* const part = p.slots + it.slot * chunk_slot_words(p.slot_rows, dim);
            const float by = sum > 0.0f ? 1.0f / sum : sum;         // a NaN stays one
            for (int d = 0; d < dim; d += 32) {
                float o[32];
                if (count > 0) {
                    tmem_load(o_at + d, o);
                    tmem_wait_load();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
                }
                if (!real) continue;
                if (it.parts > 1) {
                    float* const keep = part + 2 * p.slot_rows + static_cast<long long>(r) * dim + d;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (d + i < dim) *reinterpret_cast<float4*>(keep + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        if (d + i >= dim) break;
                        uint4 y;
                        y.x = W::pack(o[i] * by, o[i + 1] * by);
                        y.y = W::pack(o[i + 2] * by, o[i + 3] * by);
                        y.z = W::pack(o[i + 4] * by, o[i + 5] * by);
                        y.w = W::pack(o[i + 6] * by, o[i + 7] * by);
                        if (p.out_aligned) {
                            *reinterpret_cast<uint4*>(to + d + i) = y;
                        } else {
                            const T* const e = reinterpret_cast<const T*>(&y);
#pragma unroll
                            for (int k = 0; k < 8; ++k) to[d + i + k] = e[k];
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
                if (!(go = meet(smem_at(&s.tile_meet[w]), &meet_turn, &s.dead))) break;
                if (mine == 0) atomicAdd(p.work + kChunkHead + it.tile, 1);
            } else if (real && lse != nullptr) {
                *lse = sum == 0.0f ? kNegInf : (top + log2f(sum) - W::kLift) * kChunkLn2;
            }
            bar_arrive(smem_at(&s.item_empty[slot]));
        }
    }
    mma_fence_before();
    __syncthreads();
    mma_fence_after();
    if (issuer) {
        if (s.dead != 0 && lane == 0) flag(p.c.status, GS_DEV_TIMEOUT);
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

template <class T, int DP>
gs_status launch_as(const ChunkParams& p, const CUtensorMap& k, const CUtensorMap& v, int blocks, gs_stream stream) {
    constexpr int bytes = static_cast<int>(sizeof(Smem<DP>));
    if (!allow_smem<chunk_mma_kernel<T, DP>>(bytes)) return GS_ERR_CUDA;
    return launch(chunk_mma_kernel<T, DP>, dim3(blocks), Shape<DP>::THREADS, bytes, 1, stream, p, k, v);
}

template <class T>
gs_status launch_type(const ChunkParams& p, const CUtensorMap& k, const CUtensorMap& v, int blocks, gs_stream stream) {
    if (p.c.dim <= 64) return launch_as<T, 64>(p, k, v, blocks, stream);
    if (p.c.dim <= 128) return launch_as<T, 128>(p, k, v, blocks, stream);
    return launch_as<T, 256>(p, k, v, blocks, stream);
}

}  // namespace

ChunkShape chunk_mma_shape(int dim) { return {dim > 128 ? 128 : 256, sm_count()}; }

gs_status launch_chunk_mma(int dtype, const ChunkParams& p, int blocks, gs_stream stream) {
    CUtensorMap k, v;
    const int unit = p.c.dim > 128 ? 64 : 128;
    const int rows = p.c.page < unit ? p.c.page : unit;
    if (!encode(&k, dtype, p.c, p.c.k, rows) || !encode(&v, dtype, p.c, p.c.v, rows)) return GS_ERR_CUDA;
    if (dtype == GS_DTYPE_BF16) return launch_type<__nv_bfloat16>(p, k, v, blocks, stream);
    return launch_type<__half>(p, k, v, blocks, stream);
}

}  // namespace gs_decode
