// Shared by the decode kernels: checks of a cache's description, launches with
// programmatic dependent launch, storage types, block-wide scans, cluster helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "gs_decode.h"

namespace gs_decode {

constexpr float kNegInf = -__builtin_huge_valf();

inline long long elem_size(int dtype) { return dtype == GS_DTYPE_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) {
    return dtype == GS_DTYPE_F32 || dtype == GS_DTYPE_BF16 || dtype == GS_DTYPE_F16;
}
inline bool aligned(const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// The cache's description as the kernels read it.
struct CacheView {
    int layers, pages, heads, page, dim, seqs, cols;
    long long layer_stride, page_stride, head_stride, token_stride;   // elements
    char* k;
    char* v;
    int* table;
    int* lens;
    int* refs;
    unsigned* status;
    int* work;
    int* refused;                         // [seqs] of the workspace, see below; null where that is too small
};

// A cache's workspace, in words: [0] the number of copies a call asks for, [1] held pages, [4 ..]
// the copies as (from, to, tokens, -), then a word a page (compact: the rank of a moved page), then
// a word a sequence: what gs_pages_extend refused it last.  That word is the sequence's length + 1
// at the time (0: nothing), so that it says nothing of a sequence whose length has changed since.
inline long long copy_slots(const gs_kv_cache* c) {
    return c->pages > c->seqs ? c->pages : c->seqs;
}
inline long long refused_at(const gs_kv_cache* c) {
    return 4 + 4 * copy_slots(c) + static_cast<long long>(c->pages);
}
inline long long workspace_need(const gs_kv_cache* c) {
    return 4 * (refused_at(c) + c->seqs);
}
inline gs_status check_workspace(const gs_kv_cache* c) {
    if (c->workspace == nullptr || !aligned(c->workspace, 16) ||
        c->workspace_bytes < workspace_need(c))
        return GS_ERR_INVALID_ARG;
    return GS_OK;
}
// Whether gs_pages_extend left the sequence at this length: its last positions were not given to
// the tokens that come.
__device__ __forceinline__ bool was_refused(int mark, int len) { return mark == len + 1; }

// Sizes alone (what a workspace depends on).
inline gs_status check_cache_sizes(const gs_kv_cache* c) {
    if (c == nullptr) return GS_ERR_INVALID_ARG;
    if (!known_dtype(c->dtype) || c->layers < 1 || c->pages < 1 || c->kv_heads < 1 ||
        c->page < 1 || c->dim < 1 || c->seqs < 1 || c->cols < 1)
        return GS_ERR_INVALID_ARG;
    if (c->seqs > GS_MAX_SEQS || c->pages > (1 << 28) || c->page > (1 << 20) || c->kv_heads > (1 << 16) ||
        static_cast<long long>(c->cols) * c->page > (1ll << 30) ||
        static_cast<long long>(c->layers) * c->kv_heads > (1ll << 30) ||
        static_cast<long long>(c->kv_heads) * c->page * c->dim > (1ll << 30))
        return GS_ERR_UNSUPPORTED;
    if (c->dim > 256 || (c->dim * elem_size(c->dtype)) % 16 != 0) return GS_ERR_UNSUPPORTED;
    return GS_OK;
}

inline gs_status check_cache(const gs_kv_cache* c, CacheView* out) {
    const gs_status st = check_cache_sizes(c);
    if (st != GS_OK) return st;
    if (c->k == nullptr || c->v == nullptr || c->table == nullptr || c->lens == nullptr ||
        c->refs == nullptr)
        return GS_ERR_INVALID_ARG;
    const long long es = elem_size(c->dtype);
    const int64_t strides[4] = {c->layer_stride, c->page_stride, c->head_stride, c->token_stride};
    const int sizes[4] = {c->layers, c->pages, c->kv_heads, c->page};
    for (int i = 0; i < 4; ++i) {
        if (strides[i] < 0) return GS_ERR_INVALID_ARG;
        if (sizes[i] > 1 && strides[i] < c->dim) return GS_ERR_INVALID_ARG;   // rows overlap
        if ((strides[i] * es) % 16 != 0) return GS_ERR_UNSUPPORTED;
    }
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return GS_ERR_UNSUPPORTED;
    if (!aligned(c->table, 4) || !aligned(c->lens, 4) || !aligned(c->refs, 4))
        return GS_ERR_INVALID_ARG;
    out->layers = c->layers;
    out->pages = c->pages;
    out->heads = c->kv_heads;
    out->page = c->page;
    out->dim = c->dim;
    out->seqs = c->seqs;
    out->cols = c->cols;
    out->layer_stride = c->layer_stride;
    out->page_stride = c->page_stride;
    out->head_stride = c->head_stride;
    out->token_stride = c->token_stride;
    out->k = static_cast<char*>(c->k);
    out->v = static_cast<char*>(c->v);
    out->table = c->table;
    out->lens = c->lens;
    out->refs = c->refs;
    out->status = c->dev_status;
    out->work = static_cast<int*>(c->workspace);
    out->refused = check_workspace(c) == GS_OK ? out->work + refused_at(c) : nullptr;
    return GS_OK;
}

inline int sm_count() {
    static std::atomic<int> cached{0};
    int n = cached.load(std::memory_order_relaxed);
    if (n == 0) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = 152;   // GB300 (a workspace is sized before any device call may work)
            return n;
        }
        cached.store(n, std::memory_order_relaxed);
    }
    return n;
}

// Opens a kernel's dynamic shared memory to what the device allows, once a kernel and device.
template <auto K>
inline bool allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    if (bytes <= 40 * 1024) return true;         // (48 KB with the kernel's own static part)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = 1ull << (dev & 63);
    if ((done.load(std::memory_order_relaxed) & bit) != 0) return true;
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, K) != cudaSuccess ||
        cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - static_cast<int>(a.sharedSizeBytes)) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Every decode kernel is launched with programmatic stream serialization: its blocks may be
// placed before the stream's previous kernel ends, and wait for it (grid_wait) before they
// touch memory.  (So no kernel has read-only pointers - restrict, __ldg - whose loads a compiler
// may move above the wait.)
template <class... P, class... A>
inline gs_status launch(void (*kernel)(P...), dim3 grid, int threads, int smem, int cluster,
                        gs_stream stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        (void)cudaGetLastError();
        return GS_ERR_CUDA;
    }
    return GS_OK;
}

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the stream's next kernel place its blocks (it still waits for this grid's end).
__device__ __forceinline__ void grid_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ void flag(unsigned* status, unsigned bits) {
    if (status != nullptr && bits != 0u) atomicOr(status, bits);
}

// ---- clusters -----------------------------------------------------------------------------
__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of all blocks of the cluster; orders their memory accesses.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at `local` (shared memory of this block) in the block of rank r.
__device__ __forceinline__ int cluster_read(const int* local, unsigned r) {
    const unsigned a = static_cast<unsigned>(__cvta_generic_to_shared(local));
    unsigned b;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(a), "r"(r));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(b) : "memory");
    return v;
}

// Exclusive sum over the block of one value a thread; *total = the sum.  `tmp`: THREADS / 32 + 1
// values of shared memory.  Ends with every thread past its reads of tmp.
template <int THREADS, class V>
__device__ __forceinline__ V block_scan(V v, V* tmp, V* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    V inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const V o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) tmp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        V w = lane < THREADS / 32 ? tmp[lane] : V(0);
        V winc = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const V o = __shfl_up_sync(0xffffffffu, winc, d);
            if (lane >= d) winc += o;
        }
        if (lane < THREADS / 32) tmp[lane] = winc - w;
        if (lane == 31) tmp[THREADS / 32] = winc;
    }
    __syncthreads();
    const V before = tmp[warp] + inc - v;
    *total = tmp[THREADS / 32];
    __syncthreads();
    return before;
}

// ---- storage types -------------------------------------------------------------------------
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// The 16 / sizeof(T) values of a 16-byte vector.
template <class T>
__device__ __forceinline__ void unpack16(uint4 r, float* f) {
    if constexpr (sizeof(T) == 4) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    } else {
        const unsigned w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = p.x;
                f[2 * i + 1] = p.y;
            }
        }
    }
}

// 16 bytes at p, whatever p's alignment (a multiple of the element's size).
template <class T>
__device__ __forceinline__ uint4 load16_any(const T* p, bool is_aligned) {
    if (is_aligned) return *reinterpret_cast<const uint4*>(p);
    uint4 r;
    T* d = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) d[i] = p[i];
    return r;
}

}  // namespace gs_decode
