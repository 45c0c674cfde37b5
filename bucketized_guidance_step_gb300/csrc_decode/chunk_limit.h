// How long a wait of chunk attention may last.
#pragma once

#ifdef __CUDACC__
#define GS_CHUNK_BOTH __host__ __device__
#else
#define GS_CHUNK_BOTH
#endif

namespace gs_decode {

// Nanoseconds that a 16th of a position of a tile's cost may take.  Measured, GB300: 0.8 to 0.9 in 16-bit caches (prompts
// of 16384 and 32768 tokens, 32 and 8 heads of 64 to 256), 2.3 with pages of 33 tokens, 6 to 9 with pages of one; 9 to 16
// in fp32, 37 where no score is finite.
constexpr int kChunkNs = 64, kChunkNsFp32 = 512;
constexpr long long kChunkMostCost = 1ll << 36;          // (an hour and more)

// What is waited for is another block's share of the call, or an item of the own one, which is a share at most: shares
// cost `each`, and what is left of a cut tile.  So the limit grows with the share: no call is too large for it, and a
// small one has the 0.2 s in which a GPU that others use too gets to it.
GS_CHUNK_BOTH constexpr unsigned long long chunk_limit_ns(long long each, int ns) {
    return 200ull * 1000ull * 1000ull +
           static_cast<unsigned long long>(each < kChunkMostCost ? each : kChunkMostCost) * static_cast<unsigned>(ns);
}

}  // namespace gs_decode
