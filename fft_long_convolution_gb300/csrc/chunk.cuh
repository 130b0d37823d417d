// Shared by the chunked kernels of the gated delta rule: where chunks are and
// what the prep kernel leaves for them.
#pragma once
#include "delta_chunk.h"

#include "tile.cuh"

namespace fftconv {

constexpr uint32_t kWaitFinal = 1u << 18;  // polls of the waits that end a CTA

// What delta_prep_kernel leaves for a chunk of one value head: the tiles P,
// (T beta) high and low part, then float32 e[64], scale G[64], b log2(e)[64],
// beta[64], then -W^T, DK rows of 64 tokens, high and low part, then what rounding
// b log2(e) left, float32 [64].
constexpr uint32_t kImgP = 0, kImgT = tile::kTile, kImgE = 3 * tile::kTile, kImgW = kImgE + 1024;
template <int DK>
constexpr uint32_t kImgR = kImgW + DK * 256;
template <int DK>
constexpr uint32_t kImage = kImgR<DK> + 256;

// Chunk slot -> sequence and chunk: the last sequence whose first slot is not
// past it.
__device__ __forceinline__ bool find_chunk(const DeltaArgs& d, int64_t slot, Seq* s, int* i, int64_t* chunk) {
    int lo = 0, hi = d.nseq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (locate(d.offsets, d.T, m).slot <= slot) lo = m;
        else hi = m - 1;
    }
    *s = locate(d.offsets, d.T, lo);
    *i = lo;
    *chunk = slot - s->slot;
    return *chunk >= 0 && *chunk * kChunk < s->len;
}

// A chunk of a value head: where its tokens are and where its image goes.
struct ChunkItem {
    int row, t0, m, h;  // m tokens; 0: no more items
    int64_t at;
};

// The next item from *next on (a stride of the grid apart) that has tokens.
__device__ __forceinline__ ChunkItem find_item(const DeltaArgs& d, int slots, int* next) {
    const int count = slots * d.Hv;
    while (*next < count) {
        const int x = *next, slot = x / d.Hv;
        Seq s;
        int si;
        int64_t ch;
        *next = count - x > int(gridDim.x) ? x + int(gridDim.x) : count;
        if (!find_chunk(d, slot, &s, &si, &ch)) continue;
        const int64_t left = s.len - ch * kChunk;
        return {int(s.row), int(s.start + ch * kChunk), int(left < kChunk ? left : kChunk), x - slot * d.Hv, x};
    }
    return {0, 0, 0, 0, 0};
}

template <typename K>
cudaError_t opt_in(K fn, size_t smem, PerDevice& cache) {
    int* slot = cache.slot();
    if (!slot) return cudaErrorInvalidDevice;
    if (!*slot) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        *slot = 1;
    }
    return cudaSuccess;
}

}  // namespace fftconv
