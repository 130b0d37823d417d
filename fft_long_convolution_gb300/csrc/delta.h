// Shared by the gated delta rule's translation units.
#pragma once
#include "views.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mma.cuh"

struct fftconv_delta_s {
    int Dk = 0, Dv = 0, dtype = 0;
    int device = 0, num_sms = 0;
    int* dev_err = nullptr;  // error word of the bounded waits (device)
};

namespace fftconv {

constexpr int kChunk = 64;  // tokens per chunk

// Log decays below this act as a reset: exp(-120) is zero in float32, and a
// chunk's running sum stays finite.  A NaN stays a NaN.
constexpr float kMinLogDecay = -120.0f;

struct DeltaArgs {
    View q, k, v, g, beta, o;
    const int32_t* offsets;
    int64_t B, T;
    int nseq, Hk, Hv, group;  // group = Hv / Hk
    float scale;
    int* err;
};

// Sequence i: its row, its first token in the row and its length, whatever the
// offsets hold (they are clamped to the row).
struct Seq {
    int64_t row, start, len;
    int64_t slot;  // first chunk slot of the sequence
};

// Chunk slots: sequence i starts at slot pos_i / 64 + i, where pos_i is its
// first token counted over the whole batch.  Sequences of len_i tokens need
// ceil(len_i / 64) slots, so ranges never meet, and B T / 64 + nseq slots are
// enough without a prefix sum over the lengths.
__device__ __forceinline__ Seq locate(const int32_t* offsets, int64_t T, int i) {
    Seq s;
    if (!offsets) {
        s = {i, 0, T, int64_t(i) * T / kChunk + i};
    } else {
        int64_t lo = offsets[i], hi = offsets[i + 1];
        lo = lo < 0 ? 0 : (lo > T ? T : lo);
        hi = hi < lo ? lo : (hi > T ? T : hi);
        s = {0, lo, hi - lo, lo / kChunk + i};
    }
    return s;
}

inline int64_t chunk_slots(int64_t B, int64_t T, int64_t nseq) { return B * T / kChunk + nseq; }

template <int DT>
__device__ __forceinline__ float load16(const View& v, int64_t off) {
    const uint16_t w = *(reinterpret_cast<const uint16_t*>(v.p) + off);
    return Op<DT>::unpack(uint32_t(w)).r;
}

template <int DT>
__device__ __forceinline__ void store16(const View& v, int64_t off, float x) {
    *(reinterpret_cast<uint16_t*>(v.p) + off) = uint16_t(Op<DT>::pack(x, 0.0f) & 0xffffu);
}

__device__ __forceinline__ float log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

}  // namespace fftconv
