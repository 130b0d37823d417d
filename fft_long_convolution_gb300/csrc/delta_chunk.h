// Launch of the chunked gated delta rule (delta_chunk.cu).
#pragma once
#include <cuda.h>

#include "delta.h"
#include "device.h"

namespace fftconv {

struct ChunkArgs {
    CUtensorMap mq, mk, mv;  // [B][T][H][D] as boxes of 64 tokens x 64 features
    DeltaArgs d;
    const float* state_in;
    float* state_out;
    // what the backward needs, per chunk slot and value head, or null: S^T at
    // the chunk's start [DV][DK], Vn^T [DV][64], T [64][64], all 16-bit
    uint16_t *saved_s, *saved_v, *saved_t;
    // scratch: an image per chunk slot and value head, and per segment slot and
    // value head a state [DK][DV] and a transition matrix [DK][DK]
    uint8_t* images;
    float *seg_state, *seg_trans;
    int64_t slots, segments, seg_chunks;
    int sms;
};

// Bytes of an image.
constexpr size_t prep_image(int dk) { return 3 * 8192 + 1024 + size_t(dk) * 256; }

// Sets slots, segments and seg_chunks from the sizes in a->d.
void plan_segments(ChunkArgs* a, int sms);

cudaError_t launch_delta_forward(const ChunkArgs& a, int dt, int dk, int dv, cudaStream_t st);

// A tensor map over a token-major view, boxes of 64 tokens x 64 features of one
// head, swizzled by 128 bytes; tokens past T read as zeros.
inline bool encode_tokens_map(CUtensorMap* m, const View& v, int64_t B, int64_t T, int64_t H, int64_t D, int dt) {
    TensorMapEncoder enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(T), cuuint64_t(B)};
    const cuuint64_t strides[3] = {cuuint64_t(v.h) * 2, cuuint64_t(v.t) * 2, cuuint64_t(v.b) * 2};
    const cuuint32_t box[4] = {64, 1, 64, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, dt == FFTCONV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace fftconv
