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
    // what the backward needs, per chunk slot and value head, or null: S^T at the
    // chunk's start ([DK / 64] blocks of DV rows of 64), Vn^T (DV rows of 64) and
    // T (64 rows of 64), 16-bit, rows of 128 bytes in the tiles' swizzled order
    uint8_t *saved_s, *saved_v, *saved_t;
    // an image per chunk slot and value head, and per segment slot and
    // value head a state [DK][DV] and a transition matrix [DK][DK]
    uint8_t* images;
    float *seg_state, *seg_trans;
    int64_t slots, segments, seg_chunks;
    int sms;
};

// Bytes of an image.
constexpr size_t prep_image(int dk) { return 3 * 8192 + 1024 + size_t(dk) * 256 + 256; }

// Sets slots, segments and seg_chunks from the sizes in a->d.
void plan_segments(ChunkArgs* a, int sms);

// The gradients' kernels (delta_grad.cu).  d.o is not used; images, saved_s,
// saved_v and saved_t come from the forward.
struct GradArgs {
    CUtensorMap mq, mk, mv, mo, mdq, mdk, mdv;  // mo: the gradient of o
    DeltaArgs d;
    View dq, dk, dv, dg, dbeta;
    const float* d_state_out;
    float* d_state_in;
    const uint8_t *images, *saved_s, *saved_v, *saved_t;
    // scratch, per chunk slot and value head: dS^T at the chunk's end (as saved_s)
    // and dR (tiles of 64 tokens x 64 features; high parts, then low); per token and value head, when
    // value heads share a key head, dq and dk in float32, else null
    uint8_t *ds, *dr;
    float *dqh, *dkh;
    int64_t slots;
    int sms;
};

cudaError_t launch_delta_backward(const GradArgs& a, int dt, int dk, int dv, cudaStream_t st);

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
