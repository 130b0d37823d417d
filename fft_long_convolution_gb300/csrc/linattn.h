// Shared by the translation units of the linear attention.
#pragma once
#include "delta.h"

struct fftconv_linattn_s {
    int Dk = 0, Dv = 0, dtype = 0;
    int device = 0, num_sms = 0;
    int* dev_err = nullptr;  // error word of the bounded waits (device)
};

namespace fftconv {

// One walk over whole sequences: with l = exp(decay) of the head, forward in time
//   S <- l S + s_up k_t v_t^T,  o_t = s_in S'^T q_t + s_p (q_t.k_t) v_t,  S' = l S before the token
// and backward in time (reverse)
//   o_t = s_in S^T q_t + s_p (q_t.k_t) v_t,  S <- l (S + s_up k_t v_t^T).
// The outputs are a walk over (q, k, v) with s_in = s_p = scale, s_up = 1; the
// gradients are three more: dQ over (dO, V, K) from S^T; dV over (K, Q, dO) and dK
// over (V, dO, Q) in reverse, with s_up = s_p = scale, s_in = 1, from the gradient
// of the final state.
struct Walk {
    View q, k, v, o;
    float* o32;      // outputs as float32 [B][T][H][DV] instead of o, or null
    int gq, gk, gv;  // head h uses head h / g of q, k, v
    const float* decay;
    const int32_t* offsets;
    int64_t T;
    int nseq, H;
    float s_in, s_up, s_p;
    bool reverse;
    const float* state_in;  // [nseq][H][DK][DV], or (turned) [nseq][H][DV][DK]; null: zero
    bool turned;
    float* state_out;  // [nseq][H][DK][DV], or null
};

// The log decay of a head, as the kernels take it.
__device__ __forceinline__ float head_decay(const float* decay, int h) {
    const float g = decay[h];
    return g < kMinLogDecay ? kMinLogDecay : (g > 0.0f ? 0.0f : g);  // a NaN stays a NaN
}

// l = exp(g) as keep + part: where l is above 1/2 keep = 1 and part = l - 1, which
// float32 holds to its own 24 bits: a state that loses 2^-12 a token for thousands
// of tokens is then off by roundings of either sign, not by thousands of times the
// one error of a rounded l.  l x + y is keep x + (part x + y).
struct Decay {
    float keep, part;
};

__device__ __forceinline__ Decay decay_over(float g, float tokens) {
    const float x = g * tokens;
    return x > -0.69f ? Decay{1.0f, expm1f(x)} : Decay{0.0f, expf(x)};
}

__device__ __forceinline__ float decayed(const Decay& l, float x, float y) { return fmaf(l.keep, x, fmaf(l.part, x, y)); }

}  // namespace fftconv
