// What the recurrent mixers' calls share around their walks over packed rows: zeros in
// the tokens of no sequence, and the sum of a key head's gradients over the value heads
// that it is shared by.
#pragma once
#include "delta.h"

namespace fftconv {
namespace {

// The tokens of a packed row that belong to a sequence: from the first offset to the
// last one (offsets do not decrease); none without sequences.
struct Covered {
    int64_t lo, hi;
};

__device__ __forceinline__ Covered covered(const int32_t* offsets, int nseq, int64_t T) {
    int64_t lo = nseq ? offsets[0] : T, hi = nseq ? offsets[nseq] : T;
    lo = lo < 0 ? 0 : (lo > T ? T : lo);
    hi = hi < lo ? lo : (hi > T ? T : hi);
    return {lo, hi};
}

// Zero the tokens of a packed row that belong to no sequence; without sequences,
// every token of every row.
template <int N>
struct GapArgs {
    View v[N];
    int H[N], D[N];
    int n;
    const int32_t* offsets;
    int nseq;
    int64_t B, T;
};

template <int N>
__global__ void __launch_bounds__(256) gap_kernel(const GapArgs<N> a) {
    const auto [lo, hi] = covered(a.offsets, a.nseq, a.T);
    const int64_t tokens = lo + a.T - hi;
    for (int i = 0; i < a.n; ++i) {
        const int64_t per = int64_t(a.H[i]) * a.D[i], row = tokens * per, n = a.B * row;
        for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < n; e += int64_t(gridDim.x) * 256) {
            const int64_t b = e / row, t = (e - b * row) / per, r = e - b * row - t * per;
            reinterpret_cast<uint16_t*>(a.v[i].p)[b * a.v[i].b + (t < lo ? t : hi + t - lo) * a.v[i].t + r / a.D[i] * a.v[i].h +
                                                  r % a.D[i]] = 0;
        }
    }
}

// dq, dk [token][Hk][DK] = the sum over a key head's value heads, 8 features a thread, in the
// heads' order.  With offsets the tokens of no sequence are left out: no part of theirs is
// formed, and gap_kernel has zeroed them.  Bound: HBM (16 x 1000 tokens, 12 heads over 6
// of 64: 123 MB in 22 us, 5.5 TB/s).
template <int DT>
__global__ void __launch_bounds__(256) head_sum_kernel(const float* xq, const float* xk, View yq, View yk, int64_t tokens,
                                                       int64_t T, int Hk, int group, int DK, const int32_t* offsets,
                                                       int nseq) {
    const Covered in = offsets ? covered(offsets, nseq, T) : Covered{0, T};
    const int np = DK / 8;
    const int64_t n = tokens * Hk * np * 2;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < n; e += int64_t(gridDim.x) * 256) {
        const int64_t e2 = e >> 1;
        const float* x = e & 1 ? xk : xq;
        const View& y = e & 1 ? yk : yq;
        const int r = int(e2 % np) * 8;
        const int64_t hk = (e2 / np) % Hk, tok = e2 / np / Hk, b = tok / T, t = tok - b * T;
        if (t < in.lo || t >= in.hi) continue;
        float4 u = make_float4(0, 0, 0, 0), v = u;
        for (int j = 0; j < group; ++j) {
            const float* q = x + ((tok * Hk + hk) * group + j) * DK + r;
            const float4 s = *reinterpret_cast<const float4*>(q), z = *reinterpret_cast<const float4*>(q + 4);
            u.x += s.x; u.y += s.y; u.z += s.z; u.w += s.w;
            v.x += z.x; v.y += z.y; v.z += z.z; v.w += z.w;
        }
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y.p) + b * y.b + t * y.t + hk * y.h + r) =
            make_uint4(Op<DT>::pack(u.x, u.y), Op<DT>::pack(u.z, u.w), Op<DT>::pack(v.x, v.y), Op<DT>::pack(v.z, v.w));
    }
}

}  // namespace
}  // namespace fftconv
