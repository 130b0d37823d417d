// Norm of queries and keys for each head with the position rotation in the
// same pass, and its gradients.
//
// Mathematics: r = rsqrt(c sum x^2 + eps) (c = 1/D or 1), z = x r w, y = the
// rotation of z's first R features.  Backward, with dz the inverse rotation of
// dy: dw = sum dz x r and dx = r (dz w) - x r^3 c sum_d(dz w x).
//
// Bound: one read of x (and dy) and one write of y (dx) per element against a
// handful of float32 operations, so HBM bandwidth for whole batches and launch
// latency for single tokens.  Split: a row (one head of one token) belongs to
// G = 8, 16 or 32 lanes that hold 8 consecutive features (one 16-byte load)
// each; the row's sums are shuffles within the group and nothing is staged.
// A group takes a token's heads three at a time, so three (six in the backward)
// loads are in flight before the first is used, the token's cos and sin are
// read once for all its heads, and the weights once for all tokens.
#include "views.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "mma.cuh"

namespace fftconv {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
    View q, k, dyq, dyk, yq, yk;  // forward: y; backward: dy in, y = dx
    const float *wq, *wk, *cos, *sin;
    const int32_t* pos;
    int64_t rows;  // table rows
    uint32_t T, items;
    int parts, per;  // a token's heads (q's, then k's) in parts of `per`; an item is a part
    int Hq, Hk, D, R;
    float eps, c;
    float* part;  // [grid][2][D] partial weight gradients, or null
};

template <int DT>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const cpx c = Op<DT>::unpack(w[i]);
        x[2 * i] = c.r;
        x[2 * i + 1] = c.i;
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(Op<DT>::pack(x[0], x[1]), Op<DT>::pack(x[2], x[3]), Op<DT>::pack(x[4], x[5]),
                      Op<DT>::pack(x[6], x[7]));
}

// A lane's 8 features are two runs of 4, at d[0] and d[1].  With halves that
// rotate against each other (MODE 2, R a multiple of 8) the first R / 8 lanes
// hold features 4 l .. and R/2 + 4 l .., so that every pair sits in one lane;
// otherwise a lane holds 8 consecutive features.
template <int MODE>
__device__ __forceinline__ void features(int lane, int R, int (&d)[2]) {
    const bool halves = MODE == 2 && lane * 8 < R;
    d[0] = halves ? lane * 4 : lane * 8;
    d[1] = halves ? R / 2 + lane * 4 : lane * 8 + 4;
}

template <int MODE>
__device__ __forceinline__ uint4 load_row(const uint16_t* p, const int (&d)[2]) {
    if constexpr (MODE == 2) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + d[0]), b = *reinterpret_cast<const uint2*>(p + d[1]);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    return *reinterpret_cast<const uint4*>(p + d[0]);
}

template <int MODE>
__device__ __forceinline__ void store_row(uint16_t* p, const int (&d)[2], const uint4& v) {
    if constexpr (MODE == 2) {
        *reinterpret_cast<uint2*>(p + d[0]) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(p + d[1]) = make_uint2(v.z, v.w);
    } else {
        *reinterpret_cast<uint4*>(p + d[0]) = v;
    }
}

// 4 consecutive floats, by one 16-byte load where VEC.
template <bool VEC>
__device__ __forceinline__ void load4(const float* p, float* x) {
    if constexpr (VEC) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p));
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __ldg(p + j);
    }
}

// The cos and sin of a lane's features: one entry per pair (MODE 1, 2) or per
// feature (MODE 3).  Features at R or beyond get (1, 0).
template <int MODE, bool VEC, int N>
__device__ __forceinline__ void load_turn(const NormArgs& a, int64_t p, int lane, float (&c)[N], float (&s)[N]) {
    const int half = a.R >> 1;
    const float *cp = a.cos + p * half, *sp = a.sin + p * half;
    #pragma unroll
    for (int j = 0; j < N; ++j) {
        c[j] = 1.0f;
        s[j] = 0.0f;
    }
    if constexpr (MODE == 3) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = lane * 8 + j, i = d < half ? d : d - half;
            if (d < a.R) {
                c[j] = __ldg(cp + i);
                s[j] = __ldg(sp + i);
            }
        }
    } else {
        const int i = lane * 4;  // the lane's first pair
        if (MODE == 2 || VEC) {
            if (i + 4 <= half) {
                load4<VEC>(cp + i, c);
                load4<VEC>(sp + i, s);
            }
        } else {
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (i + j < half) {
                    c[j] = __ldg(cp + i + j);
                    s[j] = __ldg(sp + i + j);
                }
            }
        }
    }
}

// Rotate a row spread over the group's lanes; dir = +1 forward, -1 inverse.
// MODE 1: pairs are neighbours; 2: pairs are features j and 4 + j of a lane; 3:
// halves of another length, through the group's row buffer in shared memory.
// Features at R or beyond are not mixed: turned by (1, 0), a NaN or an infinity in
// one would reach another, so the other's part is dropped, not multiplied by 0 (8 x
// 16384 tokens of 12 heads of 128: forward 153 us, 151 by multiplying; choosing
// between the results took 177).
// WHOLE: R is a multiple of 8, so a lane's pairs are all rotated or none.
template <int MODE, bool WHOLE, int N>
__device__ __forceinline__ void turn(float (&z)[8], const float (&c)[N], const float (&s)[N], float dir, int lane, int R,
                                     float* row, unsigned mask) {
    if constexpr (MODE == 3) {
        const int half = R >> 1;
        #pragma unroll
        for (int j = 0; j < 8; ++j) row[lane * 8 + j] = z[j];
        __syncwarp(mask);
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int d = lane * 8 + j;
            if (d < R) {
                const bool low = d < half;
                z[j] = z[j] * c[j] + (low ? -dir : dir) * row[low ? d + half : d - half] * s[j];
            }
        }
        __syncwarp(mask);
    } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = lane * 8 + (MODE == 1 && !WHOLE ? 2 * j : 0) < R;
            float &x = z[MODE == 1 ? 2 * j : j], &y = z[MODE == 1 ? 2 * j + 1 : j + 4];
            const float u = x, v = y, sj = dir * s[j];
            x = u * c[j] - (on ? v : 0.0f) * sj;
            y = v * c[j] + (on ? u : 0.0f) * sj;
        }
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
    #pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o, G);
    return v;
}

// MODE 0: no rotation; 1, 2, 3 as turn().  HB: heads taken at a time.  VEC:
// weights and tables by 16-byte loads (R a multiple of 8).
template <int DT, int G, int HB, int MODE, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) qknorm_kernel(const NormArgs a) {
    __shared__ float rows[MODE == 3 ? kThreads / G : 1][MODE == 3 ? 8 * G : 1];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const bool on = lane * 8 < a.D;
    int d[2];
    features<MODE>(lane, a.R, d);
    const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << ((threadIdx.x % 32) / G * G);
    constexpr int NG = kThreads / G;
    float w[2][8];
    #pragma unroll
    for (int m = 0; m < 2; ++m) {
        const float* p = m ? a.wk : a.wq;
        #pragma unroll
        for (int j = 0; j < 8; ++j) w[m][j] = 1.0f;
        if (p && on) {
            load4<VEC>(p + d[0], w[m]);
            load4<VEC>(p + d[1], w[m] + 4);
        }
    }
    float acc[BWD ? 2 : 1][8] = {};  // weight gradients of this lane's features, q and k
    constexpr int NT = MODE == 3 ? 8 : 4;
    for (uint32_t it = blockIdx.x * NG + grp; it < a.items; it += gridDim.x * NG) {
        const uint32_t tok = it / uint32_t(a.parts);
        const int lo = int(it - tok * a.parts) * a.per, hi = min(lo + a.per, a.Hq + a.Hk);
        const int64_t b = tok / a.T, t = tok - uint32_t(b) * a.T;
        float c[NT], s[NT];
        bool lost = false;
        if constexpr (MODE != 0) {
            const int64_t p = a.pos ? a.pos[tok] : t;
            lost = p < 0 || p >= a.rows;
            load_turn<MODE, VEC>(a, lost ? 0 : p, lane, c, s);
        }
        #pragma unroll
        for (int m = 0; m < 2; ++m) {
            const View& vx = m ? a.k : a.q;
            const View& vy = m ? a.yk : a.yq;
            const View& vd = m ? a.dyk : a.dyq;
            const int first = m ? max(lo - a.Hq, 0) : lo, end = m ? hi - a.Hq : min(hi, a.Hq);
            if (first >= end) continue;
            const uint16_t* px = reinterpret_cast<const uint16_t*>(vx.p) + b * vx.b + t * vx.t;
            uint16_t* py = reinterpret_cast<uint16_t*>(vy.p) + b * vy.b + t * vy.t;
            const uint16_t* pd = BWD ? reinterpret_cast<const uint16_t*>(vd.p) + b * vd.b + t * vd.t : nullptr;
            for (int h0 = first; h0 < end; h0 += HB) {
                uint4 ux[HB], ud[BWD ? HB : 1];
                #pragma unroll
                for (int i = 0; i < HB; ++i) {
                    const bool in = on && h0 + i < end;
                    ux[i] = in ? load_row<MODE>(px + (h0 + i) * vx.h, d) : make_uint4(0, 0, 0, 0);
                    if constexpr (BWD) ud[i] = in ? load_row<MODE>(pd + (h0 + i) * vd.h, d) : make_uint4(0, 0, 0, 0);
                }
                #pragma unroll
                for (int i = 0; i < HB; ++i) {
                    if (h0 + i >= end) break;  // the same for every lane of the group
                    float x[8], z[8];
                    unpack8<DT>(ux[i], x);
                    float ss = 0.0f;
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                    ss = group_sum<G>(ss, mask);
                    const float r = rsqrtf(fmaf(a.c, ss, a.eps));
                    if constexpr (!BWD) {
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = x[j] * r * w[m][j];
                        if constexpr (MODE != 0) turn<MODE, VEC>(z, c, s, 1.0f, lane, a.R, rows[grp], mask);
                    } else {
                        unpack8<DT>(ud[i], z);
                        if constexpr (MODE != 0) turn<MODE, VEC>(z, c, s, -1.0f, lane, a.R, rows[grp], mask);
                        float dot = 0.0f;
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            acc[m][j] = fmaf(z[j] * r, x[j], acc[m][j]);
                            z[j] *= w[m][j];
                            dot = fmaf(z[j], x[j], dot);
                        }
                        dot = group_sum<G>(dot, mask) * a.c * r * r;
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = r * fmaf(-dot, x[j], z[j]);
                    }
                    if (lost) {  // the weights' gradients are sums over it, too
                        #pragma unroll
                        for (int j = 0; j < 8; ++j) z[j] = CUDART_NAN_F;
                        if constexpr (BWD) {
                            #pragma unroll
                            for (int j = 0; j < 8; ++j) acc[m][j] = CUDART_NAN_F;
                        }
                    }
                    if (on) store_row<MODE>(py + (h0 + i) * vy.h, d, pack8<DT>(z));
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        // the groups' sums, in the order of the groups
        __shared__ float red[NG][8 * G];
        #pragma unroll
        for (int m = 0; m < 2; ++m) {
            __syncthreads();
            #pragma unroll
            for (int j = 0; j < 8; ++j) red[grp][on ? d[j >> 2] + (j & 3) : lane * 8 + j] = acc[m][j];
            __syncthreads();
            for (int f = threadIdx.x; f < a.D; f += kThreads) {
                float v = 0.0f;
                for (int g = 0; g < NG; ++g) v += red[g][f];
                a.part[(int64_t(blockIdx.x) * 2 + m) * a.D + f] = v;
            }
        }
    }
}

// dw[d] = sum over the CTAs' partials, in a fixed order: a warp per feature.
__global__ void __launch_bounds__(kThreads) qknorm_dw_kernel(const float* part, int n, int D, float* dwq, float* dwk) {
    const int i = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (i >= 2 * D) return;
    float* out = i < D ? dwq : dwk;
    if (!out) return;
    float v = 0.0f;
    for (int g = lane; g < n; g += 32) v += part[int64_t(g) * 2 * D + i];
    v = group_sum<32>(v, 0xffffffffu);
    if (lane == 0) out[i < D ? i : i - D] = v;
}

int lanes_of(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

template <int DT, int G, int HB, bool BWD>
void launch_mode(const NormArgs& a, int mode, bool vec, int grid, cudaStream_t st) {
    switch (mode) {
        case 0:
            if (vec) qknorm_kernel<DT, G, HB, 0, true, BWD><<<grid, kThreads, 0, st>>>(a);
            else qknorm_kernel<DT, G, HB, 0, false, BWD><<<grid, kThreads, 0, st>>>(a);
            break;
        case 1:
            if (vec) qknorm_kernel<DT, G, HB, 1, true, BWD><<<grid, kThreads, 0, st>>>(a);
            else qknorm_kernel<DT, G, HB, 1, false, BWD><<<grid, kThreads, 0, st>>>(a);
            break;
        case 2:
            if (vec) qknorm_kernel<DT, G, HB, 2, true, BWD><<<grid, kThreads, 0, st>>>(a);
            else qknorm_kernel<DT, G, HB, 2, false, BWD><<<grid, kThreads, 0, st>>>(a);
            break;
        default: qknorm_kernel<DT, G, HB, 3, false, BWD><<<grid, kThreads, 0, st>>>(a); break;
    }
}

template <int DT, bool BWD>
void launch_dt(const NormArgs& a, int mode, bool vec, int G, int HB, int grid, cudaStream_t st) {
    if (HB == 1) {
        if (G == 8) launch_mode<DT, 8, 1, BWD>(a, mode, vec, grid, st);
        else if (G == 16) launch_mode<DT, 16, 1, BWD>(a, mode, vec, grid, st);
        else launch_mode<DT, 32, 1, BWD>(a, mode, vec, grid, st);
    } else {
        if (G == 8) launch_mode<DT, 8, 3, BWD>(a, mode, vec, grid, st);
        else if (G == 16) launch_mode<DT, 16, 3, BWD>(a, mode, vec, grid, st);
        else launch_mode<DT, 32, 3, BWD>(a, mode, vec, grid, st);
    }
}

// CTAs at most.  The forward takes a CTA per few tokens (8 x 16384 tokens of
// 12 heads of 128: 153 us, 5.3 TB/s; a resident grid that fetches ahead took
// 225 us); the backward keeps its grid small, as each CTA leaves a partial sum of
// the weights' gradients (240 us, 5.0 TB/s).
constexpr int kMaxGrid = 152 * 4, kMaxGridForward = 1 << 24;

fftconv_status_t check_args(const fftconv_qknorm_args_t* p) {
    if (!p) return FFTCONV_ERR_INVALID;
    if (p->B < 0 || p->T < 0 || p->Hq < 0 || p->Hk < 0 || !(p->eps >= 0.0f)) return FFTCONV_ERR_INVALID;
    if (p->dtype != FFTCONV_F16 && p->dtype != FFTCONV_BF16) return FFTCONV_ERR_UNSUPPORTED;
    if (p->norm != FFTCONV_NORM_RMS && p->norm != FFTCONV_NORM_L2) return FFTCONV_ERR_UNSUPPORTED;
    if (p->D < 8 || p->D > 256 || p->D % 8 || p->R < 0 || p->R > p->D || p->R % 2) return FFTCONV_ERR_UNSUPPORTED;
    // items and two steps of the grid beyond them in 32 bits
    if (p->Hq > 1023 || p->Hk > 1023 || p->T >= (int64_t(1) << 30) || (p->T && p->B >= (int64_t(1) << 30) / p->T))
        return FFTCONV_ERR_UNSUPPORTED;
    if (p->R && (!p->cos || !p->sin || p->table_rows < 1)) return FFTCONV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(p->cos) | reinterpret_cast<uintptr_t>(p->sin) |
         reinterpret_cast<uintptr_t>(p->wq) | reinterpret_cast<uintptr_t>(p->wk) |
         reinterpret_cast<uintptr_t>(p->positions)) & 3)
        return FFTCONV_ERR_ALIGN;
    return FFTCONV_OK;
}

bool same_view(const View& a, const View& b) { return a.p == b.p && a.b == b.b && a.t == b.t && a.h == b.h; }

// Shared by both directions: fills the kernel arguments and launches.
template <bool BWD>
fftconv_status_t run(const fftconv_qknorm_args_t* p, const fftconv_view_t* dy, const fftconv_view_t* y, float* dwq,
                     float* dwk, void* scratch, size_t scratch_bytes, fftconv_stream_t stream) {
    fftconv_status_t e = check_args(p);
    if (e != FFTCONV_OK) return e;
    if ((reinterpret_cast<uintptr_t>(dwq) | reinterpret_cast<uintptr_t>(dwk)) & 3) return FFTCONV_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t tokens = p->B * p->T;
    const bool want = BWD && (dwq || dwk);
    if (tokens == 0 || p->Hq + p->Hk == 0) {
        if (dwq && cudaMemsetAsync(dwq, 0, size_t(p->D) * 4, st) != cudaSuccess) return FFTCONV_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, size_t(p->D) * 4, st) != cudaSuccess) return FFTCONV_ERR_CUDA;
        return FFTCONV_OK;
    }
    NormArgs a{};
    const int64_t heads[2] = {p->Hq, p->Hk};
    const fftconv_view_t* xs[2] = {&p->q, &p->k};
    View *vx[2] = {&a.q, &a.k}, *vd[2] = {&a.dyq, &a.dyk}, *vy[2] = {&a.yq, &a.yk};
    // two outputs, both weights' gradients, scratch; inputs and given gradients, weights, tables, positions
    Span outs[5] = {}, ins[9] = {};
    int no = 0, ni = 0;
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        if ((e = take_view(*xs[i], p->B, p->T, heads[i], p->D, vx[i])) != FFTCONV_OK) return e;
        if ((e = take_view(y[i], p->B, p->T, heads[i], p->D, vy[i])) != FFTCONV_OK) return e;
        if (BWD && (e = take_view(dy[i], p->B, p->T, heads[i], p->D, vd[i])) != FFTCONV_OK) return e;
    }
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        // in place on its own input is fine (a lane reads its elements before it writes them)
        for (int j = 0; j < 2; ++j) {
            if (!heads[j]) continue;
            for (const View* x : {vx[j], vd[j]}) {
                if (!x->p || (i == j && same_view(*x, *vy[i]))) continue;
                if (share(*x, heads[j], *vy[i], heads[i], p->B, p->T, p->D)) return FFTCONV_ERR_INVALID;
            }
        }
        outs[no++] = span_of(*vy[i], p->B, p->T, heads[i], p->D);
    }
    if (heads[0] && heads[1] && share(a.yq, heads[0], a.yk, heads[1], p->B, p->T, p->D)) return FFTCONV_ERR_INVALID;
    const size_t wb = size_t(p->D) * 4, tb = size_t(p->table_rows) * (p->R / 2) * 4;
    ins[ni++] = span_of(p->wq, wb);
    ins[ni++] = span_of(p->wk, wb);
    if (p->R) {
        ins[ni++] = span_of(p->cos, tb);
        ins[ni++] = span_of(p->sin, tb);
        ins[ni++] = span_of(p->positions, size_t(tokens) * 4);
    }
    if (any_meet(outs, ins)) return FFTCONV_ERR_INVALID;
    const int first = no;
    outs[no++] = span_of(dwq, wb);
    outs[no++] = span_of(dwk, wb);
    for (int j = 0; j < 2; ++j) {
        if (vx[j]->p) ins[ni++] = span_of(*vx[j], p->B, p->T, heads[j], p->D);
        if (vd[j]->p) ins[ni++] = span_of(*vd[j], p->B, p->T, heads[j], p->D);
    }
    a.wq = p->wq;
    a.wk = p->wk;
    a.cos = p->cos;
    a.sin = p->sin;
    a.pos = p->positions;
    a.rows = p->table_rows;
    a.T = uint32_t(p->T);
    a.Hq = int(p->Hq);
    a.Hk = int(p->Hk);
    a.D = p->D;
    a.R = p->R;
    a.eps = p->eps;
    a.c = p->norm == FFTCONV_NORM_RMS ? 1.0f / float(p->D) : 1.0f;
    const int G = lanes_of(p->D);
    // As few parts of a token's heads as fill a quarter of the GPU's threads: one for
    // whole batches, one per head for single tokens.  A part waits for the weights, the
    // position and its table rows before its first row: 8 x 4096 tokens of 18 heads of
    // 64 in three parts took 1.45 times as long as in one (30.0 us); 5115 tokens of 12
    // heads of 80 in six parts 1.3 times as long as in one (8.9 us).
    const int total = a.Hq + a.Hk;
    const int64_t want_parts = (int64_t(1) * 152 * 512 + tokens * G - 1) / (tokens * G);
    a.per = int((total + want_parts - 1) / want_parts);
    a.parts = (total + a.per - 1) / a.per;
    a.items = uint32_t(tokens * a.parts);
    const int HB = a.per > 1 ? 3 : 1;
    const int64_t per = kThreads / G, need = (a.items + per - 1) / per;
    const int most = BWD ? kMaxGrid : kMaxGridForward;
    const int grid = int(need < most ? need : most);
    if (want) {
        if (!scratch || scratch_bytes < size_t(grid) * 2 * wb) return FFTCONV_ERR_WORKSPACE;
        if (off16(scratch)) return FFTCONV_ERR_ALIGN;
        a.part = static_cast<float*>(scratch);
        outs[no++] = span_of(scratch, size_t(grid) * 2 * wb);
    }
    for (int i = first; i < no; ++i) {
        for (const Span& x : ins)
            if (meets(outs[i], x)) return FFTCONV_ERR_INVALID;
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    }
    int mode = 0;
    if (p->R) mode = p->interleaved ? 1 : (p->R % 8 == 0 ? 2 : 3);
    // 16-byte loads of weights and tables: rows of tables start on 16 bytes when
    // R/2 is a multiple of 4
    const bool vec = !(off16(p->wq) || off16(p->wk) || (p->R && (off16(p->cos) || off16(p->sin) || p->R % 8)));
    if (p->dtype == FFTCONV_F16) launch_dt<0, BWD>(a, mode, vec, G, HB, grid, st);
    else launch_dt<1, BWD>(a, mode, vec, G, HB, grid, st);
    if (want) qknorm_dw_kernel<<<(2 * p->D + 7) / 8, kThreads, 0, st>>>(a.part, grid, p->D, dwq, dwk);
    return cudaGetLastError() == cudaSuccess ? FFTCONV_OK : FFTCONV_ERR_CUDA;
}

}  // namespace
}  // namespace fftconv

extern "C" fftconv_status_t fftconv_qknorm_forward(const fftconv_qknorm_args_t* args, fftconv_view_t yq,
                                                   fftconv_view_t yk, fftconv_stream_t stream) {
    const fftconv_view_t y[2] = {yq, yk};
    return fftconv::run<false>(args, nullptr, y, nullptr, nullptr, nullptr, 0, stream);
}

extern "C" size_t fftconv_qknorm_scratch_bytes(const fftconv_qknorm_args_t* args) {
    if (fftconv::check_args(args) != FFTCONV_OK) return 0;
    return size_t(fftconv::kMaxGrid) * 2 * size_t(args->D) * 4;
}

extern "C" fftconv_status_t fftconv_qknorm_backward(const fftconv_qknorm_args_t* args, fftconv_view_t dyq,
                                                    fftconv_view_t dyk, fftconv_view_t dq, fftconv_view_t dk,
                                                    float* dwq, float* dwk, void* scratch, size_t scratch_bytes,
                                                    fftconv_stream_t stream) {
    const fftconv_view_t dy[2] = {dyq, dyk}, y[2] = {dq, dk};
    return fftconv::run<true>(args, dy, y, dwq, dwk, scratch, scratch_bytes, stream);
}
