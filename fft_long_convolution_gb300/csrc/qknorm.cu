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
// A group takes HB consecutive heads of its token at once, so HB (times two in
// the backward) loads are in flight before the first is used and the token's
// cos and sin are read once for all of them.
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
    int64_t T, tokens, items;
    int Hq, Hk, D, R, inter;
    int nbq, nbk;  // blocks of HB heads of q and of k per token
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

// The cos and sin that belong to a lane's 8 features: feature j < R turns with
// entry j mod (R/2) (halves) or j / 2 (interleaved).  Features at R or beyond
// get (1, 0).
__device__ __forceinline__ void load_turn(const NormArgs& a, int64_t p, int d0, float (&c)[8], float (&s)[8]) {
    const int half = a.R >> 1;
    const float *cp = a.cos + p * half, *sp = a.sin + p * half;
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int d = d0 + j, i = a.inter ? d >> 1 : (d < half ? d : d - half);
        const bool on = d < a.R;
        c[j] = on ? __ldg(cp + i) : 1.0f;
        s[j] = on ? __ldg(sp + i) : 0.0f;
    }
}

// Rotate a row spread over the group's lanes; dir = +1 forward, -1 inverse.
// MODE 1: pairs are neighbours in the lane; 2: halves whose distance R/2 is a
// multiple of 8 (the partner sits in one other lane); 3: other halves, through
// the group's row buffer in shared memory.
template <int G, int MODE>
__device__ __forceinline__ void turn(float (&z)[8], const float (&c)[8], const float (&s)[8], float dir, int lane,
                                     int R, float* row, unsigned mask) {
    if constexpr (MODE == 1) {
        #pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float x = z[j], y = z[j + 1], sj = dir * s[j];
            z[j] = x * c[j] - y * sj;
            z[j + 1] = y * c[j] + x * sj;
        }
    } else {
        const int half = R >> 1;
        float o[8];
        if constexpr (MODE == 2) {
            const int step = half >> 3;
            const bool low = lane < step;
            const int other = lane < 2 * step ? (low ? lane + step : lane - step) : lane;
            #pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __shfl_sync(mask, z[j], other, G);
            const float sg = low ? -dir : dir;
            #pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = z[j] * c[j] + sg * o[j] * s[j];
        } else {
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
        }
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float v, unsigned mask) {
    #pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(mask, v, o, G);
    return v;
}

// MODE 0: no rotation; 1, 2, 3 as turn().
template <int DT, int G, int HB, int MODE, bool BWD>
__global__ void __launch_bounds__(kThreads) qknorm_kernel(const NormArgs a) {
    __shared__ float rows[MODE == 3 ? kThreads / G : 1][MODE == 3 ? 8 * G : 1];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int d0 = lane * 8;
    const bool on = d0 < a.D;
    const unsigned mask = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << ((threadIdx.x % 32) / G * G);
    constexpr int NG = kThreads / G;
    const int nb = a.nbq + a.nbk;
    float acc[BWD ? 2 : 1][8] = {};  // weight gradients of this lane's features, q and k
    for (int64_t it = int64_t(blockIdx.x) * NG + grp; it < a.items; it += int64_t(gridDim.x) * NG) {
        const int64_t tok = it / nb;
        const int blk = int(it - tok * nb);
        const bool isk = blk >= a.nbq;
        const int h0 = (isk ? blk - a.nbq : blk) * HB, H = isk ? a.Hk : a.Hq;
        const int64_t b = tok / a.T, t = tok - b * a.T;
        const View& vx = isk ? a.k : a.q;
        const View& vy = isk ? a.yk : a.yq;
        const uint16_t* px = reinterpret_cast<const uint16_t*>(vx.p) + b * vx.b + t * vx.t + d0;
        uint16_t* py = reinterpret_cast<uint16_t*>(vy.p) + b * vy.b + t * vy.t + d0;
        uint4 ux[HB], ud[BWD ? HB : 1];
        #pragma unroll
        for (int i = 0; i < HB; ++i)
            ux[i] = on && h0 + i < H ? *reinterpret_cast<const uint4*>(px + (h0 + i) * vx.h) : make_uint4(0, 0, 0, 0);
        if constexpr (BWD) {
            const View& vd = isk ? a.dyk : a.dyq;
            const uint16_t* pd = reinterpret_cast<const uint16_t*>(vd.p) + b * vd.b + t * vd.t + d0;
            #pragma unroll
            for (int i = 0; i < HB; ++i)
                ud[i] = on && h0 + i < H ? *reinterpret_cast<const uint4*>(pd + (h0 + i) * vd.h) : make_uint4(0, 0, 0, 0);
        }
        float c[8], s[8];
        bool lost = false;
        if constexpr (MODE != 0) {
            const int64_t p = a.pos ? a.pos[tok] : t;
            lost = p < 0 || p >= a.rows;
            load_turn(a, lost ? 0 : p, d0, c, s);
        }
        const float* wp = isk ? a.wk : a.wq;
        float w[8];
        #pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = wp && on ? __ldg(wp + d0 + j) : 1.0f;
        #pragma unroll
        for (int i = 0; i < HB; ++i) {
            if (h0 + i >= H) break;  // the same for every lane of the group
            float x[8], z[8];
            unpack8<DT>(ux[i], x);
            float ss = 0.0f;
            #pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            ss = group_sum<G>(ss, mask);
            const float r = rsqrtf(fmaf(a.c, ss, a.eps));
            if constexpr (!BWD) {
                #pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = x[j] * r * w[j];
                if constexpr (MODE != 0) turn<G, MODE>(z, c, s, 1.0f, lane, a.R, rows[grp], mask);
            } else {
                unpack8<DT>(ud[i], z);
                if constexpr (MODE != 0) turn<G, MODE>(z, c, s, -1.0f, lane, a.R, rows[grp], mask);
                float dot = 0.0f;
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float g = z[j] * x[j] * r;
                    if (isk) acc[1][j] += g;
                    else acc[0][j] += g;
                    z[j] *= w[j];
                    dot = fmaf(z[j], x[j], dot);
                }
                dot = group_sum<G>(dot, mask) * a.c * r * r;
                #pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = r * fmaf(-dot, x[j], z[j]);
            }
            if (lost) {
                #pragma unroll
                for (int j = 0; j < 8; ++j) z[j] = CUDART_NAN_F;
            }
            if (on) *reinterpret_cast<uint4*>(py + (h0 + i) * vy.h) = pack8<DT>(z);
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
            for (int j = 0; j < 8; ++j) red[grp][d0 + j] = acc[m][j];
            __syncthreads();
            for (int d = threadIdx.x; d < a.D; d += kThreads) {
                float v = 0.0f;
                for (int g = 0; g < NG; ++g) v += red[g][d];
                a.part[(int64_t(blockIdx.x) * 2 + m) * a.D + d] = v;
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
void launch_mode(const NormArgs& a, int mode, int grid, cudaStream_t st) {
    switch (mode) {
        case 0: qknorm_kernel<DT, G, HB, 0, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 1: qknorm_kernel<DT, G, HB, 1, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 2: qknorm_kernel<DT, G, HB, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        default: qknorm_kernel<DT, G, HB, 3, BWD><<<grid, kThreads, 0, st>>>(a); break;
    }
}

template <int DT, bool BWD>
void launch_dt(const NormArgs& a, int mode, int G, int HB, int grid, cudaStream_t st) {
    if (HB == 1) {
        if (G == 8) launch_mode<DT, 8, 1, BWD>(a, mode, grid, st);
        else if (G == 16) launch_mode<DT, 16, 1, BWD>(a, mode, grid, st);
        else launch_mode<DT, 32, 1, BWD>(a, mode, grid, st);
    } else {
        if (G == 8) launch_mode<DT, 8, 3, BWD>(a, mode, grid, st);
        else if (G == 16) launch_mode<DT, 16, 3, BWD>(a, mode, grid, st);
        else launch_mode<DT, 32, 3, BWD>(a, mode, grid, st);
    }
}

constexpr int kMaxGrid = 152 * 8;  // CTAs of the persistent grid; bounds the partial sums

fftconv_status_t check_args(const fftconv_qknorm_args_t* p) {
    if (!p) return FFTCONV_ERR_INVALID;
    if (p->B < 0 || p->T < 0 || p->Hq < 0 || p->Hk < 0 || !(p->eps >= 0.0f)) return FFTCONV_ERR_INVALID;
    if (p->dtype != FFTCONV_F16 && p->dtype != FFTCONV_BF16) return FFTCONV_ERR_UNSUPPORTED;
    if (p->norm != FFTCONV_NORM_RMS && p->norm != FFTCONV_NORM_L2) return FFTCONV_ERR_UNSUPPORTED;
    if (p->D < 8 || p->D > 256 || p->D % 8 || p->R < 0 || p->R > p->D || p->R % 2) return FFTCONV_ERR_UNSUPPORTED;
    if (p->Hq > 65535 || p->Hk > 65535 || p->T > (int64_t(1) << 40) || p->B > (int64_t(1) << 40) ||
        (p->T && p->B > (int64_t(1) << 40) / p->T))
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
    Span outs[4] = {}, ins[9] = {};
    int no = 0, ni = 0;
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        if ((e = take_view(*xs[i], p->B, p->T, heads[i], p->D, vx[i])) != FFTCONV_OK) return e;
        if ((e = take_view(y[i], p->B, p->T, heads[i], p->D, vy[i])) != FFTCONV_OK) return e;
        if (BWD && (e = take_view(dy[i], p->B, p->T, heads[i], p->D, vd[i])) != FFTCONV_OK) return e;
    }
    for (int i = 0; i < 2; ++i) {
        if (!heads[i]) continue;
        const Span o = span_of(*vy[i], p->B, p->T, heads[i], p->D);
        // in place on its own input is fine (a lane reads its elements before it writes them)
        for (int j = 0; j < 2; ++j) {
            if (!heads[j]) continue;
            if (!(i == j && same_view(*vx[j], *vy[i])) && meets(o, span_of(*vx[j], p->B, p->T, heads[j], p->D))) {
                // heads of q and k may be interleaved slices of one buffer; two
                // slices updated in place never share an element
                const bool both = heads[0] && heads[1] && same_view(a.q, a.yq) && same_view(a.k, a.yk);
                if (!both) return FFTCONV_ERR_INVALID;
            }
            if (BWD && !(i == j && same_view(*vd[j], *vy[i])) &&
                meets(o, span_of(*vd[j], p->B, p->T, heads[j], p->D))) {
                const bool both = heads[0] && heads[1] && same_view(a.dyq, a.yq) && same_view(a.dyk, a.yk);
                if (!both) return FFTCONV_ERR_INVALID;
            }
        }
        outs[no++] = o;
    }
    const size_t wb = size_t(p->D) * 4, tb = size_t(p->table_rows) * (p->R / 2) * 4;
    ins[ni++] = span_of(p->wq, wb);
    ins[ni++] = span_of(p->wk, wb);
    if (p->R) {
        ins[ni++] = span_of(p->cos, tb);
        ins[ni++] = span_of(p->sin, tb);
        ins[ni++] = span_of(p->positions, size_t(tokens) * 4);
    }
    if (any_meet(outs, ins)) return FFTCONV_ERR_INVALID;
    a.wq = p->wq;
    a.wk = p->wk;
    a.cos = p->cos;
    a.sin = p->sin;
    a.pos = p->positions;
    a.rows = p->table_rows;
    a.T = p->T;
    a.tokens = tokens;
    a.Hq = int(p->Hq);
    a.Hk = int(p->Hk);
    a.D = p->D;
    a.R = p->R;
    a.inter = p->interleaved != 0;
    a.eps = p->eps;
    a.c = p->norm == FFTCONV_NORM_RMS ? 1.0f / float(p->D) : 1.0f;
    const int G = lanes_of(p->D);
    // Heads per group: three when the call still fills the GPU that way, else
    // one (more groups for calls of few tokens).
    const int64_t rows = tokens * (p->Hq + p->Hk);
    const int HB = rows * G >= int64_t(3) * 152 * 2048 ? 3 : 1;
    a.nbq = (a.Hq + HB - 1) / HB;
    a.nbk = (a.Hk + HB - 1) / HB;
    a.items = tokens * (a.nbq + a.nbk);
    const int64_t per = kThreads / G, need = (a.items + per - 1) / per;
    const int grid = int(need < kMaxGrid ? need : kMaxGrid);
    if (want) {
        if (!scratch || scratch_bytes < size_t(grid) * 2 * wb) return FFTCONV_ERR_WORKSPACE;
        if (off16(scratch)) return FFTCONV_ERR_ALIGN;
        a.part = static_cast<float*>(scratch);
    }
    int mode = 0;
    if (p->R) mode = a.inter ? 1 : ((p->R / 2) % 8 == 0 ? 2 : 3);
    if (p->dtype == FFTCONV_F16) launch_dt<0, BWD>(a, mode, G, HB, grid, st);
    else launch_dt<1, BWD>(a, mode, G, HB, grid, st);
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
