// Layer norm of rows of features, and its gradients.
//
// Mathematics: m = mean x, r = rsqrt(mean (x - m)^2 + eps), h = (x - m) r,
// y = h w + b.  Backward, with dz = dy w: dx = r (dz - mean dz - h mean(dz h)),
// dw = sum dy h and db = sum dy over all tokens.  The variance is taken from the
// differences to the mean, so a mean that is large against the spread costs nothing.
//
// Bound: one read of x (and dy) and one write of y (dx) per element, so HBM
// bandwidth for whole batches and launch latency for single tokens.  Split: a row
// belongs to G lanes that hold NV runs of 8 consecutive features (a 16-byte load
// each): whole rows stay in registers, so nothing is read twice.  Up to 1024
// features G is at most a warp and the row's sums are shuffles; wider rows take a
// CTA, whose warps' sums meet in shared memory.  A group takes RB rows at a time:
// their loads are in flight together and their sums share the barriers.
#include "views.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mma.cuh"

namespace fftconv {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
    View x, dy, y;  // forward: y; backward: dy in, y = dx
    const float *w, *b;
    uint32_t T, rows;  // rows of one head
    int H, D, parts;   // CTAs that share a head
    bool vec;          // weights by 16-byte loads
    float eps, c;      // c = 1 / D
    float* part;       // [parts][2][H][D] partial weight gradients, or null
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

__device__ __forceinline__ void load8(const float* p, bool vec, float (&x)[8]) {
    if (vec) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p)), v = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
    } else {
        #pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __ldg(p + j);
    }
}

// The sums of N values over a row's G lanes, in every lane.
template <int G, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[8]) {
    #pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
        #pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (G > 32) {
        static_assert(G == kThreads, "a row takes the CTA");
        __syncthreads();  // the last sums have been read
        if (threadIdx.x % 32 == 0)
            #pragma unroll
            for (int i = 0; i < N; ++i) red[i][threadIdx.x / 32] = v[i];
        __syncthreads();
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4 a = *reinterpret_cast<const float4*>(red[i]), b = *reinterpret_cast<const float4*>(red[i] + 4);
            v[i] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
        }
    }
}

template <int DT, int G, int NV, int RB, bool BWD>
__global__ void __launch_bounds__(kThreads) layernorm_kernel(const NormArgs a) {
    constexpr int NG = kThreads / G;
    __shared__ __align__(16) float red[G > 32 ? 2 * RB : 1][8];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int h = blockIdx.x % a.H, part = blockIdx.x / a.H;
    int f[NV];
    bool on[NV];
    float w[NV][8], b[BWD ? 1 : NV][8];
    #pragma unroll
    for (int v = 0; v < NV; ++v) {
        f[v] = (v * G + lane) * 8;
        on[v] = f[v] < a.D;
        #pragma unroll
        for (int j = 0; j < 8; ++j) w[v][j] = 1.0f;
        if (a.w && on[v]) load8(a.w + int64_t(h) * a.D + f[v], a.vec, w[v]);
        if constexpr (!BWD) {
            #pragma unroll
            for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
            if (a.b && on[v]) load8(a.b + int64_t(h) * a.D + f[v], a.vec, b[v]);
        }
    }
    float aw[BWD ? NV : 1][8] = {}, ab[BWD ? NV : 1][8] = {};
    for (uint32_t base = uint32_t(part) * (NG * RB); base < a.rows; base += uint32_t(a.parts) * (NG * RB)) {
        uint4 ux[RB][NV], ud[BWD ? RB : 1][NV];
        int64_t yo[RB];
        bool live[RB];
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            const uint32_t r = base + i * NG + grp;
            live[i] = r < a.rows;
            const uint32_t bi = live[i] ? r / a.T : 0;
            const int64_t t = live[i] ? r - bi * a.T : 0;
            const uint16_t* px = reinterpret_cast<const uint16_t*>(a.x.p) + bi * a.x.b + t * a.x.t + h * a.x.h;
            const uint16_t* pd = BWD ? reinterpret_cast<const uint16_t*>(a.dy.p) + bi * a.dy.b + t * a.dy.t + h * a.dy.h : nullptr;
            yo[i] = bi * a.y.b + t * a.y.t + h * a.y.h;
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                ux[i][v] = live[i] && on[v] ? *reinterpret_cast<const uint4*>(px + f[v]) : make_uint4(0, 0, 0, 0);
                if constexpr (BWD) ud[i][v] = live[i] && on[v] ? *reinterpret_cast<const uint4*>(pd + f[v]) : make_uint4(0, 0, 0, 0);
            }
        }
        float s[BWD ? 2 * RB : RB] = {};
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                float x[8];
                unpack8<DT>(ux[i][v], x);
                #pragma unroll
                for (int j = 0; j < 8; ++j) s[i] += x[j];
                if constexpr (BWD) {
                    unpack8<DT>(ud[i][v], x);
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) s[RB + i] = fmaf(x[j], w[v][j], s[RB + i]);
                }
            }
        }
        row_sums<G>(s, red);
        float q[BWD ? 2 * RB : RB] = {}, m[RB], mz[RB];
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            m[i] = s[i] / float(a.D);  // exact for rows of equal values, as their sums are
            if constexpr (BWD) mz[i] = s[RB + i] * a.c;
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!on[v]) continue;
                float x[8];
                unpack8<DT>(ux[i][v], x);
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    x[j] -= m[i];
                    q[i] = fmaf(x[j], x[j], q[i]);
                }
                if constexpr (BWD) {
                    float d[8];
                    unpack8<DT>(ud[i][v], d);
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) q[RB + i] = fmaf(d[j] * w[v][j], x[j], q[RB + i]);
                }
            }
        }
        row_sums<G>(q, red);
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            if (!live[i]) continue;
            const float r = rsqrtf(fmaf(q[i], a.c, a.eps));
            uint16_t* py = reinterpret_cast<uint16_t*>(a.y.p) + yo[i];
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!on[v]) continue;
                float x[8];
                unpack8<DT>(ux[i][v], x);
                if constexpr (!BWD) {
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = fmaf((x[j] - m[i]) * r, w[v][j], b[v][j]);
                } else {
                    const float mh = q[RB + i] * a.c * r;  // mean of dz h
                    float d[8];
                    unpack8<DT>(ud[i][v], d);
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float hh = (x[j] - m[i]) * r;
                        aw[v][j] = fmaf(d[j], hh, aw[v][j]);
                        ab[v][j] += d[j];
                        x[j] = r * (fmaf(d[j], w[v][j], -mz[i]) - hh * mh);
                    }
                }
                *reinterpret_cast<uint4*>(py + f[v]) = pack8<DT>(x);
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        const int64_t hd = int64_t(a.H) * a.D;
        float* out = a.part + (int64_t(part) * 2 * a.H + h) * a.D;
        if constexpr (NG == 1) {
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!on[v]) continue;
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    out[f[v] + j] = aw[v][j];
                    out[hd + f[v] + j] = ab[v][j];
                }
            }
        } else {
            // the groups' sums, in the order of the groups
            __shared__ float sums[NG][NV * G * 8];
            #pragma unroll
            for (int k = 0; k < 2; ++k) {
                __syncthreads();
                #pragma unroll
                for (int v = 0; v < NV; ++v)
                    #pragma unroll
                    for (int j = 0; j < 8; ++j) sums[grp][f[v] + j] = k ? ab[v][j] : aw[v][j];
                __syncthreads();
                for (int i = threadIdx.x; i < a.D; i += kThreads) {
                    float v = 0.0f;
                    for (int g = 0; g < NG; ++g) v += sums[g][i];
                    out[k * hd + i] = v;
                }
            }
        }
    }
}

// dw, db = the sums of the CTAs' partials, in a fixed order: a CTA per 32 of the
// 2 H D sums, its warps every 8th partial each.
__global__ void __launch_bounds__(kThreads) layernorm_sum_kernel(const float* part, int n, int64_t hd, float* dw, float* db) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t i = int64_t(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (i < 2 * hd)
        #pragma unroll 8
        for (int g = warp; g < n; g += 8) v += part[g * 2 * hd + i];
    sums[warp][lane] = v;
    __syncthreads();
    if (warp || i >= 2 * hd) return;
    #pragma unroll
    for (int k = 1; k < 8; ++k) v += sums[k][lane];
    float* out = i < hd ? dw : db;
    if (out) out[i < hd ? i : i - hd] = v;
}

// How a row of D features is held: G lanes of NV runs, RB rows at a time.
struct Shape {
    int G, NV, RB;
};

Shape shape_of(int D) {
    const int n = D / 8;
    if (n <= 4) return {4, 1, 4};
    if (n <= 8) return {8, 1, 4};
    if (n <= 16) return {16, 1, 4};
    if (n <= 128) return {32, (n + 31) / 32, n <= 32 ? 4 : (n <= 96 ? 2 : 1)};
    return {kThreads, (n + kThreads - 1) / kThreads, n <= 512 ? 2 : 1};
}

// CTAs that share a head in the backward, at most: each leaves a partial sum.
constexpr int kMaxGrid = 152 * 2;

int parts_of(const fftconv_layernorm_args_t* p, bool backward) {
    const Shape s = shape_of(p->D);
    const int64_t rows = p->B * p->T, per = int64_t(kThreads / s.G) * s.RB;
    const int64_t need = (rows + per - 1) / per;
    if (!backward) return int(need);
    const int64_t most = (kMaxGrid + p->H - 1) / p->H;
    return int(need < most ? need : most);
}

template <int DT, bool BWD>
void launch(const NormArgs& a, cudaStream_t st) {
    const Shape s = shape_of(a.D);
    const unsigned grid = unsigned(a.parts) * unsigned(a.H);
    switch (s.G) {
        case 4: layernorm_kernel<DT, 4, 1, 4, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 8: layernorm_kernel<DT, 8, 1, 4, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 16: layernorm_kernel<DT, 16, 1, 4, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 32:
            if (s.NV == 1) layernorm_kernel<DT, 32, 1, 4, BWD><<<grid, kThreads, 0, st>>>(a);
            else if (s.NV == 2) layernorm_kernel<DT, 32, 2, 2, BWD><<<grid, kThreads, 0, st>>>(a);
            else if (s.NV == 3) layernorm_kernel<DT, 32, 3, 2, BWD><<<grid, kThreads, 0, st>>>(a);
            else layernorm_kernel<DT, 32, 4, 1, BWD><<<grid, kThreads, 0, st>>>(a);
            break;
        default:
            if (s.NV == 1) layernorm_kernel<DT, kThreads, 1, 2, BWD><<<grid, kThreads, 0, st>>>(a);
            else if (s.NV == 2) layernorm_kernel<DT, kThreads, 2, 2, BWD><<<grid, kThreads, 0, st>>>(a);
            else if (s.NV == 3) layernorm_kernel<DT, kThreads, 3, 1, BWD><<<grid, kThreads, 0, st>>>(a);
            else layernorm_kernel<DT, kThreads, 4, 1, BWD><<<grid, kThreads, 0, st>>>(a);
    }
}

fftconv_status_t check_args(const fftconv_layernorm_args_t* p) {
    if (!p) return FFTCONV_ERR_INVALID;
    if (p->B < 0 || p->T < 0 || p->H < 0 || !(p->eps >= 0.0f)) return FFTCONV_ERR_INVALID;
    if (p->dtype != FFTCONV_F16 && p->dtype != FFTCONV_BF16) return FFTCONV_ERR_UNSUPPORTED;
    if (p->D < 8 || p->D > 8192 || p->D % 8) return FFTCONV_ERR_UNSUPPORTED;
    const int64_t top = int64_t(1) << 30;  // rows of all heads, and a step beyond them, in 32 bits
    if (p->H > 65535 || p->T >= top || (p->T && p->B >= top / p->T)) return FFTCONV_ERR_UNSUPPORTED;
    if (p->H && p->B * p->T >= top / p->H) return FFTCONV_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(p->w) | reinterpret_cast<uintptr_t>(p->b)) & 3) return FFTCONV_ERR_ALIGN;
    return FFTCONV_OK;
}

bool same_view(const View& a, const View& b) { return a.p == b.p && a.b == b.b && a.t == b.t && a.h == b.h; }

// Shared by both directions: fills the kernel arguments and launches.
template <bool BWD>
fftconv_status_t run(const fftconv_layernorm_args_t* p, fftconv_view_t dy, fftconv_view_t y, float* dw, float* db,
                     void* scratch, size_t scratch_bytes, fftconv_stream_t stream) {
    fftconv_status_t e = check_args(p);
    if (e != FFTCONV_OK) return e;
    if ((reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(db)) & 3) return FFTCONV_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t wb = size_t(p->H) * p->D * 4;
    if (p->B == 0 || p->T == 0 || p->H == 0) {
        if (meets(span_of(dw, wb), span_of(db, wb))) return FFTCONV_ERR_INVALID;
        if (dw && wb && cudaMemsetAsync(dw, 0, wb, st) != cudaSuccess) return FFTCONV_ERR_CUDA;
        if (db && wb && cudaMemsetAsync(db, 0, wb, st) != cudaSuccess) return FFTCONV_ERR_CUDA;
        return FFTCONV_OK;
    }
    NormArgs a{};
    if ((e = take_view(p->x, p->B, p->T, p->H, p->D, &a.x)) != FFTCONV_OK) return e;
    if ((e = take_view(y, p->B, p->T, p->H, p->D, &a.y)) != FFTCONV_OK) return e;
    if (BWD && (e = take_view(dy, p->B, p->T, p->H, p->D, &a.dy)) != FFTCONV_OK) return e;
    // in place is fine: a lane reads its elements before it writes them
    for (const View* x : {&a.x, &a.dy})
        if (x->p && !same_view(*x, a.y) && share(*x, p->H, a.y, p->H, p->B, p->T, p->D)) return FFTCONV_ERR_INVALID;
    a.w = p->w;
    a.b = BWD ? nullptr : p->b;
    a.T = uint32_t(p->T);
    a.rows = uint32_t(p->B * p->T);
    a.H = int(p->H);
    a.D = p->D;
    a.eps = p->eps;
    a.c = 1.0f / float(p->D);
    a.vec = !(off16(a.w) || off16(a.b));
    a.parts = parts_of(p, BWD);
    const size_t sb = size_t(a.parts) * 2 * wb;
    if (BWD && (dw || db)) {
        if (!scratch || scratch_bytes < sb) return FFTCONV_ERR_WORKSPACE;
        if (off16(scratch)) return FFTCONV_ERR_ALIGN;
        a.part = static_cast<float*>(scratch);
    }
    const Span sy = span_of(a.y, p->B, p->T, p->H, p->D), sw = span_of(a.w, wb), sbias = span_of(a.b, wb);
    if (meets(sy, sw) || meets(sy, sbias)) return FFTCONV_ERR_INVALID;
    const Span outs[3] = {span_of(dw, wb), span_of(db, wb), span_of(a.part, sb)};
    const Span ins[4] = {sy, sw, span_of(a.x, p->B, p->T, p->H, p->D), BWD ? span_of(a.dy, p->B, p->T, p->H, p->D) : Span{}};
    if (any_meet(outs, ins)) return FFTCONV_ERR_INVALID;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    if (p->dtype == FFTCONV_F16) launch<0, BWD>(a, st);
    else launch<1, BWD>(a, st);
    if (a.part) {
        const int64_t hd = int64_t(p->H) * p->D;
        layernorm_sum_kernel<<<unsigned((2 * hd + 31) / 32), kThreads, 0, st>>>(a.part, a.parts, hd, dw, db);
    }
    return cudaGetLastError() == cudaSuccess ? FFTCONV_OK : FFTCONV_ERR_CUDA;
}

}  // namespace
}  // namespace fftconv

extern "C" fftconv_status_t fftconv_layernorm_forward(const fftconv_layernorm_args_t* args, fftconv_view_t y,
                                                      fftconv_stream_t stream) {
    return fftconv::run<false>(args, {}, y, nullptr, nullptr, nullptr, 0, stream);
}

extern "C" size_t fftconv_layernorm_scratch_bytes(const fftconv_layernorm_args_t* args) {
    if (fftconv::check_args(args) != FFTCONV_OK || !args->B || !args->T || !args->H) return 0;
    return size_t(fftconv::parts_of(args, true)) * 2 * args->H * args->D * 4;
}

extern "C" fftconv_status_t fftconv_layernorm_backward(const fftconv_layernorm_args_t* args, fftconv_view_t dy,
                                                       fftconv_view_t dx, float* dw, float* db, void* scratch,
                                                       size_t scratch_bytes, fftconv_stream_t stream) {
    return fftconv::run<true>(args, dy, dx, dw, db, scratch, scratch_bytes, stream);
}
