// Layer norm of rows of features, and its gradients.
//
// Mathematics: m = mean x, r = rsqrt(mean (x - m)^2 + eps), h = (x - m) r,
// y = h w + b.  Backward, with dz = dy w: dx = r (dz - mean dz - h mean(dz h)),
// dw = sum dy h and db = sum dy over all tokens.  The variance is taken from the
// differences to the mean, so a mean that is large against the spread costs no more than
// its own rounding (h off by 1.5e-5 where it is 500 spreads).
//
// Bound: one read of x (and dy) and one write of y (dx) per element, so HBM
// bandwidth for whole batches and launch latency for single tokens.  Split: a row
// belongs to G lanes that hold NV runs of 8 consecutive features (a 16-byte load
// each): whole rows stay in registers, so nothing is read twice.  Up to 1024
// features G is at most a warp and the row's sums are shuffles; wider rows take half
// of a CTA or all of it, whose warps' sums meet in shared memory.  Few lanes with two
// runs each cost fewer shuffles and instructions than many with one (2097152 rows of
// 32 features: 48 us, 62 us with four lanes of one run).  The grid is what the SMs
// hold at once: the weights are read once a CTA and stay in registers, and the next
// rows' loads are in flight while the current ones are worked (131072 rows of 768
// features: forward 65 us, 6.2 TB/s; 95 us with a CTA for every 16 rows).
#include "views.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "tile.cuh"

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

using tile::fma2;
using tile::mul2;
using tile::sub2;

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return fma2(a, make_float2(1.0f, 1.0f), b); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Eight values as four pairs: the arithmetic is in packed float32 pairs, which halves
// the instructions that a row costs.
template <int DT>
__device__ __forceinline__ void unpack8(const uint4& u, float2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    #pragma unroll
    for (int i = 0; i < 4; ++i) {
        const cpx c = Op<DT>::unpack(w[i]);
        x[i] = make_float2(c.r, c.i);
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
    return make_uint4(Op<DT>::pack(x[0].x, x[0].y), Op<DT>::pack(x[1].x, x[1].y), Op<DT>::pack(x[2].x, x[2].y),
                      Op<DT>::pack(x[3].x, x[3].y));
}

__device__ __forceinline__ void load8(const float* p, bool vec, float2 (&x)[4]) {
    if (vec) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p)), v = __ldg(reinterpret_cast<const float4*>(p) + 1);
        x[0] = make_float2(u.x, u.y);
        x[1] = make_float2(u.z, u.w);
        x[2] = make_float2(v.x, v.y);
        x[3] = make_float2(v.z, v.w);
    } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = make_float2(__ldg(p + 2 * j), __ldg(p + 2 * j + 1));
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
        __syncthreads();  // the last sums have been read
        if (threadIdx.x % 32 == 0)
            #pragma unroll
            for (int i = 0; i < N; ++i) red[i][threadIdx.x / 32] = v[i];
        __syncthreads();
        #pragma unroll
        for (int i = 0; i < N; ++i) {
            const float* p = red[i] + threadIdx.x / G * (G / 32);
            float4 a = *reinterpret_cast<const float4*>(p);
            v[i] = (a.x + a.y) + (a.z + a.w);
            if constexpr (G == 256) {
                a = *reinterpret_cast<const float4*>(p + 4);
                v[i] += (a.x + a.y) + (a.z + a.w);
            }
        }
    }
}

// Rows that a group takes at a time, and CTAs that an SM holds: as many rows as the
// registers of two CTAs hold.  The backward's two sums for each feature leave room
// for one row of two runs, or for one CTA (131072 rows of 768 features in two CTAs
// of one row: 178 us; in one of two rows 111 us).
__host__ __device__ constexpr int rows_at_once(int G, int NV, bool bwd) { return bwd ? (G == 32 && NV == 3 ? 2 : 1) : (NV <= (G <= 32 ? 3 : 2) ? 2 : 1); }
__host__ __device__ constexpr int ctas_per_sm(int NV, bool bwd) { return bwd && NV > 2 ? 1 : 2; }

template <int DT, int G, int NV, bool BWD>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NV, BWD)) layernorm_kernel(const NormArgs a) {
    constexpr int NG = kThreads / G, RB = rows_at_once(G, NV, BWD);
    __shared__ __align__(16) float red[G > 32 ? 2 * RB : 1][8];
    const int lane = threadIdx.x % G, grp = threadIdx.x / G;
    const int h = blockIdx.x % a.H, part = blockIdx.x / a.H;
    int f[NV];
    bool on[NV];
    float2 w[NV][4], b[BWD ? 1 : NV][4];
    #pragma unroll
    for (int v = 0; v < NV; ++v) {
        f[v] = (v * G + lane) * 8;
        on[v] = f[v] < a.D;
        #pragma unroll
        for (int j = 0; j < 4; ++j) w[v][j] = both(1.0f);
        if (a.w && on[v]) load8(a.w + int64_t(h) * a.D + f[v], a.vec, w[v]);
        if constexpr (!BWD) {
            #pragma unroll
            for (int j = 0; j < 4; ++j) b[v][j] = both(0.0f);
            if (a.b && on[v]) load8(a.b + int64_t(h) * a.D + f[v], a.vec, b[v]);
        }
    }
    float2 aw[BWD ? NV : 1][4] = {}, ab[BWD ? NV : 1][4] = {};
    // where row r of this group starts in a view, in elements
    auto at = [&](const View& v, uint32_t r) {
        const uint32_t bi = r / a.T;
        return bi * v.b + int64_t(r - bi * a.T) * v.t + h * v.h;
    };
    uint4 ux[RB][NV], ud[BWD ? RB : 1][NV];
    auto fetch = [&](uint32_t base) {
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            const uint32_t r = base + i * NG + grp;
            const bool in = r < a.rows;
            const uint16_t* px = reinterpret_cast<const uint16_t*>(a.x.p) + (in ? at(a.x, r) : 0);
            const uint16_t* pd = BWD ? reinterpret_cast<const uint16_t*>(a.dy.p) + (in ? at(a.dy, r) : 0) : nullptr;
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                ux[i][v] = in && on[v] ? *reinterpret_cast<const uint4*>(px + f[v]) : make_uint4(0, 0, 0, 0);
                if constexpr (BWD) ud[i][v] = in && on[v] ? *reinterpret_cast<const uint4*>(pd + f[v]) : make_uint4(0, 0, 0, 0);
            }
        }
    };
    const uint32_t step = uint32_t(a.parts) * (NG * RB);
    uint32_t base = uint32_t(part) * (NG * RB);
    if (base < a.rows) fetch(base);
    for (; base < a.rows; base += step) {
        // the rows as float32; the next ones are fetched while these are worked
        float2 x[RB][NV][4], d[BWD ? RB : 1][NV][4];
        #pragma unroll
        for (int i = 0; i < RB; ++i)
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                unpack8<DT>(ux[i][v], x[i][v]);
                if constexpr (BWD) unpack8<DT>(ud[i][v], d[i][v]);
            }
        if (base + step < a.rows) fetch(base + step);
        float s[BWD ? 2 * RB : RB];
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            float2 p = both(0.0f), q = p;
            #pragma unroll
            for (int v = 0; v < NV; ++v)
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p = add2(p, x[i][v][j]);
                    if constexpr (BWD) q = fma2(d[i][v][j], w[v][j], q);
                }
            s[i] = p.x + p.y;
            if constexpr (BWD) s[RB + i] = q.x + q.y;
        }
        row_sums<G>(s, red);
        float e[BWD ? 2 * RB : RB], mz[RB];
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            const float m = s[i] / float(a.D);  // exact for rows of equal values, as their sums are
            if constexpr (BWD) mz[i] = s[RB + i] * a.c;
            float2 p = both(0.0f), q = p;
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!on[v]) continue;
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2& y = x[i][v][j];
                    y = sub2(y, both(m));
                    p = fma2(y, y, p);
                    if constexpr (BWD) q = fma2(mul2(d[i][v][j], w[v][j]), y, q);
                }
            }
            e[i] = p.x + p.y;
            if constexpr (BWD) e[RB + i] = q.x + q.y;
        }
        row_sums<G>(e, red);
        #pragma unroll
        for (int i = 0; i < RB; ++i) {
            const uint32_t row = base + i * NG + grp;
            if (row >= a.rows) continue;
            const float r = rsqrtf(fmaf(e[i], a.c, a.eps));
            uint16_t* py = reinterpret_cast<uint16_t*>(a.y.p) + at(a.y, row);
            #pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!on[v]) continue;
                float2 (&y)[4] = x[i][v];
                if constexpr (!BWD) {
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = fma2(mul2(y[j], both(r)), w[v][j], b[v][j]);
                } else {
                    const float2 mh = both(-e[RB + i] * a.c * r * r), mr = both(-mz[i] * r);  // - mean(dz h) r, - mean(dz) r
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 hh = mul2(y[j], both(r)), z = d[i][v][j];
                        aw[v][j] = fma2(z, hh, aw[v][j]);
                        ab[v][j] = add2(ab[v][j], z);
                        y[j] = fma2(hh, mh, fma2(mul2(z, w[v][j]), both(r), mr));
                    }
                }
                *reinterpret_cast<uint4*>(py + f[v]) = pack8<DT>(y);
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
                for (int j = 0; j < 4; ++j) {
                    *reinterpret_cast<float2*>(out + f[v] + 2 * j) = aw[v][j];
                    *reinterpret_cast<float2*>(out + hd + f[v] + 2 * j) = ab[v][j];
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
                    for (int j = 0; j < 4; ++j) {
                        sums[grp][f[v] + 2 * j] = k ? ab[v][j].x : aw[v][j].x;
                        sums[grp][f[v] + 2 * j + 1] = k ? ab[v][j].y : aw[v][j].y;
                    }
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

// How a row of D features is held: G lanes of NV runs of 8.
struct Shape {
    int G, NV;
};

Shape shape_of(int D) {
    const int n = D / 8;
    for (int G = 2; G <= 32; G *= 2)
        if (n <= 2 * G) return {G, 2};
    if (n <= 128) return {32, (n + 31) / 32};
    if (n <= 512) return {128, (n + 127) / 128};
    return {256, (n + 255) / 256};
}

// CTAs that share a head: what fills the SMs, or what the rows need.
int parts_of(const fftconv_layernorm_args_t* p, bool backward) {
    const Shape s = shape_of(p->D);
    const int64_t per = int64_t(kThreads / s.G) * rows_at_once(s.G, s.NV, backward);
    const int64_t need = (p->B * p->T + per - 1) / per, most = 152 * ctas_per_sm(s.NV, backward) / p->H;
    return int(need < most ? need : (most > 0 ? most : 1));
}

template <int DT, bool BWD>
void launch(const NormArgs& a, cudaStream_t st) {
    const Shape s = shape_of(a.D);
    const unsigned grid = unsigned(a.parts) * unsigned(a.H);
    switch (s.G * 8 + s.NV) {
        case 2 * 8 + 2: layernorm_kernel<DT, 2, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 4 * 8 + 2: layernorm_kernel<DT, 4, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 8 * 8 + 2: layernorm_kernel<DT, 8, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 16 * 8 + 2: layernorm_kernel<DT, 16, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 32 * 8 + 2: layernorm_kernel<DT, 32, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 32 * 8 + 3: layernorm_kernel<DT, 32, 3, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 32 * 8 + 4: layernorm_kernel<DT, 32, 4, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 128 * 8 + 2: layernorm_kernel<DT, 128, 2, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 128 * 8 + 3: layernorm_kernel<DT, 128, 3, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 128 * 8 + 4: layernorm_kernel<DT, 128, 4, BWD><<<grid, kThreads, 0, st>>>(a); break;
        case 256 * 8 + 3: layernorm_kernel<DT, 256, 3, BWD><<<grid, kThreads, 0, st>>>(a); break;
        default: layernorm_kernel<DT, 256, 4, BWD><<<grid, kThreads, 0, st>>>(a);
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
