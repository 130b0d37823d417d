// Linear attention with a fixed decay for each head: C entry points and the
// token-by-token kernels.
#include "linattn.h"

#include <new>

namespace fftconv {
namespace {

// ------------------------------------------------------------ token by token
//
// S <- l S + k v^T; o = scale S^T q, one round of sums over Dk a token.
//
// A CTA of 128 threads keeps a slice of 32 of the Dv columns of one state in
// registers: lane % 8 owns 4 columns (16-byte accesses, 128 bytes per row of
// the slice), the 16 groups of 8 lanes own Dk / 16 rows each.  The sums go over
// 4 groups by shuffles and over the 4 warps through shared memory, double
// buffered so that a token costs one barrier.  The state is read and written
// once per call, all the traffic that counts for a token.
struct TokenArgs {
    View q, k, v, o;
    int64_t B, T;
    int H, group;
    float scale;
    const float* decay;
    const float* sin;  // pool of states [nslots][H][Dk][Dv]
    float* sout;
    const int32_t* slots;
    int64_t nslots;
};

template <int DT>
__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
    const cpx a = Op<DT>::unpack(u.x), b = Op<DT>::unpack(u.y);
    x[0] = a.r; x[1] = a.i; x[2] = b.r; x[3] = b.i;
}

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(128) token_kernel(const TokenArgs a) {
    constexpr int RP = DK / 16;
    __shared__ float4 red[2][4][8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int cg = lane % 8, rg = warp * 4 + lane / 8;
    const int h = blockIdx.y, col = blockIdx.z * 32 + cg * 4, hk = h / a.group;
    const int64_t i = blockIdx.x;
    const int64_t si = a.slots ? a.slots[i] : i;
    const bool live = si >= 0 && si < a.nslots;
    const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k.p) + i * a.k.b + hk * a.k.h + rg * RP;
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q.p) + i * a.q.b + hk * a.q.h + rg * RP;
    const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v.p) + i * a.v.b + h * a.v.h + col;
    uint16_t* op = reinterpret_cast<uint16_t*>(a.o.p) + i * a.o.b + h * a.o.h + col;
    if (!live) {
        if (rg == 0)
            for (int64_t t = 0; t < a.T; ++t) *reinterpret_cast<uint2*>(op + t * a.o.t) = make_uint2(0, 0);
        return;
    }
    const int64_t sbase = ((si * a.H + h) * DK + rg * RP) * DV + col;
    float4 S[RP];
    #pragma unroll
    for (int r = 0; r < RP; ++r) S[r] = *reinterpret_cast<const float4*>(a.sin + sbase + r * DV);
    const Decay al = decay_over(head_decay(a.decay, h), 1.0f);
    for (int64_t t = 0; t < a.T; ++t) {
        float k[RP], q[RP], v[4];
        #pragma unroll
        for (int r = 0; r < RP; r += 4) {
            unpack4<DT>(*reinterpret_cast<const uint2*>(kp + t * a.k.t + r), k + r);
            unpack4<DT>(*reinterpret_cast<const uint2*>(qp + t * a.q.t + r), q + r);
        }
        unpack4<DT>(*reinterpret_cast<const uint2*>(vp + t * a.v.t), v);
        float4 s = make_float4(0, 0, 0, 0);
        #pragma unroll
        for (int r = 0; r < RP; ++r) {
            S[r].x = decayed(al, S[r].x, k[r] * v[0]);
            S[r].y = decayed(al, S[r].y, k[r] * v[1]);
            S[r].z = decayed(al, S[r].z, k[r] * v[2]);
            S[r].w = decayed(al, S[r].w, k[r] * v[3]);
            s.x = fmaf(q[r], S[r].x, s.x);
            s.y = fmaf(q[r], S[r].y, s.y);
            s.z = fmaf(q[r], S[r].z, s.z);
            s.w = fmaf(q[r], S[r].w, s.w);
        }
        #pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
            s.z += __shfl_xor_sync(0xffffffffu, s.z, o);
            s.w += __shfl_xor_sync(0xffffffffu, s.w, o);
        }
        const int pb = int(t & 1);
        if (lane < 8) red[pb][warp][lane] = s;
        __syncthreads();
        if (rg == 0) {
            #pragma unroll
            for (int w = 1; w < 4; ++w) {
                const float4 x = red[pb][w][cg];
                s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
            }
            *reinterpret_cast<uint2*>(op + t * a.o.t) =
                make_uint2(Op<DT>::pack(a.scale * s.x, a.scale * s.y), Op<DT>::pack(a.scale * s.z, a.scale * s.w));
        }
    }
    #pragma unroll
    for (int r = 0; r < RP; ++r) *reinterpret_cast<float4*>(a.sout + sbase + r * DV) = S[r];
}

// Whole sequences token by token, a CTA per sequence, head and 32 columns.
template <int DT, int DK, int DV>
__global__ void __launch_bounds__(128) walk_kernel(const Walk a) {
    constexpr int RP = DK / 16;
    __shared__ float4 red[2][4][8];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int cg = lane % 8, rg = warp * 4 + lane / 8;
    const int h = blockIdx.y, col = blockIdx.z * 32 + cg * 4;
    const int i = blockIdx.x;
    const Seq s = locate(a.offsets, a.T, i);
    auto at = [&](const View& x, int hh) { return reinterpret_cast<uint16_t*>(x.p) + s.row * x.b + s.start * x.t + hh * x.h; };
    const uint16_t* kp = at(a.k, h / a.gk) + rg * RP;
    const uint16_t* qp = at(a.q, h / a.gq) + rg * RP;
    const uint16_t* vp = at(a.v, h / a.gv) + col;
    uint16_t* op = a.o32 ? nullptr : at(a.o, h) + col;
    const int64_t sb = (int64_t(i) * a.H + h) * DK * DV;
    float4 S[RP];
    #pragma unroll
    for (int r = 0; r < RP; ++r) {
        const int row = rg * RP + r;
        S[r] = make_float4(0, 0, 0, 0);
        if (!a.state_in) continue;
        const float* p = a.state_in + sb;
        S[r] = a.turned ? make_float4(p[col * DK + row], p[(col + 1) * DK + row], p[(col + 2) * DK + row], p[(col + 3) * DK + row])
                        : *reinterpret_cast<const float4*>(p + row * DV + col);
    }
    const Decay al = decay_over(head_decay(a.decay, h), 1.0f);
    auto lose = [&](const float4& x) {
        return make_float4(decayed(al, x.x, 0), decayed(al, x.y, 0), decayed(al, x.z, 0), decayed(al, x.w, 0));
    };
    for (int64_t n = 0; n < s.len; ++n) {
        const int64_t t = a.reverse ? s.len - 1 - n : n;
        float k[RP], q[RP], v[4], qk = 0.0f;
        #pragma unroll
        for (int r = 0; r < RP; r += 4) {
            unpack4<DT>(*reinterpret_cast<const uint2*>(kp + t * a.k.t + r), k + r);
            unpack4<DT>(*reinterpret_cast<const uint2*>(qp + t * a.q.t + r), q + r);
        }
        unpack4<DT>(*reinterpret_cast<const uint2*>(vp + t * a.v.t), v);
        float4 y = make_float4(0, 0, 0, 0);
        #pragma unroll
        for (int r = 0; r < RP; ++r) {
            if (!a.reverse) S[r] = lose(S[r]);
            const float qs = q[r] * a.s_in;
            qk = fmaf(q[r], k[r], qk);
            y.x = fmaf(qs, S[r].x, y.x);
            y.y = fmaf(qs, S[r].y, y.y);
            y.z = fmaf(qs, S[r].z, y.z);
            y.w = fmaf(qs, S[r].w, y.w);
            const float ku = k[r] * a.s_up;
            S[r].x = fmaf(ku, v[0], S[r].x);
            S[r].y = fmaf(ku, v[1], S[r].y);
            S[r].z = fmaf(ku, v[2], S[r].z);
            S[r].w = fmaf(ku, v[3], S[r].w);
            if (a.reverse) S[r] = lose(S[r]);
        }
        qk *= a.s_p;
        y.x = fmaf(qk, v[0], y.x); y.y = fmaf(qk, v[1], y.y); y.z = fmaf(qk, v[2], y.z); y.w = fmaf(qk, v[3], y.w);
        #pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
        }
        const int pb = int(n & 1);
        if (lane < 8) red[pb][warp][lane] = y;
        __syncthreads();
        if (rg == 0) {
            #pragma unroll
            for (int w = 1; w < 4; ++w) {
                const float4 x = red[pb][w][cg];
                y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
            }
            if (a.o32)
                *reinterpret_cast<float4*>(a.o32 + ((s.row * a.T + s.start + t) * a.H + h) * DV + col) = y;
            else
                *reinterpret_cast<uint2*>(op + t * a.o.t) = make_uint2(Op<DT>::pack(y.x, y.y), Op<DT>::pack(y.z, y.w));
        }
    }
    if (!a.state_out) return;
    #pragma unroll
    for (int r = 0; r < RP; ++r) *reinterpret_cast<float4*>(a.state_out + sb + (rg * RP + r) * DV + col) = S[r];
}

// dq, dk [token][Hk][DK] = the sum over a key head's value heads, 8 features a thread, in the
// heads' order.
template <int DT>
__global__ void __launch_bounds__(256) group_sum_kernel(const float* xq, const float* xk, View yq, View yk, int64_t tokens,
                                                        int64_t T, int Hk, int group, int DK) {
    const int np = DK / 8;
    const int64_t n = tokens * Hk * np * 2;
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < n; e += int64_t(gridDim.x) * 256) {
        const int64_t e2 = e >> 1;
        const float* x = e & 1 ? xk : xq;
        const View& y = e & 1 ? yk : yq;
        const int r = int(e2 % np) * 8;
        const int64_t hk = (e2 / np) % Hk, tok = e2 / np / Hk, b = tok / T, t = tok - b * T;
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

// Zero the tokens of a packed row that belong to no sequence: those before the
// first offset and from the last one on (offsets do not decrease); without
// sequences, every token of every row.
struct GapArgs {
    View v[3];
    int H[3], D[3];
    int n;
    const int32_t* offsets;
    int nseq;
    int64_t B, T;
};

__global__ void __launch_bounds__(256) gap_kernel(const GapArgs a) {
    int64_t lo = a.nseq ? a.offsets[0] : a.T, hi = a.nseq ? a.offsets[a.nseq] : a.T;
    lo = lo < 0 ? 0 : (lo > a.T ? a.T : lo);
    hi = hi < lo ? lo : (hi > a.T ? a.T : hi);
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

template <typename F>
cudaError_t pick(int dt, int dk, int dv, F&& f) {
    if (dt == FFTCONV_F16) {
        if (dk == 64) return dv == 64 ? f.template go<0, 64, 64>() : f.template go<0, 64, 128>();
        return dv == 64 ? f.template go<0, 128, 64>() : f.template go<0, 128, 128>();
    }
    if (dk == 64) return dv == 64 ? f.template go<1, 64, 64>() : f.template go<1, 64, 128>();
    return dv == 64 ? f.template go<1, 128, 64>() : f.template go<1, 128, 128>();
}

struct LaunchToken {
    const TokenArgs& a;
    cudaStream_t st;
    template <int DT, int DK, int DV>
    cudaError_t go() {
        token_kernel<DT, DK, DV><<<dim3(unsigned(a.B), unsigned(a.H), DV / 32), 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

struct LaunchWalk {
    const Walk& a;
    cudaStream_t st;
    template <int DT, int DK, int DV>
    cudaError_t go() {
        walk_kernel<DT, DK, DV><<<dim3(unsigned(a.nseq), unsigned(a.H), DV / 32), 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

bool wrong_device(const fftconv_linattn_s* p) {
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return d != p->device;
}

fftconv_status_t done(cudaError_t e) {
    if (e == cudaSuccess) return FFTCONV_OK;
    cudaGetLastError();
    return FFTCONV_ERR_CUDA;
}

// Sizes and input views of every call.
struct Call {
    View q, k, v;
    int64_t B, T;
    int nseq, Hk, Hv, group;
    bool any;  // there are tokens with outputs
};

fftconv_status_t take_args(const fftconv_linattn_s* p, const fftconv_linattn_args_t* x, Call* a) {
    if (!p || !x || wrong_device(p)) return FFTCONV_ERR_INVALID;
    if (x->B < 0 || x->T < 0 || x->Hk < 0 || x->Hv < 0 || x->nseq < 0) return FFTCONV_ERR_INVALID;
    if (x->Hk == 0 ? x->Hv != 0 : x->Hv % x->Hk != 0) return FFTCONV_ERR_INVALID;
    if (x->offsets ? x->B != 1 : x->nseq != x->B) return FFTCONV_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(x->offsets) | reinterpret_cast<uintptr_t>(x->decay)) & 3) return FFTCONV_ERR_ALIGN;
    const int64_t top = int64_t(1) << 31;
    if (x->B >= top || x->T >= top || x->Hv > 65535 || x->nseq >= top) return FFTCONV_ERR_UNSUPPORTED;
    *a = {};
    a->B = x->B;
    a->T = x->T;
    a->nseq = int(x->nseq);
    a->Hk = int(x->Hk);
    a->Hv = int(x->Hv);
    a->group = x->Hk ? int(x->Hv / x->Hk) : 1;
    a->any = x->B && x->T && x->Hv;
    if (!a->any) return FFTCONV_OK;
    if (!x->decay) return FFTCONV_ERR_INVALID;
    fftconv_status_t e;
    if ((e = take_view(x->q, x->B, x->T, x->Hk, p->Dk, &a->q)) != FFTCONV_OK) return e;
    if ((e = take_view(x->k, x->B, x->T, x->Hk, p->Dk, &a->k)) != FFTCONV_OK) return e;
    return take_view(x->v, x->B, x->T, x->Hv, p->Dv, &a->v);
}

// The address ranges of the inputs.
void input_spans(const fftconv_linattn_s* p, const fftconv_linattn_args_t* x, const Call& a, Span (&in)[5]) {
    in[0] = a.any ? span_of(a.q, a.B, a.T, a.Hk, p->Dk) : Span{};
    in[1] = a.any ? span_of(a.k, a.B, a.T, a.Hk, p->Dk) : Span{};
    in[2] = a.any ? span_of(a.v, a.B, a.T, a.Hv, p->Dv) : Span{};
    in[3] = span_of(x->decay, size_t(a.Hv) * 4);
    in[4] = x->offsets ? span_of(x->offsets, size_t(a.nseq + 1) * 4) : Span{};
}

size_t state_bytes(const fftconv_linattn_s* p, int64_t n, int64_t Hv) { return size_t(n) * Hv * p->Dk * p->Dv * 4; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Scratch: for a backward whose value heads share key heads, dq and dk per
// value head in float32.
struct Scratch {
    size_t q, k, total;  // byte offsets, and the size
    Scratch(const fftconv_linattn_s* p, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t, bool backward) {
        const size_t h = backward && Hk < Hv ? up256(size_t(B) * T * Hv * p->Dk * 4) : 0;
        q = 0;
        k = h;
        total = 2 * h;
    }
};

Walk walk_of(const fftconv_linattn_args_t* x, const Call& c) {
    Walk w{};
    w.decay = x->decay;
    w.offsets = x->offsets;
    w.B = c.B;
    w.T = c.T;
    w.nseq = c.nseq;
    w.H = c.Hv;
    w.gq = w.gk = w.gv = 1;
    w.s_p = x->scale;
    return w;
}

cudaError_t zero_gaps(const fftconv_linattn_args_t* x, const Call& c, int n, const View* v, const int* H, const int* D,
                      cudaStream_t st) {
    GapArgs a{};
    for (int i = 0; i < n; ++i) {
        a.v[i] = v[i];
        a.H[i] = H[i];
        a.D[i] = D[i];
    }
    a.n = n;
    a.offsets = x->offsets;
    a.nseq = x->offsets ? c.nseq : 0;
    a.B = c.B;
    a.T = c.T;
    gap_kernel<<<64, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace fftconv

using namespace fftconv;

extern "C" fftconv_status_t fftconv_linattn_create(fftconv_linattn_t* out, int Dk, int Dv, fftconv_dtype_t dtype) {
    if (!out) return FFTCONV_ERR_INVALID;
    *out = nullptr;
    if ((Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128) || (dtype != FFTCONV_F16 && dtype != FFTCONV_BF16))
        return FFTCONV_ERR_UNSUPPORTED;
    fftconv_linattn_s* p = new (std::nothrow) fftconv_linattn_s;
    if (!p) return FFTCONV_ERR_ALLOC;
    p->Dk = Dk;
    p->Dv = Dv;
    p->dtype = dtype;
    if (cudaGetDevice(&p->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return FFTCONV_ERR_CUDA;
    }
    if (cudaMalloc(&p->dev_err, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        delete p;
        return FFTCONV_ERR_ALLOC;
    }
    if (cudaMemset(p->dev_err, 0, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        cudaFree(p->dev_err);
        delete p;
        return FFTCONV_ERR_CUDA;
    }
    *out = p;
    return FFTCONV_OK;
}

extern "C" fftconv_status_t fftconv_linattn_destroy(fftconv_linattn_t p) {
    if (!p) return FFTCONV_OK;
    cudaFree(p->dev_err);
    delete p;
    return FFTCONV_OK;
}

extern "C" fftconv_status_t fftconv_linattn_status(fftconv_linattn_t p, fftconv_stream_t stream, int* out) {
    if (!p || !out || wrong_device(p)) return FFTCONV_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int v = 0;
    if (cudaMemcpyAsync(&v, p->dev_err, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaMemsetAsync(p->dev_err, 0, sizeof(int), st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) {
        cudaGetLastError();
        return FFTCONV_ERR_CUDA;
    }
    *out = v;
    return FFTCONV_OK;
}

extern "C" size_t fftconv_linattn_scratch_bytes(fftconv_linattn_t p, int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                                                int64_t nseq, int backward) {
    if (!p || B < 0 || T < 0 || Hk < 0 || Hv < 0 || nseq < 0) return 0;
    return Scratch(p, B, T, Hk, Hv, nseq, backward != 0).total;
}

extern "C" fftconv_status_t fftconv_linattn_forward(fftconv_linattn_t p, const fftconv_linattn_args_t* args,
                                                    const float* state_in, fftconv_view_t o, float* state_out,
                                                    void* scratch, size_t scratch_bytes, fftconv_stream_t stream) {
    Call c;
    fftconv_status_t e = take_args(p, args, &c);
    if (e != FFTCONV_OK) return e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((c.nseq == 0 && !args->offsets) || c.Hv == 0) return FFTCONV_OK;
    if (off16(state_in) || off16(state_out) || off16(scratch)) return FFTCONV_ERR_ALIGN;
    const size_t sb = state_bytes(p, c.nseq, c.Hv);
    const Scratch l(p, c.B, c.T, c.Hk, c.Hv, c.nseq, false);
    if (l.total && (!scratch || scratch_bytes < l.total)) return FFTCONV_ERR_WORKSPACE;
    View vo{};
    if (c.any && (e = take_view(o, c.B, c.T, c.Hv, p->Dv, &vo)) != FFTCONV_OK) return e;
    Span in[5];
    input_spans(p, args, c, in);
    const Span outs[3] = {c.any ? span_of(vo, c.B, c.T, c.Hv, p->Dv) : Span{}, span_of(state_out, sb), span_of(scratch, l.total)};
    const Span si[1] = {span_of(state_in, sb)};
    if (any_meet(outs, in) || any_meet(outs, si)) return FFTCONV_ERR_INVALID;
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    if (!c.any) {  // empty rows: the states pass through
        if (!state_out) return FFTCONV_OK;
        return done(state_in ? cudaMemcpyAsync(state_out, state_in, sb, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(state_out, 0, sb, st));
    }
    Walk w = walk_of(args, c);
    w.q = c.q;
    w.k = c.k;
    w.v = c.v;
    w.o = vo;
    w.gq = w.gk = c.group;
    w.s_in = args->scale;
    w.s_up = 1.0f;
    w.state_in = state_in;
    w.state_out = state_out;
    cudaError_t r = cudaSuccess;
    if (args->offsets) r = zero_gaps(args, c, 1, &vo, &c.Hv, &p->Dv, st);
    if (r == cudaSuccess && c.nseq) r = pick(p->dtype, p->Dk, p->Dv, LaunchWalk{w, st});
    return done(r);
}

extern "C" fftconv_status_t fftconv_linattn_backward(fftconv_linattn_t p, const fftconv_linattn_args_t* args,
                                                     const float* state_in, fftconv_view_t d_o, const float* d_state_out,
                                                     fftconv_view_t dq, fftconv_view_t dk, fftconv_view_t dv,
                                                     float* d_state_in, void* scratch, size_t scratch_bytes,
                                                     fftconv_stream_t stream) {
    Call c;
    fftconv_status_t e = take_args(p, args, &c);
    if (e != FFTCONV_OK) return e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (c.Hv == 0) {  // no value head uses the queries and keys
        if (!c.B || !c.T || !c.Hk) return FFTCONV_OK;
        View v[2];
        if ((e = take_view(dq, c.B, c.T, c.Hk, p->Dk, &v[0])) != FFTCONV_OK) return e;
        if ((e = take_view(dk, c.B, c.T, c.Hk, p->Dk, &v[1])) != FFTCONV_OK) return e;
        const int H[2] = {c.Hk, c.Hk}, D[2] = {p->Dk, p->Dk};
        c.nseq = 0;
        return done(zero_gaps(args, c, 2, v, H, D, st));
    }
    if (c.nseq == 0 && !args->offsets) return FFTCONV_OK;
    if (off16(state_in) || off16(d_state_out) || off16(d_state_in) || off16(scratch)) return FFTCONV_ERR_ALIGN;
    const size_t sb = state_bytes(p, c.nseq, c.Hv);
    if (!c.any) {
        if (!d_state_in) return FFTCONV_OK;
        if (meets(span_of(d_state_in, sb), span_of(d_state_out, sb))) return FFTCONV_ERR_INVALID;
        return done(d_state_out ? cudaMemcpyAsync(d_state_in, d_state_out, sb, cudaMemcpyDeviceToDevice, st)
                                : cudaMemsetAsync(d_state_in, 0, sb, st));
    }
    const Scratch l(p, c.B, c.T, c.Hk, c.Hv, c.nseq, true);
    if (l.total && (!scratch || scratch_bytes < l.total)) return FFTCONV_ERR_WORKSPACE;
    View vdo, vdq, vdk, vdv;
    if ((e = take_view(d_o, c.B, c.T, c.Hv, p->Dv, &vdo)) != FFTCONV_OK) return e;
    if ((e = take_view(dq, c.B, c.T, c.Hk, p->Dk, &vdq)) != FFTCONV_OK) return e;
    if ((e = take_view(dk, c.B, c.T, c.Hk, p->Dk, &vdk)) != FFTCONV_OK) return e;
    if ((e = take_view(dv, c.B, c.T, c.Hv, p->Dv, &vdv)) != FFTCONV_OK) return e;
    Span in[5];
    input_spans(p, args, c, in);
    const Span more[3] = {span_of(vdo, c.B, c.T, c.Hv, p->Dv), span_of(d_state_out, sb), span_of(state_in, sb)};
    // tokens' gradients may be slices of one buffer, so they are not checked against each other
    const Span outs[5] = {span_of(vdq, c.B, c.T, c.Hk, p->Dk), span_of(vdk, c.B, c.T, c.Hk, p->Dk),
                          span_of(vdv, c.B, c.T, c.Hv, p->Dv), span_of(d_state_in, sb), span_of(scratch, l.total)};
    if (any_meet(outs, in) || any_meet(outs, more)) return FFTCONV_ERR_INVALID;
    for (int i = 3; i < 5; ++i)  // the state's gradient and scratch overlap nothing
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    const bool shared = c.group > 1;
    float* dq32 = shared ? reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + l.q) : nullptr;
    float* dk32 = shared ? reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + l.k) : nullptr;
    Walk wq = walk_of(args, c), wv = wq, wk = wq;
    wq.q = vdo, wq.k = c.v, wq.v = c.k, wq.o = vdq, wq.o32 = dq32;
    wq.gv = c.group;
    wq.s_in = args->scale, wq.s_up = 1.0f;
    wq.state_in = state_in, wq.turned = true;
    wv.q = c.k, wv.k = c.q, wv.v = vdo, wv.o = vdv;
    wv.gq = wv.gk = c.group;
    wv.reverse = true;
    wv.s_in = 1.0f, wv.s_up = args->scale;
    wv.state_in = d_state_out, wv.state_out = d_state_in;
    wk.q = c.v, wk.k = vdo, wk.v = c.q, wk.o = vdk, wk.o32 = dk32;
    wk.gv = c.group;
    wk.reverse = true;
    wk.s_in = 1.0f, wk.s_up = args->scale;
    wk.state_in = d_state_out, wk.turned = true;
    cudaError_t r = cudaSuccess;
    if (args->offsets) {
        const View zs[3] = {vdq, vdk, vdv};
        const int zh[3] = {c.Hk, c.Hk, c.Hv}, zd[3] = {p->Dk, p->Dk, p->Dv};
        // with shared heads dq and dk are summed from float32 parts, zero in the gaps
        if (shared) r = cudaMemsetAsync(scratch, 0, l.total, st);
        if (r == cudaSuccess) r = zero_gaps(args, c, 3, zs, zh, zd, st);
    }
    if (c.nseq) {
        if (r == cudaSuccess) r = pick(p->dtype, p->Dv, p->Dk, LaunchWalk{wq, st});
        if (r == cudaSuccess) r = pick(p->dtype, p->Dk, p->Dv, LaunchWalk{wv, st});
        if (r == cudaSuccess) r = pick(p->dtype, p->Dv, p->Dk, LaunchWalk{wk, st});
        if (r == cudaSuccess && shared) {
            const int64_t n = (c.B * c.T * c.Hk * (p->Dk / 8) * 2 + 255) / 256;
            const unsigned grid = unsigned(n < 152 * 32 ? n : 152 * 32);
            auto f = p->dtype == FFTCONV_F16 ? group_sum_kernel<0> : group_sum_kernel<1>;
            f<<<grid, 256, 0, st>>>(dq32, dk32, vdq, vdk, c.B * c.T, c.T, c.Hk, c.group, p->Dk);
            r = cudaGetLastError();
        }
    }
    return done(r);
}

extern "C" fftconv_status_t fftconv_linattn_step(fftconv_linattn_t p, const fftconv_linattn_args_t* args,
                                                 const float* state_in, float* state_out, int64_t nslots,
                                                 const int32_t* slots, fftconv_view_t o, fftconv_stream_t stream) {
    Call c;
    fftconv_status_t e = take_args(p, args, &c);
    if (e != FFTCONV_OK) return e;
    if (args->offsets || nslots < 0 || (!slots && nslots < c.B)) return FFTCONV_ERR_INVALID;
    if (!c.any) return FFTCONV_OK;
    if (!state_in || !state_out) return FFTCONV_ERR_INVALID;
    if (off16(state_in) || off16(state_out) || (reinterpret_cast<uintptr_t>(slots) & 3)) return FFTCONV_ERR_ALIGN;
    TokenArgs a{};
    if ((e = take_view(o, c.B, c.T, c.Hv, p->Dv, &a.o)) != FFTCONV_OK) return e;
    const size_t sb = state_bytes(p, nslots, c.Hv);
    Span in[5];
    input_spans(p, args, c, in);
    const Span outs[2] = {span_of(a.o, c.B, c.T, c.Hv, p->Dv), span_of(state_out, sb)};
    const Span more[2] = {span_of(slots, size_t(c.B) * 4), state_in == state_out ? Span{} : span_of(state_in, sb)};
    if (any_meet(outs, in) || any_meet(outs, more) || meets(outs[0], outs[1]) || meets(outs[0], span_of(state_in, sb)))
        return FFTCONV_ERR_INVALID;
    a.q = c.q;
    a.k = c.k;
    a.v = c.v;
    a.B = c.B;
    a.T = c.T;
    a.H = c.Hv;
    a.group = c.group;
    a.scale = args->scale;
    a.decay = args->decay;
    a.sin = state_in;
    a.sout = state_out;
    a.slots = slots;
    a.nslots = nslots;
    return done(pick(p->dtype, p->Dk, p->Dv, LaunchToken{a, static_cast<cudaStream_t>(stream)}));
}
