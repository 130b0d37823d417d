// Linear attention with a fixed decay for each head: C entry points and the
// token-by-token kernels.
#include "linattn_chunk.h"
#include "packed.cuh"

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
// once per call, all the traffic that counts for a token: bound by HBM (256 rows of
// 12 heads of 128 x 128: 405 MB in 65 us, 6.2 TB/s); one row of 6 heads takes 2.4 us.
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
    const Decay al = a.T ? decay_over(head_decay(a.decay, h), 1.0f) : Decay{};
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
    if (x->B >= top || x->T >= top || x->Hv > 65535 || x->nseq >= top || chunk_slots(x->B, x->T, x->nseq) >= top)
        return FFTCONV_ERR_UNSUPPORTED;
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

// Scratch.  Forward: the segments' end states.  Backward: those of S and of its
// gradient, and, where value heads share key heads, dq and dk per value head in
// float32.
struct Scratch {
    Segments seg;
    size_t s, r, q, k, total;  // byte offsets, and the size
    Scratch(const fftconv_linattn_s* p, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t nseq, bool backward) {
        plan_segments(&seg, B, T, nseq, Hv, backward ? 3 : 1, p->dtype, p->num_sms);
        const size_t n = up256(state_bytes(p, seg.states, Hv));
        const size_t h = backward && Hk < Hv ? up256(size_t(B) * T * Hv * p->Dk * 4) : 0;
        s = 0;
        r = n;
        q = backward ? 2 * n : n;
        k = q + h;
        total = k + h;
    }
    bool cut(int nseq) const { return seg.count > nseq; }
};

// A walk of a call, its sizes and constants.
Walk walk_of(const fftconv_linattn_args_t* x, const Call& c, bool reverse) {
    Walk w{};
    w.decay = x->decay;
    w.offsets = x->offsets;
    w.T = c.T;
    w.nseq = c.nseq;
    w.H = c.Hv;
    w.gq = w.gk = w.gv = 1;
    w.s_p = x->scale;
    w.s_in = reverse ? 1.0f : x->scale;
    w.s_up = reverse ? x->scale : 1.0f;
    w.reverse = reverse;
    return w;
}

// A walk's tensors: their views, heads and features.
struct Tensor {
    View v;
    int heads, D;
};

bool encode(const fftconv_linattn_s* p, const Call& c, CUtensorMap* m, const Tensor& t) {
    return encode_tokens_map(m, t.v, c.B, c.T, t.heads, t.D, p->dtype);
}

Passes passes_of(const fftconv_linattn_s* p, const fftconv_linattn_args_t* x, const Scratch& l) {
    Passes a{};
    a.seg_chunks = l.seg.chunks;
    a.segments = l.seg.count;
    a.join = l.seg.join;
    a.most = l.seg.most;
    a.few_cut = l.seg.few_cut;
    a.longest_first = x->offsets && l.seg.by_length;
    a.err = p->dev_err;
    return a;
}

cudaError_t zero_gaps(const fftconv_linattn_args_t* x, const Call& c, int n, const View* v, const int* H, const int* D,
                      cudaStream_t st) {
    GapArgs<3> a{};
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
    gap_kernel<3><<<64, 256, 0, st>>>(a);
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
    if (l.seg.count >= (int64_t(1) << 30) / c.Hv) return FFTCONV_ERR_UNSUPPORTED;
    Passes a = passes_of(p, args, l);
    Pass& x = a.p[0];
    x.w = walk_of(args, c, false);
    x.w.gq = x.w.gk = c.group;
    x.w.o = vo;
    x.w.state_in = state_in;
    x.w.state_out = state_out;
    x.seg_state = static_cast<float*>(scratch);
    const Tensor q{c.q, c.Hk, p->Dk}, k{c.k, c.Hk, p->Dk}, v{c.v, c.Hv, p->Dv}, y{vo, c.Hv, p->Dv};
    if (!encode(p, c, &x.mq, q) || !encode(p, c, &x.mk, k) || !encode(p, c, &x.mv, v) || !encode(p, c, &x.mo, y))
        return FFTCONV_ERR_UNSUPPORTED;
    cudaError_t r = cudaSuccess;
    if (args->offsets) r = zero_gaps(args, c, 1, &vo, &c.Hv, &p->Dv, st);
    if (!c.nseq) return done(r);
    if (r == cudaSuccess && l.cut(c.nseq)) r = launch_linattn(a, 1, true, p->dtype, p->Dk, p->Dv, st);
    if (r == cudaSuccess) r = launch_linattn(a, 1, false, p->dtype, p->Dk, p->Dv, st);
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
    if (l.seg.count >= (int64_t(1) << 30) / c.Hv) return FFTCONV_ERR_UNSUPPORTED;
    const bool shared = c.group > 1;
    uint8_t* at = static_cast<uint8_t*>(scratch);
    float* dq32 = shared ? reinterpret_cast<float*>(at + l.q) : nullptr;
    float* dk32 = shared ? reinterpret_cast<float*>(at + l.k) : nullptr;
    // dQ and dK in tensors of Dv x Dk, dV of Dk x Dv: one launch where that is the same
    Passes a = passes_of(p, args, l);
    Pass &xq = a.p[0], &xk = a.p[1], &xv = a.p[2];
    xq.w = walk_of(args, c, false);
    xq.w.gv = c.group;
    xq.w.o = vdq;
    xq.w.o32 = dq32;
    xq.w.state_in = state_in;
    xq.w.turned = true;
    xk.w = walk_of(args, c, true);
    xk.w.gv = c.group;
    xk.w.o = vdk;
    xk.w.o32 = dk32;
    xk.w.state_in = d_state_out;
    xk.w.turned = true;
    xv.w = walk_of(args, c, true);
    xv.w.gq = xv.w.gk = c.group;
    xv.w.o = vdv;
    xv.w.state_in = d_state_out;
    xv.w.state_out = d_state_in;
    xq.seg_state = reinterpret_cast<float*>(at + l.s);
    xk.seg_state = xv.seg_state = reinterpret_cast<float*>(at + l.r);
    const Tensor q{c.q, c.Hk, p->Dk}, k{c.k, c.Hk, p->Dk}, v{c.v, c.Hv, p->Dv}, d{vdo, c.Hv, p->Dv};
    const Tensor yq{vdq, c.Hk, p->Dk}, yk{vdk, c.Hk, p->Dk}, yv{vdv, c.Hv, p->Dv};
    if (!encode(p, c, &xq.mq, d) || !encode(p, c, &xq.mk, v) || !encode(p, c, &xq.mv, k) || !encode(p, c, &xq.mo, yq) ||
        !encode(p, c, &xk.mq, v) || !encode(p, c, &xk.mk, d) || !encode(p, c, &xk.mv, q) || !encode(p, c, &xk.mo, yk) ||
        !encode(p, c, &xv.mq, k) || !encode(p, c, &xv.mk, q) || !encode(p, c, &xv.mv, d) || !encode(p, c, &xv.mo, yv))
        return FFTCONV_ERR_UNSUPPORTED;
    // the segments' states: S as the forward forms it, its gradient as dV's walk does
    Passes b = a;
    b.p[0] = xv;
    b.p[1] = xv;
    b.p[1].w.reverse = false;
    b.p[1].w.s_up = 1.0f;
    b.p[1].w.state_in = state_in;
    b.p[1].w.state_out = nullptr;
    b.p[1].mk = xq.mv;
    b.p[1].mv = xq.mk;
    b.p[1].seg_state = xq.seg_state;
    Passes only_dv = a;
    only_dv.p[0] = xv;
    cudaError_t r = cudaSuccess;
    if (args->offsets) {
        const View zs[3] = {vdq, vdk, vdv};
        const int zh[3] = {c.Hk, c.Hk, c.Hv}, zd[3] = {p->Dk, p->Dk, p->Dv};
        r = zero_gaps(args, c, 3, zs, zh, zd, st);
    }
    if (c.nseq) {
        const bool same = p->Dk == p->Dv;
        if (r == cudaSuccess && l.cut(c.nseq)) r = launch_linattn(b, 2, true, p->dtype, p->Dk, p->Dv, st);
        if (r == cudaSuccess) r = launch_linattn(a, same ? 3 : 2, false, p->dtype, p->Dv, p->Dk, st);
        if (r == cudaSuccess && !same) r = launch_linattn(only_dv, 1, false, p->dtype, p->Dk, p->Dv, st);
        if (r == cudaSuccess && shared) {
            const int64_t n = (c.B * c.T * c.Hk * (p->Dk / 8) * 2 + 255) / 256, most = int64_t(p->num_sms) * 32;
            const unsigned grid = unsigned(n < most ? n : most);
            auto f = p->dtype == FFTCONV_F16 ? head_sum_kernel<0> : head_sum_kernel<1>;
            f<<<grid, 256, 0, st>>>(dq32, dk32, vdq, vdk, c.B * c.T, c.T, c.Hk, c.group, p->Dk, args->offsets,
                                    c.nseq);
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
    if (!c.B || !c.Hv || (!c.T && state_in == state_out)) return FFTCONV_OK;
    if (!state_in || !state_out) return FFTCONV_ERR_INVALID;
    if (off16(state_in) || off16(state_out) || (reinterpret_cast<uintptr_t>(slots) & 3)) return FFTCONV_ERR_ALIGN;
    TokenArgs a{};
    if (c.any && (e = take_view(o, c.B, c.T, c.Hv, p->Dv, &a.o)) != FFTCONV_OK) return e;
    const size_t sb = state_bytes(p, nslots, c.Hv);
    Span in[5];
    input_spans(p, args, c, in);
    const Span outs[2] = {c.any ? span_of(a.o, c.B, c.T, c.Hv, p->Dv) : Span{}, span_of(state_out, sb)};
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
