// Gated delta rule: C entry points and the token-by-token kernels.
#include "delta.h"
#include "delta_chunk.h"
#include "packed.cuh"

#include <new>

namespace fftconv {
namespace {

// ------------------------------------------------------------ token by token
//
// S~ = exp(g) S; u = beta (v - S~^T k); S = S~ + k u^T; o = scale S^T q.
// With o = scale (S~^T q + (q.k) u) a token needs one round of sums over Dk:
// S~^T k, S~^T q and q.k together, then the rank-one update.
//
// A CTA of 128 threads keeps a slice of 32 of the Dv columns of one state in
// registers: lane % 8 owns 4 columns (16-byte accesses, 128 bytes per row of
// the slice), the 16 groups of 8 lanes own Dk / 16 rows each.  The sums go over
// 4 groups by shuffles and over the 4 warps through shared memory, double
// buffered so that a token costs one barrier.  The state is read and written
// once per call: for one token that is all the traffic that counts, so the
// bound is HBM bandwidth for large batches (Dk / 16 independent 16-byte loads
// in flight per thread; 256 rows of 12 heads of 128 x 128: 63 us, 6.4 TB/s) and
// latency for a few rows (one row: 2.2 us).
struct TokenArgs {
    DeltaArgs d;
    const float* sin;  // pool of states [nslots][Hv][Dk][Dv]
    float* sout;
    const int32_t* slots;
    int64_t nslots;
};

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(128) token_kernel(const TokenArgs a) {
    constexpr int RP = DK / 16;
    __shared__ float4 red[2][4][8][2];
    __shared__ float redqk[2][4];
    const DeltaArgs& d = a.d;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int cg = lane % 8, rg = warp * 4 + lane / 8;
    const int h = blockIdx.y, col = blockIdx.z * 32 + cg * 4, hk = h / d.group;
    const int i = blockIdx.x;
    const Seq s = locate(nullptr, d.T, i);
    const int64_t si = a.slots ? a.slots[i] : i;
    const bool live = si >= 0 && si < a.nslots;
    const uint16_t* kp = reinterpret_cast<const uint16_t*>(d.k.p) + s.row * d.k.b + s.start * d.k.t + hk * d.k.h + rg * RP;
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(d.q.p) + s.row * d.q.b + s.start * d.q.t + hk * d.q.h + rg * RP;
    const uint16_t* vp = reinterpret_cast<const uint16_t*>(d.v.p) + s.row * d.v.b + s.start * d.v.t + h * d.v.h + col;
    uint16_t* op = reinterpret_cast<uint16_t*>(d.o.p) + s.row * d.o.b + s.start * d.o.t + h * d.o.h + col;
    const int64_t go = s.row * d.g.b + s.start * d.g.t + h * d.g.h;
    const int64_t bo = s.row * d.beta.b + s.start * d.beta.t + h * d.beta.h;
    if (!live) {
        if (rg == 0)
            for (int64_t t = 0; t < s.len; ++t) *reinterpret_cast<uint2*>(op + t * d.o.t) = make_uint2(0, 0);
        return;
    }
    const int64_t sbase = ((si * d.Hv + h) * DK + rg * RP) * DV + col;
    float4 S[RP];
    #pragma unroll
    for (int r = 0; r < RP; ++r)
        S[r] = *reinterpret_cast<const float4*>(a.sin + sbase + r * DV);
    for (int64_t t = 0; t < s.len; ++t) {
        float k[RP], q[RP], v[4];
        #pragma unroll
        for (int r = 0; r < RP; r += 4) {
            const uint2 uk = *reinterpret_cast<const uint2*>(kp + t * d.k.t + r);
            const uint2 uq = *reinterpret_cast<const uint2*>(qp + t * d.q.t + r);
            const cpx k0 = Op<DT>::unpack(uk.x), k1 = Op<DT>::unpack(uk.y);
            const cpx q0 = Op<DT>::unpack(uq.x), q1 = Op<DT>::unpack(uq.y);
            k[r] = k0.r; k[r + 1] = k0.i; k[r + 2] = k1.r; k[r + 3] = k1.i;
            q[r] = q0.r; q[r + 1] = q0.i; q[r + 2] = q1.r; q[r + 3] = q1.i;
        }
        {
            const uint2 uv = *reinterpret_cast<const uint2*>(vp + t * d.v.t);
            const cpx v0 = Op<DT>::unpack(uv.x), v1 = Op<DT>::unpack(uv.y);
            v[0] = v0.r; v[1] = v0.i; v[2] = v1.r; v[3] = v1.i;
        }
        const float al = expf(log_decay(load16<DT>(d.g, go + t * d.g.t)));
        const float be = load16<DT>(d.beta, bo + t * d.beta.t);
        float ks[4] = {}, qs[4] = {}, qk = 0.0f;
        #pragma unroll
        for (int r = 0; r < RP; ++r) {
            S[r].x *= al; S[r].y *= al; S[r].z *= al; S[r].w *= al;
            ks[0] = fmaf(k[r], S[r].x, ks[0]); ks[1] = fmaf(k[r], S[r].y, ks[1]);
            ks[2] = fmaf(k[r], S[r].z, ks[2]); ks[3] = fmaf(k[r], S[r].w, ks[3]);
            qs[0] = fmaf(q[r], S[r].x, qs[0]); qs[1] = fmaf(q[r], S[r].y, qs[1]);
            qs[2] = fmaf(q[r], S[r].z, qs[2]); qs[3] = fmaf(q[r], S[r].w, qs[3]);
            qk = fmaf(q[r], k[r], qk);
        }
        #pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                ks[j] += __shfl_xor_sync(0xffffffffu, ks[j], o);
                qs[j] += __shfl_xor_sync(0xffffffffu, qs[j], o);
            }
            qk += __shfl_xor_sync(0xffffffffu, qk, o);
        }
        const int pb = int(t & 1);
        if (lane < 8) {
            red[pb][warp][lane][0] = make_float4(ks[0], ks[1], ks[2], ks[3]);
            red[pb][warp][lane][1] = make_float4(qs[0], qs[1], qs[2], qs[3]);
            if (lane == 0) redqk[pb][warp] = qk;
        }
        __syncthreads();
        float4 K = red[pb][0][cg][0], Q = red[pb][0][cg][1];
        float QK = redqk[pb][0];
        #pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 x = red[pb][w][cg][0], y = red[pb][w][cg][1];
            K.x += x.x; K.y += x.y; K.z += x.z; K.w += x.w;
            Q.x += y.x; Q.y += y.y; Q.z += y.z; Q.w += y.w;
            QK += redqk[pb][w];
        }
        const float4 u = make_float4(be * (v[0] - K.x), be * (v[1] - K.y), be * (v[2] - K.z), be * (v[3] - K.w));
        #pragma unroll
        for (int r = 0; r < RP; ++r) {
            S[r].x = fmaf(k[r], u.x, S[r].x); S[r].y = fmaf(k[r], u.y, S[r].y);
            S[r].z = fmaf(k[r], u.z, S[r].z); S[r].w = fmaf(k[r], u.w, S[r].w);
        }
        if (rg == 0) {
            const float sc = d.scale;
            *reinterpret_cast<uint2*>(op + t * d.o.t) =
                make_uint2(Op<DT>::pack(sc * fmaf(QK, u.x, Q.x), sc * fmaf(QK, u.y, Q.y)),
                           Op<DT>::pack(sc * fmaf(QK, u.z, Q.z), sc * fmaf(QK, u.w, Q.w)));
        }
    }
    #pragma unroll
    for (int r = 0; r < RP; ++r) *reinterpret_cast<float4*>(a.sout + sbase + r * DV) = S[r];
}

template <typename F>
auto pick(int dt, int dk, int dv, F&& f) {
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
        token_kernel<DT, DK, DV><<<dim3(unsigned(a.d.nseq), unsigned(a.d.Hv), DV / 32), 128, 0, st>>>(a);
        return cudaGetLastError();
    }
};

bool wrong_device(const fftconv_delta_s* p) {
    int d = -1;
    if (cudaGetDevice(&d) != cudaSuccess) {
        cudaGetLastError();
        return true;
    }
    return d != p->device;
}

// Sizes and input views of every call.
fftconv_status_t take_args(const fftconv_delta_s* p, const fftconv_delta_args_t* x, DeltaArgs* a) {
    if (!p || !x || wrong_device(p)) return FFTCONV_ERR_INVALID;
    if (x->B < 0 || x->T < 0 || x->Hk < 0 || x->Hv < 0 || x->nseq < 0) return FFTCONV_ERR_INVALID;
    if (x->Hk == 0 ? x->Hv != 0 : x->Hv % x->Hk != 0) return FFTCONV_ERR_INVALID;
    if (x->offsets ? x->B != 1 : x->nseq != x->B) return FFTCONV_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(x->offsets) & 3) return FFTCONV_ERR_ALIGN;
    const int64_t top = int64_t(1) << 31;
    if (x->B >= top || x->T >= top || x->Hv > 65535 || x->nseq >= top) return FFTCONV_ERR_UNSUPPORTED;
    a->offsets = x->offsets;
    a->B = x->B;
    a->T = x->T;
    a->nseq = int(x->nseq);
    a->Hk = int(x->Hk);
    a->Hv = int(x->Hv);
    a->group = x->Hk ? int(x->Hv / x->Hk) : 1;
    a->scale = x->scale;
    a->err = p->dev_err;
    if (x->B == 0 || x->T == 0 || x->Hv == 0) return FFTCONV_OK;
    fftconv_status_t e;
    if ((e = take_view(x->q, x->B, x->T, x->Hk, p->Dk, &a->q)) != FFTCONV_OK) return e;
    if ((e = take_view(x->k, x->B, x->T, x->Hk, p->Dk, &a->k)) != FFTCONV_OK) return e;
    if ((e = take_view(x->v, x->B, x->T, x->Hv, p->Dv, &a->v)) != FFTCONV_OK) return e;
    if ((e = take_view(x->g, x->B, x->T, x->Hv, 0, &a->g)) != FFTCONV_OK) return e;
    return take_view(x->beta, x->B, x->T, x->Hv, 0, &a->beta);
}

// The address ranges of the inputs.
void input_spans(const fftconv_delta_s* p, const DeltaArgs& a, Span (&in)[6]) {
    const bool any = a.B && a.T && a.Hv;
    in[0] = any ? span_of(a.q, a.B, a.T, a.Hk, p->Dk) : Span{};
    in[1] = any ? span_of(a.k, a.B, a.T, a.Hk, p->Dk) : Span{};
    in[2] = any ? span_of(a.v, a.B, a.T, a.Hv, p->Dv) : Span{};
    in[3] = any ? span_of(a.g, a.B, a.T, a.Hv, 0) : Span{};
    in[4] = any ? span_of(a.beta, a.B, a.T, a.Hv, 0) : Span{};
    in[5] = a.offsets ? span_of(a.offsets, size_t(a.nseq + 1) * 4) : Span{};
}

size_t state_bytes(const fftconv_delta_s* p, int64_t n, int64_t Hv) { return size_t(n) * Hv * p->Dk * p->Dv * 4; }

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// What the forward keeps for the backward, per chunk slot and value head: the
// prep kernel's images, S^T at the chunk's start, Vn^T and T.
struct SavedLayout {
    size_t s, v, t, total;  // byte offsets (the images are first), and the size
    SavedLayout(const fftconv_delta_s* p, int64_t B, int64_t T, int64_t Hv, int64_t nseq) {
        const size_t n = size_t(chunk_slots(B, T, nseq)) * Hv;
        s = n * prep_image(p->Dk);
        v = s + n * p->Dk * p->Dv * 2;
        t = v + n * p->Dv * kChunk * 2;
        total = t + n * kChunk * kChunk * 2;
    }
};

// The backward's scratch: dS'^T and dR (two parts) per chunk slot and value head, and dq, dk
// per value head where value heads share a key head.
struct BwdScratch {
    size_t r, q, k, total;  // byte offsets (dS'^T is first), and the size
    BwdScratch(const fftconv_delta_s* p, int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t nseq) {
        const size_t n = size_t(chunk_slots(B, T, nseq)) * Hv;
        const size_t h = Hk < Hv ? up256(size_t(B) * T * Hv * p->Dk * 4) : 0;
        r = up256(n * p->Dk * p->Dv * 2);
        q = r + up256(n * p->Dv * kChunk * 4);
        k = q + h;
        total = k + h;
    }
};

// The forward's scratch.
struct FwdScratch {
    ChunkArgs c{};
    size_t state, trans, total;  // byte offsets (the images are first), and the size
    FwdScratch(const fftconv_delta_s* p, int64_t B, int64_t T, int64_t Hv, int64_t nseq, bool saved) {
        c.d.B = B;
        c.d.T = T;
        c.d.Hv = int(Hv);
        c.d.nseq = int(nseq);
        plan_segments(&c, p->num_sms);
        const size_t segs = c.segments > nseq ? size_t(c.segments) * Hv * p->Dk * 4 : 0;
        state = saved ? 0 : up256(size_t(c.slots) * Hv * prep_image(p->Dk));
        trans = state + up256(segs * p->Dv);
        total = trans + up256(segs * p->Dk);
    }
};

fftconv_status_t done(cudaError_t e) {
    if (e == cudaSuccess) return FFTCONV_OK;
    cudaGetLastError();
    return FFTCONV_ERR_CUDA;
}

cudaError_t zero_gaps(const DeltaArgs& d, int n, const View* v, const int* H, const int* D, cudaStream_t st) {
    GapArgs<5> a{};
    for (int i = 0; i < n; ++i) {
        a.v[i] = v[i];
        a.H[i] = H[i];
        a.D[i] = D[i];
    }
    a.n = n;
    a.offsets = d.offsets;
    a.nseq = d.nseq;
    a.B = d.B;
    a.T = d.T;
    gap_kernel<5><<<64, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace
}  // namespace fftconv

using namespace fftconv;

extern "C" fftconv_status_t fftconv_delta_create(fftconv_delta_t* out, int Dk, int Dv, fftconv_dtype_t dtype) {
    if (!out) return FFTCONV_ERR_INVALID;
    *out = nullptr;
    if ((Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128) || (dtype != FFTCONV_F16 && dtype != FFTCONV_BF16))
        return FFTCONV_ERR_UNSUPPORTED;
    fftconv_delta_s* p = new (std::nothrow) fftconv_delta_s;
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

extern "C" fftconv_status_t fftconv_delta_destroy(fftconv_delta_t p) {
    if (!p) return FFTCONV_OK;
    cudaFree(p->dev_err);
    delete p;
    return FFTCONV_OK;
}

extern "C" fftconv_status_t fftconv_delta_status(fftconv_delta_t p, fftconv_stream_t stream, int* out) {
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

extern "C" size_t fftconv_delta_saved_bytes(fftconv_delta_t p, int64_t B, int64_t T, int64_t Hv, int64_t nseq) {
    if (!p || B < 0 || T < 0 || Hv < 0 || nseq < 0) return 0;
    const SavedLayout l(p, B, T, Hv, nseq);
    return l.total;
}

extern "C" size_t fftconv_delta_scratch_bytes(fftconv_delta_t p, int64_t B, int64_t T, int64_t Hk, int64_t Hv,
                                              int64_t nseq, int pass) {
    if (!p || B < 0 || T < 0 || Hk < 0 || Hv < 0 || nseq < 0) return 0;
    if (pass != 1) {
        const FwdScratch l(p, B, T, Hv, nseq, pass == 2);
        return l.total;
    }
    const BwdScratch l(p, B, T, Hk, Hv, nseq);
    return l.total;
}

extern "C" fftconv_status_t fftconv_delta_forward(fftconv_delta_t p, const fftconv_delta_args_t* args,
                                                  const float* state_in, fftconv_view_t o, float* state_out,
                                                  void* saved, void* scratch, size_t scratch_bytes,
                                                  fftconv_stream_t stream) {
    ChunkArgs a{};
    fftconv_status_t e = take_args(p, args, &a.d);
    if (e != FFTCONV_OK) return e;
    const DeltaArgs& d = a.d;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if ((d.nseq == 0 && !d.offsets) || d.Hv == 0) return FFTCONV_OK;
    if (off16(state_in) || off16(state_out) || off16(saved) || off16(scratch)) return FFTCONV_ERR_ALIGN;
    const size_t sb = state_bytes(p, d.nseq, d.Hv);
    const size_t vb = fftconv_delta_saved_bytes(p, d.B, d.T, d.Hv, d.nseq);
    // with `saved` the images stay there
    const FwdScratch w(p, d.B, d.T, d.Hv, d.nseq, saved != nullptr);
    const size_t need = w.total;
    if (need && (!scratch || scratch_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    const bool any = d.B && d.T;
    if (any && (e = take_view(o, d.B, d.T, d.Hv, p->Dv, &a.d.o)) != FFTCONV_OK) return e;
    Span in[6];
    input_spans(p, d, in);
    const Span outs[4] = {any ? span_of(d.o, d.B, d.T, d.Hv, p->Dv) : Span{}, span_of(state_out, sb),
                          span_of(saved, vb), span_of(scratch, need)};
    const Span si[1] = {span_of(state_in, sb)};
    if (any_meet(outs, in) || any_meet(outs, si)) return FFTCONV_ERR_INVALID;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    if (!any) {  // empty rows: the states pass through
        if (!state_out) return FFTCONV_OK;
        return done(state_in ? cudaMemcpyAsync(state_out, state_in, sb, cudaMemcpyDeviceToDevice, st)
                             : cudaMemsetAsync(state_out, 0, sb, st));
    }
    a.state_in = state_in;
    a.state_out = state_out;
    if (w.c.slots >= (int64_t(1) << 30) / d.Hv) return FFTCONV_ERR_UNSUPPORTED;
    a.slots = w.c.slots;
    a.segments = w.c.segments;
    a.seg_chunks = w.c.seg_chunks;
    a.sms = p->num_sms;
    a.images = static_cast<uint8_t*>(saved ? saved : scratch);
    a.seg_state = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + w.state);
    a.seg_trans = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + w.trans);
    if (saved) {
        const SavedLayout l(p, d.B, d.T, d.Hv, d.nseq);
        a.saved_s = a.images + l.s;
        a.saved_v = a.images + l.v;
        a.saved_t = a.images + l.t;
    }
    if (!encode_tokens_map(&a.mq, d.q, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mk, d.k, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mv, d.v, d.B, d.T, d.Hv, p->Dv, p->dtype))
        return FFTCONV_ERR_UNSUPPORTED;
    cudaError_t c = cudaSuccess;
    if (d.offsets) c = zero_gaps(d, 1, &d.o, &d.Hv, &p->Dv, st);
    if (c == cudaSuccess && d.nseq) c = launch_delta_forward(a, p->dtype, p->Dk, p->Dv, st);
    return done(c);
}

extern "C" fftconv_status_t fftconv_delta_backward(fftconv_delta_t p, const fftconv_delta_args_t* args,
                                                   fftconv_view_t d_o, const float* d_state_out, const void* saved,
                                                   fftconv_view_t dq, fftconv_view_t dk, fftconv_view_t dv,
                                                   fftconv_view_t dg, fftconv_view_t dbeta, float* d_state_in,
                                                   void* scratch, size_t scratch_bytes, fftconv_stream_t stream) {
    GradArgs a{};
    fftconv_status_t e = take_args(p, args, &a.d);
    if (e != FFTCONV_OK) return e;
    const DeltaArgs& d = a.d;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d.Hv == 0) {  // no value head uses the queries and keys
        if (!d.B || !d.T || !d.Hk) return FFTCONV_OK;
        View v[2];
        if ((e = take_view(dq, d.B, d.T, d.Hk, p->Dk, &v[0])) != FFTCONV_OK) return e;
        if ((e = take_view(dk, d.B, d.T, d.Hk, p->Dk, &v[1])) != FFTCONV_OK) return e;
        const int H[2] = {d.Hk, d.Hk}, D[2] = {p->Dk, p->Dk};
        a.d.nseq = 0;
        return done(zero_gaps(d, 2, v, H, D, st));
    }
    if (d.nseq == 0 && !d.offsets) return FFTCONV_OK;
    if (off16(d_state_out) || off16(d_state_in) || off16(saved) || off16(scratch)) return FFTCONV_ERR_ALIGN;
    const size_t sb = state_bytes(p, d.nseq, d.Hv);
    const bool any = d.B && d.T;
    if (!any) {
        if (!d_state_in) return FFTCONV_OK;
        if (meets(span_of(d_state_in, sb), span_of(d_state_out, sb))) return FFTCONV_ERR_INVALID;
        return done(d_state_out ? cudaMemcpyAsync(d_state_in, d_state_out, sb, cudaMemcpyDeviceToDevice, st)
                                : cudaMemsetAsync(d_state_in, 0, sb, st));
    }
    if (!saved) return FFTCONV_ERR_INVALID;
    const size_t need = fftconv_delta_scratch_bytes(p, d.B, d.T, d.Hk, d.Hv, d.nseq, 1);
    if (need && (!scratch || scratch_bytes < need)) return FFTCONV_ERR_WORKSPACE;
    View vdo;
    if ((e = take_view(d_o, d.B, d.T, d.Hv, p->Dv, &vdo)) != FFTCONV_OK) return e;
    if ((e = take_view(dq, d.B, d.T, d.Hk, p->Dk, &a.dq)) != FFTCONV_OK) return e;
    if ((e = take_view(dk, d.B, d.T, d.Hk, p->Dk, &a.dk)) != FFTCONV_OK) return e;
    if ((e = take_view(dv, d.B, d.T, d.Hv, p->Dv, &a.dv)) != FFTCONV_OK) return e;
    if ((e = take_view(dg, d.B, d.T, d.Hv, 0, &a.dg)) != FFTCONV_OK) return e;
    if ((e = take_view(dbeta, d.B, d.T, d.Hv, 0, &a.dbeta)) != FFTCONV_OK) return e;
    Span in[6];
    input_spans(p, d, in);
    const Span more[3] = {span_of(vdo, d.B, d.T, d.Hv, p->Dv), span_of(d_state_out, sb),
                          span_of(saved, fftconv_delta_saved_bytes(p, d.B, d.T, d.Hv, d.nseq))};
    // tokens' gradients may be slices of one buffer, so they are not checked against each other
    const Span outs[7] = {span_of(a.dq, d.B, d.T, d.Hk, p->Dk), span_of(a.dk, d.B, d.T, d.Hk, p->Dk),
                          span_of(a.dv, d.B, d.T, d.Hv, p->Dv), span_of(a.dg, d.B, d.T, d.Hv, 0),
                          span_of(a.dbeta, d.B, d.T, d.Hv, 0), span_of(d_state_in, sb), span_of(scratch, need)};
    if (any_meet(outs, in) || any_meet(outs, more)) return FFTCONV_ERR_INVALID;
    for (int i = 5; i < 7; ++i)  // the state's gradient and scratch overlap nothing
        for (int j = 0; j < i; ++j)
            if (meets(outs[i], outs[j])) return FFTCONV_ERR_INVALID;
    a.d_state_out = d_state_out;
    a.d_state_in = d_state_in;
    const SavedLayout l(p, d.B, d.T, d.Hv, d.nseq);
    a.images = static_cast<const uint8_t*>(saved);
    a.saved_s = a.images + l.s;
    a.saved_v = a.images + l.v;
    a.saved_t = a.images + l.t;
    const BwdScratch w(p, d.B, d.T, d.Hk, d.Hv, d.nseq);
    a.ds = static_cast<uint8_t*>(scratch);
    a.dr = a.ds + w.r;
    if (d.group > 1) {
        a.dqh = reinterpret_cast<float*>(a.ds + w.q);
        a.dkh = reinterpret_cast<float*>(a.ds + w.k);
    }
    a.slots = chunk_slots(d.B, d.T, d.nseq);
    a.sms = p->num_sms;
    if (a.slots >= (int64_t(1) << 30) / d.Hv) return FFTCONV_ERR_UNSUPPORTED;
    if (!encode_tokens_map(&a.mq, d.q, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mk, d.k, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mv, d.v, d.B, d.T, d.Hv, p->Dv, p->dtype) ||
        !encode_tokens_map(&a.mo, vdo, d.B, d.T, d.Hv, p->Dv, p->dtype) ||
        !encode_tokens_map(&a.mdq, a.dq, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mdk, a.dk, d.B, d.T, d.Hk, p->Dk, p->dtype) ||
        !encode_tokens_map(&a.mdv, a.dv, d.B, d.T, d.Hv, p->Dv, p->dtype))
        return FFTCONV_ERR_UNSUPPORTED;
    cudaError_t c = cudaSuccess;
    if (d.offsets) {
        const View zs[5] = {a.dq, a.dk, a.dv, a.dg, a.dbeta};
        const int zh[5] = {d.Hk, d.Hk, d.Hv, d.Hv, d.Hv}, zd[5] = {p->Dk, p->Dk, p->Dv, 1, 1};
        // with shared heads dq and dk are summed from float32 parts, zero in the gaps
        if (a.dqh) c = cudaMemsetAsync(a.dqh, 0, w.total - w.q, st);
        if (c == cudaSuccess) c = zero_gaps(d, 5, zs, zh, zd, st);
    }
    if (c == cudaSuccess && d.nseq) c = launch_delta_backward(a, p->dtype, p->Dk, p->Dv, st);
    return done(c);
}

extern "C" fftconv_status_t fftconv_delta_step(fftconv_delta_t p, const fftconv_delta_args_t* args,
                                               const float* state_in, float* state_out, int64_t nslots,
                                               const int32_t* slots, fftconv_view_t o, fftconv_stream_t stream) {
    TokenArgs a{};
    fftconv_status_t e = take_args(p, args, &a.d);
    if (e != FFTCONV_OK) return e;
    const DeltaArgs& d = a.d;
    if (d.offsets || nslots < 0 || (!slots && nslots < d.B)) return FFTCONV_ERR_INVALID;
    if (d.B == 0 || d.T == 0 || d.Hv == 0) return FFTCONV_OK;
    if (!state_in || !state_out) return FFTCONV_ERR_INVALID;
    if (off16(state_in) || off16(state_out) || (reinterpret_cast<uintptr_t>(slots) & 3)) return FFTCONV_ERR_ALIGN;
    if ((e = take_view(o, d.B, d.T, d.Hv, p->Dv, &a.d.o)) != FFTCONV_OK) return e;
    const size_t sb = state_bytes(p, nslots, d.Hv);
    Span in[6];
    input_spans(p, d, in);
    const Span outs[2] = {span_of(d.o, d.B, d.T, d.Hv, p->Dv), span_of(state_out, sb)};
    const Span more[2] = {span_of(slots, size_t(d.B) * 4), state_in == state_out ? Span{} : span_of(state_in, sb)};
    if (any_meet(outs, in) || any_meet(outs, more) || meets(outs[0], outs[1]) || meets(outs[0], span_of(state_in, sb)))
        return FFTCONV_ERR_INVALID;
    a.sin = state_in;
    a.sout = state_out;
    a.slots = slots;
    a.nslots = nslots;
    return done(pick(p->dtype, p->Dk, p->Dv, LaunchToken{a, static_cast<cudaStream_t>(stream)}));
}
