// Gated delta rule over whole sequences, 64 tokens at a time, on the
// fifth-generation tensor cores.
//
// Per chunk, with b the running sum of the log decays, G_i = exp(b_i),
// D_ij = exp(b_i - b_j), e_j = exp(b_63 - b_j):
//   A_ij = beta_i D_ij k_i.k_j (i > j),  T = (I + A)^-1
//   U = (T beta) V,  W = (T beta G) K           (columns of T scaled)
//   Vn = U - W S                                (the corrected values)
//   O = scale G (Q S) + P Vn,  P_ij = scale D_ij q_i.k_j (i >= j)
//   S <- G_63 S + (e Vn)^T K
// Only S goes from chunk to chunk.  Everything is held transposed (features
// of V in the tensor-memory lanes): S^T, Vn^T and O^T are accumulators whose
// lanes one thread owns, so S^T and Vn^T go back as A operands in tensor
// memory without passing through shared memory, and K, Q, V stay the tiles
// that the TMA engine wrote (tile.cuh).
//
// Precision: the state is float32; products that feed it take it, W, T and
// (e Vn) as two 16-bit values each (high and low part; the low x low product
// is dropped), so the state is good to about 2^-17 per chunk while K and V are
// exact.  Products that only feed O (Q S, P Vn) take one 16-bit value: O is
// rounded to 16 bits anyway.
//
// One CTA per sequence and value head; roles by warp, handing tiles over
// through mbarriers:
//   warps 0-3   chain: S (float32 -> operands, decayed in place) and Vn
//   warps 4-7   W^T -> operand in shared memory; O^T -> global memory
//   warps 8-11  T: A from K K^T, the triangular inverse, P from Q K^T
//   warp 12     issues every contraction;  warp 13  loads
#include "delta_chunk.h"

#include "tile.cuh"

namespace fftconv {
namespace {

using namespace tile;

template <int DK_, int DV_>
struct FwdCfg {
    static constexpr int DK = DK_;
    static constexpr int NKQ = 3;                          // stages of K and Q
    static constexpr uint32_t KQ = (DK / 64) * 2 * kTile;  // [feature block][K rows | Q rows]
    static constexpr uint32_t VB = 2 * kTile;              // DV = 64: the same block twice (M = 128)
    static constexpr uint32_t WB = DK * 128;               // W^T: DK rows of 64 tokens, per part
    static constexpr int LD = 68;                          // row pitch of the float32 64 x 64 scratch
    static constexpr uint32_t oKQ = 0, oV = oKQ + NKQ * KQ, oW = oV + VB, oT = oW + 2 * WB, oP = oT + 4 * kTile,
                              oA = oP + 2 * kTile, oG = oA + 64 * LD * 4, oL = oG + 4 * 132 * 4, oBar = oL + 3 * 64 * 4,
                              BYTES = oBar + 256;
    static constexpr int THREADS = 448;
    // tensor memory columns
    static constexpr uint32_t cS = 0, cHi = 128, cLo = 128 + DK / 2, cVeH = 128, cVeL = 160, cVnH = 192, cVn = 256,
                              cOS = 320, cKK = 384, cW = 448;
};

enum Bar {
    kKqFull = 0, kKqFree = 3, kVFull = 6, kRaw, kKkDone, kKkFree, kTReady, kUDone, kWtDone, kWReady, kSwDone, kSqDone,
    kVnReady, kOpRead, kSDone, kSReady, kFinal,
    kOpDone,             // [2], by chunk parity: T's warps may look back two chunks
    kGates = kOpDone + 2,  // [4], by ring slot: written up to three chunks ahead of the chain
    kBars = kGates + 4
};

constexpr uint32_t kWaitFinal = 1u << 18;  // polls of the waits that end a CTA

// T = (I + A)^-1 in place, A strictly lower triangular 64 x 64 (float32, row
// pitch LD), by 128 threads.  The four 16 x 16 diagonal blocks by forward
// substitution (a thread per column), then blocks of 32 and of 64 from
// T21 = -T22 (A21 T11): exact arithmetic of a triangular solve, no powers of A
// (which grow like binomials when keys are alike).  Intermediate products sit
// in the unused blocks above the diagonal, which are left undefined.
template <int LD, typename Sync>
__device__ __forceinline__ void inverse64(float* A, int p, Sync sync) {
    if (p < 64) {
        float* base = A + (p >> 4) * 16 * (LD + 1);
        const int col = p & 15;
        float x[16];
        #pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s0 = r == col ? 1.0f : 0.0f, s1 = 0.0f;
            #pragma unroll
            for (int k = 0; k < r; k += 4) {
                const float4 v = *reinterpret_cast<const float4*>(base + r * LD + k);
                s0 = fmaf(-v.x, x[k], s0);
                if (k + 1 < r) s1 = fmaf(-v.y, x[k + 1], s1);
                if (k + 2 < r) s0 = fmaf(-v.z, x[k + 2], s0);
                if (k + 3 < r) s1 = fmaf(-v.w, x[k + 3], s1);
            }
            x[r] = s0 + s1;
        }
        __syncwarp();
        #pragma unroll
        for (int r = 0; r < 16; ++r) base[r * LD + col] = x[r];
    }
    sync();
    {
        const int q = (p >> 6) * 32, r = (p & 63) >> 2, c = (p & 3) * 4;
        const float *A21 = A + (q + 16 + r) * LD + q, *T11 = A + q * LD + q + c;
        float* M = A + q * LD + q + 16 + c;
        const float* T22 = A + (q + 16 + r) * LD + q + 16;
        float4 m = make_float4(0, 0, 0, 0);
        #pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float x = A21[k];
            const float4 t = *reinterpret_cast<const float4*>(T11 + k * LD);
            m.x = fmaf(x, t.x, m.x); m.y = fmaf(x, t.y, m.y); m.z = fmaf(x, t.z, m.z); m.w = fmaf(x, t.w, m.w);
        }
        *reinterpret_cast<float4*>(M + r * LD) = m;
        sync();
        m = make_float4(0, 0, 0, 0);
        #pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float x = -T22[k];
            const float4 t = *reinterpret_cast<const float4*>(M + k * LD);
            m.x = fmaf(x, t.x, m.x); m.y = fmaf(x, t.y, m.y); m.z = fmaf(x, t.z, m.z); m.w = fmaf(x, t.w, m.w);
        }
        *reinterpret_cast<float4*>(A + (q + 16 + r) * LD + q + c) = m;
        sync();
    }
    {
        const int r = p >> 3, c = (p & 7) * 4, k0 = c & 16;  // T11 is zero above its diagonal blocks
        const float *A21 = A + (32 + r) * LD, *T11 = A + c, *T22 = A + (32 + r) * LD + 32;
        float* M = A + 32 + c;
        float4 m = make_float4(0, 0, 0, 0), n = m;
        #pragma unroll 8
        for (int k = k0; k < 32; ++k) {
            const float x = A21[k], y = A21[16 * LD + k];
            const float4 t = *reinterpret_cast<const float4*>(T11 + k * LD);
            m.x = fmaf(x, t.x, m.x); m.y = fmaf(x, t.y, m.y); m.z = fmaf(x, t.z, m.z); m.w = fmaf(x, t.w, m.w);
            n.x = fmaf(y, t.x, n.x); n.y = fmaf(y, t.y, n.y); n.z = fmaf(y, t.z, n.z); n.w = fmaf(y, t.w, n.w);
        }
        *reinterpret_cast<float4*>(M + r * LD) = m;
        *reinterpret_cast<float4*>(M + (r + 16) * LD) = n;
        sync();
        m = n = make_float4(0, 0, 0, 0);
        #pragma unroll 8
        for (int k = 0; k < 32; ++k) {
            const float x = k < 16 ? -T22[k] : 0.0f, y = -T22[16 * LD + k];
            const float4 t = *reinterpret_cast<const float4*>(M + k * LD);
            m.x = fmaf(x, t.x, m.x); m.y = fmaf(x, t.y, m.y); m.z = fmaf(x, t.z, m.z); m.w = fmaf(x, t.w, m.w);
            n.x = fmaf(y, t.x, n.x); n.y = fmaf(y, t.y, n.y); n.z = fmaf(y, t.z, n.z); n.w = fmaf(y, t.w, n.w);
        }
        *reinterpret_cast<float4*>(A + (32 + r) * LD + c) = m;
        *reinterpret_cast<float4*>(A + (48 + r) * LD + c) = n;
        sync();
    }
}

struct Item {
    Seq s;
    int i, h, hk;
    int n;  // chunks
};

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(FwdCfg<DK, DV>::THREADS, 1)
delta_fwd_kernel(const __grid_constant__ ChunkArgs a) {
    using C = FwdCfg<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_fail;
    const DeltaArgs& d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    Item it;
    it.i = blockIdx.x;
    it.h = blockIdx.y;
    it.hk = it.h / d.group;
    it.s = locate(d.offsets, d.T, it.i);
    it.n = int((it.s.len + kChunk - 1) / kChunk);
    const int n = it.n;
    const int64_t sbase = (int64_t(it.i) * d.Hv + it.h) * DK * DV;

    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < kBars; ++i) {
            uint32_t cnt = 1;
            if (i == kKkFree || i == kTReady || i == kWReady || i == kVnReady || i == kOpRead || i == kSReady || i >= kGates)
                cnt = 4;  // one arrival per warp of the role
            mbar_init(bar + i, cnt);
        }
        fence_mbar_init();
    }
    if (warp == 12) tc::alloc(&s_tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = s_tmem;
    volatile int* fail = &s_fail;
    const uint32_t lanes = tm + (uint32_t(32 * (warp & 3)) << 16);  // this warp's tensor-memory lanes
    const int row = 32 * (warp & 3) + lane;                         // this thread's lane

    float* gates = reinterpret_cast<float*>(sm + C::oG);  // ring of 4: e[64], scale G[64], G_63
    // one arrival per warp, after every lane's work
    auto done = [&](Bar b) {
        __syncwarp();
        if (lane == 0) arrive(bar + b);
    };

    if (n == 0) {
        // an empty sequence: the state passes through
        if (a.state_out)
            for (int x = threadIdx.x; x < DK * DV; x += C::THREADS)
                a.state_out[sbase + x] = a.state_in ? a.state_in[sbase + x] : 0.0f;
    } else if (warp < 4) {
        // ---------------------------------------------------------------- chain
        const int dv = row % DV;
        const bool mine = row < DV;
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            const float* gt = gates + (c & 3) * 132;
            if (!(ok = wait(bar + kGates + (c & 3), (c >> 2) & 1, fail))) break;
            const float gc = gt[128];
            if (c > 0) {
                if (!(ok = wait(bar + kSDone, (c - 1) & 1, fail))) break;
                tc::fence_after();
            }
            uint16_t* sv = a.saved_s ? a.saved_s + (((it.s.slot + c) * d.Hv + it.h) * DV + dv) * DK : nullptr;
            #pragma unroll
            for (int k0 = 0; k0 < DK; k0 += 32) {
                uint32_t x[32], hi[16], lo[16];
                if (c > 0) {
                    tc::ld32x32b_x32(lanes + C::cS + k0, x);
                    tc::wait_ld();
                } else {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j)
                        x[j] = a.state_in ? __float_as_uint(a.state_in[sbase + (k0 + j) * DV + dv]) : 0u;
                }
                #pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x0 = __uint_as_float(x[2 * j]), x1 = __uint_as_float(x[2 * j + 1]);
                    split<DT>(x0, x1, &hi[j], &lo[j]);
                    x[2 * j] = __float_as_uint(gc * x0);
                    x[2 * j + 1] = __float_as_uint(gc * x1);
                }
                tc::st16(lanes + C::cHi + k0 / 2, hi);
                tc::st16(lanes + C::cLo + k0 / 2, lo);
                st32(lanes + C::cS + k0, x);
                if (sv && mine) {
                    #pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        *reinterpret_cast<uint4*>(sv + k0 + 2 * j) = make_uint4(hi[j], hi[j + 1], hi[j + 2], hi[j + 3]);
                }
            }
            tc::wait_st();
            tc::fence_before();
            done(kSReady);
            // Vn^T = U^T - S^T W^T
            if (!(ok = wait(bar + kSwDone, c & 1, fail))) break;
            tc::fence_after();
            uint32_t vh[32], eh[32], el[32];
            #pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 32) {
                uint32_t x[32];
                tc::ld32x32b_x32(lanes + C::cVn + j0, x);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x0 = __uint_as_float(x[2 * j]), x1 = __uint_as_float(x[2 * j + 1]);
                    const float2 e = *reinterpret_cast<const float2*>(gt + j0 + 2 * j);
                    vh[j0 / 2 + j] = Op<DT>::pack(x0, x1);
                    split<DT>(e.x * x0, e.y * x1, &eh[j0 / 2 + j], &el[j0 / 2 + j]);
                }
            }
            // S's operands are free once Q S is done too
            if (!(ok = wait(bar + kSqDone, c & 1, fail))) break;
            st32(lanes + C::cVnH, vh);
            st32(lanes + C::cVeH, eh);
            st32(lanes + C::cVeL, el);
            tc::wait_st();
            tc::fence_before();
            done(kVnReady);
            if (a.saved_v && mine) {
                uint16_t* p = a.saved_v + (((it.s.slot + c) * d.Hv + it.h) * DV + dv) * 64;
                #pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4*>(p + 2 * j) = make_uint4(vh[j], vh[j + 1], vh[j + 2], vh[j + 3]);
            }
        }
        if (ok) ok = wait(bar + kSDone, (n - 1) & 1, fail);
        if (ok && a.state_out) {
            tc::fence_after();
            #pragma unroll
            for (int k0 = 0; k0 < DK; k0 += 32) {
                uint32_t x[32];
                tc::ld32x32b_x32(lanes + C::cS + k0, x);
                tc::wait_ld();
                if (mine) {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j) a.state_out[sbase + (k0 + j) * DV + dv] = __uint_as_float(x[j]);
                }
            }
        }
        if (!ok) s_fail = 1;
    } else if (warp < 8) {
        // ---------------------------------------------------------------- W^T and O^T
        bool ok = true;
        auto do_w = [&](int c) {  // W^T of chunk c -> shared memory
            if (!wait(bar + kWtDone, c & 1, fail)) return false;
            tc::fence_after();
            uint32_t hi[32], lo[32];
            #pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 32) {
                uint32_t x[32];
                tc::ld32x32b_x32(lanes + C::cW + j0, x);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 16; ++j)
                    split<DT>(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]), &hi[j0 / 2 + j], &lo[j0 / 2 + j]);
            }
            tc::fence_before();
            if (c > 0 && !wait(bar + kSwDone, (c - 1) & 1, fail)) return false;
            if (row < DK) {
                uint8_t* p = sm + C::oW + row * 128;
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = (j ^ (row & 7)) * 16;
                    *reinterpret_cast<uint4*>(p + at) = make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
                    *reinterpret_cast<uint4*>(p + C::WB + at) =
                        make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
                }
            }
            tc::fence_proxy_async();
            done(kWReady);
            return true;
        };
        auto do_o = [&](int c) {  // O^T of chunk c -> global memory
            if (!wait(bar + kOpDone + (c & 1), (c >> 1) & 1, fail)) return false;
            tc::fence_after();
            const float* sg = gates + (c & 3) * 132 + 64;
            uint32_t o[32];
            #pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 32) {
                uint32_t x[32], y[32];
                tc::ld32x32b_x32(lanes + C::cOS + j0, x);
                tc::ld32x32b_x32(lanes + C::cVn + j0, y);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 g = *reinterpret_cast<const float2*>(sg + j0 + 2 * j);
                    o[j0 / 2 + j] = Op<DT>::pack(fmaf(g.x, __uint_as_float(x[2 * j]), __uint_as_float(y[2 * j])),
                                                 fmaf(g.y, __uint_as_float(x[2 * j + 1]), __uint_as_float(y[2 * j + 1])));
                }
            }
            tc::fence_before();
            done(kOpRead);
            if (row < DV) {
                const int64_t t0 = it.s.start + int64_t(c) * kChunk;
                const int m = int(it.s.len - int64_t(c) * kChunk < kChunk ? it.s.len - int64_t(c) * kChunk : kChunk);
                uint16_t* p = reinterpret_cast<uint16_t*>(d.o.p) + it.s.row * d.o.b + t0 * d.o.t + it.h * d.o.h + row;
                if (m == kChunk) {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        p[(2 * j) * d.o.t] = uint16_t(o[j] & 0xffffu);
                        p[(2 * j + 1) * d.o.t] = uint16_t(o[j] >> 16);
                    }
                } else {
                    #pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (2 * j < m) p[(2 * j) * d.o.t] = uint16_t(o[j] & 0xffffu);
                        if (2 * j + 1 < m) p[(2 * j + 1) * d.o.t] = uint16_t(o[j] >> 16);
                    }
                }
            }
            return true;
        };
        ok = do_w(0);
        for (int c = 0; ok && c < n; ++c) {
            bool w = c + 1 >= n;
            // whichever came first; all four warps see the same completed phases
            // eventually, and each warp's own order does not matter to the others
            if (!w && test(bar + kWtDone, (c + 1) & 1)) {
                if (!(ok = do_w(c + 1))) break;
                w = true;
            }
            if (!(ok = do_o(c))) break;
            if (!w) ok = do_w(c + 1);
        }
        if (!ok) s_fail = 1;
    } else if (warp < 12) {
        // ---------------------------------------------------------------- T and P
        const int p = threadIdx.x - 256;
        float* A = reinterpret_cast<float*>(sm + C::oA);
        float *sbv = reinterpret_cast<float*>(sm + C::oL), *sbe = sbv + 64, *sbg = sbe + 64;  // b, beta, -beta G
        auto sync = [&] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
        // the four warps meet in barriers, so they also give up together
        auto together = [&](bool mine) { return !tc::bar_vote(1, 128, !mine); };
        bool ok = true;
        float g_next = 0.0f, b_next = 0.0f;
        auto fetch = [&](int c) {  // gates of token p of chunk c (p < 64)
            const int64_t t = int64_t(c) * kChunk + p;
            if (p < 64 && t < it.s.len) {
                const int64_t at = it.s.start + t;
                g_next = load16<DT>(d.g, it.s.row * d.g.b + at * d.g.t + it.h * d.g.h);
                b_next = load16<DT>(d.beta, it.s.row * d.beta.b + at * d.beta.t + it.h * d.beta.h);
            } else {
                g_next = 0.0f;  // past the end: no decay, no update
                b_next = 0.0f;
            }
        };
        fetch(0);
        for (int c = 0; ok && c < n; ++c) {
            float* gt = gates + (c & 3) * 132;
            // running sum of the log decays over the 64 tokens (warps 8 and 9)
            float bs = log_decay(g_next);
            const float be = b_next;
            if (c + 1 < n) fetch(c + 1);
            if (p < 64) {
                #pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float v = __shfl_up_sync(0xffffffffu, bs, o);
                    if (lane >= o) bs += v;
                }
                if (p == 31) sbv[0] = bs;
            }
            sync();
            if (p >= 32 && p < 64) bs += sbv[0];
            sync();
            if (p < 64) {
                sbv[p] = bs;
                sbe[p] = be;
                const float G = expf(bs);
                sbg[p] = -be * G;
                gt[64 + p] = d.scale * G;
                if (p == 63) gt[128] = G;
            }
            sync();
            if (p < 64) gt[p] = expf(sbv[63] - bs);
            done(Bar(kGates + (c & 3)));
            // K K^T (lanes 0-63) and Q K^T (lanes 64-127)
            ok = wait(bar + kKkDone, c & 1, fail);
            // P's buffer is free once chunk c - 2's P Vn is done
            if (ok && c > 1) ok = wait(bar + kOpDone + (c & 1), ((c >> 1) - 1) & 1, fail);
            if (!(ok = together(ok))) break;
            tc::fence_after();
            const int i = row & 63;
            const bool isp = row >= 64;
            const float bi = sbv[i], f = isp ? d.scale : sbe[i];
            #pragma unroll
            for (int j0 = 0; j0 < 64; j0 += 32) {
                uint32_t x[32];
                tc::ld32x32b_x32(lanes + C::cKK + j0, x);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 bj = *reinterpret_cast<const float4*>(sbv + j0 + j);
                    const float bb[4] = {bj.x, bj.y, bj.z, bj.w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int jj = j0 + j + q;
                        const bool on = isp ? jj <= i : jj < i;
                        // off entries take exp(0): no overflow, and the product is dropped
                        const float D = __expf(on ? bi - bb[q] : 0.0f);
                        x[j + q] = on ? __float_as_uint(f * D * __uint_as_float(x[j + q])) : 0u;
                    }
                }
                if (isp) {
                    uint8_t* pp = sm + C::oP + (c & 1) * kTile + i * 128;
                    #pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
                        #pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = Op<DT>::pack(__uint_as_float(x[8 * j + 2 * q]), __uint_as_float(x[8 * j + 2 * q + 1]));
                        *reinterpret_cast<uint4*>(pp + (((j0 / 8 + j) ^ (i & 7)) * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    #pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4*>(A + i * C::LD + j0 + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
                }
            }
            tc::fence_before();
            done(kKkFree);
            sync();
            inverse64<C::LD>(A, p, sync);
            // the scaled copies of T, as two 16-bit parts; the previous chunk's are
            // free once its U is done
            if (c > 0) ok = wait(bar + kUDone, (c - 1) & 1, fail);
            if (!(ok = together(ok))) break;
            {
                const int r = p & 63, h0 = (p >> 6) * 32;
                #pragma unroll
                for (int j0 = 0; j0 < 32; j0 += 8) {
                    uint32_t w[4][4], ts[4];
                    #pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const int jj = h0 + j0 + j;
                        const float4 t = *reinterpret_cast<const float4*>(A + r * C::LD + jj);
                        const float4 x = *reinterpret_cast<const float4*>(sbe + jj);
                        const float4 y = *reinterpret_cast<const float4*>(sbg + jj);
                        // the scratch above the diagonal holds intermediate products
                        const float t0 = jj <= r ? t.x : 0.0f, t1 = jj + 1 <= r ? t.y : 0.0f,
                                    t2 = jj + 2 <= r ? t.z : 0.0f, t3 = jj + 3 <= r ? t.w : 0.0f;
                        split<DT>(t0 * x.x, t1 * x.y, &w[0][j / 2], &w[1][j / 2]);
                        split<DT>(t2 * x.z, t3 * x.w, &w[0][j / 2 + 1], &w[1][j / 2 + 1]);
                        split<DT>(t0 * y.x, t1 * y.y, &w[2][j / 2], &w[3][j / 2]);
                        split<DT>(t2 * y.z, t3 * y.w, &w[2][j / 2 + 1], &w[3][j / 2 + 1]);
                        ts[j / 2] = Op<DT>::pack(t0, t1);
                        ts[j / 2 + 1] = Op<DT>::pack(t2, t3);
                    }
                    const int at = r * 128 + ((((h0 + j0) / 8) ^ (r & 7)) * 16);
                    #pragma unroll
                    for (int m = 0; m < 4; ++m)
                        *reinterpret_cast<uint4*>(sm + C::oT + m * kTile + at) = make_uint4(w[m][0], w[m][1], w[m][2], w[m][3]);
                    if (a.saved_t)
                        *reinterpret_cast<uint4*>(a.saved_t + (((it.s.slot + c) * d.Hv + it.h) * 64 + r) * 64 + h0 + j0) =
                            make_uint4(ts[0], ts[1], ts[2], ts[3]);
                }
            }
            tc::fence_proxy_async();
            done(kTReady);
            sync();  // the scratch and the gates are rewritten next
        }
        if (!ok) s_fail = 1;
    } else if (warp == 12) {
        // ---------------------------------------------------------------- contractions
        constexpr uint32_t id64 = tc::idesc(DT, 128, 64);
        constexpr uint32_t idS = tc::idesc(DT, 128, DK) | kMnB;
        bool ok = true;
        int kk = 0;  // next chunk of K K^T
        auto kk_issue = [&] {
            const uint32_t at = sb + C::oKQ + (kk % C::NKQ) * C::KQ;
            const uint64_t d0 = sdesc(at, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int f = 0; f < DK; f += 16) {
                    const uint64_t x = adv(d0, (f / 64) * 2 * kTile + (f % 64) * 2);
                    tc::mma_ss(tm + C::cKK, x, x, id64, f > 0);  // A: 128 rows [K; Q], B: the first 64
                }
                tc::commit(bar + kKkDone);
            }
            ++kk;
        };
        auto kk_try = [&] {
            if (kk < n && test(bar + kKqFull + kk % C::NKQ, (kk / C::NKQ) & 1) &&
                (kk == 0 || test(bar + kKkFree, (kk - 1) & 1)))
                kk_issue();
        };
        auto kk_wait = [&] {
            if (!wait(bar + kKqFull + kk % C::NKQ, (kk / C::NKQ) & 1, fail)) return false;
            if (kk > 0 && !wait(bar + kKkFree, (kk - 1) & 1, fail)) return false;
            kk_issue();
            return true;
        };
        auto wt_issue = [&](int c) {  // W^T = K^T (T beta G)^T
            const uint64_t da = sdesc(sb + C::oKQ + (c % C::NKQ) * C::KQ, DK == 128 ? 2 * kTile : kTile);
            const uint64_t db = sdesc(sb + C::oT + 2 * kTile, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)
                        tc::mma_ss(tm + C::cW, adv(da, t * 128), adv(db, m * kTile + t * 2), id64 | kMnA, m + t > 0);
                tc::commit(bar + kWtDone);
            }
        };
        auto u_issue = [&](int c) {  // U^T = V^T (T beta)^T
            const uint64_t da = sdesc(sb + C::oV, kTile);
            const uint64_t db = sdesc(sb + C::oT, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)
                        tc::mma_ss(tm + C::cVn, adv(da, t * 128), adv(db, m * kTile + t * 2), id64 | kMnA, m + t > 0);
                tc::commit(bar + kUDone);
            }
        };
        ok = kk_wait() && wait(bar + kTReady, 0, fail);
        if (ok) {
            wt_issue(0);
            ok = wait(bar + kVFull, 0, fail);
            if (ok) u_issue(0);
        }
        for (int c = 0; ok && c < n; ++c) {
            kk_try();
            if (!(ok = wait(bar + kSReady, c & 1, fail) && wait(bar + kWReady, c & 1, fail))) break;
            tc::fence_after();
            {
                const uint64_t dw = sdesc(sb + C::oW, 16);
                const uint64_t dq = sdesc(sb + C::oKQ + (c % C::NKQ) * C::KQ + kTile, 16);
                if (elect()) {
                    #pragma unroll
                    for (int f = 0; f < DK; f += 16) {  // U^T - S^T W^T (W is stored negated)
                        tc::mma(tm + C::cVn, tm + C::cHi + f / 2, adv(dw, f * 128), id64 | kMnB, 1);
                        tc::mma(tm + C::cVn, tm + C::cHi + f / 2, adv(dw, C::WB + f * 128), id64 | kMnB, 1);
                        tc::mma(tm + C::cVn, tm + C::cLo + f / 2, adv(dw, f * 128), id64 | kMnB, 1);
                    }
                    tc::commit(bar + kSwDone);
                    #pragma unroll
                    for (int f = 0; f < DK; f += 16)  // S^T Q^T
                        tc::mma(tm + C::cOS, tm + C::cHi + f / 2, adv(dq, (f / 64) * 2 * kTile + (f % 64) * 2), id64, f > 0);
                    tc::commit(bar + kSqDone);
                }
            }
            bool wt = c + 1 >= n;
            // while the chain forms Vn: the next chunks' K K^T and W^T as they get ready
            uint64_t t0 = 0;
            for (uint32_t spin = 0; !test(bar + kVnReady, c & 1); ++spin) {
                kk_try();
                if (!wt && test(bar + kTReady, (c + 1) & 1)) {
                    wt_issue(c + 1);
                    wt = true;
                }
                if ((spin & 255) == 255) {
                    const uint64_t t = globaltimer_ns();
                    if (t0 == 0) t0 = t;
                    if (*fail || t - t0 > kWaitNs) {
                        ok = false;
                        break;
                    }
                }
            }
            if (!ok) break;
            tc::fence_after();
            {
                const uint64_t dp = sdesc(sb + C::oP + (c & 1) * kTile, 16);
                const uint64_t dk = sdesc(sb + C::oKQ + (c % C::NKQ) * C::KQ, 2 * kTile);
                if (elect()) {
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)  // Vn^T P^T
                        tc::mma(tm + C::cVn, tm + C::cVnH + t / 2, adv(dp, t * 2), id64, t > 0);
                    tc::commit(bar + kOpDone + (c & 1));
                    #pragma unroll
                    for (int m = 0; m < 2; ++m)
                        #pragma unroll
                        for (int t = 0; t < 64; t += 16)  // S^T += (e Vn)^T K
                            tc::mma(tm + C::cS, tm + (m ? C::cVeL : C::cVeH) + t / 2, adv(dk, t * 128), idS, 1);
                    tc::commit(bar + kSDone);
                    tc::commit(bar + kKqFree + c % C::NKQ);
                }
            }
            if (c + 1 < n) {
                while (ok && kk <= c + 1) ok = kk_wait();
                if (ok && !wt) {
                    ok = wait(bar + kTReady, (c + 1) & 1, fail);
                    if (ok) wt_issue(c + 1);
                }
                if (ok) ok = wait(bar + kOpRead, c & 1, fail) && wait(bar + kVFull, (c + 1) & 1, fail);
                if (ok) u_issue(c + 1);
            }
        }
        if (!ok) s_fail = 1;
        // everything issued is done before tensor memory is given back
        if (elect()) tc::commit(bar + kFinal);
        mbar_wait_bounded(bar + kFinal, 0, kWaitFinal);
    } else {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int c = 0;
        const int row0 = int(it.s.row);
        auto fix = [&](uint8_t* t, int m) {  // zero rows m .. 63 of a tile
            for (int x = lane; x < (64 - m) * 8; x += 32) *reinterpret_cast<uint4*>(t + m * 128 + x * 16) = make_uint4(0, 0, 0, 0);
        };
        for (; ok && c < n; ++c) {
            const int st = c % C::NKQ;
            uint8_t* kq = sm + C::oKQ + st * C::KQ;
            const int t0 = int(it.s.start) + c * kChunk;
            const int m = int(it.s.len - int64_t(c) * kChunk < kChunk ? it.s.len - int64_t(c) * kChunk : kChunk);
            // rows past the sequence: the TMA engine writes zeros past the tensor's
            // end; in a packed row they are the next sequence's and are zeroed here
            const bool tail = d.offsets && m < kChunk;
            if (c >= C::NKQ && !(ok = wait(bar + kKqFree + st, (c / C::NKQ - 1) & 1, fail))) break;
            uint64_t* full = tail ? bar + kRaw : bar + kKqFull + st;
            if (elect()) {
                mbar_expect_tx(full, C::KQ);
                #pragma unroll
                for (int f = 0; f < DK / 64; ++f) {
                    tma_load_4d(smem_u32(kq) + f * 2 * kTile, &a.mk, f * 64, it.hk, t0, row0, full);
                    tma_load_4d(smem_u32(kq) + f * 2 * kTile + kTile, &a.mq, f * 64, it.hk, t0, row0, full);
                }
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + kRaw, 0, fail))) break;
                for (int f = 0; f < 2 * DK / 64; ++f) fix(kq + f * kTile, m);
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + kKqFull + st);
            }
            if (c >= 1 && !(ok = wait(bar + kUDone, (c - 1) & 1, fail))) break;
            full = tail ? bar + kRaw : bar + kVFull;
            if (elect()) {
                mbar_expect_tx(full, C::VB);
                #pragma unroll
                for (int f = 0; f < 2; ++f)
                    tma_load_4d(sb + C::oV + f * kTile, &a.mv, DV == 128 ? f * 64 : 0, it.h, t0, row0, full);
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + kRaw, 1, fail))) break;
                for (int f = 0; f < 2; ++f) fix(sm + C::oV + f * kTile, m);
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + kVFull);
            }
        }
        if (!ok) s_fail = 1;
        // every copy has landed before the CTA leaves (bounded waits; a phase that
        // is already over returns at once)
        for (int x = c > C::NKQ ? c - C::NKQ : 0; x < c; ++x)
            mbar_wait_bounded(bar + kKqFull + x % C::NKQ, (x / C::NKQ) & 1, kWaitFinal);
        if (c > 0) mbar_wait_bounded(bar + kVFull, (c - 1) & 1, kWaitFinal);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 12) tc::dealloc(tm, 512);
    if (threadIdx.x == 0 && s_fail) atomicExch(d.err, 7);
}

template <int DT, int DK, int DV>
cudaError_t launch(const ChunkArgs& a, cudaStream_t st) {
    static PerDevice cache;
    const size_t smem = FwdCfg<DK, DV>::BYTES + 1024;
    int* slot = cache.slot();
    if (!slot) return cudaErrorInvalidDevice;
    if (!*slot) {
        cudaError_t e = cudaFuncSetAttribute(delta_fwd_kernel<DT, DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(smem));
        if (e != cudaSuccess) return e;
        *slot = 1;
    }
    delta_fwd_kernel<DT, DK, DV><<<dim3(unsigned(a.d.nseq), unsigned(a.d.Hv)), FwdCfg<DK, DV>::THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_forward(const ChunkArgs& a, int dt, int dk, int dv, cudaStream_t st) {
    if (dt == FFTCONV_F16) {
        if (dk == 64) return dv == 64 ? launch<0, 64, 64>(a, st) : launch<0, 64, 128>(a, st);
        return dv == 64 ? launch<0, 128, 64>(a, st) : launch<0, 128, 128>(a, st);
    }
    if (dk == 64) return dv == 64 ? launch<1, 64, 64>(a, st) : launch<1, 64, 128>(a, st);
    return dv == 64 ? launch<1, 128, 64>(a, st) : launch<1, 128, 128>(a, st);
}

}  // namespace fftconv
