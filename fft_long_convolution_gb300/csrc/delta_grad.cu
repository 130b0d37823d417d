// Gradients of the gated delta rule over whole sequences.
//
// With the notation of delta_chunk.cu and dO, dS' (the gradients of a chunk's
// outputs and of the state at its end):
//   dVn = P^T dO + e (K dS'),  dR = T^T dVn,
//   dS = G_63 dS' + (scale G dO)^T-weighted Q - W^T-weighted dVn
//   X = scale D . (dO Vn^T) (i >= j),  H = -D . (dR Vn^T) (i > j)
//   dQ = scale G (dO S^T) + X K,   Y = -G (dR S^T) + H K,   dV = beta dR
//   dK = beta Y + X^T Q + (beta H)^T K + e (Vn dS'^T),   dbeta = dR.V + k.Y
//   db_i = q.dQ + k.(beta Y) - k.(dK - beta Y), and at the last token also
//          sum_j k_j.(e Vn dS'^T)_j + G_63 <S, dS'>;  dg: db summed from the end
// (rows dotted; every term of db is a row of a product that is formed anyway).  A
// pair of tokens (i, j) adds X_ij q_i.k_j and beta_i H_ij k_i.k_j to db_i and takes them
// from db_j; both sides use the same rounded X, H and beta H, or what should cancel
// in dg for pairs on one side of a token would stay as rounding (keys with a cosine of
// 0.9, beta = 0.9: dg 1.5 to 2.5 u off, 4 to 6 u with beta H rounded by itself).
//
// Two kernels, as in the forward.  delta_dstate_kernel walks the chunks from
// the last to the first with dS^T as its accumulator and leaves dS'^T and dR
// for every chunk, and dV; delta_grad_kernel takes all chunks side by side.
// The state's gradient is float32; it and dVn enter the next product as two
// 16-bit parts (T^T takes differences of dVn where keys are alike), the saved
// tensors (S, Vn, T), W, P and scale G dO as one: the gradients are rounded to 16 bits
// themselves.  The gradient of the initial state is therefore no better than a 16-bit
// result (half a rounding off for ordinary keys), although it is stored as float32.
//
// Rows are not cut into segments here as the forward's are: a row's walk takes 2.4 to
// 2.6 us a chunk however few rows there are (1 x 32768 tokens, 6 heads of 128: 1.22 ms
// on 6 SMs of a training step of 1.67 ms).
#include "chunk.cuh"

namespace fftconv {
namespace {

using namespace tile;

// ------------------------------------------------------------ dS, dR, dV
//
// Roles by warp, as in delta_fwd_kernel:
//   warps 0-15   chain: dS^T (float32 -> operands, decayed in place), dVn^T, dR^T
//   warps 16-19  scale G dO -> operand
//   warp 20      issues every contraction;  warp 21  loads;  warp 22  stores dR and
//                dV;  warp 23  stores dS'
// Bound: the chain of waits within a step, as in the forward (dS's operands, K dS',
// dVn, T^T dVn, the update): 8 x 4096 tokens, 6 heads of 128, 48 CTAs: 164 us, 2.6 us
// a chunk; 16 x 1000 tokens, 12 heads of 64, 192 CTAs on 152 SMs: 77 us.
template <int DK_, int DV_>
struct BwdCfg {
    static constexpr int DK = DK_;
    static constexpr uint32_t KQ = (DK / 64) * 2 * kTile;  // [feature block][K rows | Q rows]
    static constexpr uint32_t DO = 2 * kTile;              // DV = 64: the same block twice (M = 128)
    static constexpr uint32_t WB = DK * 128;
    // of an image, two stages: P, the decays; then T.  -W^T (high part): one
    static constexpr uint32_t iE = kTile, iT = iE + 1024, IM = iT + kTile;
    static constexpr uint32_t oKQ = 0, oDO = oKQ + 2 * KQ, oDS = oDO + DO, oI = oDS + DO, oW = oI + 2 * IM, oR = oW + WB,
                              oV = oR + 2 * DV_ * 128, oSv = oV + DV_ * 128, oBar = oSv + (DK / 64) * DV_ * 128, BYTES = oBar + 256;
    static constexpr int THREADS = 768;
    // tensor memory columns
    static constexpr uint32_t cS = 0, cHi = 128, cLo = 192, cC2 = 256, cC1 = 320, cVn = 384, cVl = 416, cR = 448;
};

enum BBar {
    bKqFull = 0, bKqFree = 2, bImFull = 4, bRead = 6,  // [2] each, by step parity
    bDoFull = 8, bRaw, bDosReady, bDosFree, bC1, bC2, bSReady, bVnReady, bSDone, bR, bStReady, bStFree, bFinal, bWFull, bSvFree, bSv = bSvFree + 2,  // [2] each, by block
    bBars = bSv + 2
};

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(BwdCfg<DK, DV>::THREADS, 1)
delta_dstate_kernel(const __grid_constant__ GradArgs a) {
    using C = BwdCfg<DK, DV>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::oBar + 240);
    volatile int& s_fail = *reinterpret_cast<volatile int*>(sm + C::oBar + 244);
    const DeltaArgs& d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int si = blockIdx.x, h = blockIdx.y, hk = h / d.group;
    if (sb & 1023) {  // not with the present layout of the window
        if (threadIdx.x == 0) atomicExch(d.err, 7);
        return;
    }
    const Seq s = locate(d.offsets, d.T, si);
    const int n = int((s.len + kChunk - 1) / kChunk);
    const int64_t sbase = (int64_t(si) * d.Hv + h) * DK * DV;
    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < bBars; ++i) {
            uint32_t cnt = 1;  // else one arrival per warp of the role
            if (i == bDosReady) cnt = 4;
            if (i == bSReady || i == bVnReady || i == bStReady || i == bRead || i == bRead + 1) cnt = 16;
            if (i >= bSv) cnt = DK == 128 ? 8 : 16;
            mbar_init(bar + i, cnt);
        }
        fence_mbar_init();
    }
    if (warp == 20) tc::alloc(&s_tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *const_cast<volatile uint32_t*>(&s_tmem);
    volatile int* fail = &s_fail;
    const uint32_t lanes = tm + (uint32_t(32 * (warp & 3)) << 16);
    const int row = 32 * (warp & 3) + lane;
    auto done = [&](int b) {
        __syncwarp();
        if (lane == 0) arrive(bar + b);
    };
    auto image = [&](int c) { return sm + C::oI + (c & 1) * C::IM; };
    auto at = [&](int c) { return (s.slot + n - 1 - c) * d.Hv + h; };  // step c takes chunk n - 1 - c

    if (n == 0) {
        if (a.d_state_in)
            for (int x = threadIdx.x; x < DK * DV; x += C::THREADS)
                a.d_state_in[sbase + x] = a.d_state_out ? a.d_state_out[sbase + x] : 0.0f;
    } else if (warp < 16) {
        // ---------------------------------------------------------------- chain
        const int dv = row % DV, quarter = warp >> 2;
        const bool mine = row < DV;
        constexpr int NC = DK / 4;
        const int k0 = quarter * NC, j0 = quarter * 16;
        // dR^T of step c (two parts), and beta dR = dV, -> shared memory as [token][feature]
        auto put_r = [&](int c) {
            const float* be = reinterpret_cast<const float*>(image(c) + C::iE) + 192 + j0;
            if (!wait(bar + bR, c & 1, fail)) return false;
            tc::fence_after();
            uint32_t r[8], l[8], v[8];
            {
                uint32_t y[16];
                ld16(lanes + C::cR + j0, y);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 u = pair(y[2 * j], y[2 * j + 1]);
                    const float2 w = mul2(u, *reinterpret_cast<const float2*>(be + 2 * j));
                    split<DT>(u, &r[j], &l[j]);
                    v[j] = Op<DT>::pack(w.x, w.y);
                }
            }
            tc::fence_before();
            done(bRead + (c & 1));
            if (c > 0 && !wait(bar + bStFree, (c - 1) & 1, fail)) return false;
            if (mine) {
                uint8_t* p = sm + C::oR + (row >> 6) * kTile + ((row >> 1) & 3) * 4;
                const int piece = (row & 63) >> 3;
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t y = __shfl_xor_sync(0xffffffffu, r[j], 1), z = __shfl_xor_sync(0xffffffffu, v[j], 1);
                    const uint32_t x = __shfl_xor_sync(0xffffffffu, l[j], 1);
                    const int t = j0 + 2 * j + (row & 1);
                    uint8_t* q = p + t * 128 + ((piece ^ (t & 7)) * 16);
                    *reinterpret_cast<uint32_t*>(q) = row & 1 ? __byte_perm(y, r[j], 0x7632) : __byte_perm(r[j], y, 0x5410);
                    *reinterpret_cast<uint32_t*>(q + DV * 128) =
                        row & 1 ? __byte_perm(x, l[j], 0x7632) : __byte_perm(l[j], x, 0x5410);
                    *reinterpret_cast<uint32_t*>(q + 2 * DV * 128) =
                        row & 1 ? __byte_perm(z, v[j], 0x7632) : __byte_perm(v[j], z, 0x5410);
                }
            }
            tc::fence_proxy_async();
            done(bStReady);
            return true;
        };
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            if (!(ok = wait(bar + bImFull + (c & 1), (c >> 1) & 1, fail))) break;
            const float* gt = reinterpret_cast<const float*>(image(c) + C::iE);
            const float g63 = exp2_fast(gt[128 + 63]);
            const float2 gc = make_float2(g63, g63);
            uint32_t x[NC], hi[NC / 2], lo[NC / 2];
            if (c > 0) {
                if (!(ok = wait(bar + bSDone, (c - 1) & 1, fail))) break;
                tc::fence_after();
                ld_cols<NC>(lanes + C::cS + k0, x);
                tc::wait_ld();
            } else {
                #pragma unroll
                for (int j = 0; j < NC; ++j)
                    x[j] = a.d_state_out ? __float_as_uint(a.d_state_out[sbase + (k0 + j) * DV + dv]) : 0u;
            }
            #pragma unroll
            for (int j = 0; j < NC / 2; ++j) {
                const float2 v = pair(x[2 * j], x[2 * j + 1]), y = mul2(gc, v);
                split<DT>(v, &hi[j], &lo[j]);
                x[2 * j] = __float_as_uint(y.x);
                x[2 * j + 1] = __float_as_uint(y.y);
            }
            st_cols<NC / 2>(lanes + C::cHi + k0 / 2, hi);
            st_cols<NC / 2>(lanes + C::cLo + k0 / 2, lo);
            st_cols<NC>(lanes + C::cS + k0, x);
            tc::wait_st();
            tc::fence_before();
            done(bSReady);
            {  // dS'^T -> global memory, a block of 64 features at a time
                const int blk = k0 >> 6;
                if (c > 0 && !(ok = wait(bar + bSvFree + blk, (c - 1) & 1, fail))) break;
                if (mine) {
                    uint8_t* p = sm + C::oSv + blk * (DV * 128) + dv * 128;
                    #pragma unroll
                    for (int j = 0; j < NC / 2; j += 4)
                        *reinterpret_cast<uint4*>(p + ((((k0 & 63) / 8 + j / 4) ^ (dv & 7)) * 16)) =
                            make_uint4(hi[j], hi[j + 1], hi[j + 2], hi[j + 3]);
                }
                tc::fence_proxy_async();
                done(bSv + blk);
            }
            if (c > 0 && !(ok = put_r(c - 1))) break;
            // dVn^T = dO^T P + e (dS'^T K^T)
            if (!(ok = wait(bar + bC1, c & 1, fail) && wait(bar + bC2, c & 1, fail))) break;
            tc::fence_after();
            uint32_t vh[8], vl[8];
            {
                uint32_t y[16], z[16];
                ld16(lanes + C::cC2 + j0, y);
                ld16(lanes + C::cC1 + j0, z);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = fma2(*reinterpret_cast<const float2*>(gt + j0 + 2 * j), pair(y[2 * j], y[2 * j + 1]),
                                          pair(z[2 * j], z[2 * j + 1]));
                    split<DT>(v, &vh[j], &vl[j]);
                }
            }
            st_cols<8>(lanes + C::cVn + j0 / 2, vh);
            st_cols<8>(lanes + C::cVl + j0 / 2, vl);
            tc::wait_st();
            tc::fence_before();
            done(bVnReady);
        }
        if (ok) ok = put_r(n - 1);
        if (ok) ok = wait(bar + bSDone, (n - 1) & 1, fail);
        if (ok && a.d_state_in) {
            tc::fence_after();
            uint32_t x[NC];
            ld_cols<NC>(lanes + C::cS + k0, x);
            tc::wait_ld();
            if (mine) {
                #pragma unroll
                for (int j = 0; j < NC; ++j) a.d_state_in[sbase + (k0 + j) * DV + dv] = __uint_as_float(x[j]);
            }
        }
        if (!ok) s_fail = 1;
    } else if (warp < 20) {
        // ---------------------------------------------------------------- scale G dO
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            ok = wait(bar + bImFull + (c & 1), (c >> 1) & 1, fail) && wait(bar + bDoFull, c & 1, fail);
            if (ok && c > 0) ok = wait(bar + bDosFree, (c - 1) & 1, fail);
            if (!ok) break;
            const int r = row & 63;
            const float sg = reinterpret_cast<const float*>(image(c) + C::iE)[64 + r];
            const float2 g = make_float2(sg, sg);
            const uint32_t base = (row >> 6) * kTile + r * 128;
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t p = base + ((j ^ (r & 7)) * 16);
                const uint4 x = *reinterpret_cast<const uint4*>(sm + C::oDO + p);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[4];
                #pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const cpx u = Op<DT>::unpack(xs[q]);
                    const float2 v = mul2(make_float2(u.r, u.i), g);
                    y[q] = Op<DT>::pack(v.x, v.y);
                }
                *reinterpret_cast<uint4*>(sm + C::oDS + p) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            tc::fence_proxy_async();
            done(bDosReady);
        }
        if (!ok) s_fail = 1;
    } else if (warp == 20) {
        // ---------------------------------------------------------------- contractions
        constexpr uint32_t id64 = tc::idesc(DT, 128, 64), idK = tc::idesc(DT, 128, DK);
        bool ok = true;
        auto c1_issue = [&](int c) {  // dO^T P
            const uint64_t da = sdesc(sb + C::oDO, kTile), db = sdesc(sb + C::oI + (c & 1) * C::IM, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int t = 0; t < 64; t += 16)
                    tc::mma_ss(tm + C::cC1, adv(da, t * 128), adv(db, t * 128), id64 | kMnA | kMnB, t > 0);
                tc::commit(bar + bC1);
            }
        };
        auto c1_wait = [&](int c) {
            return wait(bar + bImFull + (c & 1), (c >> 1) & 1, fail) && wait(bar + bDoFull, c & 1, fail);
        };
        ok = c1_wait(0);
        if (ok) c1_issue(0);
        for (int c = 0; ok && c < n; ++c) {
            if (!(ok = wait(bar + bKqFull + (c & 1), (c >> 1) & 1, fail) && wait(bar + bSReady, c & 1, fail))) break;
            tc::fence_after();
            const uint32_t kq = sb + C::oKQ + (c & 1) * C::KQ, im = sb + C::oI + (c & 1) * C::IM;
            if (elect()) {
                const uint64_t dk = sdesc(kq, 16);
                #pragma unroll
                for (int f = 0; f < DK; f += 16) {  // dS'^T K^T
                    const uint64_t x = adv(dk, (f / 64) * 2 * kTile + (f % 64) * 2);
                    tc::mma(tm + C::cC2, tm + C::cHi + f / 2, x, id64, f > 0);
                    tc::mma(tm + C::cC2, tm + C::cLo + f / 2, x, id64, 1);
                }
                tc::commit(bar + bC2);
            }
            // while the chain forms dVn: dS^T += (scale G dO)^T Q
            if (!(ok = wait(bar + bDosReady, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t da = sdesc(sb + C::oDS, kTile), dq = sdesc(kq + kTile, 2 * kTile);
                #pragma unroll
                for (int t = 0; t < 64; t += 16)
                    tc::mma_ss(tm + C::cS, adv(da, t * 128), adv(dq, t * 128), idK | kMnA | kMnB, 1);
                tc::commit(bar + bDosFree);
            }
            if (!(ok = wait(bar + bWFull, c & 1, fail) && wait(bar + bVnReady, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dw = sdesc(sb + C::oW, 16);
                #pragma unroll
                for (int t = 0; t < 64; t += 16) {  // dS^T -= dVn^T W (W is stored negated)
                    tc::mma(tm + C::cS, tm + C::cVn + t / 2, adv(dw, t * 2), idK, 1);
                    tc::mma(tm + C::cS, tm + C::cVl + t / 2, adv(dw, t * 2), idK, 1);
                }
                tc::commit(bar + bSDone);
                tc::commit(bar + bKqFree + (c & 1));
            }
            if (c > 0 && !(ok = wait(bar + bRead + ((c - 1) & 1), ((c - 1) >> 1) & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dt = sdesc(im + C::iT, 16);
                #pragma unroll
                for (int t = 0; t < 64; t += 16) {  // dR^T = dVn^T T
                    tc::mma(tm + C::cR, tm + C::cVn + t / 2, adv(dt, t * 128), id64 | kMnB, t > 0);
                    tc::mma(tm + C::cR, tm + C::cVl + t / 2, adv(dt, t * 128), id64 | kMnB, 1);
                }
                tc::commit(bar + bR);
            }
            if (c + 1 < n) {
                ok = c1_wait(c + 1);
                if (ok) c1_issue(c + 1);
            }
        }
        if (!ok) s_fail = 1;
        if (elect()) tc::commit(bar + bFinal);
        mbar_wait_bounded(bar + bFinal, 0, kWaitFinal);
    } else if (warp == 21) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int c = 0;
        const int row0 = int(s.row);
        auto fix = [&](uint8_t* t, int m) {  // zero rows m .. 63 of a tile
            for (int x = lane; x < (64 - m) * 8; x += 32) *reinterpret_cast<uint4*>(t + m * 128 + x * 16) = make_uint4(0, 0, 0, 0);
        };
        for (; ok && c < n; ++c) {
            const int ch = n - 1 - c, st = c & 1, t0 = int(s.start) + ch * kChunk;
            const int64_t left = s.len - int64_t(ch) * kChunk;
            const bool tail = d.offsets && left < kChunk;  // the first step at most
            uint8_t* kq = sm + C::oKQ + st * C::KQ;
            if (c >= 2 && !(ok = wait(bar + bKqFree + st, ((c >> 1) - 1) & 1, fail))) break;
            uint64_t* full = tail ? bar + bRaw : bar + bKqFull + st;
            if (elect()) {
                mbar_expect_tx(full, C::KQ);
                #pragma unroll
                for (int f = 0; f < DK / 64; ++f) {
                    tma_load_4d(smem_u32(kq) + f * 2 * kTile, &a.mk, f * 64, hk, t0, row0, full);
                    tma_load_4d(smem_u32(kq) + f * 2 * kTile + kTile, &a.mq, f * 64, hk, t0, row0, full);
                }
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + bRaw, 0, fail))) break;
                for (int f = 0; f < 2 * DK / 64; ++f) fix(kq + f * kTile, int(left));
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + bKqFull + st);
            }
            if (c >= 2 && !(ok = wait(bar + bRead + st, ((c >> 1) - 1) & 1, fail))) break;
            if (elect()) {
                uint64_t* b = bar + bImFull + st;
                const uint8_t* src = a.images + at(c) * kImage<DK>;
                mbar_expect_tx(b, C::IM);
                bulk_g2s(image(c), src + kImgP, kTile, b);
                bulk_g2s(image(c) + C::iE, src + kImgE, 1024, b);
                bulk_g2s(image(c) + C::iT, a.saved_t + at(c) * kTile, kTile, b);
            }
            __syncwarp();
            if (c >= 1 && !(ok = wait(bar + bC1, (c - 1) & 1, fail) && wait(bar + bDosReady, (c - 1) & 1, fail))) break;
            full = tail ? bar + bRaw : bar + bDoFull;
            if (elect()) {
                mbar_expect_tx(full, C::DO);
                #pragma unroll
                for (int f = 0; f < 2; ++f)
                    tma_load_4d(sb + C::oDO + f * kTile, &a.mo, DV == 128 ? f * 64 : 0, h, t0, row0, full);
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + bRaw, 1, fail))) break;
                for (int f = 0; f < 2; ++f) fix(sm + C::oDO + f * kTile, int(left));
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + bDoFull);
            }
            if (c >= 1 && !(ok = wait(bar + bSDone, (c - 1) & 1, fail))) break;
            if (elect()) {
                mbar_expect_tx(bar + bWFull, C::WB);
                bulk_g2s(sm + C::oW, a.images + at(c) * kImage<DK> + kImgW, C::WB, bar + bWFull);
            }
            __syncwarp();
        }
        if (!ok) s_fail = 1;
        for (int x = c > 2 ? c - 2 : 0; x < c; ++x) {  // every copy has landed before the CTA leaves
            mbar_wait_bounded(bar + bKqFull + (x & 1), (x >> 1) & 1, kWaitFinal);
            mbar_wait_bounded(bar + bImFull + (x & 1), (x >> 1) & 1, kWaitFinal);
        }
        if (c > 0) {
            mbar_wait_bounded(bar + bDoFull, (c - 1) & 1, kWaitFinal);
            mbar_wait_bounded(bar + bWFull, (c - 1) & 1, kWaitFinal);
        }
    } else if (warp == 23) {
        // ---------------------------------------------------------------- dS' -> global
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            #pragma unroll
            for (int b = 0; ok && b < DK / 64; ++b) {
                if (!(ok = wait(bar + bSv + b, c & 1, fail))) break;
                if (elect()) {
                    bulk_s2g(a.ds + at(c) * (DV * DK * 2) + b * (DV * 128), sb + C::oSv + b * (DV * 128), DV * 128);
                    bulk_wait_read();
                }
                done(bSvFree + b);
            }
        }
        if (!ok) s_fail = 1;
    } else {
        // ---------------------------------------------------------------- dR, dV -> global
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            if (!(ok = wait(bar + bStReady, c & 1, fail))) break;
            const int ch = n - 1 - c;
            const int64_t left = s.len - int64_t(ch) * kChunk, t0 = s.start + int64_t(ch) * kChunk;
            if (elect()) {
                bulk_s2g(a.dr + at(c) * (2 * DV * 128), sb + C::oR, 2 * DV * 128);
                if (!(d.offsets && left < kChunk)) {  // tokens past the tensor's end are not written
                    #pragma unroll
                    for (int f = 0; f < DV / 64; ++f)
                        tma_store_4d(&a.mdv, sb + C::oV + f * kTile, f * 64, h, int(t0), int(s.row));
                }
                bulk_wait_read();
            }
            __syncwarp();
            if (d.offsets && left < kChunk) {  // a packed row goes on with the next sequence
                constexpr int NP = DV / 8;     // 16-byte pieces of a token
                uint16_t* p = reinterpret_cast<uint16_t*>(a.dv.p) + s.row * a.dv.b + t0 * a.dv.t + h * a.dv.h;
                for (int x = lane; x < int(left) * NP; x += 32) {
                    const int t = x / NP, y = x % NP;
                    *reinterpret_cast<uint4*>(p + t * a.dv.t + y * 8) = *reinterpret_cast<const uint4*>(
                        sm + C::oV + (y >> 3) * kTile + t * 128 + (((y & 7) ^ (t & 7)) * 16));
                }
            }
            done(bStFree);
        }
        if (!ok) s_fail = 1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 20) tc::dealloc(tm, 512);
    if (threadIdx.x == 0 && s_fail) atomicExch(d.err, 7);
}

// ------------------------------------------------------------ dQ, dK, dbeta, dg
//
// One chunk of one value head at a time, one CTA per SM (two for heads of 64).  Rows 0-63 of the
// M = 128 products belong to dO (and X), rows 64-127 to dR (and H); the
// products whose rows are keys are placed at rows 64-127 too (their A operand
// starts one block early: rows 0-63 are never used), so dK's parts meet in one
// thread.  Roles: warps 0-7 form X and H and the gradients' rows, warp 8 stores
// them and forms the gates' gradients, warp 9 loads (a chunk ahead, each buffer as
// soon as it has been read) and issues the products.  Bound: HBM, 181 kB read and
// 33 kB written per chunk at Dk = Dv = 128 (8 x 4096 tokens, 6 heads, 3072 chunks:
// 114 us, 5.8 TB/s; beta H as one 16-bit part, which dg does not stand, took 109).
template <int DK, int DV>
struct GradCfg {
    static constexpr uint32_t oA = 0;                      // [feature block][dO rows | dR rows]
    static constexpr uint32_t oB = oA + (DV / 64) * 2 * kTile;  // [feature block][Q rows | K rows]
    static constexpr uint32_t oV = oB + (DK / 64) * 2 * kTile;  // V
    static constexpr uint32_t oN = oV + DV * 128;          // Vn^T: DV rows of 64 tokens
    static constexpr uint32_t oS = oN + DV * 128;          // S^T: [DK / 64] blocks of DV rows
    static constexpr uint32_t oD = oS + DK * DV * 2;       // dS'^T
    static constexpr uint32_t oX = oD + DK * DV * 2;       // [X; H], then dQ
    static constexpr uint32_t oG = oX + 2 * kTile;         // beta H, high and low part, then dK
    static constexpr uint32_t oR = oG + 2 * kTile;         // dR's low part
    static constexpr uint32_t oE = oR + DV * 128, EB = 1024 + 256;  // the image's decays, two stages
    // two stages of row sums: [4][2][64], dR.V [4][64], <S, dS'> [8]
    static constexpr uint32_t oL = oE + 2 * EB, LB = (8 * 64 + 4 * 64 + 8) * 4;
    static constexpr uint32_t oItem = oL + 2 * LB, oBar = oItem + 64, BYTES = oBar + 128;
    static constexpr int THREADS = 320;
    // small heads: two CTAs per SM
    static constexpr int PER_SM = (BYTES + 1024) * 2 <= 233472 && DK == 64 ? 2 : 1;
    // bytes of the three groups of loads
    static constexpr uint32_t B0 = 4 * DV * 128 + EB, B1 = 2 * DV * DK * 2, B2 = DK * 256 + DV * 128;
    // tensor memory columns; the scores' 64 columns are taken over by E2
    static constexpr uint32_t cE1 = 0, cE2 = DK, cSc = DK, cD1 = 2 * DK, cD2 = 3 * DK, COLS = 4 * DK;
};

enum GBar {
    gLoad = 0,  // [3] groups of loads
    gScores = 3, gD1, gD2,                    // scores; D1 and E1; D2 and E2 are done
    gIn, gX, gRv, gRows, gItem, gStFree, gBars  // dO is in order; X, H, Q, K are; dR.V is done; the rows are out
};

template <int DT, int DK, int DV>
__global__ void __launch_bounds__(GradCfg<DK, DV>::THREADS, GradCfg<DK, DV>::PER_SM)
delta_grad_kernel(const __grid_constant__ GradArgs a) {
    using C = GradCfg<DK, DV>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::oBar + 112);
    volatile int& s_fail = *reinterpret_cast<volatile int*>(sm + C::oBar + 116);
    ChunkItem* items = reinterpret_cast<ChunkItem*>(sm + C::oItem);  // [2]
    const DeltaArgs& d = a.d;
    const int p = threadIdx.x, w = __shfl_sync(0xffffffffu, p / 32, 0), lane = p % 32;
    if (sb & 1023) {  // not with the present layout of the window
        if (p == 0) atomicExch(d.err, 7);
        return;
    }
    if (p == 0) {
        s_fail = 0;
        for (int i = 0; i < gBars; ++i) mbar_init(bar + i, i == gIn || i == gX || i == gRv || i == gRows ? 8 : 1);
        fence_mbar_init();
    }
    if (w == 9) tc::alloc(&s_tmem, C::COLS);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *const_cast<volatile uint32_t*>(&s_tmem);
    volatile int* fail = &s_fail;
    auto done = [&](int b) {
        __syncwarp();
        if (lane == 0) arrive(bar + b);
    };
    bool ok = true;
    uint32_t k = 0;
    if (w < 8) {
        // ---------------------------------------------------------------- rows
        const uint32_t lanes = tm + (uint32_t(32 * (w & 3)) << 16);
        const int row = 32 * (w & 3) + lane, i = row & 63, half = w >> 2;
        const bool lower = row >= 64;  // dR, H, Y, dK
        // zero rows m .. 63 of `n` tiles `step` bytes apart: in a packed row they are
        // the next sequence's (past the tensor's end the TMA engine writes zeros)
        auto fix = [&](uint32_t off, int n, uint32_t step, int m) {
            for (int x = p; x < (64 - m) * 8 * n; x += 256) {
                const int f = x / ((64 - m) * 8), y = x % ((64 - m) * 8);
                *reinterpret_cast<uint4*>(sm + off + f * step + m * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
        };
        for (;; ++k) {
            const uint32_t par = k & 1;
            if (!(ok = wait(bar + gItem, par, fail))) break;
            const ChunkItem it = items[k & 1];
            if (!it.m) break;
            const bool tail = d.offsets && it.m < kChunk;
            const float* gt = reinterpret_cast<const float*>(sm + C::oE + par * C::EB);
            float *red = reinterpret_cast<float*>(sm + C::oL + par * C::LB), *rv = red + 512, *sd = rv + 256;
            if (!(ok = wait(bar + gLoad, par, fail))) break;
            if (tail) {
                fix(C::oA, DV / 64, 2 * kTile, it.m);
                tc::fence_proxy_async();
            }
            done(gIn);
            // <S, dS'> while the scores are formed
            if (!(ok = wait(bar + gLoad + 1, par, fail))) break;
            {
                float v = 0.0f, u = 0.0f;
                #pragma unroll 4
                for (int x = p; x < DV * DK / 8; x += 256) {
                    const uint4 y = *reinterpret_cast<const uint4*>(sm + C::oS + x * 16);
                    const uint4 z = *reinterpret_cast<const uint4*>(sm + C::oD + x * 16);
                    const uint32_t ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const cpx e = Op<DT>::unpack(ys[q]), t = Op<DT>::unpack(zs[q]);
                        v = fmaf(e.r, t.r, v);
                        u = fmaf(e.i, t.i, u);
                    }
                }
                v += u;
                #pragma unroll
                for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane == 0) sd[w] = v;
            }
            ok = wait(bar + gScores, par, fail);
            if (ok && k > 0) ok = wait(bar + gStFree, par ^ 1, fail);  // the last dQ and dK have left shared memory
            if (!ok) break;
            tc::fence_after();
            // X and H: the scores times the decays; warps 0-3 columns 0-31, 4-7 the others
            {
                uint32_t x[32];
                const int j0 = half * 32;
                tc::ld32x32b_x32(lanes + C::cSc + j0, x);
                tc::wait_ld();
                const float bi = gt[128 + i], ri = gt[256 + i], f = lower ? -1.0f : d.scale, be = gt[192 + i];
                const int last = (lower ? i - 1 : i) - j0;
                uint8_t *px = sm + C::oX + row * 128, *pg = sm + C::oG + i * 128;
                #pragma unroll
                for (int j = 0; j < 32; j += 8) {
                    uint32_t u[4];
                    #pragma unroll
                    for (int q = 0; q < 8; q += 4) {
                        const float4 b = *reinterpret_cast<const float4*>(gt + 128 + j0 + j + q);
                        const float4 s = *reinterpret_cast<const float4*>(gt + 256 + j0 + j + q);
                        const float bj[4] = {b.x, b.y, b.z, b.w}, rj[4] = {s.x, s.y, s.z, s.w};
                        float v[4];
                        #pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float y = f * exp2_fast((bi - bj[r]) + (ri - rj[r])) * __uint_as_float(x[j + q + r]);
                            v[r] = j + q + r <= last ? y : 0.0f;  // above the diagonal, whatever it holds
                        }
                        u[q / 2] = Op<DT>::pack(v[0], v[1]);
                        u[q / 2 + 1] = Op<DT>::pack(v[2], v[3]);
                    }
                    const int pos = (((j0 + j) / 8) ^ (row & 7)) * 16;
                    *reinterpret_cast<uint4*>(px + pos) = make_uint4(u[0], u[1], u[2], u[3]);
                    if (lower) {
                        // beta times the rounded H, whole in two parts: a pair's term in db's
                        // row and its term in db's column cancel where neither is after t
                        uint32_t hi[4], lo[4];
                        #pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const cpx c = Op<DT>::unpack(u[q]);
                            split<DT>(mul2(make_float2(be, be), make_float2(c.r, c.i)), &hi[q], &lo[q]);
                        }
                        *reinterpret_cast<uint4*>(pg + pos) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(pg + kTile + pos) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
            }
            if (!(ok = wait(bar + gLoad + 2, par, fail))) break;
            if (tail) {
                fix(C::oB, 2 * (DK / 64), kTile, it.m);
            }
            tc::fence_proxy_async();
            tc::fence_before();
            done(gX);
            // dR.V meanwhile, with both parts of dR (dbeta is small where it cancels
            // against k.Y): a thread per row and quarter of the features
            {
                const int r = p & 63, q0 = (p >> 6) * (DV / 32);
                float v = 0.0f;
                #pragma unroll
                for (int q = q0; q < q0 + DV / 32; ++q) {
                    const int pos = r * 128 + (((q & 7) ^ (r & 7)) * 16);
                    const uint4 y = *reinterpret_cast<const uint4*>(sm + C::oA + (q >> 3) * 2 * kTile + kTile + pos);
                    const uint4 z = *reinterpret_cast<const uint4*>(sm + C::oV + (q >> 3) * kTile + pos);
                    const uint4 l = *reinterpret_cast<const uint4*>(sm + C::oR + (q >> 3) * kTile + pos);
                    const uint32_t ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w}, ls[4] = {l.x, l.y, l.z, l.w};
                    #pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const cpx u = Op<DT>::unpack(ys[t]), x = Op<DT>::unpack(zs[t]), c = Op<DT>::unpack(ls[t]);
                        v = fmaf(u.r + c.r, x.r, fmaf(u.i + c.i, x.i, v));
                    }
                }
                rv[p] = v;
            }
            done(gRv);
            if (!(ok = wait(bar + gD1, par, fail) && wait(bar + gD2, par, fail))) break;
            tc::fence_after();
            // rows of dQ (upper) and of Y and dK (lower), a half of the features per thread
            {
                const float sg = lower ? -exp2_fast(gt[128 + i]) : gt[64 + i];
                const float ej = gt[i], be = gt[192 + i];
                float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
                const int64_t tok = int64_t(it.row) * d.T + it.t0 + i;
                float* part = a.dqh ? (lower ? a.dkh : a.dqh) + (tok * d.Hv + it.h) * DK : nullptr;
                #pragma unroll 1
                for (int f0 = half * (DK / 2); f0 < (half + 1) * (DK / 2); f0 += 16) {
                    uint32_t x[16], y[16], z[16], u[16];
                    ld16(lanes + C::cD1 + f0, x);
                    ld16(lanes + C::cD2 + f0, y);
                    if (lower) {
                        ld16(lanes + C::cE1 + f0, z);
                        ld16(lanes + C::cE2 + f0, u);
                    }
                    tc::wait_ld();
                    // this row of Q (upper) or K (lower)
                    const uint8_t* src = sm + C::oB + (f0 >> 6) * 2 * kTile + row * 128;
                    float o[16];
                    #pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint4 t = *reinterpret_cast<const uint4*>(src + ((((f0 & 63) / 8 + q) ^ (i & 7)) * 16));
                        const uint32_t ts[4] = {t.x, t.y, t.z, t.w};
                        #pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const cpx c2 = Op<DT>::unpack(ts[r / 2]);
                            const float c = r & 1 ? c2.i : c2.r;
                            const int e = 8 * q + r;
                            const float v = fmaf(sg, __uint_as_float(x[e]), __uint_as_float(y[e]));
                            s0 = fmaf(c, v, s0);
                            if (lower) {
                                const float em = ej * __uint_as_float(z[e]), dm = __uint_as_float(u[e]) + em;
                                s1 = fmaf(c, dm, s1);
                                s2 = fmaf(c, em, s2);
                                o[e] = fmaf(be, v, dm);
                            } else {
                                o[e] = v;
                            }
                        }
                    }
                    if (part) {
                        if (i < it.m) {
                            #pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<float4*>(part + f0 + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    } else {
                        uint8_t* dst = sm + (lower ? C::oG : C::oX) + (f0 >> 6) * kTile + i * 128;
                        #pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<uint4*>(dst + ((((f0 & 63) / 8 + q) ^ (i & 7)) * 16)) =
                                make_uint4(Op<DT>::pack(o[8 * q], o[8 * q + 1]), Op<DT>::pack(o[8 * q + 2], o[8 * q + 3]),
                                           Op<DT>::pack(o[8 * q + 4], o[8 * q + 5]), Op<DT>::pack(o[8 * q + 6], o[8 * q + 7]));
                    }
                }
                float* r = red + half * 64 + i;
                if (lower) {
                    r[128] = s0;
                    r[256] = s1;
                    r[384] = s2;
                } else {
                    r[0] = s0;
                }
            }
            tc::fence_proxy_async();
            tc::fence_before();
            done(gRows);
        }
    } else if (w == 8) {
        // ---------------------------------------------------------------- dq, dk, dbeta, dg -> global
        int next = blockIdx.x;
        for (;; ++k) {
            const uint32_t par = k & 1;
            const ChunkItem it = find_item(d, int(a.slots), &next);
            if (!it.m) break;
            const bool tail = d.offsets && it.m < kChunk;
            // a decay below the least one is a constant
            bool reset[2] = {};
            #pragma unroll
            for (int u = 0; u < 2; ++u)
                if (2 * lane + u < it.m)
                    reset[u] = load16<DT>(d.g, it.row * d.g.b + (it.t0 + int64_t(2 * lane + u)) * d.g.t + it.h * d.g.h) <
                               kMinLogDecay;
            if (!(ok = wait(bar + gRows, par, fail))) break;
            if (!a.dqh) {
                if (!tail) {
                    if (elect()) {  // tokens past the tensor's end are not written
                        #pragma unroll
                        for (int f = 0; f < DK / 64; ++f) {
                            tma_store_4d(&a.mdq, sb + C::oX + f * kTile, f * 64, it.h, it.t0, it.row);
                            tma_store_4d(&a.mdk, sb + C::oG + f * kTile, f * 64, it.h, it.t0, it.row);
                        }
                    }
                    __syncwarp();
                } else {
                    constexpr int NP = DK / 8;
                    for (int x = lane; x < it.m * NP; x += 32) {
                        const int t = x / NP, y = x % NP, pos = (y >> 3) * kTile + t * 128 + (((y & 7) ^ (t & 7)) * 16);
                        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dq.p) + it.row * a.dq.b + (it.t0 + int64_t(t)) * a.dq.t +
                                                  it.h * a.dq.h + y * 8) = *reinterpret_cast<const uint4*>(sm + C::oX + pos);
                        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.dk.p) + it.row * a.dk.b + (it.t0 + int64_t(t)) * a.dk.t +
                                                  it.h * a.dk.h + y * 8) = *reinterpret_cast<const uint4*>(sm + C::oG + pos);
                    }
                }
            }
            // dbeta, and db summed from the end: tokens 2 lane and 2 lane + 1
            const float* gt = reinterpret_cast<const float*>(sm + C::oE + par * C::EB);
            const float *red = reinterpret_cast<const float*>(sm + C::oL + par * C::LB), *rv = red + 512, *sd = rv + 256;
            float db[2], last = 0.0f;
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = 2 * lane + u;
                const float ky = red[128 + j] + red[192 + j], km = red[256 + j] + red[320 + j], be = gt[192 + j];
                last += red[384 + j] + red[448 + j];
                db[u] = red[j] + red[64 + j] + be * ky - km;
                if (j < it.m)
                    store16<DT>(a.dbeta, it.row * a.dbeta.b + (it.t0 + int64_t(j)) * a.dbeta.t + it.h * a.dbeta.h,
                                rv[j] + rv[64 + j] + rv[128 + j] + rv[192 + j] + ky);
            }
            #pragma unroll
            for (int o = 16; o; o >>= 1) last += __shfl_xor_sync(0xffffffffu, last, o);
            const float dot = ((sd[0] + sd[1]) + (sd[2] + sd[3])) + ((sd[4] + sd[5]) + (sd[6] + sd[7]));
            if (lane == 31) db[1] += last + exp2_fast(gt[128 + 63]) * dot;
            float x = db[0] + db[1];
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_down_sync(0xffffffffu, x, o);
                if (lane + o < 32) x += v;
            }
            const float dg[2] = {x, x - db[0]};
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int j = 2 * lane + u;
                if (j < it.m)
                    store16<DT>(a.dg, it.row * a.dg.b + (it.t0 + int64_t(j)) * a.dg.t + it.h * a.dg.h, reset[u] ? 0.0f : dg[u]);
            }
            if (elect()) bulk_wait_read();
            done(gStFree);
        }
    } else {
        // ---------------------------------------------------------------- loads and products
        int next = blockIdx.x;
        uint32_t loads = 0;  // items whose loads are under way or done
        auto load0 = [&](const ChunkItem& it, uint32_t stage) {  // dO, dR, Vn and the decays
            if (elect()) {
                mbar_expect_tx(bar, C::B0);
                #pragma unroll
                for (int f = 0; f < DV / 64; ++f) {
                    tma_load_4d(sb + C::oA + f * 2 * kTile, &a.mo, f * 64, it.h, it.t0, it.row, bar);
                    bulk_g2s(sm + C::oA + f * 2 * kTile + kTile, a.dr + it.at * (2 * DV * 128) + f * kTile, kTile, bar);
                }
                bulk_g2s(sm + C::oR, a.dr + it.at * (2 * DV * 128) + DV * 128, DV * 128, bar);
                bulk_g2s(sm + C::oN, a.saved_v + it.at * (DV * 128), DV * 128, bar);
                bulk_g2s(sm + C::oE + stage * C::EB, a.images + it.at * kImage<DK> + kImgE, 1024, bar);
                bulk_g2s(sm + C::oE + stage * C::EB + 1024, a.images + it.at * kImage<DK> + kImgR<DK>, 256, bar);
            }
            __syncwarp();
        };
        auto load1 = [&](const ChunkItem& it) {  // S and dS'
            if (elect()) {
                mbar_expect_tx(bar + 1, C::B1);
                bulk_g2s(sm + C::oS, a.saved_s + it.at * (DV * DK * 2), DV * DK * 2, bar + 1);
                bulk_g2s(sm + C::oD, a.ds + it.at * (DV * DK * 2), DV * DK * 2, bar + 1);
            }
            __syncwarp();
        };
        auto load2 = [&](const ChunkItem& it) {  // Q, K and V
            if (elect()) {
                mbar_expect_tx(bar + 2, C::B2);
                #pragma unroll
                for (int f = 0; f < DK / 64; ++f) {
                    tma_load_4d(sb + C::oB + f * 2 * kTile, &a.mq, f * 64, it.h / d.group, it.t0, it.row, bar + 2);
                    tma_load_4d(sb + C::oB + f * 2 * kTile + kTile, &a.mk, f * 64, it.h / d.group, it.t0, it.row, bar + 2);
                }
                #pragma unroll
                for (int f = 0; f < DV / 64; ++f) tma_load_4d(sb + C::oV + f * kTile, &a.mv, f * 64, it.h, it.t0, it.row, bar + 2);
            }
            __syncwarp();
        };
        auto find = [&](uint32_t to) {  // the next item, also for the rows' warps
            const ChunkItem x = find_item(d, int(a.slots), &next);
            if (lane == 0) items[to & 1] = x;
            done(gItem);
            return x;
        };
        ChunkItem it = find(0);
        if (it.m) {
            load0(it, 0);
            load1(it);
            load2(it);
            loads = 1;
        }
        for (; it.m; ++k) {
            const uint32_t par = k & 1;
            // scores [dO; dR] Vn^T; the last rows are out of tensor memory
            ok = wait(bar + gIn, par, fail);
            if (ok && k > 0) ok = wait(bar + gRows, par ^ 1, fail);
            if (!ok) break;
            const ChunkItem nx = find(k + 1);
            tc::fence_after();
            const uint64_t da = sdesc(sb + C::oA, 16);
            if (elect()) {
                const uint64_t dn = sdesc(sb + C::oN, 16);
                #pragma unroll
                for (int f = 0; f < DV; f += 16)
                    tc::mma_ss(tm + C::cSc, adv(da, (f / 64) * 2 * kTile + (f % 64) * 2), adv(dn, f * 128),
                               tc::idesc(DT, 128, 64) | kMnB, f > 0);
                tc::commit(bar + gScores);
            }
            // D1 = [dO; dR] S^T and E1 = Vn dS'^T
            if (!(ok = wait(bar + gLoad + 1, par, fail))) break;
            tc::fence_after();
            constexpr uint32_t id = tc::idesc(DT, 128, DK) | kMnB;
            if (elect()) {
                const uint64_t ds = sdesc(sb + C::oS, DV * 128);
                const uint64_t dn = sdesc(sb + C::oV, DV * 128), dd = sdesc(sb + C::oD, DV * 128);
                #pragma unroll
                for (int f = 0; f < DV; f += 16)
                    tc::mma_ss(tm + C::cD1, adv(da, (f / 64) * 2 * kTile + (f % 64) * 2), adv(ds, f * 128), id, f > 0);
                #pragma unroll
                for (int f = 0; f < DV; f += 16)
                    tc::mma_ss(tm + C::cE1, adv(dn, f * 128), adv(dd, f * 128), id | kMnA, f > 0);
                tc::commit(bar + gD1);
            }
            // D2 = [X; H] K and E2 = X^T Q + (beta H)^T K
            if (!(ok = wait(bar + gX, par, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dx = sdesc(sb + C::oX, 16), dk = sdesc(sb + C::oB + kTile, 2 * kTile);
                // A's first 64 rows are never used and come from Q's tile
                const uint64_t du = sdesc(sb + C::oB, C::oX - C::oB), dq = sdesc(sb + C::oB, 2 * kTile);
                const uint64_t dh = sdesc(sb + C::oB, C::oG - C::oB), dl = sdesc(sb + C::oB, C::oG + kTile - C::oB);
                #pragma unroll
                for (int t = 0; t < 64; t += 16)
                    tc::mma_ss(tm + C::cD2, adv(dx, t * 2), adv(dk, t * 128), id, t > 0);
                #pragma unroll
                for (int t = 0; t < 64; t += 16) {
                    tc::mma_ss(tm + C::cE2, adv(du, t * 128), adv(dq, t * 128), id | kMnA, t > 0);
                    tc::mma_ss(tm + C::cE2, adv(dh, t * 128), adv(dk, t * 128), id | kMnA, 1);
                    tc::mma_ss(tm + C::cE2, adv(dl, t * 128), adv(dk, t * 128), id | kMnA, 1);
                }
                tc::commit(bar + gD2);
            }
            if (nx.m) {
                // S and dS' (all have formed <S, dS'> before gX); dO, dR and Vn; Q, K, V
                if (!(ok = wait(bar + gD1, par, fail))) break;
                loads = k + 2;
                load1(nx);
                if (!(ok = wait(bar + gRv, par, fail))) break;
                load0(nx, par ^ 1);
                if (!(ok = wait(bar + gRows, par, fail))) break;
                load2(nx);
            }
            it = nx;
        }
        // everything issued is done and landed before the CTA leaves (bounded waits;
        // a phase that is already over returns at once)
        if (!ok && loads)
            for (int x = 0; x < 3; ++x) mbar_wait_bounded(bar + gLoad + x, (loads - 1) & 1, kWaitFinal);
        if (!ok && k > 0) mbar_wait_bounded(bar + gD2, k & 1, kWaitFinal);
    }
    if (!ok) s_fail = 1;
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (w == 9) tc::dealloc(tm, C::COLS);
    if (p == 0 && s_fail) atomicExch(d.err, 7);
}

// dq, dk [token][Hk][DK] = the sum over a key head's value heads, 8 features a thread, in the
// heads' order.  Bound: HBM (16 x 1000 tokens, 12 heads over 6 of 64: 123 MB in 22 us, 5.5 TB/s).
template <int DT>
__global__ void __launch_bounds__(256) head_sum_kernel(const float* xq, const float* xk, View yq, View yk, int64_t tokens,
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

template <int DT, int DK, int DV>
cudaError_t launch(const GradArgs& a, cudaStream_t st) {
    static PerDevice c0, c1;
    constexpr size_t sb = BwdCfg<DK, DV>::BYTES, sg = GradCfg<DK, DV>::BYTES;
    static_assert(sb <= 232448 && sg <= 232448, "shared memory");
    cudaError_t e = opt_in(delta_dstate_kernel<DT, DK, DV>, sb, c0);
    if (e == cudaSuccess) e = opt_in(delta_grad_kernel<DT, DK, DV>, sg, c1);
    if (e != cudaSuccess) return e;
    delta_dstate_kernel<DT, DK, DV><<<dim3(unsigned(a.d.nseq), unsigned(a.d.Hv)), BwdCfg<DK, DV>::THREADS, sb, st>>>(a);
    const int64_t items = a.slots * a.d.Hv;
    const int64_t most = int64_t(a.sms) * GradCfg<DK, DV>::PER_SM;
    delta_grad_kernel<DT, DK, DV><<<unsigned(items < most ? items : most), GradCfg<DK, DV>::THREADS, sg, st>>>(a);
    if (a.dqh) {
        const int64_t n = (a.d.B * a.d.T * a.d.Hk * (DK / 8) * 2 + 255) / 256;
        head_sum_kernel<DT><<<unsigned(n < 152 * 32 ? n : 152 * 32), 256, 0, st>>>(a.dqh, a.dkh, a.dq, a.dk, a.d.B * a.d.T,
                                                                                  a.d.T, a.d.Hk, a.d.group, DK);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_backward(const GradArgs& a, int dt, int dk, int dv, cudaStream_t st) {
    if (dt == FFTCONV_F16) {
        if (dk == 64) return dv == 64 ? launch<0, 64, 64>(a, st) : launch<0, 64, 128>(a, st);
        return dv == 64 ? launch<0, 128, 64>(a, st) : launch<0, 128, 128>(a, st);
    }
    if (dk == 64) return dv == 64 ? launch<1, 64, 64>(a, st) : launch<1, 64, 128>(a, st);
    return dv == 64 ? launch<1, 128, 64>(a, st) : launch<1, 128, 128>(a, st);
}

}  // namespace fftconv
