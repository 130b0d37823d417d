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
// is dropped), so the state is good to about 2^-17 per chunk (fp16: 2^-19) while K
// and V are exact.  In fp16 a low part below 2^-14 is subnormal: an entry of size x is
// good to 2^-25 / x at best (values of 1e-3: states 1e-4, outputs 2 roundings off).
// Products that only feed O (Q S, P Vn) take one 16-bit value: O is rounded to 16 bits
// anyway.
//
// Two kernels.  delta_prep_kernel forms what does not depend on S -- T, W, P
// and the decays -- for all chunks side by side, and leaves them as images of
// the shared-memory tiles that delta_fwd_kernel fetches with one bulk copy a
// chunk (58 kB at Dk = 128, next to the 49 kB of K, Q and V).  delta_fwd_kernel
// walks the chunks: one CTA per sequence (or segment of one) and value head,
// roles by warp, handing tiles over through mbarriers:
//   warps 0-15   chain: S (float32 -> operands, decayed in place), Vn and O^T, a
//                quarter of the columns for each four warps
//   warps 16-19  O -> global memory
//   warp 20      issues S W and the update of S, the two products that the walk
//                waits for;  warp 23  the others;  warp 21  loads;  warp 22
//                stores what the backward needs
// A step is a chain of waits (S's operands, S W, Vn, the update), and a wait costs
// some 200 cycles even when it is over, so what S W needs arrives on one barrier.
// That chain bounds the walk: 2 us a chunk at Dk = Dv = 128 while few CTAs walk
// (8 x 4096 tokens, 6 heads, 48 CTAs: 130 us; 149 us when it also stores what the
// backward needs), of which the products take 1 us and the conversions of S, two
// parts of 16384 values, 0.3 us of the four schedulers.  Where segments fill the SMs
// (262144 tokens, 6 heads of 128, 24576 chunks) the outputs' walks are bound by HBM: 450
// us, 108 kB read and 16 kB written a chunk, 6.8 TB/s, a copy's rate.  The states' walks
// are bound by both: 282 CTAs take two waves of 164 chunks, 1.8 us a chunk, and move
// 126 kB a chunk (83 the state, 50 the transition, none for the last segments) in 592
// us, 5.2 TB/s.
#include "delta_chunk.h"

#include "chunk.cuh"

namespace fftconv {
namespace {

using namespace tile;

// One 16 x 8 tile of a float32 product X Y over k0 <= k < k1 (multiples of 8)
// by one warp, as three products of 10-bit parts (hi hi + hi lo + lo hi: about
// 2^-20 per product).  X, Y row-major with pitch LD; acc as the MMA's C.
template <int LD>
__device__ __forceinline__ void tile_product(float (&acc)[4], const float* X, const float* Y, int k0, int k1, int lane) {
    const int g = lane >> 2, t = lane & 3;
    for (int k = k0; k < k1; k += 8) {
        const float x[4] = {X[g * LD + k + t], X[(g + 8) * LD + k + t], X[g * LD + k + t + 4], X[(g + 8) * LD + k + t + 4]};
        const float y[2] = {Y[(k + t) * LD + g], Y[(k + t + 4) * LD + g]};
        uint32_t xh[4], xl[4], yh[2], yl[2];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            xh[i] = __float_as_uint(x[i]) & 0xffffe000u;
            xl[i] = __float_as_uint(x[i] - __uint_as_float(xh[i]));
        }
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            yh[i] = __float_as_uint(y[i]) & 0xffffe000u;
            yl[i] = __float_as_uint(y[i] - __uint_as_float(yh[i]));
        }
        auto mma = [&](const uint32_t (&p)[4], const uint32_t (&q)[2]) {
            asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                : "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(q[0]), "r"(q[1]));
        };
        mma(xh, yh);
        mma(xh, yl);
        mma(xl, yh);
    }
}

// Store a 16 x 8 tile, times sgn.
template <int LD>
__device__ __forceinline__ void tile_store(float* Z, const float (&acc)[4], float sgn, int lane) {
    const int g = lane >> 2, t = lane & 3;
    *reinterpret_cast<float2*>(Z + g * LD + 2 * t) = make_float2(sgn * acc[0], sgn * acc[1]);
    *reinterpret_cast<float2*>(Z + (g + 8) * LD + 2 * t) = make_float2(sgn * acc[2], sgn * acc[3]);
}

// T = (I + A)^-1 in place, A strictly lower triangular 64 x 64 (float32, row
// pitch LD), by 256 threads (w: warp, p: thread).  The eight 8 x 8 diagonal
// blocks by forward substitution (a thread per column), then blocks of 16, 32
// and 64 from T21 = -T22 (A21 T11): a triangular solve, with no powers of A
// (which grow like binomials when keys are alike).  The products are small (up
// to 32 x 32 x 32) and wait on one another, so the larger ones run on the
// warp-level tensor path with split operands.  Intermediate products sit in
// the unused blocks above the diagonal, which are left undefined.
template <int LD, typename Sync>
__device__ __forceinline__ void inverse64(float* A, int p, int w, int lane, Sync sync) {
    if (p < 64) {
        float* base = A + (p >> 3) * 8 * (LD + 1);
        const int col = p & 7;
        float x[8];
        #pragma unroll
        for (int r = 0; r < 8; ++r) {
            float s = r == col ? 1.0f : 0.0f;
            #pragma unroll
            for (int k = 0; k < r; ++k) s = fmaf(-base[r * LD + k], x[k], s);
            x[r] = s;
        }
        __syncwarp();
        #pragma unroll
        for (int r = 0; r < 8; ++r) base[r * LD + col] = x[r];
    }
    sync();
    {
        const int q = (p >> 6) * 16, r = (p >> 3) & 7, c = p & 7;
        float* T11 = A + q * (LD + 1);
        const float* A21 = T11 + (8 + r) * LD;
        float m = 0.0f;
        #pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaf(A21[k], T11[k * LD + c], m);
        T11[r * LD + 8 + c] = m;
        sync();
        m = 0.0f;
        #pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaf(-A21[8 + k], T11[k * LD + 8 + c], m);
        T11[(8 + r) * LD + c] = m;
        sync();
        T11[r * LD + 8 + c] = 0.0f;
    }
    sync();
    {
        const int q = (w >> 1) * 32, n0 = (w & 1) * 8;
        float* M = A + q * LD + q + 16 + n0;
        float* A21 = A + (q + 16) * LD + q;
        if (w < 4) {
            float acc[4] = {};
            tile_product<LD>(acc, A21, A + q * LD + q + n0, 0, 16, lane);
            tile_store<LD>(M, acc, 1.0f, lane);
        }
        sync();
        if (w < 4) {
            float acc[4] = {};
            tile_product<LD>(acc, A21 + 16, M, 0, 16, lane);
            tile_store<LD>(A21 + n0, acc, -1.0f, lane);
        }
        sync();
    }
    {
        // T11 is zero above its diagonal blocks, T22 too
        const int m0 = (w & 1) * 16, n0 = (w >> 1) * 8;
        float* M = A + 32 + n0;
        float acc[4] = {};
        tile_product<LD>(acc, A + (32 + m0) * LD, A + n0, n0 & 16, 32, lane);
        tile_store<LD>(M + m0 * LD, acc, 1.0f, lane);
        sync();
        float acd[4] = {};
        tile_product<LD>(acd, A + (32 + m0) * LD + 32, M, 0, m0 + 16, lane);
        tile_store<LD>(A + (32 + m0) * LD + n0, acd, -1.0f, lane);
        sync();
    }
}


// Segment slot -> sequence and segment, by the same rule on the chunk slots.
__device__ __forceinline__ bool find_segment(const DeltaArgs& d, int64_t L, int64_t slot, Seq* s, int* i, int64_t* seg) {
    int lo = 0, hi = d.nseq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (locate(d.offsets, d.T, m).slot / L + m <= slot) lo = m;
        else hi = m - 1;
    }
    *s = locate(d.offsets, d.T, lo);
    *i = lo;
    *seg = slot - (s->slot / L + lo);
    return *seg == 0 || (*seg > 0 && *seg * L * kChunk < s->len);
}

template <int DK>
struct PrepCfg {
    static constexpr int LD = 68;                          // row pitch of the float32 64 x 64 scratch
    static constexpr uint32_t KQ = (DK / 64) * 2 * kTile;  // [feature block][K rows | Q rows]
    // T beta is staged where Q was (two tiles), W where the scratch was
    static constexpr uint32_t oTb = DK == 128 ? kTile : 2 * kTile, sTb = DK == 128 ? 2 * kTile : kTile;
    static constexpr uint32_t oA = 4 * kTile, oL = oA + 64 * LD * 4, oItem = oL + 352 * 4, oBar = oItem + 64, BYTES = oBar + 64;
    static constexpr int PER_SM = 4;
};

// T, W, P and the decays of one chunk and value head at a time.  Bound: HBM at
// Dk = 128 (33 kB of K and Q in, 59 kB of images out; 8 x 4096 tokens, 6 heads:
// 54 us, 5.2 TB/s, 76 % of a plain copy's rate), the latency of its steps at
// Dk = 64 (each waits for the last, the inverse's levels most of all).  Hence four
// CTAs per SM, and the next chunk's tiles and gates fetched under the current
// one's last steps.
template <int DT, int DK>
__global__ void __launch_bounds__(256, PrepCfg<DK>::PER_SM) delta_prep_kernel(const __grid_constant__ ChunkArgs a) {
    using C = PrepCfg<DK>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);  // loads, K K^T, W
    ChunkItem* items = reinterpret_cast<ChunkItem*>(sm + C::oItem);
    const DeltaArgs& d = a.d;
    const int p = threadIdx.x, w = __shfl_sync(0xffffffffu, p / 32, 0), lane = p % 32;
    if (sb & 1023) {  // not with the present layout of the window
        if (p == 0) atomicExch(d.err, 7);
        return;
    }
    if (p == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(bar + i, 1);
        fence_mbar_init();
    }
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bar + 3);
    if (w == 1) tc::alloc(s_tmem, 64);
    int next = blockIdx.x;
    auto find = [&](ChunkItem* to) {  // warp 3
        const ChunkItem x = find_item(d, int(a.slots), &next);
        if (lane == 0) *to = x;
    };
    auto load = [&](const ChunkItem& it) {  // one warp
        if (elect()) {
            mbar_expect_tx(bar, C::KQ);
            #pragma unroll
            for (int f = 0; f < DK / 64; ++f) {
                tma_load_4d(sb + f * 2 * kTile, &a.mk, f * 64, it.h / d.group, it.t0, it.row, bar);
                tma_load_4d(sb + f * 2 * kTile + kTile, &a.mq, f * 64, it.h / d.group, it.t0, it.row, bar);
            }
        }
        __syncwarp();
    };
    float g[2], e[2];  // log decays and betas of tokens 2 lane and 2 lane + 1 (warp 2)
    auto fetch = [&](const ChunkItem& it) {
        #pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int64_t t = it.t0 + 2 * lane + u;
            g[u] = e[u] = 0.0f;  // past the end: no decay, no update
            if (2 * lane + u < it.m) {
                g[u] = load16<DT>(d.g, it.row * d.g.b + t * d.g.t + it.h * d.g.h);
                e[u] = load16<DT>(d.beta, it.row * d.beta.b + t * d.beta.t + it.h * d.beta.h);
            }
        }
    };
    if (w == 3) find(items);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(s_tmem);
    const uint32_t lanes = tm + (uint32_t(32 * (w & 3)) << 16);
    float* A = reinterpret_cast<float*>(sm + C::oA);
    // b log2(e) and what rounding it left, beta, -G; decays between 16-token blocks (below)
    float *sbv = reinterpret_cast<float*>(sm + C::oL), *sbr = sbv + 64, *sbe = sbr + 64, *sng = sbe + 64, *sE2 = sng + 64,
          *sE1 = sE2 + 64;
    auto decay = [&](int i, int j) { return exp2_fast((sbv[i] - sbv[j]) + (sbr[i] - sbr[j])); };
    auto sync = [] { __syncthreads(); };
    const int row = 32 * (w & 3) + lane, i = row & 63, up = (row >> 5) & 1, half = w >> 2;
    const bool isp = row >= 64;
    if (items[0].m && w == 3) load(items[0]);
    if (w == 2) fetch(items[0]);
    bool ok = true;
    uint32_t k = 0;
    for (; items[k & 1].m; ++k) {
        const ChunkItem it = items[k & 1];
        const uint32_t par = k & 1;
        uint8_t* image = a.images + it.at * kImage<DK>;
        if (w == 2) {
            // running sum of the log decays, in units of log 2, as two floats: whole
            // numbers (exact) and fractions are summed apart, so that tokens that empty
            // the state (-173 each) cost later ratios of decays no digits
            constexpr float kLog2e = 1.44269504088896340736f;
            const float g0 = kLog2e * log_decay(g[0]), g1 = kLog2e * log_decay(g[1]);
            const float h1 = rintf(g1), f1 = g1 - h1;
            float h = rintf(g0) + h1, f = (g0 - rintf(g0)) + f1;
            #pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float v = __shfl_up_sync(0xffffffffu, h, o), y = __shfl_up_sync(0xffffffffu, f, o);
                if (lane >= o) {
                    h += v;
                    f += y;
                }
            }
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float a = u ? h : h - h1, c = u ? f : f - f1, s = a + c, t = s - a;
                sbv[2 * lane + u] = s;
                sbr[2 * lane + u] = (a - (s - t)) + (c - t);  // a + c - s, exactly
            }
            *reinterpret_cast<float2*>(sbe + 2 * lane) = make_float2(e[0], e[1]);
        }
        if (p == 0) bulk_wait_read();  // the last W has left the scratch
        tc::fence_before();
        sync();
        // D_ij for i >= 32 > j is E1_i E2_j with both factors at most 1: the decay
        // from the first token of i's 16-token block, and up to it
        if (p < 64) {
            const float b = sbv[p], G = exp2_fast(b);
            float* gt = reinterpret_cast<float*>(image + kImgE);
            gt[p] = decay(63, p);
            gt[64 + p] = d.scale * G;
            gt[128 + p] = b;
            gt[192 + p] = sbe[p];
            reinterpret_cast<float*>(image + kImgR<DK>)[p] = sbr[p];
            sng[p] = -G;
        } else if (w == 3) {
            find(items + (~k & 1));
        } else if (p >= 128 && p < 192) {
            const int q = p - 128;
            sE2[q] = decay(32 + 16 * (q >> 5), q & 31);
        } else if (p >= 192 && p < 224) {
            const int q = p - 192;
            sE1[q] = decay(32 + q, 32 + (q & 16));
        }
        ok = mbar_wait_bounded(bar, par, kWaitLimitTile);
        if (d.offsets && it.m < kChunk) {
            // rows past the sequence are the next one's: zero them (past the
            // tensor's end the TMA engine has)
            const int m = it.m;
            for (int x = p; x < (64 - m) * 8 * (DK / 32); x += 256) {
                const int f = x / ((64 - m) * 8), y = x % ((64 - m) * 8);
                *reinterpret_cast<uint4*>(sm + f * kTile + m * 128 + y * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async();
        }
        if (!(ok = !__syncthreads_or(!ok))) break;
        if (w == 0) {
            constexpr uint32_t id = tc::idesc(DT, 128, 64);
            const uint64_t d0 = sdesc(sb, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int f = 0; f < DK; f += 16) {
                    const uint64_t x = adv(d0, (f / 64) * 2 * kTile + (f % 64) * 2);
                    tc::mma_ss(tm, x, x, id, f > 0);  // A: 128 rows [K; Q], B: the first 64
                }
                tc::commit(bar + 1);
            }
        }
        ok = mbar_wait_bounded(bar + 1, par, kWaitLimitTile);
        if (!(ok = !__syncthreads_or(!ok))) break;
        tc::fence_after();
        // K K^T in lanes 0-63, Q K^T in lanes 64-127; warps 0-3 take columns 0-31,
        // warps 4-7 the others
        uint8_t* prow = image + kImgP + i * 128;
        if (up || !half) {
            const float f = isp ? d.scale : sbe[i];
            uint32_t x[32];
            const int j0 = half * 32;
            tc::ld32x32b_x32(lanes + j0, x);
            tc::wait_ld();
            if (up && !half) {  // whole blocks below the diagonal
                const float fe = f * sE1[i - 32];
                const float* e2 = sE2 + (i & 16) * 2;
                #pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 c = *reinterpret_cast<const float4*>(e2 + j);
                    const float2 u = mul2(mul2(make_float2(fe, fe), make_float2(c.x, c.y)), pair(x[j], x[j + 1]));
                    const float2 v = mul2(mul2(make_float2(fe, fe), make_float2(c.z, c.w)), pair(x[j + 2], x[j + 3]));
                    x[j] = __float_as_uint(u.x); x[j + 1] = __float_as_uint(u.y);
                    x[j + 2] = __float_as_uint(v.x); x[j + 3] = __float_as_uint(v.y);
                }
            } else {  // around the diagonal: entries above it (whatever they hold) become 0
                const float bi = sbv[i], ri = sbr[i];
                const int last = (isp ? i : i - 1) - j0;
                #pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 b = *reinterpret_cast<const float4*>(sbv + j0 + j);
                    const float4 r = *reinterpret_cast<const float4*>(sbr + j0 + j);
                    const float bj[4] = {b.x, b.y, b.z, b.w}, rj[4] = {r.x, r.y, r.z, r.w};
                    #pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float v = f * exp2_fast((bi - bj[q]) + (ri - rj[q])) * __uint_as_float(x[j + q]);
                        x[j + q] = j + q <= last ? __float_as_uint(v) : 0u;
                    }
                }
            }
            if (isp) {
                #pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
                    #pragma unroll
                    for (int q = 0; q < 4; ++q)
                        v[q] = Op<DT>::pack(__uint_as_float(x[8 * j + 2 * q]), __uint_as_float(x[8 * j + 2 * q + 1]));
                    *reinterpret_cast<uint4*>(prow + (((j0 / 8 + j) ^ (i & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            } else {
                #pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4*>(A + i * C::LD + j0 + j) = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
        } else if (isp) {
            #pragma unroll
            for (int j = 4; j < 8; ++j) *reinterpret_cast<uint4*>(prow + ((j ^ (i & 7)) * 16)) = make_uint4(0, 0, 0, 0);
        }
        if (w == 2) fetch(items[~k & 1]);
        tc::fence_before();
        sync();
        inverse64<C::LD>(A, p, w, lane, sync);
        // T with its columns times beta (staged over Q for the image), and times
        // -beta G (over the scratch, once everyone has read it), as two 16-bit parts
        {
            const int r = p & 63, h0 = (p >> 6) * 16;
            float4 t[4];
            #pragma unroll
            for (int j = 0; j < 4; ++j) t[j] = *reinterpret_cast<const float4*>(A + r * C::LD + h0 + 4 * j);
            sync();
            #pragma unroll
            for (int j0 = 0; j0 < 16; j0 += 8) {
                uint32_t v[4][4], ts[4];
                #pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const int jj = h0 + j0 + j;
                    const float4 y = t[(j0 + j) / 4];
                    const float4 x = *reinterpret_cast<const float4*>(sbe + jj), b = *reinterpret_cast<const float4*>(sng + jj);
                    // the scratch above the diagonal holds intermediate products
                    const float2 y0 = make_float2(jj <= r ? y.x : 0.0f, jj + 1 <= r ? y.y : 0.0f);
                    const float2 y1 = make_float2(jj + 2 <= r ? y.z : 0.0f, jj + 3 <= r ? y.w : 0.0f);
                    const float2 x0 = mul2(y0, make_float2(x.x, x.y)), x1 = mul2(y1, make_float2(x.z, x.w));
                    split<DT>(x0, &v[0][j / 2], &v[1][j / 2]);
                    split<DT>(x1, &v[0][j / 2 + 1], &v[1][j / 2 + 1]);
                    split<DT>(mul2(x0, make_float2(b.x, b.y)), &v[2][j / 2], &v[3][j / 2]);
                    split<DT>(mul2(x1, make_float2(b.z, b.w)), &v[2][j / 2 + 1], &v[3][j / 2 + 1]);
                    ts[j / 2] = Op<DT>::pack(y0.x, y0.y);
                    ts[j / 2 + 1] = Op<DT>::pack(y1.x, y1.y);
                }
                const int pos = r * 128 + ((((h0 + j0) / 8) ^ (r & 7)) * 16);
                #pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4*>(sm + (q < 2 ? C::oTb + q * C::sTb : C::oA + (q - 2) * kTile) + pos) =
                        make_uint4(v[q][0], v[q][1], v[q][2], v[q][3]);
                if (a.saved_t)
                    *reinterpret_cast<uint4*>(a.saved_t + it.at * kTile + pos) = make_uint4(ts[0], ts[1], ts[2], ts[3]);
            }
        }
        tc::fence_proxy_async();
        sync();
        if (p == 96) {
            bulk_s2g(image + kImgT, sb + C::oTb, kTile);
            bulk_s2g(image + kImgT + kTile, sb + C::oTb + C::sTb, kTile);
        }
        if (w == 0) {  // -W^T = K^T (-T beta G)^T
            constexpr uint32_t id = tc::idesc(DT, 128, 64) | kMnA;
            const uint64_t da = sdesc(sb, DK == 128 ? 2 * kTile : kTile), db = sdesc(sb + C::oA, 16);
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int q = 0; q < 2; ++q)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)
                        tc::mma_ss(tm, adv(da, t * 128), adv(db, q * kTile + t * 2), id, q + t > 0);
                tc::commit(bar + 2);
            }
        }
        ok = mbar_wait_bounded(bar + 2, par, kWaitLimitTile);
        if (!(ok = !__syncthreads_or(!ok))) break;
        tc::fence_after();
        if (w == 3) {  // K, Q and what was staged over Q have been read
            if (lane == 0) bulk_wait_read();
            __syncwarp();
            if (items[~k & 1].m) load(items[~k & 1]);
        }
        // W^T through the scratch, one part after the other
        uint32_t lo[16];
        uint8_t* q = sm + C::oA + row * 128;
        if (row < DK) {
            #pragma unroll
            for (int j0 = 0; j0 < 32; j0 += 16) {
                uint32_t x[16], hi[8];
                ld16(lanes + half * 32 + j0, x);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) split<DT>(pair(x[2 * j], x[2 * j + 1]), &hi[j], &lo[j0 / 2 + j]);
                #pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<uint4*>(q + ((half * 4 + j0 / 8 + j) ^ (row & 7)) * 16) =
                        make_uint4(hi[4 * j], hi[4 * j + 1], hi[4 * j + 2], hi[4 * j + 3]);
            }
        }
        tc::fence_proxy_async();
        tc::fence_before();
        sync();
        if (p == 0) {
            bulk_s2g(image + kImgW, sb + C::oA, DK * 128);
            bulk_wait_read();
        }
        sync();
        if (row < DK) {
            #pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(q + ((half * 4 + j) ^ (row & 7)) * 16) =
                    make_uint4(lo[4 * j], lo[4 * j + 1], lo[4 * j + 2], lo[4 * j + 3]);
        }
        tc::fence_proxy_async();
        sync();
        if (p == 0) bulk_s2g(image + kImgW + DK * 128, sb + C::oA, DK * 128);
    }
    if (p == 0) bulk_wait_read();
    if (p == 96) bulk_wait_read();
    if (p == 0 && !ok) {
        atomicExch(d.err, 7);
        mbar_wait_bounded(bar, k & 1, kWaitFinal);  // the copies have landed before the CTA leaves
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (w == 1) tc::dealloc(tm, 64);
}

template <int DK_, int DV_>
struct FwdCfg {
    static constexpr int DK = DK_;
    static constexpr int NKQ = 2, NI = 2;                  // stages of K and Q, and of the images (W: one)
    static constexpr uint32_t KQ = (DK / 64) * 2 * kTile;  // [feature block][K rows | Q rows]
    static constexpr uint32_t VB = 2 * kTile;              // DV = 64: the same block twice (M = 128)
    static constexpr uint32_t oKQ = 0, oV = oKQ + NKQ * KQ, oI = oV + VB, oW = oI + NI * kImgW,
                              oO = oW + DK * 256, oSv = oO + 64 * DV_ * 2,
                              oBar = oSv + (DK / 64 + 1) * DV_ * 128, BYTES = oBar + 256;
    static constexpr int THREADS = 768;
    // tensor memory columns.  The two U^T / Vn^T / P Vn accumulators take turns.
    // Vn's operand for O takes the place of S's low part (dead after S W).
    static constexpr uint32_t cS = 0, cHi = 128, cLo = 192, cVnH = 192, cVn = 256, cOS = 384, cVeH = 448, cVeL = 480;
    static __device__ __forceinline__ uint32_t vn(int c) { return cVn + (c & 1) * 64; }
};

enum Bar {
    kGo = 0,              // [2]: S's operands, K and Q, W and U are there: S W can go
    kKqFree = kGo + 2, kTFull = kKqFree + 2, kVFull = kTFull + 2, kRaw, kUDone, kSwDone, kVnReady, kSDone,
    kOReady, kOFree,
    kSv,                 // [3]: S (two blocks) and Vn are in their staging buffers
    kSvFree = kSv + 3,   // [3]: and out of them
    kFinal = kSvFree + 3,  // [2]
    kOpDone = kFinal + 2, kOpRead = kOpDone + 2,  // [2] each, by chunk parity
    kBars = kOpRead + 2
};

// STATE: only the state at the end of a segment: from zero (or the initial
// state) with the segment's values, or (blockIdx.z = 1) from the identity with
// no values, which gives the segment's transition matrix.
template <int DT, int DK, int DV, bool STATE>
__global__ void __launch_bounds__(FwdCfg<DK, DV>::THREADS, 1)
delta_fwd_kernel(const __grid_constant__ ChunkArgs a) {
    using C = FwdCfg<DK, DV>;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    // no static shared memory: the window starts 1024-byte aligned
    uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::oBar + 240);
    volatile int& s_fail = *reinterpret_cast<volatile int*>(sm + C::oBar + 244);
    const DeltaArgs& d = a.d;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int h = blockIdx.y, hk = h / d.group;
    if (sb & 1023) {  // not with the present layout of the window
        if (threadIdx.x == 0) atomicExch(d.err, 7);
        return;
    }
    Seq s;
    int si;
    int64_t seg;
    if (!find_segment(d, a.seg_chunks, blockIdx.x, &s, &si, &seg)) return;
    const int64_t c_first = seg * a.seg_chunks, c_all = (s.len + kChunk - 1) / kChunk;
    const bool last = c_first + a.seg_chunks >= c_all;
    const bool trans = STATE && blockIdx.z == 1;  // the transition matrix
    if (STATE && (last || (trans && seg == 0))) return;
    const int n = int(last ? c_all - c_first : a.seg_chunks);
    const int64_t slot0 = s.slot + c_first, tok0 = s.start + c_first * kChunk, len = s.len - c_first * kChunk;
    const int64_t hs = int64_t(si) * d.Hv + h, gs = int64_t(blockIdx.x) * d.Hv + h;
    // where the state starts and where it goes, [DK][lanes] float32
    const float* sin = seg == 0 ? (a.state_in ? a.state_in + hs * DK * DV : nullptr) : nullptr;
    if (!STATE && seg > 0) sin = a.seg_state + (gs - d.Hv) * DK * DV;
    float* sout = last && a.state_out ? a.state_out + hs * DK * DV : nullptr;
    if (STATE) sout = trans ? a.seg_trans + gs * DK * DK : a.seg_state + gs * DK * DV;
    const int LV = trans ? DK : DV;  // lanes in use (state columns)

    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < kBars; ++i) {
            uint32_t cnt = 1;  // else one arrival per warp of the role
            if (i == kOFree) cnt = 4;
            if (i == kVnReady || i == kOReady || i == kSv + 2 || i >= kOpRead) cnt = 16;
            if (i == kSv || i == kSv + 1) cnt = DK == 128 ? 8 : 16;
            if (i < kGo + 2) cnt = 16 + 3;                   // the chain, K and Q, W, U
            if (i == kKqFree || i == kKqFree + 1) cnt = 2;   // S Q and the update
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
    const uint32_t lanes = tm + (uint32_t(32 * (warp & 3)) << 16);  // this warp's tensor-memory lanes
    const int row = 32 * (warp & 3) + lane;                         // this thread's lane
    // one arrival per warp, after every lane's work
    auto done = [&](int b) {
        __syncwarp();
        if (lane == 0) arrive(bar + b);
    };
    auto image = [&](int c) { return sm + C::oI + (c % C::NI) * kImgW; };

    if (n == 0) {
        // an empty sequence: the state passes through
        if (sout)
            for (int x = threadIdx.x; x < DK * DV; x += C::THREADS) sout[x] = sin ? sin[x] : 0.0f;
    } else if (warp < 16) {
        // ---------------------------------------------------------------- chain
        const int dv = row % LV, quarter = warp >> 2;
        const bool mine = row < LV;
        constexpr int NC = DK / 4;  // columns of S of this warp
        const int k0 = quarter * NC;
        const int j0 = quarter * 16;  // and tokens of Vn and O
        // O^T of chunk c -> shared memory: done while the next chunk's S W runs
        auto put_o = [&](int c) {
            const float* gt = reinterpret_cast<const float*>(image(c) + kImgE);
            if (STATE) {
                done(kOpRead + (c & 1));
                return true;
            }
            tc::fence_after();
            uint32_t o[8];
            {
                uint32_t y[16], z[16];
                ld16(lanes + C::cOS + j0, y);
                ld16(lanes + C::vn(c) + j0, z);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 u = fma2(*reinterpret_cast<const float2*>(gt + 64 + j0 + 2 * j), pair(y[2 * j], y[2 * j + 1]),
                                          pair(z[2 * j], z[2 * j + 1]));
                    o[j] = Op<DT>::pack(u.x, u.y);
                }
            }
            tc::fence_before();
            done(kOpRead + (c & 1));
            // neighbours exchange halves, so that a lane holds two features of one
            // token; rows of odd tokens are turned by 64 bytes against bank conflicts
            if (c > 0 && !wait(bar + kOFree, (c - 1) & 1, fail)) return false;
            if (mine) {
                uint8_t* p = sm + C::oO + (((row >> 1) * 4) ^ ((row & 1) * 64)) + (j0 + (row & 1)) * (DV * 2);
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t y = __shfl_xor_sync(0xffffffffu, o[j], 1);
                    *reinterpret_cast<uint32_t*>(p + 2 * j * (DV * 2)) =
                        row & 1 ? __byte_perm(y, o[j], 0x7632) : __byte_perm(o[j], y, 0x5410);
                }
            }
            done(kOReady);
            return true;
        };
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            if (!(ok = wait(bar + kTFull + c % C::NI, (c / C::NI) & 1, fail))) break;
            const float* gt = reinterpret_cast<const float*>(image(c) + kImgE);
            const float g63 = exp2_fast(gt[128 + 63]);
            const float2 gc = make_float2(g63, g63);
            uint32_t x[NC], hi[NC / 2], lo[NC / 2];
            if (c > 0) {
                if (!(ok = wait(bar + kSDone, (c - 1) & 1, fail))) break;
                tc::fence_after();
                ld_cols<NC>(lanes + C::cS + k0, x);
                tc::wait_ld();
            } else {
                #pragma unroll
                for (int j = 0; j < NC; ++j)
                    x[j] = __float_as_uint(trans ? (k0 + j == dv ? 1.0f : 0.0f) : (sin ? sin[(k0 + j) * DV + dv] : 0.0f));
            }
            #pragma unroll
            for (int j = 0; j < NC / 2; ++j) {
                const float2 v = pair(x[2 * j], x[2 * j + 1]), y = mul2(gc, v);
                split<DT>(v, &hi[j], &lo[j]);
                x[2 * j] = __float_as_uint(y.x);
                x[2 * j + 1] = __float_as_uint(y.y);
            }
            // the places of S's operands are free after S Q and (the last) P Vn
            if (c > 0 && !(ok = wait(bar + kOpDone + ((c - 1) & 1), ((c - 1) >> 1) & 1, fail))) break;
            tc::fence_after();
            st_cols<NC / 2>(lanes + C::cHi + k0 / 2, hi);
            st_cols<NC / 2>(lanes + C::cLo + k0 / 2, lo);
            tc::wait_st();
            tc::fence_before();
            done(kGo + (c & 1));
            st_cols<NC>(lanes + C::cS + k0, x);  // complete before kVnReady
            if (!STATE && a.saved_s) {
                // a staging buffer for each block of 64 features of S, and for Vn
                const int blk = k0 >> 6;
                if (c > 0 && !(ok = wait(bar + kSvFree + blk, (c - 1) & 1, fail))) break;
                if (mine) {
                    uint8_t* sv = sm + C::oSv + blk * (DV * 128) + dv * 128;
                    #pragma unroll
                    for (int j = 0; j < NC / 2; j += 4)
                        *reinterpret_cast<uint4*>(sv + ((((k0 & 63) / 8 + j / 4) ^ (dv & 7)) * 16)) =
                            make_uint4(hi[j], hi[j + 1], hi[j + 2], hi[j + 3]);
                }
                tc::fence_proxy_async();
                done(kSv + blk);
            }
            if (c > 0 && !(ok = put_o(c - 1))) break;
            // Vn^T = U^T - S^T W^T
            if (!(ok = wait(bar + kSwDone, c & 1, fail))) break;
            tc::fence_after();
            uint32_t vh[8], eh[8], el[8];
            {
                uint32_t y[16];
                ld16(lanes + C::vn(c) + j0, y);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = pair(y[2 * j], y[2 * j + 1]);
                    vh[j] = Op<DT>::pack(v.x, v.y);
                    split<DT>(mul2(*reinterpret_cast<const float2*>(gt + j0 + 2 * j), v), &eh[j], &el[j]);
                }
            }
            st_cols<8>(lanes + C::cVnH + j0 / 2, vh);
            st_cols<8>(lanes + C::cVeH + j0 / 2, eh);
            st_cols<8>(lanes + C::cVeL + j0 / 2, el);
            tc::wait_st();
            tc::fence_before();
            done(kVnReady);
            if (!STATE && a.saved_s) {
                if (c > 0 && !(ok = wait(bar + kSvFree + 2, (c - 1) & 1, fail))) break;
                if (mine) {
                    uint8_t* sv = sm + C::oSv + (DK / 64) * (DV * 128) + dv * 128;
                    *reinterpret_cast<uint4*>(sv + ((j0 / 8) ^ (dv & 7)) * 16) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
                    *reinterpret_cast<uint4*>(sv + ((j0 / 8 + 1) ^ (dv & 7)) * 16) = make_uint4(vh[4], vh[5], vh[6], vh[7]);
                }
                tc::fence_proxy_async();
                done(kSv + 2);
            }
        }
        if (ok) ok = wait(bar + kOpDone + ((n - 1) & 1), ((n - 1) >> 1) & 1, fail) && put_o(n - 1);
        if (ok) ok = wait(bar + kSDone, (n - 1) & 1, fail);
        if (ok && sout) {
            tc::fence_after();
            uint32_t x[NC];
            ld_cols<NC>(lanes + C::cS + k0, x);
            tc::wait_ld();
            if (mine) {
                #pragma unroll
                for (int j = 0; j < NC; ++j) sout[(k0 + j) * LV + dv] = __uint_as_float(x[j]);
            }
        }
        if (!ok) s_fail = 1;
    } else if (warp < 20) {
        // ---------------------------------------------------------------- O
        bool ok = true;
        auto copy_o = [&](int c) {  // O of chunk c -> global memory
            if (!wait(bar + kOReady, c & 1, fail)) return false;
            constexpr int NP = DV / 8;  // 16-byte pieces of a token
            const int64_t left = len - int64_t(c) * kChunk;
            const int piece = row % NP;
            uint16_t* p = reinterpret_cast<uint16_t*>(d.o.p) + s.row * d.o.b + (tok0 + int64_t(c) * kChunk) * d.o.t +
                          h * d.o.h + piece * 8;
            #pragma unroll
            for (int t = row / NP; t < 64; t += 128 / NP) {
                const uint4 x = *reinterpret_cast<const uint4*>(sm + C::oO + t * (DV * 2) + ((piece ^ ((t & 1) * 4)) * 16));
                if (t < left) *reinterpret_cast<uint4*>(p + t * d.o.t) = x;
            }
            done(kOFree);
            return true;
        };
        for (int c = 0; !STATE && ok && c < n; ++c) ok = copy_o(c);
        if (!ok) s_fail = 1;
    } else if (warp == 20) {
        // ---------------------------------------------------------------- S W and the update of S
        constexpr uint32_t id64 = tc::idesc(DT, 128, 64) | kMnB, idS = tc::idesc(DT, 128, DK) | kMnB;
        bool ok = true;
        for (int c = 0; c < n; ++c) {
            if (!(ok = wait(bar + kGo + (c & 1), (c >> 1) & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dw = sdesc(sb + C::oW, 16);
                #pragma unroll
                for (int f = 0; f < DK; f += 16) {  // U^T - S^T W^T (W is stored negated)
                    tc::mma(tm + C::vn(c), tm + C::cHi + f / 2, adv(dw, f * 128), id64, !(trans && f == 0));
                    tc::mma(tm + C::vn(c), tm + C::cHi + f / 2, adv(dw, DK * 128 + f * 128), id64, 1);
                    tc::mma(tm + C::vn(c), tm + C::cLo + f / 2, adv(dw, f * 128), id64, 1);
                }
                tc::commit(bar + kSwDone);
            }
            if (!(ok = wait(bar + kVnReady, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dk = sdesc(sb + C::oKQ + (c % C::NKQ) * C::KQ, 2 * kTile);
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)  // S^T += (e Vn)^T K
                        tc::mma(tm + C::cS, tm + (m ? C::cVeL : C::cVeH) + t / 2, adv(dk, t * 128), idS, 1);
                tc::commit(bar + kSDone);
                tc::commit(bar + kKqFree + c % C::NKQ);
            }
        }
        if (!ok) s_fail = 1;
        // everything issued is done before tensor memory is given back
        if (elect()) tc::commit(bar + kFinal);
        mbar_wait_bounded(bar + kFinal, 0, kWaitFinal);
    } else if (warp == 23) {
        // ---------------------------------------------------------------- U, S Q and P Vn
        constexpr uint32_t id64 = tc::idesc(DT, 128, 64);
        bool ok = true;
        auto u_wait = [&](int c) {
            return wait(bar + kTFull + c % C::NI, (c / C::NI) & 1, fail) && wait(bar + kVFull, c & 1, fail);
        };
        auto u_issue = [&](int c) {  // U^T = V^T (T beta)^T; by one thread
            const uint64_t da = sdesc(sb + C::oV, kTile);
            const uint64_t db = sdesc(sb + C::oI + (c % C::NI) * kImgW + kImgT, 16);
            if (!trans) {
                #pragma unroll
                for (int m = 0; m < 2; ++m)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)
                        tc::mma_ss(tm + C::vn(c), adv(da, t * 128), adv(db, m * kTile + t * 2), id64 | kMnA, m + t > 0);
            }
            tc::commit(bar + kUDone);
            tc::commit(bar + kGo + (c & 1));
        };
        ok = u_wait(0);
        tc::fence_after();
        if (ok && elect()) u_issue(0);
        for (int c = 0; ok && c < n; ++c) {
            // S Q after S W, once chunk c - 1's O is out of its accumulators
            ok = wait(bar + kSwDone, c & 1, fail);
            if (ok && c > 0) ok = wait(bar + kOpRead + ((c - 1) & 1), ((c - 1) >> 1) & 1, fail);
            if (!ok) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dq = sdesc(sb + C::oKQ + (c % C::NKQ) * C::KQ + kTile, 16);
                if (!STATE) {
                    #pragma unroll
                    for (int f = 0; f < DK; f += 16)  // S^T Q^T
                        tc::mma(tm + C::cOS, tm + C::cHi + f / 2, adv(dq, (f / 64) * 2 * kTile + (f % 64) * 2), id64, f > 0);
                }
                tc::commit(bar + kKqFree + c % C::NKQ);
            }
            if (c + 1 < n && !(ok = u_wait(c + 1))) break;
            // P Vn and the next U after the update of S, while the chain turns S into operands
            if (!(ok = wait(bar + kSDone, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dp = sdesc(sb + C::oI + (c % C::NI) * kImgW + kImgP, 16);
                if (!STATE) {
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)  // Vn^T P^T
                        tc::mma(tm + C::vn(c), tm + C::cVnH + t / 2, adv(dp, t * 2), id64, t > 0);
                }
                tc::commit(bar + kOpDone + (c & 1));
                if (c + 1 < n) u_issue(c + 1);
            }
        }
        if (!ok) s_fail = 1;
        if (elect()) tc::commit(bar + kFinal + 1);
        mbar_wait_bounded(bar + kFinal + 1, 0, kWaitFinal);
    } else if (warp == 22) {
        // ---------------------------------------------------------------- S, Vn -> global
        bool ok = true;
        for (int c = 0; !STATE && a.saved_s && ok && c < n; ++c) {
            const int64_t at = (slot0 + c) * d.Hv + h;
            #pragma unroll
            for (int b = 0; ok && b <= DK / 64; ++b) {
                const bool v = b == DK / 64;
                const int x = v ? 2 : b;
                if (!(ok = wait(bar + kSv + x, c & 1, fail))) break;
                if (elect()) {
                    bulk_s2g(v ? a.saved_v + at * (DV * 128) : a.saved_s + at * (DV * DK * 2) + b * (DV * 128),
                             sb + C::oSv + b * (DV * 128), DV * 128);
                    bulk_wait_read();
                }
                done(kSvFree + x);
            }
        }
        if (!ok) s_fail = 1;
    } else {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int c = 0;
        // images are asked into L2 two chunks ahead (8 x 4096 tokens with what the
        // backward needs: 149 us, 161 us without); not by the walks of segments, which
        // fill the SMs and are at HBM's rate without it (445 us, 483 us with it)
        const bool ahead = a.seg_chunks > a.slots;
        auto fix = [&](uint8_t* t, int m) {  // zero rows m .. 63 of a tile
            for (int x = lane; x < (64 - m) * 8; x += 32) *reinterpret_cast<uint4*>(t + m * 128 + x * 16) = make_uint4(0, 0, 0, 0);
        };
        for (; ok && c < n; ++c) {
            const int st = c % C::NKQ;
            uint8_t* kq = sm + C::oKQ + st * C::KQ;
            const int t0 = int(tok0) + c * kChunk, row0 = int(s.row);
            const int64_t left = len - int64_t(c) * kChunk;
            // rows past the sequence: the TMA engine writes zeros past the tensor's
            // end; in a packed row they are the next sequence's and are zeroed here
            const bool tail = d.offsets && left < kChunk;
            if (!STATE && ahead && c + 2 < n && elect())
                bulk_prefetch(a.images + ((slot0 + c + 2) * d.Hv + h) * kImage<DK>, kImgR<DK>);
            __syncwarp();
            if (c >= C::NKQ && !(ok = wait(bar + kKqFree + st, (c / C::NKQ - 1) & 1, fail))) break;
            uint64_t* full = tail ? bar + kRaw : bar + kGo + st;
            if (elect()) {  // the state alone needs neither Q nor P
                mbar_expect_tx(full, STATE ? C::KQ / 2 : C::KQ);
                #pragma unroll
                for (int f = 0; f < DK / 64; ++f) {
                    tma_load_4d(smem_u32(kq) + f * 2 * kTile, &a.mk, f * 64, hk, t0, row0, full);
                    if (!STATE) tma_load_4d(smem_u32(kq) + f * 2 * kTile + kTile, &a.mq, f * 64, hk, t0, row0, full);
                }
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + kRaw, 0, fail))) break;
                for (int f = 0; f < 2 * DK / 64; ++f) fix(kq + f * kTile, int(left));
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + kGo + st);
            }
            if (c >= C::NI && !(ok = wait(bar + kOpRead + (c & 1), ((c - 2) >> 1) & 1, fail))) break;
            if (elect()) {
                // and the transition matrix no values: only the decays
                const uint32_t from = STATE ? (trans ? kImgE : kImgT) : 0;
                mbar_expect_tx(bar + kTFull + c % C::NI, kImgW - from);
                bulk_g2s(image(c) + from, a.images + ((slot0 + c) * d.Hv + h) * kImage<DK> + from, kImgW - from,
                         bar + kTFull + c % C::NI);
            }
            __syncwarp();
            if (c >= 1 && !(ok = wait(bar + kUDone, (c - 1) & 1, fail))) break;
            if (trans) {
                if (lane == 0) arrive(bar + kVFull);
            } else {
                full = tail ? bar + kRaw : bar + kVFull;
                if (elect()) {
                    mbar_expect_tx(full, C::VB);
                    #pragma unroll
                    for (int f = 0; f < 2; ++f)
                        tma_load_4d(sb + C::oV + f * kTile, &a.mv, DV == 128 ? f * 64 : 0, h, t0, row0, full);
                }
                __syncwarp();
                if (tail) {
                    if (!(ok = wait(bar + kRaw, 1, fail))) break;
                    for (int f = 0; f < 2; ++f) fix(sm + C::oV + f * kTile, int(left));
                    tc::fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) arrive(bar + kVFull);
                }
            }
            if (c >= 1 && !(ok = wait(bar + kSwDone, (c - 1) & 1, fail))) break;
            if (elect()) {
                mbar_expect_tx(bar + kGo + (c & 1), DK * 256);
                bulk_g2s(sm + C::oW, a.images + ((slot0 + c) * d.Hv + h) * kImage<DK> + kImgW, DK * 256, bar + kGo + (c & 1));
            }
            __syncwarp();
        }
        if (!ok) s_fail = 1;
        // every copy has landed before the CTA leaves (bounded waits; a phase that
        // is already over returns at once)
        for (int x = c > 2 ? c - 2 : 0; x < c; ++x) {
            mbar_wait_bounded(bar + kGo + (x & 1), (x >> 1) & 1, kWaitFinal);
            mbar_wait_bounded(bar + kTFull + x % C::NI, (x / C::NI) & 1, kWaitFinal);
        }
        if (c > 0) mbar_wait_bounded(bar + kVFull, (c - 1) & 1, kWaitFinal);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 20) tc::dealloc(tm, 512);
    if (threadIdx.x == 0 && s_fail) atomicExch(d.err, 7);
}

// The states at the segments' starts: S_(s+1) = M_s S_s + N_s along a
// sequence, float32; N_0 already holds the initial state's part.  The result
// replaces N_s.  A CTA takes 8 columns of S; the next M arrives by a bulk copy
// while the current one is applied (8 us a segment without, 2 us with it at
// 128 x 128; 25 segments: 76 us).  Bound: the 64 KB of M that each CTA pulls from L2
// a segment, which nothing but the chain of segments can overlap.
template <int DK, int DV>
__global__ void __launch_bounds__(256) delta_join_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(128) float join_sm[];  // M, two stages
    __shared__ float x[2][DK][8];
    __shared__ uint64_t bar[2];
    const DeltaArgs& d = a.d;
    const int i = blockIdx.x, h = blockIdx.y, col = threadIdx.x % 8, r0 = threadIdx.x / 8, v0 = blockIdx.z * 8;
    const Seq s = locate(d.offsets, d.T, i);
    const int64_t c_all = (s.len + kChunk - 1) / kChunk, nseg = (c_all + a.seg_chunks - 1) / a.seg_chunks;
    const int64_t g0 = (s.slot / a.seg_chunks + i) * d.Hv + h;
    if (nseg < 3) return;
    auto load = [&](int64_t g) {
        mbar_expect_tx(&bar[g & 1], DK * DK * 4);
        bulk_g2s(join_sm + (g & 1) * DK * DK, a.seg_trans + (g0 + g * d.Hv) * DK * DK, DK * DK * 4, &bar[g & 1]);
    };
    if (threadIdx.x == 0) {
        mbar_init(&bar[0], 1);
        mbar_init(&bar[1], 1);
        fence_mbar_init();
        load(1);
    }
    const float* N = a.seg_state + g0 * DK * DV + v0 + col;
    for (int r = r0; r < DK; r += 32) x[0][r][col] = N[r * DV];
    __syncthreads();
    bool ok = true;
    for (int64_t g = 1; g + 1 < nseg; ++g) {
        const int b = int(g & 1);
        if (threadIdx.x == 0 && g + 2 < nseg) load(g + 1);
        float* out = a.seg_state + (g0 + g * d.Hv) * DK * DV + v0 + col;
        float acc[DK / 32];
        #pragma unroll
        for (int q = 0; q < DK / 32; ++q) acc[q] = out[(r0 + 32 * q) * DV];
        ok = mbar_wait_bounded(&bar[b], uint32_t((g - 1) >> 1) & 1, kWaitLimitTile);
        if (__syncthreads_or(!ok)) {
            ok = false;
            break;
        }
        const float* M = join_sm + b * DK * DK;
        #pragma unroll 4
        for (int k = 0; k < DK; k += 4) {
            #pragma unroll
            for (int q = 0; q < DK / 32; ++q) {
                const float4 m = *reinterpret_cast<const float4*>(M + (r0 + 32 * q) * DK + k);
                acc[q] = fmaf(m.x, x[b ^ 1][k][col], acc[q]);
                acc[q] = fmaf(m.y, x[b ^ 1][k + 1][col], acc[q]);
                acc[q] = fmaf(m.z, x[b ^ 1][k + 2][col], acc[q]);
                acc[q] = fmaf(m.w, x[b ^ 1][k + 3][col], acc[q]);
            }
        }
        #pragma unroll
        for (int q = 0; q < DK / 32; ++q) {
            x[b][r0 + 32 * q][col] = acc[q];
            out[(r0 + 32 * q) * DV] = acc[q];
        }
        __syncthreads();
    }
    if (!ok && threadIdx.x == 0) {
        atomicExch(d.err, 7);
        for (int b = 0; b < 2; ++b) {  // copies have landed before the CTA leaves
            mbar_wait_bounded(&bar[b], 0, kWaitFinal);
            mbar_wait_bounded(&bar[b], 1, kWaitFinal);
        }
    }
}

template <int DT, int DK, int DV>
cudaError_t launch(const ChunkArgs& a, cudaStream_t st) {
    static PerDevice c0, c1, c2, c3;
    constexpr size_t sp = PrepCfg<DK>::BYTES, sf = FwdCfg<DK, DV>::BYTES;
    static_assert(sf <= 232448 && (sp + 1024) * PrepCfg<DK>::PER_SM <= 233472, "shared memory");
    cudaError_t e = opt_in(delta_prep_kernel<DT, DK>, sp, c0);
    if (e == cudaSuccess) e = opt_in(delta_fwd_kernel<DT, DK, DV, false>, sf, c1);
    if (e == cudaSuccess) e = opt_in(delta_fwd_kernel<DT, DK, DV, true>, sf, c2);
    if (e == cudaSuccess) e = opt_in(delta_join_kernel<DK, DV>, 2 * DK * DK * 4, c3);
    if (e != cudaSuccess) return e;
    const unsigned H = unsigned(a.d.Hv);
    const int64_t items = a.slots * a.d.Hv, most = int64_t(a.sms) * PrepCfg<DK>::PER_SM;
    delta_prep_kernel<DT, DK><<<unsigned(items < most ? items : most), 256, sp, st>>>(a);
    if (a.segments > a.d.nseq) {
        delta_fwd_kernel<DT, DK, DV, true><<<dim3(unsigned(a.segments), H, 2), FwdCfg<DK, DV>::THREADS, sf, st>>>(a);
        delta_join_kernel<DK, DV><<<dim3(unsigned(a.d.nseq), H, DV / 8), 256, 2 * DK * DK * 4, st>>>(a);
    }
    delta_fwd_kernel<DT, DK, DV, false><<<dim3(unsigned(a.segments), H), FwdCfg<DK, DV>::THREADS, sf, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Segments.  A sequence's chunks follow one another, so few long sequences
// leave SMs idle.  Cut into m segments a row costs two walks of 1/m of its
// chunks instead of one of all: the segments' end states from zero and their
// transition matrices (side by side: m - 1 and m - 2 CTAs a row; the last
// segment needs neither, the first no matrix), a join, then the outputs from the
// joined states.  The rule counts waves of CTAs over the SMs in chunks of a walk
// (2 us; 2.6 us when all SMs walk and share the bandwidth), takes a join's step as
// one more and 12 for the rest of it, and cuts when that saves a tenth.  One row
// of 262144 tokens, 6 heads of 128: 25 segments, 1.1 ms in walks and join instead
// of 8.3 ms; 8 rows of 4096: 3 segments took 148 us against 130 us uncut, and stay
// uncut.  Packed rows are taken at their mean length, as the host does not know their
// offsets: one prompt of 60000 tokens among 31 of 178 stays uncut, 1.93 ms where it
// takes 0.45 ms alone.
void plan_segments(ChunkArgs* a, int sms) {
    const DeltaArgs& d = a->d;
    a->slots = chunk_slots(d.B, d.T, d.nseq);
    a->sms = sms;
    const int64_t rows = int64_t(d.nseq) * d.Hv;
    const int64_t chunks = d.nseq ? (d.B * d.T / d.nseq + kChunk - 1) / kChunk : 0;
    int64_t best = 1, cost = chunks - chunks / 10;
    for (int64_t m = 3; rows > 0 && m * rows <= sms && m * 8 <= chunks; ++m) {
        const int64_t w1 = ((2 * m - 3) * rows + sms - 1) / sms, len = (chunks + m - 1) / m;
        const int64_t c = 13 * (w1 + 1) * len / 10 + m + 12;
        if (c < cost) {
            cost = c;
            best = m;
        }
    }
    a->seg_chunks = best == 1 ? a->slots + 1 : (chunks + best - 1) / best;
    a->segments = best == 1 ? d.nseq : a->slots / a->seg_chunks + d.nseq;
}

cudaError_t launch_delta_forward(const ChunkArgs& a, int dt, int dk, int dv, cudaStream_t st) {
    if (dt == FFTCONV_F16) {
        if (dk == 64) return dv == 64 ? launch<0, 64, 64>(a, st) : launch<0, 64, 128>(a, st);
        return dv == 64 ? launch<0, 128, 64>(a, st) : launch<0, 128, 128>(a, st);
    }
    if (dk == 64) return dv == 64 ? launch<1, 64, 64>(a, st) : launch<1, 64, 128>(a, st);
    return dv == 64 ? launch<1, 128, 64>(a, st) : launch<1, 128, 128>(a, st);
}

}  // namespace fftconv
