// Linear attention with a fixed decay for each head over whole sequences, 64 tokens
// at a time, on the fifth-generation tensor cores.
//
// Per chunk of m tokens, with l the head's decay and the walk's factors s (linattn.h):
//   KV = sum_j w_j k_j v_j^T,           w_j = s_up l^(m-1-j)   (reverse: l^(j+1))
//   P_ij = s_p l^|i-j| q_i.k_j (i >= j; reverse: i <= j)
//   O_i = u_i (S^T q_i) + sum_j P_ij v_j,  u_i = s_in l^(i+1)  (reverse: l^(m-1-i))
//   S <- l^m S + KV
// KV does not depend on S, so nothing but the update of S goes from chunk to chunk.
// Everything is held transposed (features of V in the tensor-memory lanes): S^T,
// KV^T and O^T are accumulators, S^T and the weighted V^T come back as A operands in
// tensor memory, and K, Q, V stay the tiles that the TMA engine wrote (tile.cuh).
//
// Precision: S is float32, in the registers of the warps that update it.  Operands
// that are not inputs are taken in 16-bit parts: w V as three for bf16 (24 bits) or
// two for fp16 (22 bits), so that S keeps float32's digits; S and P as two, so that
// O is as good as its one rounding to 16 bits.  In fp16 a row of each of them is
// first scaled by a power of two to a largest value in [2^14, 2^15), and the
// accumulator scaled back: neither small values nor large states leave fp16's range.
//
// One CTA per sequence (or segment of one) and value head, roles by warp, handing
// over through mbarriers:
//   warps 0-7    S: float32 += KV, and its 16-bit parts for S Q
//   warps 8-11   w V in parts
//   warps 12-15  scores -> P, then O -> shared memory
//   warp 16      loads, three chunks deep;  warp 17  issues every contraction;  warp 18  stores O
// The contractions of a chunk are issued as KV, scores, S Q, P V: while KV runs the
// last O is read out, while S Q runs the scores become P.
#include "linattn_chunk.h"

#include "chunk.cuh"

namespace fftconv {
namespace {

using namespace tile;

// ldmatrix / stmatrix of four 8 x 8 blocks, transposed.
__device__ __forceinline__ void ldsm_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Store 16 lanes x 32 columns: thread t holds, for every 4 columns, column t % 4 of
// lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void st16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A power of two that takes a row's largest size x into [2^14, 2^15), and its
// inverse; for sizes below 2^-112 that of 2^-112.
__device__ __forceinline__ float2 row_scale(float x) {
    const uint32_t e = min(max(__float_as_uint(x) >> 23, 15u), 254u);
    return make_float2(__uint_as_float((268u - e) << 23), __uint_as_float((e - 14u) << 23));
}

template <int DK_, int DV_>
struct Cfg {
    static constexpr int KT = DK_ / 64;  // tiles of K and of Q
    static constexpr int NST = 3;
    static constexpr uint32_t sK = 0, sQ = KT * kTile, sV = 2 * KT * kTile, STAGE = sV + 2 * kTile;  // V: M = 128 lanes
    static constexpr uint32_t oP = NST * STAGE, oO = oP + 2 * kTile, oT = oO + (DV_ / 64) * kTile;
    // float tables: w and u for a whole chunk and for a last one, the scales of V, S and P
    static constexpr uint32_t tW = 0, tU = 128, tV = 256, tS = 768, tP = 1024, tM = 1088, TABLE = (1088 + 256) * 4;
    static constexpr uint32_t oBar = oT + TABLE, BYTES = oBar + 256;
    static constexpr int THREADS = 640;
    // tensor memory columns: S in two parts, KV, S Q, scores and then P V, w V in parts.
    // Where only the states are wanted KV and w V take turns.
    static constexpr uint32_t cHi = 0, cLo = DK_ / 2, cKV = DK_, cOi = 2 * DK_, cX = cOi + 64, cW = cX + 64;
    static __device__ __forceinline__ uint32_t kv(bool state, int c) { return state ? (c & 1) * DK_ : cKV; }
    static __device__ __forceinline__ uint32_t w(bool state, int c) { return state ? 2 * DK_ + (c & 1) * 96 : cW; }
};

enum Bar {
    kFull = 0, kFree = 3, kParts = 6, kKvDone = 8, kKvRead = 10,  // three stages; by chunk parity
    kRaw = 12, kSop, kSqDone, kScDone, kPReady, kPvDone, kORead, kOReady, kOFree, kFinal,
    kMax, kBars = kMax + 4  // the two warps of 32 lanes of S
};

// Where a CTA's part of a sequence is.
struct Part {
    Seq s;
    int i;         // sequence
    int64_t tok0;  // its first token in the row
    int64_t left;  // tokens from there to the sequence's end
    int n;         // chunks
    bool first, last;  // in the walk's order
};

__device__ __forceinline__ bool find_part(const Walk& w, int64_t L, int64_t slot, Part* p) {
    int lo = 0, hi = w.nseq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (locate(w.offsets, w.T, m).slot / L + m <= slot) lo = m;
        else hi = m - 1;
    }
    p->i = lo;
    p->s = locate(w.offsets, w.T, lo);
    const int64_t seg = slot - (p->s.slot / L + lo), all = (p->s.len + kChunk - 1) / kChunk, from = seg * L;
    if (seg < 0 || (seg > 0 && from >= all)) return false;
    const bool low = seg == 0, high = from + L >= all;
    p->first = w.reverse ? high : low;
    p->last = w.reverse ? low : high;
    p->n = int(high ? all - from : L);
    p->tok0 = p->s.start + from * kChunk;
    p->left = p->s.len - from * kChunk;
    return true;
}

// STATE: only the state at the end of a segment (from zero, or from the initial state).
template <int DT, int DK, int DV, bool STATE>
__global__ void __launch_bounds__(Cfg<DK, DV>::THREADS, 1) linattn_walk_kernel(const __grid_constant__ Passes a) {
    using C = Cfg<DK, DV>;
    constexpr int NP = DT == 0 ? 2 : 3;      // parts of w V
    constexpr int NB = STATE ? 2 : 1;        // buffers of KV and w V
    constexpr int NC = DK / 2;               // columns of S of a thread
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    // no static shared memory: the window starts 1024-byte aligned
    uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::oBar + 240);
    volatile int& s_fail = *reinterpret_cast<volatile int*>(sm + C::oBar + 244);
    float* tab = reinterpret_cast<float*>(sm + C::oT);
    const Pass& x = a.p[blockIdx.z];
    const Walk& wk = x.w;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const int h = blockIdx.y;
    if (sb & 1023) {  // not with the present layout of the window
        if (threadIdx.x == 0) atomicExch(a.err, 7);
        return;
    }
    Part p;
    if (!find_part(wk, a.seg_chunks, blockIdx.x, &p)) return;
    if (STATE && p.last) return;
    const int n = p.n;
    const int64_t hs = int64_t(p.i) * wk.H + h, gs = int64_t(blockIdx.x) * wk.H + h;
    const float* sin = wk.state_in ? wk.state_in + hs * DK * DV : nullptr;
    if (!p.first) sin = STATE ? nullptr : x.seg_state + (gs + (wk.reverse ? wk.H : -wk.H)) * DK * DV;
    float* sout = p.last && wk.state_out ? wk.state_out + hs * DK * DV : nullptr;
    if (STATE) sout = x.seg_state + gs * DK * DV;

    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < kBars; ++i) {
            uint32_t cnt = 1;  // else one arrival per warp of the role
            if (i == kParts || i == kParts + 1 || i == kPReady || i == kORead || i == kOReady) cnt = 4;
            if (i == kKvRead || i == kKvRead + 1 || i == kSop) cnt = 8;
            if (i >= kMax) cnt = 2;
            mbar_init(bar + i, cnt);
        }
        fence_mbar_init();
    }
    const float g = head_decay(wk.decay, h);
    if (threadIdx.x < 128) {
        const int j = threadIdx.x & 63;
        const int m = threadIdx.x < 64 ? 64 : int((p.s.len - 1) % kChunk) + 1;
        const int back = m - 1 - j, on = j + 1;
        tab[C::tW + threadIdx.x] = back >= 0 ? wk.s_up * expf(g * float(wk.reverse ? on : back)) : 0.0f;
        tab[C::tU + threadIdx.x] = back >= 0 ? wk.s_in * expf(g * float(wk.reverse ? back : on)) : 0.0f;
    }
    if (warp == 17) tc::alloc(&s_tmem, 512);
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
    // step c's chunk, its tokens, and whether they are fewer than 64
    auto chunk = [&](int c) { return wk.reverse ? n - 1 - c : c; };
    auto tokens = [&](int c) {
        const int64_t l = p.left - int64_t(chunk(c)) * kChunk;
        return int(l < kChunk ? l : kChunk);
    };

    if (n == 0) {
        // an empty sequence: the state passes through
        if (sout)
            for (int e = threadIdx.x; e < DK * DV; e += C::THREADS) {
                float v = 0.0f;
                if (sin) v = wk.turned ? sin[(e % DV) * DK + e / DV] : sin[e];
                sout[e] = v;
            }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- S
        more_registers<128>();
        const int dv = row % DV, k0 = (warp >> 2) * NC;
        float2 S[NC / 2];
        #pragma unroll
        for (int j = 0; j < NC / 2; ++j) {
            S[j] = make_float2(0.0f, 0.0f);
            const int k = k0 + 2 * j;
            if (sin)
                S[j] = wk.turned ? *reinterpret_cast<const float2*>(sin + dv * DK + k)
                                 : make_float2(sin[k * DV + dv], sin[(k + 1) * DV + dv]);
        }
        auto put = [&](int c) {  // S's parts for step c
            float2 sc = make_float2(1.0f, 1.0f);
            if constexpr (DT == 0) {
                float m = 0.0f;
                #pragma unroll
                for (int j = 0; j < NC / 2; ++j) m = fmaxf(m, fmaxf(fabsf(S[j].x), fabsf(S[j].y)));
                tab[C::tM + (warp >> 2) * 128 + row] = m;
                done(kMax + (warp & 3));
                if (!wait(bar + kMax + (warp & 3), c & 1, fail)) return false;
                sc = row_scale(fmaxf(m, tab[C::tM + (~warp >> 2 & 1) * 128 + row]));
                if (warp < 4) tab[C::tS + (c & 1) * 128 + row] = sc.y;
            }
            #pragma unroll
            for (int b = 0; b < NC; b += 16) {
                uint32_t hi[8], lo[8];
                #pragma unroll
                for (int j = 0; j < 8; ++j)
                    split<DT>(DT == 0 ? mul2(S[b / 2 + j], make_float2(sc.x, sc.x)) : S[b / 2 + j], &hi[j], &lo[j]);
                st_cols<8>(lanes + C::cHi + (k0 + b) / 2, hi);
                st_cols<8>(lanes + C::cLo + (k0 + b) / 2, lo);
            }
            tc::wait_st();
            tc::fence_before();
            done(kSop);
            return true;
        };
        bool ok = STATE || put(0);
        for (int c = 0; ok && c < n; ++c) {
            const Decay l = decay_over(g, float(tokens(c)));
            if (!(ok = wait(bar + kKvDone + (c & 1), (c >> 1) & 1, fail))) break;
            tc::fence_after();
            float inv = 1.0f;
            if constexpr (DT == 0) inv = tab[C::tV + (c & 3) * 128 + row];
            #pragma unroll
            for (int b = 0; b < NC; b += 32) {
                uint32_t y[32];
                tc::ld32x32b_x32(lanes + C::kv(STATE, c) + k0 + b, y);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float2& s = S[b / 2 + j];
                    const float2 kv = pair(y[2 * j], y[2 * j + 1]), part = make_float2(l.part, l.part);
                    const float2 t = DT == 0 ? fma2(kv, make_float2(inv, inv), mul2(part, s)) : fma2(part, s, kv);
                    s = fma2(make_float2(l.keep, l.keep), s, t);
                }
            }
            tc::fence_before();
            done(kKvRead + (c & 1));
            if (!STATE && c + 1 < n) {
                if (!(ok = wait(bar + kSqDone, c & 1, fail))) break;
                tc::fence_after();
                ok = put(c + 1);
            }
        }
        if (ok && sout && row < DV) {
            #pragma unroll
            for (int j = 0; j < NC / 2; ++j) {
                sout[(k0 + 2 * j) * DV + dv] = S[j].x;
                sout[(k0 + 2 * j + 1) * DV + dv] = S[j].y;
            }
        }
        if (!ok) s_fail = 1;
    } else if (warp < 12) {
        // ---------------------------------------------------------------- w V
        fewer_registers<88>();
        const int sp = warp & 3;
        bool ok = true;
        for (int c = 0; ok && c < n; ++c) {
            const uint32_t tile_v = sb + (c % C::NST) * C::STAGE + C::sV + (sp >> 1) * kTile;
            ok = wait(bar + kFull + c % C::NST, (c / C::NST) & 1, fail);
            if (ok && c >= NB) ok = wait(bar + kKvDone + ((c - NB) & 1), ((c - NB) >> 1) & 1, fail);
            if (!ok) break;
            tc::fence_after();
            const float* wt = tab + C::tW + (tokens(c) < kChunk ? 64 : 0) + 2 * (lane & 3);
            #pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // 16 features each
                uint32_t v[16];
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = 16 * i + (lane >> 4) * 8 + (lane & 7), piece = (sp & 1) * 4 + hf * 2 + ((lane >> 3) & 1);
                    ldsm_t(tile_v + tok * 128 + ((piece ^ (tok & 7)) * 16), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
                const uint32_t to = lanes + (uint32_t(16 * hf) << 16) + C::w(STATE, c);
                uint32_t hi[16], lo[16];
                if constexpr (DT == 0) {
                    float2 y[16];
                    float m0 = 0.0f, m1 = 0.0f;
                    #pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const cpx u = Op<DT>::unpack(v[i]);
                        y[i] = mul2(make_float2(u.r, u.i), *reinterpret_cast<const float2*>(wt + 8 * (i >> 1)));
                        float& m = i & 1 ? m1 : m0;
                        m = fmaxf(m, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
                    }
                    #pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                    }
                    const float2 s0 = row_scale(m0), s1 = row_scale(m1);
                    if ((lane & 3) == 0) {
                        float* inv = tab + C::tV + (c & 3) * 128 + 32 * sp + 16 * hf + (lane >> 2);
                        inv[0] = s0.y;
                        inv[8] = s1.y;
                    }
                    #pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float s = i & 1 ? s1.x : s0.x;
                        split<DT>(mul2(y[i], make_float2(s, s)), &hi[i], &lo[i]);
                    }
                } else {
                    uint32_t l2[16];
                    #pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const cpx u = Op<DT>::unpack(v[i]);
                        const float2 y = mul2(make_float2(u.r, u.i), *reinterpret_cast<const float2*>(wt + 8 * (i >> 1)));
                        hi[i] = Op<DT>::pack(y.x, y.y);
                        const cpx e = Op<DT>::unpack(hi[i]);
                        split<DT>(sub2(y, make_float2(e.r, e.i)), &lo[i], &l2[i]);
                    }
                    st16x128b_x8(to + 64, l2);
                }
                st16x128b_x8(to, hi);
                st16x128b_x8(to + 32, lo);
            }
            tc::wait_st();
            tc::fence_before();
            done(kParts + (c & 1));
        }
        if (!ok) s_fail = 1;
    } else if (warp < 16) {
        // ---------------------------------------------------------------- P and O
        const int sp = warp & 3, q = lane >> 2, r = lane & 3;
        if constexpr (!STATE) {
            const bool mine = 32 * sp < DV;
            // decays between the chunk's tokens: rows i = 16 sp + q and i + 8, columns 8 n + 2 r and the next
            float dd[32];
            #pragma unroll
            for (int e = 0; e < 32; ++e) {
                const int i = 16 * sp + q + (e & 2) * 4, j = 8 * (e >> 2) + 2 * r + (e & 1);
                const int d = wk.reverse ? j - i : i - j;
                dd[e] = d >= 0 ? wk.s_p * expf(g * float(d)) : 0.0f;
            }
            bool ok = true;
            for (int c = 0; ok && c < n; ++c) {
                if (!(ok = wait(bar + kScDone, c & 1, fail))) break;
                tc::fence_after();
                {
                    uint32_t y[32];
                    tc::ld16x256b_x8(lanes + C::cX, y);
                    tc::wait_ld();
                    float2 z0 = make_float2(1.0f, 1.0f), z1 = z0;
                    if constexpr (DT == 0) {
                        float m0 = 0.0f, m1 = 0.0f;
                        #pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float& m = e & 2 ? m1 : m0;
                            m = fmaxf(m, fabsf(__uint_as_float(y[e]) * dd[e]));
                        }
                        #pragma unroll
                        for (int o = 1; o < 4; o <<= 1) {
                            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                        }
                        z0 = row_scale(m0);
                        z1 = row_scale(m1);
                        if (r == 0) {
                            tab[C::tP + 16 * sp + q] = z0.y;
                            tab[C::tP + 16 * sp + q + 8] = z1.y;
                        }
                    }
                    uint8_t* to = sm + C::oP + (16 * sp + q) * 128 + r * 4;
                    #pragma unroll
                    for (int b = 0; b < 8; ++b)
                        #pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float2 v = mul2(pair(y[4 * b + 2 * u], y[4 * b + 2 * u + 1]),
                                            make_float2(dd[4 * b + 2 * u], dd[4 * b + 2 * u + 1]));
                            if constexpr (DT == 0) v = mul2(v, u ? make_float2(z1.x, z1.x) : make_float2(z0.x, z0.x));
                            uint32_t hi, lo;
                            split<DT>(v, &hi, &lo);
                            uint8_t* at = to + u * 1024 + ((b ^ q) * 16);  // rows i and i + 8 turn alike
                            *reinterpret_cast<uint32_t*>(at) = hi;
                            *reinterpret_cast<uint32_t*>(at + kTile) = lo;
                        }
                }
                tc::fence_proxy_async();
                tc::fence_before();
                done(kPReady);
                // O of this chunk
                if (!(ok = wait(bar + kPvDone, c & 1, fail))) break;
                tc::fence_after();
                const int m = tokens(c);
                const float* ut = tab + C::tU + (m < kChunk ? 64 : 0) + 2 * r;
                if (!wk.o32 && c > 0 && !(ok = wait(bar + kOFree, (c - 1) & 1, fail))) break;  // the last O has left shared memory
                const int64_t t0 = p.tok0 + int64_t(chunk(c)) * kChunk;
                #pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    #pragma unroll
                    for (int b0 = 0; b0 < 8; b0 += 4) {
                        uint32_t y[16], z[16];
                        const uint32_t from = lanes + (uint32_t(16 * hf) << 16) + 8 * b0;
                        tc::ld16x256b_x4(from + C::cOi, y);
                        tc::ld16x256b_x4(from + C::cX, z);
                        tc::wait_ld();
                        const int f = mine ? 32 * sp + 16 * hf + q : 0;
                        float s0 = 1.0f, s1 = 1.0f;
                        if constexpr (DT == 0) {
                            s0 = tab[C::tS + (c & 1) * 128 + f];
                            s1 = tab[C::tS + (c & 1) * 128 + f + 8];
                        }
                        uint32_t o[8];
                        #pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float2 u = *reinterpret_cast<const float2*>(ut + 8 * (b0 + b));
                            float2 e0 = pair(z[4 * b], z[4 * b + 1]), e1 = pair(z[4 * b + 2], z[4 * b + 3]);
                            float2 u0 = u, u1 = u;
                            if constexpr (DT == 0) {
                                const float2 ps = *reinterpret_cast<const float2*>(tab + C::tP + 8 * (b0 + b) + 2 * r);
                                e0 = mul2(e0, ps);
                                e1 = mul2(e1, ps);
                                u0 = mul2(u, make_float2(s0, s0));
                                u1 = mul2(u, make_float2(s1, s1));
                            }
                            e0 = fma2(u0, pair(y[4 * b], y[4 * b + 1]), e0);
                            e1 = fma2(u1, pair(y[4 * b + 2], y[4 * b + 3]), e1);
                            if (wk.o32 && mine) {
                                const int t = 8 * (b0 + b) + 2 * r;
                                float* to = wk.o32 + ((p.s.row * wk.T + t0 + t) * wk.H + h) * DV + f;
                                if (t < m) to[0] = e0.x, to[8] = e1.x;
                                if (t + 1 < m) to[int64_t(wk.H) * DV] = e0.y, to[int64_t(wk.H) * DV + 8] = e1.y;
                            }
                            o[2 * b] = Op<DT>::pack(e0.x, e0.y);
                            o[2 * b + 1] = Op<DT>::pack(e1.x, e1.y);
                        }
                        if (hf == 1 && b0 == 4) {  // the accumulators and the scales have been read
                            tc::fence_before();
                            done(kORead);
                        }
                        if (!wk.o32 && mine) {
                            const int piece = (sp & 1) * 4 + hf * 2 + ((lane >> 3) & 1);
                            #pragma unroll
                            for (int b = 0; b < 4; b += 2) {
                                const int tok = 8 * (b0 + b) + (lane >> 4) * 8 + (lane & 7);
                                stsm_t(sb + C::oO + (sp >> 1) * kTile + tok * 128 + ((piece ^ (tok & 7)) * 16), o[2 * b],
                                       o[2 * b + 1], o[2 * b + 2], o[2 * b + 3]);
                            }
                        }
                    }
                }
                if (wk.o32) continue;
                tc::fence_proxy_async();
                done(kOReady);
            }
            if (!ok) s_fail = 1;
        }
    } else {
        fewer_registers<40>();
        bool ok = true;
        int c = 0;
        if (warp == 16) {
        // ---------------------------------------------------------------- loads
        const int row0 = int(p.s.row);
        auto fix = [&](uint8_t* t, int m) {  // zero rows m .. 63 of a tile
            for (int e = lane; e < (64 - m) * 8; e += 32) *reinterpret_cast<uint4*>(t + m * 128 + e * 16) = make_uint4(0, 0, 0, 0);
        };
        for (; ok && c < n; ++c) {
            const int st = c % C::NST, t0 = int(p.tok0) + chunk(c) * kChunk, m = tokens(c);
            // rows past the sequence: the TMA engine writes zeros past the tensor's
            // end; in a packed row they are the next sequence's and are zeroed here
            const bool tail = wk.offsets && m < kChunk;  // one chunk at most
            uint8_t* to = sm + st * C::STAGE;
            if (c >= C::NST && !(ok = wait(bar + kFree + st, (c / C::NST - 1) & 1, fail))) break;
            uint64_t* full = tail ? bar + kRaw : bar + kFull + st;
            if (elect()) {
                mbar_expect_tx(full, STATE ? C::STAGE - C::KT * kTile : C::STAGE);
                #pragma unroll
                for (int f = 0; f < C::KT; ++f) {
                    tma_load_4d(smem_u32(to) + C::sK + f * kTile, &x.mk, f * 64, h / wk.gk, t0, row0, full);
                    if (!STATE) tma_load_4d(smem_u32(to) + C::sQ + f * kTile, &x.mq, f * 64, h / wk.gq, t0, row0, full);
                }
                #pragma unroll
                for (int f = 0; f < 2; ++f)
                    tma_load_4d(smem_u32(to) + C::sV + f * kTile, &x.mv, DV == 128 ? f * 64 : 0, h / wk.gv, t0, row0, full);
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(bar + kRaw, 0, fail))) break;
                for (int f = 0; f < 2 * C::KT + 2; ++f)
                    if (!STATE || f < C::KT || f >= 2 * C::KT) fix(to + f * kTile, m);
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + kFull + st);
            }
        }
        // every copy has landed before the CTA leaves (bounded waits; a phase that
        // is already over returns at once)
        for (int y = c > C::NST ? c - C::NST : 0; y < c; ++y)
            mbar_wait_bounded(bar + kFull + y % C::NST, (y / C::NST) & 1, kWaitFinal);
        } else if (warp == 17) {
        // ---------------------------------------------------------------- contractions
        constexpr uint32_t idX = tc::idesc(DT, 64, 64), idO = tc::idesc(DT, 128, 64), idS = tc::idesc(DT, 128, DK) | kMnB;
        for (; ok && c < n; ++c) {
            const uint32_t from = sb + (c % C::NST) * C::STAGE;
            ok = wait(bar + kFull + c % C::NST, (c / C::NST) & 1, fail) && wait(bar + kParts + (c & 1), (c >> 1) & 1, fail);
            if (ok && c >= NB) ok = wait(bar + kKvRead + ((c - NB) & 1), ((c - NB) >> 1) & 1, fail);
            if (!ok) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dk = sdesc(from + C::sK, kTile);
                #pragma unroll
                for (int q = 0; q < NP; ++q)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)  // (w V)^T K
                        tc::mma(tm + C::kv(STATE, c), tm + C::w(STATE, c) + q * 32 + t / 2, adv(dk, t * 128), idS, q + t > 0);
                tc::commit(bar + kKvDone + (c & 1));
                if (STATE) tc::commit(bar + kFree + c % C::NST);
            }
            if (STATE) continue;
            if (c > 0 && !(ok = wait(bar + kORead, (c - 1) & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dq = sdesc(from + C::sQ, 16), dk = sdesc(from + C::sK, 16);
                #pragma unroll
                for (int f = 0; f < DK; f += 16)  // Q K^T
                    tc::mma_ss(tm + C::cX, adv(dq, (f / 64) * kTile + (f % 64) * 2), adv(dk, (f / 64) * kTile + (f % 64) * 2), idX, f > 0);
                tc::commit(bar + kScDone);
            }
            if (!(ok = wait(bar + kSop, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dq = sdesc(from + C::sQ, 16);
                #pragma unroll
                for (int q = 0; q < 2; ++q)
                    #pragma unroll
                    for (int f = 0; f < DK; f += 16)  // S^T Q^T
                        tc::mma(tm + C::cOi, tm + (q ? C::cLo : C::cHi) + f / 2, adv(dq, (f / 64) * kTile + (f % 64) * 2), idO, q + f > 0);
                tc::commit(bar + kSqDone);
            }
            if (!(ok = wait(bar + kPReady, c & 1, fail))) break;
            tc::fence_after();
            if (elect()) {
                const uint64_t dv = sdesc(from + C::sV, kTile), dp = sdesc(sb + C::oP, 16);
                #pragma unroll
                for (int q = 0; q < 2; ++q)
                    #pragma unroll
                    for (int t = 0; t < 64; t += 16)  // V^T P^T
                        tc::mma_ss(tm + C::cX, adv(dv, t * 128), adv(dp, q * kTile + t * 2), idO | kMnA, q + t > 0);
                tc::commit(bar + kPvDone);
                tc::commit(bar + kFree + c % C::NST);
            }
        }
        // everything issued is done before tensor memory is given back
        if (elect()) tc::commit(bar + kFinal);
        mbar_wait_bounded(bar + kFinal, 0, kWaitFinal);
        } else if (warp == 18 && !STATE && !wk.o32) {
        // ---------------------------------------------------------------- O -> global
        for (; c < n; ++c) {
            if (!(ok = wait(bar + kOReady, c & 1, fail))) break;
            const int m = tokens(c);
            const int64_t t0 = p.tok0 + int64_t(chunk(c)) * kChunk;
            if (!(wk.offsets && m < kChunk)) {  // tokens past the tensor's end are not written
                if (elect()) {
                    #pragma unroll
                    for (int f = 0; f < DV / 64; ++f)
                        tma_store_4d(&x.mo, sb + C::oO + f * kTile, f * 64, h, int(t0), int(p.s.row));
                    bulk_wait_read();
                }
            } else {  // a packed row goes on with the next sequence
                constexpr int NPC = DV / 8;  // 16-byte pieces of a token
                uint16_t* to = reinterpret_cast<uint16_t*>(wk.o.p) + p.s.row * wk.o.b + t0 * wk.o.t + h * wk.o.h;
                for (int e = lane; e < m * NPC; e += 32) {
                    const int t = e / NPC, y = e % NPC;
                    *reinterpret_cast<uint4*>(to + t * wk.o.t + y * 8) = *reinterpret_cast<const uint4*>(
                        sm + C::oO + (y >> 3) * kTile + t * 128 + (((y & 7) ^ (t & 7)) * 16));
                }
            }
            done(kOFree);
        }
        }
        if (!ok) s_fail = 1;
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 17) tc::dealloc(tm, 512);
    if (threadIdx.x == 0 && s_fail) atomicExch(a.err, 7);
}

// The states at the segments' ends, along a sequence in the walk's order: X_p =
// l^(tokens of a segment) X_(p-1) + N_p, float32, in place of N_p.  All segments but
// the walk's last are needed, all but its first are whole.  Four elements a thread,
// four segments in flight.
__global__ void __launch_bounds__(256) linattn_join_kernel(const __grid_constant__ Passes a, int size) {
    const Pass& x = a.p[blockIdx.z];
    const Walk& w = x.w;
    const int chunks = size / 1024, i = blockIdx.x / chunks, h = blockIdx.y;
    const Seq s = locate(w.offsets, w.T, i);
    const int64_t all = (s.len + kChunk - 1) / kChunk, nseg = (all + a.seg_chunks - 1) / a.seg_chunks;
    if (nseg < 3) return;
    const int64_t g0 = s.slot / a.seg_chunks + i, step = (w.reverse ? -1 : 1) * int64_t(w.H) * size;
    float4* at = reinterpret_cast<float4*>(x.seg_state + ((g0 + (w.reverse ? nseg - 1 : 0)) * w.H + h) * size +
                                           (blockIdx.x % chunks) * 1024 + threadIdx.x * 4);
    const Decay l = decay_over(head_decay(w.decay, h), float(a.seg_chunks * kChunk));
    float4 S = *at;
    for (int64_t p = 1; p + 1 < nseg; p += 4) {
        float4 N[4];
        #pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j + 1 < nseg) N[j] = *(at + (p + j) * step / 4);
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (p + j + 1 >= nseg) break;
            S = make_float4(decayed(l, S.x, N[j].x), decayed(l, S.y, N[j].y), decayed(l, S.z, N[j].z), decayed(l, S.w, N[j].w));
            *(at + (p + j) * step / 4) = S;
        }
    }
}

template <int DT, int DK, int DV>
cudaError_t launch(const Passes& a, int n, bool states, cudaStream_t st) {
    static PerDevice c0, c1;
    constexpr size_t bytes = Cfg<DK, DV>::BYTES;
    static_assert(bytes <= 232448, "shared memory");
    static_assert(kBars * 8 <= 240, "barriers");
    cudaError_t e = opt_in(linattn_walk_kernel<DT, DK, DV, false>, bytes, c0);
    if (e == cudaSuccess) e = opt_in(linattn_walk_kernel<DT, DK, DV, true>, bytes, c1);
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned(a.segments), unsigned(a.p[0].w.H), unsigned(n));
    if (states) {
        linattn_walk_kernel<DT, DK, DV, true><<<grid, Cfg<DK, DV>::THREADS, bytes, st>>>(a);
        constexpr int size = DK * DV;
        linattn_join_kernel<<<dim3(unsigned(a.p[0].w.nseq) * (size / 1024), grid.y, grid.z), 256, 0, st>>>(a, size);
    } else {
        linattn_walk_kernel<DT, DK, DV, false><<<grid, Cfg<DK, DV>::THREADS, bytes, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

// Segments.  A sequence's chunks follow one another, so few long sequences leave SMs
// idle.  Cut into segments a walk costs another over K and V for the segments' end
// states and a join.
void plan_segments(Segments* s, int64_t B, int64_t T, int64_t nseq, int64_t heads, int walks, int sms) {
    const int64_t slots = chunk_slots(B, T, nseq), rows = nseq * heads * walks;
    s->chunks = slots + 1;
    s->count = nseq;
    if (rows == 0 || rows >= sms) return;
    const int64_t L = (slots * heads * walks + sms - 1) / sms;
    if (L * 2 > (slots + nseq - 1) / nseq) return;
    s->chunks = L < 8 ? 8 : L;
    s->count = slots / s->chunks + nseq;
}

cudaError_t launch_linattn(const Passes& a, int n, bool states, int dt, int dk, int dv, cudaStream_t st) {
    if (dt == FFTCONV_F16) {
        if (dk == 64) return dv == 64 ? launch<0, 64, 64>(a, n, states, st) : launch<0, 64, 128>(a, n, states, st);
        return dv == 64 ? launch<0, 128, 64>(a, n, states, st) : launch<0, 128, 128>(a, n, states, st);
    }
    if (dk == 64) return dv == 64 ? launch<1, 64, 64>(a, n, states, st) : launch<1, 64, 128>(a, n, states, st);
    return dv == 64 ? launch<1, 128, 64>(a, n, states, st) : launch<1, 128, 128>(a, n, states, st);
}

}  // namespace fftconv
