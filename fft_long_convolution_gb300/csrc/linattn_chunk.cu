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
// Precision: S is float32, in the registers of the warps that update it.  What feeds it,
// w V, is taken in 16-bit parts: three for bf16 (24 bits) and two for fp16 (22 bits)
// where the state at the end of the walk is an output, so that it keeps float32's
// digits; two for bf16 (17 bits) where S only feeds O.  S and P enter O as one 16-bit
// value each: their roundings fall on the two terms of O's sum, by half a step of each
// factor's size.  Where the terms do not cancel O is off by about sqrt(2) times its own
// rounding alone; what is left of terms that do is off by their roundings all the same
// (two parts each, built and measured, gave O's rounding alone and took 1.3 times as
// long).  In fp16 a row of each of them is first scaled by a power of two to a largest
// value in [2^14, 2^15), and the accumulator scaled back: neither small values nor large
// states leave fp16's range.
//
// One CTA per sequence (or segment of one) and value head, roles by warp, handing
// over through mbarriers:
//   warps 0-15   w V in parts -> tensor memory; S: float32 += KV, and in 16 bits for S Q
//   warps 16-19  scores -> P;  warps 20-27  O -> shared memory
//   warp 28      loads, 3 to 5 chunks deep;  warp 30  O -> global memory
//   warp 29      issues KV and the next chunk's scores;  warp 31  S Q and P V
//
// Bound: HBM where segments fill the SMs (262144 tokens, 6 heads of 128 x 128, bf16:
// q, k, v read and o written in 250 us, 6.4 TB/s); else the chain of a chunk, 1.3 us in
// bf16 and 1.8 us in fp16 or with three parts at 128 x 128, 1.0 to 1.6 us at 64 x 64 (8 x
// 4096 tokens, 6 heads of 128: the three gradients' walks 92 us side by side).  Three
// loops of that chain are equally long: S Q, P V and the read of O; scores, P, P V and
// O; w V, KV and S.  The tensor pipe is active 40 % of the time, the schedulers issue in
// 55 %.
#include "linattn_chunk.h"

#include <algorithm>
#include <type_traits>

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

// Store 16 lanes x 8 or 16 columns: thread t holds, for every 4 columns, column t % 4 of
// lanes t / 4 and t / 4 + 8.
__device__ __forceinline__ void st16x128b_x2(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void st16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Bounded wait of a whole warp that sleeps until the phase is over, so that the roles
// that wait leave the issue slots to those that work.  Gives up after about a second,
// or when another role has (*fail set).  Each lane gets an answer of its own from a poll,
// so every one is voted on: the warp goes on as a whole, to instructions that ask for all
// its lanes, or rests as a whole.  Barriers that are waited for together share a vote
// (each by itself, prompts of uneven length in fp16 took 2 to 4 % longer).  The first poll
// nearly always suffices (it may suspend the warp for kWaitHintNs); what follows it is kept
// out of the roles' loops.
__device__ __forceinline__ bool poll(uint32_t addr, uint32_t parity) {
    uint32_t over;
    asm volatile(
        "{.reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;}"
        : "=r"(over)
        : "r"(addr), "r"(parity), "r"(kWaitHintNs)
        : "memory");
    return over;
}

__device__ __noinline__ bool rest_on(uint32_t addr, uint32_t parity, volatile int* fail) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0; it < (1u << 20); ++it) {
        if (__all_sync(0xffffffffu, poll(addr, parity))) return true;
        if (__any_sync(0xffffffffu, *fail || globaltimer_ns() - t0 > kWaitNs)) return false;
    }
    return false;
}

struct Phase {
    uint64_t* bar;
    uint32_t parity;  // of the phase; that before a barrier's first phase counts as over
    __device__ __forceinline__ uint32_t addr() const { return smem_u32(bar); }
};

__device__ __forceinline__ bool rest(volatile int* fail, const Phase& a) {
    if (__builtin_expect(__all_sync(0xffffffffu, poll(a.addr(), a.parity)), 1)) return true;
    return rest_on(a.addr(), a.parity, fail);
}

__device__ __forceinline__ bool rest(volatile int* fail, const Phase& a, const Phase& b) {
    const bool x = poll(a.addr(), a.parity), y = poll(b.addr(), b.parity);
    if (__builtin_expect(__all_sync(0xffffffffu, x && y), 1)) return true;
    return rest_on(a.addr(), a.parity, fail) && rest_on(b.addr(), b.parity, fail);
}

__device__ __forceinline__ bool rest(volatile int* fail, const Phase& a, const Phase& b, const Phase& c) {
    const bool x = poll(a.addr(), a.parity), y = poll(b.addr(), b.parity), z = poll(c.addr(), c.parity);
    if (__builtin_expect(__all_sync(0xffffffffu, x && y && z), 1)) return true;
    return rest_on(a.addr(), a.parity, fail) && rest_on(b.addr(), b.parity, fail) && rest_on(c.addr(), c.parity, fail);
}

// Pairs of 16-bit values: products, fused products, a b - c, and the larger sizes.
template <int DT>
struct Pair {
    static __device__ __forceinline__ uint32_t mul(uint32_t a, uint32_t b) {
        uint32_t r;
        if (DT == 0) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t fma(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        if (DT == 0) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    static __device__ __forceinline__ uint32_t fma_less(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        if (DT == 0) asm("{.reg .b32 n;\n neg.f16x2 n, %3;\n fma.rn.f16x2 %0, %1, %2, n;}" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        else asm("{.reg .b32 n;\n neg.bf16x2 n, %3;\n fma.rn.bf16x2 %0, %1, %2, n;}" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {  // |a|, |b|; DT 0
        uint32_t r;
        asm("{.reg .b32 x, y;\n abs.f16x2 x, %1;\n abs.f16x2 y, %2;\n max.f16x2 %0, x, y;}" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// A power of two that takes a row's largest size x into [2^14, 2^15), and its
// inverse; for sizes below 2^-112 that of 2^-112.
__device__ __forceinline__ float2 row_scale(float x) {
    const uint32_t e = min(max(__float_as_uint(x) >> 23, 15u), 254u);
    return make_float2(__uint_as_float((268u - e) << 23), __uint_as_float((e - 14u) << 23));
}

constexpr int kThreads = 1024, kMaxStages = 5;

// Shared memory: stages of K, Q (not where only the states are wanted) and V, P twice, O,
// tables, barriers.  A stage is held for one and a half steps and takes another to load
// again: as many as fit, up to 5 (three at 128 x 128; gradients of 150 rows of 4096, heads
// of 64 x 64, fp16: 316 us, with three stages 325).
// Up to 4 where only the states are wanted, as the scales' places there rely on it.
template <int DK_, int DV_, bool STATE>
struct Cfg {
    static constexpr int KT = DK_ / 64, VT = DV_ / 64;  // tiles of K and of Q, of V
    static constexpr uint32_t sK = 0, sQ = KT * kTile, sV = (STATE ? 1 : 2) * KT * kTile, STAGE = sV + VT * kTile;
    // float tables: w and u for a whole chunk and for a last one; w of two tokens in two
    // 16-bit parts, packed [2][32][2]; the decays between a chunk's tokens (pairs); the
    // scales of w V [8][128] back, S [2][128] and P [2][64]; the rows' sizes of S
    // [2][4][128]; the scales of w V
    static constexpr uint32_t tW = 0, tU = 128, tH = 256, tD = 384, tV = 640, tS = tV + 1024, tP = tS + 256;
    static constexpr uint32_t tM = tP + 128, tN = tM + 1024, TABLE = (tN + 512) * 4;
    static constexpr uint32_t kBarBytes = 336, kMost = 232448, kRest = (2 + VT) * kTile + TABLE + kBarBytes;
    static constexpr int kFit = (kMost - kRest) / STAGE, kUse = STATE ? 4 : kMaxStages, NST = kFit < kUse ? kFit : kUse;
    static_assert(NST >= 3, "stages");
    static constexpr uint32_t oP = NST * STAGE, oO = oP + 2 * kTile, oT = oO + VT * kTile, oBar = oT + TABLE, BYTES = oBar + kBarBytes;
    // Tensor memory columns: S; S Q; scores and then P V; KV; w V, all 512 at Dk = 128.
    // w V has two buffers.  With its two parts the scores have two and KV one, and two at
    // Dk = 64, where there is room (2 % of a step in bf16).  With three parts (fine) KV has
    // one, the scores one, and two at Dk = 64 (150 rows of 4096 with final states: 82 us at
    // 64 x 64, 124 at 128 x 128; with one buffer of w V and two of the scores 101 and 131).
    // Where only the states are wanted: KV and w V.
    static __host__ __device__ constexpr int nx(bool fine) { return fine && DK_ == 128 ? 1 : 2; }
    static __host__ __device__ constexpr int nkv(bool fine) { return STATE || (!fine && DK_ == 64) ? 2 : 1; }
    static constexpr uint32_t cS = 0, cOi = DK_ / 2, cX = cOi + 64;
    static __host__ __device__ constexpr uint32_t x(bool fine, int c) { return cX + (nx(fine) == 2 ? (c & 1) * 64 : 0); }
    static __host__ __device__ constexpr uint32_t kv(bool fine, int c) {
        return (STATE ? 0 : cX + nx(fine) * 64) + (nkv(fine) == 2 ? (c & 1) * DK_ : 0);
    }
    static __host__ __device__ constexpr uint32_t w(bool fine, int c) {
        return kv(fine, 0) + nkv(fine) * DK_ + (c & 1) * (fine ? 96 : 64);
    }
    static_assert(w(false, 1) + 64 <= 512 && w(true, 1) + 96 <= 512, "tensor memory");
};

enum Bar {
    kFull = 0, kFree = kMaxStages,  // by stage
    // by chunk parity
    kKvDone = 2 * kMaxStages, kKvRead = kKvDone + 2, kParts = kKvRead + 2, kScDone = kParts + 2, kORead = kScDone + 2,
    kPReady = kORead + 2, kPvDone = kPReady + 2,
    kRaw = kPvDone + 2, kSop, kSqDone, kOReady, kOFree,
    kFinal,            // [2]
    kSizes = kFinal + 2,  // [4]
    kMax = kSizes + 4, kBars = kMax + 4  // the four warps of 32 lanes of S
};

// A stage of the loads and the parity of its barriers, step after step.
template <int N>
struct Ring {
    int st = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) {
            st = 0;
            parity ^= 1;
        }
    }
};

// Where a CTA's part of a sequence is.
struct Part {
    Seq s;
    int i;              // sequence
    int64_t state;      // where the state at its end is, unless it is the walk's last one
    int64_t tok0;       // its first token in the row
    int64_t left;       // tokens from there to the sequence's end
    int n;              // chunks
    int count, before;  // segments of the sequence, and those before this one in the walk's order
    bool first, last;   // in that order
};

__device__ __forceinline__ bool find_part(const Walk& w, uint32_t L, uint32_t slot, Part* p) {
    int lo = 0, hi = w.nseq - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (uint32_t(locate(w.offsets, w.T, m).slot) / L + m <= slot) lo = m;
        else hi = m - 1;
    }
    p->i = lo;
    p->s = locate(w.offsets, w.T, lo);
    const int64_t seg = int64_t(slot) - (uint32_t(p->s.slot) / L + lo), all = (p->s.len + kChunk - 1) / kChunk, from = seg * L;
    if (seg < 0 || (seg > 0 && from >= all)) return false;
    const bool low = seg == 0, high = from + L >= all;
    p->first = w.reverse ? high : low;
    p->last = w.reverse ? low : high;
    p->n = int(high ? all - from : L);
    p->count = int((uint32_t(all) + L - 1) / L);
    p->before = int(w.reverse ? p->count - 1 - seg : seg);
    p->state = int64_t(uint32_t(p->s.slot) / L) + seg - (w.reverse ? 1 : 0);
    p->tok0 = p->s.start + from * kChunk;
    p->left = p->s.len - from * kChunk;
    return true;
}

// The slot of the part of a given rank by length, of up to 32 sequences, a lane for each;
// -1: there is none.  Whole segments come first, in the order of the row, then what is
// left of each sequence.  All lanes of a warp.  Packed sequences start in this order, as
// the longest one ends the launch: 24 sequences of 1 to 2000 tokens with 12 heads take
// 75 us, in the order of the row 94.  More than 32 start in the order of the row.
__device__ __forceinline__ int64_t by_length(const Walk& w, uint32_t L, int rank) {
    const int lane = threadIdx.x % 32;
    const bool real = lane < w.nseq;
    const Seq s = locate(w.offsets, w.T, real ? lane : 0);
    const uint32_t all = real ? uint32_t((s.len + kChunk - 1) / kChunk) : 0;
    const int full = int(all / L), left = int(all - uint32_t(full) * L);
    int upto = full;  // whole segments of this and the sequences before
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    const int whole = __shfl_sync(0xffffffffu, upto, 31);
    const bool has = real && (left > 0 || all == 0);
    const int key = has ? left : -1;
    int longer = 0;
    #pragma unroll 1
    for (int i = 0; i < 32; ++i) {
        const int y = __shfl_sync(0xffffffffu, key, i);
        longer += y > key || (y == key && i < lane);
    }
    const bool mine = rank < whole ? upto > rank && upto - full <= rank : has && longer == rank - whole;
    const uint32_t found = __ballot_sync(0xffffffffu, mine);
    const int64_t slot = int64_t(uint32_t(s.slot) / L) + lane + (rank < whole ? rank - (upto - full) : full);
    return found ? __shfl_sync(0xffffffffu, slot, __ffs(found) - 1) : -1;
}

// The slot of the part of a given rank, in the order of the row, among those of sequences
// that are cut; -1: there is none.  32 sequences at a time, a lane for each.  All lanes of
// a warp.
__device__ __forceinline__ int64_t cut_part(const Walk& w, uint32_t L, int rank) {
    const int lane = threadIdx.x % 32;
    #pragma unroll 1
    for (int i0 = 0; i0 < w.nseq; i0 += 32) {
        const bool real = i0 + lane < w.nseq;
        const Seq s = locate(w.offsets, w.T, real ? i0 + lane : 0);
        const uint32_t all = real ? uint32_t((s.len + kChunk - 1) / kChunk) : 0;
        const int parts = all > L ? int((all + L - 1) / L) : 0;
        int upto = parts;  // of this and the sequences before
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int before = upto - parts;
        const uint32_t found = __ballot_sync(0xffffffffu, upto > rank && before <= rank);
        const int64_t slot = int64_t(uint32_t(s.slot) / L) + i0 + lane + (rank - before);
        if (found) return __shfl_sync(0xffffffffu, slot, __ffs(found) - 1);
        rank -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return -1;
}

// STATE: only the state at the end of a segment (from zero, or from the initial state);
// a walk's last one, if the final state is wanted, to where that goes.  Sequences of one
// segment are left to the walk.
template <int DT, int DK, int DV, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) linattn_walk_kernel(const __grid_constant__ Passes a) {
    using C = Cfg<DK, DV, STATE>;
    constexpr int NC = DK / 4;  // columns of S of a thread
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + C::oBar);
    // no static shared memory: the window starts 1024-byte aligned
    uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + C::oBar + 320);
    volatile int& s_fail = *reinterpret_cast<volatile int*>(sm + C::oBar + 324);
    float* tab = reinterpret_cast<float*>(sm + C::oT);
    int slot = blockIdx.x, h = blockIdx.y, z = blockIdx.z;
    if (a.longest_first) {  // all heads of a sequence before the next sequence
        slot += gridDim.x * (h + gridDim.y * z);
        h = slot % gridDim.y;
        slot /= gridDim.y;
        z = slot % gridDim.z;
        slot /= gridDim.z;
    }
    const Pass& x = a.p[z];
    const Walk& wk = x.w;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    // out of the indexed parameter once, not at every use
    const bool reverse = wk.reverse, packed = wk.offsets != nullptr;
    float* o32 = wk.o32;
    if (sb & 1023) {  // not with the present layout of the window
        if (threadIdx.x == 0) atomicExch(a.err, 7);
        return;
    }
    // one warp looks for the part, the others take it from shared memory
    Part p;
    bool live;
    {
        Part* found = reinterpret_cast<Part*>(sm + C::oO);
        bool* any = reinterpret_cast<bool*>(found + 1);
        if (warp == 0) {
            int64_t at = slot;
            if (STATE ? a.few_cut : a.longest_first)
                at = STATE ? cut_part(wk, uint32_t(a.seg_chunks), slot) : by_length(wk, uint32_t(a.seg_chunks), slot);
            live = at >= 0 && find_part(wk, uint32_t(a.seg_chunks), uint32_t(at), &p);
            if (lane == 0) *found = p, *any = live;
        }
        __syncthreads();
        p = *found;
        live = *any;
        __syncthreads();
    }
    if (!live || (STATE && p.last && (p.first || !wk.state_out))) return;
    const int n = p.n;
    const int64_t hs = int64_t(p.i) * wk.H + h, gs = p.state * wk.H + h;
    const float* sin = wk.state_in ? wk.state_in + hs * DK * DV : nullptr;
    // what the walk's segment before left, and the way to those before it
    const int64_t back = (reverse ? 1 : -1) * int64_t(wk.H) * DK * DV;
    if (!p.first) sin = STATE ? nullptr : x.seg_state + gs * DK * DV + back;
    float* fin = p.last && wk.state_out ? wk.state_out + hs * DK * DV : nullptr;
    float* sout = STATE ? (p.last ? fin : x.seg_state + gs * DK * DV) : p.first ? fin : nullptr;
    // w V in three parts (bf16) where the state at the end is wanted for itself
    const bool fine = DT == 1 && (STATE || sout);
    const int parts = fine ? 3 : 2;

    if (threadIdx.x == 0) {
        s_fail = 0;
        for (int i = 0; i < kBars; ++i) {
            uint32_t cnt = 1;  // else one arrival per warp of the role
            if (i == kPReady || i == kPReady + 1 || i >= kSizes) cnt = 4;
            if (i == kORead || i == kORead + 1 || i == kOReady) cnt = 8;
            if (i >= kFree && i < kFree + kMaxStages && !STATE) cnt = 2;  // both warps that issue products
            if (i == kParts || i == kParts + 1) cnt = fine ? 16 : 8;
            if (i == kSop || i == kKvRead || i == kKvRead + 1) cnt = 16;
            mbar_init(bar + i, cnt);
        }
        fence_mbar_init();
    }
    const float g = head_decay(wk.decay, h);
    if (threadIdx.x < 128) {
        const int j = threadIdx.x & 63;
        const int m = threadIdx.x < 64 ? 64 : int((p.s.len - 1) % kChunk) + 1;
        const int back = m - 1 - j, on = j + 1;
        // fp16 holds weights of at most 1: what is common to them goes with the rows' scales
        const float w = back >= 0 ? (DT == 0 ? expf(g * float(reverse ? j : back)) : wk.s_up * expf(g * float(reverse ? on : back))) : 0.0f;
        tab[C::tW + threadIdx.x] = w;
        const float wh = Op<DT>::unpack(Op<DT>::pack(w, 0.0f)).r;
        uint16_t* half = reinterpret_cast<uint16_t*>(tab + C::tH) + (threadIdx.x >> 1) * 4 + (threadIdx.x & 1);
        half[0] = uint16_t(Op<DT>::pack(wh, 0.0f));
        half[2] = uint16_t(Op<DT>::pack(w - wh, 0.0f));
        tab[C::tU + threadIdx.x] = back >= 0 ? wk.s_in * expf(g * float(reverse ? back : on)) : 0.0f;
    } else if (threadIdx.x < 384) {
        // entry 64 + i - j: the decays of (i, j) and (i, j + 1)
        const int e = threadIdx.x - 128, d = (e >> 1) - 64 - (e & 1), t = reverse ? -d : d;
        tab[C::tD + e] = t >= 0 ? wk.s_p * expf(g * float(t)) : 0.0f;
    }
    if (warp == 29) tc::alloc(&s_tmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = *const_cast<volatile uint32_t*>(&s_tmem);
    volatile int* fail = &s_fail;
    const int sp = warp & 3;
    const uint32_t lanes = tm + (uint32_t(32 * sp) << 16);  // this warp's tensor-memory lanes
    const int row = 32 * sp + lane;                         // this thread's lane
    // 64 value features: nothing is written to the upper lanes and nothing read from them,
    // as each lane's products are its own; their warps only keep step
    const bool mine = 32 * sp < DV;
    // one arrival per warp, after every lane's work
    auto done = [&](int b) {
        __syncwarp();
        if (lane == 0) arrive(bar + b);
    };
    // a barrier's phases from 0 on; the one before them is over from the start
    auto at = [&](int b, uint32_t phase) { return Phase{bar + b, phase & 1}; };
    auto wait = [&](const auto&... phases) { return rest(fail, phases...); };
    // step c's chunk, and its tokens
    auto chunk = [&](int c) { return reverse ? n - 1 - c : c; };
    const int all = int(p.left < int64_t(n) * kChunk ? p.left : int64_t(n) * kChunk);
    auto tokens = [&](int c) { return min(all - chunk(c) * kChunk, kChunk); };
    bool ok = true;
    int c = 0;

    // The roles' loops are kept short and rolled: they share the instruction cache, and
    // straight code that runs once a chunk is fetched once a chunk (unrolled, 90 KB of
    // code, a chunk of 64 tokens took 6100 cycles).
    if (n == 0) {
        // an empty sequence: the state passes through
        if (sout)
            for (int e = threadIdx.x; e < DK * DV; e += kThreads) {
                float v = 0.0f;
                if (sin) v = wk.turned ? sin[(e % DV) * DK + e / DV] : sin[e];
                sout[e] = v;
            }
    } else if (warp < 16) {
        // ---------------------------------------------------------------- S
        const int dv = row, quarter = warp >> 2, k0 = quarter * NC;
        float2 S[NC / 2] = {};
        // the state before: one that is given or joined, or the end states of all segments
        // before, the first one first
        const bool join = !STATE && !p.first && p.count <= a.join;
        const Decay over = decay_over(g, float(a.seg_chunks * kChunk));
        #pragma unroll 1
        for (int i = join ? p.before : 1; mine && sin && i > 0; --i) {
            const float* from = sin + (i - 1) * back;
            #pragma unroll
            for (int j = 0; j < NC / 2; ++j) {
                const int k = k0 + 2 * j;
                const float2 N = wk.turned ? *reinterpret_cast<const float2*>(from + dv * DK + k)
                                           : make_float2(from[k * DV + dv], from[(k + 1) * DV + dv]);
                S[j] = make_float2(decayed(over, S[j].x, N.x), decayed(over, S[j].y, N.y));
            }
        }
        if (join && fin && mine) {  // and the sequence's final state
            float* out = fin + dv;
            const Decay rest_of = decay_over(g, float(all));
            #pragma unroll
            for (int j = 0; j < NC; ++j) {
                float& y = out[(k0 + j) * DV];
                y = decayed(rest_of, j & 1 ? S[j / 2].y : S[j / 2].x, y);
            }
        }
        const Decay whole = decay_over(g, float(kChunk));
        const Decay last = decay_over(g, float(tokens(reverse ? 0 : n - 1)));
        // w V in parts.  A warp takes 16 features; a block of 16 tokens of them comes
        // transposed from ldmatrix, as 8 features x 8 tokens four times, in the order in
        // which tensor memory takes them.
        const int hf = quarter >> 1, side = quarter & 1;
        const uint32_t v_at = sb + C::sV + (sp >> 1) * kTile + ((lane >> 4) * 8 + (lane & 7)) * 128 +
                              ((((sp & 1) * 4 + hf * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) * 16);
        auto block = [&](int st, int b, uint32_t* v) { ldsm_t(v_at + st * C::STAGE + b * 2048, v[0], v[1], v[2], v[3]); };
        const uint32_t w_at = lanes + (uint32_t(16 * hf) << 16);
        Ring<C::NST> full;
        // Three parts: a warp half of the tokens of every step.
        auto weigh_fine = [&](int e) {
            if (!wait(at(kFull + full.st, full.parity))) return false;
            tc::fence_after();
            const float* wt = tab + C::tW + (tokens(e) < kChunk ? 64 : 0) + 32 * side + 2 * (lane & 3);
            const uint32_t to = w_at + C::w(true, e) + 16 * side;
            #pragma unroll 1
            for (int b = 0; mine && b < 2; ++b) {
                uint32_t v[4], hi[4], lo[4], l2[4];
                block(full.st, 2 * side + b, v);
                #pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const cpx u = Op<DT>::unpack(v[i]);
                    const float2 y = mul2(make_float2(u.r, u.i), *reinterpret_cast<const float2*>(wt + 16 * b + 8 * (i >> 1)));
                    hi[i] = Op<DT>::pack(y.x, y.y);
                    const cpx z = Op<DT>::unpack(hi[i]);
                    split<DT>(sub2(y, make_float2(z.r, z.i)), &lo[i], &l2[i]);
                }
                st16x128b_x2(to + 8 * b, hi);
                st16x128b_x2(to + 8 * b + 32, lo);
                st16x128b_x2(to + 8 * b + 64, l2);
            }
            full.next();
            tc::wait_st();
            tc::fence_before();
            done(kParts + (e & 1));
            return true;
        };
        // Two parts, without leaving 16 bits: with w = wh + wm, the product v wh rounds to hi
        // and leaves an error that 16 bits hold exactly, which a fused multiply-add gives:
        // lo = v wm + (v wh - hi).  A warp all tokens of every other step, a step ahead.
        auto weigh = [&](int e) {
            const Phase loaded = at(kFull + full.st, full.parity);
            if (!(DT == 0 ? wait(loaded, at(kSizes + (e & 3), e >> 2)) : wait(loaded))) return false;
            tc::fence_after();
            const float* wt = tab + C::tH + (tokens(e) < kChunk ? 64 : 0) + 2 * (lane & 3);
            const uint32_t to = w_at + C::w(false, e);
            uint32_t sc[2] = {};
            if constexpr (DT == 0) {
                const uint32_t* z = reinterpret_cast<const uint32_t*>(tab + C::tN) + (e & 3) * 128 + 32 * sp + 16 * hf + (lane >> 2);
                sc[0] = z[0];
                sc[1] = z[8];
            }
            #pragma unroll 1
            for (int b = 0; mine && b < 4; b += 2) {
                uint32_t v[8], hi[8], lo[8];
                block(full.st, b, v);
                block(full.st, b + 1, v + 4);
                #pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint2 w = *reinterpret_cast<const uint2*>(wt + 16 * b + 8 * (i >> 1));
                    if constexpr (DT == 0) v[i] = Pair<DT>::mul(v[i], sc[i & 1]);
                    hi[i] = Pair<DT>::mul(v[i], w.x);
                    lo[i] = Pair<DT>::fma(v[i], w.y, Pair<DT>::fma_less(v[i], w.x, hi[i]));
                }
                st16x128b_x4(to + 8 * b, hi);
                st16x128b_x4(to + 8 * b + 32, lo);
            }
            full.next();
            full.next();
            tc::wait_st();
            tc::fence_before();
            done(kParts + (e & 1));
            return true;
        };
        // S for step e, after S Q of the step before
        auto put = [&](int e) {
            float2 sc = make_float2(1.0f, 1.0f);
            if (DT == 0 && mine) {
                float m = 0.0f;
                #pragma unroll
                for (int j = 0; j < NC / 2; ++j) m = fmaxf(m, fmaxf(fabsf(S[j].x), fabsf(S[j].y)));
                float* size = tab + C::tM + (e & 1) * 512 + row;
                size[quarter * 128] = m;
                done(kMax + sp);
                if (!wait(at(kMax + sp, e))) return false;
                #pragma unroll
                for (int j = 1; j < 4; ++j) m = fmaxf(m, size[((quarter + j) & 3) * 128]);
                sc = row_scale(m);
            }
            if (!wait(at(kSqDone, e - 1))) return false;
            tc::fence_after();
            if (DT == 0 && quarter == 0) tab[C::tS + (e & 1) * 128 + row] = sc.y;
            #pragma unroll
            for (int b = 0; b < NC; b += 16) {
                if (!mine) break;
                uint32_t y[8];
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 v = DT == 0 ? mul2(S[b / 2 + j], make_float2(sc.x, sc.x)) : S[b / 2 + j];
                    y[j] = Op<DT>::pack(v.x, v.y);
                }
                st_cols<8>(lanes + C::cS + (k0 + b) / 2, y);
            }
            tc::wait_st();
            tc::fence_before();
            done(kSop);
            return true;
        };
        // S += KV of step e
        auto add = [&](int e, auto exact) {  // exact: S is an output, else it only feeds O
            if (!wait(at(kKvDone + (e & 1), e >> 1))) return false;
            tc::fence_after();
            const Decay l = tokens(e) < kChunk ? last : whole;
            const float2 part = make_float2(l.part, l.part), keep = make_float2(l.keep, l.keep);
            const float2 whole_l = make_float2(l.keep + l.part, l.keep + l.part);
            float inv = 1.0f;
            if constexpr (DT == 0) inv = tab[C::tV + (e & 7) * 128 + row];
            #pragma unroll
            for (int b = 0; b < NC; b += 16) {
                if (!mine) break;
                uint32_t y[16];
                ld16(lanes + C::kv(fine, e) + k0 + b, y);
                tc::wait_ld();
                #pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float2& s = S[b / 2 + j];
                    const float2 kv = pair(y[2 * j], y[2 * j + 1]);
                    if constexpr (exact.value) {
                        const float2 t = DT == 0 ? fma2(kv, make_float2(inv, inv), mul2(part, s)) : fma2(part, s, kv);
                        s = fma2(keep, s, t);
                    } else {
                        s = fma2(whole_l, s, kv);
                    }
                }
            }
            tc::fence_before();
            done(kKvRead + (e & 1));
            return true;
        };
        if (fine) {
            // w V of step c goes into the buffer of step c - 2, whose products add() has
            // waited for, while KV of step c - 1 is formed
            #pragma unroll 1
            for (; ok && c <= n; ++c) {
                if (c < n) ok = weigh_fine(c);
                if (ok && c > 0) ok = add(c - 1, std::true_type());
                if (!STATE && ok && c < n) ok = put(c);
            }
        } else {
            // w V of step c goes into the buffer of step c - 2, whose products add() has
            // waited for: the warps of one side take the even steps, those of the other
            // the odd ones
            if (side) full.next();
            else ok = weigh(0);
            #pragma unroll 1
            for (; ok && c <= n; ++c) {
                if (c > 0) ok = add(c - 1, std::bool_constant<DT == 0>());
                if (!STATE && ok && c < n) ok = put(c);
                if (ok && c + 1 < n && ((c + 1) & 1) == side) ok = weigh(c + 1);
            }
        }
        if (ok && sout && mine) {
            #pragma unroll
            for (int j = 0; j < NC / 2; ++j) {
                sout[(k0 + 2 * j) * DV + dv] = S[j].x;
                sout[(k0 + 2 * j + 1) * DV + dv] = S[j].y;
            }
        }
    } else if (warp < 20) {
        // ---------------------------------------------------------------- P
        // rows i = 16 sp + q and i + 8, columns j = 8 b + 2 r and the next
        const int q = lane >> 2, r = lane & 3;
        const float2* dt = reinterpret_cast<const float2*>(tab + C::tD) + 64 + 16 * sp + q - 2 * r;
        // fp16: the scales of V's rows, two chunks ahead.  A lane takes 8 of the warp's 32
        // features, 8 tokens.  There are places for the scales of 4 chunks and for 8 of their
        // inverses.  When those of chunk e are written, w V has used the scales of chunk
        // e - 4, and S has added KV up to chunk e - 6: P V of chunk e - 4 is over (P waits
        // for it), before which all warps of S have put it, weighed V and added KV; where
        // only the states are wanted, chunk e - 4 has left its stage, so its KV is over.
        const float s_up = reverse ? wk.s_up * expf(g) : wk.s_up;  // (see the weights)
        Ring<C::NST> full;
        auto sizes = [&](int e) {
            if (!wait(at(kFull + full.st, full.parity))) return false;
            if (!mine) {
                full.next();
                done(kSizes + (e & 3));
                return true;
            }
            const int f8 = lane & 3, t8 = lane >> 2;
            const uint8_t* v = sm + full.st * C::STAGE + C::sV + (sp >> 1) * kTile + t8 * 1024;
            uint32_t m[4] = {};
            #pragma unroll
            for (int t = 0; t < 8; ++t) {
                const uint4 y = *reinterpret_cast<const uint4*>(v + t * 128 + ((((sp & 1) * 4 + f8) ^ t) * 16));
                const uint32_t z[4] = {y.x, y.y, y.z, y.w};
                #pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = Pair<DT>::larger(m[i], z[i]);
            }
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                #pragma unroll
                for (int o = 4; o < 32; o <<= 1) m[i] = Pair<DT>::larger(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
            // feature 8 f8 + t8 is this lane's: a power of two that takes its largest to
            // [2^14, 2^15) (at most 2^15 itself)
            const uint32_t z = (t8 & 4 ? (t8 & 2 ? m[3] : m[2]) : (t8 & 2 ? m[1] : m[0])) >> (t8 & 1) * 16 & 0x7fffu;
            const uint32_t x = min(44u - (z >> 10), 30u), at = (e & 3) * 128 + 32 * sp + 8 * f8 + t8;
            reinterpret_cast<uint32_t*>(tab + C::tN)[at] = x << 10 | x << 26;
            tab[C::tV + (e & 7) * 128 + (at & 127)] = s_up * __uint_as_float((142u - x) << 23);
            full.next();
            done(kSizes + (e & 3));
            return true;
        };
        if (DT == 0) ok = sizes(0) && (n < 2 || sizes(1));
        if (STATE && DT == 0)
            #pragma unroll 1
            for (c = 2; ok && c < n; ++c) ok = sizes(c);
        #pragma unroll 1
        for (; !STATE && ok && c < n; ++c) {
            // the scores are there, and the buffer's last P has been used
            ok = wait(at(kScDone + (c & 1), c >> 1), at(kPvDone + (c & 1), (c - 2) >> 1));
            if (!ok) break;
            tc::fence_after();
            uint8_t* to = sm + C::oP + (c & 1) * kTile + (16 * sp + q) * 128 + r * 4;
            uint32_t y[32];
            tc::ld16x256b_x8(lanes + C::x(fine, c), y);
            tc::wait_ld();
            float m0 = 0.0f, m1 = 0.0f;
            float2 z0 = make_float2(1.0f, 1.0f), z1 = z0;
            #pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float2 v = mul2(pair(y[2 * e], y[2 * e + 1]), dt[(e & 1) * 8 - 8 * (e >> 1)]);
                y[2 * e] = __float_as_uint(v.x);
                y[2 * e + 1] = __float_as_uint(v.y);
                float& m = e & 1 ? m1 : m0;
                if (DT == 0) m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
            if constexpr (DT == 0) {
                #pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                    m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                }
                z0 = row_scale(m0);
                z1 = row_scale(m1);
                if (r == 0) {
                    tab[C::tP + (c & 1) * 64 + 16 * sp + q] = z0.y;
                    tab[C::tP + (c & 1) * 64 + 16 * sp + q + 8] = z1.y;
                }
            }
            #pragma unroll
            for (int e = 0; e < 16; ++e) {
                float2 v = pair(y[2 * e], y[2 * e + 1]);
                const float z = e & 1 ? z1.x : z0.x;
                if (DT == 0) v = mul2(v, make_float2(z, z));
                // rows i and i + 8 turn alike
                *reinterpret_cast<uint32_t*>(to + (e & 1) * 1024 + (((e >> 1) ^ q) * 16)) = Op<DT>::pack(v.x, v.y);
            }
            tc::fence_proxy_async();
            tc::fence_before();
            done(kPReady + (c & 1));
            if (DT == 0 && c + 2 < n) ok = sizes(c + 2);
        }
    } else if (warp < 28) {
        // ---------------------------------------------------------------- O
        // 16 features a warp, 32 tokens at a time
        const int q = lane >> 2, r = lane & 3, hf = (warp >> 2) & 1, f = 32 * sp + 16 * hf + q;
        const int piece = (sp & 1) * 4 + hf * 2 + ((lane >> 3) & 1);
        const uint32_t stage = sb + C::oO + (sp >> 1) * kTile + ((lane >> 4) * 8 + (lane & 7)) * 128 + ((piece ^ (lane & 7)) * 16);
        const int o32_token = wk.H * DV;
        if (o32) o32 += (p.s.row * wk.T + p.tok0) * o32_token + h * DV + f;
        #pragma unroll 1
        for (; !STATE && c < n; ++c) {
            const Phase formed = at(kPvDone + (c & 1), c >> 1);
            ok = o32 ? wait(formed) : wait(formed, at(kOFree, c - 1));  // the last O has left shared memory
            if (!ok) break;
            tc::fence_after();
            if (!mine) {
                done(kORead + (c & 1));
                if (!o32) done(kOReady);
                continue;
            }
            const int m = tokens(c);
            const float* ut = tab + C::tU + (m < kChunk ? 64 : 0) + 2 * r;
            const float* pt = tab + C::tP + (c & 1) * 64 + 2 * r;
            float s0 = 1.0f, s1 = 1.0f;
            if constexpr (DT == 0) {
                s0 = tab[C::tS + (c & 1) * 128 + f];
                s1 = tab[C::tS + (c & 1) * 128 + f + 8];
            }
            #pragma unroll 1
            for (int t0 = 0; t0 < 64; t0 += 32) {
                uint32_t y[16], z[16];
                const uint32_t from = lanes + (uint32_t(16 * hf) << 16) + t0;
                tc::ld16x256b_x4(from + C::cOi, y);
                tc::ld16x256b_x4(from + C::x(fine, c), z);
                tc::wait_ld();
                if (DT != 0 && t0) {  // the accumulators have been read
                    tc::fence_before();
                    done(kORead + (c & 1));
                }
                #pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 u = *reinterpret_cast<const float2*>(ut + t0 + 8 * e);
                    float2 e0 = pair(z[4 * e], z[4 * e + 1]), e1 = pair(z[4 * e + 2], z[4 * e + 3]);
                    float2 u0 = u, u1 = u;
                    if constexpr (DT == 0) {
                        const float2 ps = *reinterpret_cast<const float2*>(pt + t0 + 8 * e);
                        e0 = mul2(e0, ps);
                        e1 = mul2(e1, ps);
                        u0 = mul2(u, make_float2(s0, s0));
                        u1 = mul2(u, make_float2(s1, s1));
                    }
                    e0 = fma2(u0, pair(y[4 * e], y[4 * e + 1]), e0);
                    e1 = fma2(u1, pair(y[4 * e + 2], y[4 * e + 3]), e1);
                    y[4 * e] = __float_as_uint(e0.x), y[4 * e + 1] = __float_as_uint(e0.y);
                    y[4 * e + 2] = __float_as_uint(e1.x), y[4 * e + 3] = __float_as_uint(e1.y);
                }
                if (DT == 0 && t0) {  // the accumulators and the scales have been read
                    tc::fence_before();
                    done(kORead + (c & 1));
                }
                if (o32) {
                    float* to = o32 + int64_t(chunk(c)) * kChunk * o32_token;
                    #pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = t0 + 8 * (e >> 2) + 2 * r + (e & 1);
                        if (t < m) to[int64_t(t) * o32_token + (e & 2) * 4] = __uint_as_float(y[e]);
                    }
                    continue;
                }
                #pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    uint32_t o[4];
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = Op<DT>::pack(__uint_as_float(y[4 * e + 2 * i]), __uint_as_float(y[4 * e + 2 * i + 1]));
                    stsm_t(stage + (t0 + 8 * e) * 128, o[0], o[1], o[2], o[3]);
                }
            }
            if (o32) continue;
            tc::fence_proxy_async();
            done(kOReady);
        }
    } else if (warp == 28) {
        // ---------------------------------------------------------------- loads
        const int row0 = int(p.s.row);
        auto fix = [&](uint8_t* t, int m) {  // zero rows m .. 63 of a tile
            for (int e = lane; e < (64 - m) * 8; e += 32) *reinterpret_cast<uint4*>(t + m * 128 + e * 16) = make_uint4(0, 0, 0, 0);
        };
        Ring<C::NST> ring;
        #pragma unroll 1
        for (; c < n; ++c, ring.next()) {
            const int st = ring.st, t0 = int(p.tok0) + chunk(c) * kChunk, m = tokens(c);
            // rows past the sequence: the TMA engine writes zeros past the tensor's
            // end; in a packed row they are the next sequence's and are zeroed here
            const bool tail = packed && m < kChunk;  // one chunk at most
            uint8_t* to = sm + st * C::STAGE;
            if (c >= C::NST && !(ok = wait(at(kFree + st, ring.parity ^ 1)))) break;
            uint64_t* full = tail ? bar + kRaw : bar + kFull + st;
            if (elect()) {
                mbar_expect_tx(full, C::STAGE);
                #pragma unroll
                for (int f = 0; f < C::KT; ++f) {
                    tma_load_4d(smem_u32(to) + C::sK + f * kTile, &x.mk, f * 64, h / wk.gk, t0, row0, full);
                    if (!STATE) tma_load_4d(smem_u32(to) + C::sQ + f * kTile, &x.mq, f * 64, h / wk.gq, t0, row0, full);
                }
                #pragma unroll
                for (int f = 0; f < DV / 64; ++f)
                    tma_load_4d(smem_u32(to) + C::sV + f * kTile, &x.mv, f * 64, h / wk.gv, t0, row0, full);
            }
            __syncwarp();
            if (tail) {
                if (!(ok = wait(at(kRaw, 0)))) break;
                for (int f = 0; f < int(C::STAGE / kTile); ++f) fix(to + f * kTile, m);
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) arrive(bar + kFull + st);
            }
        }
        // every copy has landed before the CTA leaves (bounded waits; a phase that
        // is already over returns at once)
        for (int y = c > C::NST ? c - C::NST : 0; y < c; ++y)
            mbar_wait_bounded(bar + kFull + y % C::NST, (y / C::NST) & 1, kWaitFinal);
    } else if (warp == 29) {
        // ---------------------------------------------------------------- KV and scores
        // The scores go one step ahead, so that P is ready when its turn comes; they and KV
        // run while O is read, which S Q waits for.
        constexpr uint32_t idX = tc::idesc(DT, 64, 64), idS = tc::idesc(DT, 128, DK) | kMnB;
        const uint64_t dk_mn = sdesc(sb + C::sK, kTile), dk = sdesc(sb + C::sK, 16), dq = sdesc(sb + C::sQ, 16);
        Ring<C::NST> ring, ahead;
        #pragma unroll 1
        for (int e = STATE ? 0 : -1; ok && e < n; ++e) {
            c = e;
            if (c >= 0) {
                const int NB = C::nkv(fine);
                const Phase ready = at(kParts + (c & 1), c >> 1), read = at(kKvRead + ((c - NB) & 1), (c - NB) >> 1);
                ok = STATE ? wait(at(kFull + ring.st, ring.parity), ready, read) : wait(ready, read);
                if (!ok) break;
                tc::fence_after();
                if (elect()) {
                    const uint64_t d = adv(dk_mn, ring.st * C::STAGE);
                    #pragma unroll 1
                    for (int q = 0; q < parts; ++q)
                        #pragma unroll
                        for (int t = 0; t < 64; t += 16)  // (w V)^T K
                            tc::mma(tm + C::kv(fine, c), tm + C::w(fine, c) + q * 32 + t / 2, adv(d, t * 128), idS, q + t > 0);
                    tc::commit(bar + kKvDone + (c & 1));
                    tc::commit(bar + kFree + ring.st);
                }
                __syncwarp();
                ring.next();
            }
            if (STATE || c + 1 >= n) continue;
            const int before = c + 1 - C::nx(fine);  // whose O has to be read: the buffer's last
            ok = wait(at(kFull + ahead.st, ahead.parity), at(kORead + (before & 1), before >> 1));
            if (!ok) break;
            tc::fence_after();
            if (elect()) {
                const uint32_t off = ahead.st * C::STAGE;
                #pragma unroll 1
                for (int f = 0; f < C::KT; ++f)
                    #pragma unroll
                    for (int t = 0; t < 128; t += 32)  // Q K^T
                        tc::mma_ss(tm + C::x(fine, c + 1), adv(dq, off + f * kTile + t), adv(dk, off + f * kTile + t), idX, f + t > 0);
                tc::commit(bar + kScDone + (~c & 1));
            }
            __syncwarp();
            ahead.next();
        }
        // everything issued is done before tensor memory is given back
        if (elect()) tc::commit(bar + kFinal);
        mbar_wait_bounded(bar + kFinal, 0, kWaitFinal);
    } else if (warp == 31 && !STATE) {
        // ---------------------------------------------------------------- S Q and P V
        constexpr uint32_t idO = tc::idesc(DT, 128, 64);
        const uint64_t dq = sdesc(sb + C::sQ, 16), dv = sdesc(sb + C::sV, kTile), dp = sdesc(sb + C::oP, 16);
        Ring<C::NST> ring;
        #pragma unroll 1
        for (; c < n; ++c, ring.next()) {
            const uint32_t off = ring.st * C::STAGE;
            ok = wait(at(kFull + ring.st, ring.parity), at(kSop, c), at(kORead + (~c & 1), (c - 1) >> 1));
            if (!ok) break;
            tc::fence_after();
            if (elect()) {
                #pragma unroll 1
                for (int f = 0; f < C::KT; ++f)  // S^T Q^T
                    #pragma unroll
                    for (int t = 0; t < 4; ++t)
                        tc::mma(tm + C::cOi, tm + C::cS + f * 32 + t * 8, adv(dq, off + f * kTile + t * 32), idO, f + t > 0);
                tc::commit(bar + kSqDone);
            }
            if (!(ok = wait(at(kPReady + (c & 1), c >> 1)))) break;
            tc::fence_after();
            if (elect()) {
                #pragma unroll
                for (int t = 0; t < 4; ++t)  // V^T P^T
                    tc::mma_ss(tm + C::x(fine, c), adv(dv, off + t * 2048), adv(dp, (c & 1) * kTile + t * 32), idO | kMnA, t > 0);
                tc::commit(bar + kPvDone + (c & 1));
                tc::commit(bar + kFree + ring.st);
            }
            __syncwarp();
        }
        if (elect()) tc::commit(bar + kFinal + 1);
        mbar_wait_bounded(bar + kFinal + 1, 0, kWaitFinal);
    } else if (warp == 30 && !STATE && !o32) {
        // ---------------------------------------------------------------- O -> global
        #pragma unroll 1
        for (; c < n; ++c) {
            if (!(ok = wait(at(kOReady, c)))) break;
            const int m = tokens(c);
            const int64_t t0 = p.tok0 + int64_t(chunk(c)) * kChunk;
            if (!(packed && m < kChunk)) {  // tokens past the tensor's end are not written
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
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    __syncwarp();
    if (warp == 29) tc::dealloc(tm, 512);
    if (threadIdx.x == 0 && s_fail) atomicExch(a.err, 7);
}

// The states at the segments' ends, along a sequence in the walk's order: X_p =
// l^(tokens of a segment) X_(p-1) + N_p, float32, in place of N_p; the walk's last one
// is the sequence's final state, if that is wanted.  Sequences of up to a.join segments
// are left to the walks' CTAs.  Four elements a thread, four segments in flight.
__global__ void __launch_bounds__(256) linattn_join_kernel(const __grid_constant__ Passes a, int size) {
    const Pass& x = a.p[blockIdx.z];
    const Walk& w = x.w;
    const int chunks = size / 1024, i = blockIdx.x / chunks, h = blockIdx.y;
    const Seq s = locate(w.offsets, w.T, i);
    const int64_t all = (s.len + kChunk - 1) / kChunk, nseg = (all + a.seg_chunks - 1) / a.seg_chunks;
    if (nseg <= a.join || nseg < (w.state_out ? 2 : 3)) return;
    const int64_t g0 = s.slot / a.seg_chunks, step = (w.reverse ? -1 : 1) * int64_t(w.H) * size;
    float4* at = reinterpret_cast<float4*>(x.seg_state + ((g0 + (w.reverse ? nseg - 2 : 0)) * w.H + h) * size +
                                           (blockIdx.x % chunks) * 1024 + threadIdx.x * 4);
    const float g = head_decay(w.decay, h);
    const Decay l = decay_over(g, float(a.seg_chunks * kChunk));
    auto after = [](const Decay& d, const float4& x, const float4& y) {
        return make_float4(decayed(d, x.x, y.x), decayed(d, x.y, y.y), decayed(d, x.z, y.z), decayed(d, x.w, y.w));
    };
    float4 S = *at;
    for (int64_t p = 1; p + 1 < nseg; p += 4) {
        float4 N[4];
        #pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j + 1 < nseg) N[j] = *(at + (p + j) * step / 4);
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (p + j + 1 >= nseg) break;
            S = after(l, S, N[j]);
            *(at + (p + j) * step / 4) = S;
        }
    }
    if (!w.state_out) return;
    float4* out = reinterpret_cast<float4*>(w.state_out + (int64_t(i) * w.H + h) * size + (blockIdx.x % chunks) * 1024 + threadIdx.x * 4);
    // backwards in time the last segment is a sequence's first one, which is whole
    const int64_t left = w.reverse ? a.seg_chunks * kChunk : s.len - (nseg - 1) * a.seg_chunks * kChunk;
    *out = after(decay_over(g, float(left)), S, *out);
}

template <int DT, int DK, int DV>
cudaError_t launch(const Passes& a, int n, bool states, cudaStream_t st) {
    static PerDevice c0, c1;
    constexpr size_t walk = Cfg<DK, DV, false>::BYTES, ends = Cfg<DK, DV, true>::BYTES;
    static_assert(kBars * 8 <= 320, "barriers");
    cudaError_t e = opt_in(linattn_walk_kernel<DT, DK, DV, false>, walk, c0);
    if (e == cudaSuccess) e = opt_in(linattn_walk_kernel<DT, DK, DV, true>, ends, c1);
    if (e != cudaSuccess) return e;
    const int64_t nseq = a.p[0].w.nseq;
    dim3 grid(unsigned(a.segments), unsigned(a.p[0].w.H), unsigned(n));
    if (states) {
        // the parts of cut sequences alone: whole segments, and at most one that is shorter
        // for each of these
        if (a.few_cut && 2 * (a.segments - nseq) < a.segments) grid.x = unsigned(2 * (a.segments - nseq));
        linattn_walk_kernel<DT, DK, DV, true><<<grid, kThreads, ends, st>>>(a);
        if (a.most <= a.join) return cudaGetLastError();
        constexpr int size = DK * DV;
        linattn_join_kernel<<<dim3(unsigned(nseq) * (size / 1024), grid.y, grid.z), 256, 0, st>>>(a, size);
    } else {
        linattn_walk_kernel<DT, DK, DV, false><<<grid, kThreads, walk, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

// Segments.  A sequence's chunks follow one another, so few long sequences leave SMs
// idle.  Cut into m segments a walk costs another over K and V for the segments' end
// states, and a join.  The rule counts waves of CTAs over the SMs.  Its unit is 0.07 us:
// a chunk's step of a walk 20 (22 uncut, where w V may take three parts; 26 in fp16), of
// the segments' states 9 (13); a CTA's start and end 106 and 100; the second launch 90,
// with the join's 160.  Fitted to 1024 to 16384 tokens with 6 to 150 rows, uncut and in
// 2 to 48 segments: 0.9 % above the fastest of them on average, 15 % at most in calls of
// more than 40 us.
//
// bf16 128 x 128, 16384 tokens, forward: 6 rows uncut 457 us, in 24 segments 62; 24 rows
// 459, in 6 134; 60 rows 461, in 5 298.  Training step's gradients: 16 rows 463, in 3
// 224, in 8 244.  2048 tokens: 36 rows forward 71, in 3 51; gradients 83, in 2 100.
// Packed rows are taken at their mean length, as the host does not know their offsets.
// Where that leaves them uncut and the estimate is above 140 us, sequences of more than
// twice the mean that would take longer by themselves than the estimate (its half for the
// gradients' three walks) are cut into pieces of that length.  It costs a launch of CTAs
// with nothing to do where no sequence is as long.  12 heads of 128 x 128, bf16, forward
// (gradients), one prompt of 60000 tokens among others of 178:
//   of 8 535 us (570), uncut 1644 (1650); 16 355 (570), with pieces of half the length 310;
//   32 311 (610), half 350, uncut 1645 (1644); 33 357 (710), uncut 1671 (1764); 64 452
//   (890), uncut 1706 (1885); 200 758 (1630), uncut 1859 (2403)
// equal prompts: 8 of 8192 tokens 265 (508), uncut 258 (502); 33 of 2048 224 (489), uncut
//   212 (478); 1000 of 178 1180 (3550), uncut 1148 (3545); 32 of uneven lengths up to 6000
//   tokens 211 (463), half 272
// Under 140 us such a launch weighs more (24 prompts in 16411 tokens take 61 us), and one
// long prompt among short ones is one chain.
//
// The walks' CTAs join up to three segments themselves (8 rows of 4096, 6 heads of 128,
// three segments: 99 us with the inputs from memory, against 107 with the join's launch;
// four segments: 128 against 129; six: 121 against 105, as the reads of the states before
// follow one another), and the few long sequences of an uneven queue (up to nine segments),
// where a launch would mostly find nothing to do.  A packed row that is cut by its mean
// length may hold a sequence of many more segments: the launch joins those (one prompt of
// 56226 tokens, 126 segments, among 49 of 190, one head of 128, bf16: 86 us, 196 with its
// segments joined one after another; 50 of 1311: 65 us, 60 without the launch).
void plan_segments(Segments* s, int64_t B, int64_t T, int64_t nseq, int64_t heads, int walks, int dt, int sms) {
    const int64_t slots = chunk_slots(B, T, nseq), rows = nseq * heads;
    s->chunks = slots + 1;
    s->count = nseq;
    s->states = 0;
    s->join = 0;
    s->most = 1;
    s->few_cut = false;
    s->by_length = nseq <= kSorted;
    if (rows == 0) return;
    // chunks of a sequence of mean length, at least one: there may be fewer tokens than sequences
    const int64_t mean = (B * T / nseq + kChunk - 1) / kChunk, n = mean > 0 ? mean : 1;
    const int64_t most = (T + kChunk - 1) / kChunk;  // chunks that one sequence may have
    const bool f16 = dt == FFTCONV_F16;
    auto waves = [&](int64_t ctas) { return (ctas + sms - 1) / sms; };
    int64_t best = 1, cost = waves(rows * walks) * (n * (f16 ? 26 : 22) + 106);
    for (int64_t m = 2; m * 2 <= n && m * rows <= 2 * sms; ++m) {
        const int64_t len = (n + m - 1) / m;
        const int64_t c = waves(m * rows * walks) * (len * (f16 ? 26 : 20) + 106) +
                          waves(m * rows * (walks > 1 ? 2 : 1)) * (len * (f16 ? 13 : 9) + 100) + (m <= 3 ? 90 : 160);
        if (c < cost) {
            cost = c;
            best = m;
        }
    }
    // an uneven queue's pieces: as long by themselves as the estimate, for several walks half
    const int64_t piece = std::max(2 * n, cost / ((f16 ? 26 : 20) * (walks > 1 ? 2 : 1)));
    s->few_cut = best == 1 && B == 1 && nseq > 1 && cost >= 2000 && most > piece;
    if (best == 1 && !s->few_cut) return;
    s->chunks = s->few_cut ? piece : (n + best - 1) / best;
    s->states = slots / s->chunks;
    s->count = s->states + nseq;
    s->join = s->few_cut ? 9 : best <= 3 ? 3 : 0;
    s->most = (most + s->chunks - 1) / s->chunks;
    s->by_length = s->few_cut && nseq <= kSorted;
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
