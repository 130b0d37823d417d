// Tiles of token-major tensors on the fifth-generation tensor cores.
//
// A tile is 64 tokens x 64 features of 16-bit values: 64 rows of 128 bytes,
// row r's 16-byte piece c at piece c ^ (r % 8) (the 128-byte swizzle that the
// TMA engine writes), 8 KB, 1024-byte aligned.  The same bytes serve as an
// operand whose contraction runs over the features (K-major: the feature is
// K) and as one whose contraction runs over the tokens (MN-major: the feature
// is M or N), so no tile is ever transposed:
// - K-major, R rows (tokens) per 64-feature block: 8-row groups 1024 bytes
//   apart (SBO), a step of 16 features is 32 bytes.
// - MN-major: 8-token groups 1024 bytes apart (SBO), 64-feature blocks LBO
//   bytes apart, a step of 16 tokens is 2048 bytes.
// The accumulator of an M = 128 contraction has row i in TMEM lane i.
#pragma once
#include "mma.cuh"
#include "tc.cuh"

namespace fftconv {
namespace tile {

constexpr uint32_t kTile = 8192;

__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{.reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;}" : "=r"(p));
    return p != 0;
}

// Shared-memory descriptor with the 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo) {
    return tc::sdesc(addr, lbo, 1024) | (uint64_t(2) << 61);
}

// Descriptor advanced by `bytes`.
__device__ __forceinline__ uint64_t adv(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

constexpr uint32_t kMnA = 1u << 15, kMnB = 1u << 16;  // MN-major A, B in the instruction descriptor

// Bring n bytes (a multiple of 16, from a 16-byte boundary) into L2.
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t n) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(__cvta_generic_to_global(src)), "r"(n) : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bounded wait of a whole warp: gives up after about a second, or sooner when
// another role of the CTA has (*fail set).  The same answer in every lane.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* fail) {
    const uint32_t addr = smem_u32(bar);
    uint64_t t0 = 0;
    bool got = false;
    for (uint32_t it = 0; it < (1u << 24); ++it) {
        uint32_t done;
        asm volatile(
            "{.reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done) {
            got = true;
            break;
        }
        if ((it & 31) == 31) {
            if (*fail) break;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            else if (t - t0 > kWaitNs) break;
        }
    }
    return __all_sync(0xffffffffu, got);
}

// Packed float32 pairs.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n sub.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float2 pair(uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}

// 2^x; 0 below the normal range.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x = hi + lo in two 16-bit values each (about 16 significant bits for bf16),
// for a pair packed low half first.
template <int DT>
__device__ __forceinline__ void split(float2 x, uint32_t* hi, uint32_t* lo) {
    const uint32_t h = Op<DT>::pack(x.x, x.y);
    const cpx f = Op<DT>::unpack(h);
    const float2 r = sub2(x, make_float2(f.r, f.i));
    *hi = h;
    *lo = Op<DT>::pack(r.x, r.y);
}

// Load 16 consecutive columns of this thread's lane (call wait_ld before use).
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Store 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
        "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Store 4 or 8 consecutive columns of this thread's lane.
__device__ __forceinline__ void st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 8) st8(taddr, r);
    else if constexpr (N == 16) tc::st16(taddr, r);
    else st32(taddr, r);
}

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 16) ld16(taddr, r);
    else tc::ld32x32b_x32(taddr, r);
}

// Copies shared -> global (one-dimensional; a box of a tensor map, clipped to
// the tensor), and the wait after which the shared memory may be reused.
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_4d(const void* tmap, uint32_t src, int x, int y, int z, int w) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

constexpr uint32_t kWaitLimitTile = 1u << 22;

}  // namespace tile
}  // namespace fftconv
