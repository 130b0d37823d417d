// Host-side checks of the strided token-major views of the token mixers.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/fftconv.h"

namespace fftconv {

inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// A view's strides with those of size-1 dimensions made harmless.
struct View {
    char* p;
    int64_t b, t, h;  // elements
};

// Check a view of [B][T][H][D] (D = 0: a [B][T][H] tensor of gates) and
// normalise it.  Sizes are positive here.
inline fftconv_status_t take_view(const fftconv_view_t& v, int64_t B, int64_t T, int64_t H, int64_t D, View* out) {
    if (!v.ptr) return FFTCONV_ERR_INVALID;
    const int64_t row = D ? D : 1;
    *out = {static_cast<char*>(v.ptr), B > 1 ? v.batch : row, T > 1 ? v.token : row, H > 1 ? v.head : row};
    if (out->b <= 0 || out->t <= 0 || out->h <= 0) return FFTCONV_ERR_INVALID;
    if (D ? (off16(v.ptr) || ((out->b | out->t | out->h) & 7)) : (reinterpret_cast<uintptr_t>(v.ptr) & 1))
        return FFTCONV_ERR_ALIGN;
    return FFTCONV_OK;
}

// An address range, for the overlap checks.
struct Span {
    uintptr_t lo, hi;
};

inline Span span_of(const View& v, int64_t B, int64_t T, int64_t H, int64_t D) {
    const int64_t last = (B - 1) * v.b + (T - 1) * v.t + (H - 1) * v.h + (D ? D : 1);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(v.p);
    return {lo, lo + uintptr_t(last) * 2};
}

inline Span span_of(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return p ? Span{lo, lo + bytes} : Span{0, 0};
}

inline bool meets(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether any of `outs` meets any of `ins`.
template <int NO, int NI>
bool any_meet(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (meets(o, i)) return true;
    return false;
}

}  // namespace fftconv
