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

// Whether two boxes of D elements, repeated along the dimensions k .. n - 1
// (strides descending; na and nb repetitions), have an element in common; b's
// first element is off elements after a's.  Only repetitions whose remaining
// dimensions' ranges meet are looked at: one or two of each dimension where these
// lie inside the stride, as in every permuted slice of one buffer.  Strides that
// overlap themselves count as shared.
struct Level {
    int64_t s, na, nb;
};
inline bool boxes_meet(const Level* lv, int k, int n, int64_t off, int64_t D) {
    if (k == n) return off < D && -off < D;
    int64_t ea = D, eb = D;
    for (int i = k + 1; i < n; ++i) {
        ea += (lv[i].na - 1) * lv[i].s;
        eb += (lv[i].nb - 1) * lv[i].s;
    }
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
    const int64_t s = lv[k].s;
    int64_t lo = floor_div(-eb - off, s) + 1, hi = -floor_div(off - ea, s) - 1;
    if (lo < 1 - lv[k].na) lo = 1 - lv[k].na;
    if (hi > lv[k].nb - 1) hi = lv[k].nb - 1;
    if (hi - lo > 3) return true;
    for (int64_t m = lo; m <= hi; ++m)
        if (boxes_meet(lv, k + 1, n, off + m * s, D)) return true;
    return false;
}

// Whether two views [B][T][Ha or Hb][D] have an element in common: exact for
// slices of one buffer (equal strides), else by their address ranges.
inline bool share(const View& a, int64_t Ha, const View& b, int64_t Hb, int64_t B, int64_t T, int64_t D) {
    if (!meets(span_of(a, B, T, Ha, D), span_of(b, B, T, Hb, D))) return false;
    if ((B > 1 && a.b != b.b) || (T > 1 && a.t != b.t) || (Ha > 1 && Hb > 1 && a.h != b.h)) return true;
    Level lv[3];
    int n = 0;
    if (B > 1) lv[n++] = {a.b, B, B};
    if (T > 1) lv[n++] = {a.t, T, T};
    if (Ha > 1 || Hb > 1) lv[n++] = {Ha > 1 ? a.h : b.h, Ha, Hb};
    for (int i = 1; i < n; ++i)
        for (int j = i; j > 0 && lv[j].s > lv[j - 1].s; --j) {
            const Level t = lv[j];
            lv[j] = lv[j - 1];
            lv[j - 1] = t;
        }
    return boxes_meet(lv, 0, n, (b.p - a.p) / 2, D);
}

// Whether any of `outs` meets any of `ins`.
template <int NO, int NI>
bool any_meet(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (const Span& o : outs)
        for (const Span& i : ins)
            if (meets(o, i)) return true;
    return false;
}

}  // namespace fftconv
