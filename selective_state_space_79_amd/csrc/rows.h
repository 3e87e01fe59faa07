// rows.h -- host-side overlap checks of arrays of rows: columns of one wider buffer are
// disjoint although their address ranges interleave.
#pragma once

#include "scan_common.h"

namespace {

// `rows` rows of `width` bytes, `pitch` bytes apart; a null pointer is no array.
struct Area {
    const void* p;
    size_t rows, pitch, width;
};

inline Area rows_of(const void* p, int64_t rows, int64_t stride, int64_t width, int64_t e) {
    return {p, static_cast<size_t>(rows), static_cast<size_t>(stride * e), static_cast<size_t>(width * e)};
}
inline Area flat(const void* p, size_t bytes) { return {p, 1, bytes, bytes}; }

inline bool overlap(const Area& a, const Area& b) {
    if (!a.p || !b.p || !a.width || !b.width) return false;
    if (!overlaps(a.p, (a.rows - 1) * a.pitch + a.width, b.p, (b.rows - 1) * b.pitch + b.width)) return false;
    if (a.pitch != b.pitch || a.rows < 2 || b.rows < 2) return true;
    // one pitch: the columns of b begin `d` bytes behind those of a, modulo the pitch
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t d = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}

// Whether an output overlaps an input or another output.
template <int NI, int NO> bool clash(const Area (&in)[NI], const Area (&out)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Area& x : in)
            if (overlap(out[i], x)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

}  // namespace
