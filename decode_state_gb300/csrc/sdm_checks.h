// Checks of arguments that the ABI layers share: alignment, element types, overlapping memory. Host only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "sdm.h"

namespace sdm {
namespace checks {

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

// Rows of `cols` elements, `stride` elements from one to the next; an array is one row of all its elements.
struct Rows {
    const void* p;
    int64_t rows, stride, cols;
    size_t es;

    uintptr_t at() const { return reinterpret_cast<uintptr_t>(p); }
    unsigned __int128 pitch() const { return (unsigned __int128)stride * es; }
    unsigned __int128 row() const { return (unsigned __int128)cols * es; }
    unsigned __int128 end() const { return at() + (rows - 1) * pitch() + row(); }
};

inline Rows array(const void* p, int64_t n, int64_t per, size_t es) { return {p, 1, 0, n * per, es}; }

// Whether any element is in both, also where the rows of one lie beside those of the other in a wider matrix.
// Rows that interleave with a different stride count as overlapping.
inline bool overlaps(const Rows& a, const Rows& b) {
    if (a.p == nullptr || b.p == nullptr || !(a.at() < b.end() && b.at() < a.end())) return false;
    if (a.rows > 1 && b.rows == 1) return overlaps(b, a);
    if (b.rows > 1 && (a.rows == 1 || a.stride == b.stride)) {
        // the place of a's first element behind the start of a row of b (of equal strides, of any row)
        const unsigned __int128 before = a.at() < b.at() ? b.at() - a.at() : 0, pitch = b.pitch();
        const unsigned __int128 place = (a.at() + (before + pitch - 1) / pitch * pitch - b.at()) % pitch;
        // beside that row, and short of the next one; an array behind the last row's columns was apart above
        if (a.rows > 1) return place < b.row() || place + a.row() > pitch;
        if (a.at() < b.at()) return true;  // it reaches the first row
        return place < b.row() || (place + a.row() > pitch && a.at() - place + pitch < b.end());
    }
    return true;
}

inline bool float_type(int dtype) { return dtype == SDM_BF16 || dtype == SDM_F32; }
inline bool index_type(int dtype) { return dtype == SDM_I32 || dtype == SDM_I64; }
inline size_t float_size(int dtype) { return dtype == SDM_BF16 ? 2 : 4; }
inline size_t index_size(int dtype) { return dtype == SDM_I64 ? 8 : 4; }

}  // namespace checks
}  // namespace sdm
