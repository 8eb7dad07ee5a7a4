// ws_host.h -- host-side helpers of the logits calls that need nothing of
// CUDA.
#pragma once

#include <cstddef>
#include <cstdint>

namespace ws {

// Whether rows of `cols` elements of `size` bytes, sa elements apart from a
// on, share an element with rows sb elements apart from b on (both aligned to
// their elements; strides of cols at least).
inline bool rows_overlap(const void* a, int64_t sa, const void* b, int64_t sb, int64_t rows, int64_t cols, size_t size) {
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / (int64_t)size;
    if (d >= (rows - 1) * sa + cols || -d >= (rows - 1) * sb + cols) return false;   // one behind the other
    auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0 ? 1 : 0); };
    auto near = [cols](int64_t x) { return x > -cols && x < cols; };
    if (sa == sb) {
        // row r of a and row r - n of b begin n sa - d elements apart
        for (int64_t n = floor_div(d, sa), i = 0; i < 2; ++n, ++i)
            if (n > -rows && n < rows && near(n * sa - d)) return true;
        return false;
    }
    for (int64_t r = 0; r < rows; ++r)
        for (int64_t x = r * sa - d, s = floor_div(x, sb), i = 0; i < 2; ++s, ++i)
            if (s >= 0 && s < rows && near(x - s * sb)) return true;
    return false;
}

// Answers of queries that are asked once: at most kA x kB whole numbers, 0 for
// a query that fails (a cluster size that a device need not support, say)
// whatever became of the others.  Where what the queries need cannot be
// prepared, nothing is kept, and the next call asks again.
template <int kA, int kB>
struct AskedOnce {
    int of[kA][kB] = {};
    bool asked = false;

    // prepare() -> bool; query(a, b, &answer) -> bool.
    template <class Prepare, class Query>
    void ask(Prepare prepare, Query query) {
        if (asked || !prepare()) return;
        for (int a = 0; a < kA; ++a)
            for (int b = 0; b < kB; ++b) {
                int n = 0;
                of[a][b] = query(a, b, &n) ? n : 0;
            }
        asked = true;
    }
};

}  // namespace ws
