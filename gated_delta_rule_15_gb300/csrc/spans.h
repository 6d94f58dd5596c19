// spans.h -- host checks of where the buffers of a call lie.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace dr {

inline bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
// n_tok rows of `width` elements, `stride` apart
struct Rows {
    const void *p;
    int64_t width, stride;
};
// Whether rows of a and b share a byte.  Rows of one stride may lie between one another (the
// parts of a fused projection's row); of different strides their whole spans count.
inline bool meet(const Rows &a, const Rows &b, int64_t n_tok, int64_t e) {
    if (!a.p || !b.p || n_tok < 1 || a.width < 1 || b.width < 1) return false;
    const char *a0 = (const char *)a.p, *b0 = (const char *)b.p;
    if (a0 + ((n_tok - 1) * a.stride + a.width) * e <= b0 || b0 + ((n_tok - 1) * b.stride + b.width) * e <= a0) return false;
    if (a.stride != b.stride) return true;
    const int64_t row = a.stride * e, off = ((b0 - a0) % row + row) % row;
    return off < a.width * e || off + b.width * e > row;
}
inline bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.width == b.width && a.stride == b.stride; }
// `bytes` bytes in one piece
struct Block {
    const void *p;
    size_t bytes;
};
inline bool meet(const Block &a, const Block &b) {
    const char *a0 = (const char *)a.p, *b0 = (const char *)b.p;
    return a.p && b.p && a.bytes && b.bytes && a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
// Whether a row shares a byte with the block, which may lie between two rows.
inline bool meet(const Rows &a, const Block &b, int64_t n_tok, int64_t e) {
    if (!a.p || !b.p || n_tok < 1 || a.width < 1 || b.bytes < 1) return false;
    const char *a0 = (const char *)a.p, *b0 = (const char *)b.p;
    if (a0 + ((n_tok - 1) * a.stride + a.width) * e <= b0 || b0 + b.bytes <= a0) return false;
    const int64_t row = a.stride * e, off = ((b0 - a0) % row + row) % row;
    return off < a.width * e || off + (int64_t)b.bytes > row;
}

}  // namespace dr
