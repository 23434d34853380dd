// Do two strided tensors share a byte?  Host code, for the argument checks of the library and of the binding.
#pragma once
#include <cstdint>

namespace msa {

// rows x heads blocks of `width` bytes, block (r, h) at base + r row + h head (strides in bytes, >= 0)
struct Blocks {
  uintptr_t base;
  int64_t rows, heads, row, head, width;
};

// the same blocks at the same places
inline bool same_blocks(const Blocks& a, const Blocks& b) {
  return a.base == b.base && a.rows == b.rows && a.heads == b.heads && a.width == b.width &&
         (a.rows <= 1 || a.row == b.row) && (a.heads <= 1 || a.head == b.head);
}

// Exact where the tensors have one row pitch (or one of them a single row) or one head pitch, and where all
// strides are multiples of a pitch within which the blocks lie apart: tensors that interleave, such as the
// slices of a fused projection, share no byte.  Others that reach into each other's range count as sharing.
inline bool share_bytes(Blocks a, Blocks b) {
  using Wide = __int128;
  for (Blocks* t : {&a, &b}) {
    if (t->rows <= 0 || t->heads <= 0 || t->width <= 0) return false;
    if (t->rows == 1 || t->row == 0) t->rows = 1, t->row = 0;
    if (t->heads == 1 || t->head == 0) t->heads = 1, t->head = 0;
  }
  auto span = [](const Blocks& t) { return (Wide)(t.rows - 1) * t.row + (Wide)(t.heads - 1) * t.head + t.width; };
  const Wide delta = (Wide)a.base - (Wide)b.base;
  if (delta >= span(b) || -delta >= span(a)) return false;
  uint64_t g = 0;  // the largest pitch that divides every stride
  for (const int64_t stride : {a.row, a.head, b.row, b.head})
    for (uint64_t s = (uint64_t)stride; s;) {
      const uint64_t r = g % s;
      g = s;
      s = r;
    }
  if (g == 0) return true;  // two blocks
  auto apart = [&](Wide pitch, Wide wa, Wide wb) {  // a's wa bytes behind b's wb in every pitch, the two side by side
    const Wide at = (delta % pitch + pitch) % pitch;
    return at >= wb && at + wa <= pitch;
  };
  if (apart(g, a.width, b.width)) return false;
  if (a.rows > 1 && b.rows > 1 && a.row != b.row) {
    if (a.heads > 1 && b.heads > 1 && a.head != b.head) return true;
    for (Blocks* t : {&a, &b}) {  // the heads have one pitch: they take the rows' part
      const Blocks u = *t;
      t->rows = u.heads, t->row = u.head, t->heads = u.rows, t->head = u.row;
    }
  }
  const int64_t R = a.row ? a.row : b.row;
  if (R && apart(R, (Wide)(a.heads - 1) * a.head + a.width, (Wide)(b.heads - 1) * b.head + b.width)) return false;
  // blocks whose heads lie `h` apart: is there a difference of rows at which they meet?
  auto meet = [&](Wide h) {
    const Wide d = delta + h, lo = -(Wide)(b.rows - 1), hi = a.rows - 1;  // d + i R in (-a.width, b.width)
    if (R == 0) return d > -(Wide)a.width && d < b.width;
    const Wide x = -(Wide)a.width - d;
    Wide i = x / R - (x % R < 0) + 1;  // the least i with d + i R > -a.width
    if (i < lo) i = lo;
    return i <= hi && d + i * R < b.width;
  };
  if (a.heads == 1 || b.heads == 1 || a.head == b.head) {
    const int64_t H = a.head ? a.head : b.head;
    for (int64_t j = -(b.heads - 1); j < a.heads; ++j)
      if (meet((Wide)j * H)) return true;
    return false;
  }
  if ((Wide)a.heads * b.heads > 4096) return true;  // (not worth the host's time)
  for (int64_t i = 0; i < a.heads; ++i)
    for (int64_t j = 0; j < b.heads; ++j)
      if (meet((Wide)i * a.head - (Wide)j * b.head)) return true;
  return false;
}

}  // namespace msa
