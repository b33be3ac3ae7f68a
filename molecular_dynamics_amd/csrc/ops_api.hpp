// Host-side checks and launches shared by the block operators.
#pragma once
#include <algorithm>

#include "ops.hpp"
#include "prof.hpp"

namespace mdmp {
namespace ops {

// rows are read and written 16 bytes at a time
inline bool rows_ok(const void* p, int64_t ld, int width, int esize) {
  return ((uintptr_t)p & 15) == 0 && ld >= width && (ld * esize) % 16 == 0;
}

// Outputs of a memory-bound pass over more bytes than this go past the caches: they would be
// evicted before a reader comes, and push out rows still to be read (131,072 x 128 float32 norms:
// backward 102 -> 86 us, forward 61 -> 52; 328,378 x 384 bf16 product 102 -> 89).  Below, the
// 256 MB last-level cache keeps them for the next operator.
inline bool streams(int64_t bytes) { return bytes > (int64_t)192 << 20; }

inline int check_width(const char* who, int32_t channels, int32_t feat_dtype) {
  if (feat_dtype != 0 && feat_dtype != 1) return arg_error(std::string(who) + ": feat_dtype must be 0 or 1");
  if (channels != 16 && channels != 32 && channels != 64 && channels != 128)
    return arg_error(std::string(who) + ": channels must be 16, 32, 64 or 128");
  if (channels == 16 && feat_dtype == 1)
    return arg_error(std::string(who) + ": 16 channels need float32 features (bf16 products contract 32 at a time)");
  return MP_OK;
}

// rows that a launch can cover (threads of a grid dimension are counted in 32 bits)
constexpr int32_t kMaxRows = 1 << 26;

#define MP_ROWS(who, name, p, ld, width, dt)                                                                     \
  do {                                                                                                           \
    if (!::mdmp::ops::rows_ok(p, ld, width, (dt) == 1 ? 2 : 4))                                                  \
      return arg_error(who ": rows of " name                                                                     \
                       " must be 16-byte aligned, with a row stride of at least their width and a multiple of 16 bytes"); \
  } while (0)

// out[j] = sum over s < S of part[s * ldp + off + j], j < N, added in a fixed order; up to three
// such segments of one set of partials in one launch.  S = 0 writes zeros.
struct Segment {
  int64_t off, N;
  void* out;  // null: no such segment
  bool bf16;
};
int reduce_rows(const float* part, int64_t S, int64_t ldp, const Segment* seg, int nseg, hipStream_t st);

}  // namespace ops
}  // namespace mdmp
