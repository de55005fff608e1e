// Argument checks shared by the C ABI's files.
#pragma once

#include <initializer_list>
#include <string>
#include <string_view>

#include "launch.h"

namespace moe {

// Records the text for moe_last_error and returns `st`.
moe_status fail(moe_status st, const std::string& what);

namespace check {

inline moe_status hip_fail(hipError_t e, const char* where) {
  return fail(MOE_ERR_HIP, std::string(where) + ": " + hipGetErrorString(e));
}

#define CHECK_PTR(p)                                                                  \
  do {                                                                                \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID_ARG, "null pointer: " #p);        \
  } while (0)

// Token-row buffers that the row kernels (gather, combine and their
// backwards) move in 16-byte pieces must start on a 16-byte boundary.
#define CHECK_ROWS(p)                                                                 \
  do {                                                                                \
    if ((reinterpret_cast<uintptr_t>(p) & 15) != 0)                                   \
      return fail(MOE_ERR_INVALID_ARG, #p " does not start on a 16-byte boundary");   \
  } while (0)

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

inline int64_t esize(int32_t dtype) { return dtype == MOE_F32 ? 4 : 2; }

struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
  const char* may_be = nullptr;  // an input: the name of the output that may be this very buffer
};

inline bool ranges_overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uintptr_t>(b.bytes) && y < x + static_cast<uintptr_t>(a.bytes);
}

// No output may overlap an input or another output, apart from the inputs that name one. The name
// decides, not the address: another input at the same address is read by blocks that the output's
// own do not wait for.
inline moe_status check_ranges(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
  for (const Range& o : outs) {
    for (const Range& i : ins)
      if (ranges_overlap(o, i) &&
          !(i.may_be && o.p == i.p && std::string_view(i.may_be) == o.name))
        return fail(MOE_ERR_INVALID_ARG, std::string(o.name) + " overlaps " + i.name);
    for (const Range& other : outs)
      if (&o != &other && ranges_overlap(o, other))
        return fail(MOE_ERR_INVALID_ARG, std::string(o.name) + " overlaps " + other.name);
  }
  return MOE_OK;
}

inline bool known_dtype(int32_t dtype) {
  return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16;
}

}  // namespace check

}  // namespace moe
