// Checks that the entry points of mc2_layer.h and mc2_layer8.h share; no HIP calls.
#pragma once
#include <initializer_list>
#include <string>

#include "mc2_layer.h"
#include "validate.hpp"

namespace mc2 {

using std::string;

constexpr int64_t kRows = (int64_t)1 << 24, kWidth = (int64_t)1 << 24, kDim = (int64_t)1 << 21,
                  kTokens = (int64_t)1 << 23, kGroups = 4096, kGroupWidth = (int64_t)1 << 29;

inline bool is_half(mc2_dtype d) { return d == MC2_F16 || d == MC2_BF16; }
inline string str(int64_t v) { return std::to_string(static_cast<long long>(v)); }

inline mc2_status shape(const char* who, const string& what) { return fail(MC2_ERR_SHAPE, string(who) + ": " + what); }

// Every pointer 16-byte aligned (NULL is).
inline mc2_status aligned(const char* who, std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15u)
      return fail(MC2_ERR_ALIGN, string(who) + ": tensor not 16-byte aligned");
  return MC2_OK;
}
inline mc2_status required(const char* who, std::initializer_list<const void*> ps, const char* names) {
  for (const void* p : ps)
    if (!p) return fail(MC2_ERR_NULL, string(who) + ": " + names + " are required");
  return MC2_OK;
}
inline mc2_status half(const char* who, mc2_dtype d) {
  return is_half(d) ? MC2_OK : fail(MC2_ERR_DTYPE, string(who) + ": dtype must be F16 or BF16");
}
inline mc2_status workspace_ok(const char* who, const void* ws, size_t bytes, size_t needed) {
  if (needed > 0 && (!ws || bytes < needed))
    return fail(MC2_ERR_WORKSPACE, string(who) + ": workspace needs " + std::to_string(needed) + " bytes");
  return needed > 0 ? aligned(who, {ws}) : MC2_OK;
}

#define MC2_TRY(call)                \
  do {                               \
    mc2_status s_ = (call);          \
    if (s_ != MC2_OK) return s_;     \
  } while (0)

}  // namespace mc2
