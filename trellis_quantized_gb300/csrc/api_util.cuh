// api_util.cuh -- host-side helpers of the C entry points: argument checks
// and the fixed head of every workspace.
#pragma once

#include "exl3_common.cuh"

#define EXL3_TRY(expr)            \
  do {                            \
    int _rc = (expr);             \
    if (_rc != EXL3_OK) return _rc; \
  } while (0)

// The calling thread's message is emptied at the start of every call.
void exl3_clear_error();

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kCtrlBytes = 256;   // device error word and reserved control words
// Arrival counters live at one fixed place of every workspace, right after
// the control block, so calls of any shape find them zero (each call resets
// the counters it used).  Capacity bounds n / 128 of one call.
constexpr size_t kMaxCounters = 8192;
constexpr size_t kCounterOff = kCtrlBytes;
constexpr size_t kDataOff = kCounterOff + kMaxCounters * sizeof(int);

inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int check_ptr(const void *p, const char *name, bool required = true) {
  if (!p) return required ? exl3_fail(EXL3_ERR_ARG, "%s is NULL", name) : EXL3_OK;
  if (!aligned16(p)) return exl3_fail(EXL3_ERR_ARG, "%s is not 16-byte aligned", name);
  return EXL3_OK;
}

inline int check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return EXL3_OK;
  if (!ws) return exl3_fail(EXL3_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
  if ((reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) != 0)
    return exl3_fail(EXL3_ERR_WORKSPACE, "workspace must be %zu-byte aligned", kAlign);
  if (have < need) return exl3_fail(EXL3_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
  return EXL3_OK;
}

template <typename T>
inline T *at(void *base, size_t off) {
  return reinterpret_cast<T *>(static_cast<char *>(base) + off);
}

}  // namespace
