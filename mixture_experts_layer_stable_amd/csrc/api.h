// Helpers shared by the C-ABI entry points (api.hip, api_block.hip): argument checks, buffer
// sizes and launch bracketing.
#pragma once
#include "common.h"

namespace mok {

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) & ~(kAlign - 1); }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline int elem_size(int act) { return act == MOK_F32 ? 4 : 2; }

// Compute units of the current device, cached per device id.
mok_status device_cus(int* out);

// Buffer sizes passed by the caller against what the descriptor needs.
inline mok_status need(size_t have, size_t want) { return have >= want ? MOK_OK : MOK_ERR_WORKSPACE; }

// ---- measurement trace (see mok_trace_bind): the calling thread's caller-owned trace ----
extern thread_local mok_trace* t_trace;
bool trace_on(const char* name);

}  // namespace mok

#define MOK_REQUIRE(p)                   \
  do {                                   \
    if ((p) == nullptr) return MOK_ERR_NULL;  \
    if (!aligned16(p)) return MOK_ERR_ALIGN; \
  } while (0)

// Launch `call` (a hipError_t expression) bracketed by trace events when traced.
#define MOK_LAUNCH(name, stream, call)                                                          \
  do {                                                                                          \
    const bool tr_ = trace_on(name);                                                            \
    if (tr_ && hipEventRecord((hipEvent_t)t_trace->events[2 * t_trace->count], stream) != hipSuccess) \
      return MOK_ERR_HIP;                                                                       \
    if ((call) != hipSuccess) return MOK_ERR_HIP;                                               \
    if (tr_) {                                                                                  \
      if (hipEventRecord((hipEvent_t)t_trace->events[2 * t_trace->count + 1], stream) != hipSuccess) \
        return MOK_ERR_HIP;                                                                     \
      t_trace->names[t_trace->count] = name;                                                    \
      ++t_trace->count;                                                                         \
    }                                                                                           \
  } while (0)
