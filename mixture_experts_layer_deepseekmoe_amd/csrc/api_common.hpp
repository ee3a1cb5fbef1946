// Host helpers shared by the C ABI's source files: alignment, formats, launch
// status and the debug build's check flags.
#pragma once

#include "moe.h"

#include <hip/hip_runtime.h>
#ifdef MOE_DEBUG
#include <cstdio>
#endif

#include "around.hpp"

namespace moe::api {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_bytes(int dt) { return dt == MOE_DTYPE_F32 ? 4 : (dt == MOE_DTYPE_BF16 ? 2 : 1); }

inline int fmt_of(int dt) { return dt == MOE_DTYPE_F32 ? FMT_F32 : (dt == MOE_DTYPE_BF16 ? FMT_BF16 : FMT_E4M3); }

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

inline int check_launch(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

// Debug build (-DMOE_DEBUG): after an entry point's launches, wait for the
// stream and read every kernel file's index-check flag; a failed check turns
// the call's status into MOE_ERR_LAUNCH and is reported on stderr.  (The
// release build never synchronises.)
#ifdef MOE_DEBUG
inline int debug_status(int rc, hipStream_t st, const char* what) {
  if (rc != MOE_OK) return rc;
  if (hipStreamSynchronize(st) != hipSuccess) return MOE_ERR_LAUNCH;
  const int flags[] = {debug_take_route(), debug_take_group(), debug_take_ggemm(), debug_take_combine(),
                       debug_take_bwd(),   debug_take_block(), debug_take_loss()};
  for (const int f : flags) {
    if (f != 0) {
      std::fprintf(stderr, "moe debug build: %s: index check %d failed\n", what, f);
      return MOE_ERR_LAUNCH;
    }
  }
  return MOE_OK;
}
#else
inline int debug_status(int rc, hipStream_t, const char*) { return rc; }
#endif

}  // namespace moe::api
