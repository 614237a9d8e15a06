// Host-side argument checks shared by the C entry points.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mtp_head.h"

namespace mtp {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two ranges of bytes share one (either may be absent).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}

// An array that a call reads or writes (either may be absent), and whether two of them share a byte, or one of
// `outs` shares one with any other array.
struct Span {
  const void* p;
  size_t bytes;
};
template <size_t N, size_t M>
bool outputs_overlap(const Span (&outs)[N], const Span (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
    for (const Span& in : ins)
      if (overlap(outs[i].p, outs[i].bytes, in.p, in.bytes)) return true;
  }
  return false;
}

inline int check_eps(float eps) { return (eps >= 0.0f && !isinf(eps)) ? MTP_OK : MTP_ERR_ARG; }

inline int map_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MTP_OK;
  if (e == cudaErrorNotSupported) return MTP_ERR_NOT_IMPLEMENTED;
  return MTP_ERR_CUDA;
}

// A C entry point's body: no C++ exception (an allocation or a lock that failed) leaves the library.
template <class Fn>
int guarded(Fn&& fn) {
  try {
    return fn();
  } catch (...) {
    return MTP_ERR_CUDA;
  }
}

}  // namespace mtp
