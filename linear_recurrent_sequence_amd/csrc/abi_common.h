// Host-side argument checks shared by the translation units of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "mlstm.h"

namespace mlstm {
namespace abi {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? MLSTM_OK : MLSTM_ERR_HIP; }

// a caller buffer's byte range; a null pointer or an empty range is skipped
struct Span {
  const void* p;
  size_t n;
};

// MLSTM_ERR_ALIAS if an output overlaps an input or another output (inputs
// may overlap each other: they are only read).  Runs after every other
// argument check, on shapes that the caller has bounded.
inline int check_alias(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    if (!o->p || o->n == 0) continue;
    for (const Span& i : ins)
      if (i.p && i.n && overlaps(o->p, o->n, i.p, i.n)) return MLSTM_ERR_ALIAS;
    for (const Span* o2 = outs.begin(); o2 != o; ++o2)
      if (o2->p && o2->n && overlaps(o->p, o->n, o2->p, o2->n)) return MLSTM_ERR_ALIAS;
  }
  return MLSTM_OK;
}

// MLSTM_ERR_ALIGN if a tensor that is given is not 16-byte aligned
inline int check_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return MLSTM_ERR_ALIGN;
  return MLSTM_OK;
}

inline int check_given(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return MLSTM_ERR_NULL;
  return MLSTM_OK;
}

}  // namespace abi
}  // namespace mlstm
