// abi_checks.h -- argument checks that the operators' C entries share.
#pragma once

#include "../../include/moe.h"
#include "ops.h"

inline bool aligned(const void* p, size_t a = 16) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// A pointer argument, and whether this call needs it.
struct Ptr {
  const void* p;
  bool needed;
};

template <size_t N>
int check_ptrs(const Ptr (&ps)[N]) {
  for (const Ptr& q : ps)
    if (q.needed && !q.p) return abi_fail(MOE_ERR_NULL, "a required pointer is NULL");
  for (const Ptr& q : ps)
    if (q.p && !aligned(q.p)) return abi_fail(MOE_ERR_ALIGN, "tensors must be 16-byte aligned");
  return MOE_OK;
}

inline int launched(hipError_t e) {
  return e == hipSuccess ? abi_ok()
                         : abi_fail(MOE_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
}
