// What the files of entry points share: checks of pointers, which come before any work.
#pragma once

#include "common.cuh"

namespace sparsp {

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define CHECK_PTR(p)                                   \
  do {                                                 \
    if ((p) == nullptr) return SPARSP_ERR_INVALID_ARG; \
    if (!aligned16(p)) return SPARSP_ERR_ALIGN;        \
  } while (0)

#define CHECK_OPT_PTR(p)                                        \
  do {                                                          \
    if ((p) != nullptr && !aligned16(p)) return SPARSP_ERR_ALIGN; \
  } while (0)

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace sparsp
