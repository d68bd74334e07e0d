// Argument checks shared by the files that define the C ABI. Internal to
// libmoe.so.
#pragma once

#include "moe_internal.cuh"

#include <math.h>

#include <mutex>

namespace moe {

static inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

static inline int host_capacity(const moe_config &c) {
  double raw = floor((double)c.k * (double)c.T * (double)c.capacity_factor / (double)c.E);
  long v = (long)raw;
  if (v > c.T) v = c.T;
  if (v < c.min_capacity) v = c.min_capacity;
  return (int)v;
}

static inline int check_cfg(const moe_config *c) {
  if (!c) return MOE_ERR_ARG;
  if (c->T < 1 || c->d < 1 || c->E < 1 || c->d_ff < 1 || c->k < 1 || c->k > c->E) return MOE_ERR_ARG;
  if (!(c->capacity_factor > 0.f) || !isfinite(c->capacity_factor)) return MOE_ERR_ARG;
  if (c->min_capacity < 1) return MOE_ERR_ARG;
  if (c->gate_mode != MOE_GATE_TOPK_SOFTMAX && c->gate_mode != MOE_GATE_SWITCH) return MOE_ERR_ARG;
  if (c->gate_mode == MOE_GATE_SWITCH && c->k != 1) return MOE_ERR_ARG;
  if (c->act_dtype != MOE_F32 && c->act_dtype != MOE_BF16) return MOE_ERR_ARG;
  if ((long long)c->T * c->k > 0x7fffffffLL || (long long)c->T * c->E > 0x7fffffffLL)
    return MOE_ERR_UNSUPPORTED;
  if (c->E > 1024 || c->k > 16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

static inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Required pointers must be non-null; every given pointer 16-byte aligned.
#define MOE_REQ(p)                                      \
  do {                                                  \
    if (!(p) || !aligned((p), 16)) return MOE_ERR_ARG;  \
  } while (0)
#define MOE_OPT(p)                                      \
  do {                                                  \
    if ((p) && !aligned((p), 16)) return MOE_ERR_ARG;   \
  } while (0)
#define MOE_CUDA(call)                                  \
  do {                                                  \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA;     \
  } while (0)

// The library's side stream for work forked from `caller`, or null (moe_api.cu);
// the lock is held while the call enqueues on it.
struct SideStream {
  cudaStream_t s = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
SideStream *side_stream(std::unique_lock<std::mutex> &lock, cudaStream_t caller);

}  // namespace moe
