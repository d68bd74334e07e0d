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

// Work of one call on a side stream beside the caller's stream s. However the call
// ends, with an error half-way too, what s gets later follows what the side
// stream got: else freeing or reusing the call's buffers in stream order would race
// with it, and a captured side stream would stay unjoined. Declared after the lock,
// so that the join is enqueued under it.
class SideFork {
 public:
  SideFork() = default;
  SideFork(const SideFork &) = delete;
  SideFork &operator=(const SideFork &) = delete;
  ~SideFork() {
    if (open_) join();
  }
  // side null: everything runs on s.
  void use(SideStream *side, cudaStream_t s) {
    side_ = side;
    s_ = s;
  }
  cudaStream_t stream() const { return side_ ? side_->s : s_; }
  // What stream() gets from here on follows what s got so far.
  int fork() {
    if (!side_) return MOE_OK;
    MOE_CUDA(cudaEventRecord(side_->fork, s_));
    MOE_CUDA(cudaStreamWaitEvent(side_->s, side_->fork, 0));
    open_ = true;
    return MOE_OK;
  }
  // The end of what stream() got so far, for await().
  int mark() {
    if (side_) MOE_CUDA(cudaEventRecord(side_->join, side_->s));
    return MOE_OK;
  }
  // What s gets from here on follows the last mark().
  int await() {
    if (side_) MOE_CUDA(cudaStreamWaitEvent(s_, side_->join, 0));
    return MOE_OK;
  }
  int join() {
    const int r = mark();
    if (r != MOE_OK) return r;
    open_ = false;
    return await();
  }

 private:
  SideStream *side_ = nullptr;
  cudaStream_t s_ = nullptr;
  bool open_ = false;
};

}  // namespace moe
