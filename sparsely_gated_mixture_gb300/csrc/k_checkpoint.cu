// Hidden activations in 8 bits between the forward and the backward.
//
// A row's columns form blocks of 32; a block stores its values as e4m3 with
// one scale 2^e, e the smallest exponent (at least -124) whose largest e4m3
// value, 448 * 2^e, reaches the block's largest. So a value keeps 4
// significant bits unless it is below 2^-6 * 2^e, that is some 2^-14 of the
// block's largest. Two properties that the backward relies on:
//   - a value over zero is never stored as zero (it is lifted to the smallest
//     one, 2^-9 * 2^e): the ReLU pattern [h > 0], and with it dpre, db1, dW1
//     and the experts' share of dx, is exactly that of the unrounded rows;
//   - every stored value is exact in bf16 (4 significant bits, exponent at
//     least -133), so loading rounds nothing.
// Values at or below zero (the rows are ReLU outputs) are stored as zero. A
// block with a NaN or an infinity over zero gets the scale byte 255 and loads
// as NaN. Scale bytes: e + 127.
//
// Both directions are HBM streams: one warp moves 1024 columns of a row,
// every 16-byte (fp32: 32-byte) load issued before the first is used; 4 lanes
// of 8 columns make a block. Widths that are not a multiple of 8 go one
// column per lane. Saving and loading the 16384 rows of 14336 of the large-expert
// layer take 215 to 223 us for 1.42 GB, 6.4 to 6.6 TB/s. Saving was bound by its
// instructions first (some 10 a value, 227 us for both): the ReLU and the
// largest value now take one packed instruction for two bf16 values, the lift
// over zero two a value, and a warp's row no 64-bit division.
#include "checkpoint.cuh"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kLow = -124;      // smallest scale exponent
constexpr int kWarps = 8;
constexpr int kPasses = 4;      // passes of 256 columns per warp
constexpr int kSeg = 256 * kPasses;

// Scale exponent of a block from its largest value (finite, >= 0): amax =
// 1.m * 2^(E - 127) and 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kLow);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// v / 2^e (v >= 0) for e4m3, at least 2^-9 where v is over zero. Saturates in
// the conversion; where 448 * 2^e passes the largest float (e >= 120) it stops
// at 240, whose value is finite.
constexpr float kLeast = 0.001953125f;
template <typename T>
__device__ __forceinline__ float scaled(float v, float inv) {
  // Any bf16 over zero (2^-133 on) times 2^127 is over 2^-9.
  if constexpr (sizeof(T) == 2) return fmaxf(v * inv, fminf(v * 0x1p127f, kLeast));
  return fmaxf(v * inv, v > 0.f ? kLeast : 0.f);
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
template <typename T>
struct Oct;
template <>
struct Oct<__nv_bfloat16> {
  uint4 v;
  // Values below zero become zero; the largest of all, NaN if one is.
  __device__ __forceinline__ float relu_top() {
    __nv_bfloat162 *w = reinterpret_cast<__nv_bfloat162 *>(&v);
    const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __hmax2_nan(w[j], zero);
    const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(w[0], w[1]), __hmax2_nan(w[2], w[3]));
    return max_nan(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      w[j] = *reinterpret_cast<uint32_t *>(&b);
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Oct<float> {
  float4 a, b;
  __device__ __forceinline__ float relu_top() {
    float f[8], top = 0.f;
    get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = max_nan(f[j], 0.f);
      top = max_nan(top, f[j]);
    }
    set(f);
    return top;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
k_ckpt_save(int cols, const FixedDiv by_seg, const int32_t *__restrict__ rows,
            const T *__restrict__ h, uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
            long long max_rows, DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5), r = by_seg(u);
  const long long row = r;
  const int seg = (int)(u - r * by_seg.d);
  if (row >= max_rows || row >= *rows) return;
  const int nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const T *src = h + row * cols;
  uint8_t *dst = q + row * cols;
  Oct<T> in[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int c = seg * kSeg + i * 256 + lane * 8;
    if (c < cols) in[i] = *reinterpret_cast<const Oct<T> *>(src + c);
  }
  uint32_t mine = 0;  // the scale byte of block `lane` of this segment
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int c = seg * kSeg + i * 256 + lane * 8;
    float f[8], top = 0.f;
    if (c < cols) top = in[i].relu_top();
    const bool bad = !(top < INFINITY);
    if (bad) top = INFINITY;
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool fine = top < INFINITY;
    const int e = fine ? scale_exp(top) : 0;
    const float inv = pow2(-e);
    const uint32_t byte = fine ? (uint32_t)(e + 127) : 255u;
    const uint32_t got = __shfl_sync(0xffffffffu, byte, 4 * (lane & 7));
    if ((lane >> 3) == i) mine = got;
    if (c < cols) {
      in[i].get(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = scaled<T>(f[j], inv);
      if (e >= 120)
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = fminf(f[j], 240.f);
      *reinterpret_cast<uint2 *>(dst + c) =
          make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16,
                     e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
    }
    if (bad) record_error(st, MOE_ERR_NONFINITE, row * cols + c);
  }
  const int b = seg * (kSeg / kCkptBlock) + lane;
  if (b < nb) scale[row * nb + b] = (uint8_t)mine;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
k_ckpt_load(int cols, const FixedDiv by_seg, const int32_t *__restrict__ rows,
            const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale, T *__restrict__ h,
            long long max_rows) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned u = blockIdx.x * kWarps + (threadIdx.x >> 5), r = by_seg(u);
  const long long row = r;
  const int seg = (int)(u - r * by_seg.d);
  if (row >= max_rows || row >= *rows) return;
  const int nb = (cols + kCkptBlock - 1) / kCkptBlock;
  const uint8_t *src = q + row * cols;
  T *dst = h + row * cols;
  uint2 in[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int c = seg * kSeg + i * 256 + lane * 8;
    if (c < cols) in[i] = *reinterpret_cast<const uint2 *>(src + c);
  }
  const int b = seg * (kSeg / kCkptBlock) + lane;
  const float mine = b < nb ? ckpt_scale(scale[row * nb + b]) : 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int c = seg * kSeg + i * 256 + lane * 8;
    const float s = __shfl_sync(0xffffffffu, mine, i * 8 + (lane >> 2));
    if (c >= cols) continue;
    const uint32_t w[4] = {in[i].x & 0xffffu, in[i].x >> 16, in[i].y & 0xffffu, in[i].y >> 16};
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 v = ckpt_e4m3x2(w[j]);
      f[2 * j] = v.x * s;
      f[2 * j + 1] = v.y * s;
    }
    Oct<T> o;
    o.set(f);
    *reinterpret_cast<Oct<T> *>(dst + c) = o;
  }
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Any width: one column of a block per lane, kAny consecutive blocks (over the
// rows' ends) a warp, all their loads in flight. A block's largest value is one
// integer reduction: bits of floats that are not below zero order as they do,
// NaN last. Saving and loading 8192 rows of 10001 bf16 columns take 260 us, bound
// by instructions (75 us is their bytes at the copy rate; one block a warp took
// 645).
constexpr int kAny = 8;

// Block u of the rows' blocks: the index of this lane's column, and whether it
// is one.
__device__ __forceinline__ bool any_at(const FixedDiv &by_block, unsigned u, unsigned total,
                                       int cols, int lane, long long &at) {
  const unsigned row = by_block(u), c = (u - row * by_block.d) * kCkptBlock + lane;
  at = (long long)row * cols + c;
  return u < total && c < (unsigned)cols;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
k_ckpt_save_any(int cols, const FixedDiv by_block, const int32_t *__restrict__ rows,
                const T *__restrict__ h, uint8_t *__restrict__ q, uint8_t *__restrict__ scale,
                long long max_rows, DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned u0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kAny;
  const unsigned total = (unsigned)min(max_rows, (long long)max(*rows, 0)) * by_block.d;
  if (u0 >= total) return;
  float v[kAny];
  long long at[kAny];
  bool live[kAny];
#pragma unroll
  for (int i = 0; i < kAny; ++i) {
    live[i] = any_at(by_block, u0 + i, total, cols, lane, at[i]);
    v[i] = live[i] ? to_f(h[at[i]]) : 0.f;
  }
  uint32_t mine = 0;  // the scale byte of block `lane`
#pragma unroll
  for (int i = 0; i < kAny; ++i) {
    const float f = max_nan(v[i], 0.f);
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(f));
    const bool fine = top < 0x7f800000u;
    const int e = fine ? scale_exp(__uint_as_float(top)) : 0;
    if (lane == i) mine = fine ? (uint32_t)(e + 127) : 255u;
    if (live[i]) {
      q[at[i]] = (uint8_t)e4m3x2(fminf(scaled<T>(f, pow2(-e)), e >= 120 ? 240.f : 448.f), 0.f);
      if (!(f < INFINITY)) record_error(st, MOE_ERR_NONFINITE, at[i]);
    }
  }
  if (lane < kAny && u0 + lane < total) scale[u0 + lane] = (uint8_t)mine;
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32)
k_ckpt_load_any(int cols, const FixedDiv by_block, const int32_t *__restrict__ rows,
                const uint8_t *__restrict__ q, const uint8_t *__restrict__ scale,
                T *__restrict__ h, long long max_rows) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const unsigned u0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kAny;
  const unsigned total = (unsigned)min(max_rows, (long long)max(*rows, 0)) * by_block.d;
  if (u0 >= total) return;
  const float mine = lane < kAny && u0 + lane < total ? ckpt_scale(scale[u0 + lane]) : 0.f;
  uint8_t v[kAny];
  long long at[kAny];
  bool live[kAny];
#pragma unroll
  for (int i = 0; i < kAny; ++i) {
    live[i] = any_at(by_block, u0 + i, total, cols, lane, at[i]);
    v[i] = live[i] ? q[at[i]] : (uint8_t)0;
  }
#pragma unroll
  for (int i = 0; i < kAny; ++i) {
    const float s = __shfl_sync(0xffffffffu, mine, i);
    if (live[i]) put(h + at[i], ckpt_e4m3x2(v[i]).x * s);
  }
}

__global__ void k_ckpt_begin(DeviceStatus *st) {
  pdl_wait();
  if (threadIdx.x == 0) *st = DeviceStatus{};
  pdl_trigger();
}

__global__ void k_ckpt_choices(int n, int E, const int32_t *__restrict__ idx,
                               int32_t *__restrict__ out, DeviceStatus *st,
                               const DeviceStatus *other) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i == 0 && other && other->code) record_error(st, other->code, other->detail);
  if (i >= n) return;
  const int e = idx[i];
  const bool ok = e >= 0 && e < E;
  if (!ok) record_error(st, MOE_ERR_BOUNDS, i);
  out[i] = ok ? e : 0;
}

// How a width is cut: segments of kSeg columns, one a warp, or (not a multiple
// of 8) blocks of 32, kAny a warp. Their number is below 2^32 (checked by the
// caller).
struct Cut {
  bool whole;
  FixedDiv by;
  dim3 grid;
  Cut(long long max_rows, int cols) : whole(cols % 8 == 0) {
    const int unit = whole ? kSeg : kCkptBlock, per_row = (cols + unit - 1) / unit;
    const long long per_block = (long long)kWarps * (whole ? 1 : kAny);
    by = FixedDiv((unsigned)per_row);
    grid = dim3((unsigned)((max_rows * per_row + per_block - 1) / per_block));
  }
};

template <typename T>
cudaError_t run_save(long long max_rows, int cols, const int32_t *rows, const void *h, uint8_t *q,
                     uint8_t *scale, DeviceStatus *st, cudaStream_t s) {
  const T *src = static_cast<const T *>(h);
  const Cut c(max_rows, cols);
  return launch_pdl(c.whole ? k_ckpt_save<T> : k_ckpt_save_any<T>, c.grid, kWarps * 32, 0, s, cols,
                    c.by, rows, src, q, scale, max_rows, st);
}

template <typename T>
cudaError_t run_load(long long max_rows, int cols, const int32_t *rows, const uint8_t *q,
                     const uint8_t *scale, void *h, cudaStream_t s) {
  T *dst = static_cast<T *>(h);
  const Cut c(max_rows, cols);
  return launch_pdl(c.whole ? k_ckpt_load<T> : k_ckpt_load_any<T>, c.grid, kWarps * 32, 0, s, cols,
                    c.by, rows, q, scale, dst, max_rows);
}

}  // namespace

cudaError_t launch_checkpoint_save(bool bf16, long long max_rows, int cols, const int32_t *rows,
                                   const void *h, uint8_t *q, uint8_t *scale, DeviceStatus *st,
                                   cudaStream_t s) {
  return bf16 ? run_save<__nv_bfloat16>(max_rows, cols, rows, h, q, scale, st, s)
              : run_save<float>(max_rows, cols, rows, h, q, scale, st, s);
}

cudaError_t launch_checkpoint_load(bool bf16, long long max_rows, int cols, const int32_t *rows,
                                   const uint8_t *q, const uint8_t *scale, void *h,
                                   cudaStream_t s) {
  return bf16 ? run_load<__nv_bfloat16>(max_rows, cols, rows, q, scale, h, s)
              : run_load<float>(max_rows, cols, rows, q, scale, h, s);
}

cudaError_t launch_checkpoint_begin(DeviceStatus *st, cudaStream_t s) {
  return launch_pdl(k_ckpt_begin, dim3(1), 32, 0, s, st);
}

cudaError_t launch_checkpoint_choices(int n, int E, const int32_t *idx, int32_t *out,
                                      DeviceStatus *st, const DeviceStatus *other,
                                      cudaStream_t s) {
  return launch_pdl(k_ckpt_choices, dim3((n + 255) / 256), 256, 0, s, n, E, idx, out, st, other);
}

}  // namespace moe
