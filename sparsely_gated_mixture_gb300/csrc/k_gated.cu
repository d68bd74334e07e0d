// What surrounds the products of the gated experts' backward: dL/dgate of each
// choice from the products' partial sums, and the gradient of x.
#include "gated.cuh"

namespace moe {
namespace {

template <typename T>
__device__ __forceinline__ float ld(const T *p, size_t i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}

__global__ void k_gated_begin(DeviceStatus *st) {
  pdl_wait();
  if (threadIdx.x < sizeof(DeviceStatus) / 4) reinterpret_cast<uint32_t *>(st)[threadIdx.x] = 0;
}

// The row of assignment a = t*k + j, or -1 (dropped, or not an expert).
__device__ __forceinline__ long long gated_row(long long a, int E, const int32_t *idx,
                                               const int32_t *pos, const uint8_t *keep,
                                               const int32_t *base) {
  if (!keep[a]) return -1;
  const int e = idx[a];
  return e >= 0 && e < E ? (long long)base[e] + pos[a] : -1;
}

// One warp per assignment; lanes in order, so the sum's order is fixed.
template <typename T>
__global__ void __launch_bounds__(256)
k_gated_dgate(long long A, int E, int k, int d, int n_blocks, const int32_t *__restrict__ idx,
              const int32_t *__restrict__ pos, const uint8_t *__restrict__ keep,
              const int32_t *__restrict__ base, const float *__restrict__ dgpart,
              const T *__restrict__ dy, const T *__restrict__ b2, float *__restrict__ dgate) {
  pdl_wait();
  pdl_trigger();
  const long long a = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (a >= A) return;
  const long long r = gated_row(a, E, idx, pos, keep, base);
  float s = 0.f;
  if (r >= 0) {
    for (int b = lane; b < n_blocks; b += 32) s += dgpart[r * n_blocks + b];
    if (b2) {
      const size_t t = (size_t)(a / k) * d, e = (size_t)idx[a] * d;
      for (int i = lane; i < d; i += 32) s = fmaf(ld(dy, t + i), ld(b2, e + i), s);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dgate[a] = s;
}

// One warp per token; choices in order.
template <typename T>
__global__ void __launch_bounds__(256)
k_gated_dx(int T_, int E, int k, int d, const int32_t *__restrict__ idx,
           const int32_t *__restrict__ pos, const uint8_t *__restrict__ keep,
           const int32_t *__restrict__ base, const float *__restrict__ dX,
           const T *__restrict__ dy, T *__restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  const long long t = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= T_) return;
  const long long mine = lane < k ? gated_row(t * k + lane, E, idx, pos, keep, base) : -1;
  for (int i0 = 0; i0 < d; i0 += 32) {
    const int i = i0 + lane;
    float s = i < d ? ld(dy, (size_t)t * d + i) : 0.f;
    for (int j = 0; j < k; ++j) {
      const long long r = __shfl_sync(0xffffffffu, mine, j);
      if (r >= 0 && i < d) s += dX[(size_t)r * d + i];
    }
    if (i < d) {
      if constexpr (sizeof(T) == 2) dx[(size_t)t * d + i] = __float2bfloat16_rn(s);
      else dx[(size_t)t * d + i] = s;
    }
  }
}

}  // namespace

cudaError_t launch_gated_begin(DeviceStatus *st, cudaStream_t s) {
  return launch_pdl(k_gated_begin, 1, 32, 0, s, st);
}

cudaError_t launch_gated_dgate(const moe_config &c, int n_blocks, const int32_t *idx,
                               const int32_t *pos, const uint8_t *keep, const int32_t *base,
                               const float *dgpart, const void *dy, const void *b2, float *dgate,
                               cudaStream_t s) {
  const long long A = (long long)c.T * c.k;
  const unsigned grid = (unsigned)((A + 7) / 8);
  if (c.act_dtype == MOE_BF16)
    return launch_pdl(k_gated_dgate<__nv_bfloat16>, grid, 256, 0, s, A, c.E, c.k, c.d, n_blocks,
                      idx, pos, keep, base, dgpart, (const __nv_bfloat16 *)dy,
                      (const __nv_bfloat16 *)b2, dgate);
  return launch_pdl(k_gated_dgate<float>, grid, 256, 0, s, A, c.E, c.k, c.d, n_blocks, idx, pos,
                    keep, base, dgpart, (const float *)dy, (const float *)b2, dgate);
}

cudaError_t launch_gated_dx(const moe_config &c, const int32_t *idx, const int32_t *pos,
                            const uint8_t *keep, const int32_t *base, const float *dX,
                            const void *dy, void *dx, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)c.T + 7) / 8);
  if (c.act_dtype == MOE_BF16)
    return launch_pdl(k_gated_dx<__nv_bfloat16>, grid, 256, 0, s, c.T, c.E, c.k, c.d, idx, pos,
                      keep, base, dX, (const __nv_bfloat16 *)dy, (__nv_bfloat16 *)dx);
  return launch_pdl(k_gated_dx<float>, grid, 256, 0, s, c.T, c.E, c.k, c.d, idx, pos, keep, base,
                    dX, (const float *)dy, (float *)dx);
}

}  // namespace moe
