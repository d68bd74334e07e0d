// Gated experts: activations, the 8-bit format and the launchers shared by the
// gated kernels. Internal to libmoe.so.
//   U(x) = (act(x W1 + b1) * (x W3 + b3)) W2 + b2
#pragma once

#include "gate_math.cuh"
#include "moe_internal.cuh"

#include <cuda_fp8.h>

#include <type_traits>

namespace moe {

// ----------------------------------------------------------------------------- activations
// act(v) and, for the backward, act'(v) with act(v). PRECISE is for fp32
// layers; bf16 layers take the fast exponential (2 ulp and 1.2 ulp for each
// unit of |v|, some 1e-6 where the result is not negligible) and division, and
// the routers' normal distribution function (1e-6 relative; erff's two branches
// take half as long again).
template <bool PRECISE>
__device__ __forceinline__ float gated_sigmoid(float v) {
  if constexpr (PRECISE) return 1.f / (1.f + expf(-v));
  return __fdividef(1.f, 1.f + fminf(__expf(-v), 1e30f));  // the fast division wants < 2^126
}
template <bool PRECISE>
__device__ __forceinline__ float gated_phi(float v) {  // the normal distribution function
  if constexpr (PRECISE) return normcdff(v);
  // Past 30 it is 0 or 1; the fit would square a larger one to infinity.
  return normal_cdf(fminf(fmaxf(v, -30.f), 30.f));
}
template <bool PRECISE, int ACT>
__device__ __forceinline__ float gated_act(float v) {
  if constexpr (ACT == MOE_ACT_SILU) return v * gated_sigmoid<PRECISE>(v);
  if constexpr (ACT == MOE_ACT_GELU) return v * gated_phi<PRECISE>(v);
  return max_nan(v, 0.f);
}
template <bool PRECISE, int ACT>
__device__ __forceinline__ void gated_act_slope(float v, float &a, float &s) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float t = gated_sigmoid<PRECISE>(v);
    a = v * t;
    s = t * fmaf(v, 1.f - t, 1.f);
  } else if constexpr (ACT == MOE_ACT_GELU) {
    const float t = gated_phi<PRECISE>(v);
    const float e = PRECISE ? expf(-0.5f * v * v) : __expf(-0.5f * v * v);
    a = v * t;
    s = fmaf(v * 0.3989422804014327f, e, t);
  } else {
    a = max_nan(v, 0.f);
    s = v > 0.f ? 1.f : 0.f;
  }
}

// Calls f with the activation as a compile-time constant.
template <typename F>
inline cudaError_t gated_dispatch(int activation, F &&f) {
  switch (activation) {
    case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>{});
    case MOE_ACT_GELU: return f(std::integral_constant<int, MOE_ACT_GELU>{});
    default: return f(std::integral_constant<int, MOE_ACT_RELU>{});
  }
}

// ----------------------------------------------------------------------------- 8-bit blocks
// e4m3 values v / 2^e, e the smallest exponent (at least -124) with 448 * 2^e
// >= the block's largest magnitude; scale byte e + 127, 255 for a block that
// holds an Inf or a NaN (its product is NaN then).
constexpr int kFp8Block = 128;
constexpr int kFp8Low = -124;
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b >= 0x7f800000u) return 255u;
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(max(e, kFp8Low) + 127);
}
// What values are multiplied by: 2^-e (a NaN for byte 255: its values are not used).
__device__ __forceinline__ float fp8_inverse(uint32_t byte) {
  return __uint_as_float((254u - (byte == 255u ? 0u : byte)) << 23);
}
__device__ __forceinline__ uint32_t fp8_pack2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
inline long long fp8_blocks(long long n) { return (n + kFp8Block - 1) / kFp8Block; }

// ----------------------------------------------------------------------------- launchers
// The routed rows of a call: packed per expert from offset[e], row r standing
// for assignment row_token[r] = t*k + j with gate row_gate[r]; mtiles [E+1] is
// the prefix of the experts' 128-row tiles.
struct GatedRows {
  const int32_t *offset, *mtiles, *row_token;
  const float *row_gate;
};

// k_gated_simt.cu: the products on the CUDA cores (fp32 layers, and bf16
// widths that the tensor-core kernels do not take).
struct GatedSimt {
  moe_config c;
  int activation, max_rows;
  GatedRows rows;
  const void *x, *W1, *b1, *W3, *b3, *W2, *b2;
  void *h;            // forward: [rows, d_ff] act_dtype
  void *pre1, *pre3;  // forward: written if not null; backward: read
  float *z;           // forward: [rows, d] gate * U
  const void *dy;     // backward
  float *hf, *dU, *dP1, *dP3, *dX, *dgpart;  // backward: fp32 rows
  void *dW1, *dW3, *dW2;                     // act_dtype
  DeviceStatus *st;
};
cudaError_t launch_gated_simt_forward(const GatedSimt &p, cudaStream_t s);
cudaError_t launch_gated_simt_backward(const GatedSimt &p, cudaStream_t s);
int gated_simt_dg_blocks(const moe_config &c, int max_rows);  // columns of dgpart [rows, ..]

// k_ffn_tc.cu: the gated first layer on the tensor cores (ffn_tc_supported
// layers; the second is launch_ffn_layer2). Buffers of max_rows packed rows;
// pre1 and pre3 may be null.
cudaError_t launch_gated_tc_layer1(const moe_config &c, int C, int activation, long long max_rows,
                                   const void *xbuf, const int32_t *offset, const void *W1,
                                   const void *b1, const void *W3, const void *b3, void *hbuf,
                                   void *pre1, void *pre3, DeviceStatus *st, cudaStream_t s);

// k_fp8.cu: to 8 bits.
// Weights [E, K, N] (bf16 or fp32) to q [E, N, Kp] (Kp = K rounded up to 128,
// zeros past K) and scale [E, ceil(N/128), Kp/128].
cudaError_t launch_fp8_weights(bool bf16, int E, int K, int N, const void *W, uint8_t *q,
                               uint8_t *scale, DeviceStatus *st, cudaStream_t s);
// Packed rows r < *count to q [max_rows, Kp] and scale [Kp/512 rounded
// up][max_rows][4], the bytes of four blocks of a row together; row r
// is that of token row_token[r] / k of src.
cudaError_t launch_fp8_rows(int max_rows, int K, int k, const int32_t *count,
                            const int32_t *row_token, const void *src, uint8_t *q,
                            uint8_t *scale, cudaStream_t s);

// k_fp8_tc.cu: one of the 8-bit layer's products on the tensor cores, any
// widths. Layer 1: a8 = x rows, W and W3 -> h8 [max_rows, d_ff rounded up to
// 128], sh; layer 2: a8 = h8, W -> z [max_rows, d] in fp32, or bf16 (d a multiple
// of 8). sa, sh: the rows' scales, as launch_fp8_rows writes them.
struct Fp8Layer {
  moe_config c;
  int layer, activation, max_rows;
  const int32_t *offset;
  const float *row_gate;
  const uint8_t *a8, *sa, *W, *sb, *W3, *sb3;
  const void *bias, *bias3;
  uint8_t *h8, *sh;
  void *z;
  bool z_bf16;
  DeviceStatus *st;
};
bool fp8_tc_supported();
cudaError_t launch_fp8_tc(const Fp8Layer &q, cudaStream_t s);

// k_gated.cu: what surrounds the products of the backward.
// dgate [T,k] = sum of a kept choice's dgpart row plus <dy, b2>; 0 for the others.
// dgpart's row of assignment (t, j) is base[e] + pos[t,j].
cudaError_t launch_gated_dgate(const moe_config &c, int n_blocks, const int32_t *idx,
                               const int32_t *pos, const uint8_t *keep, const int32_t *base,
                               const float *dgpart, const void *dy, const void *b2, float *dgate,
                               cudaStream_t s);
// dx = dy + the kept choices' rows base[e] + pos of dX.
cudaError_t launch_gated_dx(const moe_config &c, const int32_t *idx, const int32_t *pos,
                            const uint8_t *keep, const int32_t *base, const float *dX,
                            const void *dy, void *dx, cudaStream_t s);
// The status word cleared, then the choices' slots, row maps, offsets and tile
// prefix (launch_slots' outputs), in one launch. poff [E+1], or null: the
// backward's padded offsets. Up to kRouteMost assignments.
constexpr int kRouteMost = 32768;
struct GatedRouteArgs {
  int A, E, C;
  const int32_t *idx;
  const float *gate;
  int32_t *pos;
  uint8_t *keep;
  int32_t *offset, *mtiles, *poff, *row_token;
  float *row_gate;
  DeviceStatus *st;
};
cudaError_t launch_gated_route(const GatedRouteArgs &a, cudaStream_t s);
// Clears the status word: a kernel, for its place in the chain of dependent launches.
cudaError_t launch_gated_begin(DeviceStatus *st, cudaStream_t s);

}  // namespace moe
