// Gated experts: activations, the 8-bit format and the launchers shared by the
// gated kernels. Internal to libmoe.so.
//   U(x) = (act(x W1 + b1) * (x W3 + b3)) W2 + b2
#pragma once

#include "moe_internal.cuh"

#include <cuda_fp8.h>

#include <type_traits>

namespace moe {

// ----------------------------------------------------------------------------- activations
// act(v) and, for the backward, act'(v) with act(v): for the CUDA cores' kernels
// one value, for fp32 layers by CUDA's own functions.
template <int ACT>
__device__ __forceinline__ void gated_act_slope(float v, float &a, float &s) {
  if constexpr (ACT == MOE_ACT_SILU) {
    const float t = 1.f / (1.f + expf(-v));
    a = v * t;
    s = t * fmaf(v, 1.f - t, 1.f);
  } else if constexpr (ACT == MOE_ACT_GELU) {
    const float t = normcdff(v);
    a = v * t;
    s = fmaf(v * 0.3989422804014327f, expf(-0.5f * v * v), t);
  } else {
    a = max_nan(v, 0.f);
    s = v > 0.f ? 1.f : 0.f;
  }
}

// Two floats at once: packed fp32 arithmetic takes one instruction for both.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mov.b64 z, {%6, %7};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// act(v) and, with SLOPE, act'(v) of two values, for the tensor-core kernels'
// epilogues, whose instructions are what bounds short reductions. The
// exponential and the reciprocal are the hardware's (2^-22 and 2^-23 relative;
// an exponential that overflows ends in a zero). The normal distribution
// function is normal_cdf's fit (gate_math.cuh) without the compensation of z^2:
// some 1e-6 relative where it is over 1e-7. No branches, so values of either
// sign cost the same.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float2 gated_act2(float2 v, float2 *slope) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == MOE_ACT_SILU) {
    const float2 z = mul2(v, both(-kLog2e));
    const float2 d = add2(make_float2(exp2_fast(z.x), exp2_fast(z.y)), both(1.f));
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    const float2 a = mul2(v, t);
    if constexpr (SLOPE) *slope = fma2(a, fma2(t, both(-1.f), both(1.f)), t);
    return a;
  } else if constexpr (ACT == MOE_ACT_GELU) {
    const float2 m = make_float2(fabsf(v.x), fabsf(v.y));
    const float2 d = fma2(m, both(0.35355339059327376f), both(1.f));  // 1 + z / 2, z = |v| / sqrt 2
    const float2 t = make_float2(rcp_fast(d.x), rcp_fast(d.y));
    float2 q = both(0.17087277f);
    q = fma2(t, q, both(-0.82215223f));
    q = fma2(t, q, both(1.48851587f));
    q = fma2(t, q, both(-1.13520398f));
    q = fma2(t, q, both(0.27886807f));
    q = fma2(t, q, both(-0.18628806f));
    q = fma2(t, q, both(0.09678418f));
    q = fma2(t, q, both(0.37409196f));
    q = fma2(t, q, both(1.00002368f));
    q = fma2(t, q, both(-1.26551223f - 0.69314718f));  // with the half of erfc / 2
    const float2 zz = mul2(mul2(m, m), both(-0.5f * kLog2e));
    const float2 x = fma2(q, both(kLog2e), zz);
    const float2 tail = mul2(t, make_float2(exp2_fast(x.x), exp2_fast(x.y)));  // Phi(-|v|)
    if constexpr (SLOPE) {
      const float2 g = mul2(v, both(0.3989422804014327f));
      const float2 phi = make_float2(v.x < 0.f ? tail.x : 1.f - tail.x,
                                     v.y < 0.f ? tail.y : 1.f - tail.y);
      *slope = fma2(g, make_float2(exp2_fast(zz.x), exp2_fast(zz.y)), phi);
    }
    // v Phi(v) = max(v, 0) - |v| Phi(-|v|). At +Inf the second term is finite * 0, so
    // that the value is Inf, as the CUDA cores' form has it (Inf * 0 would be a NaN);
    // at -Inf both are a NaN, and a NaN is one by its tail.
    constexpr float kMost = 3.402823466e38f;
    const float2 w = make_float2(-fabsf(fminf(v.x, kMost)), -fabsf(fminf(v.y, kMost)));
    return fma2(w, tail, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
  } else {
    if constexpr (SLOPE) *slope = make_float2(v.x > 0.f ? 1.f : 0.f, v.y > 0.f ? 1.f : 0.f);
    return make_float2(max_nan(v.x, 0.f), max_nan(v.y, 0.f));
  }
}
// A bf16 pair as floats, and two floats as one.
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16x2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t *>(&b);
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
// holds an Inf or a NaN (its product is a NaN by that byte, whatever its values).
constexpr int kFp8Block = 128;
constexpr int kFp8Low = -124;
__device__ __forceinline__ uint32_t fp8_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b >= 0x7f800000u) return 255u;
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (uint32_t)(max(e, kFp8Low) + 127);
}
// What values are multiplied by: 2^-e; for byte 255 2^127, which leaves zeros, NaNs and
// +-448.
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
  float *xf, *hf, *dU, *dP1, *dP3, *dX, *dgpart;  // backward: fp32 rows
  void *dW1, *dW3, *dW2;                     // act_dtype
  float *wpart;  // backward: gated_simt_wpart bytes, the weight gradients by slices of rows
  DeviceStatus *st;
};
cudaError_t launch_gated_simt_forward(const GatedSimt &p, cudaStream_t s);
// Backward: x, g dy, dP1, dP3, h and dgpart first; then dX, and the weight gradients.
cudaError_t launch_gated_simt_front(const GatedSimt &p, cudaStream_t s);
cudaError_t launch_gated_simt_dx(const GatedSimt &p, cudaStream_t s);
cudaError_t launch_gated_simt_weights(const GatedSimt &p, cudaStream_t s);
size_t gated_simt_wpart(const moe_config &c, int max_rows);
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

// k_gated_few.cu: the whole layer for up to kGatedFewRows rows an
// expert and kGatedFewChoices choices, bf16 (widths in steps of 64) or 8 bits.
constexpr int kGatedFewRows = 64, kGatedFewChoices = 512;
// Blocks: one an SM, up to what the workspace (sized without a device) holds.
constexpr int kGatedFewMaxBlocks = 160;
int gated_few_blocks();
struct GatedFew {
  moe_config c;
  bool fp8;
  int activation, C, max_rows, toks;  // toks: rows an expert at most, in steps of 16
  const void *x;
  const int32_t *idx;
  const float *gate;
  const void *W1, *b1, *W3, *b3, *W2, *b2;
  const uint8_t *s1, *s3, *s2;
  int32_t *pos;
  uint8_t *keep;
  int32_t *offset;
  float *row_gate;
  int4 *list;         // [choices]
  int32_t *counters;  // [1 + 2 blocks]
  float *part;        // [blocks][2][toks][256]
  void *xbuf, *h;     // bf16, or e4m3 with scales sx, sh
  uint8_t *sx, *sh;
  void *pre1, *pre3, *z;  // z: bf16 (d a multiple of 8) or fp32
  bool z_bf16;
  void *y;
  DeviceStatus *st;
};
cudaError_t launch_gated_few(const GatedFew &q, cudaStream_t s);

// k_gated_few_simt.cu: both products and the combine for few rows on the CUDA
// cores, after routing. part, part2: gated_few_simt_part bytes for the layers.
struct GatedFewSimt {
  moe_config c;
  int activation, max_rows;
  GatedRows rows;
  const void *x;
  const int32_t *idx, *pos;
  const uint8_t *keep;
  const float *gate;
  const void *W1, *b1, *W3, *b3, *W2, *b2;
  void *h, *pre1, *pre3, *y;
  float *part, *part2;
  DeviceStatus *st;
};
size_t gated_few_simt_part(const moe_config &c, int max_rows, int layer);
cudaError_t launch_gated_few_simt(const GatedFewSimt &p, cudaStream_t s);

// k_gated.cu: what surrounds the products of the backward.
// The backward's rows in bf16 (d a multiple of 64): xbuf = x in packed rows, dY =
// dy in padded blocks, pad rows zero; and zero rows behind the last packed ones of
// xbuf and h, which the weight gradients' K tails read.
cudaError_t launch_gated_gather(const moe_config &c, long long P_max, const GatedRows &rows,
                                const int32_t *poff, const void *x, const void *dy, void *xbuf,
                                void *h, void *dY, cudaStream_t s);
// dgate [T,k] = sum of a kept choice's dgpart row plus <dy, b2>; 0 for the others.
// dgpart's row of assignment (t, j) is base[e] + pos[t,j].
cudaError_t launch_gated_dgate(const moe_config &c, int n_blocks, const int32_t *idx,
                               const int32_t *pos, const uint8_t *keep, const int32_t *base,
                               const float *dgpart, const void *dy, const void *b2, float *dgate,
                               cudaStream_t s);
// The bias gradients (each may be null) db2 = the column sums of dY [rows, d],
// each row times its gate (row_gate null: of dY as it is), db1 and db3 of dP1 and
// dP3 [rows, d_ff], over each expert's rows from base[e] on; rows in act_dtype, or
// fp32 (src_f32), sums in act_dtype.
cudaError_t launch_gated_colsum(const moe_config &c, bool src_f32, const int32_t *offset,
                                const int32_t *base, const void *dY, const float *row_gate,
                                void *db2, const void *dP1, void *db1, const void *dP3, void *db3,
                                cudaStream_t s);
// y = x + the kept choices' rows of z, for widths that launch_combine reads a value
// at a time.
cudaError_t launch_gated_combine(const moe_config &c, const void *x, const float *z,
                                 const int32_t *idx, const int32_t *pos, const uint8_t *keep,
                                 const int32_t *offset, void *y, DeviceStatus *st,
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
