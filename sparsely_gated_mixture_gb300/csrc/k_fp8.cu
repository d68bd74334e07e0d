// To 8 bits for the experts' products: e4m3 values with a power-of-two scale
// for each block, which the tensor cores apply themselves (their scales are
// such bytes). A weight's blocks are 128 x 128, a row's are 128 columns.
#include "gated.cuh"

namespace moe {
namespace {

constexpr int B = kFp8Block;

// Eight values along N of one row, as floats; VEC: 16-byte loads (the row
// starts on 16 bytes and N is a multiple of 8, or 4 for fp32).
template <typename T, bool VEC>
struct Eight {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *row, int n, int N) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i)
        u[i] = n + i * 4 < N ? *reinterpret_cast<const uint4 *>(row + n + i * 4)
                             : make_uint4(0, 0, 0, 0);
    } else {
      __align__(16) T t[8];
      static_assert(__alignof__(t) % alignof(uint4) == 0, "read as uint4");
#pragma unroll
      for (int j = 0; j < 8; ++j) t[j] = n + j < N ? row[n + j] : T(0.f);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(t)[i];
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
    if constexpr (sizeof(T) == 2)
      return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    return __uint_as_float(w[j]);
  }
};

// One block of 256 threads for a 128 x 128 block of one expert's weight, read
// along N and written along K. A thread holds 8 rows of 8 columns (v = tid % 16
// its eighth of columns, q = tid / 16 of rows), all of its loads in flight at
// once; its bytes change places through shared memory, where the 8-byte piece q
// of column n stands at q ^ v, so that neither side meets bank conflicts.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
k_fp8_weights(int K, int N, int KB, const T *__restrict__ W, uint8_t *__restrict__ out,
              uint8_t *__restrict__ scale, DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  __shared__ __align__(16) uint2 tile[B * 16];
  static_assert(__alignof__(tile) % alignof(uint4) == 0, "read as uint4");
  __shared__ float tops[8];
  const int nb = blockIdx.x, kb = blockIdx.y, e = blockIdx.z;
  const int tid = threadIdx.x, v = tid & 15, q = tid >> 4;
  const int n = nb * B + v * 8, k0 = kb * B + q * 8;
  const T *src = W + (size_t)e * K * N;
  Eight<T, VEC> r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (k0 + i < K) r[i].load(src + (size_t)(k0 + i) * N, n, N);
    else r[i].zero();
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(r[i].get(j)));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max_nan(top, tops[w]);
  const uint32_t byte = fp8_scale_byte(top);
  const float inv = fp8_inverse(byte);
  if (tid == 0) {
    const size_t at = ((size_t)e * gridDim.x + nb) * KB + kb;
    scale[at] = (uint8_t)byte;
    if (byte == 255u) record_error(st, MOE_ERR_NONFINITE, (long long)at);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = fp8_pack2(r[4 * h].get(j) * inv, r[4 * h + 1].get(j) * inv) |
             fp8_pack2(r[4 * h + 2].get(j) * inv, r[4 * h + 3].get(j) * inv) << 16;
    tile[(v * 8 + j) * 16 + (q ^ v)] = make_uint2(w[0], w[1]);
  }
  __syncthreads();
  // Eight lanes write a column's 128 bytes.
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = i * 32 + (tid >> 3), piece = tid & 7, vc = c >> 3;
    uint4 u = reinterpret_cast<const uint4 *>(tile)[c * 8 + (piece ^ (vc >> 1))];
    if (vc & 1) u = make_uint4(u.z, u.w, u.x, u.y);
    if (nb * B + c < N)
      reinterpret_cast<uint4 *>(out + ((size_t)e * N + nb * B + c) * KB * B + kb * B)[piece] = u;
  }
}

// A warp a row: blocks of 128 columns, 4 a lane, eight blocks in flight.
// VEC: 8-byte loads (K a multiple of 4).
template <bool VEC>
__global__ void __launch_bounds__(256)
k_fp8_rows(int max_rows, int K, int KB, int k, const int32_t *__restrict__ count,
           const int32_t *__restrict__ row_token, const __nv_bfloat16 *__restrict__ src,
           uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int r = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), lane = threadIdx.x & 31;
  if (r >= max_rows || r >= *count) return;
  const __nv_bfloat16 *row = src + (size_t)(row_token[r] / k) * K;
  uint32_t *out = reinterpret_cast<uint32_t *>(q + (size_t)r * KB * B) + lane;
  constexpr int N = 8;
  for (int kb0 = 0; kb0 < KB; kb0 += N) {
    uint2 u[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (kb0 + i) * B + lane * 4;
      if constexpr (VEC) {
        u[i] = c < K ? *reinterpret_cast<const uint2 *>(row + c) : make_uint2(0, 0);
      } else {
        const unsigned short *w = reinterpret_cast<const unsigned short *>(row);
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = c + j < K ? w[c + j] : 0u;
        u[i] = make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
      }
    }
    uint32_t bytes[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (kb0 + i >= KB) break;
      const float2 a = unpack2(u[i].x), b = unpack2(u[i].y);
      float top = max_nan(max_nan(fabsf(a.x), fabsf(a.y)), max_nan(fabsf(b.x), fabsf(b.y)));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      bytes[i] = fp8_scale_byte(top);
      const float inv = fp8_inverse(bytes[i]);
      out[(kb0 + i) * 32] = fp8_pack2(a.x * inv, a.y * inv) | fp8_pack2(b.x * inv, b.y * inv) << 16;
    }
    // Four blocks' bytes of a row are a word (those past KB are not read).
    if (lane < 2 && kb0 + 4 * lane < KB) {
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i / 4 == lane && kb0 + i < KB) w |= bytes[i] << 8 * (i & 3);
      reinterpret_cast<uint32_t *>(scale)[(size_t)(kb0 / 4 + lane) * max_rows + r] = w;
    }
  }
}

}  // namespace

cudaError_t launch_fp8_weights(bool bf16, int E, int K, int N, const void *W, uint8_t *q,
                               uint8_t *scale, DeviceStatus *st, cudaStream_t s) {
  const int KB = (int)fp8_blocks(K);
  const dim3 grid((unsigned)fp8_blocks(N), KB, E);  // blocks side by side read on along a row
  const auto run = [&](auto kernel, auto *w) {
    return launch_pdl(kernel, grid, 256, 0, s, K, N, KB, w, q, scale, st);
  };
  if (bf16) {
    const auto *w = static_cast<const __nv_bfloat16 *>(W);
    return N % 8 == 0 ? run(k_fp8_weights<__nv_bfloat16, true>, w)
                      : run(k_fp8_weights<__nv_bfloat16, false>, w);
  }
  const auto *w = static_cast<const float *>(W);
  return N % 4 == 0 ? run(k_fp8_weights<float, true>, w) : run(k_fp8_weights<float, false>, w);
}

cudaError_t launch_fp8_rows(int max_rows, int K, int k, const int32_t *count,
                            const int32_t *row_token, const void *src, uint8_t *q,
                            uint8_t *scale, cudaStream_t s) {
  const int KB = (int)fp8_blocks(K);
  const auto run = [&](auto kernel) {
    return launch_pdl(kernel, (unsigned)((max_rows + 7ll) / 8), 256, 0, s, max_rows, K, KB, k,
                      count, row_token, (const __nv_bfloat16 *)src, q, scale);
  };
  return K % 4 == 0 ? run(k_fp8_rows<true>) : run(k_fp8_rows<false>);
}

}  // namespace moe
