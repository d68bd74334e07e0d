// To 8 bits for the experts' products: e4m3 values with a power-of-two scale
// for each block, which the tensor cores apply themselves (their scales are
// such bytes). A weight's blocks are 128 x 128, a row's are 128 columns.
#include "gated.cuh"

namespace moe {
namespace {

constexpr int B = kFp8Block;

template <typename T>
__device__ __forceinline__ float ld(const T *p, size_t i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}

// One block of 256 threads for a 128 x 128 block of one expert's weight: read
// along N, written along K.
template <typename T>
__global__ void __launch_bounds__(256)
k_fp8_weights(int K, int N, int KB, const T *__restrict__ W, uint8_t *__restrict__ q,
              uint8_t *__restrict__ scale, DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float tile[];  // [128 k][129]
  __shared__ float tops[8];
  const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
  const int tid = threadIdx.x, n = tid & 127;
  const T *src = W + (size_t)e * K * N;
  float top = 0.f;
  for (int i = tid >> 7; i < B; i += 2) {
    const int kk = kb * B + i, nn = nb * B + n;
    const float v = kk < K && nn < N ? ld(src, (size_t)kk * N + nn) : 0.f;
    tile[i * 129 + n] = v;
    top = max_nan(top, fabsf(v));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) tops[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = max_nan(top, tops[w]);
  const uint32_t byte = fp8_scale_byte(top);
  const float inv = fp8_inverse(byte);
  const size_t at = ((size_t)e * gridDim.y + nb) * KB + kb;
  if (tid == 0) {
    scale[at] = (uint8_t)byte;
    if (byte == 255u) record_error(st, MOE_ERR_NONFINITE, (long long)at);
  }
  // Each warp a column, 4 values a lane.
  const int lane = tid & 31;
  for (int c = tid >> 5; c < B && nb * B + c < N; c += 8) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = tile[(lane * 4 + j) * 129 + c] * inv;
    const uint32_t u = fp8_pack2(v[0], v[1]) | fp8_pack2(v[2], v[3]) << 16;
    *reinterpret_cast<uint32_t *>(q + ((size_t)e * N + nb * B + c) * KB * B + kb * B + lane * 4) = u;
  }
}

// A warp for a block of 128 columns of a row, 4 a lane.
__global__ void __launch_bounds__(256)
k_fp8_rows(int max_rows, int K, int KB, int k, const int32_t *__restrict__ count,
           const int32_t *__restrict__ row_token, const __nv_bfloat16 *__restrict__ src,
           uint8_t *__restrict__ q, uint8_t *__restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const long long w = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long r = w / KB;
  const int kb = (int)(w - r * KB);
  if (r >= max_rows || r >= *count) return;
  const size_t row = (size_t)(row_token[r] / k);
  float v[4], top = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = kb * B + lane * 4 + j;
    v[j] = c < K ? __bfloat162float(src[row * K + c]) : 0.f;
    top = max_nan(top, fabsf(v[j]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  const uint32_t byte = fp8_scale_byte(top);
  const float inv = fp8_inverse(byte);
  *reinterpret_cast<uint32_t *>(q + (size_t)r * KB * B + kb * B + lane * 4) =
      fp8_pack2(v[0] * inv, v[1] * inv) | fp8_pack2(v[2] * inv, v[3] * inv) << 16;
  if (lane == 0) scale[((size_t)(kb >> 2) * max_rows + r) * 4 + (kb & 3)] = (uint8_t)byte;
}

}  // namespace

cudaError_t launch_fp8_weights(bool bf16, int E, int K, int N, const void *W, uint8_t *q,
                               uint8_t *scale, DeviceStatus *st, cudaStream_t s) {
  const int KB = (int)fp8_blocks(K);
  const dim3 grid(KB, (unsigned)fp8_blocks(N), E);
  constexpr size_t smem = 128 * 129 * 4;
  if (bf16) {
    const cudaError_t err = allow_smem(k_fp8_weights<__nv_bfloat16>, smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(k_fp8_weights<__nv_bfloat16>, grid, 256, smem, s, K, N, KB,
                      (const __nv_bfloat16 *)W, q, scale, st);
  }
  const cudaError_t err = allow_smem(k_fp8_weights<float>, smem);
  if (err != cudaSuccess) return err;
  return launch_pdl(k_fp8_weights<float>, grid, 256, smem, s, K, N, KB, (const float *)W, q, scale,
                    st);
}

cudaError_t launch_fp8_rows(int max_rows, int K, int k, const int32_t *count,
                            const int32_t *row_token, const void *src, uint8_t *q,
                            uint8_t *scale, cudaStream_t s) {
  const int KB = (int)fp8_blocks(K);
  const long long warps = (long long)max_rows * KB;
  return launch_pdl(k_fp8_rows, (unsigned)((warps + 7) / 8), 256, 0, s, max_rows, K, KB, k, count,
                    row_token, (const __nv_bfloat16 *)src, q, scale);
}

}  // namespace moe
