// The gated experts for a few rows on the CUDA cores: fp32 layers, and bf16
// widths that the tensor-core kernels do not take. Bound by reading the weights
// of the experts in use once, so a thread owns a column (layer 1: of W1 and W3),
// keeps the sums of up to eight rows in registers and walks a slice of K with
// sixteen weights in flight; the rows' values come from shared memory. Slices of K
// make enough blocks to ask for the weights at once; their sums leave in fp32 and
// are added in order of K: layer 1's by the pass that makes the hidden rows,
// layer 2's by the combine. Experts of more than eight rows are walked again, from
// L2. (8 tokens, top-2 of 8 experts,
// fp32, d 512, d_ff 1024: 37 us; with k_gated_simt.cu's tiles 147.)
#include "gated.cuh"

namespace moe {
namespace {

constexpr int kCols = 128, kRows = 8, kMaxSlice = 512, kFlight = 8;

template <typename T>
__device__ __forceinline__ float ld(const T *p, size_t i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}
template <typename T>
__device__ __forceinline__ void put(T *p, size_t i, float v) {
  if constexpr (sizeof(T) == 2) p[i] = __float2bfloat16_rn(v);
  else p[i] = v;
}

// Blocks (column tile, slice of K, expert). LAYER 1: A = x through row_token, sums
// of W1 and W3 to part [slice][2][rows][N]; LAYER 2: A = h, part [slice][rows][N].
template <typename T, int LAYER>
__global__ void __launch_bounds__(kCols)
k_few_simt(const GatedFewSimt p, int K, int N, int slice) {
  pdl_wait();
  pdl_trigger();
  __shared__ float a[kRows][kMaxSlice];
  const int e = blockIdx.z, tid = threadIdx.x, n = blockIdx.x * kCols + tid;
  const int r0 = p.rows.offset[e], rows = p.rows.offset[e + 1] - r0;
  if (rows == 0) return;
  const int k0 = blockIdx.y * slice, k1 = min(K, k0 + slice);
  const size_t at = (size_t)e * K * N + n;
  const T *W1 = static_cast<const T *>(LAYER == 1 ? p.W1 : p.W2) + at;
  const T *W3 = static_cast<const T *>(p.W3) + at;
  constexpr int M = LAYER == 1 ? 2 : 1;
  for (int m0 = 0; m0 < rows; m0 += kRows) {
    __syncthreads();
    for (int i = 0; i < kRows && m0 + i < rows; ++i) {
      const int r = r0 + m0 + i;
      const T *src = LAYER == 1
                         ? static_cast<const T *>(p.x) + (size_t)(p.rows.row_token[r] / p.c.k) * K
                         : static_cast<const T *>(p.h) + (size_t)r * K;
      for (int k = k0 + tid; k < k1; k += kCols) a[i][k - k0] = ld(src, k);
    }
    __syncthreads();
    if (n >= N) continue;
    float acc[M][kRows] = {};
    for (int kb = k0; kb < k1; kb += kFlight) {
      float w[M][kFlight];
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        const bool in = kb + j < k1;
        w[0][j] = in ? ld(W1, (size_t)(kb + j) * N) : 0.f;
        if (LAYER == 1) w[M - 1][j] = in ? ld(W3, (size_t)(kb + j) * N) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < kFlight; ++j) {
        if (kb + j >= k1) break;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (m0 + i >= rows) break;
          const float v = a[i][kb + j - k0];
#pragma unroll
          for (int q = 0; q < M; ++q) acc[q][i] = fmaf(v, w[q][j], acc[q][i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (m0 + i >= rows) break;
#pragma unroll
      for (int q = 0; q < M; ++q)
        p.part[(((size_t)blockIdx.y * M + q) * p.max_rows + r0 + m0 + i) * N + n] = acc[q][i];
    }
  }
}

// h = act(p1) * p3 from layer 1's sums; a thread a column of a row (rows along y).
template <typename T, int ACT>
__global__ void __launch_bounds__(256) k_few_simt_hidden(const GatedFewSimt p, int slices) {
  pdl_wait();
  pdl_trigger();
  const int F = p.c.d_ff, n = blockIdx.x * 256 + threadIdx.x, r = blockIdx.y;
  if (n >= F || r >= p.rows.offset[p.c.E]) return;
  const int e = p.idx[p.rows.row_token[r]];
  float p1 = p.b1 ? ld(static_cast<const T *>(p.b1), (size_t)e * F + n) : 0.f;
  float p3 = p.b3 ? ld(static_cast<const T *>(p.b3), (size_t)e * F + n) : 0.f;
  const size_t step = (size_t)p.max_rows * F, at = (size_t)r * F + n;
#pragma unroll 4
  for (int s = 0; s < slices; ++s) {
    p1 += p.part[(2 * s) * step + at];
    p3 += p.part[(2 * s + 1) * step + at];
  }
  if (p.pre1) {
    put(static_cast<T *>(p.pre1), at, p1);
    put(static_cast<T *>(p.pre3), at, p3);
  }
  float v, slope;
  gated_act_slope<ACT>(p1, v, slope);
  put(static_cast<T *>(p.h), at, v * p3);
}

// y = x + the kept choices' gate * (layer 2's sums + b2), in choice order; a
// thread a column of a token (tokens along y).
template <typename T>
__global__ void __launch_bounds__(256) k_few_simt_combine(const GatedFewSimt p, int slices) {
  pdl_wait();
  pdl_trigger();
  const int d = p.c.d, k = p.c.k, n = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (n >= d) return;
  float y = ld(static_cast<const T *>(p.x), (size_t)t * d + n);
  const size_t step = (size_t)p.max_rows * d;
  for (int j = 0; j < k; ++j) {
    const int a = t * k + j;
    if (!p.keep[a]) continue;
    const int e = p.idx[a];
    const float *src = p.part2 + (size_t)(p.rows.offset[e] + p.pos[a]) * d + n;
    float z = p.b2 ? ld(static_cast<const T *>(p.b2), (size_t)e * d + n) : 0.f;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) z += src[s * step];
    y = fmaf(p.gate[a], z, y);
  }
  if (!isfinite(y)) record_error(p.st, MOE_ERR_NONFINITE, (long long)t);
  put(static_cast<T *>(p.y), (size_t)t * d + n, y);
}

// Columns of K a slice: enough blocks for two waves of four an SM over the experts
// that can be in use, at least 64 columns, at most what shared memory holds.
int slice_of(const moe_config &c, int K, int N) {
  const long long A = (long long)c.T * c.k, used = A < c.E ? A : c.E;
  const long long tiles = used * ((N + kCols - 1) / kCols);
  long long slices = (8ll * kPlanSms + tiles - 1) / tiles;
  long long s = (K + slices - 1) / slices;
  s = s < 64 ? 64 : s > kMaxSlice ? kMaxSlice : s;
  return (int)((s + kFlight - 1) / kFlight * kFlight);
}
int slices_of(const moe_config &c, int K, int N) {
  const int s = slice_of(c, K, N);
  return (K + s - 1) / s;
}

template <typename T>
cudaError_t few_simt(GatedFewSimt p, cudaStream_t s) {
  const moe_config &c = p.c;
  const int s1 = slices_of(c, c.d, c.d_ff), s2 = slices_of(c, c.d_ff, c.d);
  const dim3 g1((c.d_ff + kCols - 1) / kCols, s1, c.E), g2((c.d + kCols - 1) / kCols, s2, c.E);
  cudaError_t err = launch_pdl_c(kPdlGemm, k_few_simt<T, 1>, g1, kCols, 0, s, p, c.d, c.d_ff,
                                 slice_of(c, c.d, c.d_ff));
  if (err != cudaSuccess) return err;
  err = gated_dispatch(p.activation, [&](auto act) {
    return launch_pdl(k_few_simt_hidden<T, decltype(act)::value>,
                      dim3((c.d_ff + 255) / 256, p.max_rows), 256, 0, s, p, s1);
  });
  if (err != cudaSuccess) return err;
  GatedFewSimt q = p;
  q.part = p.part2;
  err = launch_pdl_c(kPdlGemm, k_few_simt<T, 2>, g2, kCols, 0, s, q, c.d_ff, c.d,
                     slice_of(c, c.d_ff, c.d));
  if (err != cudaSuccess) return err;
  return launch_pdl_c(kPdlCombine, k_few_simt_combine<T>, dim3((c.d + 255) / 256, c.T), 256, 0, s, p,
                      s2);
}

}  // namespace

size_t gated_few_simt_part(const moe_config &c, int max_rows, int layer) {
  return layer == 1 ? 2ull * slices_of(c, c.d, c.d_ff) * max_rows * c.d_ff * 4
                    : 1ull * slices_of(c, c.d_ff, c.d) * max_rows * c.d * 4;
}

cudaError_t launch_gated_few_simt(const GatedFewSimt &p, cudaStream_t s) {
  return p.c.act_dtype == MOE_BF16 ? few_simt<__nv_bfloat16>(p, s) : few_simt<float>(p, s);
}

}  // namespace moe
