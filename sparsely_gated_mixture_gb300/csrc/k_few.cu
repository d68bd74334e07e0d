// The few-token layer on the CUDA cores: fp32 layers, and bf16 layers of
// widths that are not multiples of 8. The weights of the experts in use are
// read once, in 16-byte vectors where the widths allow it, and multiplied
// with up to 8 rows at a time from registers.
#include "few.cuh"

#include <atomic>
#include <chrono>

namespace moe {
namespace {

// ----------------------------------------------------------------------------- experts
// out[s][row][n] = sum over slice s of K of A[row][k] W[e][k][n]. A unit is an
// expert, a block of 32 * VEC columns and a slice of K; the block's 8 warps
// share the slice's rows (each loads whole 32 * VEC column segments), and
// their sums are joined in shared memory in warp order.
constexpr int kUnitRows = 256;  // rows of K staged at a time: 32 a warp

struct FewUnits {
  int blocks, slices, per;  // column blocks, slices of K, rows of K per slice
};
__host__ __device__ inline FewUnits few_units(int n_experts, int K, int N, int cols, int grid) {
  FewUnits u;
  u.blocks = (N + cols - 1) / cols;
  const int tiles = n_experts * u.blocks;
  int s = tiles > 0 ? (2 * grid + tiles - 1) / tiles : 1;
  const int most = (K + kUnitRows - 1) / kUnitRows;
  if (s > most) s = most;
  u.per = ((K + s - 1) / s + kUnitRows - 1) / kUnitRows * kUnitRows;
  u.slices = (K + u.per - 1) / u.per;
  return u;
}

template <typename T, int VEC>
struct FewVec;
template <>
struct FewVec<float, 4> {
  float4 v;
  __device__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <>
struct FewVec<float, 1> {
  float v;
  __device__ void get(float (&f)[1]) const { f[0] = v; }
};
template <>
struct FewVec<__nv_bfloat16, 2> {
  uint32_t v;
  __device__ void get(float (&f)[2]) const {
    f[0] = __uint_as_float(v << 16);
    f[1] = __uint_as_float(v & 0xffff0000u);
  }
};
template <>
struct FewVec<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ void get(float (&f)[1]) const { f[0] = __bfloat162float(v); }
};

// smem: xs [kUnitRows][8], red [8 warps][8 rows][VEC][32 lanes].
constexpr int kSimtSmemFloats = kUnitRows * 8 + 8 * 8 * 32 * 4;

template <typename T, int VEC>
__device__ void few_product(const FewRows &R, const T *A, bool by_token, const T *Wall, int K,
                            int N, float *out, float *smem) {
  constexpr int COLS = 32 * VEC;
  using V = FewVec<T, VEC>;
  const FewUnits u = few_units(R.n, K, N, COLS, gridDim.x);
  float *xs = smem, *red = smem + kUnitRows * 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int total = R.n * u.blocks * u.slices;
  for (int w = blockIdx.x; w < total; w += gridDim.x) {
    const int i = w / (u.blocks * u.slices), q = w % (u.blocks * u.slices);
    const int cb = q % u.blocks, s = q / u.blocks;
    const int k0 = s * u.per, k1 = min(K, k0 + u.per);
    const int c = cb * COLS + lane * VEC;
    const T *W = Wall + (size_t)R.expert[i] * K * N + c;
    const int r1 = R.first[i + 1];
    for (int r0 = R.first[i]; r0 < r1; r0 += 8) {
      float acc[8][VEC] = {};
      for (int kb = k0; kb < k1; kb += kUnitRows) {
        const int n = min(kUnitRows, k1 - kb);
        __syncthreads();
        for (int j = tid; j < 8 * kUnitRows; j += kFewThreads) {
          const int r = j / kUnitRows, kk = j % kUnitRows;
          float v = 0.f;
          if (r0 + r < r1 && kk < n) {
            const size_t row = by_token ? R.token[r0 + r] : r0 + r;
            v = few_f(A[row * K + kb + kk]);
          }
          xs[kk * 8 + r] = v;
        }
        __syncthreads();
        if (c < N) {
          const int m0 = warp * 32, m1 = min(n, m0 + 32);
          for (int m = m0; m < m1; m += 8) {
            V wv[8];
#pragma unroll
            for (int z = 0; z < 8; ++z)
              if (m + z < m1)
                wv[z] = *reinterpret_cast<const V *>(W + (size_t)(kb + m + z) * N);
#pragma unroll
            for (int z = 0; z < 8; ++z) {
              if (m + z >= m1) break;
              float f[VEC];
              wv[z].get(f);
              const float4 a = *reinterpret_cast<const float4 *>(xs + (m + z) * 8);
              const float4 b = *reinterpret_cast<const float4 *>(xs + (m + z) * 8 + 4);
              const float xr[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
              for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[r][v] = fmaf(xr[r], f[v], acc[r][v]);
            }
          }
        }
      }
      // Join the warps.
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int v = 0; v < VEC; ++v) red[((warp * 8 + r) * VEC + v) * 32 + lane] = acc[r][v];
      __syncthreads();
      for (int j = tid; j < 8 * VEC * 32; j += kFewThreads) {
        const int r = j / (VEC * 32), l = j % 32, v = j / 32 % VEC;
        const int col = cb * COLS + l * VEC + v;
        if (r0 + r >= r1 || col >= N) continue;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) sum += red[((x * 8 + r) * VEC + v) * 32 + l];
        out[((size_t)s * R.rows + r0 + r) * N + col] = sum;
      }
    }
  }
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kFewThreads, 2) k_few_simt(const FewArgs p) {
  extern __shared__ __align__(16) char smem[];
  float *work = reinterpret_cast<float *>(smem);
  few_start(p);
  few_route<T>(p, work);
  if (!few_barrier(p, 0)) return;
  few_select<T>(p, work);
  if (!few_barrier(p, 1)) return;
  const FewRows R = few_rows(p, smem + kSimtSmemFloats * 4);
  few_product<T, VEC>(R, static_cast<const T *>(p.x), true, static_cast<const T *>(p.W1), p.d,
                      p.F, p.hpart, work);
  if (!few_barrier(p, 2)) return;
  constexpr int V = VEC < 4 ? VEC : 4;
  const int s1 = few_units(R.n, p.d, p.F, 32 * VEC, gridDim.x).slices;
  const int s2 = few_units(R.n, p.F, p.d, 32 * VEC, gridDim.x).slices;
  few_hidden<T, V>(p, R, [&](int, int) { return s1; }, threadIdx.x, kFewThreads);
  if (!few_barrier(p, 3)) return;
  few_product<T, VEC>(R, static_cast<const T *>(p.h), false, static_cast<const T *>(p.W2), p.F,
                      p.d, p.zpart, work);
  if (!few_barrier(p, 4)) return;
  few_combine<T, V>(p, R, [&](int, int) { return s2; });
}

template <typename T, int VEC>
cudaError_t run_simt(const FewArgs &p, cudaStream_t s) {
  const size_t smem = kSimtSmemFloats * 4 + few_rows_bytes(p.E, p.T * p.k);
  int grid = 2 * sm_count();  // two blocks fit an SM (launch bounds, 62 KB at most)
  if (grid > kFewMaxGrid) grid = kFewMaxGrid;
  FewArgs a = p;
  a.rt = few_router(p.T, p.d, p.E, p.Wn != nullptr, grid);
  void *args[1] = {&a};
  return launch_few_grid(reinterpret_cast<const void *>(k_few_simt<T, VEC>), args, grid, smem, s);
}

}  // namespace

cudaError_t launch_few_grid(const void *kernel, void **args, int grid, size_t smem,
                            cudaStream_t s) {
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

FewLayout few_layout(const moe_config &c) {
  FewLayout L{};
  const size_t T = c.T, E = c.E, k = c.k, d = c.d, F = c.d_ff, A = T * k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) / 256 * 256;
    return o;
  };
  L.status = take(sizeof(DeviceStatus));
  L.flags = take((size_t)kFewBarriers * kFewMaxGrid * kFewFlag * 8);
  L.n_tiles = few_tc_supported(c) ? few_tc_tiles(c) : 0;
  L.tiles = take((size_t)L.n_tiles * 4);
  L.idx = take(A * 4);
  L.gate = take(A * 4);
  // Router: slices * columns <= (grid + groups) * 32, with noise or without.
  L.rpart = take(T * 32 * (kFewMaxGrid + 2 * (2 * E + 31) / 32 + 1) * 4);
  // A layer's partials: with at most 2 grid / (experts in use * column blocks)
  // + 2 of them per column (both forms) and rows <= T * experts in use (and <=
  // T k), partials * rows * N <= T * 2 grid * (columns of a block) + 2 T k N.
  L.hpart = take((T * 2 * kFewMaxGrid * kFewColsMax + 2 * A * F) * 4);
  L.zpart = take((T * 2 * kFewMaxGrid * kFewColsMax + 2 * A * d) * 4);
  L.h = take(A * F * elem_bytes(c.act_dtype));
  L.total = off;
  return L;
}

cudaError_t launch_few(const FewCall &q, cudaStream_t s) {
  const moe_config &c = q.cfg;
  const FewLayout L = few_layout(c);
  FewArgs p{};
  p.T = c.T;
  p.d = c.d;
  p.E = c.E;
  p.F = c.d_ff;
  p.k = c.k;
  p.C = q.capacity;
  p.mode = q.thr ? kFewThreshold : c.gate_mode == MOE_GATE_SWITCH ? kFewSwitch : kFewTopk;
  p.by_k = FewDiv(c.k);
  p.by_d4 = FewDiv(c.d % 4 == 0 ? c.d / 4 : 1);
  p.by_f4 = FewDiv(c.d_ff % 4 == 0 ? c.d_ff / 4 : 1);
  p.x = q.x;
  p.Wg = q.Wg;
  p.Wn = q.Wn;
  p.noise = q.noise;
  p.bias = q.bias;
  p.thr = q.thr;
  p.W1 = q.W1;
  p.b1 = q.b1;
  p.W2 = q.W2;
  p.b2 = q.b2;
  p.y = q.y;
  p.idx = q.idx ? q.idx : ws_at<int32_t>(q.ws, L.idx);
  p.gate = q.gate ? q.gate : ws_at<float>(q.ws, L.gate);
  p.pos = q.pos;
  p.keep = q.keep;
  p.mask = q.mask;
  p.st = ws_at<DeviceStatus>(q.ws, L.status);
  p.flags = ws_at<unsigned long long>(q.ws, L.flags);
  p.tiles = ws_at<uint32_t>(q.ws, L.tiles);
  p.n_tiles = L.n_tiles;
  p.rpart = ws_at<float>(q.ws, L.rpart);
  p.hpart = ws_at<float>(q.ws, L.hpart);
  p.zpart = ws_at<float>(q.ws, L.zpart);
  p.h = ws_at<char>(q.ws, L.h);
  // A value that no earlier launch and no stale memory holds.
  static std::atomic<unsigned long long> launches{
      (unsigned long long)std::chrono::steady_clock::now().time_since_epoch().count() << 20};
  p.nonce = (launches.fetch_add(1) + 1) * 0x9E3779B97F4A7C15ull | 1ull;
  p.wait_ns = wait_limit_ns();
  if (c.act_dtype == MOE_F32) {
    if (c.d % 4 == 0 && c.d_ff % 4 == 0) return run_simt<float, 4>(p, s);
    return run_simt<float, 1>(p, s);
  }
  if (few_tc_supported(c)) return launch_few_tc(p, s);
  if (c.d % 2 == 0 && c.d_ff % 2 == 0) return run_simt<__nv_bfloat16, 2>(p, s);
  return run_simt<__nv_bfloat16, 1>(p, s);
}

}  // namespace moe
