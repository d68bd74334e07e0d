// The few-token layer on the CUDA cores: fp32 layers, and bf16 layers of
// widths that are not multiples of 8. The weights of the experts in use are
// read in vectors of 2, 4, 8 or 16 bytes, as the widths allow, and multiplied
// with up to 8 rows at a time from registers; more rows read them again, from
// L2 or HBM. A warp asks for nothing while it multiplies a chunk, which is what
// bounds the form: in fp32 one token of the large-expert layer takes 164 us (141
// us at the copy rate), 64 tokens 1.92 ms (0.56). The 128 registers that two
// blocks an SM leave a thread are all in use; fp32 with vectors of four and of
// one and bf16 with vectors of one spill 28 to 36 bytes. moe_forward takes 4.5
// and 6.9 ms there.
#include "few.cuh"

#include <atomic>
#include <chrono>

namespace moe {
namespace {

// ----------------------------------------------------------------------------- experts
// out[s][row][n] = sum over slice s of K of A[row][k] W[e][k][n]. A unit is an
// expert, a block of 32 * VEC columns and a slice of K. The block stages a
// chunk of K of up to 8 rows of A in shared memory, transposed; each of its 8
// warps takes an eighth of the chunk's K and has all its weights (32 values a
// lane) in flight before the rows are staged. The warps' sums are joined in
// shared memory in warp order.
template <int VEC>
struct FewChunk {
  static constexpr int per_warp = 32 / VEC;  // 4 KB in flight a warp (fp32)
  static constexpr int rows = 8 * per_warp;
};

constexpr int kSlices = 8;

// The slices of K, up to kSlices: as many as make the fewest rows of K for the
// busiest block, a chunk begun counted as a whole one (its loads wait as long)
// and a unit's own cost (staging, joining) as 128 rows: 13 tokens in fp32 35.6 ->
// 34.6 us against rows as they are and 64.
struct FewUnits {
  int blocks, slices, per;  // column blocks, slices of K, rows of K per slice
  int total;
  FixedDiv by_blocks, by_tile;  // column blocks; units of an expert
  __device__ void make(int n_experts, int K, int N, int cols, int chunk, int grid) {
    blocks = (N + cols - 1) / cols;
    const int tiles = n_experts * blocks;
    int best = 0x7fffffff;
    slices = 1;
    per = K;
    for (int s = 1; s <= kSlices; ++s) {
      const int rows = ((K + s - 1) / s + 31) / 32 * 32, n = (K + rows - 1) / rows;
      const int cost = (tiles * n + grid - 1) / grid * ((rows + chunk - 1) / chunk * chunk + 128);
      if (cost < best) {
        best = cost;
        slices = n;
        per = rows;
      }
    }
    total = tiles * slices;
    by_blocks = FixedDiv(blocks);
    by_tile = FixedDiv(blocks * slices);
  }
};

template <typename T, int VEC>
struct FewVec;
template <>
struct FewVec<float, 4> {
  float4 v;
  __device__ void get(float (&f)[4]) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};
template <>
struct FewVec<float, 2> {
  float2 v;
  __device__ void get(float (&f)[2]) const { f[0] = v.x; f[1] = v.y; }
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

// smem: xs [chunk rows][8], red [8 warps][8 rows][VEC][32 lanes].
constexpr int kSimtSmemFloats = 256 * 8 + 8 * 8 * 32 * 4;

// The rows of a product's left operand: layer 1's are tokens' x; layer 2's the
// hidden ones, made of layer 1's partial sums where they are staged (ReLU of
// their sum and b1, rounded once to the layer's type: the layer's hidden rows are
// of that type, in moe_expert_ffn and on the tensor cores too).
template <typename T>
struct FewX {
  const FewRows &rows;
  const T *x;
  int K;
  __device__ float operator()(int row, int k, int) const {
    return few_f(x[(size_t)rows.token[row] * K + k]);
  }
};
template <typename T>
struct FewH {
  const float *part;
  size_t step;  // between the slices
  const T *b1;
  int K, slices;
  __device__ float operator()(int row, int k, int e) const {
    const float *p = part + (size_t)row * K + k;
    float v = 0.f;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) v += __ldcg(p + s * step);
    if (b1) v += few_f(b1[(size_t)e * K + k]);
    return few_f(few_t<T>(max_nan(v, 0.f)));
  }
};

// One unit's sums of rows r0 .. r0 + R - 1 (those below r1) of expert e.
template <typename T, int VEC, int R, typename AF>
__device__ __forceinline__ void few_unit(const AF &A, int e, const T *W, bool live, int N, int k0,
                                         int k1, int r0, int r1, int c0, float *out,
                                         float *smem) {
  using V = FewVec<T, VEC>;
  constexpr int PW = FewChunk<VEC>::per_warp, CH = FewChunk<VEC>::rows;
  float *xs = smem, *red = smem + CH * 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float acc[R][VEC] = {};
  for (int kb = k0; kb < k1; kb += CH) {
    const int n = min(CH, k1 - kb), m0 = warp * PW;
    V wv[PW];
#pragma unroll
    for (int z = 0; z < PW; ++z)
      if (live && m0 + z < n) wv[z] = *reinterpret_cast<const V *>(W + (size_t)(kb + m0 + z) * N);
    constexpr int NX = (R * CH + kFewThreads - 1) / kFewThreads;
    float xv[NX];
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int i = j * kFewThreads + tid, r = i / CH, kk = i % CH;
      xv[j] = 0.f;
      if (r < R && r0 + r < r1 && kk < n) xv[j] = A(r0 + r, kb + kk, e);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int i = j * kFewThreads + tid;
      if (i < R * CH) xs[i % CH * R + i / CH] = xv[j];
    }
    __syncthreads();
    if (live) {
#pragma unroll
      for (int z = 0; z < PW; ++z) {
        if (m0 + z >= n) break;
        float f[VEC], x[R];
        wv[z].get(f);
        if constexpr (R == 8) {
          const float4 a = *reinterpret_cast<const float4 *>(xs + (m0 + z) * 8);
          const float4 b = *reinterpret_cast<const float4 *>(xs + (m0 + z) * 8 + 4);
          x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
          x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
          const float2 a = *reinterpret_cast<const float2 *>(xs + (m0 + z) * 2);
          x[0] = a.x; x[1] = a.y;
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < VEC; ++v) acc[r][v] = fmaf(x[r], f[v], acc[r][v]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < VEC; ++v) red[((warp * R + r) * VEC + v) * 32 + lane] = acc[r][v];
  __syncthreads();
  for (int j = tid; j < R * VEC * 32; j += kFewThreads) {
    const int r = j / (VEC * 32), l = j % 32, v = j / 32 % VEC;
    const int col = c0 + l * VEC + v;
    if (r0 + r >= r1 || col >= N) continue;
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) sum += red[((x * R + r) * VEC + v) * 32 + l];
    out[(size_t)(r0 + r) * N + col] = sum;
  }
}

// One or two rows, the usual number, cost a quarter of eight's arithmetic.
template <typename T, int VEC, typename AF>
__device__ void few_product(const FewRows &R, const FewUnits &u, const AF &A, const T *Wall, int K,
                            int N, float *out, float *smem) {
  constexpr int COLS = 32 * VEC;
  const int lane = threadIdx.x & 31;
  for (int w = blockIdx.x; w < u.total; w += gridDim.x) {
    const int i = (int)u.by_tile(w), q = w - i * u.blocks * u.slices;
    const int s = (int)u.by_blocks(q), cb = q - s * u.blocks;
    const int k0 = s * u.per, k1 = min(K, k0 + u.per), c = cb * COLS + lane * VEC;
    const int e = R.expert[i];
    const T *W = Wall + (size_t)e * K * N + c;
    float *o = out + (size_t)s * R.rows * N;
    const int r1 = R.first[i + 1];
    for (int r0 = R.first[i]; r0 < r1;) {
      if (r1 - r0 <= 2) {
        few_unit<T, VEC, 2>(A, e, W, c < N, N, k0, k1, r0, r1, cb * COLS, o, smem);
        r0 += 2;
      } else {
        few_unit<T, VEC, 8>(A, e, W, c < N, N, k0, k1, r0, r1, cb * COLS, o, smem);
        r0 += 8;
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
  __shared__ FewAlone alone;
  few_select<T>(p, work, alone);
  if (p.T == 1) __syncthreads();
  else if (!few_barrier(p, 1)) return;
  const FewRows R = few_rows(p, smem + kSimtSmemFloats * 4, alone);
  __shared__ __align__(8) unsigned char unit_mem[2 * sizeof(FewUnits)];
  FewUnits *u = reinterpret_cast<FewUnits *>(unit_mem);
  if (threadIdx.x < 64 && threadIdx.x % 32 == 0) {
    const bool second = threadIdx.x == 32;
    u[second].make(R.n, second ? p.F : p.d, second ? p.d : p.F, 32 * VEC,
                   FewChunk<VEC>::rows, gridDim.x);
  }
  __syncthreads();
  const FewX<T> x{R, static_cast<const T *>(p.x), p.d};
  few_product<T, VEC>(R, u[0], x, static_cast<const T *>(p.W1), p.d, p.F, p.hpart, work);
  if (!few_barrier(p, 2)) return;
  const FewH<T> h{p.hpart, (size_t)R.rows * p.F, static_cast<const T *>(p.b1), p.F, u[0].slices};
  few_product<T, VEC>(R, u[1], h, static_cast<const T *>(p.W2), p.F, p.d, p.zpart, work);
  few_combine<T, VEC>(p, R, [&](int, int) { return u[1].slices; });
}

template <typename T, int VEC>
cudaError_t run_simt(const FewArgs &p, cudaStream_t s) {
  const size_t smem = kSimtSmemFloats * 4 + few_rows_bytes(p.E, p.T * p.k);
  constexpr size_t most = kSimtSmemFloats * 4 + few_rows_bytes(1024, kFewRows);
  int grid = 2 * sm_count();  // two blocks fit an SM (launch bounds, 72 KB at most)
  if (grid > kFewMaxGrid) grid = kFewMaxGrid;
  FewArgs a = p;
  a.rt = few_router(p.T, p.d, p.E, p.Wn != nullptr, grid);
  void *args[1] = {&a};
  return launch_few_grid(reinterpret_cast<const void *>(k_few_simt<T, VEC>), args, grid, smem,
                         most, s);
}

}  // namespace

cudaError_t launch_few_grid(const void *kernel, void **args, int grid, size_t smem, size_t most,
                            cudaStream_t s) {
  cudaError_t err = allow_smem(kernel, most);
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
  err = cudaLaunchKernelExC(&cfg, kernel, args);
  if (err != cudaSuccess) cudaGetLastError();  // reported here, not by the next call
  return err;
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
  L.flags = take((size_t)(kFewMaxGrid + kFewBarriers - 1) * kFewFlag * 8);
  L.n_tiles = few_on_tc(c) ? few_tc_tiles(c) : 0;
  L.tiles = take((size_t)L.n_tiles * 4);
  L.idx = take(A * 4);
  L.gate = take(A * 4);
  // Router: slices * columns <= (grid + groups) * 32, with noise or without.
  L.rpart = take(T * 32 * (kFewMaxGrid + 2 * (2 * E + 31) / 32 + 1) * 4);
  // A layer's partial sums. On the CUDA cores: at most kSlices of every value.
  // On the tensor cores a tile has at most KC / (a run's length) + 2, and a run
  // at least 2 / 3 of total / G units (total / G rounded down, 2 at least); with
  // total = experts in use * NT * KC and rows <= T * experts in use that is
  // 1.5 T G kFewTile floats and two of every value.
  const auto partials = [&](size_t N) {
    return few_on_tc(c) ? T * 2 * kFewMaxGrid * kFewTile + 2 * A * N : kSlices * A * N;
  };
  L.hpart = take(partials(F) * 4);
  L.zpart = take(partials(d) * 4);
  L.h = take(few_on_tc(c) ? A * F * 2 : 0);
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
  p.by_k = FixedDiv(c.k);
  p.by_d4 = FixedDiv(c.d % 4 == 0 ? c.d / 4 : 1);
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
  p.n_tiles = c.T > 1 ? L.n_tiles : 0;  // a single token's tiles are not joined
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
    if (c.d % 2 == 0 && c.d_ff % 2 == 0) return run_simt<float, 2>(p, s);
    return run_simt<float, 1>(p, s);
  }
  if (few_on_tc(c)) return launch_few_tc(p, s);
  if (c.d % 2 == 0 && c.d_ff % 2 == 0) return run_simt<__nv_bfloat16, 2>(p, s);
  return run_simt<__nv_bfloat16, 1>(p, s);
}

}  // namespace moe
