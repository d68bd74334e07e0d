// Gated experts on the CUDA cores: fp32 layers (the tensor cores have no fp32
// input kind) and bf16 widths that the tensor-core kernels do not take. With
// the packed rows r of expert e (token t, gate g):
//   forward 1:  p1 = x W1 + b1, p3 = x W3 + b3, h = act(p1) * p3
//   forward 2:  z = g * (h W2 + b2)
//   backward 1: D = dy W2^T; dgate's <D, h>; dP1 = g D p3 act'(p1), dP3 = g D act(p1)
//   backward 2: dX = dP1 W1^T + dP3 W3^T
//   backward 3: dW1 = x^T dP1, dW3 = x^T dP3, dW2 = h^T (g dy)
// One tiled product with these operands and epilogues: 16 TM x 16 TN outputs a
// block of 256 threads, TM x TN a thread, packed fp32 multiply-adds (two a lane and
// instruction), K in chunks whose next one is fetched while this one is multiplied.
// Tiles of 128 x 128: chunks of 16, two in shared memory, two blocks an SM (bound by
// the multiply-adds: 5019 tokens, top-4 of 5 experts of 181 x 683, layer 1 249 us
// with that pipe active 66% of the time). Tiles of 64 x 64: chunks of 64 in the
// forward, whose blocks are few and wait for each (75 -> 61 us for 517 rows of 130
// through 6 experts of 234); of 16 in the backward, whose launches share the SMs
// (108 -> 98). Both projections of forward 1 share a block's columns, so that a
// thread holds p1 and p3 of the same places. The three weight gradients are one
// launch; where their tiles are fewer than four an SM, slices of an expert's rows
// go to fp32 sums that a second launch adds in order (4246 tokens, top-3 of 3
// experts of 96 x 208: the backward 425 -> 188 us).
#include "gated.cuh"

#include <algorithm>

namespace moe {
namespace {

constexpr int kThreads = 256, kSliceRows = 256;

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

enum Op { kF1, kF2, kB1, kB2, kW };  // kW: the weight gradients

// c += a * b on two floats at once, kept as they are in registers.
__device__ __forceinline__ void fma_pair(unsigned long long &c, unsigned long long a,
                                     unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}

template <int OP, typename T, int ACT, int TM, int TN>
__global__ void __launch_bounds__(kThreads, TM == 8 ? 2 : 1)
k_gated_simt(const GatedSimt p) {
  pdl_wait();
  pdl_trigger();
  constexpr int BM = 16 * TM, BN = 16 * TN, BK = TM == 8 ? 16 : OP == kF1 || OP == kF2 ? 64 : 16;
  constexpr int KL = BK, KR = kThreads / BK;  // K-contiguous operands: lanes along K, rows a pass
  constexpr bool kWeight = OP == kW;
  constexpr int LA = BM * BK / kThreads, LB = BN * BK / kThreads;
  constexpr int NB = TM == 8 ? 2 : 1;  // chunks in shared memory
  __shared__ __align__(16) float As[NB][BK][BM + (TM == 8 ? 4 : 2)];
  __shared__ __align__(16) float Bs[NB][BK][BN + (TN == 8 ? 4 : 2)];
  const int E = p.c.E, d = p.c.d, F = p.c.d_ff, k = p.c.k;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;

  // The block's expert, first row and row count. A weight gradient's blocks are
  // (weight, row block, column block) along x, experts along y.
  int e, m0, n0, which = 0;
  constexpr int BNu = OP == kF1 ? BN / 2 : BN;  // columns of the output a block covers
  if constexpr (kWeight) {
    const int db = (d + BM - 1) / BM, fb = (F + BM - 1) / BM;  // BM = BN
    int i = blockIdx.x;
    which = i / (db * fb);
    i -= which * db * fb;
    const int mb = which == 2 ? fb : db;  // dW1, dW3: [d, F]; dW2: [F, d]
    e = blockIdx.y;
    n0 = i / mb * BN;
    m0 = i % mb * BM;
  } else {
    constexpr int kSplit = kTcBM / BM;  // blocks for each 128-row tile
    __shared__ int starts[1025];
    const int tile = blockIdx.x / kSplit;
    for (int i = tid; i <= E; i += kThreads) starts[i] = p.rows.mtiles[i];
    __syncthreads();
    if (tile >= starts[E]) return;
    int lo = 0, hi = E;  // largest e with starts[e] <= tile
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= tile) lo = mid;
      else hi = mid;
    }
    e = lo;
    m0 = (tile - starts[e]) * kTcBM + (blockIdx.x % kSplit) * BM;
    n0 = blockIdx.y * BNu;
  }
  const int r0 = p.rows.offset[e], rows = p.rows.offset[e + 1] - r0;
  if (!kWeight && m0 >= rows) return;
  const int M = kWeight ? (which == 2 ? F : d) : rows;
  const int N = kWeight ? (which == 2 ? d : F) : OP == kF1 || OP == kB1 ? F : d;
  // A weight gradient's slice of the rows (along z): [kbeg, kbeg + K).
  const int slice = kWeight ? ((rows + (int)gridDim.z - 1) / (int)gridDim.z + BK - 1) / BK * BK : 0;
  const int kbeg = kWeight ? min(rows, (int)blockIdx.z * slice) : 0;
  const int K = kWeight ? min(rows - kbeg, slice)
                        : OP == kF1 || OP == kB1 ? d : OP == kF2 ? F : 2 * F;
  const size_t we = (size_t)e * d * F;  // this expert's place in each weight

  // A: rows (K contiguous; K in lanes) or, for a weight gradient, columns of
  // the rows (M contiguous). Rows of x and dy are read through their token.
  size_t arow[kWeight ? 1 : LA];
  if (!kWeight) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int m = m0 + tid / KL + KR * i;
      const int r = r0 + min(m, rows - 1);
      if (OP == kF1 || OP == kB1) arow[i] = (size_t)(p.rows.row_token[r] / k) * d;
      else arow[i] = (size_t)r * F;
    }
  }
  const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
  const T *W1 = static_cast<const T *>(p.W1) + we, *W3 = static_cast<const T *>(p.W3) + we;
  const T *W2 = static_cast<const T *>(p.W2) + we;
  // A weight gradient's rows [rows, M] and [rows, N].
  const float *wa = nullptr, *wb = nullptr;
  if constexpr (kWeight) {
    wa = (which == 2 ? p.hf : p.xf) + (size_t)(r0 + kbeg) * M;
    wb = (which == 0 ? p.dP1 : which == 1 ? p.dP3 : p.dU) + (size_t)(r0 + kbeg) * N;
  }

  float ra[LA] = {}, rb[LB] = {};
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      float v = 0.f;
      if constexpr (kWeight) {
        const int mm = tid % BM, kk = k0 + tid / BM + i * (kThreads / BM), m = m0 + mm;
        if (m < M && kk < K) v = wa[(size_t)kk * M + m];
      } else {
        const int kk = k0 + tid % KL, m = m0 + tid / KL + KR * i;
        if (m < M && kk < K) {
          if (OP == kF1) v = ld(x, arow[i] + kk);
          else if (OP == kF2) v = ld(static_cast<const T *>(p.h), arow[i] + kk);
          else if (OP == kB1) v = ld(dy, arow[i] + kk);
          else v = (kk < F ? p.dP1 + kk : p.dP3 + (kk - F))[arow[i]];
        }
      }
      ra[i] = v;
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      float v = 0.f;
      if constexpr (OP == kB1 || OP == kB2) {  // the weight's rows are the output's columns
        const int kk = k0 + tid % KL, n = n0 + tid / KL + KR * i;
        if (n < N && kk < K) {
          if (OP == kB1) v = ld(W2, (size_t)n * d + kk);
          else v = ld(kk < F ? W1 + kk : W3 + (kk - F), (size_t)n * F);
        }
      } else {
        const int nn = tid % BN, kk = k0 + tid / BN + i * (kThreads / BN);
        const bool second = OP == kF1 && nn >= BNu;
        const int n = n0 + (second ? nn - BNu : nn);
        if (n < N && kk < K) {
          if (OP == kF1) v = ld(second ? W3 : W1, (size_t)kk * F + n);
          else if (OP == kF2) v = ld(W2, (size_t)kk * d + n);
          else v = wb[(size_t)kk * N + n];
        }
      }
      rb[i] = v;
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      if (kWeight) As[buf][tid / BM + i * (kThreads / BM)][tid % BM] = ra[i];
      else As[buf][tid % KL][tid / KL + KR * i] = ra[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      if (OP == kB1 || OP == kB2) Bs[buf][tid % KL][tid / KL + KR * i] = rb[i];
      else Bs[buf][tid / BN + i * (kThreads / BN)][tid % BN] = rb[i];
    }
  };

  // Thread (ty, tx) holds rows {0, BM/2} + ty TM/2 + .. and columns {0, BN/2} +
  // tx TN/2 + .., so that its operands are short vectors and, in forward 1, the
  // second half of its columns is W3's.
  constexpr int HM = TM / 2, HN = TN / 2;
  unsigned long long acc[TM][TN / 2] = {};
  int buf = 0;
  if (K > 0) fetch(0);
  if (NB == 2) {
    stage(0);
    __syncthreads();
  }
  for (int k0 = 0; k0 < K; k0 += BK) {
    if (NB == 1) {
      stage(0);
      __syncthreads();
    }
    if (k0 + BK < K) fetch(k0 + BK);
#pragma unroll 16
    for (int kk = 0; kk < BK; ++kk) {
      __align__(16) float a[TM];
      unsigned long long b[TN / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float *row = &As[buf][kk][h * (BM / 2) + ty * HM];
        if constexpr (HM == 4)
          *reinterpret_cast<float4 *>(&a[4 * h]) = *reinterpret_cast<const float4 *>(row);
        else
          *reinterpret_cast<float2 *>(&a[2 * h]) = *reinterpret_cast<const float2 *>(row);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float *row = &Bs[buf][kk][h * (BN / 2) + tx * HN];
        if constexpr (HN == 4) {
          const ulonglong2 u = *reinterpret_cast<const ulonglong2 *>(row);
          b[2 * h] = u.x;
          b[2 * h + 1] = u.y;
        } else {
          b[h] = *reinterpret_cast<const unsigned long long *>(row);
        }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const unsigned long long aa = pack2(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) fma_pair(acc[i][j], aa, b[j]);
      }
    }
    if (NB == 2 && k0 + BK < K) stage(buf ^= 1);
    __syncthreads();
  }

  const T *b1 = static_cast<const T *>(p.b1), *b3 = static_cast<const T *>(p.b3);
  const T *b2 = static_cast<const T *>(p.b2);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + (i / HM) * (BM / 2) + ty * HM + i % HM;
    float v[TN];
#pragma unroll
    for (int j = 0; j < TN / 2; ++j)
      asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "l"(acc[i][j]));
    const bool live = m < M;
    const size_t r = (size_t)r0 + m;
    bool bad = false;
    if constexpr (OP == kF1) {
      if (!live) continue;
#pragma unroll
      for (int j = 0; j < HN; ++j) {
        const int n = n0 + tx * HN + j;
        if (n >= N) continue;
        float p1 = v[j], p3 = v[HN + j];
        if (b1) p1 += ld(b1, (size_t)e * F + n);
        if (b3) p3 += ld(b3, (size_t)e * F + n);
        if (p.pre1) put(static_cast<T *>(p.pre1), r * F + n, p1);
        if (p.pre3) put(static_cast<T *>(p.pre3), r * F + n, p3);
        float a, sl;
        gated_act_slope<ACT>(p1, a, sl);
        put(static_cast<T *>(p.h), r * F + n, a * p3);
      }
    } else if constexpr (OP == kB1) {
      const float g = live ? p.rows.row_gate[r] : 0.f;
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + (j / HN) * (BN / 2) + tx * HN + j % HN;
        if (!live || n >= N) continue;
        const float p1 = ld(static_cast<const T *>(p.pre1), r * F + n);
        const float p3 = ld(static_cast<const T *>(p.pre3), r * F + n);
        float a, sl;
        gated_act_slope<ACT>(p1, a, sl);
        const float h = a * p3, D = v[j];
        part = fmaf(D, h, part);
        p.hf[r * F + n] = h;
        p.dP1[r * F + n] = g * D * p3 * sl;
        p.dP3[r * F + n] = g * D * a;
      }
      // Over the 16 lanes that share the row.
#pragma unroll
      for (int o = 8; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
      if (live && tx == 0) p.dgpart[r * gridDim.y + blockIdx.y] = part;
    } else {
      if (!live) continue;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + (j / HN) * (BN / 2) + tx * HN + j % HN;
        if (n >= N) continue;
        float u = v[j];
        if constexpr (OP == kF2) {
          if (b2) u += ld(b2, (size_t)e * d + n);
          u *= p.rows.row_gate[r];
          p.z[r * d + n] = u;
        } else if constexpr (OP == kB2) {
          p.dX[r * d + n] = u;
        } else if (gridDim.z > 1) {
          p.wpart[((size_t)blockIdx.z * 3 + which) * E * d * F + we + (size_t)m * N + n] = u;
          continue;
        } else {
          void *out = which == 0 ? p.dW1 : which == 1 ? p.dW3 : p.dW2;
          put(static_cast<T *>(out), we + (size_t)m * N + n, u);
        }
        bad |= !isfinite(u);
      }
    }
    if (bad) record_error(p.st, MOE_ERR_NONFINITE, (long long)(kWeight ? m : r));
  }
}

// dU[r] = g * dy and xf[r] = x of the row's token, in fp32; one warp per packed
// row.
template <typename T>
__global__ void __launch_bounds__(256) k_gated_rows(const GatedSimt p) {
  pdl_wait();
  pdl_trigger();
  const long long r = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  if (r >= p.max_rows || r >= p.rows.offset[p.c.E]) return;
  const size_t src = (size_t)(p.rows.row_token[r] / p.c.k) * p.c.d;
  const float g = p.rows.row_gate[r];
#pragma unroll 4
  for (int i = threadIdx.x & 31; i < p.c.d; i += 32) {
    p.dU[r * p.c.d + i] = g * ld(static_cast<const T *>(p.dy), src + i);
    p.xf[r * p.c.d + i] = ld(static_cast<const T *>(p.x), src + i);
  }
}

// The weight gradients from their slices' sums, in order; grid (elements of one, 3).
template <typename T>
__global__ void __launch_bounds__(256) k_gated_wsum(const GatedSimt p, int slices) {
  pdl_wait();
  pdl_trigger();
  const size_t n = (size_t)p.c.E * p.c.d * p.c.d_ff, i = blockIdx.x * (size_t)256 + threadIdx.x;
  if (i >= n) return;
  const int which = blockIdx.y;
  const float *src = p.wpart + which * n + i;
  float v = 0.f;
#pragma unroll 4
  for (int s = 0; s < slices; ++s) v += src[(size_t)s * 3 * n];
  void *out = which == 0 ? p.dW1 : which == 1 ? p.dW3 : p.dW2;
  put(static_cast<T *>(out), i, v);
  if (!isfinite(v))
    record_error(p.st, MOE_ERR_NONFINITE,
                 (long long)(i % ((size_t)p.c.d * p.c.d_ff) / (which == 2 ? p.c.d : p.c.d_ff)));
}

// Rows in 128-row tiles at most: every expert's last one may be short.
long long max_tiles(const GatedSimt &p) {
  return ((long long)p.max_rows + kTcBM - 1) / kTcBM + (p.c.E < p.max_rows ? p.c.E : p.max_rows);
}

// The weight gradients' tiles, and the slices of an expert's rows that give every
// SM four blocks where the tiles alone do not. Workspaces are sized by these, so
// they count on kPlanSms.
// Slices of kSliceRows rows at least, at uniform loads (of 128: the same times).
struct WeightSplit {
  bool wide;
  int slices;
};
WeightSplit weight_split(const moe_config &c, int max_rows) {
  const auto blocks = [&](int t) {
    return 3ll * c.E * ((c.d + t - 1) / t) * ((c.d_ff + t - 1) / t);
  };
  const long long most = std::min(16, std::max(1, max_rows / c.E / kSliceRows));
  const bool wide = max_rows >= 64 * c.E && blocks(128) * most >= 2 * kPlanSms;
  const long long b = blocks(wide ? 128 : 64);
  return {wide, (int)std::min(most, (4ll * kPlanSms + b - 1) / b)};
}

template <int OP, typename T, int ACT, int TM, int TN>
cudaError_t run_one(const GatedSimt &p, cudaStream_t s) {
  constexpr int BM = 16 * TM, BN = 16 * TN;
  const int N = OP == kF1 || OP == kB1 ? p.c.d_ff : p.c.d;
  const int BNu = OP == kF1 ? BN / 2 : BN;
  dim3 grid;
  if (OP == kW)
    grid = dim3(3 * ((p.c.d + BM - 1) / BM) * ((p.c.d_ff + BM - 1) / BM), p.c.E,
                weight_split(p.c, p.max_rows).slices);
  else  // row blocks fastest: they share the weight's columns
    grid = dim3((unsigned)(max_tiles(p) * (kTcBM / BM)), (N + BNu - 1) / BNu);
  return launch_pdl_c(kPdlGemm, k_gated_simt<OP, T, ACT, TM, TN>, grid, kThreads, 0, s, p);
}

// 128 x 128 tiles where they give every SM a block and rows to fill them, else
// 64 x 64 (517 rows of 130 through 6 experts of 234: 23 us a layer 1 with tiles
// of 32 x 64, whose threads hold 2 x 4 and spend their instructions on loads).
bool wide_tiles(const moe_config &c, int max_rows, int op) {
  if (op == kW) return weight_split(c, max_rows).wide;
  const int N = (op == kF1 ? 2 : 1) * (op == kF2 || op == kB2 ? c.d : c.d_ff);
  return ((long long)max_rows + 127) / 128 * ((N + 127) / 128) >= 2 * kPlanSms &&
         max_rows >= 64 * c.E;
}

template <int OP, typename T, int ACT>
cudaError_t run_op(const GatedSimt &p, cudaStream_t s) {
  if (!wide_tiles(p.c, p.max_rows, OP)) return run_one<OP, T, ACT, 4, 4>(p, s);
  // Columns that leave half a tile empty (5019 tokens through 5 experts of 181 x
  // 683: 505 -> 470 us; from 256 columns on the half tiles cost what they save).
  if constexpr (OP == kF2 || OP == kB2) {
    if (p.c.d < 256 && (p.c.d + 63) / 64 % 2) return run_one<OP, T, ACT, 8, 4>(p, s);
  }
  return run_one<OP, T, ACT, 8, 8>(p, s);
}

template <typename T>
cudaError_t forward(const GatedSimt &p, cudaStream_t s) {
  const cudaError_t err = gated_dispatch(p.activation, [&](auto act) {
    return run_op<kF1, T, decltype(act)::value>(p, s);
  });
  return err != cudaSuccess ? err : run_op<kF2, T, MOE_ACT_RELU>(p, s);
}

template <typename T>
cudaError_t backward_front(const GatedSimt &p, cudaStream_t s) {
  const cudaError_t err =
      launch_pdl(k_gated_rows<T>, (unsigned)((p.max_rows + 7ll) / 8), 256, 0, s, p);
  if (err != cudaSuccess) return err;
  return gated_dispatch(p.activation, [&](auto act) {
    return run_op<kB1, T, decltype(act)::value>(p, s);
  });
}

}  // namespace

int gated_simt_dg_blocks(const moe_config &c, int max_rows) {
  const int cols = wide_tiles(c, max_rows, kB1) ? 128 : 64;
  return (c.d_ff + cols - 1) / cols;
}

cudaError_t launch_gated_simt_forward(const GatedSimt &p, cudaStream_t s) {
  return p.c.act_dtype == MOE_BF16 ? forward<__nv_bfloat16>(p, s) : forward<float>(p, s);
}

cudaError_t launch_gated_simt_front(const GatedSimt &p, cudaStream_t s) {
  return p.c.act_dtype == MOE_BF16 ? backward_front<__nv_bfloat16>(p, s)
                                   : backward_front<float>(p, s);
}

cudaError_t launch_gated_simt_dx(const GatedSimt &p, cudaStream_t s) {
  return p.c.act_dtype == MOE_BF16 ? run_op<kB2, __nv_bfloat16, MOE_ACT_RELU>(p, s)
                                   : run_op<kB2, float, MOE_ACT_RELU>(p, s);
}

size_t gated_simt_wpart(const moe_config &c, int max_rows) {
  const int slices = weight_split(c, max_rows).slices;
  return slices > 1 ? 12ull * slices * c.E * c.d * c.d_ff : 0;
}

template <typename T>
static cudaError_t weights(const GatedSimt &p, cudaStream_t s) {
  const cudaError_t err = run_op<kW, T, MOE_ACT_RELU>(p, s);
  const int slices = weight_split(p.c, p.max_rows).slices;
  if (err != cudaSuccess || slices == 1) return err;
  const size_t n = (size_t)p.c.E * p.c.d * p.c.d_ff;
  return launch_pdl(k_gated_wsum<T>, dim3((unsigned)((n + 255) / 256), 3), 256, 0, s, p, slices);
}

cudaError_t launch_gated_simt_weights(const GatedSimt &p, cudaStream_t s) {
  return p.c.act_dtype == MOE_BF16 ? weights<__nv_bfloat16>(p, s) : weights<float>(p, s);
}

}  // namespace moe
