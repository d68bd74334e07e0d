// The few-token layer (moe_forward_few, moe_forward_threshold_few): arguments
// of its kernels, the barrier between its phases, and the phases that both
// forms of the experts share. Internal to libmoe.so.
//
// One persistent cooperative grid runs the whole layer for T <= 64 tokens:
//   router     partial sums of x W_g (and x W_noise) over slices of d
//   selection  one block per token: logits, top-k or threshold mask, gates
//   (every block then derives the capacity's slots and the experts' rows)
//   layer 1    partial sums of x W1 over slices of d, for the experts in use
//   layer 2    H = ReLU(sum + b1), rounded to the layer's type, and the partial
//              sums of H W2 over slices of d_ff
//   combine    y = x + sum of gate * (sum + b2)
// with a barrier over the grid after each but the last.
#pragma once

#include "moe_internal.cuh"
#include "tc_ptx.cuh"

#include <math.h>

namespace moe {

constexpr int kFewTokens = 64;     // T at most: an expert's tokens are one 64-bit mask
constexpr int kFewRows = 1024;     // T * k at most (k <= 16)
constexpr int kFewThreads = 256;
constexpr int kFewMaxGrid = 320;   // blocks at most (sizes the flags and partial sums)
constexpr int kFewBarriers = 4;
constexpr int kFewFlag = 16;       // 64-bit words from one flag or count to the next (128 bytes)
constexpr int kFewTile = 256;      // weight columns of a unit on the tensor cores
enum FewMode { kFewTopk = 0, kFewSwitch = 1, kFewThreshold = 2 };

// The router's units (few_router).
struct FewRouter {
  int NC, groups, slices, rows_per_slice;
  int lcw;  // log2 of the columns of a unit (8 to 32)
  int lt;   // log2 of the groups of 8 tokens (2 to 8)
  FixedDiv by_group;
};

struct FewArgs {
  int T, d, E, F, k, C, mode;
  FewRouter rt;
  FixedDiv by_k, by_d4;  // k; d / 4 (1 where it is not whole)
  const void *x;
  const float *Wg, *Wn, *noise, *bias, *thr;
  const void *W1, *b1, *W2, *b2;
  void *y;
  int32_t *idx;    // [T, k]
  float *gate;     // [T, k]
  int32_t *pos;    // [T, k] or null
  uint8_t *keep;   // [T, k] or null
  uint32_t *mask;  // [T, ceil(E/32)] or null (threshold)
  // Workspace.
  DeviceStatus *st;
  // The first word of each kFewFlag: the first barrier's flags [kFewMaxGrid], the others' counts.
  unsigned long long *flags;
  uint32_t *tiles;            // pieces of layer 1's tiles that are written (tensor-core form)
  int n_tiles;
  float *rpart;               // router partials [slices][T][columns]
  float *hpart, *zpart;       // partials of the layers [slices][rows][N]
  void *h;                    // [rows, F] in bf16 (tensor-core form)
  unsigned long long nonce, wait_ns;
};

namespace {

// ----------------------------------------------------------------------------- grid barrier
// The first barrier: every block stores the launch's nonce to a flag of its
// own, on a 128-byte line of its own (152 blocks polling 152 flags on ten lines
// took 2 to 5 us: every poll went to the same few L2 slices), and all wait for
// all flags. So the workspace need not be zeroed: flags of an earlier call hold
// another nonce. A replayed graph has the same nonce each time; a block clears
// its flag once it has passed the last barrier, or leaves early. The later
// barriers count arrivals on one word each, which block 0 clears before it
// arrives at the first: one poll a block instead of 152 (one token 22.2 -> 21.1
// us for the noisy top-4 layer). For the first barrier, a tagged count that
// whoever arrives first sets up costs 304 blocks more than the flags do (13
// tokens, fp32: 36.9 against 40.2 us) and gains 152 blocks little.
// Waits are bounded: past the limit the block records MOE_ERR_TIMEOUT and
// leaves, and so does, within the limit, every block that waits for it.
__device__ __forceinline__ void few_flag_set(unsigned long long *f, unsigned long long v) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(f), "l"(v) : "memory");
}
// Relaxed: several can be in flight; the caller fences once it has seen them.
__device__ __forceinline__ unsigned long long few_flag_get(const unsigned long long *f) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(f) : "memory");
  return v;
}

__device__ __forceinline__ unsigned long long *few_flag(const FewArgs &p, int block) {
  return p.flags + (size_t)block * kFewFlag;
}
__device__ __forceinline__ unsigned long long *few_count(const FewArgs &p, int b) {  // b > 0
  return few_flag(p, kFewMaxGrid + b - 1);
}

__device__ __forceinline__ void few_start(const FewArgs &p) {
  if (blockIdx.x == 0) {
    if (threadIdx.x > 0 && threadIdx.x < kFewBarriers) *few_count(p, threadIdx.x) = 0;
    if (threadIdx.x == 0) *p.st = DeviceStatus{};
  }
  for (int i = blockIdx.x * kFewThreads + threadIdx.x; i < p.n_tiles;
       i += gridDim.x * kFewThreads)
    p.tiles[i] = 0;
}

// Arrive at barrier b (one thread, after a barrier of the block's threads that
// wrote): what they wrote before is visible to a block that has waited (a
// release, cumulative over the barrier).
__device__ __forceinline__ void few_arrive(const FewArgs &p, int b) {
  if (b == 0)
    few_flag_set(few_flag(p, blockIdx.x), p.nonce);
  else
    asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(few_count(p, b)) : "memory");
}

// Wait until `done()`; false: leave the kernel. With an abort flag, a set one
// ends the wait too.
template <typename F>
__device__ __forceinline__ bool few_poll(const FewArgs &p, int b, volatile int *abort_flag,
                                         const F &done) {
  unsigned long long t0 = 0;
  while (!done()) {
    const unsigned long long now = globaltimer();
    if (t0 == 0) t0 = now;
    if (abort_flag && *abort_flag) return false;
    if (now - t0 >= p.wait_ns) {
      record_error(p.st, MOE_ERR_TIMEOUT, 100 + b);
      return false;
    }
  }
  return true;
}

// The first barrier, by all threads of the block: up to two flags each.
__device__ __forceinline__ bool few_wait_first(const FewArgs &p) {
  static_assert(kFewMaxGrid <= 2 * kFewThreads);
  const int i = threadIdx.x, j = i + kFewThreads, n = gridDim.x;
  const bool ok = few_poll(p, 0, nullptr, [&] {
    return (i >= n || few_flag_get(few_flag(p, i)) == p.nonce) &
           (j >= n || few_flag_get(few_flag(p, j)) == p.nonce);
  });
  __threadfence();  // the flags' acquire
  return ok;
}
// A later one, by one thread.
__device__ __forceinline__ bool few_wait(const FewArgs &p, int b,
                                         volatile int *abort_flag = nullptr) {
  const bool ok =
      few_poll(p, b, abort_flag, [&] { return few_flag_get(few_count(p, b)) == gridDim.x; });
  __threadfence();  // the count's acquire
  return ok;
}

// A block that leaves the kernel, or has passed the last barrier (then every
// block has passed the first).
__device__ __forceinline__ void few_leave(const FewArgs &p) { *few_flag(p, blockIdx.x) = 0; }

// A barrier in two steps, by all threads; between them the block may do what
// neither the others nor it itself waits for.
__device__ __forceinline__ void few_barrier_arrive(const FewArgs &p, int b) {
  __syncthreads();
  if (threadIdx.x == 0) few_arrive(p, b);
}
__device__ __forceinline__ bool few_barrier_wait(const FewArgs &p, int b) {
  const bool ok = b == 0 ? few_wait_first(p) : threadIdx.x == 0 ? few_wait(p, b) : true;
  const bool fail = __syncthreads_or(!ok);
  if (threadIdx.x == 0 && (b == kFewBarriers - 1 || fail)) few_leave(p);
  return !fail;
}
__device__ __forceinline__ bool few_barrier(const FewArgs &p, int b) {
  few_barrier_arrive(p, b);
  return few_barrier_wait(p, b);
}

// ----------------------------------------------------------------------------- element types
__device__ __forceinline__ float few_f(float v) { return v; }
__device__ __forceinline__ float few_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T few_t(float v);
template <>
__device__ __forceinline__ float few_t<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 few_t<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// ----------------------------------------------------------------------------- router
// Columns: E of W_g, then E of W_noise. A unit is 32 columns (8 or 16 where
// there are no more) and one slice of d, as many units as blocks where that is
// possible.
// 64 rows of the weights and of x (for every token) are staged in shared
// memory at a time.
constexpr int kRtRows = 64;

inline FewRouter few_router(int T, int d, int E, bool noisy, int grid) {
  FewRouter r;
  r.NC = noisy ? 2 * E : E;
  r.lcw = 3;
  while (r.lcw < 5 && (1 << r.lcw) < r.NC) ++r.lcw;
  r.groups = (r.NC + (1 << r.lcw) - 1) >> r.lcw;
  int s = grid / r.groups;
  const int most = (d + 31) / 32;  // slices of at least 32 rows
  if (s > most) s = most;
  if (s < 1) s = 1;
  r.rows_per_slice = ((d + s - 1) / s + 7) / 8 * 8;
  r.slices = (d + r.rows_per_slice - 1) / r.rows_per_slice;
  r.lt = 1;
  while ((8 << r.lt) < T) ++r.lt;
  r.by_group = FixedDiv((unsigned)r.groups);
  return r;
}

// x[t, k .. k+7] as floats, zero past the end.
template <typename T>
__device__ __forceinline__ void few_x8(const T *x, int d, int k, float (&f)[8]) {
  if (d % 8 == 0 && k + 8 <= d) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4 *>(x + k);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4 *>(x + k);
      const float4 b = *reinterpret_cast<const float4 *>(x + k + 4);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
      f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = k + j < d ? few_f(x[k + j]) : 0.f;
  }
}

// fp32 x, on the CUDA cores: a warp takes 8 tokens, and with fewer than 64
// tokens the warps of the same tokens share the rows.
// smem: xs [kRtRows][tokens, a multiple of 8], w [kRtRows][cw], red [8 warps][8][32]:
// 32 KB at most.
template <typename T>
__device__ __forceinline__ void few_route_f32(const FewArgs &p, float *smem) {
  const FewRouter &r = p.rt;
  const int tgp = 1 << r.lt, tp = 8 << r.lt;  // warps, tokens side by side
  const int ks = 8 >> r.lt;                   // warps that share a token group's rows
  const int cw = 1 << r.lcw;
  float *xs = smem, *ws = xs + kRtRows * tp, *red = ws + kRtRows * cw;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tgi = warp & (tgp - 1), kp = warp >> r.lt;
  const int lrows = 32 >> r.lcw, lr = lane >> r.lcw, lc = lane & (cw - 1);
  const T *x = static_cast<const T *>(p.x);
  int xt[2], xo[2];  // the token and the 8 columns that this thread stages
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xo[i] = ((i * kFewThreads + tid) >> (3 + r.lt)) * 8;
    xt[i] = (i * kFewThreads + tid) & (tp - 1);
  }
  for (int u = blockIdx.x; u < r.groups * r.slices; u += gridDim.x) {
    const int s = (int)r.by_group(u), g = u - s * r.groups;
    const int k0 = s * r.rows_per_slice, k1 = min(p.d, k0 + r.rows_per_slice);
    const int col0 = g << r.lcw;
    float acc[8] = {};
    float wv[8], xv[2][8];
    // The next 64 rows are in flight while these are multiplied.
    auto fetch = [&](int kb) {
      const int n = min(kRtRows, k1 - kb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = i * kFewThreads + tid, kk = at >> r.lcw, col = col0 + (at & (cw - 1));
        wv[i] = 0.f;
        if (kk < n && col < r.NC)
          wv[i] = col < p.E ? p.Wg[(size_t)(kb + kk) * p.E + col]
                            : p.Wn[(size_t)(kb + kk) * p.E + col - p.E];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (xt[i] < p.T && xo[i] < n) {
          few_x8<T>(x + (size_t)xt[i] * p.d, p.d, kb + xo[i], xv[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) xv[i][j] = 0.f;
        }
      }
    };
    fetch(k0);
    for (int kb = k0; kb < k1; kb += kRtRows) {
      const int n = min(kRtRows, k1 - kb);
      __syncthreads();  // the previous rows have been used
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = i * kFewThreads + tid;
        if (at < kRtRows * cw) ws[at] = wv[i];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (xo[i] < kRtRows)
#pragma unroll
          for (int j = 0; j < 8; ++j) xs[(xo[i] + j) * tp + xt[i]] = xv[i][j];
      __syncthreads();
      if (kb + kRtRows < k1) fetch(kb + kRtRows);
      if (tgi * 8 < p.T) {
#pragma unroll 4
        for (int kk = kp * lrows + lr; kk < n; kk += ks * lrows) {
          const float w = ws[kk * cw + lc];
          const float4 a = *reinterpret_cast<const float4 *>(xs + kk * tp + tgi * 8);
          const float4 b = *reinterpret_cast<const float4 *>(xs + kk * tp + tgi * 8 + 4);
          acc[0] = fmaf(w, a.x, acc[0]);
          acc[1] = fmaf(w, a.y, acc[1]);
          acc[2] = fmaf(w, a.z, acc[2]);
          acc[3] = fmaf(w, a.w, acc[3]);
          acc[4] = fmaf(w, b.x, acc[4]);
          acc[5] = fmaf(w, b.y, acc[5]);
          acc[6] = fmaf(w, b.z, acc[6]);
          acc[7] = fmaf(w, b.w, acc[7]);
        }
      }
    }
    // Over the lanes' rows, then over the warps of the same tokens.
#pragma unroll
    for (int t = 0; t < 8; ++t)
      for (int o = cw; o < 32; o <<= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
    if (lr == 0)
#pragma unroll
      for (int t = 0; t < 8; ++t) red[(warp * 8 + t) * 32 + lc] = acc[t];
    __syncthreads();
    for (int i = tid; i < tp * cw; i += kFewThreads) {
      const int t = i >> r.lcw, c = i & (cw - 1), col = col0 + c;
      if (t >= p.T || col >= r.NC) continue;
      float v = 0.f;
      for (int w = 0; w < ks; ++w) v += red[((w * tgp + t / 8) * 8 + t % 8) * 32 + c];
      p.rpart[((size_t)s * p.T + t) * r.NC + col] = v;
    }
  }
}

__device__ __forceinline__ void few_mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// bf16 x: a weight is the sum of three bf16 numbers (exact from 2^-110 on, below
// that within 2^-134), so three bf16 products with fp32 accumulation give the
// fp32 product. The CUDA-core form above is bound by its shared-memory reads (9
// for 8 multiply-adds: 8 us for 40 tokens and 1024 columns); here a 16-row step
// takes 28 for the whole block's 64 tokens x 16 columns. The products are too
// small and the weights too few for tcgen05's operands (they would first have to
// be split into memory).
// Warps: 4 steps of 16 rows x 2 halves of the columns; joined in shared memory.
// smem: xs bf16 [tokens][72], w bf16 [3][cw][72] (rows of 64 with a pad that
// spreads the fragments' reads over the banks); then red [4][tokens][cw] floats.
__device__ __forceinline__ void few_route_bf16(const FewArgs &p, float *smem) {
  const FewRouter &r = p.rt;
  const int tp = 8 << r.lt, mt = tp >> 4, cw = 1 << r.lcw, nt = cw >> 3;
  constexpr int P = 36;  // 32-bit words of a staged row
  uint32_t *xs = reinterpret_cast<uint32_t *>(smem), *ws = xs + tp * P;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int step = warp & 3, nh = warp >> 2, g = lane >> 2, q = lane & 3;
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x);
  int xt[2], xo[2];  // the token and the 8 columns that this thread stages
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xo[i] = ((i * kFewThreads + tid) >> (3 + r.lt)) * 8;
    xt[i] = (i * kFewThreads + tid) & (tp - 1);
  }
  for (int u = blockIdx.x; u < r.groups * r.slices; u += gridDim.x) {
    const int s = (int)r.by_group(u), gr = u - s * r.groups;
    const int k0 = s * r.rows_per_slice, k1 = min(p.d, k0 + r.rows_per_slice);
    const int col0 = gr << r.lcw;
    float acc[4][2][4] = {};
    float wv[4][2], xv[2][8];
    // The next 64 rows are in flight while these are multiplied.
    auto fetch = [&](int kb) {
      const int n = min(kRtRows, k1 - kb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = i * kFewThreads + tid, kk = (at >> r.lcw) * 2, col = col0 + (at & (cw - 1));
        const float *w = col < p.E ? p.Wg + col : p.Wn + col - p.E;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          wv[i][j] = kk + j < n && col < r.NC ? w[(size_t)(kb + kk + j) * p.E] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (xt[i] < p.T && xo[i] < n) {
          few_x8(x + (size_t)xt[i] * p.d, p.d, kb + xo[i], xv[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) xv[i][j] = 0.f;
        }
      }
    };
    fetch(k0);
    for (int kb = k0; kb < k1; kb += kRtRows) {
      __syncthreads();  // the previous rows have been used
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = i * kFewThreads + tid;
        if (at >= (kRtRows / 2) << r.lcw) break;
        uint32_t *dst = ws + (at & (cw - 1)) * P + (at >> r.lcw);
        float a = wv[i][0], b = wv[i][1];
#pragma unroll
        for (int z = 0; z < 3; ++z) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
          const uint32_t u = z ? *reinterpret_cast<const uint32_t *>(&h) : bf16x2_finite(a, b);
          dst[z * cw * P] = u;
          a -= __uint_as_float(u << 16);
          b -= __uint_as_float(u & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (xo[i] < kRtRows) {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // Exact: x is bf16.
            const __nv_bfloat162 h = __floats2bfloat162_rn(xv[i][2 * j], xv[i][2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t *>(&h);
          }
          *reinterpret_cast<uint4 *>(xs + xt[i] * P + xo[i] / 2) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      __syncthreads();
      if (kb + kRtRows < k1) fetch(kb + kRtRows);
      if (nh < nt) {
        uint32_t b[2][3][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if (nh + 2 * n >= nt) break;
#pragma unroll
          for (int z = 0; z < 3; ++z) {
            const uint32_t *w = ws + (z * cw + (nh + 2 * n) * 8 + g) * P + step * 8 + q;
            b[n][z][0] = w[0];
            b[n][z][1] = w[4];
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          if (m >= mt) break;
          const uint32_t *at = xs + (m * 16 + g) * P + step * 8 + q;
          const uint32_t a[4] = {at[0], at[8 * P], at[4], at[8 * P + 4]};
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (nh + 2 * n >= nt) break;
#pragma unroll
            for (int z = 2; z >= 0; --z) few_mma16816(acc[m][n], a, b[n][z][0], b[n][z][1]);
          }
        }
      }
    }
    __syncthreads();  // the staged rows have been used: red takes their place
    float *red = smem;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      if (m >= mt) break;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        if (nh + 2 * n >= nt) break;
        float *o = red + ((step * tp + m * 16 + g) << r.lcw) + (nh + 2 * n) * 8 + q * 2;
        o[0] = acc[m][n][0];
        o[1] = acc[m][n][1];
        o[8 << r.lcw] = acc[m][n][2];
        o[(8 << r.lcw) + 1] = acc[m][n][3];
      }
    }
    __syncthreads();
    for (int i = tid; i < tp << r.lcw; i += kFewThreads) {
      const int t = i >> r.lcw, col = col0 + (i & (cw - 1));
      if (t >= p.T || col >= r.NC) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) v += red[(w * tp << r.lcw) + i];
      p.rpart[((size_t)s * p.T + t) * r.NC + col] = v;
    }
  }
}

template <typename T>
__device__ __forceinline__ void few_route(const FewArgs &p, float *smem) {
  if constexpr (sizeof(T) == 2)
    few_route_bf16(p, smem);
  else
    few_route_f32<T>(p, smem);
}

// ----------------------------------------------------------------------------- selection
__device__ __forceinline__ float few_softplus(float z) {
  return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
}

// A float's order as an unsigned number; NaN is lowest.
__device__ __forceinline__ uint32_t few_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return isnan(v) ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Block reduction of a float over 256 threads (red: 8 floats of shared memory).
template <bool MAX>
__device__ __forceinline__ float few_block(float v, float *red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) v = MAX ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

// The choices of a single token, which every block selects for itself.
struct FewAlone {
  int32_t idx[16];
  float gate[16];
};

// One block per token t (a single token: every block, into `alone`, which saves
// the barrier between this and the rows: 94.0 -> 92.0 us for the large-expert
// layer's token): sums the router's slices in order, then
//   top-k:     the k largest H (lower index on ties), softmax over them;
//   Switch:    the largest, its gate from the softmax over all experts;
//   threshold: the experts with Softmax(H) > thr, in order, renormalised.
// A NaN logit ranks last; a non-finite one is recorded.
// smem: H [E] floats, red [8], taken words [32], sums [2][256], in whose place
// then the candidates [128] (64 bits each) and the chosen [16].
template <typename T>
__device__ __forceinline__ void few_select(const FewArgs &p, float *smem, FewAlone &alone) {
  const FewRouter &r = p.rt;
  float *H = smem;
  float *red = smem + (p.E + 1) / 2 * 2;  // what follows is 8-byte aligned
  uint32_t *words = reinterpret_cast<uint32_t *>(red + 8);
  float *sums = red + 40;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Threads side by side over the experts, the rest over the slices.
  const int lpe = min(8, 32 - __clz(p.E - 1)), pe = 1 << lpe;
  const int nl = kFewThreads >> lpe, sl = tid >> lpe;
  const bool single = p.T == 1, tell = !single || blockIdx.x == 0;
  for (int t = single ? 0 : blockIdx.x; t < p.T; t += gridDim.x) {
    float mx = -INFINITY;
    __syncthreads();
    // Up to four experts a thread, four slices at a time, all the loads of a
    // round in flight together (places past the end read the first one).
    float c[4] = {}, z[4] = {}, add[4] = {}, noise[4] = {}, thr[4] = {};
    const int e0 = tid & (pe - 1);
    const float *q = p.rpart + (size_t)t * r.NC;
    const size_t step = (size_t)p.T * r.NC;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i * pe;
      if (sl == 0 && e < p.E) {
        if (p.bias) add[i] = p.bias[e];
        if (p.Wn) noise[i] = p.noise[(size_t)t * p.E + e];
      }
      if (p.mode == kFewThreshold && i * kFewThreads + tid < p.E)
        thr[i] = p.thr[i * kFewThreads + tid];
    }
    for (int s0 = sl; s0 < r.slices; s0 += 4 * nl) {
      float vc[4][4], vz[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i * pe >= p.E) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = e0 + i * pe, s = s0 + j * nl;
          const float *at = q + (s < r.slices ? s * step : 0) + (e < p.E ? e : 0);
          vc[i][j] = __ldcg(at);
          if (p.Wn) vz[i][j] = __ldcg(at + p.E);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i * pe >= p.E) break;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (s0 + j * nl < r.slices) {
            c[i] += vc[i][j];
            if (p.Wn) z[i] += vz[i][j];
          }
      }
    }
    if (nl > 1) {  // then E <= 128: one expert a thread
      sums[tid] = c[0];
      sums[kFewThreads + tid] = z[0];
      __syncthreads();
      if (sl == 0) {
        float cs = 0.f, zs = 0.f;
#pragma unroll 8
        for (int i = 0; i < nl; ++i) {
          cs += sums[i * pe + tid];
          zs += sums[kFewThreads + i * pe + tid];
        }
        c[0] = cs;
        z[0] = zs;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + i * pe;
      if (sl != 0 || e >= p.E) continue;
      float h = c[i] + add[i];
      if (p.Wn) h = fmaf(noise[i], few_softplus(z[i]), h);
      if (!isfinite(h)) record_error(p.st, MOE_ERR_NONFINITE, (long long)t * p.E + e);
      H[e] = h;
      mx = fmaxf(mx, h);
    }
    const auto put = [&](int j, int e, float g) {  // choice j of the token
      if (single) {
        alone.idx[j] = e;
        alone.gate[j] = g;
      }
      if (tell) {
        p.idx[(size_t)t * p.k + j] = e;
        p.gate[(size_t)t * p.k + j] = g;
      }
    };
    float se = 0.f;
    if (p.mode != kFewTopk) {
      mx = few_block<true>(mx, red);
      for (int e = tid; e < p.E; e += kFewThreads) {
        const float v = expf(H[e] - mx);
        if (p.mode == kFewThreshold) H[e] = v;
        se += v;
      }
      se = few_block<false>(se, red);
    }
    __syncthreads();
    if (p.mode == kFewThreshold) {
      const int nw = (p.E + 31) / 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int w = i * 8 + warp, e = i * kFewThreads + tid;
        if (w >= nw) break;
        const float P = e < p.E ? H[e] / se : 0.f;
        const uint32_t b = __ballot_sync(0xffffffffu, e < p.E && P > thr[i]);
        if (e < p.E) H[e] = P;
        if (lane == 0) {
          words[w] = b;
          if (p.mask && tell) p.mask[(size_t)t * nw + w] = b;
        }
      }
      __syncthreads();
      if (warp == 0) {
        // Picks before this lane's word, then each pick at its place.
        const uint32_t mine = lane < nw ? words[lane] : 0u;
        int incl = __popc(mine);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const int total = __shfl_sync(0xffffffffu, incl, 31);
        int at = incl - __popc(mine);
        float sum = 0.f;
        for (uint32_t b = mine; b; b &= b - 1)
          sum += H[lane * 32 + __ffs(b) - 1];
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        for (uint32_t b = mine; b; b &= b - 1, ++at) {
          if (at >= p.k) break;
          const int e = lane * 32 + __ffs(b) - 1;
          put(at, e, H[e] / sum);
        }
        for (int j = total + lane; j < p.k; j += 32) put(j, p.E, 0.f);
        if (total > p.k && lane == 0) record_error(p.st, MOE_ERR_BOUNDS, t);
      }
    } else if (p.mode == kFewSwitch) {
      if (warp == 0) {
        int e = 0x7fffffff;
        for (int i = lane; i < p.E && e >= p.E; i += 32)
          if (H[i] == mx) e = i;
        e = __reduce_min_sync(0xffffffffu, e);
        if (lane == 0) put(0, e < p.E ? e : 0, 1.f / se);
      }
    } else {
      // Candidates, each ranked by one thread that counts those before it (a
      // larger key, or the same and a lower index). Up to 128 experts are all
      // candidates (three instructions each, where a pick below is some 300
      // cycles); of more, every warp picks the k best of its own by two integer
      // reductions a pick: the largest key, then the lowest index that has it.
      unsigned long long *cand = reinterpret_cast<unsigned long long *>(sums);
      int *chosen = reinterpret_cast<int *>(cand + 128), nc = p.E;
      const auto rank = [](uint32_t key, int e) {  // one number to compare
        return (unsigned long long)key << 32 | (uint32_t)~e;
      };
      if (p.E <= min(128, 64 * p.k)) {
        if (tid < p.E) cand[tid] = rank(few_key(H[tid]), tid);
      } else {
        constexpr int kNone = 0x7fffffff;
        uint32_t key[4];
        int left = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = i * kFewThreads + tid;
          key[i] = e < p.E ? few_key(H[e]) : 0u;
          left |= (e < p.E) << i;
        }
        nc = 8 * p.k;
        for (int j = 0; j < p.k; ++j) {
          uint32_t lk = 0;
          int li = kNone;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((left >> i & 1) && (li == kNone || key[i] > lk)) {
              lk = key[i];
              li = i * kFewThreads + tid;
            }
          const uint32_t best = __reduce_max_sync(0xffffffffu, lk);
          const int e = __reduce_min_sync(0xffffffffu, lk == best ? li : kNone);
          if (e == li && e != kNone) left &= ~(1 << (e / kFewThreads));
          if (lane == 0) cand[warp * p.k + j] = rank(best, e);  // kNone: behind every expert
        }
      }
      __syncthreads();
      if (tid < nc) {
        const unsigned long long mine = cand[tid];
        int before = 0;
        for (int c0 = 0; c0 < nc; c0 += 8) {  // past nc: other words of sums, not counted
#pragma unroll
          for (int c = 0; c < 8; ++c) before += (cand[c0 + c] > mine) & (c0 + c < nc);
        }
        if (before < p.k) chosen[before] = (int)~(uint32_t)mine;
      }
      __syncthreads();
      if (warp != 0) continue;
      const int mine = lane < p.k ? chosen[lane] : 0;
      const float v = lane < p.k ? H[mine] : -INFINITY;
      const float top = __shfl_sync(0xffffffffu, v, 0);  // every lane takes part
      const float w = lane < p.k ? expf(v - top) : 0.f;
      float sum = w;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane < p.k) put(lane, mine, w / sum);
    }
  }
}

// ----------------------------------------------------------------------------- rows of the experts
// Every block derives, from the choices, what each needs: the experts in use
// (ascending), their packed rows (token order, under capacity) and each row's
// token. A token picks an expert at most once, so a choice's slot is the
// number of earlier tokens in the expert's 64-bit mask.
struct FewRows {
  unsigned long long *tokens;  // [E] tokens of each expert (bit t)
  int *expert;                 // [<= kFewRows] experts in use
  int *first;                  // [<= kFewRows + 1] their first packed row
  int *base;                   // [E] first packed row of every expert
  int16_t *place;              // [E] its place in `expert`
  uint16_t *owner;             // [<= kFewRows] each packed row's place in `expert`
  int16_t *row;                // [T k] packed row of each choice, or -1
  float *gate;                 // [T k]
  uint8_t *token;              // [<= kFewRows] token of each packed row
  int n, rows;                 // experts in use; rows
};
constexpr size_t few_rows_bytes(int E, int A) {
  return ((size_t)E * 14 + ((size_t)2 * A + 2) * 4 + (size_t)A * 9 + 63) / 64 * 64;
}

__device__ FewRows few_rows(const FewArgs &p, char *smem, const FewAlone &alone) {
  FewRows R;
  R.tokens = reinterpret_cast<unsigned long long *>(smem);
  R.base = reinterpret_cast<int *>(R.tokens + p.E);
  R.expert = R.base + p.E;
  const int A = p.T * p.k;
  R.first = R.expert + A;
  R.gate = reinterpret_cast<float *>(R.first + A + 1);
  R.owner = reinterpret_cast<uint16_t *>(R.gate + A);
  R.row = reinterpret_cast<int16_t *>(R.owner + A);
  R.place = R.row + A;
  R.token = reinterpret_cast<uint8_t *>(R.place + p.E);
  __shared__ int scan[8][2], total[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.T == 1) {
    // A single token: each pick is kept, in a row of its own; sorted by every
    // warp's lanes, without the sums over the experts (1.5 -> 0.6 us).
    const int e = lane < A ? alone.idx[lane] : p.E;
    const uint32_t some = __ballot_sync(0xffffffffu, e < p.E);
    int at = 0;
    for (int a = 0; a < A; ++a) at += __shfl_sync(0xffffffffu, e, a) < e;
    R.n = R.rows = __popc(some);
    if (warp == 0 && lane < A) {
      const bool kept = e < p.E;
      R.gate[lane] = alone.gate[lane];
      R.row[lane] = kept ? (int16_t)at : (int16_t)-1;
      if (kept) {
        R.expert[at] = e;
        R.owner[at] = (uint16_t)at;
        R.token[at] = 0;
      }
      if (blockIdx.x == 0) {
        if (p.pos) p.pos[lane] = kept ? 0 : -1;
        if (p.keep) p.keep[lane] = kept;
      }
    }
    if (tid <= A) R.first[tid] = min(tid, R.n);
    __syncthreads();
    return R;
  }
  int choice[kFewRows / kFewThreads];
#pragma unroll
  for (int i = 0; i < kFewRows / kFewThreads; ++i) {
    const int a = i * kFewThreads + tid;
    choice[i] = -1;
    if (a < A) {
      choice[i] = p.idx[a];
      R.gate[a] = p.gate[a];
    }
  }
  for (int e = tid; e < p.E; e += kFewThreads) R.tokens[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kFewRows / kFewThreads; ++i)
    if (choice[i] >= 0 && choice[i] < p.E) {
      const int t = (int)p.by_k(i * kFewThreads + tid);  // 32-bit halves: one native atomic each
      atomicOr(reinterpret_cast<uint32_t *>(&R.tokens[choice[i]]) + (t >> 5), 1u << (t & 31));
    }
  __syncthreads();
  // Exclusive sums over the experts of (in use, rows), 4 experts a thread.
  int use = 0, rows = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = tid * 4 + q;
    const int n = e < p.E ? min(p.C, __popcll(R.tokens[e])) : 0;
    use += n > 0;
    rows += n;
  }
  int iu = use, ir = rows;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, iu, o), b = __shfl_up_sync(0xffffffffu, ir, o);
    if (lane >= o) {
      iu += a;
      ir += b;
    }
  }
  if (lane == 31) {
    scan[warp][0] = iu;
    scan[warp][1] = ir;
  }
  __syncthreads();
  int bu = iu - use, br = ir - rows;
  for (int w = 0; w < warp; ++w) {
    bu += scan[w][0];
    br += scan[w][1];
  }
  if (tid == kFewThreads - 1) {
    total[0] = bu + use;
    total[1] = br + rows;
    R.first[bu + use] = br + rows;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = tid * 4 + q;
    if (e >= p.E) break;
    const int n = min(p.C, __popcll(R.tokens[e]));
    R.base[e] = br;
    if (n > 0) {
      R.expert[bu] = e;
      R.first[bu] = br;
      R.place[e] = (int16_t)bu;
      ++bu;
      br += n;
    }
  }
  __syncthreads();
  R.n = total[0];
  R.rows = total[1];
#pragma unroll
  for (int i = 0; i < kFewRows / kFewThreads; ++i) {
    const int a = i * kFewThreads + tid, e = choice[i], t = (int)p.by_k(a);
    if (a >= A) break;
    const bool some = e >= 0 && e < p.E;
    const int pos = some ? __popcll(R.tokens[e] & ((1ull << t) - 1)) : -1;
    const bool kept = some && pos < p.C;
    R.row[a] = kept ? (int16_t)(R.base[e] + pos) : (int16_t)-1;
    if (kept) {
      R.token[R.base[e] + pos] = (uint8_t)t;
      R.owner[R.base[e] + pos] = (uint16_t)R.place[e];
    }
    if (blockIdx.x == 0) {
      if (p.pos) p.pos[a] = pos;
      if (p.keep) p.keep[a] = kept;
    }
  }
  __syncthreads();
  return R;
}

// ----------------------------------------------------------------------------- combine
// V floats at p (aligned to V floats), written by other blocks, from L2; zero
// unless `some`. Predicated: behind a branch each would be waited for before the
// next is asked for.
template <int V>
__device__ __forceinline__ void few_get(const float *p, bool some, float (&v)[V]) {
  if constexpr (V == 4) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.f32 %0, 0f00000000;\n"
        " mov.f32 %1, 0f00000000;\n mov.f32 %2, 0f00000000;\n mov.f32 %3, 0f00000000;\n"
        " @p ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n}\n"
        : "=&f"(v[0]), "=&f"(v[1]), "=&f"(v[2]), "=&f"(v[3])
        : "l"(p), "r"((uint32_t)some));
  } else if constexpr (V == 2) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %3, 0;\n mov.f32 %0, 0f00000000;\n"
        " mov.f32 %1, 0f00000000;\n @p ld.global.cg.v2.f32 {%0, %1}, [%2];\n}\n"
        : "=&f"(v[0]), "=&f"(v[1])
        : "l"(p), "r"((uint32_t)some));
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n mov.f32 %0, 0f00000000;\n"
        " @p ld.global.cg.f32 %0, [%1];\n}\n"
        : "=&f"(v[0])
        : "l"(p), "r"((uint32_t)some));
  }
}
template <typename T, int V>
__device__ __forceinline__ void few_ld(const T *p, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = few_f(p[i]);
}
template <typename T, int V>
__device__ __forceinline__ void few_st(T *p, const float (&v)[V]) {
  struct alignas(sizeof(T) * V) Pack {
    T t[V];
  } o;
#pragma unroll
  for (int i = 0; i < V; ++i) o.t[i] = few_t<T>(v[i]);
  *reinterpret_cast<Pack *>(p) = o;
}

template <int Q_, int S_>
struct FewRound {
  static constexpr int Q = Q_, S = S_;
};

// y[t] = x[t] + sum over the kept choices, in order, of gate * (sum of the
// partial sums + b2), in fp32, rounded once. V columns a thread; where that
// leaves most threads idle (few tokens, whose partials are many), 8 lanes share
// the same columns' choices and their partials, joined in a fixed order.
// The last barrier is inside, after what does not depend on it.
template <typename T, int V, typename PF>
__device__ __forceinline__ void few_combine(const FewArgs &p, const FewRows &R,
                                            const PF &pieces) {
  const T *x = static_cast<const T *>(p.x), *b2 = static_cast<const T *>(p.b2);
  T *y = static_cast<T *>(p.y);
  const unsigned cols = p.d / V, total = p.T * cols;
  const size_t step = (size_t)R.rows * p.d;
  const FixedDiv by = V == 4 ? p.by_d4 : FixedDiv(cols);
  const int K = p.T == 1 ? R.n : p.k;  // a single token's picks are its first choices
  // Token t's columns c .. c + V - 1: every dq-th choice from q0 on, Q at a time,
  // of its partials every ds-th from s0 on, S at a time.
  const auto add = [&](auto rounds, unsigned t, unsigned c, int q0, int dq, int s0, int ds,
                       bool live, float (&acc)[V]) {
    constexpr int Q = decltype(rounds)::Q, S = decltype(rounds)::S;
    for (int qb = q0; qb < K; qb += Q * dq) {
      float v[Q][V] = {};
      int row[Q], np[Q], most = 0;
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        const int q = qb + i * dq;
        row[i] = live && q < K ? R.row[t * p.k + q] : -1;
        np[i] = row[i] >= 0 ? pieces(R.owner[row[i]], (int)c) : 0;
        most = max(most, np[i]);
        if (b2 && s0 == 0 && row[i] >= 0)
          few_ld<T, V>(b2 + (size_t)R.expert[R.owner[row[i]]] * p.d + c, v[i]);
      }
      for (int sb = s0; sb < most; sb += S * ds) {
        float w[S][Q][V];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < Q; ++i)
            few_get<V>(p.zpart + (sb + s * ds) * step + (size_t)row[i] * p.d + c,
                       sb + s * ds < np[i], w[s][i]);
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int i = 0; i < Q; ++i)
#pragma unroll
            for (int z = 0; z < V; ++z) v[i][z] += w[s][i][z];
      }
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        if (row[i] < 0) continue;
        const float g = R.gate[t * p.k + qb + i * dq];
#pragma unroll
        for (int z = 0; z < V; ++z) acc[z] = fmaf(g, v[i][z], acc[z]);
      }
    }
  };
  const auto store = [&](unsigned t, unsigned c, const float (&acc)[V]) {
    bool bad = false;
#pragma unroll
    for (int z = 0; z < V; ++z) bad |= !isfinite(acc[z]);
    if (bad) record_error(p.st, MOE_ERR_NONFINITE, t);
    few_st<T, V>(y + (size_t)t * p.d + c, acc);
  };
  const unsigned first = blockIdx.x * kFewThreads + threadIdx.x, stride = gridDim.x * kFewThreads;
  if (total * 8 <= stride) {
    const unsigned i = first >> 3, sub = first & 7;
    const bool live = i < total;
    const unsigned t = live ? by(i) : 0, c = live ? (i - t * cols) * V : 0;
    // Lanes over the choices that a token keeps on average, the rest over their
    // partials.
    const int lk = R.rows > 4 * p.T ? 3 : R.rows > 2 * p.T ? 2 : R.rows > p.T ? 1 : 0;
    float acc[V] = {};
    if (live && sub == 0) few_ld<T, V>(x + (size_t)t * p.d + c, acc);
    if (!few_barrier(p, kFewBarriers - 1)) return;
    if (first - (threadIdx.x & 31) >= total * 8) return;  // whole warps leave
    add(FewRound<1, 4>{}, t, c, sub & ((1 << lk) - 1), 1 << lk, (int)sub >> lk,
        8 >> lk, live, acc);
#pragma unroll
    for (int z = 0; z < V; ++z)
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) acc[z] += __shfl_xor_sync(0xffffffffu, acc[z], o);
    if (live && sub == 0) store(t, c, acc);
    return;
  }
  if (!few_barrier(p, kFewBarriers - 1)) return;
  for (unsigned i = first; i < total; i += stride) {
    const unsigned t = by(i), c = (i - t * cols) * V;
    float acc[V];
    few_ld<T, V>(x + (size_t)t * p.d + c, acc);
    add(FewRound<4, 2>{}, t, c, 0, 1, 0, 1, true, acc);
    store(t, c, acc);
  }
}

}  // namespace

// Launches a kernel of one cooperative grid of kFewThreads-thread blocks; no
// launch of it takes more than `most` of dynamic shared memory.
cudaError_t launch_few_grid(const void *kernel, void **args, int grid, size_t smem, size_t most,
                            cudaStream_t s);
// k_few_tc.cu: bf16 layers whose widths are multiples of 8, experts on tcgen05.
inline bool few_on_tc(const moe_config &c) {
  return c.act_dtype == MOE_BF16 && c.d % 8 == 0 && c.d_ff % 8 == 0;
}
int few_tc_tiles(const moe_config &cfg);  // layer 1's tiles at most
cudaError_t launch_few_tc(const FewArgs &p, cudaStream_t s);

}  // namespace moe
