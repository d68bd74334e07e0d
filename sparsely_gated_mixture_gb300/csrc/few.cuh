// The few-token layer (moe_forward_few, moe_forward_threshold_few): arguments
// of its kernels, the barrier between its phases, and the phases that both
// forms of the experts share. Internal to libmoe.so.
//
// One persistent cooperative grid runs the whole layer for T <= 64 tokens:
//   router     partial sums of x W_g (and x W_noise) over slices of d
//   selection  one block per token: logits, top-k or threshold mask, gates
//   (every block then derives the capacity's slots and the experts' rows)
//   layer 1    partial sums of x W1 over slices of d, for the experts in use
//   hidden     H = ReLU(sum + b1), rounded to the layer's type
//   layer 2    partial sums of H W2 over slices of d_ff
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
constexpr int kFewMaxGrid = 512;   // blocks at most (sizes the partial buffers)
constexpr int kFewBarriers = 5;
constexpr int kFewColsMax = 256;   // columns of one unit of the experts' products at most
enum FewMode { kFewTopk = 0, kFewSwitch = 1, kFewThreshold = 2 };

struct FewArgs {
  int T, d, E, F, k, C, mode;
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
  unsigned long long *flags;  // [kFewBarriers][kFewMaxGrid]
  float *rpart;               // router partials [slices][T][columns]
  float *hpart, *zpart;       // partials of the layers [slices][rows][N]
  void *h;                    // [rows, F], the layer's type
  unsigned long long nonce, wait_ns;
};

namespace {

// ----------------------------------------------------------------------------- grid barrier
// Every block has one flag per barrier; it arrives by storing the launch's
// nonce there and waits until all blocks' flags hold it: one hop, where a
// shared counter would take one atomic per block in turn. The workspace need
// not be zeroed: flags of an earlier call hold another nonce, and for a
// replayed graph, whose nonce is the same each time, the flags are cleared:
// a block clears its flags of the barriers after the first before it arrives
// at the first (no block looks at them earlier), and its flag of the first
// once it has passed the second (every block has passed the first by then).
// Waits are bounded: past the limit the block records MOE_ERR_TIMEOUT and
// leaves, and so does, within the limit, every block that waits for it.
__device__ __forceinline__ void few_flag_set(unsigned long long *f, unsigned long long v) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(f), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long few_flag_get(const unsigned long long *f) {
  unsigned long long v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(f) : "memory");
  return v;
}

__device__ __forceinline__ void few_start(const FewArgs &p) {
  if (threadIdx.x == 0) {
    for (int b = 1; b < kFewBarriers; ++b)
      p.flags[(size_t)b * kFewMaxGrid + blockIdx.x] = 0;
    if (blockIdx.x == 0) *p.st = DeviceStatus{};
  }
}

// Arrive at barrier b (one thread, after a barrier of the block's threads that
// wrote): what they wrote before is visible to a block that has waited.
__device__ __forceinline__ void few_arrive(const FewArgs &p, int b) {
  __threadfence();
  few_flag_set(p.flags + (size_t)b * kFewMaxGrid + blockIdx.x, p.nonce);
}

// Wait for barrier b (threads tid of n_threads of the block); false: leave the
// kernel. With an abort flag, a set one ends the wait too.
__device__ __forceinline__ bool few_wait(const FewArgs &p, int b, int tid, int n_threads,
                                         volatile int *abort_flag = nullptr) {
  bool ok = true;
  unsigned long long t0 = 0;
  for (int i = tid; i < (int)gridDim.x && ok; i += n_threads) {
    const unsigned long long *f = p.flags + (size_t)b * kFewMaxGrid + i;
    while (few_flag_get(f) != p.nonce) {
      const unsigned long long now = globaltimer();
      if (t0 == 0) t0 = now;
      if (abort_flag && *abort_flag) {
        ok = false;
        break;
      }
      if (now - t0 >= p.wait_ns) {
        record_error(p.st, MOE_ERR_TIMEOUT, 100 + b);
        ok = false;
        break;
      }
    }
  }
  return ok;
}

__device__ __forceinline__ bool few_barrier(const FewArgs &p, int b) {
  __syncthreads();
  if (threadIdx.x == 0) few_arrive(p, b);
  const bool ok = few_wait(p, b, threadIdx.x, blockDim.x);
  const bool fail = __syncthreads_or(!ok);
  if (threadIdx.x == 0 && (b == 1 || fail))
    p.flags[blockIdx.x] = 0;
  return !fail;
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
// Columns: E of W_g, then E of W_noise. A unit is 32 columns (or the next
// power of two over their number, the warp's lanes then also covering rows)
// and one slice of d; the block's warps share the slice's rows, each thread
// holding the sums of 8 tokens in registers, and are summed in shared memory.
constexpr int kRtRows = 128;  // rows of x staged at a time

struct FewRouter {
  int NC, cw, groups, slices, rows_per_slice;
};
__host__ __device__ inline FewRouter few_router(int d, int E, bool noisy, int grid) {
  FewRouter r;
  r.NC = noisy ? 2 * E : E;
  r.cw = 1;
  while (r.cw < 32 && r.cw < r.NC) r.cw *= 2;
  r.groups = (r.NC + r.cw - 1) / r.cw;
  int s = (grid + r.groups - 1) / r.groups;
  const int most = (d + 31) / 32;  // slices of at least 32 rows
  if (s > most) s = most;
  r.rows_per_slice = (d + s - 1) / s;
  r.slices = (d + r.rows_per_slice - 1) / r.rows_per_slice;
  return r;
}

// smem: xs [kRtRows][8] floats, red [8 warps][8][32] floats (12 KB).
template <typename T>
__device__ void few_route(const FewArgs &p, float *smem) {
  const FewRouter r = few_router(p.d, p.E, p.Wn != nullptr, gridDim.x);
  float *xs = smem;
  float *red = smem + kRtRows * 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lr = lane / r.cw, lrows = 32 / r.cw;  // this lane's row among the warp's
  const T *x = static_cast<const T *>(p.x);
  for (int u = blockIdx.x; u < r.groups * r.slices; u += gridDim.x) {
    const int g = u % r.groups, s = u / r.groups;
    const int k0 = s * r.rows_per_slice, k1 = min(p.d, k0 + r.rows_per_slice);
    const int col = g * r.cw + (lane & (r.cw - 1));
    const float *W = nullptr;
    if (col < p.E) W = p.Wg + col;
    else if (col < r.NC) W = p.Wn + (col - p.E);
    for (int t0 = 0; t0 < p.T; t0 += 8) {
      float acc[8] = {};
      for (int kb = k0; kb < k1; kb += kRtRows) {
        const int n = min(kRtRows, k1 - kb);
        __syncthreads();
        for (int i = tid; i < 8 * n; i += kFewThreads) {
          const int t = i / n, kk = i - t * n;
          xs[kk * 8 + t] = t0 + t < p.T ? few_f(x[(size_t)(t0 + t) * p.d + kb + kk]) : 0.f;
        }
        __syncthreads();
        if (W) {
#pragma unroll 4
          for (int kk = warp * lrows + lr; kk < n; kk += 8 * lrows) {
            const float w = W[(size_t)(kb + kk) * p.E];
            const float4 a = *reinterpret_cast<const float4 *>(xs + kk * 8);
            const float4 b = *reinterpret_cast<const float4 *>(xs + kk * 8 + 4);
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
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 8; ++t) red[(warp * 8 + t) * 32 + lane] = acc[t];
      __syncthreads();
      // Thread (t, column): the sum over the warps and the lanes' rows.
      const int t = tid >> 5;
      if (lane < r.cw && t0 + t < p.T && col < r.NC) {
        float v = 0.f;
        for (int w = 0; w < 8; ++w)
          for (int q = 0; q < lrows; ++q) v += red[(w * 8 + t) * 32 + q * r.cw + lane];
        p.rpart[((size_t)s * p.T + t0 + t) * r.NC + col] = v;
      }
    }
  }
}

// ----------------------------------------------------------------------------- selection
__device__ __forceinline__ float few_softplus(float z) {
  return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
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

// One block per token t: sums the router's slices in order, then
//   top-k:     the k largest H (lower index on ties), softmax over them;
//   Switch:    the largest, its gate from the softmax over all experts;
//   threshold: the experts with Softmax(H) > thr, in order, renormalised.
// A NaN logit ranks last; a non-finite one is recorded.
// smem: H [E] floats, red [8], taken words [32].
template <typename T>
__device__ void few_select(const FewArgs &p, float *smem) {
  const FewRouter r = few_router(p.d, p.E, p.Wn != nullptr, gridDim.x);
  float *H = smem;
  float *red = smem + p.E;
  uint32_t *words = reinterpret_cast<uint32_t *>(red + 8);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
    float mx = -INFINITY;
    __syncthreads();
    for (int e = tid; e < p.E; e += kFewThreads) {
      const float *q = p.rpart + (size_t)t * r.NC + e;
      const size_t step = (size_t)p.T * r.NC;
      float c = 0.f, z = 0.f;
#pragma unroll 8
      for (int s = 0; s < r.slices; ++s) c += q[s * step];
      if (p.bias) c += p.bias[e];
      if (p.Wn) {
#pragma unroll 8
        for (int s = 0; s < r.slices; ++s) z += q[s * step + p.E];
        c = fmaf(p.noise[(size_t)t * p.E + e], few_softplus(z), c);
      }
      if (!isfinite(c)) record_error(p.st, MOE_ERR_NONFINITE, (long long)t * p.E + e);
      H[e] = c;
      mx = fmaxf(mx, c);
    }
    int32_t *oi = p.idx + (size_t)t * p.k;
    float *og = p.gate + (size_t)t * p.k;
    float se = 0.f;
    if (p.mode != kFewTopk) {
      mx = few_block<true>(mx, red);
      for (int e = tid; e < p.E; e += kFewThreads) se += expf(H[e] - mx);
      se = few_block<false>(se, red);
    }
    __syncthreads();
    if (p.mode == kFewThreshold) {
      const int nw = (p.E + 31) / 32;
      for (int w = warp; w < nw; w += 8) {
        const int e = w * 32 + lane;
        const bool take = e < p.E && expf(H[e] - mx) / se > p.thr[e];
        const uint32_t b = __ballot_sync(0xffffffffu, take);
        if (lane == 0) {
          words[w] = b;
          if (p.mask) p.mask[(size_t)t * nw + w] = b;
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
          sum += expf(H[lane * 32 + __ffs(b) - 1] - mx) / se;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        for (uint32_t b = mine; b; b &= b - 1, ++at) {
          if (at >= p.k) break;
          const int e = lane * 32 + __ffs(b) - 1;
          oi[at] = e;
          og[at] = expf(H[e] - mx) / se / sum;
        }
        for (int j = total + lane; j < p.k; j += 32) {
          oi[j] = p.E;
          og[j] = 0.f;
        }
        if (total > p.k && lane == 0) record_error(p.st, MOE_ERR_BOUNDS, t);
      }
    } else if (warp == 0) {
      // Lane l ranks experts l, l + 32, ...; `done` marks the chosen ones.
      uint32_t done = 0;
      float top = 0.f, g = 0.f, sum = 0.f;
      int mine = 0;
      for (int j = 0; j < p.k; ++j) {
        float bv = -INFINITY;
        int be = 0x7fffffff;
        for (int e = lane, q = 0; e < p.E; e += 32, ++q) {
          if ((done >> q) & 1u) continue;
          const float v = isnan(H[e]) ? -INFINITY : H[e];
          if (be == 0x7fffffff || v > bv) {
            bv = v;
            be = e;
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
          const int oe = __shfl_xor_sync(0xffffffffu, be, o);
          if (oe != 0x7fffffff && (be == 0x7fffffff || ov > bv || (ov == bv && oe < be))) {
            bv = ov;
            be = oe;
          }
        }
        if ((be & 31) == lane) done |= 1u << (be >> 5);
        if (j == 0) top = bv;
        const float w = expf(bv - top);
        sum += w;
        if (lane == j) {
          g = w;
          mine = be;
        }
      }
      if (lane < p.k) {
        oi[lane] = mine;
        og[lane] = p.mode == kFewSwitch ? 1.f / se : g / sum;
      }
    }
  }
}

// ----------------------------------------------------------------------------- rows of the experts
// Every block derives, from the choices, what each needs: the experts in use
// (ascending), their packed rows (token order, under capacity) and each row's
// token. A token picks an expert at most once, so a choice's slot is the
// number of earlier tokens in the expert's 64-bit mask.
struct FewRows {
  unsigned long long *tokens;  // [E] tokens of each expert
  int *expert;                 // [<= kFewRows] experts in use
  int *first;                  // [<= kFewRows + 1] their first packed row
  int *base;                   // [E] first packed row of every expert
  uint16_t *owner;             // [<= kFewRows] each packed row's place in `expert`
  uint8_t *token;              // [<= kFewRows] token of each packed row
  int n, rows;                 // experts in use; rows
};
constexpr size_t few_rows_bytes(int E, int A) {
  return ((size_t)E * 12 + ((size_t)2 * A + 2) * 4 + (size_t)A * 3 + 63) / 64 * 64;
}

__device__ FewRows few_rows(const FewArgs &p, char *smem) {
  FewRows R;
  R.tokens = reinterpret_cast<unsigned long long *>(smem);
  R.base = reinterpret_cast<int *>(R.tokens + p.E);
  R.expert = R.base + p.E;
  const int A = p.T * p.k;
  R.first = R.expert + A;
  R.owner = reinterpret_cast<uint16_t *>(R.first + A + 1);
  R.token = reinterpret_cast<uint8_t *>(R.owner + A);
  __shared__ int scan[8][2], total[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int e = tid; e < p.E; e += kFewThreads) R.tokens[e] = 0;
  __syncthreads();
  for (int a = tid; a < A; a += kFewThreads) {
    const int e = p.idx[a];
    if (e >= 0 && e < p.E) atomicOr(&R.tokens[e], 1ull << (a / p.k));
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
      for (int r = 0; r < n; ++r) R.owner[br + r] = (uint16_t)bu;
      ++bu;
      br += n;
    }
  }
  __syncthreads();
  R.n = total[0];
  R.rows = total[1];
  for (int a = tid; a < A; a += kFewThreads) {
    const int e = p.idx[a], t = a / p.k;
    const bool some = e >= 0 && e < p.E;
    const int pos = some ? __popcll(R.tokens[e] & ((1ull << t) - 1)) : -1;
    const bool kept = some && pos < p.C;
    if (kept) R.token[R.base[e] + pos] = (uint8_t)t;
    if (blockIdx.x == 0) {
      if (p.pos) p.pos[a] = pos;
      if (p.keep) p.keep[a] = kept;
    }
  }
  __syncthreads();
  return R;
}

// ----------------------------------------------------------------------------- hidden, combine
// V floats at p (aligned to V floats).
template <int V>
__device__ __forceinline__ void few_add(const float *p, float (&v)[V]) {
  if constexpr (V == 4) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    v[0] += f.x;
    v[1] += f.y;
    v[2] += f.z;
    v[3] += f.w;
  } else if constexpr (V == 2) {
    const float2 f = *reinterpret_cast<const float2 *>(p);
    v[0] += f.x;
    v[1] += f.y;
  } else {
    v[0] += *p;
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

// h[r] = ReLU(sum of the partial sums + b1), rounded once to the layer's
// type, V columns at a time, by threads tid of n_threads of each block.
// pieces(j, c): the number of partial sums of column c of expert j of R.
template <typename T, int V, typename PF>
__device__ __forceinline__ void few_hidden(const FewArgs &p, const FewRows &R, const PF &pieces,
                                           int tid, int n_threads) {
  const T *b1 = static_cast<const T *>(p.b1);
  T *h = static_cast<T *>(p.h);
  const unsigned cols = p.F / V, total = R.rows * cols;
  const size_t step = (size_t)R.rows * p.F;
  for (unsigned i = blockIdx.x * n_threads + tid; i < total; i += gridDim.x * n_threads) {
    const unsigned row = i / cols, c = (i - row * cols) * V;
    const int j = R.owner[row], np = pieces(j, (int)c);
    const float *src = p.hpart + (size_t)row * p.F + c;
    float v[V] = {};
#pragma unroll 4
    for (int s = 0; s < np; ++s) few_add<V>(src + s * step, v);
    if (b1) {
      float b[V];
      few_ld<T, V>(b1 + (size_t)R.expert[j] * p.F + c, b);
#pragma unroll
      for (int q = 0; q < V; ++q) v[q] += b[q];
    }
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = fmaxf(v[q], 0.f);
    few_st<T, V>(h + (size_t)row * p.F + c, v);
  }
}

// y[t] = x[t] + sum over the kept choices, in order, of gate * (sum of the
// partial sums + b2), in fp32, rounded once.
template <typename T, int V, typename PF>
__device__ __forceinline__ void few_combine(const FewArgs &p, const FewRows &R,
                                            const PF &pieces) {
  const T *x = static_cast<const T *>(p.x), *b2 = static_cast<const T *>(p.b2);
  T *y = static_cast<T *>(p.y);
  const unsigned cols = p.d / V, total = p.T * cols;
  const size_t step = (size_t)R.rows * p.d;
  for (unsigned i = blockIdx.x * kFewThreads + threadIdx.x; i < total;
       i += gridDim.x * kFewThreads) {
    const unsigned t = i / cols, c = (i - t * cols) * V;
    float acc[V];
    few_ld<T, V>(x + (size_t)t * p.d + c, acc);
    for (int q = 0; q < p.k; ++q) {
      const int e = p.idx[t * p.k + q];
      if (e < 0 || e >= p.E) continue;
      const int pos = __popcll(R.tokens[e] & ((1ull << t) - 1));
      if (pos >= p.C) continue;
      const int row = R.base[e] + pos, np = pieces(R.owner[row], (int)c);
      const float *src = p.zpart + (size_t)row * p.d + c;
      float v[V] = {};
#pragma unroll 4
      for (int s = 0; s < np; ++s) few_add<V>(src + s * step, v);
      if (b2) {
        float b[V];
        few_ld<T, V>(b2 + (size_t)e * p.d + c, b);
#pragma unroll
        for (int z = 0; z < V; ++z) v[z] += b[z];
      }
      const float g = p.gate[t * p.k + q];
#pragma unroll
      for (int z = 0; z < V; ++z) acc[z] = fmaf(g, v[z], acc[z]);
    }
    bool bad = false;
#pragma unroll
    for (int z = 0; z < V; ++z) bad |= !isfinite(acc[z]);
    if (bad) record_error(p.st, MOE_ERR_NONFINITE, t);
    few_st<T, V>(y + (size_t)t * p.d + c, acc);
  }
}

}  // namespace

// Launches a kernel of one cooperative grid of kFewThreads-thread blocks.
cudaError_t launch_few_grid(const void *kernel, void **args, int grid, size_t smem,
                            cudaStream_t s);
// k_few_tc.cu: bf16 layers whose widths are multiples of 8, experts on tcgen05.
bool few_tc_supported(const moe_config &cfg);
cudaError_t launch_few_tc(const FewArgs &p, cudaStream_t s);

}  // namespace moe
