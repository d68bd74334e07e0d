// What surrounds the gated experts' products: the choices' slots in one launch,
// dL/dgate of each choice from the products' partial sums, the gradient of x.
#include "gated.cuh"

namespace moe {
namespace {

// Up to three arrays of rows and what their column sums are; weight: by packed
// row, or null.
template <typename S, typename O>
struct GatedColumns {
  const S *src[3];
  const float *weight[3];
  O *out[3];
  int cols[3], blocks[3];
};

template <typename T>
__device__ __forceinline__ float ld(const T *p, size_t i) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(p[i]);
  else return p[i];
}

__global__ void k_gated_begin(DeviceStatus *st) {
  pdl_wait();
  if (threadIdx.x < sizeof(DeviceStatus) / 4) reinterpret_cast<uint32_t *>(st)[threadIdx.x] = 0;
}

// Exclusive sum of v over the block's 256 threads; *total gets the whole.
__device__ __forceinline__ int block_scan(int v, int *warps, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();  // the last call's reads of warps are done
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) before += warps[w];
    all += warps[w];
  }
  *total = all;
  return before + incl - v;
}

// Slots without a pass over the grid between: a block ranks 256 assignments
// and counts, for itself, all of them before its own and all after. A batch of
// kRouteMost choices is 128 KB that every block reads from L2; the histogram,
// scan and rank passes for long batches and a separate clearing of the status
// word take four launches (4096 tokens of top 4: 17 us against 6).
constexpr int kRouteChunk = 256;
__host__ __device__ constexpr int route_copies(int E) { return E <= 256 ? 8 : 1; }
__global__ void __launch_bounds__(kRouteChunk) k_gated_route(const GatedRouteArgs p) {
  pdl_wait();
  pdl_trigger();
  // Counts before and from the block's own on, `copies` of each (lanes take
  // turns, so that few experts do not mean long queues for one counter), offsets.
  extern __shared__ int route_mem[];
  const int copies = route_copies(p.E);
  int *before = route_mem, *total = before + p.E, *off = route_mem + 2 * copies * p.E;
  __shared__ int own[kRouteChunk];
  __shared__ int warps[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int a0 = (int)blockIdx.x * kRouteChunk, a = a0 + tid;
  const bool first = blockIdx.x == 0;
  if (first && tid < (int)(sizeof(DeviceStatus) / 4)) reinterpret_cast<uint32_t *>(p.st)[tid] = 0;
  for (int e = tid; e < 2 * copies * p.E; e += kRouteChunk) route_mem[e] = 0;
  int mine = a < p.A ? p.idx[a] : -1;
  if (mine >= p.E) mine = -1;
  own[tid] = mine;
  __syncthreads();
  // Eight loads of four in flight a thread (own chunks begin on a multiple of 4).
  int *const hist = route_mem + (lane & (copies - 1)) * 2 * p.E;
  for (int i0 = 4 * tid; i0 < p.A; i0 += 32 * kRouteChunk) {
    int4 u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * 4 * kRouteChunk;
      if (i + 3 < p.A) {
        u[j] = *reinterpret_cast<const int4 *>(p.idx + i);
      } else {
        u[j].x = i < p.A ? p.idx[i] : -1;
        u[j].y = i + 1 < p.A ? p.idx[i + 1] : -1;
        u[j].z = i + 2 < p.A ? p.idx[i + 2] : -1;
        u[j].w = -1;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * 4 * kRouteChunk, e[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (e[q] >= 0 && e[q] < p.E) atomicAdd(hist + (i < a0 ? 0 : p.E) + e[q], 1);
        else if (first && i + q < p.A) record_error(p.st, MOE_ERR_BOUNDS, (long long)(i + q));
      }
    }
  }
  __syncthreads();
  if (copies > 1) {
    for (int e = tid; e < 2 * p.E; e += kRouteChunk) {
      int n = 0;
      for (int c = 0; c < copies; ++c) n += route_mem[c * 2 * p.E + e];
      route_mem[e] = n;
    }
    __syncthreads();
  }
  // Kept rows, their offsets and the tiles of 128 rows, four experts a thread.
  int rows[4], n = 0, tiles = 0, pads = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * tid + j;
    rows[j] = 0;
    if (e < p.E) {
      rows[j] = min(before[e] + total[e], p.C);
      tiles += (rows[j] + kTcBM - 1) / kTcBM;
      pads += max(kBwdRowPad, (rows[j] + kBwdRowPad - 1) / kBwdRowPad * kBwdRowPad);
    }
    n += rows[j];
  }
  int all;
  int at = block_scan(n, warps, &all);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (4 * tid + j < p.E) {
      off[4 * tid + j] = at;
      if (first) p.offset[4 * tid + j] = at;
    }
    at += rows[j];
  }
  if (first) {
    if (tid == 0) p.offset[p.E] = all;
    int tile = block_scan(tiles, warps, &all);
    if (tid == 0) p.mtiles[p.E] = all;
    int pad = block_scan(pads, warps, &all);
    if (tid == 0 && p.poff) p.poff[p.E] = all;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * tid + j;
      if (e >= p.E) break;
      p.mtiles[e] = tile;
      tile += (rows[j] + kTcBM - 1) / kTcBM;
      if (p.poff) p.poff[e] = pad;
      pad += max(kBwdRowPad, (rows[j] + kBwdRowPad - 1) / kBwdRowPad * kBwdRowPad);
    }
  }
  __syncthreads();
  // The rank among the block's own: equal lanes before this one, and the warps
  // before.
  const unsigned peers = __match_any_sync(0xffffffffu, mine);
  int rank = __popc(peers & ((1u << lane) - 1u));
  for (int i = 0; i < warp * 32; ++i) rank += own[i] == mine;
  if (a >= p.A) return;
  const int ps = mine < 0 ? -1 : before[mine] + rank;
  const bool kept = mine >= 0 && ps < p.C;
  p.pos[a] = ps;
  p.keep[a] = kept ? 1 : 0;
  if (kept) {
    p.row_token[off[mine] + ps] = a;
    p.row_gate[off[mine] + ps] = p.gate[a];
  }
}

// The row of assignment a = t*k + j, or -1 (dropped, or not an expert).
__device__ __forceinline__ long long gated_row(long long a, int E, const int32_t *idx,
                                               const int32_t *pos, const uint8_t *keep,
                                               const int32_t *base) {
  if (!keep[a]) return -1;
  const int e = idx[a];
  return e >= 0 && e < E ? (long long)base[e] + pos[a] : -1;
}

// One warp per assignment; lanes in order, so the sum's order is fixed.
template <typename T>
__global__ void __launch_bounds__(256)
k_gated_dgate(long long A, int E, int k, int d, int n_blocks, const int32_t *__restrict__ idx,
              const int32_t *__restrict__ pos, const uint8_t *__restrict__ keep,
              const int32_t *__restrict__ base, const float *__restrict__ dgpart,
              const T *__restrict__ dy, const T *__restrict__ b2, float *__restrict__ dgate) {
  pdl_wait();
  pdl_trigger();
  const long long a = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (a >= A) return;
  const long long r = gated_row(a, E, idx, pos, keep, base);
  float s = 0.f;
  if (r >= 0) {
    for (int b = lane; b < n_blocks; b += 32) s += dgpart[r * n_blocks + b];
    if (b2) {
      const T *y = dy + (size_t)(a / k) * d, *b = b2 + (size_t)idx[a] * d;
      constexpr int V = 16 / (int)sizeof(T);
      if (d % V == 0) {
        for (int i = lane * V; i < d; i += 32 * V) {
          const uint4 u = *reinterpret_cast<const uint4 *>(y + i);
          const uint4 w = *reinterpret_cast<const uint4 *>(b + i);
#pragma unroll
          for (int j = 0; j < V; ++j)
            s = fmaf(ld(reinterpret_cast<const T *>(&u), j), ld(reinterpret_cast<const T *>(&w), j),
                     s);
        }
      } else {
        for (int i = lane; i < d; i += 32) s = fmaf(ld(y, i), ld(b, i), s);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dgate[a] = s;
}

// One warp per padded row, then one per zero row: 16 bytes a lane, four in flight
// of each operand.
__global__ void __launch_bounds__(256)
k_gated_gather(long long P_max, int E, int k, int nv, int fv, const int32_t *__restrict__ offset,
               const int32_t *__restrict__ poff, const int32_t *__restrict__ row_token,
               const uint4 *__restrict__ x, const uint4 *__restrict__ dy,
               uint4 *__restrict__ xbuf, uint4 *__restrict__ h, uint4 *__restrict__ dY) {
  pdl_wait();
  pdl_trigger();
  const long long w = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const uint4 z = make_uint4(0, 0, 0, 0);
  if (w >= P_max) {  // a row behind the last packed one
    if (w >= P_max + kBwdRowPad) return;  // the grid's last block has warps to spare
    const size_t r = (size_t)offset[E] + (w - P_max);
    for (int i = lane; i < nv; i += 32) xbuf[r * nv + i] = z;
    for (int i = lane; i < fv; i += 32) h[r * fv + i] = z;
    return;
  }
  if (w >= poff[E]) return;
  int lo = 0, hi = E;  // largest e with poff[e] <= w
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (poff[mid] <= w) lo = mid;
    else hi = mid;
  }
  const int m = (int)(w - poff[lo]), q = offset[lo] + m;
  uint4 *oy = dY + w * nv;
  if (q >= offset[lo + 1]) {
    for (int i = lane; i < nv; i += 32) oy[i] = z;
    return;
  }
  const size_t t = (size_t)(row_token[q] / k) * nv;
  uint4 *ox = xbuf + (size_t)q * nv;
  constexpr int N = 4;
  for (int i0 = lane; i0 < nv; i0 += 32 * N) {
    uint4 a[N], b[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + 32 * j;
      a[j] = i < nv ? x[t + i] : z;
      b[j] = i < nv ? dy[t + i] : z;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = i0 + 32 * j;
      if (i >= nv) break;
      ox[i] = a[j];
      oy[i] = b[j];
    }
  }
}

// The bias gradients: column sums of each expert's rows, a block for 64 columns
// and an expert. Eight warps take rows in turn, 16 bytes a lane and eight of
// them in flight (widths of an odd size: a value a lane); lanes, then warps,
// add in a fixed order. The pad rows behind an expert's are not read.
template <typename S, typename O, bool VEC>
__global__ void __launch_bounds__(256)
k_gated_colsum(const int32_t *__restrict__ offset, const int32_t *__restrict__ base,
               const GatedColumns<S, O> p) {
  pdl_wait();
  pdl_trigger();
  constexpr int V = VEC ? 16 / (int)sizeof(S) : 1, LANES = VEC ? 64 / V : 32, PER = 32 / LANES;
  constexpr int Q = 64 / (LANES * V);  // column groups of a lane
  __shared__ float sums[8][64];
  int job = 0, cb = blockIdx.x;
  while (cb >= p.blocks[job]) cb -= p.blocks[job++];
  const int e = blockIdx.y, cols = p.cols[job], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = offset[e + 1] - offset[e];
  const int c0 = cb * 64 + (lane % LANES) * V;
  const S *src = p.src[job] + (size_t)base[e] * cols;
  const float *weight = p.weight[job] ? p.weight[job] + offset[e] : nullptr;
  float acc[Q][V] = {};
  for (int r0 = warp * PER + lane / LANES; r0 < rows; r0 += 64 * PER) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int c = c0 + q * 32;
      if (c >= cols) continue;
      if constexpr (VEC) {
        uint4 u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + i * 8 * PER;
          u[i] = r < rows ? *reinterpret_cast<const uint4 *>(src + (size_t)r * cols + c)
                          : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float w = weight ? weight[min(r0 + i * 8 * PER, rows - 1)] : 1.f;
#pragma unroll
          for (int v = 0; v < V; ++v)
            acc[q][v] = fmaf(w, ld(reinterpret_cast<const S *>(&u[i]), v), acc[q][v]);
        }
      } else {
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + i * 8 * PER;
          u[i] = r < rows ? ld(src, (size_t)r * cols + c) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          acc[q][0] =
              fmaf(weight ? weight[min(r0 + i * 8 * PER, rows - 1)] : 1.f, u[i], acc[q][0]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int o = LANES; o < 32; o <<= 1)
        acc[q][v] += __shfl_xor_sync(0xffffffffu, acc[q][v], o);
      if (lane < LANES) sums[warp][lane * V + q * 32 + v] = acc[q][v];
    }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 64 && cb * 64 + c < cols) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][c];
    O *out = p.out[job] + (size_t)e * cols + cb * 64 + c;
    if constexpr (sizeof(O) == 2) *out = __float2bfloat16_rn(s);
    else *out = s;
  }
}

// One warp per token; choices in order.
template <typename T>
__global__ void __launch_bounds__(256)
k_gated_dx(int T_, int E, int k, int d, const int32_t *__restrict__ idx,
           const int32_t *__restrict__ pos, const uint8_t *__restrict__ keep,
           const int32_t *__restrict__ base, const float *__restrict__ dX,
           const T *__restrict__ dy, T *__restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  const long long t = (blockIdx.x * 256ll + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (t >= T_) return;
  const long long mine = lane < k ? gated_row(t * k + lane, E, idx, pos, keep, base) : -1;
  constexpr int N = 4;  // columns of a lane in flight
  for (int i0 = lane; i0 - lane < d; i0 += 32 * N) {
    float s[N];
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int i = i0 + 32 * q;
      s[q] = i < d ? ld(dy, (size_t)t * d + i) : 0.f;
    }
    for (int j = 0; j < k; ++j) {
      const long long r = __shfl_sync(0xffffffffu, mine, j);
      if (r < 0) continue;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const int i = i0 + 32 * q;
        if (i < d) s[q] += dX[(size_t)r * d + i];
      }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int i = i0 + 32 * q;
      if (i >= d) continue;
      if constexpr (sizeof(T) == 2) dx[(size_t)t * d + i] = __float2bfloat16_rn(s[q]);
      else dx[(size_t)t * d + i] = s[q];
    }
  }
}

// y = x + the kept choices' rows of z, in choice order; a block a token, a thread a
// column, four rows in flight (a warp a token takes 10 us for 517 tokens of 130).
template <typename T>
__global__ void __launch_bounds__(128)
k_gated_combine(int E, int k, int d, const T *x, const float *__restrict__ z,
                const int32_t *__restrict__ idx, const int32_t *__restrict__ pos,
                const uint8_t *__restrict__ keep, const int32_t *__restrict__ offset, T *y,
                DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  __shared__ long long rows[16];
  const long long t = blockIdx.x;
  if (threadIdx.x < 16)
    rows[threadIdx.x] =
        threadIdx.x < k ? gated_row(t * k + threadIdx.x, E, idx, pos, keep, offset) : -1;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < d; i += 128) {
    float s = ld(x, (size_t)t * d + i);
    for (int j0 = 0; j0 < k; j0 += 4) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = rows[j0 + j] >= 0 ? z[(size_t)rows[j0 + j] * d + i] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) s += v[j];
    }
    bad |= !isfinite(s);
    if constexpr (sizeof(T) == 2) y[(size_t)t * d + i] = __float2bfloat16_rn(s);
    else y[(size_t)t * d + i] = s;
  }
  if (bad) record_error(st, MOE_ERR_NONFINITE, t);
}

}  // namespace

cudaError_t launch_gated_combine(const moe_config &c, const void *x, const float *z,
                                 const int32_t *idx, const int32_t *pos, const uint8_t *keep,
                                 const int32_t *offset, void *y, DeviceStatus *st,
                                 cudaStream_t s) {
  if (c.act_dtype == MOE_BF16)
    return launch_pdl_c(kPdlCombine, k_gated_combine<__nv_bfloat16>, c.T, 128, 0, s, c.E, c.k, c.d,
                        (const __nv_bfloat16 *)x, z, idx, pos, keep, offset, (__nv_bfloat16 *)y, st);
  return launch_pdl_c(kPdlCombine, k_gated_combine<float>, c.T, 128, 0, s, c.E, c.k, c.d,
                      (const float *)x, z, idx, pos, keep, offset, (float *)y, st);
}

cudaError_t launch_gated_route(const GatedRouteArgs &a, cudaStream_t s) {
  return launch_pdl(k_gated_route, (a.A + kRouteChunk - 1) / kRouteChunk, kRouteChunk,
                    ((2 * (size_t)route_copies(a.E) + 1) * a.E + 1) * 4, s, a);
}

cudaError_t launch_gated_gather(const moe_config &c, long long P_max, const GatedRows &rows,
                                const int32_t *poff, const void *x, const void *dy, void *xbuf,
                                void *h, void *dY, cudaStream_t s) {
  const long long warps = P_max + kBwdRowPad;
  return launch_pdl(k_gated_gather, (unsigned)((warps + 7) / 8), 256, 0, s, P_max, c.E, c.k,
                    c.d / 8, c.d_ff / 8, rows.offset, poff, rows.row_token, (const uint4 *)x,
                    (const uint4 *)dy, (uint4 *)xbuf, (uint4 *)h, (uint4 *)dY);
}

cudaError_t launch_gated_begin(DeviceStatus *st, cudaStream_t s) {
  return launch_pdl(k_gated_begin, 1, 32, 0, s, st);
}

cudaError_t launch_gated_dgate(const moe_config &c, int n_blocks, const int32_t *idx,
                               const int32_t *pos, const uint8_t *keep, const int32_t *base,
                               const float *dgpart, const void *dy, const void *b2, float *dgate,
                               cudaStream_t s) {
  const long long A = (long long)c.T * c.k;
  const unsigned grid = (unsigned)((A + 7) / 8);
  if (c.act_dtype == MOE_BF16)
    return launch_pdl(k_gated_dgate<__nv_bfloat16>, grid, 256, 0, s, A, c.E, c.k, c.d, n_blocks,
                      idx, pos, keep, base, dgpart, (const __nv_bfloat16 *)dy,
                      (const __nv_bfloat16 *)b2, dgate);
  return launch_pdl(k_gated_dgate<float>, grid, 256, 0, s, A, c.E, c.k, c.d, n_blocks, idx, pos,
                    keep, base, dgpart, (const float *)dy, (const float *)b2, dgate);
}

template <typename S, typename O>
static cudaError_t run_colsum(int E, const int32_t *offset, const int32_t *base,
                              const void *const (&src)[3], const float *weight,
                              void *const (&out)[3], const int (&cols)[3], cudaStream_t s) {
  GatedColumns<S, O> p{};
  int n = 0, blocks = 0;
  bool vec = true;
  for (int j = 0; j < 3; ++j) {
    if (!out[j]) continue;
    p.src[n] = static_cast<const S *>(src[j]);
    p.weight[n] = j == 0 ? weight : nullptr;
    p.out[n] = static_cast<O *>(out[j]);
    p.cols[n] = cols[j];
    p.blocks[n] = (cols[j] + 63) / 64;
    blocks += p.blocks[n++];
    vec = vec && cols[j] % (16 / (int)sizeof(S)) == 0;
  }
  if (!n) return cudaSuccess;
  const dim3 grid(blocks, E);
  return vec ? launch_pdl(k_gated_colsum<S, O, true>, grid, 256, 0, s, offset, base, p)
             : launch_pdl(k_gated_colsum<S, O, false>, grid, 256, 0, s, offset, base, p);
}

cudaError_t launch_gated_colsum(const moe_config &c, bool src_f32, const int32_t *offset,
                                const int32_t *base, const void *dY, const float *row_gate,
                                void *db2, const void *dP1, void *db1, const void *dP3, void *db3,
                                cudaStream_t s) {
  const void *const src[3] = {dY, dP1, dP3};
  void *const out[3] = {db2, db1, db3};
  const int cols[3] = {c.d, c.d_ff, c.d_ff};
  const auto run = [&](auto kernel) {
    return kernel(c.E, offset, base, src, row_gate, out, cols, s);
  };
  if (c.act_dtype == MOE_F32) return run(run_colsum<float, float>);
  return src_f32 ? run(run_colsum<float, __nv_bfloat16>)
                 : run(run_colsum<__nv_bfloat16, __nv_bfloat16>);
}

cudaError_t launch_gated_dx(const moe_config &c, const int32_t *idx, const int32_t *pos,
                            const uint8_t *keep, const int32_t *base, const float *dX,
                            const void *dy, void *dx, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)c.T + 7) / 8);
  if (c.act_dtype == MOE_BF16)
    return launch_pdl(k_gated_dx<__nv_bfloat16>, grid, 256, 0, s, c.T, c.E, c.k, c.d, idx, pos,
                      keep, base, dX, (const __nv_bfloat16 *)dy, (__nv_bfloat16 *)dx);
  return launch_pdl(k_gated_dx<float>, grid, 256, 0, s, c.T, c.E, c.k, c.d, idx, pos, keep, base,
                    dX, (const float *)dy, (float *)dx);
}

}  // namespace moe
