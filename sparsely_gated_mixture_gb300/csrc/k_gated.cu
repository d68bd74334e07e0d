// What surrounds the gated experts' products: the choices' slots in one launch,
// dL/dgate of each choice from the products' partial sums, the gradient of x.
#include "gated.cuh"

namespace moe {
namespace {

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
__global__ void __launch_bounds__(kRouteChunk) k_gated_route(const GatedRouteArgs p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int route_mem[];
  int *before = route_mem, *total = before + p.E, *off = total + p.E;  // [E], [E], [E + 1]
  __shared__ int own[kRouteChunk];
  __shared__ int warps[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int a0 = (int)blockIdx.x * kRouteChunk, a = a0 + tid;
  const bool first = blockIdx.x == 0;
  if (first && tid < (int)(sizeof(DeviceStatus) / 4)) reinterpret_cast<uint32_t *>(p.st)[tid] = 0;
  for (int e = tid; e < 2 * p.E; e += kRouteChunk) route_mem[e] = 0;
  int mine = a < p.A ? p.idx[a] : -1;
  if (mine >= p.E) mine = -1;
  own[tid] = mine;
  __syncthreads();
  // Sixteen loads in flight a thread.
  for (int i0 = tid; i0 < p.A; i0 += 16 * kRouteChunk) {
    int e[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int i = i0 + j * kRouteChunk;
      e[j] = i < p.A ? p.idx[i] : -1;
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int i = i0 + j * kRouteChunk;
      if (e[j] >= 0 && e[j] < p.E)
        atomicAdd(i < a0 ? &before[e[j]] : &total[e[j]], 1);
      else if (first && i < p.A)
        record_error(p.st, MOE_ERR_BOUNDS, (long long)i);  // after block 0's clearing
    }
  }
  __syncthreads();
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
      const size_t t = (size_t)(a / k) * d, e = (size_t)idx[a] * d;
      for (int i = lane; i < d; i += 32) s = fmaf(ld(dy, t + i), ld(b2, e + i), s);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) dgate[a] = s;
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
  for (int i0 = 0; i0 < d; i0 += 32) {
    const int i = i0 + lane;
    float s = i < d ? ld(dy, (size_t)t * d + i) : 0.f;
    for (int j = 0; j < k; ++j) {
      const long long r = __shfl_sync(0xffffffffu, mine, j);
      if (r >= 0 && i < d) s += dX[(size_t)r * d + i];
    }
    if (i < d) {
      if constexpr (sizeof(T) == 2) dx[(size_t)t * d + i] = __float2bfloat16_rn(s);
      else dx[(size_t)t * d + i] = s;
    }
  }
}

}  // namespace

cudaError_t launch_gated_route(const GatedRouteArgs &a, cudaStream_t s) {
  return launch_pdl(k_gated_route, (a.A + kRouteChunk - 1) / kRouteChunk, kRouteChunk,
                    (3 * (size_t)a.E + 1) * 4, s, a);
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
