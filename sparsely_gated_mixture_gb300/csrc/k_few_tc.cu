// The few-token layer with the experts on tcgen05: bf16 layers whose widths
// are multiples of 8.
//
// The products are bound by reading the weights once, so the weights are the
// tall operand: D[n, token] = sum_k W[k, n] A[token, k] with M = 128 weight
// columns on the TMEM lanes and the tokens as the instruction's N (16 to 64).
// Weight tiles go from HBM by TMA straight into the MMA's shared memory, and
// no thread touches them.
//
// The work of a layer, (experts in use) x (256-column tiles) x (64-row chunks
// of K), is one line of units of 32 KB of weights that the blocks share in
// equal contiguous runs. A tile that one run holds whole goes on directly; the
// parts of a shared one leave as partial sums, added in order of K: for layer
// 1 by the block that writes the tile's last part, which then makes H of them,
// for layer 2 in the combine. With a single token all of layer 1 leaves as
// partial sums, and the warp that feeds layer 2's tokens adds them (few_tokens):
// one row is little to read again, and the join before the barrier took 2.4 us
// more.
//
// Warps: 0 weight producer (TMA), 1 MMA issuer and TMEM owner, 2 producer of
// the token operand (TMA: x for layer 1, H for layer 2), 4-7 epilogue. The
// weight producer knows both layers' tiles once the experts are selected, so
// it runs ahead into layer 2 while the grid joins layer 1's partials: the ring
// of stages holds some 4 us of HBM time per SM, which covers the two barriers
// between the layers.
#include "few.cuh"

namespace moe {
namespace {

constexpr int kTile = kFewTile;               // weight columns of a unit
constexpr int kChunk = 64;                    // rows of K of a unit
constexpr int kWBytes = kTile * kChunk * 2;   // 32 KB
constexpr int kBoxBytes = 64 * kChunk * 2;    // one [64 x 64] box, 8 KB
constexpr int kMaxStages = 8;
constexpr int kTmemCols = 256;                // 2 buffers x 2 halves x 64 tokens
constexpr int kEpiThreads = 128;

// D = A B with fp32 accumulation, bf16 operands, A (weights) MN-major, B
// (tokens) K-major, M = 128, N tokens.
__device__ __forceinline__ uint32_t few_idesc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void few_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A box of weights, first to leave L2: each is read once, and what the blocks
// exchange should stay (40 tokens over 1024 experts 93 -> 87 us).
__device__ __forceinline__ void few_tma_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                           int y, int z) {
  asm volatile(
      "{\n .reg .b64 pol;\n createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n"
      " cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], pol;\n}\n" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// Eight TMEM columns of this warp's lanes, at any addresses, and one wait.
__device__ __forceinline__ void few_tmem8(const uint32_t (&a)[8], uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%8];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%9];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%2}, [%10];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%3}, [%11];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%4}, [%12];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%5}, [%13];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%6}, [%14];\n"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%7}, [%15];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7])
      : "memory");
}

// Whether v holds for all threads of the four epilogue warps (and a barrier of
// them).
__device__ __forceinline__ bool epi_all(bool v) {
  uint32_t out;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(out)
      : "r"((uint32_t)v), "n"(kEpiThreads)
      : "memory");
  return out != 0;
}

// One layer's units and this block's run of them, [lo, hi). G: the blocks that
// get any (every one of them at least two units, unless there is but one: with
// one unit each, the smallest layers gain less from the wider load than the
// doubled partial sums cost, 19.3 against 18.9 us for the noisy top-4 layer's
// token). total * G stays below 2^32: MOE_FEW_MAX_WIDTH bounds the units of few
// columns, and 2^32 / 152 units of half their 32 KB or more would not fit the
// device.
struct FewLine {
  int N, KC, NT;
  unsigned total, G, lo, hi;
  FixedDiv by_total;
  // Where the run begins: expert j of those in use, column tile nt, chunk kb;
  // the piece of its tile that it makes.
  int j, nt, kb, piece;

  // By one thread, for all others to use.
  __device__ void make(int n_experts, int K, int n, int grid) {
    N = n;
    KC = (K + kChunk - 1) / kChunk;
    NT = (n + kTile - 1) / kTile;
    total = (unsigned)n_experts * NT * KC;
    G = max(1u, min((unsigned)grid, total / 2));
    by_total = FixedDiv(total);
    const FixedDiv by_g(G);
    const unsigned b = min((unsigned)blockIdx.x, G);
    lo = b == G ? total : by_g(total * b);
    hi = b == G ? total : by_g(total * (b + 1));
    const unsigned tile = lo / KC;
    j = (int)(tile / NT);
    nt = (int)(tile - (unsigned)j * NT);
    kb = (int)(lo - tile * KC);
    piece = (int)(blockIdx.x - owner(tile * KC));
  }
  // The block whose run holds unit u: the largest b with floor(total b / G) <= u.
  __device__ unsigned owner(unsigned u) const { return by_total((u + 1) * G - 1); }
  // Partial sums of column c of expert jj.
  __device__ int pieces(int jj, int c) const {
    const unsigned u = ((unsigned)jj * NT + c / kTile) * KC;
    return (int)(owner(u + KC - 1) - owner(u)) + 1;
  }
};

// The shares of tiles that make up a block's run, in order: expert j, columns
// from nt * kTile, chunks [kb0, kb1), and which piece of the tile it is.
struct FewSeg {
  int j, nt, kb0, kb1, piece;
  unsigned left;  // units from kb0 to the run's end
  __device__ explicit FewSeg(const FewLine &l)
      : j(l.j), nt(l.nt), kb0(l.kb), piece(l.piece), left(l.hi - l.lo) {
    kb1 = (int)min((unsigned)l.KC, kb0 + left);
  }
  __device__ bool more() const { return left > 0; }
  __device__ void next(const FewLine &l) {
    left -= kb1 - kb0;
    kb0 = piece = 0;  // a tile begun by this run: its first piece
    if (++nt == l.NT) {
      nt = 0;
      ++j;
    }
    kb1 = (int)min((unsigned)l.KC, left);
  }
};

struct FewTc {
  int stages, tok_bytes;  // ring stages; bytes of a stage's token operand
};

// Layer 1's results are complete when every block has arrived at barrier 2 (one
// warp waits).
__device__ __forceinline__ bool few_wait_warp(const FewArgs &p, volatile int *abort_flag) {
  const bool done = (threadIdx.x & 31) == 0 ? few_wait(p, 2, abort_flag) : true;
  const bool all = __all_sync(0xffffffffu, done);
  if (!all) *abort_flag = 1;
  __syncwarp();
  return all;
}

// Layer 2's token operand where the layer has a single token (one row for each
// expert in use), by one warp, which waits for barrier 2 first: two columns a lane of a unit's 64,
// H = ReLU(sum of layer 1's parts + b1) rounded to bf16, as the join of a tile's
// parts would make it, without that join before the barrier. The loads of four
// units are in flight together. Returns the ring position after the last unit.
__device__ __forceinline__ uint32_t few_tokens(const FewArgs &p, const FewTc &q, const FewRows &R,
                                               const FewLine *line, uint8_t *ring,
                                               uint64_t *full_t, uint64_t *empty, uint32_t it,
                                               volatile int *abort_flag) {
  constexpr int B = 4, Z = 4;
  const FewLine &l = line[1];
  const int lane = threadIdx.x & 31, stage = kWBytes + q.tok_bytes;
  const __nv_bfloat162 *b1 = static_cast<const __nv_bfloat162 *>(p.b1);
  const size_t step = (size_t)R.rows * p.F;
  int j = l.j, nt = l.nt, kb = l.kb;
  for (unsigned u = l.lo; u < l.hi; u += B) {
    float2 v[B];
    const float *src[B];
    int np[B], most = 0;
    __nv_bfloat162 bias[B];
#pragma unroll
    for (int m = 0; m < B; ++m) {
      const int k = kb * kChunk + 2 * lane;
      const bool in = u + m < l.hi && k < p.F;
      v[m] = make_float2(0.f, 0.f);
      bias[m] = __floats2bfloat162_rn(0.f, 0.f);
      np[m] = in ? line[0].pieces(j, k) : 0;
      src[m] = p.hpart + (size_t)j * p.F + k;
      if (in && b1) bias[m] = b1[((size_t)R.expert[j] * p.F + k) / 2];
      most = max(most, np[m]);
      if (++kb == l.KC) {
        kb = 0;
        if (++nt == l.NT) {
          nt = 0;
          ++j;
        }
      }
    }
    if (u == l.lo && !few_wait_warp(p, abort_flag)) return it;
    for (int z0 = 0; z0 < most; z0 += Z) {
      float w[Z][B][2];
#pragma unroll
      for (int z = 0; z < Z; ++z)
#pragma unroll
        for (int m = 0; m < B; ++m)
          few_get<2>(src[m] + (z0 + z) * step, z0 + z < np[m], w[z][m]);
#pragma unroll
      for (int z = 0; z < Z; ++z)
#pragma unroll
        for (int m = 0; m < B; ++m) {
          v[m].x += w[z][m][0];
          v[m].y += w[z][m][1];
        }
    }
#pragma unroll
    for (int m = 0; m < B; ++m) {
      if (u + m >= l.hi) break;
      const int st = it % q.stages;
      const bool free =
          mbar_wait(&empty[st], ((it / q.stages) & 1u) ^ 1u, abort_flag, p.st, 117, p.wait_ns);
      if (!__all_sync(0xffffffffu, free)) return it;
      const __nv_bfloat162 h =
          __floats2bfloat162_rn(max_nan(v[m].x + __low2float(bias[m]), 0.f),
                                max_nan(v[m].y + __high2float(bias[m]), 0.f));
      // Row 0 of the operand: the swizzle leaves it in place.
      *reinterpret_cast<__nv_bfloat162 *>(ring + (size_t)st * stage + kWBytes + lane * 4) = h;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full_t[st]);
      ++it;
    }
  }
  return it;
}

// tmX: x [T, d], box [roundup(T, 16), 64]; tmH: H [T k, d_ff], box [16, 64];
// tm1, tm2: W1 [E, d, d_ff], W2 [E, d_ff, d], box [1, 64, 64]. All bf16 in the
// 128-byte swizzle; out-of-range rows and columns read as zero.
__global__ void __launch_bounds__(kFewThreads, 1)
k_few_tc(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmH,
         const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
         const __grid_constant__ FewArgs p, const FewTc q) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t full_w[kMaxStages], full_t[kMaxStages], empty[kMaxStages];
  __shared__ uint64_t acc_full[2], acc_empty[2], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ bool last_part;
  __shared__ FewAlone alone;
  __shared__ __align__(16) unsigned char line_mem[2 * sizeof(FewLine)];
  FewLine *line = reinterpret_cast<FewLine *>(line_mem);
  volatile int *abort_flag = &abort_word;
  // 1024-byte aligned, by an offset: through an integer the compiler would lose
  // that this is shared memory (generic loads took the router 8 us, not 4).
  uint8_t *ring = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const int stage = kWBytes + q.tok_bytes, S = q.stages;
  uint8_t *rows_mem = ring + (size_t)S * stage;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool direct = p.T == 1;  // layer 2's tokens straight from layer 1's partial sums

  few_start(p);
  // The ring's memory serves the router and the selection first.
  float *work = reinterpret_cast<float *>(ring);
  few_route<__nv_bfloat16>(p, work);
  few_barrier_arrive(p, 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full_w[s], 1);
      mbar_init(&full_t[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(&drain, 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (const CUtensorMap *m : {&tmX, &tmH, &tm1, &tm2})
      asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)m) : "memory");
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  bool ok = few_barrier_wait(p, 0);
  if (ok) {
    few_select<__nv_bfloat16>(p, work, alone);
    if (p.T > 1) ok = few_barrier(p, 1);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  FewRows R{};
  if (ok) R = few_rows(p, reinterpret_cast<char *>(rows_mem), alone);
  if (ok && R.n > 0 && lane == 0 && warp < 2)
    line[warp].make(R.n, warp ? p.F : p.d, warp ? p.d : p.F, gridDim.x);
  fence_proxy_async_smem();  // generic accesses to the ring come before TMA's
  __syncthreads();
  if (ok && R.n > 0) {
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------ weight producer
        uint32_t it = 0;
        bool go = true;
        for (int layer = 0; layer < 2 && go; ++layer) {
          const FewLine &l = line[layer];
          const CUtensorMap *tm = layer ? &tm2 : &tm1;
          for (FewSeg s(l); s.more() && go; s.next(l)) {
            const int n0 = s.nt * kTile;
            const int e = R.expert[s.j], boxes = min(4, (l.N - n0 + 63) / 64);
            for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
              const int st = it % S;
              if (!mbar_wait(&empty[st], ((it / S) & 1u) ^ 1u, abort_flag, p.st, 111, p.wait_ns)) {
                go = false;
                break;
              }
              mbar_expect_tx(&full_w[st], boxes * kBoxBytes);
              for (int b = 0; b < boxes; ++b)
                few_tma_3d(ring + (size_t)st * stage + b * kBoxBytes, tm, &full_w[st],
                           n0 + b * 64, kb * kChunk, e);
            }
          }
        }
        for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i)
          mbar_drain(&full_w[i % S], (i / S) & 1u);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // ------------------------------------------------------ MMA issuer
        uint32_t it = 0;
        int local = 0;
        bool go = true;
        for (int layer = 0; layer < 2 && go; ++layer) {
          const FewLine &l = line[layer];
          for (FewSeg s(l); s.more() && go; s.next(l), ++local) {
            const int buf = local & 1;
            if (!mbar_wait(&acc_empty[buf], ((local >> 1) & 1u) ^ 1u, abort_flag, p.st, 112,
                           p.wait_ns))
              break;
            tc_fence_after();
            const int toks = layer ? R.first[s.j + 1] - R.first[s.j] : p.T;
            const uint32_t idesc = few_idesc((toks + 15) / 16 * 16);
            const uint32_t d0 = tmem + (uint32_t)(buf * 128);
            const int halves = l.N - s.nt * kTile > 128 ? 2 : 1;
            for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
              const int st = it % S;
              const uint32_t ph = (it / S) & 1u;
              if (!mbar_wait(&full_w[st], ph, abort_flag, p.st, 113, p.wait_ns) ||
                  !mbar_wait(&full_t[st], ph, abort_flag, p.st, 114, p.wait_ns)) {
                go = false;
                break;
              }
              tc_fence_after();
              const uint32_t a0 = smem_u32(ring + (size_t)st * stage);
              const uint32_t b0 = a0 + kWBytes;
              for (int h = 0; h < halves; ++h)
#pragma unroll
                for (int kk = 0; kk < kChunk / 16; ++kk)
                  few_mma(d0 + h * 64, sdesc(a0 + h * 2 * kBoxBytes + kk * 2048, kBoxBytes, 1024),
                          sdesc(b0 + kk * 32, 16, 1024), idesc, (kb > s.kb0 || kk) ? 1u : 0u);
              umma_commit(&empty[st]);
            }
            if (go) umma_commit(&acc_full[buf]);
          }
        }
        umma_commit(&drain);
        mbar_drain(&drain, 0);
      }
    } else if (warp == 2) {
      // -------------------------------------------------------- token producer
      uint32_t it = 0;
      bool go = true;
      for (int layer = 0; layer < 2 && go; ++layer) {
        const FewLine &l = line[layer];
        if (layer && direct) {
          it = few_tokens(p, q, R, line, ring, full_t, empty, __shfl_sync(0xffffffffu, it, 0),
                          abort_flag);
          break;
        }
        if (layer) {
          if (!few_wait_warp(p, abort_flag)) break;
          asm volatile("fence.proxy.async.global;" ::: "memory");
        }
        for (FewSeg s(l); s.more() && go; s.next(l)) {
          if (lane == 0) {
            const int r0 = R.first[s.j], rows = R.first[s.j + 1] - r0;
            const int boxes = layer ? (rows + 15) / 16 : 1;
            const uint32_t bytes = layer ? boxes * 2048 : q.tok_bytes;
            for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
              const int st = it % S;
              if (!mbar_wait(&empty[st], ((it / S) & 1u) ^ 1u, abort_flag, p.st, 115, p.wait_ns)) {
                go = false;
                break;
              }
              uint8_t *dst = ring + (size_t)st * stage + kWBytes;
              mbar_expect_tx(&full_t[st], bytes);
              for (int b = 0; b < boxes; ++b)
                tma_load_2d(dst + b * 2048, layer ? &tmH : &tmX, &full_t[st], kb * kChunk,
                            layer ? r0 + b * 16 : 0);
            }
          }
          go = __shfl_sync(0xffffffffu, go, 0);
        }
      }
      if (lane == 0)
        for (uint32_t i = it > (uint32_t)S ? it - S : 0; i < it; ++i)
          mbar_drain(&full_t[i % S], (i / S) & 1u);
    } else if (warp >= 4) {
      // -------------------------------------------------------- epilogue
      const int quad = warp & 3, et = threadIdx.x - 128;
      const __nv_bfloat16 *b1 = static_cast<const __nv_bfloat16 *>(p.b1);
      __nv_bfloat16 *hout = static_cast<__nv_bfloat16 *>(p.h);
      int local = 0;
      bool go = true;
      for (int layer = 0; layer < 2 && go; ++layer) {
        const FewLine &l = line[layer];
        float *part = layer ? p.zpart : p.hpart;
        for (FewSeg s(l); s.more(); s.next(l), ++local) {
          const int buf = local & 1, n0 = s.nt * kTile;
          // In layer 1 the four warps meet below: they go on or leave together.
          go = mbar_wait(&acc_full[buf], (local >> 1) & 1u, abort_flag, p.st, 116, p.wait_ns);
          go = layer ? __all_sync(0xffffffffu, go) : epi_all(go);
          if (!go) break;
          tc_fence_after();
          const int r0 = R.first[s.j], rows = R.first[s.j + 1] - r0;
          const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * 128);
          float *out = part + ((size_t)s.piece * R.rows + r0) * l.N;
          // A whole tile of layer 1 becomes H here; a part of one leaves as a
          // partial sum, and whoever writes a tile's last part joins them.
          const bool whole = layer == 0 && !direct && s.kb0 == 0 && s.kb1 == l.KC;
          const int e = R.expert[s.j];
          for (int h = 0; h < 2; ++h) {
            if (n0 + h * 128 >= l.N) break;
            const int n = n0 + h * 128 + quad * 32 + lane;
            const float bias =
                whole && b1 && n < l.N ? __bfloat162float(b1[(size_t)e * l.N + n]) : 0.f;
            for (int r = 0; r < rows; r += 8) {
              uint32_t a[8], v[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int rr = min(r + i, rows - 1);
                a[i] = lanes + h * 64 + (uint32_t)(layer ? rr : R.token[r0 + rr]);
              }
              few_tmem8(a, v);
              if (n < l.N) {
                if (whole) {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (r + i < rows)
                      hout[(size_t)(r0 + r + i) * l.N + n] =
                          __float2bfloat16_rn(max_nan(__uint_as_float(v[i]) + bias, 0.f));
                } else {
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    if (r + i < rows) out[(size_t)(r + i) * l.N + n] = __uint_as_float(v[i]);
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[buf]);
          if (layer == 0 && !whole && !direct) {
            const int np = l.pieces(s.j, n0);
            epi_all(true);  // the part is written
            if (et == 0) {
              __threadfence();
              last_part = atomicAdd(p.tiles + s.j * l.NT + s.nt, 1u) == (unsigned)np - 1;
              __threadfence();
            }
            epi_all(true);
            if (last_part) {
              const int cols = min(kTile, l.N - n0) / 4;
              const size_t step = (size_t)R.rows * l.N;
              const float *src = part + (size_t)r0 * l.N + n0;
              // Four places a thread at a time, so that their loads overlap.
              for (int i0 = et; i0 < rows * cols; i0 += 4 * kEpiThreads) {
                float v[4][4] = {};
                int r[4], c[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  const int i = i0 + m * kEpiThreads;
                  r[m] = i < rows * cols ? (cols == kTile / 4 ? i / (kTile / 4) : i / cols) : -1;
                  c[m] = (i - r[m] * cols) * 4;
                }
#pragma unroll 2
                for (int z = 0; z < np; ++z) {
                  float w[4][4];
#pragma unroll
                  for (int m = 0; m < 4; ++m)
                    few_get<4>(src + z * step + (size_t)r[m] * l.N + c[m], r[m] >= 0, w[m]);
#pragma unroll
                  for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int x = 0; x < 4; ++x) v[m][x] += w[m][x];
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                  if (r[m] < 0) continue;
                  if (b1) {
                    float b[4];
                    few_ld<__nv_bfloat16, 4>(b1 + (size_t)e * l.N + n0 + c[m], b);
#pragma unroll
                    for (int z = 0; z < 4; ++z) v[m][z] += b[z];
                  }
#pragma unroll
                  for (int z = 0; z < 4; ++z) v[m][z] = max_nan(v[m][z], 0.f);
                  few_st<__nv_bfloat16, 4>(hout + (size_t)(r0 + r[m]) * l.N + n0 + c[m], v[m]);
                }
              }
            }
          }
        }
        if (layer == 0) {
          // H's share of this block is written: TMA of every block may read it.
          asm volatile("fence.proxy.async.global;" ::: "memory");
          go = epi_all(go && *abort_flag == 0);
          if (!go) *abort_flag = 1;
          else if (et == 0) few_arrive(p, 2);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
  if (!ok || *abort_flag) {
    if (threadIdx.x == 0) few_leave(p);
    return;
  }
  few_combine<__nv_bfloat16, 4>(p, R, [&](int j, int c) { return line[1].pieces(j, c); });
}

// 3-D bf16 tensor [E, K, N], box [1, 64, 64], 128-byte swizzle; rows past K of
// an expert and columns past N read as zero.
bool make_weight_map(CUtensorMap *m, const void *base, int E, int K, int N) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)N, (cuuint64_t)K, (cuuint64_t)E};
  cuuint64_t strides[2] = {(cuuint64_t)N * 2, (cuuint64_t)K * N * 2};
  cuuint32_t box[3] = {64, kChunk, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kSmemMax = kSmemMost - 1024;  // less the static part

}  // namespace

int few_tc_tiles(const moe_config &c) {
  const long long A = (long long)c.T * c.k;
  return (int)((A < c.E ? A : c.E) * ((c.d_ff + kTile - 1) / kTile));
}

cudaError_t launch_few_tc(const FewArgs &p, cudaStream_t s) {
  const int box = (p.T + 15) / 16 * 16;
  FewTc q;
  q.tok_bytes = box * kChunk * 2;
  const size_t rows = few_rows_bytes(p.E, p.T * p.k);
  const size_t stage = kWBytes + q.tok_bytes;
  q.stages = (int)((kSmemMax - 1024 - rows) / stage);
  if (q.stages > kMaxStages) q.stages = kMaxStages;
  CUtensorMap tx, th, t1, t2;
  if (!make_map(&tx, p.x, (uint64_t)p.T, (uint64_t)p.d, (uint32_t)box) ||
      !make_map(&th, p.h, (uint64_t)p.T * p.k, (uint64_t)p.F, 16) ||
      !make_weight_map(&t1, p.W1, p.E, p.d, p.F) || !make_weight_map(&t2, p.W2, p.E, p.F, p.d))
    return cudaErrorInvalidValue;
  int grid = sm_count();
  if (grid > kFewMaxGrid) grid = kFewMaxGrid;
  FewArgs a = p;
  a.rt = few_router(p.T, p.d, p.E, p.Wn != nullptr, grid);
  void *args[6] = {&tx, &th, &t1, &t2, &a, &q};
  return launch_few_grid(reinterpret_cast<const void *>(k_few_tc), args, grid,
                         1024 + q.stages * stage + rows, kSmemMax, s);
}

}  // namespace moe
