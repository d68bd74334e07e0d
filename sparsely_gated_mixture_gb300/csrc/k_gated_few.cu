// The gated experts for a few tokens, in bf16 and in 8 bits: bound by reading
// the weights of the experts in use once. As in the few-token layer (k_few_tc.cu)
// the weights are the tall operand, D[n, token] = sum_k W[k, n] A[token, k], with
// M = 128 weight columns on the TMEM lanes and an expert's rows, 16 to 64, as the
// instruction's N; weight tiles go from HBM by TMA straight to the MMA.
//
// A unit of work is 32 KB of weights: 128 bytes of K (64 bf16, 128 e4m3) of 256
// columns -- layer 1: 128 of W1 and the same 128 of W3; layer 2: 256 of W2. The
// units of all experts in use are one line that the blocks share in equal runs,
// so any number of experts and columns loads every SM alike. A tile that one
// run holds whole goes on from TMEM; the parts of a shared one leave as partial
// sums, and the block that comes last adds them in order of K.
//
// The launches follow one another by programmatic dependence: a block of layer 2
// starts when an SM's block of layer 1 ends, and fills its ring with weights,
// which do not depend on layer 1, before it waits for the hidden rows. (Rings of
// half the size, so that both layers' blocks fit an SM: one token through the
// large experts 122 us instead of 121, in 8 bits 74 instead of 73.)
#include "gated.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kHalf = 16384;              // a unit's bytes of one half of its columns
constexpr int kUnit = 2 * kHalf;
constexpr int kBox = 8192;                // bf16: 64 columns of 64 K
constexpr int kMaxStages = 5;
constexpr int kSfBytes = 3 * 512;         // 8 bits: scales of both halves and of the rows
constexpr int kSfSlots = 2;

// ----------------------------------------------------------------------------- routing
// One block for each choice: its slot, its row of the packed x (copied, or put
// in 8 bits); block 0 also writes the offsets, the list of experts in use and
// the cleared status and counters.
struct RouteArgs {
  int A, E, C, k, d, max_rows, n_counters;
  const int32_t *idx;
  const float *gate;
  const __nv_bfloat16 *x;
  int32_t *pos;
  uint8_t *keep;
  int32_t *offset;
  float *row_gate;
  int4 *list;         // [n] {expert, first row, rows, 0} of the experts in use
  int32_t *counters;  // [0]: n; then the joins' counters
  void *xbuf;         // bf16 [rows, d], or e4m3 [rows, 128 KB]
  uint8_t *sx;        // 8 bits: [KB / 4][max_rows][4]
  DeviceStatus *st;
};

template <bool FP8>
__global__ void __launch_bounds__(256) k_few_gated_route(const RouteArgs p) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int hist[];  // [E]
  __shared__ int part[3][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int a = blockIdx.x;
  const bool first = a == 0;
  if (first) {
    if (tid < (int)(sizeof(DeviceStatus) / 4)) reinterpret_cast<uint32_t *>(p.st)[tid] = 0;
    for (int i = 1 + tid; i < p.n_counters; i += 256) p.counters[i] = 0;
  }
  for (int e = tid; e < p.E; e += 256) hist[e] = 0;
  const int mine = p.idx[a];
  __syncthreads();
  int before = 0;  // earlier choices of the same expert
  for (int i = tid; i < p.A; i += 256) {
    const int e = p.idx[i];
    if (e >= 0 && e < p.E) {
      atomicAdd(&hist[e], 1);
      before += e == mine && i < a;
    } else if (first) {
      record_error(p.st, MOE_ERR_BOUNDS, (long long)i);
    }
  }
  __syncthreads();
  int base = 0;  // rows of earlier experts
  for (int e = tid; e < min(mine, p.E); e += 256) base += min(hist[e], p.C);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    base += __shfl_xor_sync(0xffffffffu, base, o);
  }
  if (lane == 0) {
    part[0][warp] = before;
    part[1][warp] = base;
  }
  __syncthreads();
  before = base = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += part[0][w];
    base += part[1][w];
  }
  const bool valid = mine >= 0 && mine < p.E, kept = valid && before < p.C;
  const int row = base + before;
  if (tid == 0) {
    p.pos[a] = valid ? before : -1;
    p.keep[a] = kept ? 1 : 0;
    if (kept) p.row_gate[row] = p.gate[a];
  }
  if (first) {  // offsets and the list, 4 experts a thread
    int rows[4], n = 0, used = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * tid + j;
      rows[j] = e < p.E ? min(hist[e], p.C) : 0;
      n += rows[j];
      used += rows[j] > 0;
    }
    int in = n, iu = used;  // inclusive over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, in, o), v = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) {
        in += u;
        iu += v;
      }
    }
    __syncthreads();
    if (lane == 31) {
      part[0][warp] = in;
      part[1][warp] = iu;
    }
    __syncthreads();
    int at = in - n, slot = iu - used, all = 0, count = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) {
        at += part[0][w];
        slot += part[1][w];
      }
      all += part[0][w];
      count += part[1][w];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 4 * tid + j;
      if (e >= p.E) break;
      p.offset[e] = at;
      if (rows[j] > 0) p.list[slot++] = make_int4(e, at, rows[j], 0);
      at += rows[j];
    }
    if (tid == 0) {
      p.offset[p.E] = all;
      p.counters[0] = count;
    }
  }
  if (!kept) return;
  const __nv_bfloat16 *src = p.x + (size_t)(a / p.k) * p.d;
  if constexpr (!FP8) {  // d is a multiple of 64
    uint4 *out = static_cast<uint4 *>(p.xbuf) + (size_t)row * (p.d / 8);
    for (int i = tid; i < p.d / 8; i += 256) out[i] = reinterpret_cast<const uint4 *>(src)[i];
  } else {
    const int KB = (p.d + kFp8Block - 1) / kFp8Block;
    for (int kb = warp; kb < KB; kb += 8) {
      float v[4], top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = kb * kFp8Block + lane * 4 + j;
        v[j] = c < p.d ? __bfloat162float(src[c]) : 0.f;
        top = max_nan(top, fabsf(v[j]));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t byte = fp8_scale_byte(top);
      const float inv = fp8_inverse(byte);
      reinterpret_cast<uint32_t *>(p.xbuf)[((size_t)row * KB + kb) * 32 + lane] =
          fp8_pack2(v[0] * inv, v[1] * inv) | fp8_pack2(v[2] * inv, v[3] * inv) << 16;
      if (lane == 0) p.sx[((size_t)(kb >> 2) * p.max_rows + row) * 4 + (kb & 3)] = (uint8_t)byte;
    }
  }
}

// ----------------------------------------------------------------------------- the products
struct FewParams {
  int KC, N, NT, toks, stages, max_rows;  // chunks of K; columns; tiles; rows a tile holds
  int NB;                                 // 8 bits: scale blocks of the weight's columns
  const int4 *list;
  int32_t *counters;                      // [0] experts in use
  int32_t *joins;                         // [blocks]
  float *part;                            // [blocks][2][toks][256]
  const float *row_gate;
  const __nv_bfloat16 *bias, *bias3;
  __nv_bfloat16 *h, *pre1, *pre3;         // layer 1, bf16
  uint8_t *h8, *sh;                       // layer 1, 8 bits
  void *z;                                // layer 2
  int z_bf16;
  const uint32_t *sa;                     // 8 bits: the rows' scales
  const uint8_t *sb, *sb3;                // and the weights'
  DeviceStatus *st;
  unsigned long long wait_ns;
};

// This block's run of units, as pieces of tiles.
struct Run {
  unsigned total, G, lo, hi;
  int KC, NT;
  __device__ Run(int experts, int nt, int kc) : KC(kc), NT(nt) {
    total = (unsigned)experts * nt * kc;
    // At least two units each, unless there is but one.
    G = total ? max(1u, min(gridDim.x, total / 2)) : 1u;
    lo = blockIdx.x < G ? first(blockIdx.x) : total;
    hi = blockIdx.x < G ? first(blockIdx.x + 1) : total;
  }
  __device__ unsigned first(unsigned b) const {
    return (unsigned)((unsigned long long)total * b / G);
  }
  // The block whose run holds unit u: the largest b with first(b) <= u.
  __device__ unsigned owner(unsigned u) const {
    return (unsigned)(((unsigned long long)(u + 1) * G - 1) / total);
  }
};
struct Seg {
  int j, nt, kb0, kb1;  // expert of the list, tile, chunks [kb0, kb1)
  unsigned at, end;
  __device__ explicit Seg(const Run &r) : at(r.lo), end(r.hi) { set(r); }
  __device__ void set(const Run &r) {
    if (at >= end) return;
    const unsigned tile = at / r.KC;
    j = (int)(tile / r.NT);
    nt = (int)(tile - (unsigned)j * r.NT);
    kb0 = (int)(at - tile * r.KC);
    kb1 = (int)min((unsigned)r.KC, kb0 + (end - at));
  }
  __device__ bool more() const { return at < end; }
  __device__ void next(const Run &r) {
    at += kb1 - kb0;
    set(r);
  }
};

__device__ __forceinline__ void tma_load_3d_first(void *dst, const CUtensorMap *map, uint64_t *bar,
                                                  int x, int y, int z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

template <bool FP8>
__device__ __forceinline__ uint32_t few_desc(int n, uint32_t id) {
  const uint32_t shape = (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
  if constexpr (FP8) return shape | 1u << 23 | id << 4 | id << 29;  // e4m3, K-major, UE8M0
  // fp32 sums of bf16; the weights MN-major, the rows K-major.
  return shape | 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15;
}
template <bool FP8>
__device__ __forceinline__ void few_mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t acc) {
  if constexpr (FP8)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X"
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void few_scales(uint32_t tmem, uint32_t smem) {
  const uint64_t d = (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 |
                     (uint64_t)1 << 46;
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}
// The routing's results, from L2. Layer 2 reads them before it waits for layer 1: all of
// layer 1's threads wait for the routing launch before they let layer 2 start, and
// a launch that was waited for has its writes performed for the whole GPU, so L2 has
// them; only a copy in an SM's L1 could be older, which these loads do not read.
__device__ __forceinline__ int experts_in_use(const FewParams &p) { return __ldcg(p.counters); }
__device__ __forceinline__ int4 expert_of(const FewParams &p, int j) { return __ldcg(p.list + j); }
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// tmA, tmA3: weights (bf16: [E, K, N], box [1, 64, 64]; e4m3: [E, N, K], box [1,
// 128, 128]; layer 2: tmA3 is tmA). tmB: the packed rows, box [16, 128 bytes].
template <int LAYER, int ACT, bool FP8>
__global__ void __launch_bounds__(kThreads, 2)
k_gated_few(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA3,
            const __grid_constant__ CUtensorMap tmB, const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const int stage = kUnit + p.toks * 128, S = p.stages;
  uint8_t *sf = ring + S * stage;  // 8 bits
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  __shared__ uint64_t sf_full[kSfSlots], sf_empty[kSfSlots], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_word;
  __shared__ int joined;
  __shared__ float tops[2][4][16];  // 8 bits: a token's largest of 32 columns
  volatile int *abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t acc_cols = 2 * (uint32_t)p.toks;  // both halves
  const uint32_t need = 2 * acc_cols + (FP8 ? 32 : 0);
  const uint32_t cols = need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
      mbar_init(&sf_full[b], 1);
      mbar_init(&sf_empty[b], 1);
    }
    mbar_init(&drain, 1);
    abort_word = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&tmem_slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // The list is complete: layer 1 follows the routing, layer 2 starts after that.
  if (LAYER == 1) pdl_wait();
  const Run run(experts_in_use(p), p.NT, p.KC);
  tc_fence_before();
  __syncthreads();
  pdl_trigger();  // this block has its TMEM: a dependent one cannot keep it from it
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const auto halves_of = [&](int nt) { return LAYER == 1 || nt * 256 + 128 < p.N ? 2 : 1; };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------- producer
      uint64_t policy;  // weights are read once: what the blocks exchange should stay in L2
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      const auto weights = [&](const Seg &g, const int4 &who, int kb, int s) {
        const int halves = halves_of(g.nt), boxes = (who.z + 15) / 16;
        uint8_t *dst = ring + s * stage;
        mbar_expect_tx(&full[s], halves * kHalf + boxes * 2048);
        for (int q = 0; q < halves; ++q) {
          const CUtensorMap *tm = q ? &tmA3 : &tmA;
          const int n = LAYER == 1 ? g.nt * 128 : g.nt * 256 + q * 128;
          if constexpr (FP8) {
            tma_load_3d_first(dst + q * kHalf, tm, &full[s], kb * 128, n, who.x, policy);
          } else {
            tma_load_3d_first(dst + q * kHalf, tm, &full[s], n, kb * 64, who.x, policy);
            tma_load_3d_first(dst + q * kHalf + kBox, tm, &full[s], n + 64, kb * 64, who.x, policy);
          }
        }
      };
      const auto rows = [&](const int4 &who, int kb, int s) {
        for (int b = 0; b < (who.z + 15) / 16; ++b)
          tma_load_2d(ring + s * stage + kUnit + b * 2048, &tmB, &full[s], kb * (FP8 ? 128 : 64),
                      who.y + b * 16);
      };
      uint32_t it = 0;
      // Layer 2: the first ring of weights before layer 1 is done.
      const uint32_t ahead = LAYER == 2 ? min((uint32_t)S, run.hi - run.lo) : 0;
      if (LAYER == 2) {
        uint32_t i = 0;
        for (Seg g(run); g.more() && i < ahead; g.next(run)) {
          const int4 who = expert_of(p, g.j);
          for (int kb = g.kb0; kb < g.kb1 && i < ahead; ++kb, ++i) weights(g, who, kb, i);
        }
        pdl_wait();
      }
      bool ok = true;
      for (Seg g(run); ok && g.more(); g.next(run)) {
        const int4 who = expert_of(p, g.j);
        for (int kb = g.kb0; kb < g.kb1; ++kb, ++it) {
          const int s = it % S;
          if (it >= ahead) {
            if (!mbar_wait(&empty[s], ((it / S) & 1u) ^ 1u, abort_flag, p.st, 131, p.wait_ns)) {
              ok = false;
              break;
            }
            weights(g, who, kb, s);
          }
          rows(who, kb, s);
        }
      }
      // Copies in flight land before the block leaves (bounded).
      for (uint32_t q = it > (uint32_t)S ? it - S : 0; q < it; ++q)
        mbar_drain(&full[q % S], (q / S) & 1u);
    }
  } else if (warp == 2) {
    // --------------------------------------------------------------- scales
    if constexpr (FP8) {
      if (LAYER == 2) pdl_wait();
      uint32_t g4 = 0;
      bool ok = true;
      for (Seg g(run); ok && g.more(); g.next(run)) {
        const int4 who = expert_of(p, g.j);
        // Lane l < 8: half l / 4's byte of chunk l % 4 of a group of four.
        const int half = (lane >> 2) & 1;
        const int nb = LAYER == 1 ? g.nt : min(2 * g.nt + half, p.NB - 1);
        const uint8_t *sb =
            (LAYER == 1 && half ? p.sb3 : p.sb) + ((size_t)who.x * p.NB + nb) * p.KC;
        for (int k0 = g.kb0 & ~3; k0 < g.kb1; k0 += 4, ++g4) {
          uint32_t a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a[j] = lane + 32 * j < who.z
                       ? p.sa[(size_t)(k0 >> 2) * p.max_rows + who.y + lane + 32 * j]
                       : 0x7f7f7f7fu;
          const int kb = k0 + (lane & 3);
          uint32_t b = lane < 8 && kb < p.KC ? (uint32_t)sb[kb] << 8 * (lane & 3) : 0u;
          b |= __shfl_xor_sync(0xffffffffu, b, 1);
          b |= __shfl_xor_sync(0xffffffffu, b, 2);
          const uint32_t b0 = __shfl_sync(0xffffffffu, b, 0), b1 = __shfl_sync(0xffffffffu, b, 4);
          const int s = g4 % kSfSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(&sf_empty[s], ((g4 / kSfSlots) & 1u) ^ 1u,
                                                 abort_flag, p.st, 132, p.wait_ns));
          if (!ok) break;
          uint4 *out = reinterpret_cast<uint4 *>(sf + s * kSfBytes) + lane;
          out[0] = make_uint4(b0, b0, b0, b0);
          out[32] = make_uint4(b1, b1, b1, b1);
          out[64] = make_uint4(a[0], a[1], a[2], a[3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf_full[s]);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------- MMA issuer
      uint32_t it = 0, g4 = 0;
      int local = 0;
      bool ok = true;
      for (Seg g(run); ok && g.more(); g.next(run), ++local) {
        const int buf = local & 1;
        if (!mbar_wait(&acc_empty[buf], ((local >> 1) & 1u) ^ 1u, abort_flag, p.st, 133, p.wait_ns))
          break;
        tc_fence_after();
        const int n = (expert_of(p, g.j).z + 15) / 16 * 16, halves = halves_of(g.nt);
        const uint32_t d0 = tmem + (uint32_t)buf * acc_cols;
        uint32_t sft = 0;
        for (int kb = g.kb0; kb < g.kb1; ++kb, ++it) {
          if (FP8 && (kb == g.kb0 || (kb & 3) == 0)) {
            const int q = g4 % kSfSlots;
            if (!mbar_wait(&sf_full[q], (g4 / kSfSlots) & 1u, abort_flag, p.st, 134, p.wait_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            sft = tmem + 2 * acc_cols + (g4 & 1u) * 16;
            const uint32_t ss = smem_u32(sf + q * kSfBytes);
            few_scales(sft, ss);
            few_scales(sft + 4, ss + 512);
            few_scales(sft + 8, ss + 1024);
            umma_commit(&sf_empty[q]);
            ++g4;
          }
          const int s = it % S;
          if (!mbar_wait(&full[s], (it / S) & 1u, abort_flag, p.st, 135, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(ring + s * stage), b0 = a0 + kUnit;
          const uint32_t idesc = few_desc<FP8>(n, (uint32_t)kb & 3u);
          for (int q = 0; q < halves; ++q)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const uint32_t aq = a0 + q * kHalf;
              few_mma8<FP8>(d0 + q * p.toks,
                            FP8 ? sdesc(aq + kk * 32, 16, 1024) : sdesc(aq + kk * 2048, kBox, 1024),
                            sdesc(b0 + kk * 32, 16, 1024), idesc, sft + q * 4, sft + 8,
                            (kb > g.kb0 || kk) ? 1u : 0u);
            }
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&acc_full[buf]);
      }
      umma_commit(&drain);
      mbar_drain(&drain, 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // --------------------------------------------------------------- epilogue
    if (LAYER == 2) pdl_wait();
    const int quad = warp & 3, col = quad * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    int local = 0, flip = 0;
    for (Seg g(run); g.more(); g.next(run), ++local) {
      const int buf = local & 1;
      const bool ready = mbar_wait(&acc_full[buf], (local >> 1) & 1u, abort_flag, p.st, 136,
                                   p.wait_ns);
      // All four warps leave together: barriers follow.
      int go;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.red.and.pred q, 2, 128, p;\n"
          " selp.b32 %0, 1, 0, q;\n}\n"
          : "=r"(go)
          : "r"((int)ready)
          : "memory");
      if (!go) break;
      tc_fence_after();
      const int4 who = expert_of(p, g.j);
      const int e = who.x, row0 = who.y, rows = who.z, halves = halves_of(g.nt);
      const uint32_t acc = lanes + (uint32_t)buf * acc_cols;
      const bool whole = g.kb0 == 0 && g.kb1 == run.KC;
      unsigned b0 = 0, b1 = 0;  // the blocks that share the tile
      bool finish = whole;
      if (!whole) {
        const unsigned u = ((unsigned)g.j * run.NT + g.nt) * run.KC;
        b0 = run.owner(u);
        b1 = run.owner(u + run.KC - 1);
        float *out = p.part + ((size_t)blockIdx.x * 2 + (g.kb0 == 0 ? 1 : 0)) * p.toks * 256 + col;
        for (int i0 = 0; i0 < rows; i0 += 16)
          for (int q = 0; q < halves; ++q) {
            uint32_t v[16];
            tmem_ld16(acc + q * p.toks + i0, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i0 + i < rows) out[(i0 + i) * 256 + q * 128] = __uint_as_float(v[i]);
          }
        __threadfence();
        epi_sync();
        if (threadIdx.x == 128) joined = atomicAdd(&p.joins[b0], 1);
        epi_sync();
        finish = joined == (int)(b1 - b0);
        if (finish) __threadfence();
      }
      if (finish) {
        const int n0 = LAYER == 1 ? g.nt * 128 + col : g.nt * 256 + col;
        for (int i0 = 0; i0 < rows; i0 += 16) {
          float v[2][16];
          if (whole) {
            uint32_t u[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              if (q < halves) tmem_ld16(acc + q * p.toks + i0, u);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[q][i] = __uint_as_float(u[i]);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i = 0; i < 16; ++i) v[q][i] = 0.f;
            for (unsigned b = b0; b <= b1; ++b) {
              const float *in = p.part + ((size_t)b * 2 + (b == b0 ? 1 : 0)) * p.toks * 256 + col;
              float w[2][16];
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  w[q][i] =
                      i0 + i < rows && q < halves ? __ldcg(in + (i0 + i) * 256 + q * 128) : 0.f;
#pragma unroll
              for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < 16; ++i) v[q][i] += w[q][i];
            }
          }
          if constexpr (LAYER == 1) {
            const bool in = n0 < p.N;
            const float c1 = p.bias && in ? __bfloat162float(p.bias[(size_t)e * p.N + n0]) : 0.f;
            const float c3 = p.bias3 && in ? __bfloat162float(p.bias3[(size_t)e * p.N + n0]) : 0.f;
            float h[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 p1 = add2(make_float2(v[0][i], v[0][i + 1]), both(c1));
              const float2 p3 = add2(make_float2(v[1][i], v[1][i + 1]), both(c3));
              const float2 r = mul2(gated_act2<ACT, false>(p1, nullptr), p3);
              h[i] = r.x;
              h[i + 1] = r.y;
              if (!FP8 && p.pre1) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                  if (in && i0 + i + u < rows) {
                    const size_t at = (size_t)(row0 + i0 + i + u) * p.N + n0;
                    p.pre1[at] = __float2bfloat16_rn(u ? p1.y : p1.x);
                    p.pre3[at] = __float2bfloat16_rn(u ? p3.y : p3.x);
                  }
              }
            }
            if constexpr (!FP8) {
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (in && i0 + i < rows)
                  p.h[(size_t)(row0 + i0 + i) * p.N + n0] = __float2bfloat16_rn(h[i]);
            } else {
              // A block of 128 columns is the tile: its largest over the four warps.
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                h[i] = in ? __bfloat162float(__float2bfloat16_rn(h[i])) : 0.f;
                float top = fabsf(h[i]);
#pragma unroll
                for (int o = 16; o; o >>= 1)
                  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
                if (lane == 0) tops[flip][quad][i] = top;
              }
              epi_sync();
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (i0 + i >= rows) continue;
                const float top = max_nan(max_nan(tops[flip][0][i], tops[flip][1][i]),
                                          max_nan(tops[flip][2][i], tops[flip][3][i]));
                const uint32_t byte = fp8_scale_byte(top);
                const size_t r = (size_t)row0 + i0 + i;
                p.h8[(r * p.NB + g.nt) * 128 + col] =
                    (uint8_t)fp8_pack2(h[i] * fp8_inverse(byte), 0.f);
                if (col == 0) p.sh[((size_t)(g.nt >> 2) * p.max_rows + r) * 4 + (g.nt & 3)] =
                    (uint8_t)byte;
              }
              flip ^= 1;  // the other's readers are past the next barrier
            }
          } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int n = n0 + q * 128;
              if (q >= halves || n >= p.N) continue;
              const float c = p.bias ? __bfloat162float(p.bias[(size_t)e * p.N + n]) : 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (i0 + i >= rows) continue;
                const size_t r = (size_t)row0 + i0 + i;
                const float u = (v[q][i] + c) * p.row_gate[r];
                if (!isfinite(u)) record_error(p.st, MOE_ERR_NONFINITE, (long long)r);
                if (p.z_bf16)
                  static_cast<__nv_bfloat16 *>(p.z)[r * p.N + n] = __float2bfloat16_rn(u);
                else
                  static_cast<float *>(p.z)[r * p.N + n] = u;
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols)
                 : "memory");
  }
}

// y = x + the kept choices' rows of z, a block for 1024 columns of a token (a
// warp a token, as for long batches, is 10 us for one token of 4096 columns).
// VEC: 8 columns a thread (d a multiple of 8).
template <bool VEC, bool ZB>
__global__ void __launch_bounds__(128)
k_few_gated_combine(int E, int k, int d, const __nv_bfloat16 *x, const void *__restrict__ z,
                    const int32_t *__restrict__ idx, const int32_t *__restrict__ pos,
                    const uint8_t *__restrict__ keep, const int32_t *__restrict__ offset,
                    __nv_bfloat16 *y, DeviceStatus *st) {
  pdl_wait();
  pdl_trigger();
  __shared__ int rows[16];
  const int t = blockIdx.y, tid = threadIdx.x;
  if (tid < k) {
    const int a = t * k + tid, e = idx[a];
    rows[tid] = keep[a] && e >= 0 && e < E ? offset[e] + pos[a] : -1;
  }
  __syncthreads();
  constexpr int V = VEC ? 8 : 1;
  bool bad = false;
  for (int q = 0; q < 8 / V; ++q) {
    const int c = blockIdx.x * 1024 + (q * 128 + tid) * V;
    if (c >= d) break;
    float f[V];
    const size_t at = (size_t)t * d + c;
    if constexpr (VEC) {
      const uint4 u = *reinterpret_cast<const uint4 *>(x + at);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = unpack2(w[j]);
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
      }
    } else {
      f[0] = __bfloat162float(x[at]);
    }
#pragma unroll 4
    for (int j = 0; j < k; ++j) {
      if (rows[j] < 0) continue;
      const size_t r = (size_t)rows[j] * d + c;
      if constexpr (VEC && ZB) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(z) + r);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack2(w[i]);
          f[2 * i] += v.x;
          f[2 * i + 1] += v.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += static_cast<const float *>(z)[r + i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bad |= !isfinite(f[i]);
    if constexpr (VEC) {
      uint4 o;
      o.x = pack_bf16x2(make_float2(f[0], f[1]));
      o.y = pack_bf16x2(make_float2(f[2], f[3]));
      o.z = pack_bf16x2(make_float2(f[4], f[5]));
      o.w = pack_bf16x2(make_float2(f[6], f[7]));
      *reinterpret_cast<uint4 *>(y + at) = o;
    } else {
      y[at] = __float2bfloat16_rn(f[0]);
    }
  }
  if (bad) record_error(st, MOE_ERR_NONFINITE, (long long)t);
}

// ----------------------------------------------------------------------------- host
bool map3(CUtensorMap *m, const void *base, uint64_t x, uint64_t y, uint64_t z, uint32_t bx,
          uint32_t by, bool fp8) {
  auto fn = encode_fn();
  if (!fn) return false;
  const uint64_t es = fp8 ? 1 : 2;
  cuuint64_t dims[3] = {x, y, z}, strides[2] = {x * es, x * y * es};
  cuuint32_t box[3] = {bx, by, 1}, one[3] = {1, 1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_few_rows(CUtensorMap *m, const void *base, uint64_t rows, uint64_t cols, bool fp8) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * (fp8 ? 1 : 2)};
  cuuint32_t box[2] = {fp8 ? 128u : 64u, 16}, one[2] = {1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
            const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int LAYER, int ACT, bool FP8>
cudaError_t run_few(const CUtensorMap &a, const CUtensorMap &a3, const CUtensorMap &b,
                    const FewParams &p, cudaStream_t s) {
  const size_t smem = 1024 + (size_t)p.stages * (kUnit + p.toks * 128) +
                      (FP8 ? kSfSlots * kSfBytes : 0);
  const cudaError_t err = allow_smem(k_gated_few<LAYER, ACT, FP8>, kSmemMost - 2048);
  if (err != cudaSuccess) return err;
  return launch_pdl_c(kPdlGemm, k_gated_few<LAYER, ACT, FP8>, gated_few_blocks(), kThreads, smem, s,
                      a, a3, b, p);
}

template <bool FP8>
cudaError_t few_layer(const GatedFew &q, int layer, cudaStream_t s) {
  const moe_config &c = q.c;
  const int K = layer == 1 ? c.d : c.d_ff, N = layer == 1 ? c.d_ff : c.d;
  const uint64_t Kp = FP8 ? (uint64_t)fp8_blocks(K) * 128 : (uint64_t)K;
  FewParams p{};
  p.KC = (int)((Kp * (FP8 ? 1 : 2) + 127) / 128);
  p.N = N;
  p.NT = layer == 1 ? (N + 127) / 128 : (N + 255) / 256;
  p.toks = q.toks;
  p.stages = (int)((kSmemMost - 2048 - 1024 - kSfSlots * kSfBytes) / (kUnit + q.toks * 128));
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  p.max_rows = q.max_rows;
  p.NB = (int)fp8_blocks(N);
  p.list = q.list;
  p.counters = q.counters;
  p.joins = q.counters + 1 + (layer == 2 ? gated_few_blocks() : 0);
  p.part = q.part;
  p.row_gate = q.row_gate;
  p.bias = static_cast<const __nv_bfloat16 *>(layer == 1 ? q.b1 : q.b2);
  p.bias3 = static_cast<const __nv_bfloat16 *>(q.b3);
  p.h = static_cast<__nv_bfloat16 *>(q.h);
  p.pre1 = static_cast<__nv_bfloat16 *>(q.pre1);
  p.pre3 = static_cast<__nv_bfloat16 *>(q.pre3);
  p.h8 = static_cast<uint8_t *>(q.h);
  p.sh = q.sh;
  p.z = q.z;
  p.z_bf16 = q.z_bf16 ? 1 : 0;
  p.sa = reinterpret_cast<const uint32_t *>(layer == 1 ? q.sx : q.sh);
  p.sb = layer == 1 ? q.s1 : q.s2;
  p.sb3 = q.s3;
  p.st = q.st;
  p.wait_ns = wait_limit_ns();
  const void *W = layer == 1 ? q.W1 : q.W2, *W3 = layer == 1 ? q.W3 : q.W2;
  CUtensorMap a, a3, b;
  const bool maps =
      FP8 ? map3(&a, W, Kp, N, c.E, 128, 128, true) && map3(&a3, W3, Kp, N, c.E, 128, 128, true)
          : map3(&a, W, N, K, c.E, 64, 64, false) && map3(&a3, W3, N, K, c.E, 64, 64, false);
  if (!maps || !map_few_rows(&b, layer == 1 ? q.xbuf : q.h, (uint64_t)q.max_rows, Kp, FP8))
    return cudaErrorInvalidValue;
  if (layer == 2) return run_few<2, 0, FP8>(a, a3, b, p, s);
  return gated_dispatch(q.activation, [&](auto act) {
    return run_few<1, decltype(act)::value, FP8>(a, a3, b, p, s);
  });
}

}  // namespace

int gated_few_blocks() {
  const int n = sm_count();
  return n < kGatedFewMaxBlocks ? n : kGatedFewMaxBlocks;
}

cudaError_t launch_gated_few(const GatedFew &q, cudaStream_t s) {
  const moe_config &c = q.c;
  const RouteArgs r{c.T * c.k, c.E, q.C, c.k, c.d, q.max_rows, 1 + 2 * gated_few_blocks(), q.idx,
                    q.gate, static_cast<const __nv_bfloat16 *>(q.x), q.pos, q.keep, q.offset,
                    q.row_gate, q.list, q.counters, q.xbuf, q.sx, q.st};
  const size_t smem = (size_t)c.E * 4;
  cudaError_t err = q.fp8 ? launch_pdl(k_few_gated_route<true>, r.A, 256, smem, s, r)
                          : launch_pdl(k_few_gated_route<false>, r.A, 256, smem, s, r);
  if (err == cudaSuccess) err = q.fp8 ? few_layer<true>(q, 1, s) : few_layer<false>(q, 1, s);
  if (err == cudaSuccess) err = q.fp8 ? few_layer<true>(q, 2, s) : few_layer<false>(q, 2, s);
  if (err != cudaSuccess) return err;
  const auto combine = [&](auto kernel) {
    return launch_pdl_c(kPdlCombine, kernel, dim3((c.d + 1023) / 1024, c.T), 128, 0, s, c.E, c.k,
                        c.d, static_cast<const __nv_bfloat16 *>(q.x), (const void *)q.z, q.idx,
                        (const int32_t *)q.pos, (const uint8_t *)q.keep, (const int32_t *)q.offset,
                        static_cast<__nv_bfloat16 *>(q.y), q.st);
  };
  if (q.z_bf16) return combine(k_few_gated_combine<true, true>);
  return c.d % 8 == 0 ? combine(k_few_gated_combine<true, false>)
                      : combine(k_few_gated_combine<false, false>);
}

}  // namespace moe
