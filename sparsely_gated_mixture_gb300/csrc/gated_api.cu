// C ABI of the gated experts (declared in include/moe.h): argument checks,
// workspace layouts and the order of launches. No computation happens here.
#include "api.cuh"
#include "gated.cuh"

namespace moe {

// Rows that any call has at most.
static long long gated_max_rows(const moe_config &c) {
  const long long A = (long long)c.T * c.k, full = (long long)c.E * host_capacity(c);
  return A < full ? A : full;
}

static int check_gated(const moe_config *c) {
  const int r = check_cfg(c);
  if (r != MOE_OK) return r;
  if (c->d > MOE_GATED_MAX_WIDTH || c->d_ff > MOE_GATED_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
  // Kernels count warps of 128 columns of a row in 32 bits, and step over rows, a
  // few hundred at a time, in as many with a sign.
  const long long w = fp8_blocks(c->d > c->d_ff ? c->d : c->d_ff), rows = gated_max_rows(*c);
  return rows * w < (1ll << 32) && rows <= (1ll << 31) - 1024 ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// What routing needs, at the start of every gated workspace.
struct GatedRoute {
  size_t status, hist, chunk_base, count, offset, mtiles, pos, keep, row_token, row_gate;
  int n_chunks;
};

struct GatedTake {
  size_t off = 0;
  size_t operator()(size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  }
};

static GatedRoute gated_route(const moe_config &c, GatedTake &take) {
  GatedRoute L{};
  const size_t A = (size_t)c.T * c.k, E = c.E;
  L.n_chunks = (int)((A + kSlotChunk - 1) / kSlotChunk);
  L.status = take(sizeof(DeviceStatus));
  L.hist = take((size_t)L.n_chunks * E * 4);
  L.chunk_base = take((size_t)L.n_chunks * E * 4);
  L.count = take(E * 4);
  L.offset = take((E + 1) * 4);
  L.mtiles = take((E + 1) * 4);
  L.pos = take(A * 4);
  L.keep = take(A);
  L.row_token = take(A * 4);
  L.row_gate = take(A * 4);
  return L;
}

// The products run on the tensor cores for bf16 layers whose widths are
// multiples of 64, else on the CUDA cores.
static bool gated_tc_shape(const moe_config &c) {
  return c.act_dtype == MOE_BF16 && c.d % 64 == 0 && c.d_ff % 64 == 0;
}
// The experts' outputs in bf16 before the combine, where that reads 16 bytes
// at a time: half the bytes of moe_expert_ffn's fp32 rows, one more rounding a
// term, as in moe_forward.
static bool gated_z_bf16(const moe_config &c) { return gated_tc_shape(c) && c.k <= 4; }

// Few rows an expert: the kernels that are bound by reading the weights once.
static int gated_few_toks(const moe_config &c) {
  const long long A = (long long)c.T * c.k, C = host_capacity(c), rows = A < C ? A : C;
  if (A > kGatedFewChoices || rows > kGatedFewRows) return 0;
  return (int)((rows + 15) / 16 * 16);
}
// In bf16 the kernels for long batches read the weights as fast (64 tokens
// through 8 large experts 419 us against 437) once the experts in use, at
// uniform choices, have tiles of layer 2 for three quarters of the SMs; with
// fewer they leave most of them idle (one token 227 us against 127). In 8 bits
// they do not (64 tokens 253 us against 235; 64 tokens through 16 experts of 512 x 1024
// 36 either way). Many narrow experts do better by these kernels beyond the rule too
// (top-8 of experts of 2048 x 1024, bf16: 64 tokens through 64 of them 178 us against
// 147, through 256 409 against 385).
static bool gated_few_pays(const moe_config &c) {
  if (!gated_few_toks(c)) return false;
  const double used = c.E * (1.0 - pow(1.0 - (double)c.k / c.E, (double)c.T));
  return used * ((c.d + 255) / 256) < 0.75 * gated_few_blocks();
}
struct GatedFewLayout {
  size_t list, counters, part;
};
static GatedFewLayout gated_few_layout(const moe_config &c, GatedTake &take) {
  const size_t toks = (size_t)gated_few_toks(c), blocks = kGatedFewMaxBlocks;
  GatedFewLayout L{};
  L.list = take(toks ? (size_t)c.T * c.k * sizeof(int4) : 0);
  L.counters = take(toks ? (1 + 2 * blocks) * 4 : 0);
  L.part = take(blocks * 2 * toks * 256 * 4);
  return L;
}

struct GatedLayout {
  GatedRoute r;
  GatedFewLayout few;
  size_t xbuf, h, z, part, part2, total;
};
static GatedLayout gated_layout(const moe_config &c) {
  GatedLayout L{};
  GatedTake take;
  const size_t R = (size_t)gated_max_rows(c);
  L.r = gated_route(c, take);
  L.xbuf = take(gated_tc_shape(c) ? R * c.d * 2 : 0);
  L.h = take(R * c.d_ff * elem_bytes(c.act_dtype));
  L.z = take(R * c.d * (gated_z_bf16(c) ? 2 : 4));
  if (gated_tc_shape(c)) {
    L.few = gated_few_layout(c, take);
  } else if (gated_few_toks(c)) {
    L.part = take(gated_few_simt_part(c, (int)R, 1));
    L.part2 = take(gated_few_simt_part(c, (int)R, 2));
  }
  L.total = take.off;
  return L;
}

static bool gated_fp8_z_bf16(const moe_config &c) { return c.d % 8 == 0 && c.k <= 4; }

struct GatedFp8Layout {
  GatedRoute r;
  GatedFewLayout few;
  size_t x8, sx, h8, sh, z, total;
};
static GatedFp8Layout gated_fp8_layout(const moe_config &c) {
  GatedFp8Layout L{};
  GatedTake take;
  const size_t R = (size_t)gated_max_rows(c);
  const size_t db = (size_t)fp8_blocks(c.d), fb = (size_t)fp8_blocks(c.d_ff);
  L.r = gated_route(c, take);
  L.x8 = take(R * db * kFp8Block);
  L.sx = take(R * ((db + 3) / 4 * 4));
  L.h8 = take(R * fb * kFp8Block);
  L.sh = take(R * ((fb + 3) / 4 * 4));
  L.z = take(R * c.d * (gated_fp8_z_bf16(c) ? 2 : 4));
  L.few = gated_few_layout(c, take);
  L.total = take.off;
  return L;
}

// Tensor cores: xbuf and h are packed rows (64 more than there can be, for the
// zeroed tail that the weight gradients read; h's are gate * h), dY, dP1, dP3 and
// dX rows of padded blocks (offsets poff). CUDA cores: fp32 packed rows, dU = gate *
// dy in dY's place.
struct GatedBwdLayout {
  GatedRoute r;
  size_t poff, xbuf, h, dY, dU, dP1, dP3, dX, dgpart, wpart, total;
  long long P_max;
  int dg_blocks;
};
static GatedBwdLayout gated_bwd_layout(const moe_config &c) {
  GatedBwdLayout L{};
  GatedTake take;
  const bool tc = gated_tc_shape(c);
  const size_t R = (size_t)gated_max_rows(c), d = c.d, F = c.d_ff;
  L.P_max = (long long)R + (tc ? (long long)kBwdRowPad * c.E : 0);
  const size_t P = (size_t)L.P_max, eb = tc ? 2 : 4;
  L.r = gated_route(c, take);
  L.dg_blocks = tc ? 2 * ((c.d_ff + 255) / 256) : gated_simt_dg_blocks(c, (int)R);
  L.poff = take(((size_t)c.E + 1) * 4);
  L.xbuf = take(tc ? (R + kBwdRowPad) * d * 2 : R * d * 4);
  L.h = take((R + (tc ? kBwdRowPad : 0)) * F * eb);
  L.dY = take(tc ? P * d * 2 : 0);
  L.dU = take(tc ? 0 : P * d * 4);
  L.dP1 = take(P * F * eb);
  L.dP3 = take(P * F * eb);
  L.dX = take(P * d * 4);
  L.dgpart = take(P * L.dg_blocks * 4);
  L.wpart = take(tc ? 0 : gated_simt_wpart(c, (int)R));
  L.total = take.off;
  return L;
}

// The status cleared and the choices' slots; pos and keep go to the caller's
// arrays where given. poff: the backward's padded offsets, or null.
static int gated_slots(const moe_config &c, const GatedRoute &L, const int32_t *idx,
                       const float *gate, int32_t *pos, uint8_t *keep, int32_t *poff, void *ws,
                       cudaStream_t s) {
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.status);
  if ((long long)c.T * c.k <= kRouteMost) {
    MOE_CUDA(launch_gated_route({c.T * c.k, c.E, host_capacity(c), idx, gate, pos, keep,
                                 ws_at<int32_t>(ws, L.offset), ws_at<int32_t>(ws, L.mtiles), poff,
                                 ws_at<int32_t>(ws, L.row_token), ws_at<float>(ws, L.row_gate),
                                 st}, s));
    return MOE_OK;
  }
  MOE_CUDA(launch_gated_begin(st, s));
  MOE_CUDA(launch_slots(c, host_capacity(c), idx, gate, ws_at<int32_t>(ws, L.hist),
                        ws_at<int32_t>(ws, L.chunk_base), ws_at<int32_t>(ws, L.count),
                        ws_at<int32_t>(ws, L.offset), ws_at<int32_t>(ws, L.mtiles), pos, keep,
                        ws_at<int32_t>(ws, L.row_token), ws_at<float>(ws, L.row_gate), L.n_chunks,
                        st, s));
  if (poff) MOE_CUDA(launch_bwd_offsets(c.E, ws_at<int32_t>(ws, L.offset), poff, s));
  return MOE_OK;
}

static GatedRows gated_rows(const GatedRoute &L, void *ws) {
  return {ws_at<int32_t>(ws, L.offset), ws_at<int32_t>(ws, L.mtiles),
          ws_at<int32_t>(ws, L.row_token), ws_at<float>(ws, L.row_gate)};
}

// The backward's products on the tensor cores, dx included.
struct GatedBwdCall {
  int activation;
  const void *x;
  const int32_t *idx;
  const void *pre1, *pre3, *W1, *W3, *W2, *b2, *dy;
  void *dx;
  float *dgate;
  void *dW1, *db1, *dW3, *db3, *dW2, *db2;
};
static int gated_backward_tc(const moe_config &c, const GatedBwdLayout &L, const GatedBwdCall &q,
                             void *ws, cudaStream_t s) {
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.r.status);
  const GatedRows rows = gated_rows(L.r, ws);
  const int32_t *pos = ws_at<int32_t>(ws, L.r.pos);
  const uint8_t *keep = ws_at<uint8_t>(ws, L.r.keep);
  const int32_t *poff = ws_at<int32_t>(ws, L.poff);
  void *xbuf = ws_at<char>(ws, L.xbuf), *h = ws_at<char>(ws, L.h);
  void *dY = ws_at<char>(ws, L.dY);
  void *dP1 = ws_at<char>(ws, L.dP1), *dP3 = ws_at<char>(ws, L.dP3);
  float *dX = ws_at<float>(ws, L.dX), *dgpart = ws_at<float>(ws, L.dgpart);
  const long long R = gated_max_rows(c), cap = host_capacity(c);
  MOE_CUDA(launch_gated_gather(c, L.P_max, rows, poff, q.x, q.dy, xbuf, h, dY, s));
  // dgate's partials are of D as the tensor cores sum it: in fp32, cut at each add of
  // 16 products, some 5e-6 too small at d = 4096 (moe_backward's dL/dgate alike).
  BwdGemm g{3, c.d, c.d_ff, 0, c.E, L.P_max, 0, 0, dY, q.W2, rows.offset, poff, rows.row_gate,
            nullptr, dP1, dgpart, false};
  g.activation = q.activation;
  g.pre1 = q.pre1;
  g.pre3 = q.pre3;
  g.out3 = dP3;
  g.h = h;
  MOE_CUDA(launch_bwd_gemm(g, st, s));
  // Beside the products that follow, on the library's side stream: dL/dgate and
  // the bias gradients, whose small blocks fit next to the GEMMs' one an SM.
  std::unique_lock<std::mutex> side_lock;
  SideFork side;
  side.use(side_stream(side_lock, s), s);
  const int r = side.fork();
  if (r != MOE_OK) return r;
  const cudaStream_t fs = side.stream();
  MOE_CUDA(launch_gated_dgate(c, L.dg_blocks, q.idx, pos, keep, poff, dgpart, q.dy, q.b2, q.dgate,
                              fs));
  MOE_CUDA(launch_gated_colsum(c, false, rows.offset, poff, dY, rows.row_gate, q.db2, dP1, q.db1,
                               dP3, q.db3, fs));
  BwdGemm gx{4, c.d_ff, c.d, 0, c.E, L.P_max, 0, 0, dP1, q.W1, rows.offset, poff, nullptr, nullptr,
             dX, nullptr, false};
  gx.A3 = dP3;
  gx.B3 = q.W3;
  // The pairs' lower traffic pays from one wave on (top-4 layer's backward 229 us
  // with none of them, 219 with dX's and the weight gradients', 226 with all; none,
  // all and by this rule, top-2 of 8 experts: 4096 tokens of 1024 x 2048 259, 251,
  // 243; 8192 of 768 x 2048 365, 346, 331; 8192 of 2048 x 4096 1238, 1105, 1104; 1024 of
  // 4096 x 14336, whose weight gradients have short sums, 2077, 1761, 1959; 2048
  // tokens, top-2 of 32 of 1024 x 2048: 310, 313, 297).
  gx.pair_waves = 1;
  MOE_CUDA(launch_bwd_gemm(gx, st, s));
  const auto wgrad = [&](const void *A, int M, const void *B, int N, void *out) {
    BwdGemm w{2, 0, N, M, c.E, R, L.P_max, cap, A, B, rows.offset, poff, nullptr, nullptr, out,
              nullptr, true};
    w.pair_waves = 1;
    return launch_bwd_gemm(w, st, s);
  };
  MOE_CUDA(wgrad(h, c.d_ff, dY, c.d, q.dW2));
  MOE_CUDA(wgrad(xbuf, c.d, dP1, c.d_ff, q.dW1));
  MOE_CUDA(wgrad(xbuf, c.d, dP3, c.d_ff, q.dW3));
  if (side.join() != MOE_OK) return MOE_ERR_CUDA;
  MOE_CUDA(launch_bwd_dx(c, q.idx, pos, keep, poff, dX, nullptr, q.dy, q.dx, s));
  return MOE_OK;
}

// What the few-row kernels take from the routing part of a workspace.
static GatedFew gated_few(const moe_config &c, const GatedRoute &L, const GatedFewLayout &F,
                          int activation, const void *x, const int32_t *idx, const float *gate,
                          int32_t *pos, uint8_t *keep, void *ws) {
  GatedFew q{};
  q.c = c;
  q.activation = activation;
  q.C = host_capacity(c);
  q.max_rows = (int)gated_max_rows(c);
  q.toks = gated_few_toks(c);
  q.x = x;
  q.idx = idx;
  q.gate = gate;
  q.pos = pos;
  q.keep = keep;
  q.offset = ws_at<int32_t>(ws, L.offset);
  q.row_gate = ws_at<float>(ws, L.row_gate);
  q.list = ws_at<int4>(ws, F.list);
  q.counters = ws_at<int32_t>(ws, F.counters);
  q.part = ws_at<float>(ws, F.part);
  q.st = ws_at<DeviceStatus>(ws, L.status);
  return q;
}

static bool known_activation(int a) {
  return a == MOE_ACT_SILU || a == MOE_ACT_GELU || a == MOE_ACT_RELU;
}

static int check_weights_fp8(int32_t E, int32_t K, int32_t N) {
  if (E < 1 || K < 1 || N < 1) return MOE_ERR_ARG;
  // The grid's y and z extents.
  return E <= 1024 && K <= MOE_GATED_MAX_WIDTH && N <= MOE_GATED_MAX_WIDTH ? MOE_OK
                                                                          : MOE_ERR_UNSUPPORTED;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_gated_workspace_size(const moe_config *cfg, size_t *bytes) {
  const int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (!bytes) return MOE_ERR_ARG;
  *bytes = gated_layout(*cfg).total;
  return MOE_OK;
}

int moe_experts_gated(const moe_config *cfg, int32_t activation, const void *x,
                      const int32_t *expert_idx, const float *gate, const void *W1,
                      const void *b1, const void *W3, const void *b3, const void *W2,
                      const void *b2, void *y, void *pre1, void *pre3, int32_t *pos,
                      uint8_t *keep, void *ws, moe_stream_t stream) {
  int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (!known_activation(activation)) return MOE_ERR_ARG;
  MOE_REQ(x); MOE_REQ(expert_idx); MOE_REQ(gate); MOE_REQ(W1); MOE_OPT(b1); MOE_REQ(W3);
  MOE_OPT(b3); MOE_REQ(W2); MOE_OPT(b2); MOE_REQ(y); MOE_OPT(pre1); MOE_OPT(pre3);
  MOE_OPT(pos); MOE_OPT(keep);
  if (!ws || !aligned(ws, 256)) return MOE_ERR_ARG;
  if ((pre1 == nullptr) != (pre3 == nullptr)) return MOE_ERR_ARG;
  const moe_config &c = *cfg;
  if (gated_tc_shape(c) && !ffn_tc_supported(c)) return MOE_ERR_UNSUPPORTED;
  const GatedLayout L = gated_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.r.status);
  int32_t *ps = pos ? pos : ws_at<int32_t>(ws, L.r.pos);
  uint8_t *kp = keep ? keep : ws_at<uint8_t>(ws, L.r.keep);
  const long long R = gated_max_rows(c);
  void *z = ws_at<char>(ws, L.z);
  if (gated_tc_shape(c) && gated_few_pays(c)) {
    GatedFew q = gated_few(c, L.r, L.few, activation, x, expert_idx, gate, ps, kp, ws);
    q.W1 = W1; q.b1 = b1; q.W3 = W3; q.b3 = b3; q.W2 = W2; q.b2 = b2;
    q.xbuf = ws_at<char>(ws, L.xbuf);
    q.h = ws_at<char>(ws, L.h);
    q.pre1 = pre1;
    q.pre3 = pre3;
    q.z = z;
    q.z_bf16 = gated_z_bf16(c);
    q.y = y;
    MOE_CUDA(launch_gated_few(q, s));
    return MOE_OK;
  }
  r = gated_slots(c, L.r, expert_idx, gate, ps, kp, nullptr, ws, s);
  if (r != MOE_OK) return r;
  if (gated_tc_shape(c)) {
    const GatedRows rows = gated_rows(L.r, ws);
    void *xbuf = ws_at<char>(ws, L.xbuf), *h = ws_at<char>(ws, L.h);
    const int C = host_capacity(c);
    const bool zb = gated_z_bf16(c);
    MOE_CUDA(launch_gather(c, x, rows.offset, rows.row_token, xbuf, st, s));
    MOE_CUDA(launch_gated_tc_layer1(c, C, activation, R, xbuf, rows.offset, W1, b1, W3, b3, h,
                                    pre1, pre3, st, s));
    MOE_CUDA(launch_ffn_layer2(c, C, R, h, rows.offset, rows.row_gate, W2, b2, z, zb, st, s));
    MOE_CUDA(launch_combine(c, x, z, zb, ps, kp, expert_idx, rows.offset, y, st, s));
    return MOE_OK;
  }
  if (gated_few_toks(c)) {
    GatedFewSimt p{};
    p.c = c;
    p.activation = activation;
    p.max_rows = (int)R;
    p.rows = gated_rows(L.r, ws);
    p.x = x;
    p.idx = expert_idx;
    p.pos = ps;
    p.keep = kp;
    p.gate = gate;
    p.W1 = W1; p.b1 = b1; p.W3 = W3; p.b3 = b3; p.W2 = W2; p.b2 = b2;
    p.h = ws_at<char>(ws, L.h);
    p.pre1 = pre1;
    p.pre3 = pre3;
    p.y = y;
    p.part = ws_at<float>(ws, L.part);
    p.part2 = ws_at<float>(ws, L.part2);
    p.st = st;
    MOE_CUDA(launch_gated_few_simt(p, s));
    return MOE_OK;
  }
  GatedSimt p{};
  p.c = c;
  p.activation = activation;
  p.max_rows = (int)R;
  p.rows = gated_rows(L.r, ws);
  p.x = x;
  p.W1 = W1; p.b1 = b1; p.W3 = W3; p.b3 = b3; p.W2 = W2; p.b2 = b2;
  p.h = ws_at<char>(ws, L.h);
  p.pre1 = pre1;
  p.pre3 = pre3;
  p.z = static_cast<float *>(z);
  p.st = st;
  MOE_CUDA(launch_gated_simt_forward(p, s));
  if (c.d % 4 == 0)
    MOE_CUDA(launch_combine(c, x, p.z, false, ps, kp, expert_idx, p.rows.offset, y, st, s));
  else
    MOE_CUDA(launch_gated_combine(c, x, p.z, expert_idx, ps, kp, p.rows.offset, y, st, s));
  return MOE_OK;
}

int moe_gated_backward_workspace_size(const moe_config *cfg, size_t *bytes) {
  const int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (!bytes) return MOE_ERR_ARG;
  *bytes = gated_bwd_layout(*cfg).total;
  return MOE_OK;
}

int moe_experts_gated_backward(const moe_config *cfg, int32_t activation, const void *x,
                               const int32_t *expert_idx, const float *gate, const void *pre1,
                               const void *pre3, const void *W1, const void *W3, const void *W2,
                               const void *b2, const void *dy, void *dx, float *dgate, void *dW1,
                               void *db1, void *dW3, void *db3, void *dW2, void *db2, void *ws,
                               moe_stream_t stream) {
  int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (!known_activation(activation)) return MOE_ERR_ARG;
  MOE_REQ(x); MOE_REQ(expert_idx); MOE_REQ(gate); MOE_REQ(pre1); MOE_REQ(pre3); MOE_REQ(W1);
  MOE_REQ(W3); MOE_REQ(W2); MOE_OPT(b2); MOE_REQ(dy); MOE_REQ(dx); MOE_REQ(dgate);
  MOE_REQ(dW1); MOE_OPT(db1); MOE_REQ(dW3); MOE_OPT(db3); MOE_REQ(dW2); MOE_OPT(db2);
  if (!ws || !aligned(ws, 256)) return MOE_ERR_ARG;
  const moe_config &c = *cfg;
  if (gated_tc_shape(c) && !bwd_tc_supported(c)) return MOE_ERR_UNSUPPORTED;
  const GatedBwdLayout L = gated_bwd_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  int32_t *pos = ws_at<int32_t>(ws, L.r.pos);
  uint8_t *keep = ws_at<uint8_t>(ws, L.r.keep);
  r = gated_slots(c, L.r, expert_idx, gate, pos, keep,
                  gated_tc_shape(c) ? ws_at<int32_t>(ws, L.poff) : nullptr, ws, s);
  if (r != MOE_OK) return r;
  if (gated_tc_shape(c)) {
    const GatedBwdCall q{activation, x, expert_idx, pre1, pre3, W1, W3, W2, b2, dy, dx,
                         dgate, dW1, db1, dW3, db3, dW2, db2};
    return gated_backward_tc(c, L, q, ws, s);
  }
  GatedSimt p{};
  p.c = c;
  p.activation = activation;
  p.max_rows = (int)gated_max_rows(c);
  p.rows = gated_rows(L.r, ws);
  p.x = x;
  p.W1 = W1; p.W3 = W3; p.W2 = W2; p.b2 = b2;
  p.pre1 = const_cast<void *>(pre1);
  p.pre3 = const_cast<void *>(pre3);
  p.dy = dy;
  p.xf = ws_at<float>(ws, L.xbuf);
  p.hf = ws_at<float>(ws, L.h);
  p.dU = ws_at<float>(ws, L.dU);
  p.dP1 = ws_at<float>(ws, L.dP1);
  p.dP3 = ws_at<float>(ws, L.dP3);
  p.dX = ws_at<float>(ws, L.dX);
  p.dgpart = ws_at<float>(ws, L.dgpart);
  p.wpart = ws_at<float>(ws, L.wpart);
  p.dW1 = dW1; p.dW3 = dW3; p.dW2 = dW2;
  p.st = ws_at<DeviceStatus>(ws, L.r.status);
  MOE_CUDA(launch_gated_simt_front(p, s));
  // The weight gradients beside all that dx needs, and the small sums.
  std::unique_lock<std::mutex> side_lock;
  SideFork side;
  side.use(side_stream(side_lock, s), s);
  r = side.fork();
  if (r != MOE_OK) return r;
  const cudaStream_t fs = side.stream();
  const int32_t *off = p.rows.offset;
  MOE_CUDA(launch_gated_simt_weights(p, fs));
  MOE_CUDA(launch_gated_simt_dx(p, s));
  MOE_CUDA(launch_gated_dgate(c, L.dg_blocks, expert_idx, pos, keep, off, p.dgpart, dy, b2, dgate,
                              s));
  MOE_CUDA(launch_gated_colsum(c, true, off, off, p.dU, nullptr, db2, p.dP1, db1, p.dP3, db3, fs));
  MOE_CUDA(launch_gated_dx(c, expert_idx, pos, keep, off, p.dX, dy, dx, s));
  return side.join();
}

int moe_weights_fp8_size(int32_t E, int32_t K, int32_t N, size_t *w8_bytes,
                         size_t *wscale_bytes) {
  const int r = check_weights_fp8(E, K, N);
  if (r != MOE_OK) return r;
  if (!w8_bytes || !wscale_bytes) return MOE_ERR_ARG;
  const size_t KB = (size_t)fp8_blocks(K);
  *w8_bytes = (size_t)E * N * KB * kFp8Block;
  *wscale_bytes = (size_t)E * (size_t)fp8_blocks(N) * KB;
  return MOE_OK;
}

int moe_weights_fp8(int32_t E, int32_t K, int32_t N, int32_t dtype, const void *W, uint8_t *w8,
                    uint8_t *wscale, void *ws, moe_stream_t stream) {
  const int r = check_weights_fp8(E, K, N);
  if (r != MOE_OK) return r;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_ARG;
  MOE_REQ(W); MOE_REQ(w8); MOE_REQ(wscale);
  if (!ws || !aligned(ws, 256)) return MOE_ERR_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  MOE_CUDA(launch_fp8_weights(dtype == MOE_BF16, E, K, N, W, w8, wscale,
                              ws_at<DeviceStatus>(ws, 0), s));
  return MOE_OK;
}

int moe_gated_fp8_workspace_size(const moe_config *cfg, size_t *bytes) {
  const int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (cfg->act_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!bytes) return MOE_ERR_ARG;
  *bytes = gated_fp8_layout(*cfg).total;
  return MOE_OK;
}

int moe_experts_gated_fp8(const moe_config *cfg, int32_t activation, const void *x,
                          const int32_t *expert_idx, const float *gate, const uint8_t *W1,
                          const uint8_t *s1, const void *b1, const uint8_t *W3,
                          const uint8_t *s3, const void *b3, const uint8_t *W2,
                          const uint8_t *s2, const void *b2, void *y, int32_t *pos,
                          uint8_t *keep, void *ws, moe_stream_t stream) {
  int r = check_gated(cfg);
  if (r != MOE_OK) return r;
  if (cfg->act_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (!known_activation(activation)) return MOE_ERR_ARG;
  MOE_REQ(x); MOE_REQ(expert_idx); MOE_REQ(gate); MOE_REQ(W1); MOE_REQ(s1); MOE_OPT(b1);
  MOE_REQ(W3); MOE_REQ(s3); MOE_OPT(b3); MOE_REQ(W2); MOE_REQ(s2); MOE_OPT(b2); MOE_REQ(y);
  MOE_OPT(pos); MOE_OPT(keep);
  if (!ws || !aligned(ws, 256)) return MOE_ERR_ARG;
  const moe_config &c = *cfg;
  if (!fp8_tc_supported()) return MOE_ERR_UNSUPPORTED;
  const GatedFp8Layout L = gated_fp8_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.r.status);
  int32_t *ps = pos ? pos : ws_at<int32_t>(ws, L.r.pos);
  uint8_t *kp = keep ? keep : ws_at<uint8_t>(ws, L.r.keep);
  const int R = (int)gated_max_rows(c);
  uint8_t *x8 = ws_at<uint8_t>(ws, L.x8), *sx = ws_at<uint8_t>(ws, L.sx);
  uint8_t *h8 = ws_at<uint8_t>(ws, L.h8), *sh = ws_at<uint8_t>(ws, L.sh);
  void *z = ws_at<char>(ws, L.z);
  const bool zb = gated_fp8_z_bf16(c);
  if (gated_few_toks(c)) {
    GatedFew q = gated_few(c, L.r, L.few, activation, x, expert_idx, gate, ps, kp, ws);
    q.fp8 = true;
    q.W1 = W1; q.s1 = s1; q.b1 = b1; q.W3 = W3; q.s3 = s3; q.b3 = b3;
    q.W2 = W2; q.s2 = s2; q.b2 = b2;
    q.xbuf = x8;
    q.sx = sx;
    q.h = h8;
    q.sh = sh;
    q.z = z;
    q.z_bf16 = zb;
    q.y = y;
    MOE_CUDA(launch_gated_few(q, s));
    return MOE_OK;
  }
  r = gated_slots(c, L.r, expert_idx, gate, ps, kp, nullptr, ws, s);
  if (r != MOE_OK) return r;
  const GatedRows rows = gated_rows(L.r, ws);
  MOE_CUDA(launch_fp8_rows(R, c.d, c.k, rows.offset + c.E, rows.row_token, x, x8, sx, s));
  MOE_CUDA(launch_fp8_tc({c, 1, activation, R, rows.offset, nullptr, x8, sx, W1, s1, W3, s3, b1,
                          b3, h8, sh, nullptr, false, st}, s));
  MOE_CUDA(launch_fp8_tc({c, 2, activation, R, rows.offset, rows.row_gate, h8, sh, W2, s2, nullptr,
                          nullptr, b2, nullptr, nullptr, nullptr, z, zb, st}, s));
  MOE_CUDA(launch_combine(c, x, z, zb, ps, kp, expert_idx, rows.offset, y, st, s));
  return MOE_OK;
}

}  // extern "C"
