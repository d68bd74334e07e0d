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
  // Kernels count warps of 128 columns of a row in 32 bits.
  const long long w = fp8_blocks(c->d > c->d_ff ? c->d : c->d_ff);
  return gated_max_rows(*c) * w < (1ll << 32) ? MOE_OK : MOE_ERR_UNSUPPORTED;
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

struct GatedLayout {
  GatedRoute r;
  size_t h, z, total;
};
static GatedLayout gated_layout(const moe_config &c) {
  GatedLayout L{};
  GatedTake take;
  const size_t R = (size_t)gated_max_rows(c);
  L.r = gated_route(c, take);
  L.h = take(R * c.d_ff * elem_bytes(c.act_dtype));
  L.z = take(R * c.d * 4);
  L.total = take.off;
  return L;
}

struct GatedFp8Layout {
  GatedRoute r;
  size_t x8, sx, h, h8, sh, z, total;
};
static GatedFp8Layout gated_fp8_layout(const moe_config &c) {
  GatedFp8Layout L{};
  GatedTake take;
  const size_t R = (size_t)gated_max_rows(c);
  const size_t db = (size_t)fp8_blocks(c.d), fb = (size_t)fp8_blocks(c.d_ff);
  L.r = gated_route(c, take);
  L.x8 = take(R * db * kFp8Block);
  L.sx = take(R * db);
  L.h = take(R * c.d_ff * 2);
  L.h8 = take(R * fb * kFp8Block);
  L.sh = take(R * fb);
  L.z = take(R * c.d * 4);
  L.total = take.off;
  return L;
}

struct GatedBwdLayout {
  GatedRoute r;
  size_t h, dU, dP1, dP3, dX, dgpart, cpart, total;
  int dg_blocks, chunks;
};
static GatedBwdLayout gated_bwd_layout(const moe_config &c) {
  GatedBwdLayout L{};
  GatedTake take;
  const size_t R = (size_t)gated_max_rows(c), d = c.d, F = c.d_ff;
  L.r = gated_route(c, take);
  L.dg_blocks = gated_simt_dg_blocks(c, (int)R);
  L.chunks = colsum_chunks(host_capacity(c));
  L.h = take(R * F * 4);
  L.dU = take(R * d * 4);
  L.dP1 = take(R * F * 4);
  L.dP3 = take(R * F * 4);
  L.dX = take(R * d * 4);
  L.dgpart = take(R * L.dg_blocks * 4);
  L.cpart = take((size_t)L.chunks * c.E * (d + F) * 4);
  L.total = take.off;
  return L;
}

// The status cleared and the choices' slots; pos and keep go to the caller's
// arrays where given.
static int gated_slots(const moe_config &c, const GatedRoute &L, const int32_t *idx,
                       const float *gate, int32_t *pos, uint8_t *keep, void *ws, cudaStream_t s) {
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.status);
  MOE_CUDA(launch_gated_begin(st, s));
  MOE_CUDA(launch_slots(c, host_capacity(c), idx, gate, ws_at<int32_t>(ws, L.hist),
                        ws_at<int32_t>(ws, L.chunk_base), ws_at<int32_t>(ws, L.count),
                        ws_at<int32_t>(ws, L.offset), ws_at<int32_t>(ws, L.mtiles), pos, keep,
                        ws_at<int32_t>(ws, L.row_token), ws_at<float>(ws, L.row_gate), L.n_chunks,
                        st, s));
  return MOE_OK;
}

static GatedRows gated_rows(const GatedRoute &L, void *ws) {
  return {ws_at<int32_t>(ws, L.offset), ws_at<int32_t>(ws, L.mtiles),
          ws_at<int32_t>(ws, L.row_token), ws_at<float>(ws, L.row_gate)};
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
  const GatedLayout L = gated_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.r.status);
  int32_t *ps = pos ? pos : ws_at<int32_t>(ws, L.r.pos);
  uint8_t *kp = keep ? keep : ws_at<uint8_t>(ws, L.r.keep);
  r = gated_slots(c, L.r, expert_idx, gate, ps, kp, ws, s);
  if (r != MOE_OK) return r;
  GatedSimt p{};
  p.c = c;
  p.activation = activation;
  p.max_rows = (int)gated_max_rows(c);
  p.rows = gated_rows(L.r, ws);
  p.x = x;
  p.W1 = W1; p.b1 = b1; p.W3 = W3; p.b3 = b3; p.W2 = W2; p.b2 = b2;
  p.h = ws_at<char>(ws, L.h);
  p.pre1 = pre1;
  p.pre3 = pre3;
  p.z = ws_at<float>(ws, L.z);
  p.st = st;
  MOE_CUDA(launch_gated_simt_forward(p, s));
  MOE_CUDA(launch_combine(c, x, p.z, false, ps, kp, expert_idx, p.rows.offset, y, st, s));
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
  const GatedBwdLayout L = gated_bwd_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  int32_t *pos = ws_at<int32_t>(ws, L.r.pos);
  uint8_t *keep = ws_at<uint8_t>(ws, L.r.keep);
  r = gated_slots(c, L.r, expert_idx, gate, pos, keep, ws, s);
  if (r != MOE_OK) return r;
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
  p.hf = ws_at<float>(ws, L.h);
  p.dU = ws_at<float>(ws, L.dU);
  p.dP1 = ws_at<float>(ws, L.dP1);
  p.dP3 = ws_at<float>(ws, L.dP3);
  p.dX = ws_at<float>(ws, L.dX);
  p.dgpart = ws_at<float>(ws, L.dgpart);
  p.dW1 = dW1; p.dW3 = dW3; p.dW2 = dW2;
  p.st = ws_at<DeviceStatus>(ws, L.r.status);
  MOE_CUDA(launch_gated_simt_backward(p, s));
  const int32_t *off = p.rows.offset;
  MOE_CUDA(launch_gated_dgate(c, L.dg_blocks, expert_idx, pos, keep, off, p.dgpart, dy, b2, dgate,
                              s));
  float *cpart = ws_at<float>(ws, L.cpart);
  const bool bf16 = c.act_dtype == MOE_BF16;
  MOE_CUDA(launch_bwd_colsum(c, L.chunks, off, off, nullptr, p.dU, p.dP1, true, cpart, db2, db1,
                             bf16, s));
  MOE_CUDA(launch_bwd_colsum(c, L.chunks, off, off, nullptr, p.dU, p.dP3, true, cpart, nullptr,
                             db3, bf16, s));
  MOE_CUDA(launch_gated_dx(c, expert_idx, pos, keep, off, p.dX, dy, dx, s));
  return MOE_OK;
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
  DeviceStatus *st = ws_at<DeviceStatus>(ws, 0);
  MOE_CUDA(launch_gated_begin(st, s));
  MOE_CUDA(launch_fp8_weights(dtype == MOE_BF16, E, K, N, W, w8, wscale, st, s));
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
  const GatedFp8Layout L = gated_fp8_layout(c);
  cudaStream_t s = (cudaStream_t)stream;
  DeviceStatus *st = ws_at<DeviceStatus>(ws, L.r.status);
  int32_t *ps = pos ? pos : ws_at<int32_t>(ws, L.r.pos);
  uint8_t *kp = keep ? keep : ws_at<uint8_t>(ws, L.r.keep);
  r = gated_slots(c, L.r, expert_idx, gate, ps, kp, ws, s);
  if (r != MOE_OK) return r;
  GatedSimt p{};
  p.c = c;
  p.activation = activation;
  p.max_rows = (int)gated_max_rows(c);
  p.rows = gated_rows(L.r, ws);
  p.x = x;
  p.W1 = W1; p.b1 = b1; p.W3 = W3; p.b3 = b3; p.W2 = W2; p.b2 = b2;
  p.s1 = s1; p.s3 = s3; p.s2 = s2;
  p.h = ws_at<char>(ws, L.h);
  p.z = ws_at<float>(ws, L.z);
  p.st = st;
  uint8_t *x8 = ws_at<uint8_t>(ws, L.x8), *sx = ws_at<uint8_t>(ws, L.sx);
  uint8_t *h8 = ws_at<uint8_t>(ws, L.h8), *sh = ws_at<uint8_t>(ws, L.sh);
  const int32_t *count = p.rows.offset + c.E;
  MOE_CUDA(launch_fp8_rows(p.max_rows, c.d, c.k, count, p.rows.row_token, x, x8, sx, s));
  p.a8 = x8; p.sa = sx;
  MOE_CUDA(launch_gated_simt_fp8(p, 1, s));
  MOE_CUDA(launch_fp8_rows(p.max_rows, c.d_ff, c.k, count, nullptr, p.h, h8, sh, s));
  p.a8 = h8; p.sa = sh;
  MOE_CUDA(launch_gated_simt_fp8(p, 2, s));
  MOE_CUDA(launch_combine(c, x, p.z, false, ps, kp, expert_idx, p.rows.offset, y, st, s));
  return MOE_OK;
}

}  // extern "C"
