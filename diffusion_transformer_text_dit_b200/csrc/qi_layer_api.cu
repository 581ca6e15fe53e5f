// C ABI of the prompt-encoder layer operators (declared in include/qi.h):
// packed causal attention, Linear with activation and residual, gated
// feed-forward block.  Every argument check runs before the first launch of a
// call.
#include <string.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "qi_host.h"

using namespace qi_host;

static_assert(QI_MAX_SEQS == qi::AP_MAX_SEQS, "sequence table");
static_assert(QI_ACT_NONE == qi::ACT_NONE && QI_ACT_GELU_TANH == qi::ACT_GELU_TANH &&
                  QI_ACT_SILU == qi::ACT_SILU,
              "activation codes");

namespace {

// Largest extent of a matrix (rows, columns, K) and length of a sequence: the
// kernels' indexes, rounded up to whole tiles, stay below 2^31.
constexpr int MAX_EXTENT = 1 << 30;

// Makes the context's device current for the duration of a call, so that a
// call works whatever device its thread uses otherwise.
struct DeviceScope {
  int before;
  bool ok, moved;
  explicit DeviceScope(const qi_ctx* ctx) : before(-1), ok(false), moved(false) {
    if (cudaGetDevice(&before) != cudaSuccess) return;
    if (before != ctx->device) {
      if (cudaSetDevice(ctx->device) != cudaSuccess) return;
      moved = true;
    }
    ok = true;
  }
  ~DeviceScope() {
    if (moved) cudaSetDevice(before);
  }
};

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an > 0 && bn > 0 && x < y + bn && y < x + an;
}

// Bytes from the first to the last value of a [rows, cols] matrix of 2-byte values.
size_t span_bytes(int rows, int cols, int ld) {
  return rows == 0 ? 0 : (static_cast<size_t>(rows - 1) * ld + cols) * 2;
}

// A [rows, cols] matrix of 2-byte values.
struct Rows {
  const void* p;
  int rows, cols, ld;
};

// Whether two matrices share a byte.  Column ranges of the same rows (a fused
// q | k | v | o block) lie between each other without sharing one.
bool overlap(const Rows& a, const Rows& b) {
  if (!overlap(a.p, span_bytes(a.rows, a.cols, a.ld), b.p, span_bytes(b.rows, b.cols, b.ld))) return false;
  const int lda = a.rows == 1 ? std::max(a.cols, b.ld) : a.ld, ldb = b.rows == 1 ? std::max(b.cols, lda) : b.ld;
  const intptr_t bytes = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
  if (lda != ldb || bytes % 2 != 0) return true;
  const intptr_t at = (bytes / 2 % lda + lda) % lda;   // b's first column, counted in a's rows
  return at < a.cols || at + b.cols > lda;
}

int check_act(int act, bool none_ok) {
  if (act == QI_ACT_GELU_TANH || act == QI_ACT_SILU || (none_ok && act == QI_ACT_NONE)) return QI_OK;
  return fail(QI_ERR_INVALID_ARG, "unknown activation %d", act);
}

// A row matrix that TMA or 16-byte loads read: base and rows 16-byte aligned.
int check_rows(const char* name, const void* p, int cols, int ld, bool required) {
  if (!p) return required ? fail(QI_ERR_INVALID_ARG, "%s is NULL", name) : QI_OK;
  if (ld < cols) return fail(QI_ERR_INVALID_ARG, "%s: leading dimension %d < %d columns", name, ld, cols);
  if (ld % 8 != 0 || !aligned16(p))
    return fail(QI_ERR_ALIGNMENT, "%s: rows must be 16-byte aligned (pointer, ld %% 8 == 0)", name);
  return QI_OK;
}

int check_launch(int r, const char* what) {
  if (r == -2) return fail(QI_ERR_CUDA, "cuTensorMapEncodeTiled failed (%s)", what);
  if (r != 0) return cuda_fail(what);
  return QI_OK;
}

// ---------------------------------------------------------------- packed attention

int check_spans(const int32_t* spans, int n, int heads, int kv_heads, long long q_rows, long long k_rows) {
  if (n < 0 || n > QI_MAX_SEQS)
    return fail(QI_ERR_INVALID_ARG, "n_seqs = %d outside 0..%d", n, QI_MAX_SEQS);
  if (n > 0 && !spans) return fail(QI_ERR_INVALID_ARG, "spans is NULL");
  if (heads < 1 || kv_heads < 1 || heads % kv_heads != 0)
    return fail(QI_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
  if (heads / kv_heads > 128 || heads > 4096)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "at most 128 query heads per key/value head, 4096 heads");
  std::vector<std::pair<long long, long long>> q;
  q.reserve(n);
  long long keys = 0;
  for (int i = 0; i < n; ++i) {
    const long long q0 = spans[4 * i], ql = spans[4 * i + 1], k0 = spans[4 * i + 2], kl = spans[4 * i + 3];
    if (q0 < 0 || ql < 0 || k0 < 0 || kl < 0)
      return fail(QI_ERR_INVALID_ARG, "sequence %d: negative start or length", i);
    if ((q_rows >= 0 && q0 + ql > q_rows) || (k_rows >= 0 && k0 + kl > k_rows))
      return fail(QI_ERR_INVALID_ARG, "sequence %d: rows outside the q or k buffer", i);
    if (ql > MAX_EXTENT || kl > MAX_EXTENT)
      return fail(QI_ERR_UNSUPPORTED_SHAPE, "sequence %d: more than 2^30 queries or keys", i);
    if (ql > 0) q.emplace_back(q0, q0 + ql);
    keys += kl;
  }
  // (ranges of 256 keys: units of work stay below 2^31)
  if (keys * kv_heads >= 1ll << 38)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "keys x kv_heads of all sequences must stay below 2^38");
  std::sort(q.begin(), q.end());
  for (size_t i = 1; i < q.size(); ++i)
    if (q[i].first < q[i - 1].second)
      return fail(QI_ERR_INVALID_ARG, "two sequences share query rows");
  long long rows = 0;
  for (const auto& x : q) rows += x.second - x.first;
  if (rows * heads > (1ll << 31) - 1)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "query rows x heads must stay below 2^31");
  return QI_OK;
}

}  // namespace

int qi_attn_causal_packed_workspace_bytes(qi_ctx* ctx, const int32_t* spans, int n_seqs, int heads,
                                          int kv_heads, size_t* bytes) try {
  if (!ctx || !bytes) return fail(QI_ERR_INVALID_ARG, "NULL argument");
  int r;
  if ((r = check_spans(spans, n_seqs, heads, kv_heads, -1, -1))) return r;
  qi::PackedPlan tile, token;
  qi::packed_plan(spans, n_seqs, heads, kv_heads, ctx->num_sms, &tile, &token);
  *bytes = qi::packed_plan_bytes(tile) + qi::packed_plan_bytes(token);
  return QI_OK;
} catch (const std::bad_alloc&) {
  return fail(QI_ERR_INVALID_ARG, "out of host memory");
}

int qi_attn_causal_packed(qi_ctx* ctx, const uint16_t* q, int ldq, int q_rows, const uint16_t* k,
                          int ldk, const uint16_t* v, int ldv, int k_rows, int heads, int kv_heads,
                          int head_dim, const int32_t* spans, int n_seqs, float sm_scale,
                          uint16_t* o, int ldo, void* workspace, size_t workspace_bytes,
                          void* stream) try {
  if (!ctx) return fail(QI_ERR_INVALID_ARG, "ctx is NULL");
  if (head_dim != 128) return fail(QI_ERR_UNSUPPORTED_SHAPE, "head_dim must be 128");
  if (q_rows < 0 || k_rows < 0) return fail(QI_ERR_INVALID_ARG, "negative row count");
  if (!(sm_scale > 0.f) || sm_scale > 1e30f) return fail(QI_ERR_INVALID_ARG, "sm_scale must be positive and finite");
  int r;
  if ((r = check_spans(spans, n_seqs, heads, kv_heads, q_rows, k_rows))) return r;
  if ((r = check_rows("q", q, heads * 128, ldq, q_rows > 0)) ||
      (r = check_rows("o", o, heads * 128, ldo, q_rows > 0)) ||
      (r = check_rows("k", k, kv_heads * 128, ldk, k_rows > 0)) ||
      (r = check_rows("v", v, kv_heads * 128, ldv, k_rows > 0)))
    return r;
  const Rows qr{q, q_rows, heads * 128, ldq}, orows{o, q_rows, heads * 128, ldo}, kr{k, k_rows, kv_heads * 128, ldk},
      vr{v, k_rows, kv_heads * 128, ldv};
  if (overlap(orows, kr) || overlap(orows, vr) || overlap(orows, qr))
    return fail(QI_ERR_INVALID_ARG, "o overlaps q, k or v");
  qi::PackedPlan tile, token;
  qi::packed_plan(spans, n_seqs, heads, kv_heads, ctx->num_sms, &tile, &token);
  const size_t need = qi::packed_plan_bytes(tile) + qi::packed_plan_bytes(token);
  if (need > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(QI_ERR_WORKSPACE, "packed attention needs %zu bytes of workspace, got %zu", need,
                  workspace ? workspace_bytes : static_cast<size_t>(0));
    if (!aligned16(workspace)) return fail(QI_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    for (const Rows& r : {qr, kr, vr, orows})
      if (overlap(workspace, need, r.p, span_bytes(r.rows, r.cols, r.ld)))
        return fail(QI_ERR_INVALID_ARG, "the workspace overlaps q, k, v or o");
  }
  if (tile.units == 0 && token.units == 0) return QI_OK;
  qi::PackedAttnParams p;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = o;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.ldo = ldo;
  p.q_rows = q_rows;
  p.k_rows = k_rows;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.sm_scale = sm_scale;
  p.num_sms = ctx->num_sms;
  p.scratch = need > 0 ? workspace : nullptr;
  p.status = ctx->status;
  DeviceScope dev(ctx);
  if (!dev.ok) return cuda_fail("cudaSetDevice");
  Prof pr(ctx, QI_KCLASS_ATTN, S(stream));
  return check_launch(qi::launch_attention_packed(p, tile, token, S(stream)), "packed attention launch");
} catch (const std::bad_alloc&) {
  return fail(QI_ERR_INVALID_ARG, "out of host memory");
}

// ---------------------------------------------------------------- Linear

int qi_linear_act(qi_ctx* ctx, const uint16_t* a, int M, int lda, const qi_linear_bf16* w, int act,
                  const uint16_t* residual, int ld_residual, uint16_t* y, int ldy, void* stream) {
  if (!ctx || !w || !w->w) return fail(QI_ERR_INVALID_ARG, "NULL argument");
  if (M < 0 || w->n < 1 || w->k < 1) return fail(QI_ERR_INVALID_ARG, "need M >= 0, n >= 1, k >= 1");
  if (w->k % 8 != 0) return fail(QI_ERR_UNSUPPORTED_SHAPE, "k = %d is not a multiple of 8", w->k);
  if (M > MAX_EXTENT || w->n > MAX_EXTENT || w->k > MAX_EXTENT)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "M, n and k must not exceed 2^30");
  if (!aligned16(w->w) || (w->bias && !aligned16(w->bias)))
    return fail(QI_ERR_ALIGNMENT, "weight and bias must be 16-byte aligned");
  int r;
  if ((r = check_act(act, true))) return r;
  if ((r = check_rows("a", a, w->k, lda, M > 0))) return r;
  if (M > 0 && !y) return fail(QI_ERR_INVALID_ARG, "y is NULL");
  if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(residual)) & 1)
    return fail(QI_ERR_ALIGNMENT, "y and residual must be 2-byte aligned");
  if (ldy < w->n || (residual && ld_residual < w->n))
    return fail(QI_ERR_INVALID_ARG, "leading dimension of y or residual < n");
  const size_t yb = span_bytes(M, w->n, ldy);
  const Rows yr{y, M, w->n, ldy};
  if (overlap(yr, {a, M, w->k, lda}) || overlap(y, yb, w->w, span_bytes(w->n, w->k, w->k)) ||
      overlap(y, yb, w->bias, static_cast<size_t>(w->n) * 2) ||
      (residual && (residual != y || ld_residual != ldy) && overlap(yr, {residual, M, w->n, ld_residual})))
    return fail(QI_ERR_INVALID_ARG, "y overlaps an input (only residual == y with the same ld is allowed)");
  if (M == 0) return QI_OK;
  qi::LinearActParams p;
  p.a = a;
  p.M = M;
  p.K = w->k;
  p.N = w->n;
  p.lda = lda;
  p.w = w->w;
  p.bias = w->bias;
  p.act = act;
  p.res = residual;
  p.ld_res = ld_residual;
  p.y = y;
  p.ldy = ldy;
  p.num_sms = ctx->num_sms;
  p.status = ctx->status;
  p.after_tiles = false;
  DeviceScope dev(ctx);
  if (!dev.ok) return cuda_fail("cudaSetDevice");
  Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
  return check_launch(qi::launch_linear_act(p, S(stream)), "linear_act launch");
}

// ---------------------------------------------------------------- gated feed-forward block

namespace {

struct GatedBufs {
  uint16_t *h, *dg, *du;   // [M, F]
};

GatedBufs carve_gated(Carve& c, int M, int F, bool backward) {
  GatedBufs b{nullptr, nullptr, nullptr};
  const size_t n = static_cast<size_t>(M) * F;
  b.h = c.take<uint16_t>(n);
  if (backward) {
    b.dg = c.take<uint16_t>(n);
    b.du = c.take<uint16_t>(n);
  }
  return b;
}

int check_gated(const qi_gated_ffn* w) {
  if (!w || !w->gate || !w->up || !w->down) return fail(QI_ERR_INVALID_ARG, "gated ffn: NULL weight");
  if (w->hidden < 8 || w->mlp < 8 || w->hidden % 8 != 0 || w->mlp % 8 != 0)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "gated ffn: hidden and mlp must be positive multiples of 8");
  if (w->hidden > MAX_EXTENT || w->mlp > MAX_EXTENT / 2)   // (gate | up is one row)
    return fail(QI_ERR_UNSUPPORTED_SHAPE, "gated ffn: hidden must not exceed 2^30, mlp 2^29");
  if (!aligned16(w->gate) || !aligned16(w->up) || !aligned16(w->down))
    return fail(QI_ERR_ALIGNMENT, "gated ffn: weights must be 16-byte aligned");
  return check_act(w->act, false);
}

int check_m(int M) {
  if (M < 0) return fail(QI_ERR_INVALID_ARG, "M must be >= 0");
  if (M > MAX_EXTENT) return fail(QI_ERR_UNSUPPORTED_SHAPE, "M must not exceed 2^30");
  return QI_OK;
}

size_t gated_bytes(const qi_gated_ffn& w, int M, bool backward) {
  Carve c{nullptr, 0, 0};
  carve_gated(c, M, w.mlp, backward);
  return M == 0 ? 0 : c.off + 256;
}

// Aligned start of the caller's workspace, or an error.
int take_workspace(void* ws, size_t have, size_t need, Carve* c) {
  if (!ws || have < need)
    return fail(QI_ERR_WORKSPACE, "gated ffn needs %zu bytes of workspace, got %zu", need,
                ws ? have : static_cast<size_t>(0));
  const uintptr_t a = (reinterpret_cast<uintptr_t>(ws) + 255) & ~static_cast<uintptr_t>(255);
  *c = Carve{reinterpret_cast<uint8_t*>(a), need, 0};
  return QI_OK;
}

}  // namespace

int qi_gated_ffn_workspace_bytes(const qi_gated_ffn* w, int M, int backward, size_t* bytes) {
  if (!bytes) return fail(QI_ERR_INVALID_ARG, "NULL output");
  int r;
  if ((r = check_gated(w))) return r;
  if ((r = check_m(M))) return r;
  *bytes = gated_bytes(*w, M, backward != 0);
  return QI_OK;
}

int qi_gated_ffn_forward(qi_ctx* ctx, const qi_gated_ffn* w, const uint16_t* x, int M, int ldx,
                         const uint16_t* residual, int ld_residual, uint16_t* y, int ldy,
                         float* gate_up, void* workspace, size_t workspace_bytes, void* stream) {
  if (!ctx) return fail(QI_ERR_INVALID_ARG, "ctx is NULL");
  int r;
  if ((r = check_gated(w))) return r;
  if ((r = check_m(M))) return r;
  const int H = w->hidden, F = w->mlp;
  if ((r = check_rows("x", x, H, ldx, M > 0)) || (r = check_rows("y", y, H, ldy, M > 0)) ||
      (r = check_rows("residual", residual, H, ld_residual, false)) ||
      (r = check_rows("gate_up", gate_up, 2 * F, 2 * F, false)))
    return r;
  if (M == 0) return QI_OK;
  Carve c{nullptr, 0, 0};
  const size_t need = gated_bytes(*w, M, false);
  if ((r = take_workspace(workspace, workspace_bytes, need, &c))) return r;
  const GatedBufs b = carve_gated(c, M, F, false);
  // y may be x (the input is read before y is written) or the residual itself
  const size_t yb = span_bytes(M, H, ldy), gb = gate_up ? static_cast<size_t>(M) * 2 * F * 4 : 0,
               wb = static_cast<size_t>(H) * F * 2;
  if (overlap(y, yb, workspace, workspace_bytes) || overlap(gate_up, gb, workspace, workspace_bytes) ||
      overlap(y, yb, gate_up, gb) || overlap(gate_up, gb, x, span_bytes(M, H, ldx)) ||
      overlap(gate_up, gb, residual, span_bytes(M, H, ld_residual)) ||
      overlap(x, span_bytes(M, H, ldx), workspace, workspace_bytes) ||
      overlap(residual, span_bytes(M, H, ld_residual), workspace, workspace_bytes) ||
      overlap(y, yb, w->down, wb) || overlap(y, yb, w->gate, wb) || overlap(y, yb, w->up, wb) ||
      overlap(gate_up, gb, w->down, wb) || overlap(gate_up, gb, w->gate, wb) || overlap(gate_up, gb, w->up, wb) ||
      overlap(workspace, workspace_bytes, w->down, wb) || overlap(workspace, workspace_bytes, w->gate, wb) ||
      overlap(workspace, workspace_bytes, w->up, wb) ||
      (residual && (residual != y || ld_residual != ldy) &&
       overlap({y, M, H, ldy}, Rows{residual, M, H, ld_residual})))
    return fail(QI_ERR_INVALID_ARG, "gated ffn: an output overlaps an input, the workspace or the other output");
  qi::GateUpParams g;
  g.x = x;
  g.M = M;
  g.H = H;
  g.F = F;
  g.ldx = ldx;
  g.gate = w->gate;
  g.up = w->up;
  g.act = w->act;
  g.h = b.h;
  g.gu = gate_up;
  g.num_sms = ctx->num_sms;
  g.status = ctx->status;
  qi::LinearActParams p;
  p.a = b.h;
  p.M = M;
  p.K = F;
  p.N = H;
  p.lda = F;
  p.w = w->down;
  p.bias = nullptr;
  p.act = QI_ACT_NONE;
  p.res = residual;
  p.ld_res = ld_residual;
  p.y = y;
  p.ldy = ldy;
  p.num_sms = ctx->num_sms;
  p.status = ctx->status;
  p.after_tiles = qi::gate_up_on_tiles(M, H, F, ctx->num_sms);
  DeviceScope dev(ctx);
  if (!dev.ok) return cuda_fail("cudaSetDevice");
  {
    Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
    if ((r = check_launch(qi::launch_gate_up(g, S(stream)), "gate/up launch"))) return r;
  }
  Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
  return check_launch(qi::launch_linear_act(p, S(stream)), "down projection launch");
}

int qi_gated_ffn_backward(qi_ctx* ctx, const qi_gated_ffn* w, const uint16_t* x, int M, int ldx,
                          const uint16_t* dy, int ld_dy, const float* gate_up, uint16_t* dx,
                          int ld_dx, uint16_t* dgate, uint16_t* dup, uint16_t* ddown,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!ctx) return fail(QI_ERR_INVALID_ARG, "ctx is NULL");
  int r;
  if ((r = check_gated(w))) return r;
  if ((r = check_m(M))) return r;
  const int H = w->hidden, F = w->mlp;
  if ((r = check_rows("x", x, H, ldx, M > 0)) || (r = check_rows("dy", dy, H, ld_dy, M > 0)) ||
      (r = check_rows("gate_up", gate_up, 2 * F, 2 * F, M > 0)) ||
      (r = check_rows("dx", dx, H, ld_dx, false)) || (r = check_rows("dgate", dgate, H, H, false)) ||
      (r = check_rows("dup", dup, H, H, false)) || (r = check_rows("ddown", ddown, F, F, false)))
    return r;
  const size_t wb = static_cast<size_t>(H) * F * 2, xb = span_bytes(M, H, ldx), yb = span_bytes(M, H, ld_dy),
               gb = static_cast<size_t>(M) * 2 * F * 4;
  const Rows xr{x, M, H, ldx}, yr{dy, M, H, ld_dy}, dr{dx, M, H, ld_dx};
  struct Range {
    const void* p;
    size_t n;
  };
  const Range outs[5] = {{dx, dx ? span_bytes(M, H, ld_dx) : 0}, {dgate, wb}, {dup, wb}, {ddown, wb},
                         {workspace, workspace_bytes}};
  const Range ins[6] = {{x, xb}, {dy, yb}, {gate_up, gb}, {w->gate, wb}, {w->up, wb}, {w->down, wb}};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < 6; ++j)
      if (i == 0 && j < 2 ? overlap(dr, j == 0 ? xr : yr) : overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
        return fail(QI_ERR_INVALID_ARG, "gated ffn backward: an output or the workspace overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return fail(QI_ERR_INVALID_ARG, "gated ffn backward: outputs or the workspace overlap");
  }
  if (M > 0 && !dx && !dgate && !dup && !ddown) return QI_OK;
  Carve c{nullptr, 0, 0};
  if (M > 0 && (r = take_workspace(workspace, workspace_bytes, gated_bytes(*w, M, true), &c))) return r;
  DeviceScope dev(ctx);
  if (!dev.ok) return cuda_fail("cudaSetDevice");
  if (M == 0) {   // a sum over no rows
    for (uint16_t* p : {dgate, dup, ddown})
      if (p && cudaMemsetAsync(p, 0, wb, S(stream)) != cudaSuccess) return cuda_fail("zero gradient");
    return QI_OK;
  }
  const GatedBufs b = carve_gated(c, M, F, true);
  qi::GatedBackwardParams p;
  p.x = x;
  p.dy = dy;
  p.gu = gate_up;
  p.M = M;
  p.H = H;
  p.F = F;
  p.ldx = ldx;
  p.ld_dy = ld_dy;
  p.gate = w->gate;
  p.up = w->up;
  p.down = w->down;
  p.act = w->act;
  p.dg = b.dg;
  p.du = b.du;
  p.h = b.h;
  p.dx = dx;
  p.ld_dx = ld_dx;
  p.dgate = dgate;
  p.dup = dup;
  p.ddown = ddown;
  p.num_sms = ctx->num_sms;
  p.status = ctx->status;
  {
    Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
    if ((r = check_launch(qi::launch_gated_dh(p, S(stream)), "hidden gradient launch"))) return r;
  }
  if (dx) {
    Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
    if ((r = check_launch(qi::launch_gated_dx(p, S(stream)), "input gradient launch"))) return r;
  }
  if (dgate || dup || ddown) {
    Prof pr(ctx, QI_KCLASS_GEMM_BF16, S(stream));
    if ((r = check_launch(qi::launch_gated_dw(p, S(stream)), "weight gradient launch"))) return r;
  }
  return QI_OK;
}
