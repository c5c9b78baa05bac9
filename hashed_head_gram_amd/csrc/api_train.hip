// C ABI entry points of the training-step operators: argument validation and
// dispatch. Every check that can fail runs before anything is enqueued.
#include <limits.h>
#include <math.h>

#include "train.h"

namespace {

constexpr int64_t kMaxEmbedTokens = ((int64_t)1 << 26) - 1;
constexpr int kMaxEmbedD = 16384;
constexpr int64_t kMaxNormRows = (int64_t)1 << 31;
constexpr int64_t kMaxHeadTokens = ((int64_t)1 << 26) - 1;
constexpr int kMaxOrthoSide = 16384;
constexpr int kMaxOrthoSteps = 64;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
int hip_status(hipError_t e) { return e == hipSuccess ? PG_OK : PG_EHIP; }
bool float_dtype(int32_t t) { return t == PG_F32 || t == PG_BF16; }
uintptr_t elt(int32_t t) { return t == PG_F32 ? 4 : 2; }

int check_embed(int64_t n_tok, int64_t V, int32_t d) {
  if (n_tok < 0 || V < 1 || d < 1) return PG_EINVAL;
  if (d > kMaxEmbedD) return PG_EUNSUPPORTED;
  if (n_tok > kMaxEmbedTokens || V > INT_MAX - 1) return PG_ERANGE;
  return PG_OK;
}

// The checks both gradient forms share (n_tok > 0).
int check_embed_backward(const void* dout, int32_t dtype, int64_t ld, const int32_t* tokens,
                         int32_t d, const pg::EmbedPlan& p, const void* ws, int64_t ws_bytes) {
  if (!dout || !tokens || !aligned(dout, elt(dtype)) || !aligned(tokens, 4) || ld < d)
    return PG_EINVAL;
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256)) return PG_EINVAL;
  return PG_OK;
}

int check_norm(int32_t dtype, int64_t n, int32_t d) {
  if (!float_dtype(dtype) || n < 0 || d < 1) return PG_EINVAL;
  if (d > pg::kNormMaxD) return PG_EUNSUPPORTED;
  if (n > kMaxNormRows) return PG_ERANGE;
  return PG_OK;
}

int check_ortho(int64_t n_mat, int32_t rows, int32_t cols) {
  if (n_mat < 0 || rows < 1 || cols < 1) return PG_EINVAL;
  if (rows > kMaxOrthoSide || cols > kMaxOrthoSide) return PG_EUNSUPPORTED;
  if (n_mat > 65535) return PG_ERANGE;
  // the tile kernels' grid: 2^34 padded elements are 2^22 blocks at most
  const auto pad = [](int64_t x) { return (x + 127) / 128 * 128; };
  if (n_mat * pad(rows) * pad(cols) > (int64_t)1 << 34) return PG_ERANGE;
  return PG_OK;
}

int check_head(int64_t n, int32_t d, int64_t V, int32_t dtype, int32_t k) {
  if (n < 0 || d < 1 || V < 1 || k < 1 || !float_dtype(dtype)) return PG_EINVAL;
  if (d > pg::kHeadMaxD || k > pg::kHeadMaxK) return PG_EUNSUPPORTED;
  if (n > kMaxHeadTokens || V > INT_MAX - 1) return PG_ERANGE;
  // tiles are numbered in 32 bits
  if ((n / 128 + 1) * (V / 128 + 1) > INT_MAX) return PG_ERANGE;
  return PG_OK;
}

// The checks of all four head calls. n, the sizes and the flags are looked at
// before n = 0 returns; g.logits: distillation.
int check_head_call(const pg::HeadArgs& g, const pg_table* table, int32_t d, float temperature,
                    bool distill) {
  if (!table || !table->data || !aligned(table->data, 16)) return PG_EINVAL;
  if (table->dtype == PG_NF4) return PG_EUNSUPPORTED;
  const int st = check_head(g.n, d, table->n_rows, table->dtype, g.k);
  if (st != PG_OK) return st;
  if (!float_dtype(g.dtype)) return PG_EINVAL;
  if (g.dtype != table->dtype) return PG_EUNSUPPORTED;
  if (!isfinite(g.scale) || !(temperature > 0.f) || !isfinite(temperature) ||
      !isfinite(1.f / temperature) || !isfinite(g.scale / temperature * 1.4427f))
    return PG_EINVAL;
  if (g.ld_h < d) return PG_EINVAL;
  if (g.n == 0) return PG_OK;
  if (!g.h || !aligned(g.h, elt(g.dtype)) || !g.ids || !aligned(g.ids, 4)) return PG_EINVAL;
  if (!g.lse || !aligned(g.lse, 4)) return PG_EINVAL;
  if (distill && (!g.teacher || !aligned(g.teacher, 4) || !g.logits || !aligned(g.logits, 4)))
    return PG_EINVAL;
  return PG_OK;
}

int head_forward(pg::HeadArgs& g, const pg_table* table, int32_t d, float temperature,
                 bool distill, void* ws, int64_t ws_bytes, hipStream_t stream) {
  const int st = check_head_call(g, table, d, temperature, distill);
  if (st != PG_OK || g.n == 0) return st;
  if (!g.loss || !aligned(g.loss, 4)) return PG_EINVAL;
  g.d = d;
  g.table = table->data;
  g.V = table->n_rows;
  g.inv_tau = 1.f / temperature;
  const pg::HeadPlan p = pg::head_plan(g.n, d, g.V, g.dtype, g.k, false);
  if (!ws || ws_bytes < p.bytes || !aligned(ws, 256)) return PG_EINVAL;
  return hip_status(pg::launch_head_forward(p, g, ws, stream));
}

int head_backward(pg::HeadArgs& g, const pg_table* table, int32_t d, float temperature,
                  bool distill, void* ws, int64_t ws_bytes, hipStream_t stream) {
  if (g.accumulate != 0 && g.accumulate != 1) return PG_EINVAL;
  if (!g.dh && !g.dw) return PG_EINVAL;
  if (g.dw && (!float_dtype(g.dw_dtype) || !aligned(g.dw, elt(g.dw_dtype)))) return PG_EINVAL;
  if (g.dw && g.accumulate && g.dw_dtype != PG_F32) return PG_EUNSUPPORTED;
  const int st = check_head_call(g, table, d, temperature, distill);
  if (st != PG_OK) return st;
  if (g.dh && (g.ld_dh < d || !aligned(g.dh, elt(g.dtype)))) return PG_EINVAL;
  g.d = d;
  g.table = table->data;
  g.V = table->n_rows;
  g.inv_tau = 1.f / temperature;
  if (g.n > 0 && (!g.dloss || !aligned(g.dloss, 4) || !aligned(g.dlse, 4))) return PG_EINVAL;
  // later pieces read h again, and dh reads T while dT is written
  if (g.n > 0 && ((g.dh && g.dh == g.h) || (g.dw && g.dw == g.table))) return PG_EINVAL;
  const pg::HeadPlan p = pg::head_plan(g.n, d, g.V, g.dtype, g.k, true);
  if (g.n > 0 && (!ws || ws_bytes < p.bytes || !aligned(ws, 256))) return PG_EINVAL;
  return hip_status(pg::launch_head_backward(p, g, ws, stream));
}

// Largest workspace of any batch up to n: pieces get narrower as batches grow.
int64_t head_workspace(int64_t n, int32_t d, int64_t V, int32_t dtype, int32_t k, bool backward) {
  const int st = check_head(n, d, V, dtype, k);
  if (st != PG_OK) return st;
  int64_t most = pg::head_plan(n, d, V, dtype, k, backward).bytes;
  if (backward)
    for (int64_t m = 128; m < n && m <= 32768; m += 128) {
      const int64_t b = pg::head_plan(m, d, V, dtype, k, true).bytes;
      if (b > most) most = b;
    }
  return most;
}

// Largest |a s + b s^3 + c s^5| over 0 <= s <= m: the ends and the interior
// extrema, where a + 3 b t + 5 c t^2 = 0 with t = s^2.
double quintic_max(double a, double b, double c, double m) {
  auto p = [&](double s) { return fabs(s * (a + s * s * (b + c * s * s))); };
  double best = p(m);
  auto extremum = [&](double t) {
    if (t > 0 && t < m * m && p(sqrt(t)) > best) best = p(sqrt(t));
  };
  if (c != 0) {
    const double disc = 9 * b * b - 20 * a * c;
    if (disc >= 0) {
      extremum((-3 * b + sqrt(disc)) / (10 * c));
      extremum((-3 * b - sqrt(disc)) / (10 * c));
    }
  } else if (b != 0) {
    extremum(-a / (3 * b));
  }
  return best;
}

// Largest |b t + c t^2| over t = s^2, 0 <= s <= m.
double factor_max(double b, double c, double m) {
  const double t = m * m;
  const double best = fabs(b * t + c * t * t);
  return c != 0 && -b / (2 * c) > 0 && -b / (2 * c) < t ? fmax(best, fabs(b * b / (4 * c))) : best;
}

// Whether every iterate a step reads stays where the fp16 copies hold it:
// singular values at most 3 before each step, |b t + c t^2| at most 100 for t = s^2.
bool ortho_in_range(double a, double b, double c, int steps) {
  double m = 1.0;
  for (int k = 0; k < steps; ++k) {
    if (!(m <= 3.0)) return false;
    if (!(factor_max(b, c, m) <= 100.0)) return false;
    m = quintic_max(a, b, c, m);
  }
  return isfinite(m);                                // the result itself stays in fp32
}

// Leading steps whose operands have to be split in halves. The rounding of the
// fp16 operands of step k enters in proportion to B's size there and is moved
// by the steps behind it as s is: their composed slope, largest on 33 points
// of [0, m] (at 0 it is |a| a step). On spectra that suffer most (an eighth to
// half of the directions strong, the others 1e-2 to 1e-4 of them), simulated in
// float64 with fp16 operands, a sum of size times slope of 1 moves the result
// by up to 7e-6 of it in the 2-norm: 600 are about half a step of the result's
// bf16, 2^-8. Five steps of the usual coefficients come to 548 and 4.0e-3.
// Where all steps together pass 600, only the last ones stay unsplit, up to 80:
// by then the singular values are large, and with them what is rounded. Seven
// polynomials at 5 to 20 steps: none moved the result by more than 4.0e-3.
constexpr double kSumAll = 600, kSumLast = 80;
int ortho_split(double a, double b, double c, int steps) {
  double m[kMaxOrthoSteps + 1];
  m[0] = 1.0;
  for (int k = 0; k < steps; ++k) m[k + 1] = quintic_max(a, b, c, m[k]);
  double sum = 0;
  int last = 0;
  for (int k = steps - 1; k >= 0; --k) {
    const double size = factor_max(b, c, m[k]);
    if (size > 0) {
      double slope = 0;
      for (int i = 0; i <= 32; ++i) {
        double s = m[k + 1] * i / 32, g = 1;
        for (int j = k + 1; j < steps; ++j) {
          const double t = s * s;
          g *= a + t * (3 * b + 5 * c * t);
          s *= a + t * (b + c * t);
        }
        slope = fmax(slope, fabs(g));
      }
      sum += size * slope;
    }
    if (sum <= kSumLast) last = steps - k;
    if (sum > kSumAll) return steps - last;
  }
  return 0;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------
// Token embedding

PG_API int pg_embed(const pg_table* table, int32_t d, float scale, const int32_t* tokens,
                    int64_t n_tok, int32_t out_dtype, void* out, int64_t ld_out,
                    int32_t* dev_status, hipStream_t stream) {
  if (!table || !table->data || !aligned(table->data, 16)) return PG_EINVAL;
  if (table->dtype == PG_NF4) return PG_EUNSUPPORTED;
  if (!float_dtype(table->dtype) || !float_dtype(out_dtype)) return PG_EINVAL;
  const int st = check_embed(n_tok, table->n_rows, d);
  if (st != PG_OK) return st;
  if (ld_out < d) return PG_EINVAL;
  if (n_tok == 0) return PG_OK;
  if (!tokens || !out || !aligned(tokens, 4) || !aligned(out, elt(out_dtype))) return PG_EINVAL;
  if (dev_status && !aligned(dev_status, 4)) return PG_EINVAL;
  return hip_status(pg::launch_embed(table->dtype, table->data, table->n_rows, d, scale, tokens,
                                     n_tok, out_dtype, out, ld_out, dev_status, stream));
}

PG_API int64_t pg_embed_workspace_size(int64_t n_tok, int64_t V, int32_t d) {
  const int st = check_embed(n_tok, V, d);
  if (st != PG_OK) return st;
  return pg::embed_plan(n_tok, V, d).bytes;
}

PG_API int pg_embed_backward(const void* dout, int32_t dtype, int64_t ld, const int32_t* tokens,
                             int64_t n_tok, int64_t V, int32_t d, float scale, int64_t* urows,
                             float* ugrad, int64_t* n_unique, void* workspace,
                             int64_t workspace_bytes, hipStream_t stream) {
  int st = check_embed(n_tok, V, d);
  if (st != PG_OK) return st;
  if (!float_dtype(dtype) || !n_unique || !aligned(n_unique, 8)) return PG_EINVAL;
  if (n_tok == 0) return hip_status(pg::launch_set_i64(n_unique, 0, stream));
  if (!urows || !ugrad || !aligned(urows, 8) || !aligned(ugrad, 4)) return PG_EINVAL;
  const pg::EmbedPlan p = pg::embed_plan(n_tok, V, d);
  st = check_embed_backward(dout, dtype, ld, tokens, d, p, workspace, workspace_bytes);
  if (st != PG_OK) return st;
  return hip_status(pg::launch_embed_backward(p, dout, dtype, ld, tokens, n_tok, V, d, scale,
                                              urows, ugrad, n_unique, nullptr, 0, workspace,
                                              stream));
}

PG_API int pg_embed_backward_dense(const void* dout, int32_t dtype, int64_t ld,
                                   const int32_t* tokens, int64_t n_tok, int64_t V, int32_t d,
                                   float scale, float* dtable, int32_t accumulate,
                                   void* workspace, int64_t workspace_bytes,
                                   hipStream_t stream) {
  int st = check_embed(n_tok, V, d);
  if (st != PG_OK) return st;
  if (!float_dtype(dtype) || (accumulate != 0 && accumulate != 1)) return PG_EINVAL;
  if (n_tok == 0 && accumulate) return PG_OK;
  if (!dtable || !aligned(dtable, 4)) return PG_EINVAL;
  const pg::EmbedPlan p = pg::embed_plan(n_tok, V, d);
  if (n_tok > 0) {
    st = check_embed_backward(dout, dtype, ld, tokens, d, p, workspace, workspace_bytes);
    if (st != PG_OK) return st;
  }
  return hip_status(pg::launch_embed_backward(p, dout, dtype, ld, tokens, n_tok, V, d, scale,
                                              nullptr, nullptr, nullptr, dtable, accumulate,
                                              workspace, stream));
}

// ---------------------------------------------------------------------------
// Layer norm

PG_API int pg_layer_norm(const void* x, int32_t dtype, int64_t n, int32_t d, int64_t ld_x,
                         const float* gamma, const float* beta, float eps, void* y, int64_t ld_y,
                         float* mean, float* rstd, hipStream_t stream) {
  const int st = check_norm(dtype, n, d);
  if (st != PG_OK) return st;
  if (!(eps >= 0.f) || ld_x < d || ld_y < d) return PG_EINVAL;
  if (n == 0) return PG_OK;
  if (!x || !y || !gamma || !aligned(x, elt(dtype)) || !aligned(y, elt(dtype)) ||
      !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return PG_EINVAL;
  if (x == y && ld_x != ld_y) return PG_EINVAL;
  return hip_status(pg::launch_layer_norm(x, dtype, n, d, ld_x, gamma, beta, eps, y, ld_y, mean,
                                          rstd, stream));
}

PG_API int64_t pg_layer_norm_workspace_size(int64_t n, int32_t d) {
  const int st = check_norm(PG_F32, n, d);
  if (st != PG_OK) return st;
  return pg::layer_norm_partials(n, d) * 2 * (((int64_t)d + 7) / 8 * 8) * 4;
}

PG_API int pg_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                  int32_t dtype, int64_t n, int32_t d, const float* gamma,
                                  const float* mean, const float* rstd, const void* add,
                                  int64_t ld_add, void* dx, int64_t ld_dx, float* dgamma,
                                  float* dbeta, void* workspace, int64_t workspace_bytes,
                                  hipStream_t stream) {
  const int st = check_norm(dtype, n, d);
  if (st != PG_OK) return st;
  if (!dgamma || !aligned(dgamma, 4) || !aligned(dbeta, 4)) return PG_EINVAL;
  if (n > 0) {
    if (ld_dy < d || ld_x < d || ld_dx < d || (add && ld_add < d)) return PG_EINVAL;
    if (!dy || !x || !gamma || !mean || !rstd || !dx) return PG_EINVAL;
    const uintptr_t e = elt(dtype);
    if (!aligned(dy, e) || !aligned(x, e) || !aligned(dx, e) || !aligned(add, e) ||
        !aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
      return PG_EINVAL;
    if (dx == x || (dx == dy && ld_dx != ld_dy) || (dx == add && ld_dx != ld_add))
      return PG_EINVAL;
    if (!workspace || workspace_bytes < pg_layer_norm_workspace_size(n, d) ||
        !aligned(workspace, 256))
      return PG_EINVAL;
  }
  return hip_status(pg::launch_layer_norm_backward(
      dy, ld_dy, x, ld_x, dtype, n, d, gamma, mean, rstd, add, ld_add, dx, ld_dx, dgamma, dbeta,
      static_cast<float*>(workspace), stream));
}

// ---------------------------------------------------------------------------
// Orthogonalised update

PG_API int64_t pg_orthogonalize_workspace_size(int64_t n_mat, int32_t rows, int32_t cols) {
  const int st = check_ortho(n_mat, rows, cols);
  if (st != PG_OK) return st;
  return pg::ortho_plan(n_mat, rows, cols).bytes;
}

PG_API int pg_orthogonalize(const void* G, int32_t dtype, int64_t n_mat, int32_t rows,
                            int32_t cols, int32_t steps, float a, float b, float c, float eps,
                            float scale, void* out, void* workspace, int64_t workspace_bytes,
                            hipStream_t stream) {
  const int st = check_ortho(n_mat, rows, cols);
  if (st != PG_OK) return st;
  if (!float_dtype(dtype) || steps < 1 || steps > kMaxOrthoSteps || !(eps >= 0.f))
    return PG_EINVAL;
  if (!ortho_in_range(a, b, c, steps)) return PG_EUNSUPPORTED;
  if (n_mat == 0) return PG_OK;
  if (!G || !out || !aligned(G, elt(dtype)) || !aligned(out, 2)) return PG_EINVAL;
  const pg::OrthoPlan p = pg::ortho_plan(n_mat, rows, cols);
  if (!workspace || workspace_bytes < p.bytes || !aligned(workspace, 256)) return PG_EINVAL;
  const pg::OrthoArgs oa{steps, p.small ? 0 : ortho_split(a, b, c, steps), a, b, c, eps, scale};
  return hip_status(pg::launch_orthogonalize(p, G, dtype, n_mat, rows, cols, oa,
                                             static_cast<uint16_t*>(out), workspace, stream));
}

// ---------------------------------------------------------------------------
// Losses of the head

PG_API int64_t pg_head_loss_workspace_size(int64_t n, int32_t d, int64_t V, int32_t dtype) {
  return head_workspace(n, d, V, dtype, 1, false);
}

PG_API int64_t pg_head_loss_backward_workspace_size(int64_t n, int32_t d, int64_t V,
                                                    int32_t dtype) {
  return head_workspace(n, d, V, dtype, 1, true);
}

PG_API int64_t pg_head_distill_workspace_size(int64_t n, int32_t d, int64_t V, int32_t k,
                                              int32_t dtype) {
  return head_workspace(n, d, V, dtype, k, false);
}

PG_API int64_t pg_head_distill_backward_workspace_size(int64_t n, int32_t d, int64_t V, int32_t k,
                                                       int32_t dtype) {
  return head_workspace(n, d, V, dtype, k, true);
}

PG_API int pg_head_loss(const void* h, int32_t dtype, int64_t n, int32_t d, int64_t ld_h,
                        const pg_table* table, float scale, const int32_t* targets, float* loss,
                        float* lse, void* workspace, int64_t workspace_bytes,
                        hipStream_t stream) {
  pg::HeadArgs g{};
  g.h = h;
  g.dtype = dtype;
  g.n = n;
  g.ld_h = ld_h;
  g.scale = scale;
  g.ids = targets;
  g.k = 1;
  g.loss = loss;
  g.lse = lse;
  return head_forward(g, table, d, 1.f, false, workspace, workspace_bytes, stream);
}

PG_API int pg_head_loss_backward(const void* h, int32_t dtype, int64_t n, int32_t d, int64_t ld_h,
                                 const pg_table* table, float scale, const int32_t* targets,
                                 const float* lse, const float* dloss, const float* dlse,
                                 void* dh, int64_t ld_dh, void* dw, int32_t dw_dtype,
                                 int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                 hipStream_t stream) {
  pg::HeadArgs g{};
  g.h = h;
  g.dtype = dtype;
  g.n = n;
  g.ld_h = ld_h;
  g.scale = scale;
  g.ids = targets;
  g.k = 1;
  g.lse = const_cast<float*>(lse);
  g.dloss = dloss;
  g.dlse = dlse;
  g.dh = dh;
  g.ld_dh = ld_dh;
  g.dw = dw;
  g.dw_dtype = dw_dtype;
  g.accumulate = accumulate;
  return head_backward(g, table, d, 1.f, false, workspace, workspace_bytes, stream);
}

PG_API int pg_head_distill(const void* h, int32_t dtype, int64_t n, int32_t d, int64_t ld_h,
                           const pg_table* table, float scale, const int32_t* ids,
                           const float* teacher, int32_t k, float temperature, float* loss,
                           float* lse, float* logits, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream) {
  pg::HeadArgs g{};
  g.h = h;
  g.dtype = dtype;
  g.n = n;
  g.ld_h = ld_h;
  g.scale = scale;
  g.ids = ids;
  g.teacher = teacher;
  g.k = k;
  g.loss = loss;
  g.lse = lse;
  g.logits = logits;
  return head_forward(g, table, d, temperature, true, workspace, workspace_bytes, stream);
}

PG_API int pg_head_distill_backward(const void* h, int32_t dtype, int64_t n, int32_t d,
                                    int64_t ld_h, const pg_table* table, float scale,
                                    const int32_t* ids, const float* teacher, int32_t k,
                                    float temperature, const float* lse, const float* logits,
                                    const float* dloss, void* dh, int64_t ld_dh, void* dw,
                                    int32_t dw_dtype, int32_t accumulate, void* workspace,
                                    int64_t workspace_bytes, hipStream_t stream) {
  pg::HeadArgs g{};
  g.h = h;
  g.dtype = dtype;
  g.n = n;
  g.ld_h = ld_h;
  g.scale = scale;
  g.ids = ids;
  g.teacher = teacher;
  g.k = k;
  g.lse = const_cast<float*>(lse);
  g.logits = const_cast<float*>(logits);
  g.dloss = dloss;
  g.dh = dh;
  g.ld_dh = ld_dh;
  g.dw = dw;
  g.dw_dtype = dw_dtype;
  g.accumulate = accumulate;
  return head_backward(g, table, d, temperature, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
