// C ABI of sampling, embedding and layer norm: argument validation and workspaces (see include/dh.h).
#include <cmath>

#include "layers.cuh"

using namespace dh;

namespace {

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool aligned256(const void* p) { return aligned_to(p, 256); }
bool valid_dtype(int dt) { return dt == DH_F32 || dt == DH_BF16; }
int elem_bytes(int dt) { return dt == DH_BF16 ? 2 : 4; }

// Rows of a call: their numbers, rounded up to a block's, stay below 2^31.
constexpr int MAX_ROWS = 0x7FFFFF00;

// Whether the rows of d elements at p and q (n and m of them, strides in elements) may share memory.
bool overlap(const void* p, int64_t ps, int64_t n, const void* q, int64_t qs, int64_t m, int64_t d, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t an = ((uintptr_t)(n - 1) * (uintptr_t)ps + (uintptr_t)d) * (uintptr_t)elem;
  const uintptr_t bn = ((uintptr_t)(m - 1) * (uintptr_t)qs + (uintptr_t)d) * (uintptr_t)elem;
  if (!(a < b + bn && b < a + an)) return false;
  // other columns of the same rows
  const uintptr_t step = (uintptr_t)ps * (uintptr_t)elem, row = (uintptr_t)d * (uintptr_t)elem;
  if (ps != qs || step < 2 * row) return true;
  const uintptr_t apart = (a < b ? b - a : a - b) % step;
  return apart < row || step - apart < row;
}
// The same, other than being the same rows.
bool clash(const void* p, int64_t ps, const void* q, int64_t qs, int64_t n, int64_t d, int elem) {
  return !(p == q && (ps == qs || n == 1)) && overlap(p, ps, n, q, qs, n, d, elem);
}

// Whether two arrays share memory (a null one none).
bool shared(const void* p, uint64_t p_bytes, const void* q, uint64_t q_bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + q_bytes && b < a + p_bytes;
}
// Whether n rows of d elements at p share memory with an array; it may lie between two of them.
bool touches(const void* p, int64_t ld, int64_t n, int64_t d, int elem, const void* q, uint64_t bytes) {
  const uint64_t step = (uint64_t)ld * (uint64_t)elem, row = (uint64_t)d * (uint64_t)elem;
  if (!shared(p, (uint64_t)(n - 1) * step + row, q, bytes)) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  if (b < a || step <= row) return true;
  return (b - a) % step < row || (b - a) % step + bytes > step;
}

int done(cudaError_t e, const char* what) { return note_error(e, what) == cudaSuccess ? DH_OK : DH_ERR_CUDA; }

}  // namespace

extern "C" {

// ------------------------------------------------------------------ sampling

size_t dh_sample_workspace(int N, int vocab, int dtype) {
  if (N <= 0 || N > MAX_ROWS || vocab <= 0 || vocab > DH_MAX_VOCAB || !valid_dtype(dtype)) return 0;
  return sample_workspace(N, vocab, dtype);
}

int dh_sample(const void* logits, int64_t row_stride, const float* u, const float* temperature, const int32_t* top_k,
              const float* top_p, const float* min_p, float temperature_all, int top_k_all, float top_p_all,
              float min_p_all, int N, int vocab, int dtype, int32_t* token_out, float* prob_out, void* workspace,
              size_t ws_bytes, void* stream) {
  if (N < 0 || vocab <= 0 || row_stride < 0) return DH_ERR_INVALID_ARG;
  if (!temperature && !(temperature_all >= 0.f && std::isfinite(temperature_all))) return DH_ERR_INVALID_ARG;
  if (!top_k && top_k_all < 0) return DH_ERR_INVALID_ARG;
  if (!top_p && !(top_p_all >= 0.f && top_p_all <= 1.f)) return DH_ERR_INVALID_ARG;
  if (!min_p && !(min_p_all >= 0.f && min_p_all <= 1.f)) return DH_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || vocab > DH_MAX_VOCAB || N > MAX_ROWS) return DH_ERR_UNSUPPORTED;
  if (N == 0) return DH_OK;
  if (!logits || !u || !token_out) return DH_ERR_INVALID_ARG;
  if (!aligned_to(logits, elem_bytes(dtype))) return DH_ERR_UNSUPPORTED;
  // a row's results may take the place of its uniform or of a setting: they are written when those have been read
  const uint64_t each = 4ull * (uint64_t)N;
  const void* const out[] = {token_out, prob_out};
  const void* const per_row[] = {u, temperature, top_k, top_p, min_p};
  if (shared(token_out, each, prob_out, each)) return DH_ERR_INVALID_ARG;
  for (const void* o : out) {
    if (touches(logits, row_stride, N, vocab, elem_bytes(dtype), o, each)) return DH_ERR_INVALID_ARG;
    for (const void* r : per_row)
      if (o != r && shared(o, each, r, each)) return DH_ERR_INVALID_ARG;
  }
  const size_t need = dh_sample_workspace(N, vocab, dtype);
  if (need && (!workspace || !aligned256(workspace) || ws_bytes < need)) return DH_ERR_WORKSPACE;
  Ctx c;
  if (!get_ctx(stream, &c)) return DH_ERR_CUDA;
  SampleArgs a = {};
  a.logits = logits;
  a.ld = row_stride;
  a.u = u;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.temperature0 = temperature_all;
  a.top_k0 = top_k_all;
  a.top_p0 = top_p_all;
  a.min_p0 = min_p_all;
  a.N = N;
  a.vocab = vocab;
  a.token = token_out;
  a.prob = prob_out;
  a.ws = workspace;
  return done(launch_sample(c, a, dtype), "sampling");
}

// ------------------------------------------------------------------ embedding

int dh_embed(const void* table, int64_t table_stride, const int32_t* tokens, int N, int vocab, int d, int dtype,
             float scale, void* out, int64_t out_stride, void* stream) {
  if (N < 0 || vocab <= 0 || d <= 0 || table_stride < 0 || (N > 1 && out_stride < d)) return DH_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || vocab > DH_MAX_VOCAB || d > DH_MAX_WIDTH || N > DH_MAX_TOKENS) return DH_ERR_UNSUPPORTED;
  if (N == 0) return DH_OK;
  if (!table || !tokens || !out) return DH_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype);
  if (!aligned_to(table, e) || !aligned_to(out, e)) return DH_ERR_UNSUPPORTED;
  if (overlap(table, table_stride, vocab, out, out_stride, N, d, e) ||
      touches(out, out_stride, N, d, e, tokens, 4ull * (uint64_t)N))
    return DH_ERR_INVALID_ARG;
  Ctx c;
  if (!get_ctx(stream, &c)) return DH_ERR_CUDA;
  EmbedArgs a = {};
  a.src = table;
  a.src_ld = table_stride;
  a.dst = out;
  a.dst_ld = out_stride;
  a.tokens = tokens;
  a.N = N;
  a.vocab = vocab;
  a.d = d;
  a.scale = scale;
  return done(launch_embed(c, a, dtype), "embedding");
}

size_t dh_embed_backward_workspace(int N, int vocab, int d, int dtype) {
  if (N <= 0 || N > DH_MAX_TOKENS || vocab <= 0 || vocab > DH_MAX_VOCAB || d <= 0 || d > DH_MAX_WIDTH ||
      !valid_dtype(dtype))
    return 0;
  return embed_backward_workspace(N, vocab, d, dtype);
}

int dh_embed_backward(const void* grad_out, int64_t grad_stride, const int32_t* tokens, int N, int vocab, int d,
                      int dtype, float scale, int accumulate, void* grad_table, int64_t table_stride, void* workspace,
                      size_t ws_bytes, void* stream) {
  if (N < 0 || vocab <= 0 || d <= 0 || grad_stride < 0 || (vocab > 1 && table_stride < d) || accumulate < 0 ||
      accumulate > 1)
    return DH_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || vocab > DH_MAX_VOCAB || d > DH_MAX_WIDTH || N > DH_MAX_TOKENS) return DH_ERR_UNSUPPORTED;
  if (N == 0 && accumulate) return DH_OK;
  if (!grad_table || (N > 0 && (!grad_out || !tokens))) return DH_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype);
  if (!aligned_to(grad_table, e) || !aligned_to(grad_out, e)) return DH_ERR_UNSUPPORTED;
  if (N > 0 && (overlap(grad_out, grad_stride, N, grad_table, table_stride, vocab, d, e) ||
                touches(grad_table, table_stride, vocab, d, e, tokens, 4ull * (uint64_t)N)))
    return DH_ERR_INVALID_ARG;
  const size_t need = dh_embed_backward_workspace(N, vocab, d, dtype);
  if (need && (!workspace || !aligned256(workspace) || ws_bytes < need)) return DH_ERR_WORKSPACE;
  Ctx c;
  if (!get_ctx(stream, &c)) return DH_ERR_CUDA;
  EmbedArgs a = {};
  a.src = grad_out;
  a.src_ld = grad_stride;
  a.dst = grad_table;
  a.dst_ld = table_stride;
  a.tokens = tokens;
  a.N = N;
  a.vocab = vocab;
  a.d = d;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  a.ws = static_cast<char*>(workspace);
  return done(launch_embed_backward(c, a, dtype), "embedding gradient");
}

// ------------------------------------------------------------------ layer norm

namespace {

// The checks that both calls share.
int check_norm(int N, int d, int dtype, int param_dtype, int64_t row_stride) {
  if (N < 0 || d <= 0 || row_stride < 0) return DH_ERR_INVALID_ARG;
  if (!valid_dtype(dtype) || (param_dtype != DH_F32 && param_dtype != dtype) || d > DH_MAX_WIDTH || N > MAX_ROWS)
    return DH_ERR_UNSUPPORTED;
  return DH_OK;
}

}  // namespace

int dh_layer_norm(const void* x, int64_t row_stride, const void* weight, const void* bias, int N, int d, int dtype,
                  int param_dtype, float eps, void* y, int64_t y_stride, float* stats_out, void* stream) {
  const int st = check_norm(N, d, dtype, param_dtype, row_stride);
  if (st != DH_OK) return st;
  if (!(eps >= 0.f && std::isfinite(eps)) || (N > 1 && y_stride < d)) return DH_ERR_INVALID_ARG;
  if (N == 0) return DH_OK;
  if (!x || !y) return DH_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, pe) || !aligned_to(bias, pe) ||
      !aligned_to(stats_out, 8))
    return DH_ERR_UNSUPPORTED;
  const uint64_t stats_bytes = 8ull * (uint64_t)N, param_bytes = (uint64_t)d * (uint64_t)pe;
  if (clash(x, row_stride, y, y_stride, N, d, e) || touches(y, y_stride, N, d, e, weight, param_bytes) ||
      touches(y, y_stride, N, d, e, bias, param_bytes) || touches(y, y_stride, N, d, e, stats_out, stats_bytes) ||
      touches(x, row_stride, N, d, e, stats_out, stats_bytes) || shared(stats_out, stats_bytes, weight, param_bytes) ||
      shared(stats_out, stats_bytes, bias, param_bytes))
    return DH_ERR_INVALID_ARG;
  Ctx c;
  if (!get_ctx(stream, &c)) return DH_ERR_CUDA;
  NormArgs a = {};
  a.x = x;
  a.ld = row_stride;
  a.weight = weight;
  a.bias = bias;
  a.eps = eps;
  a.y = y;
  a.y_ld = y_stride;
  a.stats_out = reinterpret_cast<float2*>(stats_out);
  a.N = N;
  a.d = d;
  return done(launch_norm(c, a, dtype, param_dtype), "layer norm");
}

size_t dh_layer_norm_backward_workspace(int N, int d, int dtype) {
  if (N <= 0 || N > MAX_ROWS || d <= 0 || d > DH_MAX_WIDTH || !valid_dtype(dtype)) return 0;
  return norm_backward_workspace(N, d, dtype);
}

int dh_layer_norm_backward(const void* grad_out, int64_t grad_stride, const void* x, int64_t row_stride,
                           const float* stats, const void* weight, int N, int d, int dtype, int param_dtype,
                           void* grad_x, int64_t grad_x_stride, void* grad_weight, void* grad_bias, void* workspace,
                           size_t ws_bytes, void* stream) {
  const int st = check_norm(N, d, dtype, param_dtype, row_stride);
  if (st != DH_OK) return st;
  if (grad_stride < 0 || (grad_x && N > 1 && grad_x_stride < d)) return DH_ERR_INVALID_ARG;
  if (!grad_x && !grad_weight && !grad_bias) return DH_OK;
  if (N > 0 && (!grad_out || !x || !stats)) return DH_ERR_INVALID_ARG;
  const int e = elem_bytes(dtype), pe = elem_bytes(param_dtype);
  if (!aligned_to(grad_out, e) || !aligned_to(x, e) || !aligned_to(grad_x, e) || !aligned_to(stats, 8) ||
      !aligned_to(weight, pe) || !aligned_to(grad_weight, pe) || !aligned_to(grad_bias, pe))
    return DH_ERR_UNSUPPORTED;
  if (N > 0 && grad_x && (clash(grad_out, grad_stride, grad_x, grad_x_stride, N, d, e) ||
                          clash(x, row_stride, grad_x, grad_x_stride, N, d, e)))
    return DH_ERR_INVALID_ARG;
  const uint64_t stats_bytes = 8ull * (uint64_t)N, param_bytes = (uint64_t)d * (uint64_t)pe;
  if (N > 0 && (touches(grad_x, grad_x_stride, N, d, e, stats, stats_bytes) ||
                touches(grad_x, grad_x_stride, N, d, e, weight, param_bytes)))
    return DH_ERR_INVALID_ARG;
  const void* const params[] = {grad_weight, grad_bias};
  for (const void* p : params)
    if (shared(p, param_bytes, weight, param_bytes) ||
        (N > 0 && (touches(grad_out, grad_stride, N, d, e, p, param_bytes) ||
                   touches(x, row_stride, N, d, e, p, param_bytes) || shared(p, param_bytes, stats, stats_bytes) ||
                   touches(grad_x, grad_x_stride, N, d, e, p, param_bytes))))
      return DH_ERR_INVALID_ARG;
  if (shared(grad_weight, param_bytes, grad_bias, param_bytes)) return DH_ERR_INVALID_ARG;
  const bool sums = grad_weight || grad_bias;
  const size_t need = sums ? dh_layer_norm_backward_workspace(N, d, dtype) : 0;
  if (need && (!workspace || !aligned256(workspace) || ws_bytes < need)) return DH_ERR_WORKSPACE;
  Ctx c;
  if (!get_ctx(stream, &c)) return DH_ERR_CUDA;
  if (N == 0 && !sums) return DH_OK;
  NormArgs a = {};
  a.x = x;
  a.ld = row_stride;
  a.weight = weight;
  a.y = grad_x;
  a.y_ld = grad_x_stride;
  a.stats = reinterpret_cast<const float2*>(stats);
  a.grad = grad_out;
  a.grad_ld = grad_stride;
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.N = N;
  a.d = d;
  a.ws = need ? reinterpret_cast<float*>(static_cast<char*>(workspace) + WS_HEADER) : nullptr;
  return done(launch_norm_backward(c, a, dtype, param_dtype), "layer norm gradient");
}

}  // extern "C"
