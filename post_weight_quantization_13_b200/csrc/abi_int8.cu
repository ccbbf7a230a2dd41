// extern "C" entry points of the 8-bit serving path (declared in
// include/gptq.h): every argument is checked on the host before anything is
// launched.
#include <cmath>

#include "internal.cuh"

using namespace gptq;

namespace gptq {
namespace {

constexpr int64_t kMaxIn = 32768;
constexpr int64_t kMaxOut = 65535;
constexpr int64_t kMaxTokens = 1ll << 26;

bool dtype_ok(gptq_dtype_t t) { return t == GPTQ_F16 || t == GPTQ_BF16 || t == GPTQ_F32; }
bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
uintptr_t esize(gptq_dtype_t t) { return t == GPTQ_F32 ? 4 : 2; }

gptq_status_t check_sizes(int64_t tokens, int64_t in, int64_t out) {
  if (tokens < 0) return fail(GPTQ_ERR_INVALID_ARG, "tokens must be >= 0 (got %lld)", (long long)tokens);
  if (in < 1) return fail(GPTQ_ERR_INVALID_ARG, "in must be >= 1 (got %lld)", (long long)in);
  if (out < 0) return fail(GPTQ_ERR_INVALID_ARG, "out must be >= 0 (got %lld)", (long long)out);
  if (tokens > kMaxTokens || in > kMaxIn || out > kMaxOut)
    return fail(GPTQ_ERR_UNSUPPORTED,
                "%lld tokens of a %lld x %lld layer exceed this build's limits (tokens <= %lld, in <= %lld, out <= "
                "%lld)",
                (long long)tokens, (long long)out, (long long)in, (long long)kMaxTokens, (long long)kMaxIn,
                (long long)kMaxOut);
  return GPTQ_OK;
}

// An int8 matrix the kernels read in 16-byte units.
gptq_status_t check_int8(const char* name, const void* p, int64_t ld, int64_t in) {
  if (!p) return fail(GPTQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 16)) return fail(GPTQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (ld < in || ld % 16 != 0)
    return fail(GPTQ_ERR_INVALID_ARG, "%s: the row stride (%lld) must be a multiple of 16 and >= in (%lld)", name,
                (long long)ld, (long long)in);
  return GPTQ_OK;
}

// A floating matrix: rows of `cols` elements of type t, stride ld.
gptq_status_t check_rows(const char* name, const void* p, int64_t ld, int64_t cols, gptq_dtype_t t) {
  if (!p) return fail(GPTQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, esize(t))) return fail(GPTQ_ERR_INVALID_ARG, "%s is not aligned to its element type", name);
  if (ld < cols)
    return fail(GPTQ_ERR_INVALID_ARG, "%s: row stride %lld < %lld columns", name, (long long)ld, (long long)cols);
  return GPTQ_OK;
}

gptq_status_t check_vector(const char* name, const void* p, uintptr_t element) {
  if (!p) return fail(GPTQ_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, element)) return fail(GPTQ_ERR_INVALID_ARG, "%s is not aligned to its element type", name);
  return GPTQ_OK;
}

#define TRY(x)                                \
  do {                                        \
    const gptq_status_t s_ = (x);             \
    if (s_ != GPTQ_OK) return s_;             \
  } while (0)

gptq_status_t check_tokens(const gptq_int8_tokens_t* x, int64_t in) {
  if (!x) return fail(GPTQ_ERR_INVALID_ARG, "x is NULL");
  TRY(check_int8("x.q", x->q, x->ldq, in));
  TRY(check_vector("x.scale", x->scale, 4));
  return check_vector("x.sum", x->sum, 4);
}

gptq_status_t check_layer(const char* name, const gptq_int8_layer_t* w, int64_t in) {
  if (!w) return fail(GPTQ_ERR_INVALID_ARG, "%s is NULL", name);
  TRY(check_int8(name, w->w, w->ldw, in));
  TRY(check_vector(name, w->scale, 4));
  if (w->zero) TRY(check_vector(name, w->zero, 4));
  return GPTQ_OK;
}

gptq_status_t check_norm(const gptq_norm_t* a) {
  if (!dtype_ok(a->yt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown yt %d", (int)a->yt);
  if (a->ht != a->yt && a->ht != GPTQ_F32)
    return fail(GPTQ_ERR_INVALID_ARG, "the residual stream's type must be yt or fp32");
  if (a->kind != GPTQ_NORM_RMS && a->kind != GPTQ_NORM_LAYER)
    return fail(GPTQ_ERR_INVALID_ARG, "unknown norm kind %d", (int)a->kind);
  if (!std::isfinite(a->eps) || a->eps < 0.f) return fail(GPTQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (a->tokens == 0) return GPTQ_OK;
  const int64_t d = a->d;
  TRY(check_rows("h", a->h, a->ldh, d, a->ht));
  if (a->y) TRY(check_rows("y", a->y, a->ldy, d, a->yt));
  if (!a->y && (a->post_weight || a->gate)) return fail(GPTQ_ERR_INVALID_ARG, "post_weight and gate need y");
  if (a->post_weight) TRY(check_vector("post_weight", a->post_weight, esize(a->yt)));
  if (a->post_bias && !a->post_weight) return fail(GPTQ_ERR_INVALID_ARG, "post_bias needs post_weight");
  if (a->post_bias) TRY(check_vector("post_bias", a->post_bias, esize(a->yt)));
  if (a->gate) {
    TRY(check_vector("gate", a->gate, esize(a->yt)));
    if (a->ldgate != 0 && a->ldgate < d)
      return fail(GPTQ_ERR_INVALID_ARG, "gate: row stride %lld is neither 0 nor >= %lld", (long long)a->ldgate,
                  (long long)d);
  }
  if (a->weight) TRY(check_vector("weight", a->weight, esize(a->yt)));
  if (a->bias && !a->weight) return fail(GPTQ_ERR_INVALID_ARG, "bias needs weight");
  if (a->bias) TRY(check_vector("bias", a->bias, esize(a->yt)));
  if (a->h_out) TRY(check_rows("h_out", a->h_out, a->ldh_out, d, a->ht));
  if (a->h_out == a->h && a->ldh_out != a->ldh)
    return fail(GPTQ_ERR_INVALID_ARG, "h_out == h needs ldh_out == ldh");
  if ((a->x || a->q) && !a->weight) return fail(GPTQ_ERR_INVALID_ARG, "x and q need weight");
  if (a->weight && !a->x && !a->q) return fail(GPTQ_ERR_INVALID_ARG, "weight needs x or q");
  if (!a->h_out && !a->x && !a->q) return fail(GPTQ_ERR_INVALID_ARG, "no output is requested");
  if (a->x) TRY(check_rows("x", a->x, a->ldx, d, a->yt));
  if (a->q) {
    TRY(check_int8("q", a->q, a->ldq, d));
    TRY(check_vector("scale", a->scale, 4));
    TRY(check_vector("sum", a->sum, 4));
  }
  return GPTQ_OK;
}

}  // namespace
}  // namespace gptq

extern "C" {

gptq_status_t gptq_layout_int8(const uint32_t* qweight, const int32_t* zeros, int64_t out, int64_t in, int bits,
                               int8_t* w, int64_t ldw, int32_t* zero, void* stream) {
  clear_error();
  if (bits != 2 && bits != 3 && bits != 4 && bits != 8)
    return fail(GPTQ_ERR_INVALID_ARG, "bits must be 2, 3, 4 or 8 (got %d)", bits);
  TRY(check_sizes(0, in, out));
  if ((in * bits) % 32 != 0)
    return fail(GPTQ_ERR_UNSUPPORTED, "packed codes need in*bits %% 32 == 0 (in=%lld, bits=%d)", (long long)in, bits);
  if (out == 0) return GPTQ_OK;
  TRY(check_vector("qweight", qweight, 4));
  TRY(check_vector("zeros", zeros, 4));
  TRY(check_int8("w", w, ldw, in));
  if (zero) TRY(check_vector("zero", zero, 4));
  TRY(check_device());
  return layout_int8(qweight, zeros, out, in, bits, w, ldw, zero, (cudaStream_t)stream);
}

gptq_status_t gptq_quantize_tokens(const void* X, gptq_dtype_t xt, int64_t tokens, int64_t in, int64_t ldx, int8_t* q,
                                   int64_t ldq, float* scale, int32_t* sum, void* stream) {
  clear_error();
  TRY(check_sizes(tokens, in, 0));
  if (!dtype_ok(xt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown X dtype %d", (int)xt);
  if (tokens == 0) return GPTQ_OK;
  TRY(check_rows("X", X, ldx, in, xt));
  TRY(check_int8("q", q, ldq, in));
  TRY(check_vector("scale", scale, 4));
  TRY(check_vector("sum", sum, 4));
  TRY(check_device());
  return quantize_tokens(X, xt, tokens, in, ldx, q, ldq, scale, sum, (cudaStream_t)stream);
}

gptq_status_t gptq_norm_tokens(const gptq_norm_t* args, void* stream) {
  clear_error();
  if (!args) return fail(GPTQ_ERR_INVALID_ARG, "args is NULL");
  TRY(check_sizes(args->tokens, args->d, 0));
  TRY(check_norm(args));
  if (args->tokens == 0) return GPTQ_OK;
  TRY(check_device());
  return norm_tokens(args, (cudaStream_t)stream);
}

gptq_status_t gptq_matmul_int8(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in, const gptq_int8_layer_t* w,
                               int64_t out, const float* bias, void* Y, gptq_dtype_t yt, int64_t ldy, void* stream) {
  clear_error();
  TRY(check_sizes(tokens, in, out));
  if (!dtype_ok(yt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown Y dtype %d", (int)yt);
  if (tokens == 0 || out == 0) return GPTQ_OK;
  TRY(check_tokens(x, in));
  TRY(check_layer("w", w, in));
  if (bias) TRY(check_vector("bias", bias, 4));
  TRY(check_rows("Y", Y, ldy, out, yt));
  TRY(check_device());
  return matmul_int8(x, tokens, in, w, out, bias, Y, yt, ldy, (cudaStream_t)stream);
}

gptq_status_t gptq_matmul_int8_gated(const gptq_int8_tokens_t* x, int64_t tokens, int64_t in,
                                     const gptq_int8_layer_t* gate, const gptq_int8_layer_t* up, int64_t out,
                                     gptq_act_t act, void* Y, gptq_dtype_t yt, int64_t ldy, void* stream) {
  clear_error();
  TRY(check_sizes(tokens, in, out));
  if (!dtype_ok(yt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown Y dtype %d", (int)yt);
  if (act != GPTQ_ACT_SILU && act != GPTQ_ACT_GELU && act != GPTQ_ACT_GELU_TANH)
    return fail(GPTQ_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  if (tokens == 0 || out == 0) return GPTQ_OK;
  TRY(check_tokens(x, in));
  TRY(check_layer("gate", gate, in));
  TRY(check_layer("up", up, in));
  TRY(check_rows("Y", Y, ldy, out, yt));
  TRY(check_device());
  return matmul_int8_gated(x, tokens, in, gate, up, out, (int)act, Y, yt, ldy, (cudaStream_t)stream);
}

size_t gptq_linear_int8_ws_bytes(int64_t tokens, int64_t in) {
  if (tokens < 0 || tokens > kMaxTokens || in < 1 || in > kMaxIn) return 0;
  return linear_int8_ws_bytes(tokens, in);
}

gptq_status_t gptq_linear_int8(const void* X, gptq_dtype_t xt, int64_t tokens, int64_t in, int64_t ldx,
                               const gptq_int8_layer_t* w, int64_t out, const float* bias, void* Y, gptq_dtype_t yt,
                               int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  TRY(check_sizes(tokens, in, out));
  if (!dtype_ok(xt) || !dtype_ok(yt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown dtype (X %d, Y %d)", (int)xt, (int)yt);
  if (tokens == 0 || out == 0) return GPTQ_OK;
  TRY(check_rows("X", X, ldx, in, xt));
  TRY(check_layer("w", w, in));
  if (bias) TRY(check_vector("bias", bias, 4));
  TRY(check_rows("Y", Y, ldy, out, yt));
  const size_t need = linear_int8_ws_bytes(tokens, in);
  if (need) TRY(check_ws(ws, ws_bytes, need));
  TRY(check_device());
  return linear_int8(X, xt, tokens, in, ldx, w, nullptr, out, bias, 0, Y, yt, ldy, ws, (cudaStream_t)stream);
}

gptq_status_t gptq_linear_int8_gated(const void* X, gptq_dtype_t xt, int64_t tokens, int64_t in, int64_t ldx,
                                     const gptq_int8_layer_t* gate, const gptq_int8_layer_t* up, int64_t out,
                                     gptq_act_t act, void* Y, gptq_dtype_t yt, int64_t ldy, void* ws, size_t ws_bytes,
                                     void* stream) {
  clear_error();
  TRY(check_sizes(tokens, in, out));
  if (!dtype_ok(xt) || !dtype_ok(yt)) return fail(GPTQ_ERR_INVALID_ARG, "unknown dtype (X %d, Y %d)", (int)xt, (int)yt);
  if (act != GPTQ_ACT_SILU && act != GPTQ_ACT_GELU && act != GPTQ_ACT_GELU_TANH)
    return fail(GPTQ_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  if (tokens == 0 || out == 0) return GPTQ_OK;
  TRY(check_rows("X", X, ldx, in, xt));
  TRY(check_layer("gate", gate, in));
  TRY(check_layer("up", up, in));
  TRY(check_rows("Y", Y, ldy, out, yt));
  const size_t need = linear_int8_ws_bytes(tokens, in);
  if (need) TRY(check_ws(ws, ws_bytes, need));
  TRY(check_device());
  return linear_int8(X, xt, tokens, in, ldx, gate, up, out, nullptr, (int)act, Y, yt, ldy, ws, (cudaStream_t)stream);
}

gptq_status_t gptq_int8_status(void* stream) {
  clear_error();
  TRY(check_device());
  return int8_status((cudaStream_t)stream);
}

}  // extern "C"
