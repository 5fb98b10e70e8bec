// C ABI of the decode step's operators around the matrix products: argument
// checks and dispatch (contracts in include/wobs.h).
#include <cstdarg>
#include <cstdio>

#include "../../include/wobs.h"
#include "internal.h"

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return wobs::set_error(code, msg);
}

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int bytes_of(int dtype) { return dtype == WOBS_DTYPE_F32 ? 4 : 2; }
bool known(int dtype) { return dtype >= WOBS_DTYPE_F16 && dtype <= WOBS_DTYPE_F32; }

// A row-major operand whose rows must start on 16-byte boundaries.
int check_rows(const char* op, const char* what, const void* p, int dtype, int64_t ld, int M, int K) {
  if (!known(dtype)) return fail(WOBS_ERR_INVALID_ARG, "%s: %s dtype %d (1 fp16, 2 bf16, 3 fp32)", op, what, dtype);
  if (M > 1 && ld < K) return fail(WOBS_ERR_INVALID_ARG, "%s: %s pitch smaller than K", op, what);
  if (!aligned(p, 16) || (M > 1 && (ld * bytes_of(dtype)) % 16))
    return fail(WOBS_ERR_MISALIGNED, "%s: %s rows must be 16-byte aligned", op, what);
  return WOBS_OK;
}

// The cache and the sequences' tables; fills the kernels' view of them.
int check_cache(const char* op, const wobs_kv4_cache* c, int B, int L, const int32_t* table, int64_t ldt,
                int max_pages, const int32_t* lens, wobs::Kv4Args* out) {
  if (!c || !c->kq || !c->kd || !c->vq || !c->vd || !table || !lens)
    return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (B < 1 || L < 1 || max_pages < 1 || c->pages < 1 || c->heads < 1)
    return fail(WOBS_ERR_INVALID_ARG, "%s: B=%d L=%d max_pages=%d pages=%d heads=%d (all at least 1)", op, B, L, max_pages, c->pages, c->heads);
  if (B > 1 && ldt < max_pages) return fail(WOBS_ERR_INVALID_ARG, "%s: table pitch smaller than max_pages", op);
  if (c->page_size < 16 || c->page_size % 16)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: page_size=%d not a positive multiple of 16", op, c->page_size);
  if (c->dim != 64 && c->dim != 128 && c->dim != 256)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: dim=%d (64, 128 or 256)", op, c->dim);
  if (static_cast<double>(c->heads) * c->page_size * c->dim > 2147483647.0)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: a page of more than 2^31 elements", op);
  // positions are 32-bit, those of the steps that a kernel looks ahead among them
  if (static_cast<int64_t>(max_pages) * c->page_size > (1ll << 31) - 1024)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: %d pages of %d tokens a sequence, more than 2^31 - 1024", op, max_pages, c->page_size);
  if (!aligned(c->kq, 16) || !aligned(c->vq, 16) || !aligned(c->kd, 16) || !aligned(c->vd, 16))
    return fail(WOBS_ERR_MISALIGNED, "%s: cache planes must be 16-byte aligned", op);
  if (!aligned(table, 4) || !aligned(lens, 4)) return fail(WOBS_ERR_MISALIGNED, "%s: table / lens not 4-byte aligned", op);
  *out = wobs::Kv4Args{c->kq, c->vq, static_cast<__half*>(c->kd), static_cast<__half*>(c->vd), c->pages, c->page_size,
                       c->heads, c->dim, table, ldt, max_pages, lens, wobs::error_word_ptr()};
  return WOBS_OK;
}

// The grid of the token kernels: a row a sequence, a lane for four elements or eight.
bool too_many_tokens(const wobs::Kv4Args& c, int B, int L) {
  return B > 65535 || static_cast<double>(L) * c.heads * (c.dim >> 2) > 4294967040.0;
}

int check_strided(const char* op, const char* what, const void* p, const int64_t* strides, int es) {
  if (!p || !strides) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (!aligned(p, es)) return fail(WOBS_ERR_MISALIGNED, "%s: %s not aligned to its element size", op, what);
  return WOBS_OK;
}

}  // namespace

extern "C" {

int wobs_rmsnorm_q8_1(int x_dtype, const void* X, int64_t ldx, int res_dtype, const void* residual, int64_t ldr,
                      void* residual_out, int64_t ldh, int w_dtype, const void* w, float eps, int M, int K, void* xq,
                      int y_dtype, void* Y, int64_t ldy, void* stream) {
  const char* op = "rmsnorm_q8_1";
  if (!X || !w || (!xq && !Y)) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if ((residual == nullptr) != (residual_out == nullptr))
    return fail(WOBS_ERR_INVALID_ARG, "%s: residual and residual_out go together", op);
  if (M < 1) return fail(WOBS_ERR_INVALID_ARG, "%s: M=%d", op, M);
  if (!(eps >= 0.f)) return fail(WOBS_ERR_INVALID_ARG, "%s: eps must not be negative", op);
  if (K < 32 || K % 32 || K > wobs::kRmsNormMaxK)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: K=%d not a positive multiple of 32, at most %d", op, K, wobs::kRmsNormMaxK);
  int rc = check_rows(op, "X", X, x_dtype, ldx, M, K);
  if (!rc) rc = check_rows(op, "w", w, w_dtype, K, 1, K);
  if (!rc && residual) rc = check_rows(op, "residual", residual, res_dtype, ldr, M, K);
  if (!rc && residual) rc = check_rows(op, "residual_out", residual_out, res_dtype, ldh, M, K);
  if (!rc && Y) rc = check_rows(op, "Y", Y, y_dtype, ldy, M, K);
  if (rc) return rc;
  if (!aligned(xq, 4)) return fail(WOBS_ERR_MISALIGNED, "%s: xq not 4-byte aligned", op);
  wobs::RmsNormArgs a;
  a.x = X; a.residual = residual; a.w = w; a.h = residual_out; a.y = Y;
  a.xq = static_cast<uint8_t*>(xq);
  a.ldx = ldx; a.ldr = ldr; a.ldh = ldh; a.ldy = ldy;
  a.x_dtype = x_dtype; a.r_dtype = res_dtype; a.w_dtype = w_dtype; a.y_dtype = y_dtype;
  a.K = K; a.eps = eps;
  wobs::Launch L;
  const cudaError_t e = wobs::launch_rmsnorm_q8_1(a, M, static_cast<cudaStream_t>(stream), &L);
  return wobs::report_launch(e, op, M, 0, K, L, 1);
}

int wobs_dequantize_q8_1(const void* xq, int M, int K, int dtype, void* X, void* stream) {
  const char* op = "dequantize_q8_1";
  if (!xq || !X) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (!known(dtype)) return fail(WOBS_ERR_INVALID_ARG, "%s: dtype %d (1 fp16, 2 bf16, 3 fp32)", op, dtype);
  if (M < 1) return fail(WOBS_ERR_INVALID_ARG, "%s: M=%d", op, M);
  if (K < 32 || K % 32) return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: K=%d not a positive multiple of 32", op, K);
  const int64_t blocks = static_cast<int64_t>(M) * (K >> 5);
  if (blocks > (1ll << 36)) return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: more than 2^36 blocks", op);
  if (!aligned(xq, 4) || !aligned(X, 16)) return fail(WOBS_ERR_MISALIGNED, "%s: xq 4-byte, X 16-byte aligned", op);
  wobs::Launch L;
  const cudaError_t e = wobs::launch_dequantize_q8_1(xq, blocks, dtype, X, static_cast<cudaStream_t>(stream), &L);
  return wobs::report_launch(e, op, M, 0, K, L, 1);
}

int wobs_kv4_append(const wobs_kv4_cache* cache, int dtype, const void* K, const int64_t* k_strides, const void* V,
                    const int64_t* v_strides, int B, int L, const int32_t* table, int64_t ld_table, int max_pages,
                    const int32_t* lens, void* stream) {
  const char* op = "kv4_append";
  wobs::Kv4Args c;
  int rc = check_cache(op, cache, B, L, table, ld_table, max_pages, lens, &c);
  if (rc) return rc;
  if (!known(dtype)) return fail(WOBS_ERR_INVALID_ARG, "%s: dtype %d (1 fp16, 2 bf16, 3 fp32)", op, dtype);
  rc = check_strided(op, "K", K, k_strides, bytes_of(dtype));
  if (!rc) rc = check_strided(op, "V", V, v_strides, bytes_of(dtype));
  if (rc) return rc;
  if (too_many_tokens(c, B, L)) return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: more than 65535 sequences, or L x heads x dim past 2^34", op);
  wobs::Launch info;
  const cudaError_t e = wobs::launch_kv4_append(c, dtype, {K, k_strides[0], k_strides[1], k_strides[2]},
                                                {V, v_strides[0], v_strides[1], v_strides[2]}, B, L,
                                                static_cast<cudaStream_t>(stream), &info);
  return wobs::report_launch(e, op, B * L, c.heads, c.dim, info, 1);
}

int wobs_kv4_read(const wobs_kv4_cache* cache, const int32_t* table, int64_t ld_table, int max_pages,
                  const int32_t* lens, int B, int L, int dtype, void* K, void* V, void* stream) {
  const char* op = "kv4_read";
  wobs::Kv4Args c;
  int rc = check_cache(op, cache, B, L, table, ld_table, max_pages, lens, &c);
  if (rc) return rc;
  if (!K || !V) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (!known(dtype)) return fail(WOBS_ERR_INVALID_ARG, "%s: dtype %d (1 fp16, 2 bf16, 3 fp32)", op, dtype);
  if (!aligned(K, 16) || !aligned(V, 16)) return fail(WOBS_ERR_MISALIGNED, "%s: K and V must be 16-byte aligned", op);
  if (too_many_tokens(c, B, L)) return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: more than 65535 sequences, or L x heads x dim past 2^34", op);
  wobs::Launch info;
  const cudaError_t e = wobs::launch_kv4_read(c, dtype, K, V, B, L, static_cast<cudaStream_t>(stream), &info);
  return wobs::report_launch(e, op, B * L, c.heads, c.dim, info, 1);
}

int wobs_attn_kv4(const wobs_kv4_cache* cache, int dtype, const void* Q, const int64_t* q_strides, int B, int L,
                  int q_heads, float scale, const int32_t* table, int64_t ld_table, int max_pages, const int32_t* lens,
                  int out_dtype, void* O, void* ws, size_t ws_bytes, void* stream) {
  const char* op = "attn_kv4";
  wobs::Kv4Args c;
  int rc = check_cache(op, cache, B, L, table, ld_table, max_pages, lens, &c);
  if (rc) return rc;
  if (!O) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (dtype != WOBS_DTYPE_F16 && dtype != WOBS_DTYPE_BF16)
    return fail(WOBS_ERR_INVALID_ARG, "%s: Q dtype %d (1 fp16, 2 bf16)", op, dtype);
  if (out_dtype != dtype && out_dtype != WOBS_DTYPE_F32)
    return fail(WOBS_ERR_INVALID_ARG, "%s: output dtype %d (the queries' or 3 fp32)", op, out_dtype);
  if (L > WOBS_MAX_M) return fail(WOBS_ERR_INVALID_ARG, "%s: L=%d outside 1..%d", op, L, WOBS_MAX_M);
  if (q_heads < 1 || q_heads % c.heads)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: %d query heads over %d cache heads", op, q_heads, c.heads);
  rc = check_strided(op, "Q", Q, q_strides, 2);
  if (rc) return rc;
  if (!aligned(O, 16)) return fail(WOBS_ERR_MISALIGNED, "%s: O must be 16-byte aligned", op);
  const int group = q_heads / c.heads;
  // one arrival counter for each row tile of a sequence's cache head
  if (static_cast<double>(B) * c.heads * wobs::attn_kv4_tiles(L, group, c.dim) > 65536.0)
    return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: more than 65536 row tiles (B x heads x L x group)", op);
  wobs::SplitArgs sk{nullptr, nullptr, 1};
  wobs::ArgmaxArgs am;
  rc = wobs::prepare_workspace(WOBS_OP_ATTN_KV4, B * L, q_heads, c.dim, nullptr, ws, ws_bytes, &sk, &am);
  if (rc) return rc;
  const bool q_vec = aligned(Q, 8) && q_strides[0] % 4 == 0 && q_strides[1] % 4 == 0 && q_strides[2] % 4 == 0;
  wobs::AttnKv4Args a{{Q, q_strides[0], q_strides[1], q_strides[2]}, dtype, out_dtype, q_vec, O, B, L, group, scale, sk.partials, sk.counters};
  wobs::Launch info;
  const cudaError_t e = wobs::launch_attn_kv4(c, a, static_cast<cudaStream_t>(stream), &info);
  return wobs::report_launch(e, op, B * L, q_heads, c.dim, info, 1);
}

int wobs_sample(int dtype, const void* logits, int64_t ld, int M, int N, const float* u, const float* temperature,
                const int32_t* top_k, const float* top_p, const float* min_p, int64_t* token, float* prob,
                void* stream) {
  const char* op = "sample";
  if (!logits || !u || !token) return fail(WOBS_ERR_INVALID_ARG, "%s: null pointer", op);
  if (!known(dtype)) return fail(WOBS_ERR_INVALID_ARG, "%s: dtype %d (1 fp16, 2 bf16, 3 fp32)", op, dtype);
  if (M < 1 || M > 65535) return fail(WOBS_ERR_INVALID_ARG, "%s: M=%d outside 1..65535", op, M);
  if (N < 1 || N > wobs::kSampleMaxN) return fail(WOBS_ERR_UNSUPPORTED_SHAPE, "%s: N=%d outside 1..%d", op, N, wobs::kSampleMaxN);
  if (M > 1 && ld < N) return fail(WOBS_ERR_INVALID_ARG, "%s: ld < N", op);
  if (!aligned(logits, bytes_of(dtype))) return fail(WOBS_ERR_MISALIGNED, "%s: logits not aligned to their element size", op);
  if (!aligned(token, 8) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) || !aligned(top_p, 4) ||
      !aligned(min_p, 4) || !aligned(prob, 4))
    return fail(WOBS_ERR_MISALIGNED, "%s: token 8-byte, the other arrays 4-byte aligned", op);
  wobs::SampleArgs a{logits, M > 1 ? ld : N, dtype, M, N, u, temperature, top_p, min_p, top_k, token, prob};
  wobs::Launch L;
  const cudaError_t e = wobs::launch_sample(a, static_cast<cudaStream_t>(stream), &L);
  return wobs::report_launch(e, op, M, N, 0, L, 1);
}

}  // extern "C"
