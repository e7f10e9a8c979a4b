// attn_api.cu — the extern "C" entry points of the paged cache and attention
// operators (declared in mxq.h): host-side checks, then one launch function.
#include <algorithm>
#include <cmath>
#include <string>

#include "attn.h"
#include "internal.h"
#include "mxq.h"

using namespace mxq;

namespace {

mxq_status fail(mxq_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}

mxq_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MXQ_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A tensor [n0, n1, D] of `es`-byte elements read and written in `bytes`-byte
// pieces: its base and both outer strides are multiples of that.
mxq_status check_rows(const char* name, const void* p, int64_t n0, int64_t n1, int64_t s0,
                      int64_t s1, int64_t D, int es, size_t bytes) {
  if (!p) return fail(MXQ_ERR_INVALID_ARG, std::string(name) + " must be non-NULL");
  if ((n0 > 1 && s0 < D) || (n1 > 1 && s1 < D))
    return fail(MXQ_ERR_INVALID_ARG, std::string(name) + ": strides below the head dimension");
  if (!aligned(p, bytes) || (n0 > 1 && s0 * es % static_cast<int64_t>(bytes) != 0) ||
      (n1 > 1 && s1 * es % static_cast<int64_t>(bytes) != 0))
    return fail(MXQ_ERR_UNSUPPORTED, std::string(name) + " needs a base and strides of " +
                                         std::to_string(bytes) + "-byte multiples");
  return MXQ_OK;
}

mxq_status check_cache(const char* name, const void* p, int32_t dtype, int64_t pages,
                       int32_t page_size, int32_t Hkv, int32_t D, int64_t sp, int64_t st,
                       int64_t sh, bool scaled, size_t bytes) {
  if (dtype != MXQ_BF16 && dtype != MXQ_E4M3)
    return fail(MXQ_ERR_UNSUPPORTED, "cache_dtype must be MXQ_BF16 or MXQ_E4M3");
  if (scaled && dtype != MXQ_E4M3)
    return fail(MXQ_ERR_INVALID_ARG, "a bf16 cache takes no scales");
  const int es = dtype == MXQ_E4M3 ? 1 : 2;
  const mxq_status r = check_rows(name, p, page_size, Hkv, st, sh, D, es, bytes);
  if (r != MXQ_OK) return r;
  if (pages > 1 && sp < D)
    return fail(MXQ_ERR_INVALID_ARG, std::string(name) + ": strides below the head dimension");
  if (pages > 1 && sp * es % static_cast<int64_t>(bytes) != 0)
    return fail(MXQ_ERR_UNSUPPORTED, std::string(name) + " needs a base and strides of " +
                                         std::to_string(bytes) + "-byte multiples");
  return MXQ_OK;
}

// Head counts and head dimension of the two attention operators.
mxq_status check_heads(int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hq <= 0 || Hkv <= 0) return fail(MXQ_ERR_INVALID_ARG, "need Hq > 0 and Hkv > 0");
  if (Hq % Hkv != 0)
    return fail(MXQ_ERR_INVALID_ARG, "Hq (" + std::to_string(Hq) + ") must be a multiple of Hkv (" +
                                         std::to_string(Hkv) + ")");
  if (Hq / Hkv > 128 || Hkv > 65535)
    return fail(MXQ_ERR_UNSUPPORTED, "at most 128 query heads per key/value head, 65535 of those");
  if (D != 64 && D != 128)
    return fail(MXQ_ERR_UNSUPPORTED, "the head dimension must be 64 or 128; got " +
                                         std::to_string(D));
  return MXQ_OK;
}

mxq_status check_scale(float scale, int32_t window, int32_t first) {
  // (the kernels multiply it by log2 e)
  if (!(scale > 0.f) || !std::isfinite(scale * 1.44269504088896340736f))
    return fail(MXQ_ERR_INVALID_ARG, "scale must be positive and finite, times log2 e as well");
  if (window < 0 || first < 0)
    return fail(MXQ_ERR_INVALID_ARG, "window and first must be >= 0 (0: none)");
  return MXQ_OK;
}

// first keys that stay visible before a window: without one all do
int first_keys(int32_t window, int32_t first) {
  return window > 0 ? std::min(first, 1 << 30) : 0;
}

mxq_status check_workspace(const void* ws, size_t have, size_t need, const char* query) {
  if (need == 0) return MXQ_OK;
  if (!ws || have < need)
    return fail(MXQ_ERR_INVALID_ARG, "workspace of " + std::to_string(ws ? have : 0) +
                                         " bytes is smaller than the " + std::to_string(need) +
                                         " of " + query);
  if (!aligned(ws, 256))
    return fail(MXQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return MXQ_OK;
}

}  // namespace

#define MXQ_TRY(expr)                       \
  do {                                      \
    const mxq_status st_ = (expr);          \
    if (st_ != MXQ_OK) return st_;          \
  } while (0)

extern "C" mxq_status mxq_rope_append_kv(
    const void* q, int64_t sq_t, int64_t sq_h, int32_t Hq, void* q_out, int64_t so_t, int64_t so_h,
    const void* k, int64_t sk_t, int64_t sk_h, const void* v, int64_t sv_t, int64_t sv_h, int64_t T,
    int32_t Hkv, int32_t D, const float* cos_sin, int64_t max_pos, int32_t rot,
    const int32_t* positions, int32_t interleaved, const int64_t* slots, void* k_cache,
    void* v_cache, int32_t cache_dtype, int64_t pages, int32_t page_size, int64_t sck_p,
    int64_t sck_t, int64_t sck_h, int64_t scv_p, int64_t scv_t, int64_t scv_h,
    const float* k_scale, const float* v_scale, mxq_stream_t stream) {
  if (T < 0 || Hkv <= 0 || D <= 0 || Hq < 0)
    return fail(MXQ_ERR_INVALID_ARG, "need T >= 0, Hq >= 0, Hkv > 0 and D > 0");
  if (D % 16 != 0 || D > 512)
    return fail(MXQ_ERR_UNSUPPORTED, "the head dimension must be a multiple of 16 up to 512");
  if (rot < 0 || rot > D || rot % 16 != 0)
    return fail(MXQ_ERR_INVALID_ARG, "rot must be a multiple of 16 in [0, D]");
  if (Hq > 65535 || Hkv > 65535) return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 heads");
  if (pages <= 0 || page_size <= 0 || pages > (int64_t(1) << 40))
    return fail(MXQ_ERR_INVALID_ARG, "need pages > 0 and page_size > 0");
  if (pages > (int64_t(1) << 60) / page_size)
    return fail(MXQ_ERR_INVALID_ARG, "more than 2^60 cache slots");
  if ((q == nullptr) != (Hq == 0) || (q && !q_out))
    return fail(MXQ_ERR_INVALID_ARG, "q, q_out and Hq > 0 go together");
  if (T == 0) return MXQ_OK;
  if (!slots) return fail(MXQ_ERR_INVALID_ARG, "slots must be non-NULL");
  if (!aligned(slots, 8)) return fail(MXQ_ERR_INVALID_ARG, "slots must be 8-byte aligned");
  if (rot > 0) {
    if (!cos_sin || !positions || max_pos <= 0)
      return fail(MXQ_ERR_INVALID_ARG, "a rotation needs cos_sin, max_pos > 0 and positions");
    if (!aligned(cos_sin, 16) || !aligned(positions, 4))
      return fail(MXQ_ERR_UNSUPPORTED,
                  "cos_sin needs a 16-byte aligned base, positions a 4-byte one");
  }
  if (q) {
    MXQ_TRY(check_rows("q", q, T, Hq, sq_t, sq_h, D, 2, 16));
    MXQ_TRY(check_rows("q_out", q_out, T, Hq, so_t, so_h, D, 2, 16));
    if (q == q_out && (sq_t != so_t || sq_h != so_h))
      return fail(MXQ_ERR_INVALID_ARG, "q rotated in place needs equal strides of q and q_out");
  }
  MXQ_TRY(check_rows("k", k, T, Hkv, sk_t, sk_h, D, 2, 16));
  MXQ_TRY(check_rows("v", v, T, Hkv, sv_t, sv_h, D, 2, 16));
  const size_t piece = cache_dtype == MXQ_E4M3 ? 8 : 16;
  const bool scaled = k_scale || v_scale;
  MXQ_TRY(check_cache("k_cache", k_cache, cache_dtype, pages, page_size, Hkv, D, sck_p, sck_t,
                      sck_h, scaled, piece));
  MXQ_TRY(check_cache("v_cache", v_cache, cache_dtype, pages, page_size, Hkv, D, scv_p, scv_t,
                      scv_h, scaled, piece));
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(MXQ_ERR_INVALID_ARG, "the cache scales must be 4-byte aligned");
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  RopeAppendParams p = {};
  p.q = q, p.k = k, p.v = v;
  p.q_t = sq_t, p.q_h = sq_h, p.k_t = sk_t, p.k_h = sk_h, p.v_t = sv_t, p.v_h = sv_h;
  p.q_out = q_out, p.o_t = so_t, p.o_h = so_h;
  p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.D = D, p.rot = rot;
  p.interleaved = interleaved != 0, p.fp8 = cache_dtype == MXQ_E4M3;
  p.cos_sin = cos_sin, p.max_pos = max_pos, p.positions = positions, p.slots = slots;
  p.k_cache = k_cache, p.v_cache = v_cache;
  p.slots_total = pages * page_size, p.page_size = page_size;
  p.ck_p = sck_p, p.ck_t = sck_t, p.ck_h = sck_h, p.cv_p = scv_p, p.cv_t = scv_t, p.cv_h = scv_h;
  p.k_scale = k_scale, p.v_scale = v_scale, p.status = d.status;
  const cudaError_t e = launch_rope_append(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "rope append launch");
}

extern "C" mxq_status mxq_paged_attention_decode_workspace_size(int64_t B, int32_t Hq, int32_t Hkv,
                                                                int32_t D, size_t* bytes) {
  if (!bytes || B < 0) return fail(MXQ_ERR_INVALID_ARG, "bad sizes or NULL result pointer");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  *bytes = 0;
  if (B == 0) return MXQ_OK;
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  *bytes = decode_workspace_bytes(B, Hq, Hkv, D, d.num_sms);
  return MXQ_OK;
}

extern "C" mxq_status mxq_paged_attention_decode_ex(
    const void* q, int64_t sq_b, int64_t sq_h, int64_t B, int32_t Hq, int32_t Hkv, int32_t D,
    const void* k_cache, const void* v_cache, int32_t cache_dtype, int64_t pages, int32_t page_size,
    int64_t sck_p, int64_t sck_t, int64_t sck_h, int64_t scv_p, int64_t scv_t, int64_t scv_h,
    const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* seq_lens,
    float scale, int32_t window, int32_t first, const float* sinks, const float* k_scale,
    const float* v_scale, void* out, int64_t so_b, int64_t so_h, float* lse, void* workspace,
    size_t ws_bytes, mxq_stream_t stream) {
  if (B < 0 || max_pages < 0) return fail(MXQ_ERR_INVALID_ARG, "need B >= 0 and max_pages >= 0");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  MXQ_TRY(check_scale(scale, window, first));
  if (pages <= 0 || page_size <= 0 || pages > 0x7fffffff)
    return fail(MXQ_ERR_INVALID_ARG, "need 0 < pages < 2^31 and page_size > 0");
  if (B == 0) return MXQ_OK;
  if (B > 65535) return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 sequences");
  if (max_pages > 0x7fffffff / 2 / page_size)
    return fail(MXQ_ERR_UNSUPPORTED, "sequences of more than 2^30 keys");
  if (!seq_lens || (max_pages > 0 && !page_table))
    return fail(MXQ_ERR_INVALID_ARG, "page_table and seq_lens must be non-NULL");
  if (ld_table < max_pages) return fail(MXQ_ERR_INVALID_ARG, "ld_table must be >= max_pages");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(sinks, 4) || !aligned(lse, 4) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  MXQ_TRY(check_rows("q", q, B, Hq, sq_b, sq_h, D, 2, 16));
  MXQ_TRY(check_rows("out", out, B, Hq, so_b, so_h, D, 2, 16));
  const bool scaled = k_scale || v_scale;
  MXQ_TRY(check_cache("k_cache", k_cache, cache_dtype, pages, page_size, Hkv, D, sck_p, sck_t,
                      sck_h, scaled, 16));
  MXQ_TRY(check_cache("v_cache", v_cache, cache_dtype, pages, page_size, Hkv, D, scv_p, scv_t,
                      scv_h, scaled, 16));
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  MXQ_TRY(check_workspace(workspace, ws_bytes, decode_workspace_bytes(B, Hq, Hkv, D, d.num_sms),
                          "mxq_paged_attention_decode_workspace_size"));
  DecodeParams p = {};
  p.q = q, p.q_b = sq_b, p.q_h = sq_h;
  p.B = static_cast<int>(B), p.Hq = Hq, p.Hkv = Hkv, p.D = D;
  p.k_cache = k_cache, p.v_cache = v_cache, p.fp8 = cache_dtype == MXQ_E4M3;
  p.pages = pages, p.page_size = page_size;
  p.ck_p = sck_p, p.ck_t = sck_t, p.ck_h = sck_h, p.cv_p = scv_p, p.cv_t = scv_t, p.cv_h = scv_h;
  p.page_table = page_table, p.ld_table = ld_table, p.max_pages = max_pages, p.seq_lens = seq_lens;
  p.scale = scale, p.window = std::min(window, 1 << 30), p.first = first_keys(window, first);
  p.sinks = sinks, p.k_scale = k_scale, p.v_scale = v_scale;
  p.out = out, p.o_b = so_b, p.o_h = so_h, p.lse = lse, p.workspace = workspace;
  p.status = d.status;
  const cudaError_t e = launch_decode(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "decode attention launch");
}

extern "C" mxq_status mxq_paged_attention_decode(
    const void* q, int64_t sq_b, int64_t sq_h, int64_t B, int32_t Hq, int32_t Hkv, int32_t D,
    const void* k_cache, const void* v_cache, int32_t cache_dtype, int64_t pages, int32_t page_size,
    int64_t sck_p, int64_t sck_t, int64_t sck_h, int64_t scv_p, int64_t scv_t, int64_t scv_h,
    const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* seq_lens,
    float scale, int32_t window, const float* sinks, const float* k_scale, const float* v_scale,
    void* out, int64_t so_b, int64_t so_h, float* lse, void* workspace, size_t ws_bytes,
    mxq_stream_t stream) {
  return mxq_paged_attention_decode_ex(q, sq_b, sq_h, B, Hq, Hkv, D, k_cache, v_cache, cache_dtype,
                                       pages, page_size, sck_p, sck_t, sck_h, scv_p, scv_t, scv_h,
                                       page_table, ld_table, max_pages, seq_lens, scale, window, 0,
                                       sinks, k_scale, v_scale, out, so_b, so_h, lse, workspace,
                                       ws_bytes, stream);
}

extern "C" mxq_status mxq_attention_varlen_workspace_size(int64_t Tq, int64_t B, int32_t Hq,
                                                          int32_t Hkv, int32_t D, size_t* bytes) {
  if (!bytes || B < 0 || Tq < 0)
    return fail(MXQ_ERR_INVALID_ARG, "bad sizes or NULL result pointer");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  *bytes = 0;
  if (B == 0 || Tq == 0) return MXQ_OK;
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  *bytes = prompt_workspace_bytes(Tq, B, Hq, Hkv, D, d.num_sms);
  return MXQ_OK;
}

extern "C" mxq_status mxq_attention_varlen_ex(
    const void* q, int64_t sq_t, int64_t sq_h, const void* k, int64_t sk_t, int64_t sk_h,
    const void* v, int64_t sv_t, int64_t sv_h, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int64_t B, int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hkv,
    int32_t D, float scale, int32_t causal, int32_t window, int32_t first, const float* sinks,
    void* out, int64_t so_t, int64_t so_h, float* lse, void* workspace, size_t ws_bytes,
    mxq_stream_t stream) {
  if (B < 0 || Tq < 0 || Tk < 0) return fail(MXQ_ERR_INVALID_ARG, "need B, Tq, Tk >= 0");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  MXQ_TRY(check_scale(scale, window, first));
  if (window > 0 && !causal)
    return fail(MXQ_ERR_INVALID_ARG, "a window needs a causal mask");
  if (B == 0 || Tq == 0) return MXQ_OK;
  if (B > 65535 || Tq > (1 << 30) || Tk > (1 << 30))
    return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 sequences or 2^30 tokens");
  if (!cu_seqlens_q || !cu_seqlens_k)
    return fail(MXQ_ERR_INVALID_ARG, "cu_seqlens_q and cu_seqlens_k must be non-NULL");
  if (!aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4) || !aligned(sinks, 4) ||
      !aligned(lse, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  MXQ_TRY(check_rows("q", q, Tq, Hq, sq_t, sq_h, D, 2, 16));
  MXQ_TRY(check_rows("out", out, Tq, Hq, so_t, so_h, D, 2, 16));
  if (Tk > 0) {
    MXQ_TRY(check_rows("k", k, Tk, Hkv, sk_t, sk_h, D, 2, 16));
    MXQ_TRY(check_rows("v", v, Tk, Hkv, sv_t, sv_h, D, 2, 16));
  }
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  MXQ_TRY(check_workspace(workspace, ws_bytes,
                          prompt_workspace_bytes(Tq, B, Hq, Hkv, D, d.num_sms),
                          "mxq_attention_varlen_workspace_size"));
  PromptParams p = {};
  p.q = q, p.q_t = sq_t, p.q_h = sq_h;
  p.k = k, p.k_t = sk_t, p.k_h = sk_h, p.v = v, p.v_t = sv_t, p.v_h = sv_h;
  p.cu_q = cu_seqlens_q, p.cu_k = cu_seqlens_k;
  p.B = static_cast<int>(B), p.Tq = Tq, p.Tk = Tk, p.Hq = Hq, p.Hkv = Hkv, p.D = D;
  p.scale = scale, p.causal = causal != 0, p.window = std::min(window, 1 << 30), p.sinks = sinks;
  p.first = first_keys(window, first);
  p.out = out, p.o_t = so_t, p.o_h = so_h, p.lse = lse, p.workspace = workspace;
  p.status = d.status;
  const cudaError_t e = launch_prompt(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream), &err);
  if (!err.empty()) return fail(MXQ_ERR_CUDA, err);
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "prompt attention launch");
}

extern "C" mxq_status mxq_attention_varlen(
    const void* q, int64_t sq_t, int64_t sq_h, const void* k, int64_t sk_t, int64_t sk_h,
    const void* v, int64_t sv_t, int64_t sv_h, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int64_t B, int64_t Tq, int64_t Tk, int32_t Hq, int32_t Hkv,
    int32_t D, float scale, int32_t causal, int32_t window, const float* sinks, void* out,
    int64_t so_t, int64_t so_h, float* lse, void* workspace, size_t ws_bytes,
    mxq_stream_t stream) {
  return mxq_attention_varlen_ex(q, sq_t, sq_h, k, sk_t, sk_h, v, sv_t, sv_h, cu_seqlens_q,
                                 cu_seqlens_k, B, Tq, Tk, Hq, Hkv, D, scale, causal, window, 0,
                                 sinks, out, so_t, so_h, lse, workspace, ws_bytes, stream);
}

namespace {

// `n` int32 places from p on; none where there are no rows
struct Extent {
  const int32_t* p;
  int64_t n, rows;
  bool overlaps(const Extent& o) const {
    if (!p || !o.p || rows <= 0 || o.rows <= 0) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
    return a < b + 4 * o.n && b < a + 4 * n;
  }
};

// A page table and the counts of its pages.
mxq_status check_table(const char* name, const void* table, int64_t ld, int64_t rows,
                       int64_t max_pages) {
  if (rows > 0 && max_pages > 0 && !table)
    return fail(MXQ_ERR_INVALID_ARG, std::string(name) + " must be non-NULL");
  if (!aligned(table, 4))
    return fail(MXQ_ERR_INVALID_ARG, std::string(name) + " must be 4-byte aligned");
  if (ld < max_pages)
    return fail(MXQ_ERR_INVALID_ARG, std::string(name) + ": row stride below max_pages");
  return MXQ_OK;
}

mxq_status check_pages(int64_t B, int64_t max_pages, int64_t pages, int32_t page_size,
                       const int32_t* refs) {
  if (B < 0 || max_pages < 0) return fail(MXQ_ERR_INVALID_ARG, "need B >= 0 and max_pages >= 0");
  if (pages <= 0 || page_size <= 0 || pages > 0x7fffffff)
    return fail(MXQ_ERR_INVALID_ARG, "need 0 < pages < 2^31 and page_size > 0");
  if (B > 0x3fffffff) return fail(MXQ_ERR_UNSUPPORTED, "more than 2^30 rows");
  if (max_pages > 0x7fffffff / 2 / page_size)
    return fail(MXQ_ERR_UNSUPPORTED, "sequences of more than 2^30 keys");
  if (!refs) return fail(MXQ_ERR_INVALID_ARG, "page_refs must be non-NULL");
  if (!aligned(refs, 16))
    return fail(MXQ_ERR_UNSUPPORTED, "page_refs needs a 16-byte aligned base");
  return MXQ_OK;
}

mxq_status fill_move(MoveParams* p, void* k_cache, void* v_cache, int32_t dtype, int64_t pages,
                     int32_t page_size, int32_t Hkv, int32_t D, int64_t sck_p, int64_t sck_t,
                     int64_t sck_h, int64_t scv_p, int64_t scv_t, int64_t scv_h) {
  if (Hkv <= 0 || D <= 0) return fail(MXQ_ERR_INVALID_ARG, "need Hkv > 0 and D > 0");
  if (D % 16 != 0 || D > 512)
    return fail(MXQ_ERR_UNSUPPORTED, "the head dimension must be a multiple of 16 up to 512");
  if (Hkv > 65535) return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 heads");
  if (pages <= 0 || page_size <= 0 || pages > 0x7fffffff)
    return fail(MXQ_ERR_INVALID_ARG, "need 0 < pages < 2^31 and page_size > 0");
  MXQ_TRY(check_cache("k_cache", k_cache, dtype, pages, page_size, Hkv, D, sck_p, sck_t, sck_h,
                      false, 16));
  MXQ_TRY(check_cache("v_cache", v_cache, dtype, pages, page_size, Hkv, D, scv_p, scv_t, scv_h,
                      false, 16));
  p->k_cache = k_cache, p->v_cache = v_cache;
  p->es = dtype == MXQ_E4M3 ? 1 : 2;
  p->per_head = D * p->es / 16, p->cols = Hkv * p->per_head;
  p->pages = pages, p->page_size = page_size;
  p->ck_p = sck_p, p->ck_t = sck_t, p->ck_h = sck_h;
  p->cv_p = scv_p, p->cv_t = scv_t, p->cv_h = scv_h;
  return MXQ_OK;
}

}  // namespace

extern "C" mxq_status mxq_cache_pages_workspace_size(int64_t rows, int64_t pages, size_t* bytes) {
  if (!bytes || rows < 0 || pages <= 0 || rows > 0x3fffffff || pages > 0x7fffffff)
    return fail(MXQ_ERR_INVALID_ARG, "bad sizes or NULL result pointer");
  *bytes = pages_workspace_bytes(rows, pages);
  return MXQ_OK;
}

extern "C" mxq_status mxq_cache_resize(int32_t* page_table, int64_t ld_table, int64_t B,
                                       int64_t max_pages, const int32_t* seq_lens,
                                       const int32_t* new_lens, int32_t* page_refs, int64_t pages,
                                       int32_t page_size, int32_t window, int32_t first,
                                       void* workspace, size_t ws_bytes, mxq_stream_t stream) {
  MXQ_TRY(check_pages(B, max_pages, pages, page_size, page_refs));
  if (window < 0 || first < 0)
    return fail(MXQ_ERR_INVALID_ARG, "window and first must be >= 0 (0: none)");
  if (B == 0) return MXQ_OK;
  MXQ_TRY(check_table("page_table", page_table, ld_table, B, max_pages));
  if (!seq_lens || !new_lens)
    return fail(MXQ_ERR_INVALID_ARG, "seq_lens and new_lens must be non-NULL");
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  MXQ_TRY(check_workspace(workspace, ws_bytes, pages_workspace_bytes(B, pages),
                          "mxq_cache_pages_workspace_size"));
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  PagesParams p = {};
  p.table = page_table, p.ld = ld_table, p.B = B, p.max_pages = max_pages;
  p.lens = seq_lens, p.new_lens = new_lens, p.refs = page_refs, p.pages = pages;
  // (the kernel counts pages from the first keys' end on in 32 bits; no row has more than 2^30 keys)
  p.page_size = page_size, p.window = std::min(window, 1 << 30);
  p.first = first_keys(window, first);
  p.workspace = workspace, p.status = d.status;
  const cudaError_t e = launch_resize_pages(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "cache resize launch");
}

extern "C" mxq_status mxq_cache_fork(const int32_t* page_table, int64_t ld_table, int64_t B,
                                     int64_t max_pages, const int32_t* seq_lens,
                                     int32_t* page_refs, int64_t pages, int32_t page_size,
                                     const int32_t* parents, int64_t n, int32_t* new_table,
                                     int64_t ld_new, int32_t* new_lens, int32_t* copies,
                                     void* workspace, size_t ws_bytes, mxq_stream_t stream) {
  MXQ_TRY(check_pages(B, max_pages, pages, page_size, page_refs));
  if (n < 0) return fail(MXQ_ERR_INVALID_ARG, "need n >= 0");
  if (n > 0x3fffffff) return fail(MXQ_ERR_UNSUPPORTED, "more than 2^30 rows");
  if (B == 0 && n == 0) return MXQ_OK;
  MXQ_TRY(check_table("page_table", page_table, ld_table, B, max_pages));
  MXQ_TRY(check_table("new_table", new_table, ld_new, n, max_pages));
  if ((B > 0 && !seq_lens) || (n > 0 && (!parents || !new_lens || !copies)))
    return fail(MXQ_ERR_INVALID_ARG, "seq_lens, parents, new_lens and copies must be non-NULL");
  if (!aligned(seq_lens, 4) || !aligned(parents, 4) || !aligned(new_lens, 4) ||
      !aligned(copies, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  // (what the call reads again after it has begun to write)
  const Extent in[] = {{page_table, (B - 1) * ld_table + max_pages, B},
                       {seq_lens, B, B},
                       {parents, n, n},
                       {page_refs, pages, pages}};
  const Extent results[] = {{new_table, (n - 1) * ld_new + max_pages, n}, {new_lens, n, n},
                            {copies, 3 * n, n}};
  for (const Extent& x : in)
    for (const Extent& y : results)
      if (x.overlaps(y))
        return fail(MXQ_ERR_INVALID_ARG, "new_table, new_lens and copies must not overlap what "
                                         "the call reads");
  MXQ_TRY(check_workspace(workspace, ws_bytes, pages_workspace_bytes(std::max(B, n), pages),
                          "mxq_cache_pages_workspace_size"));
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  PagesParams p = {};
  p.table = const_cast<int32_t*>(page_table), p.ld = ld_table, p.B = B, p.max_pages = max_pages;
  p.lens = seq_lens, p.refs = page_refs, p.pages = pages, p.page_size = page_size;
  p.parents = parents, p.n = n, p.new_table = new_table, p.ld_new = ld_new;
  p.new_lens_out = new_lens, p.copies = copies;
  p.workspace = workspace, p.status = d.status;
  const cudaError_t e = launch_fork_pages(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "cache fork launch");
}

extern "C" mxq_status mxq_cache_copy_pages(void* k_cache, void* v_cache, int32_t cache_dtype,
                                           int64_t pages, int32_t page_size, int32_t Hkv,
                                           int32_t D, int64_t sck_p, int64_t sck_t, int64_t sck_h,
                                           int64_t scv_p, int64_t scv_t, int64_t scv_h,
                                           const int32_t* copies, int64_t n,
                                           mxq_stream_t stream) {
  if (n < 0) return fail(MXQ_ERR_INVALID_ARG, "need n >= 0");
  MoveParams p = {};
  MXQ_TRY(fill_move(&p, k_cache, v_cache, cache_dtype, pages, page_size, Hkv, D, sck_p, sck_t,
                    sck_h, scv_p, scv_t, scv_h));
  if (n == 0) return MXQ_OK;
  if (n > 0x3fffffff) return fail(MXQ_ERR_UNSUPPORTED, "more than 2^30 copies");
  if (!copies) return fail(MXQ_ERR_INVALID_ARG, "copies must be non-NULL");
  if (!aligned(copies, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  p.copies = copies, p.n = n, p.status = d.status;
  const cudaError_t e =
      launch_copy_pages(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "cache copy launch");
}

extern "C" mxq_status mxq_cache_compact(void* k_cache, void* v_cache, int32_t cache_dtype,
                                        int64_t pages, int32_t page_size, int32_t Hkv, int32_t D,
                                        int64_t sck_p, int64_t sck_t, int64_t sck_h, int64_t scv_p,
                                        int64_t scv_t, int64_t scv_h, const int32_t* page_table,
                                        int64_t ld_table, int64_t B, int64_t max_pages,
                                        const int32_t* starts, const int32_t* kept,
                                        int64_t ld_kept, int64_t most, const int32_t* counts,
                                        mxq_stream_t stream) {
  if (B < 0 || max_pages < 0 || most < 0)
    return fail(MXQ_ERR_INVALID_ARG, "need B, max_pages and the kept rows >= 0");
  MoveParams p = {};
  MXQ_TRY(fill_move(&p, k_cache, v_cache, cache_dtype, pages, page_size, Hkv, D, sck_p, sck_t,
                    sck_h, scv_p, scv_t, scv_h));
  if (B == 0 || most == 0) return MXQ_OK;
  if (B > 65535) return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 sequences");
  if (most > 0x3fffffff || max_pages > 0x7fffffff / 2 / page_size)
    return fail(MXQ_ERR_UNSUPPORTED, "sequences of more than 2^30 keys");
  MXQ_TRY(check_table("page_table", page_table, ld_table, B, max_pages));
  if (!starts || !kept || !counts)
    return fail(MXQ_ERR_INVALID_ARG, "starts, kept and counts must be non-NULL");
  if (!aligned(starts, 4) || !aligned(kept, 4) || !aligned(counts, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  if (ld_kept < most) return fail(MXQ_ERR_INVALID_ARG, "kept: row stride below its width");
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  p.table = page_table, p.ld = ld_table, p.B = B, p.max_pages = max_pages;
  p.starts = starts, p.kept = kept, p.counts = counts, p.ld_kept = ld_kept, p.most = most;
  p.status = d.status;
  const cudaError_t e = launch_compact(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "cache compact launch");
}

extern "C" mxq_status mxq_paged_attention_tree_workspace_size(int64_t T, int64_t B, int32_t Hq,
                                                              int32_t Hkv, int32_t D,
                                                              size_t* bytes) {
  if (!bytes || B < 0 || T < 0)
    return fail(MXQ_ERR_INVALID_ARG, "bad sizes or NULL result pointer");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  *bytes = 0;
  if (B == 0 || T == 0) return MXQ_OK;
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  *bytes = tree_workspace_bytes(T, B, Hq, Hkv, D, d.num_sms);
  return MXQ_OK;
}

extern "C" mxq_status mxq_paged_attention_tree(
    const void* q, int64_t sq_t, int64_t sq_h, int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
    const void* k_cache, const void* v_cache, int32_t cache_dtype, int64_t pages, int32_t page_size,
    int64_t sck_p, int64_t sck_t, int64_t sck_h, int64_t scv_p, int64_t scv_t, int64_t scv_h,
    const int32_t* page_table, int64_t ld_table, int64_t max_pages, const int32_t* seq_lens,
    const int32_t* cu_seqlens_q, const int32_t* parents, int64_t B, float scale, int32_t window,
    int32_t first, const float* sinks, const float* k_scale, const float* v_scale, void* out,
    int64_t so_t, int64_t so_h, float* lse, void* workspace, size_t ws_bytes,
    mxq_stream_t stream) {
  if (B < 0 || T < 0 || max_pages < 0)
    return fail(MXQ_ERR_INVALID_ARG, "need B, T and max_pages >= 0");
  MXQ_TRY(check_heads(Hq, Hkv, D));
  MXQ_TRY(check_scale(scale, window, first));
  if (pages <= 0 || page_size <= 0 || pages > 0x7fffffff)
    return fail(MXQ_ERR_INVALID_ARG, "need 0 < pages < 2^31 and page_size > 0");
  if (B == 0 || T == 0) return MXQ_OK;
  if (B > 65535 || T > (1 << 30))
    return fail(MXQ_ERR_UNSUPPORTED, "more than 65535 sequences or 2^30 tokens");
  if (max_pages > 0x7fffffff / 2 / page_size)
    return fail(MXQ_ERR_UNSUPPORTED, "sequences of more than 2^30 keys");
  if (!seq_lens || !cu_seqlens_q || (max_pages > 0 && !page_table))
    return fail(MXQ_ERR_INVALID_ARG, "page_table, seq_lens and cu_seqlens_q must be non-NULL");
  if (ld_table < max_pages) return fail(MXQ_ERR_INVALID_ARG, "ld_table must be >= max_pages");
  if (!aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(parents, 4) || !aligned(sinks, 4) || !aligned(lse, 4) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4))
    return fail(MXQ_ERR_INVALID_ARG, "4-byte arrays must be 4-byte aligned");
  MXQ_TRY(check_rows("q", q, T, Hq, sq_t, sq_h, D, 2, 16));
  MXQ_TRY(check_rows("out", out, T, Hq, so_t, so_h, D, 2, 16));
  const bool scaled = k_scale || v_scale;
  MXQ_TRY(check_cache("k_cache", k_cache, cache_dtype, pages, page_size, Hkv, D, sck_p, sck_t,
                      sck_h, scaled, 16));
  MXQ_TRY(check_cache("v_cache", v_cache, cache_dtype, pages, page_size, Hkv, D, scv_p, scv_t,
                      scv_h, scaled, 16));
  // (the kernel counts them in 16 bytes, in 32 bits)
  const int64_t far = int64_t(1) << 35;
  if ((pages > 1 && (sck_p >= far || scv_p >= far)) ||
      (page_size > 1 && (sck_t >= far || scv_t >= far)))
    return fail(MXQ_ERR_UNSUPPORTED, "a page or token stride of 2^35 elements or more");
  DeviceInfo d;
  std::string err;
  if (!device_info(&d, &err)) return fail(MXQ_ERR_UNSUPPORTED, err);
  MXQ_TRY(check_workspace(workspace, ws_bytes, tree_workspace_bytes(T, B, Hq, Hkv, D, d.num_sms),
                          "mxq_paged_attention_tree_workspace_size"));
  TreeParams p = {};
  p.q = q, p.q_t = sq_t, p.q_h = sq_h, p.T = T;
  p.B = static_cast<int>(B), p.Hq = Hq, p.Hkv = Hkv, p.D = D;
  p.k_cache = k_cache, p.v_cache = v_cache, p.fp8 = cache_dtype == MXQ_E4M3;
  p.pages = pages, p.page_size = page_size;
  p.ck_p = sck_p, p.ck_t = sck_t, p.ck_h = sck_h, p.cv_p = scv_p, p.cv_t = scv_t, p.cv_h = scv_h;
  p.page_table = page_table, p.ld_table = ld_table, p.max_pages = max_pages;
  p.seq_lens = seq_lens, p.cu_q = cu_seqlens_q, p.parents = parents;
  p.scale = scale, p.window = std::min(window, 1 << 30), p.first = first_keys(window, first);
  p.sinks = sinks, p.k_scale = k_scale, p.v_scale = v_scale;
  p.out = out, p.o_t = so_t, p.o_h = so_h, p.lse = lse, p.workspace = workspace;
  p.status = d.status;
  const cudaError_t e = launch_tree(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MXQ_OK : cuda_fail(e, "tree attention launch");
}
