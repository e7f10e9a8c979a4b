// attn.h — parameters of the paged-cache and attention kernels (checked and
// filled by attn_api.cu) and their launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <string>

namespace mxq {

// Strides are in elements; the innermost (head dimension) stride is 1.
struct RopeAppendParams {
  const void *q, *k, *v;   // bf16; q may be null
  int64_t q_t, q_h, k_t, k_h, v_t, v_h;
  void* q_out;
  int64_t o_t, o_h;
  int64_t T;
  int Hq, Hkv, D, rot;
  bool interleaved, fp8;
  const float* cos_sin;    // [max_pos, rot]: cosines, then sines
  int64_t max_pos;
  const int32_t* positions;
  const int64_t* slots;
  void *k_cache, *v_cache;
  int64_t slots_total;     // pages * page_size
  int page_size;
  int64_t ck_p, ck_t, ck_h, cv_p, cv_t, cv_h;
  const float *k_scale, *v_scale;   // fp32 [Hkv] or null (1)
  int* status;
};

struct DecodeParams {
  const void* q;
  int64_t q_b, q_h;
  int B, Hq, Hkv, D;
  const void *k_cache, *v_cache;
  bool fp8;
  int64_t pages;
  int page_size;
  int64_t ck_p, ck_t, ck_h, cv_p, cv_t, cv_h;
  const int32_t* page_table;
  int64_t ld_table;
  int64_t max_pages;       // columns of page_table
  const int32_t* seq_lens;
  float scale;
  int window;              // 0: none
  const float *sinks, *k_scale, *v_scale;
  void* out;
  int64_t o_b, o_h;
  float* lse;              // [B, Hq] or null
  void* workspace;
  int* status;
};

struct PromptParams {
  const void *q, *k, *v;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h;
  const int32_t *cu_q, *cu_k;
  int B;
  int64_t Tq, Tk;
  int Hq, Hkv, D;
  float scale;
  bool causal;
  int window;
  const float* sinks;
  void* out;
  int64_t o_t, o_h;
  float* lse;              // [Tq, Hq] or null
  void* workspace;
  int* status;
};

cudaError_t launch_rope_append(const RopeAppendParams& p, int num_sms, cudaStream_t stream);
size_t decode_workspace_bytes(int64_t B, int Hq, int Hkv, int D, int num_sms);
cudaError_t launch_decode(const DecodeParams& p, int num_sms, cudaStream_t stream);
size_t prompt_workspace_bytes(int64_t Tq, int64_t B, int Hq, int Hkv, int D, int num_sms);
// err: set where the tensor maps cannot be made
cudaError_t launch_prompt(const PromptParams& p, int num_sms, cudaStream_t stream,
                          std::string* err);

}  // namespace mxq
