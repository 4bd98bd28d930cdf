// Kernels of the paged 8-bit history cache (include/lime_kv.h): launchers
// called by kv_api.cu after the arguments are checked.
#pragma once
#include "lime_common.cuh"
#include "lime_kv.h"

namespace lime {

__host__ __device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A request's row count, clamped into its table's range (flagged when it was not).
__device__ __forceinline__ int kv_len(const int32_t* lens, int64_t u, int64_t most,
                                      unsigned* status) {
  const int n = lens[u];
  if (n < 0 || n > most) {
    raise_flag(status, LIME_FLAG_BAD_OFFSETS);
    return n < 0 ? 0 : (int)most;
  }
  return n;
}

// Scratch of an attention call, apart from its tickets: counters that are zero
// between calls and stand at a fixed place of the workspace.
size_t kv_attention_ws_bytes(const lime_kv_dims& D, int64_t B, int64_t total_q);
size_t kv_ticket_bytes();

int kv_reserve(const lime_kv_dims& D, int64_t B, const int32_t* lens, const int64_t* off,
               int64_t total, int32_t* table, const int32_t* free_blocks, int64_t free_cap,
               const int32_t* n_free, int32_t* lens_out, int32_t* n_free_out, int64_t* slots,
               void* ws, unsigned* status, cudaStream_t st);
int kv_release(const lime_kv_dims& D, int64_t B, const int32_t* lens, const int32_t* keep,
               int32_t* table, int32_t* free_blocks, int64_t free_cap, const int32_t* n_free,
               int32_t* lens_out, int32_t* n_free_out, void* ws, unsigned* status,
               cudaStream_t st);
int kv_append(const lime_kv_dims& D, const void* K, int64_t ldk, const void* V, int64_t ldv,
              int64_t total, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
              unsigned* status, cudaStream_t st);
int kv_attention(const lime_kv_dims& D, int64_t B, const void* Q, int64_t ldq, const int64_t* off,
                 int64_t total_q, const int32_t* table, const int32_t* lens, const int8_t* kc,
                 const int8_t* vc, const float* scale, float sm_scale, bool causal, void* O,
                 float* lse, void* ws, int* tickets, unsigned* status, cudaStream_t st);

}  // namespace lime
