// C ABI of the paged 8-bit history cache (include/lime_kv.h): argument checks
// and dispatch.  Every numeric step runs in kv_reserve.cu, kv_append.cu and
// kv_attn.cu.
#include <math.h>
#include <stdio.h>

#include "lime_kv.cuh"

using namespace lime;

namespace {

constexpr size_t kStatusBytes = 256;  // status word + padding at the workspace head

int check_dims(const lime_kv_dims* D) {
  if (!D || (D->dtype != LIME_F32 && D->dtype != LIME_BF16)) return LIME_ERR_ARG;
  if (D->Hq <= 0 || D->Hkv <= 0 || D->max_blocks <= 0 || D->n_blocks <= 0) return LIME_ERR_ARG;
  if (D->Hq % D->Hkv != 0 || D->Hq > 1024) return LIME_ERR_SHAPE;
  if (D->dh != 16 && D->dh != 32 && D->dh != 64 && D->dh != 128) return LIME_ERR_SHAPE;
  if (D->block != 16 && D->block != 32 && D->block != 64 && D->block != 128) return LIME_ERR_SHAPE;
  if (D->n_blocks > INT32_MAX / D->Hkv || D->max_blocks > (1 << 30) / D->block)
    return LIME_ERR_SHAPE;
  return LIME_OK;
}

size_t esize(const lime_kv_dims* D) { return D->dtype == LIME_BF16 ? 2 : 4; }
size_t cache_bytes(const lime_kv_dims* D) {
  return (size_t)D->n_blocks * D->Hkv * D->block * D->dh;
}
size_t scale_bytes(const lime_kv_dims* D) { return (size_t)D->n_blocks * D->Hkv * 8; }

// Bytes from the first element of row 0 to the last of row n - 1.
size_t pitched(int64_t n, int64_t ld, int64_t width, size_t es) {
  return n > 0 ? ((size_t)(n - 1) * ld + width) * es : 0;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Span {
  const void* p;
  size_t n;
};

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}

// Whether any of the nw written spans overlaps another span of the call (the
// written ones come first).
bool clash(const Span* s, int nw, int n) {
  for (int i = 0; i < nw; ++i)
    for (int j = i + 1; j < n; ++j)
      if (overlap(s[i], s[j])) return true;
  return false;
}

int check_ws(void* ws, size_t bytes, const lime_kv_dims* D, int64_t B, int64_t total_q) {
  if (!ws || !aligned(ws, 256)) return LIME_ERR_ARG;
  return bytes < lime_kv_workspace_bytes(D, B, total_q) ? LIME_ERR_ARG : LIME_OK;
}

unsigned* status_of(void* ws) { return (unsigned*)ws; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
// status word, tickets (zero between calls), scratch
int* tickets_of(void* ws) { return (int*)((char*)ws + kStatusBytes); }
size_t head_bytes() { return kStatusBytes + round256(kv_ticket_bytes()); }
void* scratch_of(void* ws) { return (char*)ws + head_bytes(); }

int launch_status(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return LIME_OK;
  fprintf(stderr, "liblime: %s: %s\n", what, cudaGetErrorString(e));
  return LIME_ERR_CUDA;
}

bool bad_count(int64_t n) { return n < 0 || n > INT32_MAX; }

}  // namespace

extern "C" {

size_t lime_kv_workspace_bytes(const lime_kv_dims* dims, int64_t B, int64_t total_q) {
  if (check_dims(dims) != LIME_OK || bad_count(B) || bad_count(total_q)) return 0;
  const size_t ranks = (size_t)B * 8, attn = kv_attention_ws_bytes(*dims, B, total_q);
  return head_bytes() + round256(attn > ranks ? attn : ranks);
}

int lime_kv_workspace_init(void* workspace, size_t bytes, cudaStream_t stream) {
  if (!workspace || bytes < head_bytes() || !aligned(workspace, 256)) return LIME_ERR_ARG;
  return cudaMemsetAsync(workspace, 0, head_bytes(), stream) == cudaSuccess ? LIME_OK
                                                                            : LIME_ERR_CUDA;
}

int lime_kv_reserve(const lime_kv_dims* dims, int64_t B, const int32_t* lens,
                    const int64_t* new_offsets, int64_t total_new, int32_t* block_table,
                    const int32_t* free_blocks, int64_t free_cap, const int32_t* n_free,
                    int32_t* lens_out, int32_t* n_free_out, int64_t* slot_map, void* workspace,
                    size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_dims(dims);
  if (rc) return rc;
  if (bad_count(B) || bad_count(total_new) || bad_count(free_cap)) return LIME_ERR_ARG;
  if ((rc = check_ws(workspace, workspace_bytes, dims, B, 0))) return rc;
  if (B == 0 && total_new > 0) return LIME_ERR_ARG;
  if (!n_free || !n_free_out || (free_cap > 0 && !free_blocks)) return LIME_ERR_ARG;
  if (B > 0 && (!lens || !new_offsets || !block_table || !lens_out)) return LIME_ERR_ARG;
  if (total_new > 0 && !slot_map) return LIME_ERR_ARG;
  if (!aligned(lens, 4) || !aligned(new_offsets, 8) || !aligned(block_table, 4) ||
      !aligned(free_blocks, 4) || !aligned(n_free, 4) || !aligned(lens_out, 4) ||
      !aligned(n_free_out, 4) || !aligned(slot_map, 8))
    return LIME_ERR_ARG;
  const Span s[] = {{block_table, (size_t)B * dims->max_blocks * 4},
                    {lens_out, (size_t)B * 4},
                    {n_free_out, 4},
                    {slot_map, (size_t)total_new * 8},
                    {workspace, workspace_bytes},
                    {lens, (size_t)B * 4},
                    {new_offsets, (size_t)(B + 1) * 8},
                    {free_blocks, (size_t)free_cap * 4},
                    {n_free, 4}};
  if (clash(s, 5, 9)) return LIME_ERR_ALIAS;
  if ((rc = kv_reserve(*dims, B, lens, new_offsets, total_new, block_table, free_blocks, free_cap,
                       n_free, lens_out, n_free_out, slot_map, scratch_of(workspace),
                       status_of(workspace), stream)))
    return rc;
  return launch_status("lime_kv_reserve");
}

int lime_kv_release(const lime_kv_dims* dims, int64_t B, const int32_t* lens,
                    const int32_t* keep, int32_t* block_table, int32_t* free_blocks,
                    int64_t free_cap, const int32_t* n_free, int32_t* lens_out,
                    int32_t* n_free_out, void* workspace, size_t workspace_bytes,
                    cudaStream_t stream) {
  int rc = check_dims(dims);
  if (rc) return rc;
  if (bad_count(B) || bad_count(free_cap)) return LIME_ERR_ARG;
  if ((rc = check_ws(workspace, workspace_bytes, dims, B, 0))) return rc;
  if (!n_free || !n_free_out || (free_cap > 0 && !free_blocks)) return LIME_ERR_ARG;
  if (B > 0 && (!lens || !block_table || !lens_out)) return LIME_ERR_ARG;
  if (!aligned(lens, 4) || !aligned(keep, 4) || !aligned(block_table, 4) ||
      !aligned(free_blocks, 4) || !aligned(n_free, 4) || !aligned(lens_out, 4) ||
      !aligned(n_free_out, 4))
    return LIME_ERR_ARG;
  const Span s[] = {{block_table, (size_t)B * dims->max_blocks * 4},
                    {free_blocks, (size_t)free_cap * 4},
                    {lens_out, (size_t)B * 4},
                    {n_free_out, 4},
                    {workspace, workspace_bytes},
                    {lens, (size_t)B * 4},
                    {keep, (size_t)B * 4},
                    {n_free, 4}};
  if (clash(s, 5, 8)) return LIME_ERR_ALIAS;
  if ((rc = kv_release(*dims, B, lens, keep, block_table, free_blocks, free_cap, n_free, lens_out,
                       n_free_out, scratch_of(workspace), status_of(workspace), stream)))
    return rc;
  return launch_status("lime_kv_release");
}

int lime_kv_append(const lime_kv_dims* dims, const void* K, int64_t ldk, const void* V,
                   int64_t ldv, int64_t total_new, const int64_t* slot_map, int8_t* k_cache,
                   int8_t* v_cache, float* scale, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream) {
  int rc = check_dims(dims);
  if (rc) return rc;
  if (bad_count(total_new)) return LIME_ERR_ARG;
  if ((rc = check_ws(workspace, workspace_bytes, dims, 0, 0))) return rc;
  if (total_new == 0) return LIME_OK;
  if (!K || !V || !slot_map || !k_cache || !v_cache || !scale) return LIME_ERR_ARG;
  const size_t es = esize(dims);
  const int64_t width = (int64_t)dims->Hkv * dims->dh;
  if (ldk < width || ldv < width || ldk > INT32_MAX || ldv > INT32_MAX || ldk * es % 16 != 0 ||
      ldv * es % 16 != 0)
    return LIME_ERR_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slot_map, 8) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(scale, 16))
    return LIME_ERR_ARG;
  const Span s[] = {{k_cache, cache_bytes(dims)},
                    {v_cache, cache_bytes(dims)},
                    {scale, scale_bytes(dims)},
                    {workspace, workspace_bytes},
                    {K, pitched(total_new, ldk, width, es)},
                    {V, pitched(total_new, ldv, width, es)},
                    {slot_map, (size_t)total_new * 8}};
  if (clash(s, 4, 7)) return LIME_ERR_ALIAS;
  if ((rc = kv_append(*dims, K, ldk, V, ldv, total_new, slot_map, k_cache, v_cache, scale,
                      status_of(workspace), stream)))
    return rc;
  return launch_status("lime_kv_append");
}

int lime_kv_attention(const lime_kv_dims* dims, int64_t B, const void* Q, int64_t ldq,
                      const int64_t* q_offsets, int64_t total_q, const int32_t* block_table,
                      const int32_t* lens, const int8_t* k_cache, const int8_t* v_cache,
                      const float* scale, float sm_scale, int32_t causal, void* O, float* lse,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  int rc = check_dims(dims);
  if (rc) return rc;
  if (bad_count(B) || bad_count(total_q) || (causal != 0 && causal != 1) || !(fabsf(sm_scale) <= 0x1p100f))
    return LIME_ERR_ARG;
  // rows of all heads are counted in 32 bits
  if (total_q * dims->Hq > INT32_MAX) return LIME_ERR_ARG;
  if ((rc = check_ws(workspace, workspace_bytes, dims, B, total_q))) return rc;
  if (B == 0) return total_q == 0 ? LIME_OK : LIME_ERR_ARG;
  if (total_q == 0) return LIME_OK;
  if (!Q || !q_offsets || !block_table || !lens || !k_cache || !v_cache || !scale || !O)
    return LIME_ERR_ARG;
  const size_t es = esize(dims);
  const int64_t width = (int64_t)dims->Hq * dims->dh;
  if (ldq < width || ldq > INT32_MAX || ldq * es % 16 != 0) return LIME_ERR_ARG;
  if (!aligned(Q, 16) || !aligned(O, 16) || !aligned(lse, 4) || !aligned(q_offsets, 8) ||
      !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(scale, 16))
    return LIME_ERR_ARG;
  const Span s[] = {{O, (size_t)total_q * width * es},
                    {lse, (size_t)total_q * dims->Hq * 4},
                    {workspace, workspace_bytes},
                    {Q, pitched(total_q, ldq, width, es)},
                    {q_offsets, (size_t)(B + 1) * 8},
                    {block_table, (size_t)B * dims->max_blocks * 4},
                    {lens, (size_t)B * 4},
                    {k_cache, cache_bytes(dims)},
                    {v_cache, cache_bytes(dims)},
                    {scale, scale_bytes(dims)}};
  if (clash(s, 3, 10)) return LIME_ERR_ALIAS;
  if ((rc = kv_attention(*dims, B, Q, ldq, q_offsets, total_q, block_table, lens, k_cache, v_cache,
                         scale, sm_scale, causal != 0, O, lse, scratch_of(workspace),
                         tickets_of(workspace), status_of(workspace), stream)))
    return rc;
  return launch_status("lime_kv_attention");
}

}  // extern "C"
