// Attention over the paged 8-bit history cache.
#include <math.h>

#include "lime_kv.cuh"

namespace lime {

namespace {

// One warp per (query row, head): 32 keys at a time, a key per lane for the
// scores and a few dims per lane for the values, with the running maximum and
// sum of the softmax.
template <class T, int DH>
__global__ void k_attn_rows(lime_kv_dims D, int64_t B, const T* Q, int64_t ldq, const int64_t* off,
                            int64_t total_q, const int32_t* table, const int32_t* lens,
                            const int8_t* kc, const int8_t* vc, const float* scale, float sm_scale,
                            bool causal, T* O, float* lse, unsigned* status) {
  constexpr int PER = (DH + 31) / 32;
  __shared__ float qs[4][DH];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * 4 + warp;
  if (r >= total_q * D.Hq) return;
  const int64_t i = r / D.Hq;
  const int hq = (int)(r % D.Hq), h = hq / (D.Hq / D.Hkv);
  const int64_t u = owner_of(off, B, i);
  int64_t a, b;
  user_range(off, u, B, total_q, &a, &b, status);
  const int n = kv_len(lens, u, (int64_t)D.max_blocks * D.block, status);
  int64_t limit = causal ? n - (b - a) + (i - a) + 1 : n;
  if (limit > n) limit = n;
  for (int d = lane; d < DH; d += 32) qs[warp][d] = to_f(Q[i * ldq + (int64_t)hq * DH + d]);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[PER];
  for (int k = 0; k < PER; ++k) o[k] = 0.0f;
  for (int64_t j0 = 0; j0 < limit; j0 += 32) {
    const int64_t j = j0 + lane;
    float s = -INFINITY, vs = 0.0f;
    int64_t base = -1;
    if (j < limit) {
      const int64_t block = table[u * D.max_blocks + j / D.block];
      if (block >= 0 && block < D.n_blocks) {
        base = ((block * D.Hkv + h) * D.block + j % D.block) * DH;
        const float2 sc = reinterpret_cast<const float2*>(scale)[block * D.Hkv + h];
        float acc = 0.0f;
        for (int d = 0; d < DH; ++d) acc += qs[warp][d] * (float)kc[base + d];
        s = acc * sc.x * sm_scale;
        vs = sc.y;
      } else {
        raise_flag(status, LIME_FLAG_BAD_BLOCK);
      }
    }
    const float top = fmaxf(m, warp_max(s));
    const float ref = top == -INFINITY ? 0.0f : top;
    const float p = expf(s - ref), keep = expf(m - ref);
    m = top;
    l = l * keep + warp_sum(p);
    const float pv = p * vs;
    for (int k = 0; k < PER; ++k) o[k] *= keep;
    for (int t = 0; t < 32; ++t) {
      const float w = __shfl_sync(0xffffffffu, pv, t);
      const int64_t at = __shfl_sync(0xffffffffu, base, t);
      if (at < 0) continue;
      for (int k = 0; k < PER; ++k)
        if (lane + 32 * k < DH) o[k] += w * (float)vc[at + lane + 32 * k];
    }
  }
  for (int k = 0; k < PER; ++k)
    if (lane + 32 * k < DH) O[r * DH + lane + 32 * k] = from_f<T>(l > 0.0f || l != l ? o[k] / l : 0.0f);
  if (lse && lane == 0) lse[r] = m + logf(l);
}

template <class T>
void launch(const lime_kv_dims& D, int64_t B, const void* Q, int64_t ldq, const int64_t* off,
            int64_t total_q, const int32_t* table, const int32_t* lens, const int8_t* kc,
            const int8_t* vc, const float* scale, float sm_scale, bool causal, void* O, float* lse,
            unsigned* status, cudaStream_t st) {
  const unsigned grid = (unsigned)ceil_div(total_q * D.Hq, 4);
#define LAUNCH(DH)                                                                             \
  k_attn_rows<T, DH><<<grid, 128, 0, st>>>(D, B, (const T*)Q, ldq, off, total_q, table, lens, \
                                           kc, vc, scale, sm_scale, causal, (T*)O, lse, status)
  if (D.dh == 16) LAUNCH(16);
  else if (D.dh == 32) LAUNCH(32);
  else if (D.dh == 64) LAUNCH(64);
  else LAUNCH(128);
#undef LAUNCH
  note_launches(1);
}

}  // namespace

size_t kv_ws_bytes(const lime_kv_dims& D, int64_t B, int64_t total_q) {
  return (size_t)B * 8;  // ranks of the requests' blocks
}

int kv_attention(const lime_kv_dims& D, int64_t B, const void* Q, int64_t ldq, const int64_t* off,
                 int64_t total_q, const int32_t* table, const int32_t* lens, const int8_t* kc,
                 const int8_t* vc, const float* scale, float sm_scale, bool causal, void* O,
                 float* lse, void* ws, unsigned* status, cudaStream_t st) {
  if (D.dtype == LIME_BF16)
    launch<bf16>(D, B, Q, ldq, off, total_q, table, lens, kc, vc, scale, sm_scale, causal, O, lse,
                 status, st);
  else
    launch<float>(D, B, Q, ldq, off, total_q, table, lens, kc, vc, scale, sm_scale, causal, O, lse,
                  status, st);
  return LIME_OK;
}

}  // namespace lime
