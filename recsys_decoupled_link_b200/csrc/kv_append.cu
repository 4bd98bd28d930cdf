// Quantising append of the paged history cache: new key and value rows become
// int8 codes under one scale per (block, head).
#include "lime_kv.cuh"

namespace lime {

namespace {

__device__ __forceinline__ float finite_abs(float x, bool* odd) {
  const float a = fabsf(x);
  if (a <= 3.402823466e38f) return a;
  *odd = true;  // NaN or infinite
  return 0.0f;
}

// rint(x / s) in 64 bits: the quotient of two fp32 values lies on a half-way
// point only when it is one exactly, so this is the exact rounding.
__device__ __forceinline__ int8_t code_of(float x, float s) {
  if (x != x || s == 0.0f) return 0;
  const double r = rint((double)x / (double)s);
  return (int8_t)(r > 127.0 ? 127.0 : (r < -127.0 ? -127.0 : r));
}

// One warp per (new row, head); the row that begins a group does the group.
template <class T>
__global__ void k_append(int Hkv, int dh, int bs, int64_t n_slots, const T* K, int64_t ldk,
                         const T* V, int64_t ldv, int64_t total, const int64_t* slots, int8_t* kc,
                         int8_t* vc, float* scale, unsigned* status) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t t = w / Hkv;
  const int h = (int)(w % Hkv);
  if (t >= total) return;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= n_slots) {
    if (slot != -1) raise_flag(status, LIME_FLAG_BAD_BLOCK);
    return;
  }
  const int row = (int)(slot % bs);
  if (t > 0 && row != 0 && slots[t - 1] == slot - 1) return;
  int n = 1;
  while (row + n < bs && t + n < total && slots[t + n] == slot + n) ++n;
  const int64_t tile = (slot / bs) * Hkv + h;
  bool odd = false;
  for (int side = 0; side < 2; ++side) {
    const T* X = side ? V : K;
    const int64_t ld = side ? ldv : ldk;
    int8_t* codes = (side ? vc : kc) + tile * bs * dh;
    float a = 0.0f;
    for (int i = lane; i < n * dh; i += 32)
      a = fmaxf(a, finite_abs(to_f(X[(t + i / dh) * ld + h * dh + i % dh]), &odd));
    a = warp_max(a);
    float had = row ? scale[tile * 2 + side] : 0.0f;
    if (!(had >= 0.0f && had <= 3.402823466e38f)) had = 0.0f;
    const float s = fmaxf(had, __fdiv_rn(a, 127.0f));
    if (s > had)
      for (int i = lane; i < row * dh; i += 32)
        codes[i] = (int8_t)rint((double)codes[i] * (double)had / (double)s);
    for (int i = lane; i < n * dh; i += 32)
      codes[row * dh + i] = code_of(to_f(X[(t + i / dh) * ld + h * dh + i % dh]), s);
    if (lane == 0) scale[tile * 2 + side] = s;
  }
  if (odd) raise_flag(status, LIME_FLAG_NONFINITE);
}

}  // namespace

int kv_append(const lime_kv_dims& D, const void* K, int64_t ldk, const void* V, int64_t ldv,
              int64_t total, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
              unsigned* status, cudaStream_t st) {
  const unsigned grid = (unsigned)ceil_div(total * D.Hkv, 8);
  const int64_t n_slots = D.n_blocks * D.block;
  if (D.dtype == LIME_BF16)
    k_append<bf16><<<grid, 256, 0, st>>>(D.Hkv, D.dh, D.block, n_slots, (const bf16*)K, ldk,
                                         (const bf16*)V, ldv, total, slots, kc, vc, scale, status);
  else
    k_append<float><<<grid, 256, 0, st>>>(D.Hkv, D.dh, D.block, n_slots, (const float*)K, ldk,
                                          (const float*)V, ldv, total, slots, kc, vc, scale,
                                          status);
  note_launches(1);
  return LIME_OK;
}

}  // namespace lime
