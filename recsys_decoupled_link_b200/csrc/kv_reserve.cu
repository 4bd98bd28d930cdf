// Block tables and slot maps of the paged history cache, built on the GPU from
// the requests' lengths, and the release of blocks.
#include "lime_kv.cuh"

namespace lime {

namespace {

constexpr int kScanThreads = 1024;


// Exclusive sum of one value per thread over the block; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t part[kScanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t p = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[kScanThreads / 32 - 1];
  const int64_t before = warp ? part[warp - 1] : 0;
  __syncthreads();
  return before + x - v;
}

__device__ __forceinline__ int stack_height(const int32_t* n_free, int64_t cap, unsigned* status) {
  const int n = *n_free;
  if (n < 0 || n > cap) {
    raise_flag(status, LIME_FLAG_BAD_BLOCK);
    return n < 0 ? 0 : (int)cap;
  }
  return n;
}

// One block of threads walks the requests once: thread t owns `per`
// consecutive ones.  first[u] becomes the rank of request u's first new block
// on the stack, or -1 where the request is refused.
__global__ void __launch_bounds__(kScanThreads)
    k_reserve_scan(int64_t B, int64_t total, int bs, int max_blocks, const int32_t* lens,
                   const int64_t* off, int64_t cap, const int32_t* n_free, int32_t* lens_out,
                   int32_t* n_free_out, int32_t* first, unsigned* status) {
  const int64_t most = (int64_t)max_blocks * bs;
  const int64_t per = ceil_div(B, kScanThreads);
  const int64_t u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : B;
  const int height = stack_height(n_free, cap, status);
  int64_t sum = 0;
  for (int64_t u = u0; u < u1; ++u) {
    int64_t a, b;
    user_range(off, u, B, total, &a, &b, status);
    const int n = kv_len(lens, u, most, status);
    const int64_t after = ceil_div(n + (b - a), bs);
    if (after <= max_blocks) sum += after - ceil_div(n, bs);
  }
  int64_t all;
  int64_t rank = block_scan(sum, &all);
  __shared__ int taken;
  if (threadIdx.x == 0) taken = 0;
  __syncthreads();
  for (int64_t u = u0; u < u1; ++u) {
    int64_t a, b;
    user_range(off, u, B, total, &a, &b, status);
    const int n = kv_len(lens, u, most, status);
    const int64_t after = ceil_div(n + (b - a), bs);
    const int64_t need = after <= max_blocks ? after - ceil_div(n, bs) : 0;
    const bool ok = after <= max_blocks && (need == 0 || rank + need <= height);
    first[u] = ok ? (int32_t)(rank < height ? rank : height) : -1;
    lens_out[u] = ok ? n + (int)(b - a) : n;
    rank += need;
    if (!ok) raise_flag(status, LIME_FLAG_NO_BLOCKS);
    if (ok && need > 0) atomicMax(&taken, (int)rank);
  }
  __syncthreads();
  if (threadIdx.x == 0) *n_free_out = height - taken;
}

// One thread per new row: its slot, and the table entry of a block it starts.
__global__ void k_reserve_fill(int64_t B, int64_t total, int bs, int max_blocks, int64_t n_blocks,
                               const int32_t* lens, const int64_t* off, int32_t* table,
                               const int32_t* free_blocks, int64_t cap, const int32_t* n_free,
                               const int32_t* first, int64_t* slots, unsigned* status) {
  const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= total) return;
  const int64_t u = owner_of(off, B, t);
  const int64_t n = kv_len(lens, u, (int64_t)max_blocks * bs, status);
  const int64_t pos = n + (t - off[u]), col = pos / bs;
  int64_t slot = -1;
  if (first[u] >= 0 && pos >= n && col < max_blocks) {
    const int64_t held = ceil_div(n, bs);
    int64_t block;
    if (col < held) {
      block = table[u * max_blocks + col];
    } else {
      const int64_t at = stack_height(n_free, cap, status) - 1 - (first[u] + col - held);
      block = at >= 0 ? free_blocks[at] : -1;
      if (pos % bs == 0) table[u * max_blocks + col] = (int32_t)block;
    }
    if (block >= 0 && block < n_blocks)
      slot = block * bs + pos % bs;
    else
      raise_flag(status, LIME_FLAG_BAD_BLOCK);
  }
  slots[t] = slot;
}

__device__ __forceinline__ int kept_rows(const int32_t* keep, int64_t u, int n) {
  const int k = keep ? keep[u] : 0;
  return k < 0 ? 0 : (k < n ? k : n);
}

__global__ void __launch_bounds__(kScanThreads)
    k_release_scan(int64_t B, int bs, int max_blocks, const int32_t* lens, const int32_t* keep,
                   int64_t cap, const int32_t* n_free, int32_t* lens_out, int32_t* n_free_out,
                   int64_t* first, unsigned* status) {
  const int64_t most = (int64_t)max_blocks * bs;
  const int64_t per = ceil_div(B, kScanThreads);
  const int64_t u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : B;
  const int height = stack_height(n_free, cap, status);
  int64_t sum = 0;
  for (int64_t u = u0; u < u1; ++u) {
    const int n = kv_len(lens, u, most, status);
    sum += ceil_div(n, bs) - ceil_div(kept_rows(keep, u, n), bs);
  }
  int64_t all;
  int64_t at = height + block_scan(sum, &all);
  for (int64_t u = u0; u < u1; ++u) {
    const int n = kv_len(lens, u, most, status);
    const int k = kept_rows(keep, u, n);
    first[u] = at;
    at += ceil_div(n, bs) - ceil_div(k, bs);
    lens_out[u] = k;
  }
  if (threadIdx.x == 0) {
    if (height + all > cap) raise_flag(status, LIME_FLAG_BAD_BLOCK);
    *n_free_out = (int32_t)(height + all < cap ? height + all : cap);
  }
}

// A warp per request pushes its released blocks.
__global__ void k_release_fill(int64_t B, int bs, int max_blocks, const int32_t* lens,
                               const int32_t* keep, int32_t* table, int32_t* free_blocks,
                               int64_t cap, const int64_t* first, unsigned* status) {
  const int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (u >= B) return;
  const int n = kv_len(lens, u, (int64_t)max_blocks * bs, status);
  const int64_t c0 = ceil_div(kept_rows(keep, u, n), bs), c1 = ceil_div(n, bs);
  for (int64_t c = c0 + (threadIdx.x & 31); c < c1; c += 32) {
    const int64_t at = first[u] + (c - c0);
    if (at < cap) free_blocks[at] = table[u * max_blocks + c];
    table[u * max_blocks + c] = -1;
  }
}

}  // namespace

int kv_reserve(const lime_kv_dims& D, int64_t B, const int32_t* lens, const int64_t* off,
               int64_t total, int32_t* table, const int32_t* free_blocks, int64_t free_cap,
               const int32_t* n_free, int32_t* lens_out, int32_t* n_free_out, int64_t* slots,
               void* ws, unsigned* status, cudaStream_t st) {
  int32_t* first = (int32_t*)ws;
  k_reserve_scan<<<1, kScanThreads, 0, st>>>(B, total, D.block, D.max_blocks, lens, off, free_cap,
                                             n_free, lens_out, n_free_out, first, status);
  note_launches(1);
  if (total > 0) {
    k_reserve_fill<<<(unsigned)ceil_div(total, 256), 256, 0, st>>>(
        B, total, D.block, D.max_blocks, D.n_blocks, lens, off, table, free_blocks, free_cap,
        n_free, first, slots, status);
    note_launches(1);
  }
  return LIME_OK;
}

int kv_release(const lime_kv_dims& D, int64_t B, const int32_t* lens, const int32_t* keep,
               int32_t* table, int32_t* free_blocks, int64_t free_cap, const int32_t* n_free,
               int32_t* lens_out, int32_t* n_free_out, void* ws, unsigned* status,
               cudaStream_t st) {
  int64_t* first = (int64_t*)ws;
  k_release_scan<<<1, kScanThreads, 0, st>>>(B, D.block, D.max_blocks, lens, keep, free_cap,
                                             n_free, lens_out, n_free_out, first, status);
  note_launches(1);
  if (B > 0) {
    k_release_fill<<<(unsigned)ceil_div(B, 8), 256, 0, st>>>(B, D.block, D.max_blocks, lens, keep,
                                                             table, free_blocks, free_cap, first,
                                                             status);
    note_launches(1);
  }
  return LIME_OK;
}

}  // namespace lime
