// Block tables and slot maps of the paged history cache, built on the GPU from
// the requests' lengths, and the release of blocks.
#include "lime_fast.cuh"
#include "lime_kv.cuh"
#include "sm100.cuh"

namespace lime {

using namespace sm100;

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

// Blocks request u's new rows need, or -1 where they pass its table.
__device__ __forceinline__ int blocks_needed(int n, int64_t rows, int log_bs, int max_blocks) {
  const int64_t bs = 1 << log_bs;
  const int64_t after = (n + rows + bs - 1) >> log_bs;
  return after <= max_blocks ? (int)(after - ((n + bs - 1) >> log_bs)) : -1;
}

// Whether a request gets its blocks, given the rank of the first.
__device__ __forceinline__ bool served(int need, int64_t rank, int height) {
  return need == 0 || (need > 0 && rank + need <= height);
}

// The slot of row t of a request with n rows whose new rows are [a, b) of the
// packed ones, and the table entry of a block that it starts.  first: rank of
// the request's first new block, or -1 where it is refused.
__device__ __forceinline__ int64_t place(int64_t t, int64_t u, int64_t a, int64_t b, int n, int64_t first,
                                         int log_bs, int max_blocks, int64_t n_blocks,
                                         int32_t* table, const int32_t* free_blocks, int height,
                                         unsigned* status) {
  const int64_t bs = 1 << log_bs, pos = n + (t - a), col = pos >> log_bs;
  if (first < 0 || t < a || t >= b || col >= max_blocks) return -1;
  const int64_t held = (n + bs - 1) >> log_bs;
  int64_t block = -1;
  if (col < held) {
    block = table[u * max_blocks + col];
  } else {
    const int64_t at = height - 1 - (first + col - held);
    if (at >= 0 && at < height) block = free_blocks[at];
    if ((pos & (bs - 1)) == 0) table[u * max_blocks + col] = (int32_t)block;
  }
  if (block >= 0 && block < n_blocks) return (block << log_bs) + (pos & (bs - 1));
  raise_flag(status, LIME_FLAG_BAD_BLOCK);
  return -1;
}

// Up to kFusedRequests requests: one kernel.  Every thread block scans all of
// them (12 bytes each, from L2) and places its own kFusedRows rows, so nothing
// passes between blocks: 4.1 us for 256 requests with a row each, where two
// kernels took 6.9.
constexpr int kFusedRequests = 2048;
constexpr int kFusedRows = 2048;

__global__ void __launch_bounds__(kScanThreads)
    k_reserve_fused(int64_t B, int64_t total, int log_bs, int max_blocks, int64_t n_blocks,
                    const int32_t* lens, const int64_t* off, int32_t* table,
                    const int32_t* free_blocks, int64_t cap, const int32_t* n_free,
                    int32_t* lens_out, int32_t* n_free_out, int64_t* slots, unsigned* status) {
  __shared__ int32_t s_off[kFusedRequests], s_end[kFusedRequests], s_len[kFusedRequests],
      s_need[kFusedRequests], s_first[kFusedRequests];
  __shared__ int taken;
  if (threadIdx.x == 0) taken = 0;
  const int64_t most = (int64_t)max_blocks << log_bs;
  const int height = stack_height(n_free, cap, status);
  for (int u = threadIdx.x; u < B; u += kScanThreads) {
    int64_t a, b;
    user_range(off, u, B, total, &a, &b, status);
    const int n = kv_len(lens, u, most, status);
    s_off[u] = (int32_t)a;
    s_len[u] = n;
    s_need[u] = blocks_needed(n, b - a, log_bs, max_blocks);
    s_end[u] = (int32_t)b;
  }
  __syncthreads();
  const int per = (int)ceil_div(B, kScanThreads);
  const int u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : (int)B;
  int64_t sum = 0;
  for (int u = u0; u < u1; ++u) sum += s_need[u] > 0 ? s_need[u] : 0;
  int64_t all;
  int64_t rank = block_scan(sum, &all);
  for (int u = u0; u < u1; ++u) {
    const int need = s_need[u], rows = s_end[u] - s_off[u];
    const bool ok = served(need, rank, height);
    s_first[u] = ok ? (int32_t)(rank < height ? rank : height) : -1;
    if (need > 0) rank += need;
    if (blockIdx.x == 0) {
      lens_out[u] = s_len[u] + (ok ? rows : 0);
      if (!ok) raise_flag(status, LIME_FLAG_NO_BLOCKS);
      if (ok && need > 0) atomicMax(&taken, (int)rank);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_free_out = height - taken;
  const int64_t t0 = (int64_t)blockIdx.x * kFusedRows;
  for (int64_t t = t0 + threadIdx.x; t < t0 + kFusedRows && t < total; t += kScanThreads) {
    int lo = 0, hi = (int)B;                       // the largest u with off[u] <= t is in [lo, hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid] <= t) lo = mid; else hi = mid;
    }
    slots[t] = place(t, lo, s_off[lo], s_end[lo], s_len[lo], s_first[lo], log_bs, max_blocks, n_blocks, table,
                     free_blocks, height, status);
  }
}

// More requests: a scan and a placing kernel.  A block of threads owns
// kScanThreads requests and sums the needs of all before them itself.
// first[u] becomes the rank of request u's first new block on the stack, or -1
// where the request is refused.
__global__ void __launch_bounds__(kScanThreads)
    k_reserve_scan(int64_t B, int64_t total, int log_bs, int max_blocks, const int32_t* lens,
                   const int64_t* off, int64_t cap, const int32_t* n_free, int32_t* lens_out,
                   int32_t* n_free_out, int32_t* first, unsigned* status) {
  __shared__ int taken;
  pdl_launch();
  pdl_wait();
  const int64_t most = (int64_t)max_blocks << log_bs;
  const int height = stack_height(n_free, cap, status);
  const int64_t begin = (int64_t)blockIdx.x * kScanThreads, u = begin + threadIdx.x;
  int64_t sum = 0;
#pragma unroll 4
  for (int64_t v = threadIdx.x; v < begin; v += kScanThreads) {
    int64_t a, b;
    user_range(off, v, B, total, &a, &b, status);
    const int need = blocks_needed(kv_len(lens, v, most, status), b - a, log_bs, max_blocks);
    sum += need > 0 ? need : 0;
  }
  int64_t a = 0, b = 0, before, all;
  int n = 0, need = 0;
  if (u < B) {
    user_range(off, u, B, total, &a, &b, status);
    n = kv_len(lens, u, most, status);
    need = blocks_needed(n, b - a, log_bs, max_blocks);
  }
  block_scan(sum, &before);
  const int64_t rank = before + block_scan(need > 0 ? need : 0, &all);
  if (threadIdx.x == 0) taken = (int)(before < height ? before : height);
  __syncthreads();
  if (u < B) {
    const bool ok = served(need, rank, height);
    first[u] = ok ? (int32_t)(rank < height ? rank : height) : -1;
    lens_out[u] = n + (ok ? (int)(b - a) : 0);
    if (!ok) raise_flag(status, LIME_FLAG_NO_BLOCKS);
    if (ok && need > 0) atomicMax(&taken, (int)(rank + need));
  }
  __syncthreads();
  // the block in which the stack runs out, or the last one, knows what is taken
  const bool last = begin + kScanThreads >= B;
  if (threadIdx.x == 0 && before <= height && (last || before + all > height))
    *n_free_out = height - taken;
}

// One thread per new row: its slot, and the table entry of a block it starts.
__global__ void k_reserve_fill(int64_t B, int64_t total, int log_bs, int max_blocks,
                               int64_t n_blocks, const int32_t* lens, const int64_t* off,
                               int32_t* table, const int32_t* free_blocks, int64_t cap,
                               const int32_t* n_free, const int32_t* first, int64_t* slots,
                               unsigned* status) {
  pdl_launch();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= total) return;
  const int64_t u = owner_of(off, B, t);
  const int n = kv_len(lens, u, (int64_t)max_blocks << log_bs, status);
  slots[t] = place(t, u, off[u], off[u + 1], n, first[u], log_bs, max_blocks, n_blocks, table, free_blocks,
                   stack_height(n_free, cap, status), status);
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
  int log_bs = 4;
  while (1 << log_bs < D.block) ++log_bs;
  if (B <= kFusedRequests) {
    const int64_t grid = ceil_div(total, kFusedRows);
    k_reserve_fused<<<(unsigned)(grid > 0 ? grid : 1), kScanThreads, 0, st>>>(
        B, total, log_bs, D.max_blocks, D.n_blocks, lens, off, table, free_blocks, free_cap, n_free,
        lens_out, n_free_out, slots, status);
    note_launches(1);
    return LIME_OK;
  }
  int32_t* first = (int32_t*)ws;
  const int rc = launch_pdl(k_reserve_scan, dim3((unsigned)ceil_div(B, kScanThreads)),
                            dim3(kScanThreads), 0, st, 1, B, total, log_bs, (int)D.max_blocks, lens,
                            off, free_cap, n_free, lens_out, n_free_out, first, status);
  if (rc || total == 0) return rc;
  return launch_pdl(k_reserve_fill, dim3((unsigned)ceil_div(total, 256)), dim3(256), 0, st, 1, B,
                    total, log_bs, (int)D.max_blocks, D.n_blocks, lens, off, table, free_blocks,
                    free_cap, n_free, (const int32_t*)first, slots, status);
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
