// Block tables and slot maps of the paged history cache, built on the GPU from
// the requests' lengths, and the release of blocks.  Bound by latency: a scan
// over the requests between two rounds of loads.  Release: 256 requests' 25,000
// blocks 8.3 us, 16,384 requests' 365,000 41 us (one block of threads scans them).
#include "lime_fast.cuh"
#include "lime_kv.cuh"
#include "sm100.cuh"

namespace lime {

using namespace sm100;

namespace {

constexpr int kScanThreads = 1024;

// Exclusive sum of one value per thread over the block's THREADS; *total gets
// the sum.
template <int THREADS>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* total) {
  __shared__ int64_t part[32];
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
    int64_t p = lane < THREADS / 32 ? part[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) p += y;
    }
    part[lane] = p;
  }
  __syncthreads();
  *total = part[31];
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
// passes between blocks.  A thread places ROWS rows in a row, with one search for
// their request and mostly one block: 4 where there are rows enough to fill the
// GPU (633,000 rows: 8.1 us against 11.7 with one), 1 where not (256 rows: 3.9
// against 5.7 with four).
constexpr int kFusedRequests = 2048;
constexpr int kFusedThreads = 256;

template <int ROWS>
__global__ void __launch_bounds__(kFusedThreads)
    k_reserve_fused(int B, int64_t total, int log_bs, int max_blocks, int64_t n_blocks,
                    const int32_t* lens, const int64_t* off, int32_t* table,
                    const int32_t* free_blocks, int64_t cap, const int32_t* n_free,
                    int32_t* lens_out, int32_t* n_free_out, int64_t* slots, unsigned* status) {
  extern __shared__ int32_t s_off[];
  int32_t *s_end = s_off + B, *s_len = s_end + B, *s_need = s_len + B, *s_first = s_need + B;
  __shared__ int taken;
  if (threadIdx.x == 0) taken = 0;
  const int64_t most = (int64_t)max_blocks << log_bs;
  const int height = stack_height(n_free, cap, status);
  for (int u = threadIdx.x; u < B; u += kFusedThreads) {
    int64_t a, b;
    user_range(off, u, B, total, &a, &b, status);
    const int n = kv_len(lens, u, most, status);
    s_off[u] = (int32_t)a;
    s_end[u] = (int32_t)b;
    s_len[u] = n;
    s_need[u] = blocks_needed(n, b - a, log_bs, max_blocks);
  }
  __syncthreads();
  const int per = (B + kFusedThreads - 1) / kFusedThreads;
  const int u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : B;
  int64_t sum = 0;
  for (int u = u0; u < u1; ++u) sum += s_need[u] > 0 ? s_need[u] : 0;
  int64_t all;
  int64_t rank = block_scan<kFusedThreads>(sum, &all);
  bool refused = false;
  for (int u = u0; u < u1; ++u) {
    const int need = s_need[u], rows = s_end[u] - s_off[u];
    const bool ok = served(need, rank, height);
    s_first[u] = ok ? (int32_t)(rank < height ? rank : height) : -1;
    if (need > 0) rank += need;
    refused |= !ok;
    if (blockIdx.x == 0) {
      lens_out[u] = s_len[u] + (ok ? rows : 0);
      if (ok && need > 0) atomicMax(&taken, (int)rank);
    }
  }
  refused = __syncthreads_or(refused);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *n_free_out = height - taken;
    if (refused) raise_flag(status, LIME_FLAG_NO_BLOCKS);
  }

  const int64_t t0 = ((int64_t)blockIdx.x * kFusedThreads + threadIdx.x) * ROWS;
  if (t0 >= total) return;
  int u = 0;
  for (int hi = B; hi - u > 1;) {                  // the largest u with off[u] <= t0 is in [u, hi)
    const int mid = (u + hi) >> 1;
    if (s_off[mid] <= t0) u = mid; else hi = mid;
  }
  int64_t out[ROWS], col = -1, base = -1;          // base: first slot of the block in column col
  const int64_t mask = (1 << log_bs) - 1;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t t = t0 + i;
    while (u + 1 < B && t >= s_off[u + 1]) ++u, col = -1;
    const int64_t pos = s_len[u] + (t - s_off[u]);
    if (col != pos >> log_bs || (pos & mask) == 0) {
      const int64_t slot = t < total ? place(t, u, s_off[u], s_end[u], s_len[u], s_first[u], log_bs, max_blocks,
                                             n_blocks, table, free_blocks, height, status)
                                     : -1;
      col = slot < 0 ? -1 : pos >> log_bs;         // the next row may be placed in the same block
      base = slot < 0 ? -1 : slot - (pos & mask);
    }
    out[i] = base < 0 || t >= s_end[u] ? -1 : base + (pos & mask);
  }
  if (ROWS % 2 == 0 && t0 + ROWS <= total && ((uintptr_t)slots & 15) == 0) {
#pragma unroll
    for (int i = 0; i + 1 < ROWS; i += 2)
      *reinterpret_cast<longlong2*>(slots + t0 + i) = make_longlong2(out[i], out[i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (t0 + i < total) slots[t0 + i] = out[i];
  }
}

// More requests: a block of threads owns kScanThreads of them and sums the needs
// of all before them itself.  With at most kShortRows rows to a request on
// average (slots != NULL) it also places them, a thread or, beyond 32 rows, a
// warp to a request; otherwise a second kernel does, by rows, which first[u]
// tells the rank of request u's first new block on the stack, or -1 where the
// request is refused.  65,000 rows of 16,384 requests: one kernel 12.0 us, two
// 15.2.
constexpr int kShortRows = 32;

__global__ void __launch_bounds__(kScanThreads)
    k_reserve_scan(int64_t B, int64_t total, int log_bs, int max_blocks, int64_t n_blocks,
                   const int32_t* lens, const int64_t* off, int32_t* table,
                   const int32_t* free_blocks, int64_t cap, const int32_t* n_free,
                   int32_t* lens_out, int32_t* n_free_out, int32_t* first, int64_t* slots,
                   unsigned* status) {
  __shared__ int taken;
  pdl_launch();
  pdl_wait();
  const int64_t most = (int64_t)max_blocks << log_bs;
  const int height = stack_height(n_free, cap, status);
  const int64_t begin = (int64_t)blockIdx.x * kScanThreads, u = begin + threadIdx.x;
  int64_t sum = 0;
  // (their own blocks of threads flag what is wrong with them)
#pragma unroll 8
  for (int64_t v = threadIdx.x; v < begin; v += kScanThreads) {
    int64_t x = off[v], y = off[v + 1], n = lens[v];
    x = x < 0 ? 0 : x > total ? total : x;
    y = y < x ? x : y > total ? total : y;
    n = n < 0 ? 0 : n > most ? most : n;
    const int need = blocks_needed((int)n, y - x, log_bs, max_blocks);
    sum += need > 0 ? need : 0;
  }
  int64_t a = 0, b = 0, before, all;
  int n = 0, need = 0;
  if (u < B) {
    user_range(off, u, B, total, &a, &b, status);
    n = kv_len(lens, u, most, status);
    need = blocks_needed(n, b - a, log_bs, max_blocks);
  }
  block_scan<kScanThreads>(sum, &before);
  const int64_t rank = before + block_scan<kScanThreads>(need > 0 ? need : 0, &all);
  if (threadIdx.x == 0) taken = (int)(before < height ? before : height);
  __syncthreads();
  int64_t mine = -1;                               // rank of this request's first block
  bool refused = false;
  if (u < B) {
    const bool ok = served(need, rank, height);
    if (!slots) first[u] = ok ? (int32_t)(rank < height ? rank : height) : -1;
    lens_out[u] = n + (ok ? (int)(b - a) : 0);
    if (ok && need > 0) atomicMax(&taken, (int)(rank + need));
    refused = !ok;
    mine = ok ? (rank < height ? rank : height) : -1;
  }
  refused = __syncthreads_or(refused);
  if (refused && threadIdx.x == 0) raise_flag(status, LIME_FLAG_NO_BLOCKS);
  // the block in which the stack runs out, or the last one, knows what is taken
  const bool last = begin + kScanThreads >= B;
  if (threadIdx.x == 0 && before <= height && (last || before + all > height))
    *n_free_out = height - taken;
  if (!slots) return;
  const bool few = b - a <= 32;
  if (few) {
    const int64_t mask = (1 << log_bs) - 1;
    int64_t base = -1;                             // first slot of the current block
    for (int64_t t = a; t < b; ++t) {
      const int64_t pos = n + (t - a);
      if (t == a || (pos & mask) == 0) {
        const int64_t slot = place(t, u, a, b, n, mine, log_bs, max_blocks, n_blocks, table, free_blocks, height,
                                   status);
        base = slot < 0 ? -1 : slot - (pos & mask);
      }
      slots[t] = base < 0 ? -1 : base + (pos & mask);
    }
  }
  for (unsigned left = __ballot_sync(0xffffffffu, !few); left; left &= left - 1) {
    const int src = __ffs(left) - 1;
    const int64_t wa = __shfl_sync(0xffffffffu, a, src), wb = __shfl_sync(0xffffffffu, b, src);
    const int64_t wu = __shfl_sync(0xffffffffu, u, src), wm = __shfl_sync(0xffffffffu, mine, src);
    const int wn = __shfl_sync(0xffffffffu, n, src);
    for (int64_t t = wa + (threadIdx.x & 31); t < wb; t += 32)
      slots[t] = place(t, wu, wa, wb, wn, wm, log_bs, max_blocks, n_blocks, table, free_blocks, height, status);
  }
  // rows that the offsets give to nobody
  if (u == 0)
    for (int64_t t = 0; t < a; ++t) slots[t] = -1;
  if (u == B - 1)
    for (int64_t t = b; t < total; ++t) slots[t] = -1;
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

// Table columns [c0, c1) whose blocks request u gives back.
__device__ __forceinline__ void released(const int32_t* lens, const int32_t* keep, int64_t u, int bs, int max_blocks,
                                         unsigned* status, int* rows, int64_t* c0, int64_t* c1) {
  const int n = kv_len(lens, u, (int64_t)max_blocks * bs, status);
  *rows = kept_rows(keep, u, n);
  *c0 = ceil_div(*rows, bs);
  *c1 = ceil_div(n, bs);
}

// A warp per request counts the blocks it gives back.  Entries outside the pool
// are no blocks: on the stack they would be handed out again and again.
__global__ void k_release_count(int64_t B, int bs, int max_blocks, int64_t n_blocks, const int32_t* lens,
                                const int32_t* keep, const int32_t* table, int32_t* lens_out, int64_t* first,
                                unsigned* status) {
  const int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (u >= B) return;
  int rows;
  int64_t c0, c1;
  released(lens, keep, u, bs, max_blocks, status, &rows, &c0, &c1);
  int count = 0;
  bool odd = false;
  for (int64_t c = c0 + (threadIdx.x & 31); c < c1; c += 32) {
    const int32_t id = table[u * max_blocks + c];
    const bool ok = id >= 0 && id < n_blocks;
    count += ok;
    odd |= !ok;
  }
  if (odd) raise_flag(status, LIME_FLAG_BAD_BLOCK);
  count = __reduce_add_sync(0xffffffffu, count);
  if ((threadIdx.x & 31) == 0) {
    first[u] = count;
    lens_out[u] = rows;
  }
}

// first[u]: from the number of blocks that u gives back to the place of the first.
__global__ void __launch_bounds__(kScanThreads)
    k_release_scan(int64_t B, int64_t cap, const int32_t* n_free, int32_t* n_free_out, int64_t* first,
                   unsigned* status) {
  const int64_t per = ceil_div(B, kScanThreads);
  const int64_t u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : B;
  const int height = stack_height(n_free, cap, status);
  int64_t sum = 0;
  for (int64_t u = u0; u < u1; ++u) sum += first[u];
  int64_t all;
  int64_t at = height + block_scan<kScanThreads>(sum, &all);
  for (int64_t u = u0; u < u1; ++u) {
    const int64_t count = first[u];
    first[u] = at;
    at += count;
  }
  if (threadIdx.x == 0) {
    if (height + all > cap) raise_flag(status, LIME_FLAG_BAD_BLOCK);
    *n_free_out = (int32_t)(height + all < cap ? height + all : cap);
  }
}

// A warp per request pushes its released blocks.
__global__ void k_release_fill(int64_t B, int bs, int max_blocks, int64_t n_blocks, const int32_t* lens,
                               const int32_t* keep, int32_t* table, int32_t* free_blocks, int64_t cap,
                               const int64_t* first, unsigned* status) {
  const int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (u >= B) return;
  const int lane = threadIdx.x & 31;
  int rows;
  int64_t c0, c1, at = first[u];
  released(lens, keep, u, bs, max_blocks, status, &rows, &c0, &c1);
  for (; c0 < c1; c0 += 32) {
    const int64_t c = c0 + lane;
    const int32_t id = c < c1 ? table[u * max_blocks + c] : -1;
    const bool ok = id >= 0 && id < n_blocks;
    const unsigned good = __ballot_sync(0xffffffffu, ok);
    const int64_t to = at + __popc(good & ((1u << lane) - 1u));
    if (ok && to < cap) free_blocks[to] = id;
    if (c < c1) table[u * max_blocks + c] = -1;
    at += __popc(good);
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
    const int rows = total >= (int64_t)num_sms() * 2 * kFusedThreads ? 4 : 1;
    const int64_t grid = ceil_div(total, rows * kFusedThreads);
    auto kernel = rows == 4 ? k_reserve_fused<4> : k_reserve_fused<1>;
    kernel<<<(unsigned)(grid > 0 ? grid : 1), kFusedThreads, (size_t)B * 20, st>>>(
        (int)B, total, log_bs, D.max_blocks, D.n_blocks, lens, off, table, free_blocks, free_cap,
        n_free, lens_out, n_free_out, slots, status);
    note_launches(1);
    return LIME_OK;
  }
  int32_t* first = (int32_t*)ws;
  const bool alone = total <= B * kShortRows;
  const int rc = launch_pdl(k_reserve_scan, dim3((unsigned)ceil_div(B, kScanThreads)),
                            dim3(kScanThreads), 0, st, 1, B, total, log_bs, (int)D.max_blocks,
                            D.n_blocks, lens, off, table, free_blocks, free_cap, n_free, lens_out,
                            n_free_out, first, alone ? slots : (int64_t*)nullptr, status);
  if (rc || alone) return rc;
  return launch_pdl(k_reserve_fill, dim3((unsigned)ceil_div(total, 256)), dim3(256), 0, st, 1, B,
                    total, log_bs, (int)D.max_blocks, D.n_blocks, lens, off, table, free_blocks,
                    free_cap, n_free, (const int32_t*)first, slots, status);
}

int kv_release(const lime_kv_dims& D, int64_t B, const int32_t* lens, const int32_t* keep,
               int32_t* table, int32_t* free_blocks, int64_t free_cap, const int32_t* n_free,
               int32_t* lens_out, int32_t* n_free_out, void* ws, unsigned* status,
               cudaStream_t st) {
  int64_t* first = (int64_t*)ws;
  const unsigned grid = (unsigned)ceil_div(B, 8);
  if (B > 0) {
    k_release_count<<<grid, 256, 0, st>>>(B, D.block, D.max_blocks, D.n_blocks, lens, keep, table, lens_out, first,
                                          status);
    note_launches(1);
  }
  k_release_scan<<<1, kScanThreads, 0, st>>>(B, free_cap, n_free, n_free_out, first, status);
  note_launches(1);
  if (B > 0) {
    k_release_fill<<<grid, 256, 0, st>>>(B, D.block, D.max_blocks, D.n_blocks, lens, keep, table, free_blocks,
                                         free_cap, first, status);
    note_launches(1);
  }
  return LIME_OK;
}

}  // namespace lime
