// Parts of the cache attention (kv_attn.cu): the division of ragged requests over
// persistent workers, the joining of cut pairs, and the arithmetic of codes and
// probabilities.
#pragma once
#include <cuda_fp16.h>
#include <math.h>

#include "lime_fast.cuh"
#include "lime_kv.cuh"
#include "sm100.cuh"

namespace lime {
namespace kv {

using namespace sm100;

constexpr int kMaxWorkers = 2560;        // of a persistent grid
constexpr int kInlineRequests = 2048;    // most requests whose weights every block sums itself
constexpr int kJoin = 8;                 // parts of a cut pair read at a time
constexpr float kOffset = 14.0f;         // probabilities enter fp16 times 2^14
constexpr float kSlack = 1.5f;           // log2 by which a row's reference may lag its maximum
constexpr float kTiny = 1e-37f;          // least factor of a masked score
constexpr float kUnseen = 3.0e38f;       // kOffset less the reference of a row that has seen no key
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
  const void* Q;
  int64_t ldq;
  const int64_t* off;
  const int32_t* table;
  const int32_t* lens;
  const float2* scale;
  const int64_t* prefix;  // [B + 2] weight before each request, then the
                          // number of pairs (NULL: summed by every block)
  int* tickets;           // [grid] zero between calls
  float* part;            // [2 * grid] partial results
  void* O;
  float* lse;
  unsigned* status;
  int64_t B, total_q, n_blocks;
  int Hq, Hkv, G, max_blocks;
  int log_block;
  int log_g;         // of G, or -1 where it is no power of two
  float scale_log2;  // |sm_scale| log2 e
  bool negative;     // sm_scale < 0
  bool causal;
};

// Host: launches k_kv_plan for requests too many to be summed by every block.
struct Cut;
int launch_plan(const Args& a, const Cut& cut, int64_t* prefix, cudaStream_t st);

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x / y, in 32 bits where they suffice (a 64-bit division takes most of a
// microsecond of a segment's start).
__device__ __forceinline__ int64_t div_by(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}

// How requests are cut into pairs, and pairs into tiles.
struct Cut {
  int heads;  // kv heads of a request
  int R;      // rows of a pair
  int TK;     // keys of a tile
  int cost;   // a pair's fixed cost, in tiles
  int least;  // fewest tiles worth a worker of their own, with a pair's cost
  __device__ __forceinline__ int64_t pairs(int64_t rows, int G) const {
    return ceil_div(rows * G, R) * heads;
  }
  __device__ __forceinline__ int weight(int n) const { return (n + TK - 1) / TK + cost; }
  // A worker's share of all weight.  Where there are more workers than pairs,
  // one below `least` would only add joins, and one above the pairs' mean would
  // put two of them into one worker.
  __device__ __forceinline__ int64_t share(int64_t total, int64_t pairs, int workers) const {
    const int64_t s = div_by(total + workers - 1, workers), mean = div_by(total + pairs - 1, pairs);
    const int64_t floor = least < mean ? least : mean;
    return s > floor ? s : floor;
  }
};

// The request whose weights hold position s: the largest u with prefix[u] <= s
// (a warp probes 32 places at a time).
__device__ __forceinline__ int64_t find_request(const int64_t* prefix, int64_t B, int64_t s) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = B;  // answer in [lo, hi)
  while (hi - lo > 1) {
    const int64_t step = ceil_div(hi - lo, 32);
    const int64_t p = lo + step * lane;
    const bool ok = p < hi && prefix[p] <= s;
    const int n = __popc(__ballot_sync(0xffffffffu, ok));  // n >= 1
    lo += step * (n - 1);
    hi = lo + step < hi ? lo + step : hi;
  }
  return lo;
}

// Where a worker's share begins.
struct Place {
  int64_t u, before;  // request, and the weight before it
  int64_t total, share;
};

template <int WARPS, int GROUPS> struct LocateSmem {
  int64_t sum[WARPS], pairs[WARPS], found[GROUPS][2];
};

// Finds worker `blockIdx.x * GROUPS + group`'s place (all threads of the block
// call it, with WARPS warps); false where it has nothing to do.
template <int WARPS, int GROUPS>
__device__ __forceinline__ bool locate(const Args& a, const Cut& cut, LocateSmem<WARPS, GROUPS>& sm,
                                       int group, Place* at) {
  const int worker = blockIdx.x * GROUPS + group, workers = gridDim.x * GROUPS;
  if (a.prefix) {
    at->total = a.prefix[a.B];
    if (at->total == 0) return false;
    at->share = cut.share(at->total, a.prefix[a.B + 1], workers);
    if (at->share * worker >= at->total) return false;
    at->u = find_request(a.prefix, a.B, at->share * worker);
    at->before = a.prefix[at->u];
    return true;
  }
  const int64_t most = (int64_t)a.max_blocks << a.log_block;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (int)ceil_div(a.B, WARPS * 32);
  const int64_t u0 = (int64_t)per * threadIdx.x, u1 = u0 + per < a.B ? u0 + per : a.B;
  int64_t sum = 0, count = 0;
  for (int64_t v = u0; v < u1; ++v) {
    int64_t x, y;
    user_range(a.off, v, a.B, a.total_q, &x, &y, a.status);
    const int64_t p = cut.pairs(y - x, a.G);
    sum += p * cut.weight(kv_len(a.lens, v, most, a.status));
    count += p;
  }
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  if (lane == 31) sm.sum[warp] = x, sm.pairs[warp] = count;
  __syncthreads();
  int64_t total = 0, from = x - sum, pairs = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) from += sm.sum[w];
    total += sm.sum[w];
    pairs += sm.pairs[w];
  }
  if (total == 0) return false;
  const int64_t share = cut.share(total, pairs, workers);
  if (share * blockIdx.x * GROUPS >= total) return false;  // the whole block
#pragma unroll
  for (int i = 0; i < GROUPS; ++i) {
    const int64_t pos = share * (blockIdx.x * GROUPS + i);
    if (from <= pos && pos < from + sum) {
      int64_t v = u0, f = from;
      for (;; ++v) {
        int64_t p, q;
        user_range(a.off, v, a.B, a.total_q, &p, &q, a.status);
        const int64_t w = cut.pairs(q - p, a.G) * cut.weight(kv_len(a.lens, v, most, a.status));
        if (pos < f + w) break;
        f += w;
      }
      sm.found[i][0] = v;
      sm.found[i][1] = f;
    }
  }
  __syncthreads();
  if (share * worker >= total) return false;
  at->u = sm.found[group][0];
  at->before = sm.found[group][1];
  at->total = total;
  at->share = share;
  return true;
}

// What a segment's start and end know and its tile loop hardly needs: kept in
// shared memory, a copy per warp, for the registers it would hold meanwhile.
struct Segment {
  int64_t pos, pos_end;       // this block's place in the weights, and its end
  int64_t share;              // of every block
  int64_t u, before;          // request, and the weight before it
  int64_t pair_pos, seg_end;  // where the pair begins and the segment ends
  int64_t q0;                 // the request's first query row
  int n, m_rows;              // its cached and its query rows
  int r_base, rows;           // the pair's rows (query, head of the group)
  int w_pair;
};

// The segment at sg.pos, found from the request of the one before it (every
// lane of a warp calls it; sg is the warp's own copy).
struct Head {
  int h, rt;   // kv head, tile of rows
  int t0, t1;  // tiles of the pair
};
__device__ __forceinline__ Head next_segment(const Args& a, const Cut& cut, volatile Segment& sg) {
  const int64_t most = (int64_t)a.max_blocks << a.log_block;
  const int64_t pos = sg.pos, pos_end = sg.pos_end;
  int64_t u = sg.u, before = sg.before, q0, q1;
  int n, w_pair;
  for (;;) {
    user_range(a.off, u, a.B, a.total_q, &q0, &q1, a.status);
    n = kv_len(a.lens, u, most, a.status);
    w_pair = cut.weight(n);
    const int64_t w = cut.pairs(q1 - q0, a.G) * w_pair;
    if (pos < before + w) break;
    before += w;
    ++u;
  }
  const int m_rows = (int)(q1 - q0);
  const int rts = (int)ceil_div((int64_t)m_rows * a.G, cut.R);
  const int64_t pair = div_by(pos - before, w_pair);
  const int64_t pair_pos = before + pair * w_pair;
  const int64_t seg_end = pair_pos + w_pair < pos_end ? pair_pos + w_pair : pos_end;
  Head head;
  head.h = (int)((uint32_t)pair / (uint32_t)rts);
  head.rt = (int)pair - head.h * rts;
  head.t0 = (int)(pos - pair_pos) - cut.cost;
  head.t1 = (int)(seg_end - pair_pos) - cut.cost;
  if (head.t0 < 0) head.t0 = 0;
  if (head.t1 < 0) head.t1 = 0;
  const int r_base = head.rt * cut.R, left = m_rows * a.G - r_base;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    sg.u = u, sg.before = before;
    sg.pair_pos = pair_pos, sg.seg_end = seg_end, sg.q0 = q0;
    sg.n = n, sg.m_rows = m_rows, sg.r_base = r_base, sg.rows = left < cut.R ? left : cut.R;
    sg.w_pair = w_pair;
  }
  __syncwarp();
  return head;
}

// Query row (of its request) that row r of a pair's request belongs to.
__device__ __forceinline__ int query_of(const Args& a, int r) {
  return a.log_g >= 0 ? r >> a.log_g : r / a.G;
}

// Rows of the cache that the segment's row r sees.
__device__ __forceinline__ int limit_of(const Args& a, volatile Segment& sg, int r) {
  if (!a.causal) return sg.n;
  const int lim = sg.n - sg.m_rows + query_of(a, sg.r_base + r) + 1;
  return lim < 0 ? 0 : lim;
}

// One (key, value) scale entry of the table: block `col` of the segment's
// request, for kv head h, and the pair's place among the (block, head)s.  A
// negative key scale hides the block.
__device__ __forceinline__ void load_entry(const Args& a, volatile Segment& sg, int h, int col,
                                           int* place, float2* sc) {
  *place = -1;
  *sc = make_float2(-1.0f, 0.0f);
  if (col >= (sg.n + (1 << a.log_block) - 1) >> a.log_block) return;
  const int b = a.table[sg.u * a.max_blocks + col];
  if (b >= 0 && b < a.n_blocks) {
    *place = b * a.Hkv + h;
    *sc = a.scale[(int64_t)b * a.Hkv + h];
  } else {
    raise_flag(a.status, LIME_FLAG_BAD_BLOCK);
  }
}

// A cut pair's partial results: R rows of DH normalised outputs, then R pairs
// (reference, sum).  Part c of a pair whose first part is worker `first`'s:
template <int R, int DH>
__device__ __forceinline__ float* part_of(const Args& a, int c, int first) {
  return a.part + (2 * (int64_t)c + (c == first ? 1 : 0)) * (R * DH + 2 * R);
}

// Joins the parts of workers first..last in their order; threads 0..threads-1
// each take outputs (row, 4 dims).
template <int R, int DH, typename Store>
__device__ __forceinline__ void join_parts(const Args& a, int first, int last, int thread,
                                           int threads, int rows, Store store) {
  for (int i = thread; i < rows * (DH / 4); i += threads) {
    const int r = i / (DH / 4), d = i % (DH / 4) * 4;
    float top = -INFINITY, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int c0 = first; c0 <= last; c0 += kJoin) {
      float2 x[kJoin];  // kJoin parts in flight
      float4 y[kJoin];
#pragma unroll
      for (int c = 0; c < kJoin; ++c) {
        x[c] = make_float2(-INFINITY, 0.0f);
        y[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c0 + c <= last) {
          const float* p = part_of<R, DH>(a, c0 + c, first);
          x[c] = __ldcg(reinterpret_cast<const float2*>(p + R * DH + 2 * r));
          y[c] = __ldcg(reinterpret_cast<const float4*>(p + r * DH + d));
        }
      }
      float best = top;
#pragma unroll
      for (int c = 0; c < kJoin; ++c) best = fmaxf(best, x[c].x);
      // v stays normalised: outputs near fp32's largest would overflow times a sum
      const float ref = best == -INFINITY ? 0.0f : best;
      float keep = sum * ex2(top - ref);
      sum = keep;
#pragma unroll
      for (int c = 0; c < kJoin; ++c) sum += x[c].y *= ex2(x[c].x - ref);
      top = best;
      const float by = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
      keep *= by;
      v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
      for (int c = 0; c < kJoin; ++c) {
        const float k = x[c].y * by;
        v.x = fmaf(k, y[c].x, v.x), v.y = fmaf(k, y[c].y, v.y);
        v.z = fmaf(k, y[c].z, v.z), v.w = fmaf(k, y[c].w, v.w);
      }
    }
    store(r, d, v, top, sum);
  }
}

// Four outputs of row `at` (query row and head), and its lse.
template <typename T, int DH>
__device__ __forceinline__ void store_out(const Args& a, int64_t at, int d, float4 v, float top,
                                          float sum) {
  T* dst = (T*)a.O + at * DH + d;
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(dst) = v;
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  if (a.lse && d == 0) a.lse[at] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// Powers of two that bring a row whose largest magnitude is top (finite, or
// the exponent's largest) to [2^14, 2^15): s1 * s2; c is scale_log2 over them.
__device__ __forceinline__ void row_scale(const Args& a, float top, float* s1, float* s2, float* c) {
  const int exp = (__float_as_int(top) >> 23) & 255;
  const int shift = 14 + 127 - (exp < 254 ? exp : 254);
  const int e1 = shift >> 1, e2 = shift - e1;
  *s1 = __int_as_float((127 + e1) << 23) * (a.negative ? -1.0f : 1.0f);
  *s2 = __int_as_float((127 + e2) << 23);
  *c = a.scale_log2 * __int_as_float((127 - e1) << 23) * __int_as_float((127 - e2) << 23);
}

// log2 of a value scale over the unit, at least -60 (what is smaller adds
// nothing), and the factor that takes it out of a sum again.  Both may be any
// finite numbers: the fast division gives 0 for a unit above 2^126.
__device__ __forceinline__ void unit_log2(float vs, float unit, float* lr, float* inv) {
  const float ratio = __log2f(__fdiv_rn(vs, unit));
  *lr = unit > 0.0f ? (ratio > -60.0f ? ratio : -60.0f) : 0.0f;
  *inv = ex2(-*lr);
}

// Two fp32 values to an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The same, the largest finite fp16 in place of an overflow: a probability is at
// most 2^(kOffset + kSlack), unless scores beyond 2^22 cost its exponent half a
// unit.
__device__ __forceinline__ uint32_t half2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// {1024 + b0, 1024 + b1} - 1152 of two biased bytes (code + 128) picked by SEL.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
  const uint32_t m = __byte_perm(w, 0x64646464u, SEL);
  const uint32_t bias = 0x64806480u;
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&m),
                            *reinterpret_cast<const __half2*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A wait has run out: lets the copies and products still in flight land
// before the block gives up its memory.
__device__ __forceinline__ void drain_after_timeout(volatile int* abort_flag) {
  if (!*abort_flag) return;
  const uint64_t t0 = global_ns();
  while (global_ns() - t0 < 1000000ull) {
  }
}

}  // namespace kv

}  // namespace lime
