// Attention over the paged 8-bit history cache (include/lime_kv.h).
//
// A pair is one (request, kv head, tile of R query rows).  Its cached rows are
// cut into tiles of TK keys; all pairs' tiles, laid end to end, are divided
// evenly over the workers of a persistent grid, so that ragged requests load
// every SM alike.  A worker's share of one pair is a segment.  A worker is a
// block of four warps, which take the segment's tiles in turn, each with its own
// softmax state and its own ring of TMA stages, and join their states at the
// segment's end; or, in large calls (kv_attention has the rule), one warp.  A pair cut
// by workers' borders leaves partial results, which the last worker to finish
// joins in the workers' order.
//
// Both products run on mma.sync with fp16 operands and fp32 sums.  A code is
// exact in fp16, and becomes a matrix fragment in registers: the byte under the
// exponent of 1024 (0x64) is 1024 + code + 128, less 1152.  tcgen05 reads its
// operands from shared memory or TMEM, which adds a store and a load of two
// bytes for every code read once (and block-diagonal queries where a head has
// fewer than 128 rows); built that way, with the probabilities in TMEM, the
// kernel took 76 us where this one takes 54 (32 links over 16,384 rows), 71
// against 55 (causal chunks) and 133 against 128 (64 links, ragged).  mma.sync
// reaches 552 TFLOP/s here, which is never the bound.  Which key a fragment's
// column stands for, and which dims a lane holds, are free as long as both
// products agree; KeyMap picks them so that every shared-memory read is a wide
// one without bank conflicts.
//
// Measured (B200, graph replay): 64 requests' single tokens, 32 query heads on 8,
// dh 128, 508,000 rows in all: 173 us, 6.0 TB/s, 92 % of the copy bandwidth (1.05 GB
// of DRAM reads by its counters); called one by one over inputs that change, 194 us.
// 32 x 32 links over 16,384 rows, 4 heads of 32: 54 us, 2.5 TB/s; there a warp
// holds 32 rows and two blocks of four warps fill an SM's registers.  A tile of
// 64 keys takes a warp about 700 instructions, 64 of them mma.sync at four to
// five issue slots each: 1,000 of the 1,800 cycles that a scheduler spends on it
// (tensor and special-function pipe: 500 each).  Three blocks spill (58 us) or,
// with steps of 32 keys, spend more on their steps (62 us); row tiles of 16 took
// 74 us, of 64 (64 links, ragged) 159 against 134.
#include "kv_attn.cuh"

namespace lime {

using namespace kv;

namespace {

constexpr int kWarps = 4;

// How a worker of NW warps divides the work: a pair's fixed cost in its tiles
// (about 5 us beside 1 us a tile and warp; 2 to 10 tiles measured), and the
// fewest tiles worth a worker of their own.
template <int NW> constexpr int kPairCost = 5 * NW;
template <int NW> constexpr int kLeast = kPairCost<NW> + 4 * NW;

// Per head dim: keys of a warp's tile (one ring stage), keys of one softmax
// step, stages of the ring.
template <int DH> struct Tile {
  static constexpr int TK = DH == 128 ? 32 : 64;
  static constexpr int SK = DH <= 32 ? 64 : 32;
  static constexpr int kStages = DH <= 32 ? 3 : DH == 64 ? 2 : 2;
  static constexpr int kBytes = TK * DH;             // keys (or values) of a tile
  static constexpr int kRing = kStages * 2 * kBytes; // per warp
};

// ------------------------------------------------------------------- plan

// Prefix sums of the requests' weights, where there are too many requests for
// every block to sum them.
__global__ void __launch_bounds__(1024)
    k_kv_plan(int64_t B, const int64_t* off, int64_t total_q, const int32_t* lens, int G, int64_t most,
              Cut cut, int64_t* prefix, unsigned* status) {
  __shared__ int64_t part[32];
  __shared__ unsigned long long all_pairs;
  if (threadIdx.x == 0) all_pairs = 0;
  __syncthreads();
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = ceil_div(B, 1024);
  const int64_t u0 = per * threadIdx.x, u1 = u0 + per < B ? u0 + per : B;
  int64_t sum = 0, pairs = 0;
  for (int64_t u = u0; u < u1; ++u) {
    int64_t a, b;
    user_range(off, u, B, total_q, &a, &b, status);
    const int64_t p = cut.pairs(b - a, G);
    const int64_t w = p * cut.weight(kv_len(lens, u, most, status));
    prefix[u] = w;
    sum += w;
    pairs += p;
  }
  if (pairs) atomicAdd(&all_pairs, (unsigned long long)pairs);
  int64_t x = sum;
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
  int64_t at = (warp ? part[warp - 1] : 0) + x - sum;
  for (int64_t u = u0; u < u1; ++u) {
    const int64_t w = prefix[u];
    prefix[u] = at;
    at += w;
  }
  if (threadIdx.x == 0) {
    prefix[B] = part[31];
    prefix[B + 1] = (int64_t)all_pairs;
  }
}

// -------------------------------------------------------------- fragments

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The same onto zero.
__device__ __forceinline__ void mma16816_first(float* c, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Byte offset inside a tile, through the 128-byte swizzle the TMA applies.
__device__ __forceinline__ uint32_t swz(uint32_t off) { return off ^ (((off >> 7) & 7u) << 4); }

// swz(lane | c) from at = swz(lane), where lane and the constant c share no bit.
__device__ __forceinline__ uint32_t swz_at(uint32_t at, uint32_t c) {
  return (at ^ (((c >> 7) & 7u) << 4)) + c;
}

// Which of 16 keys a fragment's columns stand for.  Column c of the first
// (second) 8-key product is key col(c) (col(c) + odd): lane t of a quad then
// holds in both products the scores, and as value rows the codes, of keys
// key(t, 0..3).  With the tiles' swizzle, no two lanes of a shared-memory
// access phase meet in a bank, for the key reads (a row per lane group g) and
// for the value reads (a row per lane t).
template <int DH> struct KeyMap {
  static constexpr int odd = DH == 64 ? 2 : 8;
  __device__ static __forceinline__ int col(int c) {
    const int t = c >> 1;
    if (DH == 64) return 4 * t + (c & 1);
    if (DH == 32) return (c & 1) ? 4 + (t ^ 2) : t;
    return c;
  }
  __device__ static __forceinline__ int key(int t, int i) { return col(2 * t + (i & 1)) + (i >> 1) * odd; }
};

// BYTES of shared memory into words.
template <int BYTES>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t* w) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

// ----------------------------------------------------------------- kernel

// Blocks an SM holds, by registers.
template <typename T, int DH, int MT>
constexpr int min_blocks() {
  return DH <= 32 ? (MT == 2 ? 2 : 4) : DH == 64 ? (MT == 2 ? 2 : 3) : (sizeof(T) == 2 ? 3 : 2);
}

// ONE: a softmax step's keys lie in one block (block >= SK), under one scale.
// NW: warps of a worker, which share a segment's tiles (kWarps), or each take
// segments of their own (1).
template <typename T, int DH, int MT, bool ONE, int NW>
__global__ void __launch_bounds__(kWarps * 32, min_blocks<T, DH, MT>())
    k_kv_attn(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const Args a) {
  constexpr bool kSplit = sizeof(T) == 4;  // fp32 rows: operands as two fp16 terms
  constexpr int NQ = kSplit ? 2 : 1;
  // A tensor core's adds truncate, which over thousands of keys costs fp32 outputs
  // more than all else: single queries over 4,096 keys of 32 dims are 1.4e-6 of their
  // size off, and 4e-7 with a step's products summed apart, added with rounding, and
  // the scores' small terms summed first.  That takes 5 to 8 % more time (32 links over
  // 2,048 rows 72.5 to 78 us).  Heads of 128 have no registers for sums apart; the
  // scores' order alone brings them to 7.5e-7 (from 1.3e-6), for 3 to 6 %.
  constexpr bool kApart = kSplit && DH <= 64;
  constexpr int TK = Tile<DH>::TK, SK = Tile<DH>::SK, S = Tile<DH>::kStages, NG = SK / 16;
  constexpr int kGroups = kWarps / NW;     // workers of a block
  constexpr int NC = ONE ? 1 : NG;         // scales of a step
  constexpr int R = 16 * MT;
  constexpr int KS = DH / 16;              // k-steps of the score product
  constexpr int NT = DH / 8;               // 8-dim tiles of the output
  constexpr int E = DH / 4;                // dims of a lane
  constexpr int VB = DH / 8;               // value bytes of a lane and key
  typedef KeyMap<DH> Map;

  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kWarps][S];
  __shared__ float2 ml[kWarps][R];
  __shared__ int abort_flag, arrived;
  __shared__ Segment segments[kWarps];
  __shared__ LocateSmem<kWarps, kGroups> locate_smem;
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);  // 1,024-byte aligned: the swizzle's period

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = warp / NW, gw = warp % NW, gt = threadIdx.x % (NW * 32);  // worker, warp and thread in it
  const int worker = blockIdx.x * kGroups + group;
  auto sync = [&] {                        // of a worker
    if (NW == 1) __syncwarp();
    else __syncthreads();
  };
  uint8_t* ring = smem + warp * Tile<DH>::kRing;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  const int bs = 1 << a.log_block;
  const int nb = bs >= TK ? 1 : TK / bs;   // blocks of a tile, each with an arrival of its own
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(&full[warp][s], nb);
  fence_mbar_init();
  __syncthreads();
  pdl_launch();
  pdl_wait();

  const Cut cut = {a.Hkv, R, TK, kPairCost<NW>, kLeast<NW>};
  Place place;
  if (!locate<kWarps, kGroups>(a, cut, locate_smem, group, &place)) return;
  volatile Segment& sg = segments[warp];
  if (lane == 0) {
    const int64_t pos = place.share * worker;
    sg.pos = pos;
    sg.pos_end = pos + place.share < place.total ? pos + place.share : place.total;
    sg.share = place.share;
    sg.u = place.u;
    sg.before = place.before;
  }
  __syncwarp();

  const int box_rows = bs >= TK ? TK : bs;
  const uint32_t box_bytes = (uint32_t)box_rows * DH;
  const int batch = 32 / nb;               // tiles whose table entries a warp holds

  // this lane's reads: key rows, and value rows of the keys key(t, 0) and key(t, 1)
  const uint32_t k_at = swz(Map::col(g) * DH + E * t);
  const uint32_t v_at0 = swz(Map::key(t, 0) * DH + VB * g), v_at1 = swz(Map::key(t, 1) * DH + VB * g);
  uint32_t stage = 0, phase = 0;           // of the ring; phase: one bit per stage

  while (sg.pos < sg.pos_end) {
    const Head head = next_segment(a, cut, sg);
    const int h = head.h, t0 = head.t0, rows = sg.rows, r_base = sg.r_base;
    const int64_t q0 = sg.q0;
    const int lim_low = limit_of(a, sg, 0), lim_high = limit_of(a, sg, rows - 1);
    const int t_live = (lim_high + TK - 1) / TK;
    const int t1 = head.t1 < t_live ? head.t1 : t_live;

    // from: kOffset less the row's reference; a probability's exponent adds it
    float o[MT][NT][4], from[MT][2], vref = 0.0f;
    uint64_t l[MT][2];                   // sums of the even and the odd columns
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      from[mt][0] = from[mt][1] = kUnseen;
      l[mt][0] = l[mt][1] = 0;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.0f;
    }

    // ---- queries, raw: asked for before the tiles, which would delay them
    constexpr int NV = E * (int)sizeof(T) / 16 > 0 ? E * (int)sizeof(T) / 16 : 1;
    uint4 raw[MT][2][NV];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = mt * 16 + hf * 8 + g;
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[mt][hf][i] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
          const int rr = r_base + r, qi = query_of(a, rr);
          const T* src = (const T*)a.Q + (q0 + qi) * a.ldq + (h * a.G + rr - qi * a.G) * DH + E * t;
          if constexpr (E * sizeof(T) >= 16) {
#pragma unroll
            for (int i = 0; i < NV; ++i) raw[mt][hf][i] = reinterpret_cast<const uint4*>(src)[i];
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            raw[mt][hf][0] = make_uint4(v.x, v.y, 0, 0);
          }
        }
      }
    }

    // ---- table entries and scales of 32 / nb tiles ahead, one block per lane
    const int count = t1 - t0 > gw ? (t1 - t0 - gw + NW - 1) / NW : 0;
    auto load_batch = [&](int first, int& ent, float2& sc) {
      const int j = first + lane / nb;
      const int col = (((t0 + gw + j * NW) * TK) >> a.log_block) + lane % nb;
      load_entry(a, sg, h, j < count ? col : INT32_MAX, &ent, &sc);
    };
    int ent0, ent1;
    float2 sc0, sc1;
    load_batch(0, ent0, sc0);
    load_batch(batch, ent1, sc1);
    int base = 0;                        // first tile of batch 0

    // Brings tile j into ring stage `st`.  An elected lane asks for the copies,
    // in fewer instructions than one picked by its number (single tokens 174 us
    // against 178, 64 links 127 against 130).
    auto issue = [&](int j, uint32_t st) {
      const int src = (j - base) * nb;
      const int mine = src < 32 ? ent0 : ent1;
      const int row = bs >= TK ? (((t0 + gw + j * NW) * TK) & (bs - 1)) * DH / 128 : 0;
      uint8_t* dst = ring + st * 2 * Tile<DH>::kBytes;
#pragma unroll 1
      for (int i = 0; i < nb; ++i, dst += box_bytes) {
        const int z = __shfl_sync(0xffffffffu, mine, src + i);
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[warp][st], z >= 0 ? 2 * box_bytes : 0);
          if (z >= 0) {
            tma_load_3d(dst, &map_k, 0, row, z, &full[warp][st]);
            tma_load_3d(dst + Tile<DH>::kBytes, &map_v, 0, row, z, &full[warp][st]);
          }
        }
      }
    };

    {
      uint32_t st = stage;
      for (int j = 0; j < S && j < count; ++j) {
        issue(j, st);
        st = st + 1 == S ? 0 : st + 1;
      }
    }

    // ---- queries: fp16 fragments of rows scaled to [2^14, 2^15)
    uint32_t qf[MT][KS][NQ][4];
    float c_row[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float x[E < 8 ? 8 : E];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (sizeof(T) == 2) {
            unpack8(raw[mt][hf][i], x + 8 * i);
          } else {
            x[4 * i] = __uint_as_float(raw[mt][hf][i].x), x[4 * i + 1] = __uint_as_float(raw[mt][hf][i].y);
            x[4 * i + 2] = __uint_as_float(raw[mt][hf][i].z), x[4 * i + 3] = __uint_as_float(raw[mt][hf][i].w);
          }
        }
        float top = 0.0f;
#pragma unroll
        for (int d = 0; d < E; ++d) top = fmaxf(top, fabsf(x[d]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float s1, s2;
        row_scale(a, top, &s1, &s2, &c_row[mt][hf]);
#pragma unroll
        for (int w = 0; w < KS; ++w) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = x[4 * w + i] * s1 * s2;
          const uint32_t h0 = half2_of(y[0], y[1]), h1 = half2_of(y[2], y[3]);
          qf[mt][w][0][hf] = h0;
          qf[mt][w][0][hf + 2] = h1;
          if constexpr (kSplit) {
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
            qf[mt][w][NQ - 1][hf] = half2_of(y[0] - f0.x, y[1] - f0.y);
            qf[mt][w][NQ - 1][hf + 2] = half2_of(y[2] - f1.x, y[3] - f1.y);
          }
        }
      }
    }

    // Probabilities carry their block's value scale over a unit, the largest
    // scale so far: log2 of the ratio joins the exponent, and the sum takes it
    // out again.  A lane holds both for its block of the batch.
    float lr0, inv0;
    auto new_unit = [&] {
      const float most = fmaxf(vref, warp_max(sc0.y));
      if (most > vref) {
        const float keep = vref / most;
        vref = most;
        const uint64_t keep2 = pack2(keep, keep);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              unpack2(mul2(pack2(o[mt][i][2 * hf], o[mt][i][2 * hf + 1]), keep2), o[mt][i][2 * hf],
                      o[mt][i][2 * hf + 1]);
      }
      unit_log2(sc0.y, vref, &lr0, &inv0);
    };
    new_unit();

    for (int j = 0; j < count; ++j) {
      if (__builtin_expect(j - base == batch, 0)) {  // batch 0 is used up
        base += batch;
        ent0 = ent1;
        sc0 = sc1;
        load_batch(base + batch, ent1, sc1);
        new_unit();
      }
      const uint8_t *ks = ring + stage * 2 * Tile<DH>::kBytes, *vs = ks + Tile<DH>::kBytes;
      mbar_wait(&full[warp][stage], (phase >> stage) & 1u, a.status, &abort_flag);
      phase ^= 1u << stage;

#pragma unroll 1
      for (int sub = 0; sub < TK; sub += SK) {
        const int key0 = (t0 + gw + j * NW) * TK + sub;
        if (sub > 0 && key0 >= lim_high) break;
        const uint32_t flip = ((sub * DH >> 7) & 7) << 4;  // of the step's first row (0 but for DH 16)

        // ---- the blocks' scales; hidden keys
        float kg[NC], lr[NC], inv[NC];
        bool hidden = false;
#pragma unroll
        for (int x = 0; x < NC; ++x) {
          const int src = (j - base) * nb + (nb > 1 ? (sub + x * 16) >> a.log_block : 0);
          kg[x] = __shfl_sync(0xffffffffu, sc0.x, src);
          lr[x] = __shfl_sync(0xffffffffu, lr0, src);
          inv[x] = __shfl_sync(0xffffffffu, inv0, src);
          hidden |= kg[x] < 0.0f;
        }
        float c[MT][2][NC];                  // factors of a score to units of log2
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int x = 0; x < NC; ++x) c[mt][hf][x] = c_row[mt][hf] * kg[x];

        // ---- scores
        float s[MT][2 * NG][4];
#pragma unroll
        for (int x = 0; x < 2 * NG; ++x) {
          const uint32_t row = ((x >> 1) * 16 + (x & 1) * Map::odd) * DH;
          uint32_t w[KS];
#pragma unroll
          for (int c = 0; c < E; c += 16)
            lds<E < 16 ? E : 16>(ks + sub * DH + (swz_at(k_at, row) ^ c ^ flip), w + c / 4);
          auto key_frags = [&](int k, uint32_t& b0, uint32_t& b1) {
            const uint32_t b = w[k] ^ 0x80808080u;
            b0 = codes_to_half2<0x4140>(b), b1 = codes_to_half2<0x4342>(b);
          };
          if constexpr (kSplit) {
            // second terms first: a tensor core's adds truncate, and onto a whole
            // score that of a small term costs as much as a large one's
            uint32_t b0[KS], b1[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) key_frags(k, b0[k], b1[k]);
#pragma unroll
            for (int p = NQ - 1; p >= 0; --p)
#pragma unroll
              for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                  if (p == NQ - 1 && k == 0) mma16816_first(s[mt][x], qf[mt][k][p], b0[k], b1[k]);
                  else mma16816(s[mt][x], qf[mt][k][p], b0[k], b1[k]);
                }
          } else {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              uint32_t b0, b1;
              key_frags(k, b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                if (k == 0) mma16816_first(s[mt][x], qf[mt][k][0], b0, b1);
                else mma16816(s[mt][x], qf[mt][k][0], b0, b1);
              }
            }
          }
        }

        if (__builtin_expect(hidden || key0 + SK > lim_low, 0)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int r = mt * 16 + hf * 8 + g;
              const int lim = r < sg.rows ? limit_of(a, sg, r) : 0;
#pragma unroll
              for (int x = 0; x < 2 * NG; ++x) {
                const int key = key0 + (x >> 1) * 16 + (x & 1) * Map::odd;
                const bool off = kg[ONE ? 0 : x >> 1] < 0.0f;
                if (off || key + Map::col(2 * t) >= lim) s[mt][x][2 * hf] = -INFINITY;
                if (off || key + Map::col(2 * t + 1) >= lim) s[mt][x][2 * hf + 1] = -INFINITY;
              }
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int x = 0; x < NC; ++x) c[mt][hf][x] = fmaxf(c[mt][hf][x], kTiny);  // -inf times 0 is NaN
        }

        // ---- running maximum, in units of log2
        float top[MT][2];
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float best = -INFINITY;
#pragma unroll
            for (int x = 0; x < NG; ++x) {
              const float v = max3(s[mt][2 * x][2 * hf], s[mt][2 * x][2 * hf + 1], s[mt][2 * x + 1][2 * hf]);
              if (ONE) best = max3(best, v, s[mt][2 * x + 1][2 * hf + 1]);
              else best = fmaxf(best, fmaxf(v, s[mt][2 * x + 1][2 * hf + 1]) * c[mt][hf][ONE ? 0 : x]);
            }
            top[mt][hf] = best;
            grow |= (ONE ? fmaf(best, c[mt][hf][0], from[mt][hf]) : best + from[mt][hf]) > kOffset + kSlack;
          }
        }
        if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float v = top[mt][hf];
              if (ONE) v *= c[mt][hf][0];
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
              const float to = fminf(from[mt][hf], kOffset - v), keep = ex2(to - from[mt][hf]);
              from[mt][hf] = to;
              const uint64_t keep2 = pack2(keep, keep);
              l[mt][hf] = mul2(l[mt][hf], keep2);
#pragma unroll
              for (int i = 0; i < NT; ++i)
                unpack2(mul2(pack2(o[mt][i][2 * hf], o[mt][i][2 * hf + 1]), keep2), o[mt][i][2 * hf],
                       o[mt][i][2 * hf + 1]);
            }
          }
        }

        // ---- probabilities
        uint32_t pf[MT][NG][NQ][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int x = 0; x < NG; ++x) {
              const float by_c = c[mt][hf][ONE ? 0 : x], add = from[mt][hf] + lr[ONE ? 0 : x];
              float p[4];
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                unpack2(fma2(pack2(s[mt][2 * x + (i >> 1)][2 * hf], s[mt][2 * x + (i >> 1)][2 * hf + 1]),
                            pack2(by_c, by_c), pack2(add, add)),
                       p[i], p[i + 1]);
                p[i] = ex2(p[i]);
                p[i + 1] = ex2(p[i + 1]);
              }
              const float by = inv[ONE ? 0 : x];
              l[mt][hf] = fma2(add2(pack2(p[0], p[1]), pack2(p[2], p[3])), pack2(by, by), l[mt][hf]);
              const uint32_t h0 = half2_sat(p[0], p[1]), h1 = half2_sat(p[2], p[3]);
              pf[mt][x][0][hf] = h0;
              pf[mt][x][0][hf + 2] = h1;
              if constexpr (kSplit) {
                const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                pf[mt][x][NQ - 1][hf] = half2_of(p[0] - f0.x, p[1] - f0.y);
                pf[mt][x][NQ - 1][hf + 2] = half2_of(p[2] - f1.x, p[3] - f1.y);
              }
            }
          }
        }

        // ---- values
        constexpr int W = VB < 4 ? 1 : VB / 4, NI = VB < 4 ? VB : 4;
        auto load_values = [&](int x, uint32_t (&w)[4][W]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lds<VB>(vs + sub * DH +
                        (swz_at(i & 1 ? v_at1 : v_at0, (x * 16 + (i >> 1) * Map::odd) * DH) ^ flip),
                    w[i]);
#pragma unroll
            for (int c = 0; c < W; ++c) w[i][c] ^= 0x80808080u;
          }
        };
        // fragments of dims 4 c + i: bytes of two keys side by side, two dims at a time
        auto value_frags = [&](uint32_t (&w)[4][W], int c, int i, uint32_t& b0, uint32_t& b1) {
          const uint32_t ab = __byte_perm(w[0][c], w[1][c], i < 2 ? 0x5140 : 0x7362);
          const uint32_t cd = __byte_perm(w[2][c], w[3][c], i < 2 ? 0x5140 : 0x7362);
          b0 = (i & 1) ? codes_to_half2<0x4342>(ab) : codes_to_half2<0x4140>(ab);
          b1 = (i & 1) ? codes_to_half2<0x4342>(cd) : codes_to_half2<0x4140>(cd);
        };
        if constexpr (kApart) {
          uint32_t w[NG][4][W];
#pragma unroll
          for (int x = 0; x < NG; ++x) load_values(x, w[x]);
#pragma unroll
          for (int c = 0; c < W; ++c) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              float part[MT][4];
#pragma unroll
              for (int x = 0; x < NG; ++x) {
                uint32_t b0, b1;
                value_frags(w[x], c, i, b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int p = 0; p < NQ; ++p) {
                    if (x + p == 0) mma16816_first(part[mt], pf[mt][x][p], b0, b1);
                    else mma16816(part[mt], pf[mt][x][p], b0, b1);
                  }
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                float* to = o[mt][4 * c + i];
#pragma unroll
                for (int k = 0; k < 4; k += 2)
                  unpack2(add2(pack2(to[k], to[k + 1]), pack2(part[mt][k], part[mt][k + 1])), to[k], to[k + 1]);
              }
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < NG; ++x) {
            uint32_t w[4][W];
            load_values(x, w);
#pragma unroll
            for (int c = 0; c < W; ++c) {
              // bytes of two keys side by side, two dims at a time
              const uint32_t ab0 = __byte_perm(w[0][c], w[1][c], 0x5140), cd0 = __byte_perm(w[2][c], w[3][c], 0x5140);
              const uint32_t ab1 = __byte_perm(w[0][c], w[1][c], 0x7362), cd1 = __byte_perm(w[2][c], w[3][c], 0x7362);
#pragma unroll
              for (int i = 0; i < NI; ++i) {
                const uint32_t ab = i < 2 ? ab0 : ab1, cd = i < 2 ? cd0 : cd1;
                const uint32_t b0 = (i & 1) ? codes_to_half2<0x4342>(ab) : codes_to_half2<0x4140>(ab);
                const uint32_t b1 = (i & 1) ? codes_to_half2<0x4342>(cd) : codes_to_half2<0x4140>(cd);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int p = 0; p < NQ; ++p) mma16816(o[mt][4 * c + i], pf[mt][x][p], b0, b1);
              }
            }
          }
        }
      }

      __syncwarp();                      // every lane has read the stage
      if (j + S < count) issue(j + S, stage);
      stage = stage + 1 == S ? 0 : stage + 1;
    }

    // ---- join the warps: each leaves its normalised output in its ring
    float* mine = (float*)ring;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float sum, odd;
        unpack2(l[mt][hf], sum, odd);
        sum += odd;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const int r = mt * 16 + hf * 8 + g;
        if (t == 0) ml[warp][r] = make_float2(from[mt][hf] == kUnseen ? -INFINITY : -from[mt][hf], sum);
        // NaN sums stay NaN; a row that saw no key gives 0
        const float by = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
        float out[E];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          out[i] = o[mt][i][2 * hf] * by * vref;
          out[NT + i] = o[mt][i][2 * hf + 1] * by * vref;
        }
#pragma unroll
        for (int d = 0; d < E; d += 4)
          *reinterpret_cast<float4*>(mine + r * DH + E * t + d) =
              make_float4(out[d], out[d + 1], out[d + 2], out[d + 3]);
      }
    }
    sync();

    const int first = (int)div_by(sg.pair_pos, sg.share);
    const int last = (int)div_by(sg.pair_pos + sg.w_pair - 1, sg.share);
    const int out_rows = sg.rows;
    const int64_t q_first = sg.q0;
    const bool whole = first == last;
    float* part = part_of<R, DH>(a, worker, first);
    auto store = [&](int r, int d, float4 v, float top, float sum) {
      const int rr = sg.r_base + r, qi = query_of(a, rr);
      store_out<T, DH>(a, (q_first + qi) * a.Hq + h * a.G + rr - qi * a.G, d, v, top, sum);
    };
    for (int i = gt; i < out_rows * (DH / 4); i += NW * 32) {
      const int r = i / (DH / 4), d = i % (DH / 4) * 4;
      float2 x[NW];
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        x[w] = ml[group * NW + w][r];
        top = fmaxf(top, x[w].x);
      }
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        x[w].y *= ex2(x[w].x - (top == -INFINITY ? 0.0f : top));
        sum += x[w].y;
      }
      const float by = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 y = *reinterpret_cast<const float4*>((float*)(smem + (group * NW + w) * Tile<DH>::kRing) + r * DH + d);
        const float k = x[w].y * by;
        v.x = fmaf(k, y.x, v.x), v.y = fmaf(k, y.y, v.y), v.z = fmaf(k, y.z, v.z), v.w = fmaf(k, y.w, v.w);
      }
      if (whole) {
        store(r, d, v, top, sum);
      } else {
        *reinterpret_cast<float4*>(part + r * DH + d) = v;
        if (d == 0) *reinterpret_cast<float2*>(part + R * DH + 2 * r) = make_float2(top, sum);
      }
    }
    if (!whole) {
      // the last block to arrive joins the pair's parts in the blocks' order
      __threadfence();
      sync();
      int before_me = 0;
      if (gt == 0) before_me = atomicAdd(a.tickets + first, 1);
      if (NW == 1) {
        before_me = __shfl_sync(0xffffffffu, before_me, 0);
      } else {
        if (gt == 0) arrived = before_me;
        __syncthreads();
        before_me = arrived;
      }
      if (before_me == last - first) {
        if (gt == 0) a.tickets[first] = 0;
        __threadfence();
        join_parts<R, DH>(a, first, last, gt, NW * 32, out_rows, store);
      }
    }
    fence_proxy_async_smem();            // the ring's next writes are TMA's
    sync();
    if (lane == 0) sg.pos = sg.seg_end;
    __syncwarp();
  }
  drain_after_timeout(&abort_flag);
}

// ------------------------------------------------------------------- host

size_t part_floats(int R, int DH) { return (size_t)R * DH + 2 * R; }

// Query rows of a pair: 32 where a warp's registers hold two row tiles.
int pair_rows(const lime_kv_dims& D, int64_t rows_per_head) {
  return D.dtype == LIME_BF16 && D.dh <= 64 && rows_per_head > 16 ? 32 : 16;
}

template <typename T, int DH, int MT, bool ONE, int NW>
int launch(Args a, CUtensorMap mk, CUtensorMap mv, int64_t* prefix, cudaStream_t st) {
  auto kernel = k_kv_attn<T, DH, MT, ONE, NW>;
  const size_t smem = kWarps * Tile<DH>::kRing + 1024;
  static int per_sm[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LIME_ERR_CUDA;
  if (dev < 0 || dev >= 64) dev = 0;
  if (!per_sm[dev]) {
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kWarps * 32, smem) != cudaSuccess ||
        n < 1)
      return LIME_ERR_CUDA;
    per_sm[dev] = n;
  }
  int grid = num_sms() * per_sm[dev];
  if (grid > kMaxWorkers / kWarps) grid = kMaxWorkers / kWarps;
  if (a.B > kInlineRequests) {
    a.prefix = prefix;
    const Cut cut = {a.Hkv, 16 * MT, Tile<DH>::TK, kPairCost<NW>, kLeast<NW>};
    if (const int rc = launch_plan(a, cut, prefix, st)) return rc;
  }
  return launch_pdl(kernel, dim3(grid), dim3(kWarps * 32), smem, st, 1, mk, mv, a);
}

}  // namespace

namespace kv {
int launch_plan(const Args& a, const Cut& cut, int64_t* prefix, cudaStream_t st) {
  return launch_pdl(k_kv_plan, dim3(1), dim3(1024), 0, st, 1, a.B, a.off, a.total_q, a.lens, a.G,
                    (int64_t)a.max_blocks << a.log_block, cut, prefix, a.status);
}
}  // namespace kv

size_t kv_ticket_bytes() { return kMaxWorkers * sizeof(int); }

size_t kv_attention_ws_bytes(const lime_kv_dims& D, int64_t B, int64_t total_q) {
  if (total_q == 0) return 0;
  const size_t prefix = B > kInlineRequests ? ((size_t)(B + 2) * 8 + 255) / 256 * 256 : 0;
  return prefix + 2 * kMaxWorkers * part_floats(D.dh <= 64 ? 32 : 16, D.dh) * sizeof(float);
}

int kv_attention(const lime_kv_dims& D, int64_t B, const void* Q, int64_t ldq, const int64_t* off,
                 int64_t total_q, const int32_t* table, const int32_t* lens, const int8_t* kc,
                 const int8_t* vc, const float* scale, float sm_scale, bool causal, void* O,
                 float* lse, void* ws, int* tickets, unsigned* status, cudaStream_t st) {
  const int G = D.Hq / D.Hkv;
  const int R = pair_rows(D, ceil_div(total_q, B) * G);
  const int TK = D.dh == 128 ? 32 : 64;
  int64_t* prefix = (int64_t*)ws;
  const size_t prefix_bytes = B > kInlineRequests ? ((size_t)(B + 2) * 8 + 255) / 256 * 256 : 0;

  Args a = {};
  a.Q = Q, a.ldq = ldq, a.off = off, a.table = table, a.lens = lens;
  a.scale = (const float2*)scale;
  a.tickets = tickets, a.part = (float*)((char*)ws + prefix_bytes);
  a.O = O, a.lse = lse, a.status = status;
  a.B = B, a.total_q = total_q, a.n_blocks = D.n_blocks;
  a.Hq = D.Hq, a.Hkv = D.Hkv, a.G = G, a.max_blocks = D.max_blocks;
  a.log_block = 4;
  while (1 << a.log_block < D.block) ++a.log_block;
  a.log_g = (G & (G - 1)) ? -1 : 0;
  while (a.log_g >= 0 && 1 << a.log_g < G) ++a.log_g;
  a.scale_log2 = fabsf(sm_scale) * 1.4426950408889634f, a.negative = sm_scale < 0.0f, a.causal = causal;
  CUtensorMap mk, mv;
  const int box = D.block < TK ? D.block : TK;
  if (!make_tmap_kv(&mk, kc, D.block * D.dh, D.n_blocks * D.Hkv, box * D.dh) ||
      !make_tmap_kv(&mv, vc, D.block * D.dh, D.n_blocks * D.Hkv, box * D.dh))
    return LIME_ERR_CUDA;
  // Workers of one warp where all requests' query rows, packed together, fill a pair
  // for each of 8 warps an SM (what it holds of the kernels with 32 rows to a pair):
  // their segments are longer, and one warp's start and end run beside the others'
  // tiles.  Four warps / one, in us: 32 links, 4 heads of 32, up to 1,024 rows: 160
  // requests 33 / 38, 296 (the border) 48 / 47, 512 75 / 60.  Single tokens, 32 heads
  // on 8, dh 128, where requests do not fill their tiles and the border lies at 592:
  // up to 16,384 rows, 256 requests 628 / 706, 600 1,659 / 1,713, 1,200 3,456 / 3,420;
  // up to 2,048 rows, 64 requests 49 / 47, 560 272 / 223, 600 289 / 238.
  const int64_t packed = ceil_div(total_q * G, R) * D.Hkv;
  const bool own = packed >= (int64_t)num_sms() * 2 * kWarps;
#define RUN2(T, DH, MT, ONE)                                        \
  return own ? launch<T, DH, MT, ONE, 1>(a, mk, mv, prefix, st)     \
             : launch<T, DH, MT, ONE, kWarps>(a, mk, mv, prefix, st)
#define RUN(T, DH, MT)                        \
  do {                                        \
    if (D.block >= Tile<DH>::SK) RUN2(T, DH, MT, true); \
    RUN2(T, DH, MT, false);                   \
  } while (0)
  if (D.dtype == LIME_BF16) {
    if (D.dh == 16) { if (R == 32) RUN(bf16, 16, 2); RUN(bf16, 16, 1); }
    if (D.dh == 32) { if (R == 32) RUN(bf16, 32, 2); RUN(bf16, 32, 1); }
    if (D.dh == 64) { if (R == 32) RUN(bf16, 64, 2); RUN(bf16, 64, 1); }
    RUN(bf16, 128, 1);
  }
  if (D.dh == 16) RUN(float, 16, 1);
  if (D.dh == 32) RUN(float, 32, 1);
  if (D.dh == 64) RUN(float, 64, 1);
  RUN(float, 128, 1);
#undef RUN2
#undef RUN
}

}  // namespace lime
