// Quantising append of the paged history cache: new key and value rows become
// int8 codes under one scale per (block, head).
//
// A unit is one group of new rows (consecutive slots of a block) in one head,
// keys or values: read once into registers, its largest magnitude found, its
// codes written.  A team of TW warps holds a unit, 16-byte loads, at most
// kVecs of them per lane in flight.  633,000 bf16 rows of 4 x 32 keys and values
// take 115 us, 65 % of the copy bandwidth for 2 + 1 bytes a value: a warp loads,
// reduces, codes and stores one unit after another, and waits for loads most.
#include <math.h>

#include "lime_kv.cuh"
#include "sm100.cuh"

namespace lime {

using namespace sm100;

namespace {

constexpr float kMax = 3.402823466e38f;

// 16-byte loads of a lane that hold its part of a unit.
template <typename T> constexpr int kVecs = sizeof(T) == 2 ? 8 : 16;

// Warps that hold bs rows of DH values.
template <typename T, int DH>
__host__ __device__ constexpr int team_warps(int bs) {
  const int vec = 16 / (int)sizeof(T), rows = 32 * vec / DH * kVecs<T>;
  return bs <= rows ? 1 : bs / rows;
}

__device__ __forceinline__ void unpack(const uint4& v, float* x, bf16) { unpack8(v, x); }
__device__ __forceinline__ void unpack(const uint4& v, float* x, float) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Running largest magnitude; NaN once one has been seen.
template <typename T> struct AbsMax;
template <> struct AbsMax<bf16> {
  __nv_bfloat162 m = __float2bfloat162_rn(0.0f);
  __device__ __forceinline__ void add(const uint4& v) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2_nan(m, __habs2(p[i]));
  }
  __device__ __forceinline__ float get() const {
    return max_nan(__low2float(m), __high2float(m));
  }
};
template <> struct AbsMax<float> {
  float m = 0.0f;
  __device__ __forceinline__ void add(const uint4& v) {
    m = max_nan(m, max_nan(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y))));
    m = max_nan(m, max_nan(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w))));
  }
  __device__ __forceinline__ float get() const { return m; }
};

// rint(x / s) in 64 bits: exact, since the quotient of two fp32 values lies
// on a half-way point only if it is one.  NaN gives 0.
__device__ __forceinline__ int code_of(float x, float s) {
  if (x != x || s == 0.0f) return 0;
  const double r = rint((double)x / (double)s);
  return (int)(r > 127.0 ? 127.0 : (r < -127.0 ? -127.0 : r));
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
  return (uint64_t)__float_as_uint(a) | (uint64_t)__float_as_uint(b) << 32;
}
__device__ __forceinline__ float lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// N values to N codes (packed four to a word).  x * (1 / s) rounds to the right
// code unless x / s is next to a half-way point: with r that code, x - r s is
// exact in fp32 (a multiple of the unit of s, at most s), so |x - r s| against
// s / 2 decides between r and its neighbours.  Half the largest value, which
// bf16 rows often hold, sits there: the branch is short.
template <int N>
__device__ __forceinline__ void to_codes(const float* x, float s, float inv, bool plain, uint32_t* w) {
  float t[N], worst = 0.0f;
  const float magic = 12582912.0f;  // 1.5 * 2^23: the integer lands in the low bits
  // two values to an instruction
  const uint64_t inv2 = pair(inv, inv), magic2 = pair(magic, magic), s2 = pair(s, s);
  const uint64_t minus2 = pair(-1.0f, -1.0f);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t x2 = pair(x[i], x[i + 1]), t2 = fma2(x2, inv2, magic2);
    const uint64_t e2 = fma2(fma2(t2, minus2, magic2), s2, x2);
    t[i] = lo(t2), t[i + 1] = hi(t2);
    worst = fmaxf(worst, fmaxf(fabsf(lo(e2)), fabsf(hi(e2))));
  }
  uint32_t c[N];
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = __float_as_uint(t[i]);
  const float half = 0.5f * s;
  if (!plain) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = (uint32_t)code_of(x[i], s);
  } else if (worst >= half) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float e = fmaf(magic - t[i], s, x[i]);
      const bool odd = c[i] & 1u;
      c[i] += (e > half || (e == half && odd)) ? 1u : 0u;
      c[i] -= (e < -half || (e == -half && odd)) ? 1u : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < N; i += 4)
    w[i / 4] = __byte_perm(__byte_perm(c[i], c[i + 1], 0x0040), __byte_perm(c[i + 2], c[i + 3], 0x0040), 0x5410);
}

// Threads of a block: four warps, or one team where that is more.  An SM takes
// 24 warps of 80 registers (bf16) or 16 of 128 (fp32).
__host__ __device__ constexpr int block_threads(int TW) { return TW > 4 ? TW * 32 : 128; }

template <typename T, int DH, int TW>
__global__ void __launch_bounds__(block_threads(TW), (sizeof(T) == 2 ? 768 : 512) / block_threads(TW))
    k_append(int Hkv, int log_bs, int64_t n_slots, const T* K, int64_t ldk, const T* V, int64_t ldv,
             int64_t total, int tile, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
             unsigned* status) {
  constexpr int kThreads = block_threads(TW);
  constexpr int VEC = 16 / sizeof(T), LR = DH / VEC, RPL = 32 / LR, NV = kVecs<T>;
  constexpr int kTeams = kThreads / 32 / TW;
  const int bs = 1 << log_bs;
  extern __shared__ int64_t sl[];                  // slots of the tile, one before and bs behind
  __shared__ int n_runs;
  __shared__ float team_max[kThreads / 32];
  int* runs = (int*)(sl + tile + bs + 1);          // first rows of the tile's groups

  // blocks of the same rows run side by side: together they read whole rows
  const int unit = (int)(blockIdx.x % (2 * Hkv)), side = unit & 1, h = unit >> 1;
  const int64_t t0 = (int64_t)(blockIdx.x / (2 * Hkv)) * tile;
  if (threadIdx.x == 0) n_runs = 0;
  for (int i = threadIdx.x; i < tile + bs + 1; i += kThreads) {
    const int64_t t = t0 - 1 + i;
    sl[i] = t >= 0 && t < total ? slots[t] : -1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < tile; i += kThreads) {
    if (t0 + i >= total) break;
    const int64_t s = sl[i + 1];
    if (s < 0 || s >= n_slots) {
      if (s != -1) raise_flag(status, LIME_FLAG_BAD_BLOCK);
    } else if ((s & (bs - 1)) == 0 || sl[i] != s - 1) {
      runs[atomicAdd(&n_runs, 1)] = i;             // units are independent: any order
    }
  }
  __syncthreads();

  const T* X = side ? V : K;
  const int64_t ld = side ? ldv : ldk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int team = warp / TW, tw = warp % TW;
  for (int k = team; k < n_runs; k += kTeams) {
    const int i0 = runs[k];
    const int64_t slot = sl[i0 + 1];
    const int row = (int)(slot & (bs - 1));
    int n = 1;                                     // rows of the group
    for (; row + n < bs; n += 32) {
      const int i = n + lane;
      const bool ok = row + i < bs && sl[i0 + 1 + i] == slot + i;
      const unsigned b = __ballot_sync(0xffffffffu, ok);
      if (b != 0xffffffffu) {
        n += __ffs(~b) - 1;
        break;
      }
    }
    if (n > bs - row) n = bs - row;
    const int64_t cell = (slot >> log_bs) * Hkv + h;
    int8_t* codes = (side ? vc : kc) + (cell << log_bs) * DH;

    uint4 v[NV];
    const int r0 = tw * RPL + lane / LR;
    const T* src = X + (t0 + i0 + r0) * ld + (int64_t)h * DH + lane % LR * VEC;
#pragma unroll
    for (int j = 0; j < NV; ++j, src += TW * RPL * ld)
      v[j] = j * TW * RPL + r0 < n ? __ldcs(reinterpret_cast<const uint4*>(src))
                                   : make_uint4(0, 0, 0, 0);
    float had = row ? scale[cell * 2 + side] : 0.0f;
    if (!(had >= 0.0f && had <= kMax)) had = 0.0f;
    AbsMax<T> most;
#pragma unroll
    for (int j = 0; j < NV; ++j) most.add(v[j]);
    float a = most.get();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    bool odd = !(a <= kMax);
    if (odd) {                                     // NaN or infinite: the finite values' maximum
      raise_flag(status, LIME_FLAG_NONFINITE);
      a = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[VEC];
        unpack(v[j], x, T());
#pragma unroll
        for (int d = 0; d < VEC; ++d)
          if (fabsf(x[d]) <= kMax) a = fmaxf(a, fabsf(x[d]));
      }
      a = warp_max(a);
    }
    if constexpr (TW > 1) {
      if (lane == 0) team_max[warp] = a;
      named_bar_sync(1 + team, TW * 32);
#pragma unroll
      for (int w = 0; w < TW; ++w) a = fmaxf(a, team_max[team * TW + w]);
      named_bar_sync(1 + team, TW * 32);           // every warp has read both
    }
    const float s = fmaxf(had, __fdiv_rn(a, 127.0f));
    if (s > had)
      for (int i = tw * 32 + lane; i < row * DH; i += TW * 32)
        codes[i] = (int8_t)rint((double)codes[i] * (double)had / (double)s);
    if ((s > had || row == 0) && tw == 0 && lane == 0) scale[cell * 2 + side] = s;
    // 1 / s and the test by s / 2 want a scale well inside fp32's range
    const bool plain = !odd && s > 1e-30f && s < 1e36f;
    const float inv = plain ? __frcp_rn(s) : 0.0f;
    int8_t* to = codes + (row + r0) * DH + lane % LR * VEC;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (j * TW * RPL + r0 < n) {
        float x[VEC];
        uint32_t w[VEC / 4];
        unpack(v[j], x, T());
        to_codes<VEC>(x, s, inv, plain, w);
        int8_t* dst = to + j * TW * RPL * DH;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = w[0];
      }
    }
  }
}

template <typename T, int DH, int TW>
int launch(const lime_kv_dims& D, const void* K, int64_t ldk, const void* V, int64_t ldv,
           int64_t total, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
           unsigned* status, cudaStream_t st) {
  // Rows of a thread block: so many that its teams have a full block's group
  // each where there are enough rows to fill the GPU, fewer where not (every
  // row may be a group of its own).
  const int sides = 2 * D.Hkv, sms = num_sms(), threads = block_threads(TW);
  int tile = 8, log_bs = 4;
  while (1 << log_bs < D.block) ++log_bs;
  while (tile < threads / 32 / TW * 2 * D.block && tile * 2 * (int64_t)sms * 8 <= total * sides) tile *= 2;
  const size_t smem = (size_t)(tile + D.block + 1) * 8 + (size_t)tile * 4;
  k_append<T, DH, TW><<<(unsigned)(ceil_div(total, tile) * sides), threads, smem, st>>>(
      D.Hkv, log_bs, D.n_blocks * D.block, (const T*)K, ldk, (const T*)V, ldv, total, tile, slots,
      kc, vc, scale, status);
  note_launches(1);
  return LIME_OK;
}

template <typename T, int DH>
int launch_team(const lime_kv_dims& D, const void* K, int64_t ldk, const void* V, int64_t ldv,
                int64_t total, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
                unsigned* status, cudaStream_t st) {
  const int tw = team_warps<T, DH>(D.block);
#define RUN(TW)            \
  if (tw == TW)            \
  return launch<T, DH, TW>(D, K, ldk, V, ldv, total, slots, kc, vc, scale, status, st)
  if constexpr (team_warps<T, DH>(128) >= 8) RUN(8);
  if constexpr (team_warps<T, DH>(128) >= 4) RUN(4);
  if constexpr (team_warps<T, DH>(128) >= 2) RUN(2);
#undef RUN
  return launch<T, DH, 1>(D, K, ldk, V, ldv, total, slots, kc, vc, scale, status, st);
}

}  // namespace

int kv_append(const lime_kv_dims& D, const void* K, int64_t ldk, const void* V, int64_t ldv,
              int64_t total, const int64_t* slots, int8_t* kc, int8_t* vc, float* scale,
              unsigned* status, cudaStream_t st) {
#define RUN(T, DH) \
  return launch_team<T, DH>(D, K, ldk, V, ldv, total, slots, kc, vc, scale, status, st)
  if (D.dtype == LIME_BF16) {
    if (D.dh == 16) RUN(bf16, 16);
    if (D.dh == 32) RUN(bf16, 32);
    if (D.dh == 64) RUN(bf16, 64);
    RUN(bf16, 128);
  }
  if (D.dh == 16) RUN(float, 16);
  if (D.dh == 32) RUN(float, 32);
  if (D.dh == 64) RUN(float, 64);
  RUN(float, 128);
#undef RUN
}

}  // namespace lime
