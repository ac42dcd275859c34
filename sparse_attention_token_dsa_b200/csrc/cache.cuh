// cache.cuh — rotary positions, and the paged cache of a DSA layer: rows written
// (quantised) into pages and read back.
//
// Rotary positions: the pair (x_a, x_b) number i of a token at position p becomes
//     y_a = m (x_a cos t - x_b sin t),  y_b = m (x_b cos t + x_a sin t),  t = p f_i,
// with a factor m (1 unless positions are scaled) and a table f of frequencies in
// radians a position.  The transpose, which is also the gradient, turns by -t.
// The angle of a far position has no digits left in 32 bits, so turns = p (f / 2 pi)
// is formed in 64 bits and its whole part is dropped.  The remaining fraction goes to
// sincospif rounded to 32 bits, and for results in 32 bits what the rounding took turns them
// once more to first order: without that the angle's error is as large as the function's own
// (largest error of a cosine 1.9 steps of 2^-24, with it 1.25).  Results in fewer bits do
// without it (8192 x 64 heads of bf16 values 46 us for 47).
//
// The paged cache holds a row's first dim_q values as e4m3 codes in groups of 128 with
// one fp32 scale a group, and its last dim_raw values as bf16, in three planes
// [page][row][..] (a page's rows lie together in each plane, so a group of 128 codes is
// one aligned 128-byte run and the bf16 part can be an operand of a TMA copy).
//
// All three are bound by memory: they read a row once, write it once and hold it in
// registers between.
#pragma once
#include "operand.cuh"

namespace dsa {

// ------------------------------------------------------------- conversions --
template <typename T>
struct RowType;
template <>
struct RowType<float> {
  static constexpr int kVec = 4;      // values in 16 bytes
  __device__ static float get(const float* p) { return *p; }
  __device__ static void put(float* p, float v) { *p = v; }
  __device__ static void unpack(const uint4& u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x);
    v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z);
    v[3] = __uint_as_float(u.w);
  }
  __device__ static uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

template <>
struct RowType<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ static void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  __device__ static void unpack(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static uint4 pack(const float (&v)[8]) {
    return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                      bf16x2(v[6], v[7]));
  }
};

// cos and sin of position * freq.
template <bool WHOLE = false>
__device__ __forceinline__ float2 turn_of(int32_t position, double freq) {
  const double turns = (double)position * (freq * 0.15915494309189533577);   // 1 / (2 pi)
  const double part = turns - rint(turns);                                   // [-1/2, 1/2]
  const float near = (float)part;
  float s, c;
  sincospif(2.f * near, &s, &c);
  if constexpr (!WHOLE) return make_float2(c, s);
  const float rest = (float)(part - near) * 6.2831853f;                      // in radians
  return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// -------------------------------------------------------- rotary positions --
struct RopeArgs {
  const void* x;
  void* out;
  const int32_t* pos;      // [n_tokens]
  const double* freq;      // [rot / 2]
  int64_t n_tokens;
  int64_t x_ts, x_hs, o_ts, o_hs;   // token and head strides (elements)
  int32_t heads, offset, rot;
  int32_t pairs;           // pair units of a head (see below)
  int32_t units;           // pair and copy units of a head
  uint32_t per_unit;       // 2^32 / units, rounded up; 0 where that is not exact
  int32_t tpb;             // tokens of a block
  int32_t span;            // units that one block of a token takes (blockIdx.y of them)
  float mscale;
  float sign;              // +1, or -1 for the transpose
};

constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 3;    // units a thread holds at once

// The work of a head is cut into units of one 16-byte vector: in the half layout a
// pair unit is one vector of the first half and its partner in the second, in the
// interleaved layout one vector holding whole pairs; the values outside the rotated
// part are copy units (none when the call is in place).  A thread issues the loads of
// three units before it uses any, and the block forms the cosines and sines of its
// tokens (once for all heads) while they are in flight.  Rows that are not aligned to
// 16 bytes take the same path one pair at a time (VEC = false).
// Measured (B200, copy 6545 GB/s; here and below replays of a graph over three inputs in turn):
// 8192 tokens x 64 heads x 128 bf16 values, 64 of them rotated in halves, 46 us, 5.8 TB/s; 2049
// tokens x 64 heads x 576 fp32 values, interleaved, 94 us, 6.4 TB/s.  Four units and 4 blocks an
// SM took 51 and 96 us, two and 6 54 and 99.  At 5 blocks the half layouts spill 24 and 32 bytes
// a thread; at 4, with nothing spilled, the two took 47 and 104 us.
template <typename T, bool VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_kernel(const RopeArgs a) {
  using R = RowType<T>;
  constexpr int N = VEC ? R::kVec : 1;
  // m cos, m sin of the tokens' angles, [tpb][rot / 2]; vectors take them two pairs at a
  // time, [tpb][two of a unit][unit], so lanes beside one another read places beside one
  // another
  constexpr int P = VEC ? (INTER ? N / 2 : N) : 1;   // pairs of a unit
  extern __shared__ __align__(16) float2 turns[];
  const int64_t t0 = (int64_t)blockIdx.x * a.tpb;
  const int nt = (int)(a.n_tokens - t0 < a.tpb ? a.n_tokens - t0 : a.tpb);
  const int half = a.rot >> 1;
  const uint32_t per_token = (uint32_t)a.heads * a.units;
  const uint32_t first = blockIdx.y * (uint32_t)a.span;
  uint32_t last = a.tpb > 1 ? per_token * nt : first + a.span;
  if (a.tpb == 1 && last > per_token) last = per_token;
  const T* x = reinterpret_cast<const T*>(a.x);
  T* out = reinterpret_cast<T*>(a.out);
  bool ready = false;
  for (uint32_t base = first + threadIdx.x; base - threadIdx.x < last;
       base += kRopeBatch * kRopeThreads) {
    uint4 va[kRopeBatch], vb[kRopeBatch];
    float sa[kRopeBatch], sb[kRopeBatch];
    int64_t oa[kRopeBatch];
    int tab[kRopeBatch];                             // place in `turns`; -1: a copy unit
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const uint32_t i = base + k * kRopeThreads;
      if (i >= last) continue;
      const uint32_t tl = a.tpb > 1 ? i / per_token : 0;
      const uint32_t r = i - tl * per_token;
      const uint32_t h = a.per_unit ? __umulhi(r, a.per_unit) : r / (uint32_t)a.units;
      const int u = (int)(r - h * a.units);
      int d;
      if (u < a.pairs) {
        d = a.offset + (INTER ? 2 * P : P) * u;
        tab[k] = (int)tl * half + (VEC ? 2 : 1) * u;
      } else {
        d = (u - a.pairs) * N;
        if (d >= a.offset) d += a.rot;
        tab[k] = -1;
      }
      const T* px = x + (t0 + tl) * a.x_ts + (int64_t)h * a.x_hs + d;
      oa[k] = (t0 + tl) * a.o_ts + (int64_t)h * a.o_hs + d;
      const int part = INTER ? 1 : half;             // distance of the partner
      if constexpr (VEC) {
        va[k] = __ldcs(reinterpret_cast<const uint4*>(px));
        if (!INTER && tab[k] >= 0) vb[k] = __ldcs(reinterpret_cast<const uint4*>(px + half));
      } else {
        sa[k] = R::get(px);
        if (tab[k] >= 0) sb[k] = R::get(px + part);
      }
    }
    if (!ready) {
      for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
        const int tl = i / half, pair = i - tl * half;
        const float2 cs = turn_of<sizeof(T) == 4>(a.pos[t0 + tl], a.freq[pair]);
        const int at = VEC ? (pair % P / 2 * a.pairs + pair / P) * 2 + (pair & 1) : pair;
        turns[tl * half + at] = make_float2(cs.x * a.mscale, cs.y * a.mscale * a.sign);
      }
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int k = 0; k < kRopeBatch; ++k) {
      const uint32_t i = base + k * kRopeThreads;
      if (i >= last) continue;
      T* po = out + oa[k];
      if (tab[k] < 0) {
        if constexpr (VEC)
          __stcs(reinterpret_cast<uint4*>(po), va[k]);
        else
          R::put(po, sa[k]);
      } else if constexpr (!VEC) {
        const float2 cs = turns[tab[k]];
        R::put(po, sa[k] * cs.x - sb[k] * cs.y);
        R::put(po + (INTER ? 1 : half), sb[k] * cs.x + sa[k] * cs.y);
      } else if constexpr (INTER) {
        float v[N];
        R::unpack(va[k], v);
#pragma unroll
        for (int j = 0; j < P; j += 2) {
          const float4 cs = *reinterpret_cast<const float4*>(turns + tab[k] + j * a.pairs);
          const float p = v[2 * j], q = v[2 * j + 1], r = v[2 * j + 2], s = v[2 * j + 3];
          v[2 * j] = p * cs.x - q * cs.y;
          v[2 * j + 1] = q * cs.x + p * cs.y;
          v[2 * j + 2] = r * cs.z - s * cs.w;
          v[2 * j + 3] = s * cs.z + r * cs.w;
        }
        __stcs(reinterpret_cast<uint4*>(po), R::pack(v));
      } else {
        float v[N], w[N];
        R::unpack(va[k], v);
        R::unpack(vb[k], w);
#pragma unroll
        for (int j = 0; j < P; j += 2) {
          const float4 cs = *reinterpret_cast<const float4*>(turns + tab[k] + j * a.pairs);
          const float p = v[j], q = w[j], r = v[j + 1], s = w[j + 1];
          v[j] = p * cs.x - q * cs.y;
          w[j] = q * cs.x + p * cs.y;
          v[j + 1] = r * cs.z - s * cs.w;
          w[j + 1] = s * cs.z + r * cs.w;
        }
        __stcs(reinterpret_cast<uint4*>(po), R::pack(v));
        __stcs(reinterpret_cast<uint4*>(po + half), R::pack(w));
      }
    }
  }
}

// -------------------------------------------------------------- paged cache --
struct CachePlanes {
  uint8_t* codes;          // [page][row][dim_q]
  float* scale;            // [page][row][dim_q / 128]
  __nv_bfloat16* raw;      // [page][row][dim_raw]
  int64_t codes_ps, scale_ps, raw_ps;   // page strides (elements)
  int32_t n_pages, page_shift, dim_q, dim_raw;
};

constexpr int kCacheThreads = 256;
constexpr int kCacheUnits = kCacheThreads / 8;   // 8 lanes take a row, in chunks of 128 values
constexpr int kCacheBatch = 4;                   // chunks a lane holds at once
constexpr int kReadBatch = 5;                    // where it reads values

struct CacheWriteArgs {
  CachePlanes c;
  const void* x;           // rows of dim_q + dim_raw values, x_ts apart
  int64_t x_ts;
  const int64_t* slots;    // [n_tokens] page * page_size + row; outside the cache: not written
  int64_t n_tokens;
  const int32_t* pos;      // rotation of [offset, offset + rot) (null: none)
  const double* freq;
  int32_t offset, rot, inter;
  float mscale;
  float sign;              // +1, or -1 for the transpose
  int32_t items;           // chunks of a row
  int32_t pow2;            // scale: least power of two >= amax / 448 (else amax / 448)
};

// 8 consecutive values of a row as they were loaded.
template <typename T, bool VEC>
struct Run8 {
  using R = RowType<T>;
  static constexpr int kWords = 8 / R::kVec;
  uint4 word[VEC ? kWords : 1];
  float value[VEC ? 1 : 8];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) word[i] = *reinterpret_cast<const uint4*>(p + i * R::kVec);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) value[j] = R::get(p + j);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        float u[R::kVec];
        R::unpack(word[i], u);
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) v[i * R::kVec + j] = u[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = value[j];
    }
  }
};

// Rotates the 8 values of a row that start at d (a multiple of 8) where they lie in the
// rotated part (in the half layout with their partners, read here).
template <typename T, bool VEC>
__device__ __forceinline__ void turn8(const CacheWriteArgs& a, const T* row, int64_t token, int d,
                                      float (&v)[8]) {
  if (d < a.offset || d >= a.offset + a.rot) return;
  const int r = d - a.offset, half = a.rot >> 1;
  const int32_t p = a.pos[token];
  if (a.inter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 cs = turn_of(p, a.freq[(r >> 1) + j]);
      cs.x *= a.mscale;
      cs.y *= a.mscale * a.sign;
      const float x0 = v[2 * j], x1 = v[2 * j + 1];
      v[2 * j] = x0 * cs.x - x1 * cs.y;
      v[2 * j + 1] = x1 * cs.x + x0 * cs.y;
    }
  } else {
    const bool low = r < half;
    Run8<T, VEC> mate;
    mate.load(row + (low ? d + half : d - half));
    float w[8];
    mate.get(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 cs = turn_of(p, a.freq[(low ? r : r - half) + j]);
      cs.x *= a.mscale;
      cs.y *= (low ? -a.mscale : a.mscale) * a.sign;
      v[j] = v[j] * cs.x + w[j] * cs.y;
    }
  }
}

// Codes of 8 values: f turns a value into its quotient by the scale.
template <typename F>
__device__ __forceinline__ uint2 codes8(const float (&v)[8], F f) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f(v[4 * h]), f(v[4 * h + 1])),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f(v[4 * h + 2]), f(v[4 * h + 3])),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[h] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Scale of a group and its codes: two runs of 8 values a lane.
__device__ __forceinline__ float quantise(const float (&v)[2][8], float amax, bool pow2,
                                          uint2 (&code)[2]) {
  if (pow2) {
    // amax = m 2^e with m in [1/2, 1), 448 = 0.875 2^9
    int e;
    const float m = frexpf(amax, &e);
    e = amax > 3.0e38f ? 120 : max(m > 0.875f ? e - 8 : e - 9, -126);
    float s = 1.f, inv = 1.f;
    if (amax > 0.f) {
      s = __int_as_float((e + 127) << 23);
      inv = __int_as_float((127 - e) << 23);         // 2^-e
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) code[h] = codes8(v[h], [&](float x) { return x * inv; });
    return s;
  }
  const float s = e4m3_scale(amax);
  if (s > 0x1p-90f && s < 0x1p90f) {
    // The IEEE quotient by Markstein's method: from the correctly rounded reciprocal y,
    // q = x y, its exact remainder r = x - q s, and q + r y rounds to x / s.  (Where x is so
    // small that r is not exact, q is far below the smallest code.)
    const float y = __frcp_rn(s);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      code[h] = codes8(v[h], [&](float x) {
        const float q = x * y;
        return fmaf(fmaf(-q, s, x), y, q);
      });
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) code[h] = codes8(v[h], [&](float x) { return __fdiv_rn(x, s); });
  }
  return s;
}

// 8 lanes take four chunks of 128 values of a row (blockIdx.y: which four), or, where rows
// have less than four chunks, one chunk of each of two rows (of four took registers that
// cost more threads), and hold them at once, two runs of 8 values a lane, 64 apart, so each
// access of the 8 lanes is one contiguous run; a group's largest magnitude is a three-step exchange between them and
// nothing is reread.  A scale that is a power of two makes code * scale exact in bf16, so
// attention on the tensor cores reads the quantised values without a second rounding;
// e4m3 being a floating format, it costs at most one binade at the bottom of its range.
// Measured (B200): 131072 keys of 128 values 11.5 us, 4.5 TB/s, and 524288 of them 36 us, 5.7
// TB/s (the same 131072 again and again 10.3; with the values waiting for the slots 12.3, and
// one row at a time 14.4); 8191 latent rows of 512 + 64 values, the 64 rotated, 5.3 us and 32
// of them 3.1: launch and latency.
template <typename T, bool VEC, bool TURN, int ROWS>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int BATCH = ROWS > 1 ? ROWS : kCacheBatch, CHUNKS = BATCH / ROWS;
  const int l = threadIdx.x & 7, q_chunks = a.c.dim_q >> 7, width = a.c.dim_q + a.c.dim_raw;
  const uint32_t mates = 0xffu << (threadIdx.x & 24);
  // (tokens and pages fit 32 bits; their places do not)
  const uint32_t token0 = blockIdx.x * (uint32_t)(ROWS * kCacheUnits) + (threadIdx.x >> 3);
  const int c0 = blockIdx.y * CHUNKS;
  auto x_at = [&](int r) {
    return reinterpret_cast<const T*>(a.x) + (int64_t)(token0 + r * kCacheUnits) * a.x_ts;
  };
  int64_t slot[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const uint32_t token = token0 + r * kCacheUnits;
    slot[r] = token < a.n_tokens ? a.slots[token] : -1;
  }
  // the values do not wait for the slots (a token that is skipped is read for nothing)
  Run8<T, VEC> held[BATCH][2];
#pragma unroll
  for (int k = 0; k < BATCH; ++k)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = (c0 + k % CHUNKS) * 128 + h * 64 + l * 8;
      if (token0 + k / CHUNKS * kCacheUnits < a.n_tokens && d < width)
        held[k][h].load(x_at(k / CHUNKS) + d);
    }
#pragma unroll
  for (int k = 0; k < BATCH; ++k) {
    const int r = k / CHUNKS, c = c0 + k % CHUNKS;
    const int64_t page = slot[r] >> a.c.page_shift;
    if (slot[r] < 0 || page >= a.c.n_pages || c >= a.items) continue;   // the same for the 8 lanes
    const int row = (int)slot[r] & ((1 << a.c.page_shift) - 1);
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      held[k][h].get(v[h]);
      if constexpr (TURN) {
        const int d = c * 128 + h * 64 + l * 8;
        if (d < width) turn8<T, VEC>(a, x_at(r), token0 + r * kCacheUnits, d, v[h]);
      }
    }
    if (c < q_chunks) {
      float amax = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[h][j]));
      amax = fmaxf(amax, __shfl_xor_sync(mates, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(mates, amax, 2));
      amax = fmaxf(amax, __shfl_xor_sync(mates, amax, 4));
      uint2 code[2];
      const float s = quantise(v, amax, a.pow2, code);
      uint8_t* dst = a.c.codes + page * a.c.codes_ps + (int64_t)row * a.c.dim_q + c * 128;
      *reinterpret_cast<uint2*>(dst + l * 8) = code[0];
      *reinterpret_cast<uint2*>(dst + 64 + l * 8) = code[1];
      if (l == 0) a.c.scale[page * a.c.scale_ps + row * q_chunks + c] = s;
    } else {
      __nv_bfloat16* dst = a.c.raw + page * a.c.raw_ps + (int64_t)row * a.c.dim_raw;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = (c - q_chunks) * 128 + h * 64 + l * 8;
        if (d < a.c.dim_raw)
          *reinterpret_cast<uint4*>(dst + d) = RowType<__nv_bfloat16>::pack(v[h]);
      }
    }
  }
}

struct CacheReadArgs {
  CachePlanes c;
  const int32_t* table;    // [batch][max_pages]
  const int32_t* k_len;    // [batch] or null
  int32_t batch, max_pages, n_k;
  void* out;               // [batch][n_k][dim_q + dim_raw], or codes [batch][n_k][dim_q]
  float* out_scale;        // [batch][n_k][dim_q / 128] (codes)
};

// Page of a sequence's row, or -1 for a table entry outside the cache.
__device__ __forceinline__ int32_t page_of(const int32_t* table, int32_t key, int shift,
                                           int32_t n_pages) {
  const int32_t p = table[key >> shift];
  return (uint32_t)p < (uint32_t)n_pages ? p : -1;
}

__device__ __forceinline__ void e4m3x4_values(uint32_t w, float s, float* v) {
  const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
  const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
  const float2 a = __half22float2(lo), b = __half22float2(hi);
  v[0] = a.x * s;
  v[1] = a.y * s;
  v[2] = b.x * s;
  v[3] = b.y * s;
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  using R = RowType<T>;
  if constexpr (R::kVec == 8) {
    *reinterpret_cast<uint4*>(p) = R::pack(v);
  } else {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    *reinterpret_cast<uint4*>(p) = R::pack(lo);
    *reinterpret_cast<uint4*>(p + 4) = R::pack(hi);
  }
}

// Rows of a sequence for 8 lanes: their pages, -1 behind the length (`out` stays as it
// was there), -2 for a table entry outside the cache (zeros).
template <int ROWS>
__device__ __forceinline__ void rows_to_read(const CacheReadArgs& a, int (&s)[ROWS],
                                             int (&page)[ROWS]) {
  const int b = blockIdx.y;
  const int len = a.k_len ? min(a.k_len[b], a.n_k) : a.n_k;
  const int32_t* table = a.table + (int64_t)b * a.max_pages;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    s[r] = (blockIdx.x * ROWS + r) * kCacheUnits + (threadIdx.x >> 3);
    // (the table is read up to n_k, so as not to wait for the length)
    const int p = s[r] < a.n_k ? page_of(table, s[r], a.c.page_shift, a.c.n_pages) : -1;
    page[r] = s[r] < len ? (p < 0 ? -2 : p) : -1;
  }
}

// Values of a sequence's first n_k rows.  8 lanes take five chunks of 128 values of a row
// (blockIdx.z: which five; a latent row is one run) or one chunk of each of four rows, and
// hold them at once, two runs of 8 values a lane, 64 apart, so that each store of the 8
// lanes is one contiguous run (16 codes a lane took 24 us where this takes 20).
// Measured (B200): 65536 latent rows of 512 e4m3 + 64 bf16 values (1808 bytes read and
// written) to bf16 21.3 us, 5.6 TB/s, and 262144 rows 75 us, 6.3 TB/s; two ragged sequences of
// up to 32768, 49 thousand rows, 18 us.  Runs of four chunks took a seventh longer: the second
// run of a row holds 64 values and looks its page up again.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheReadArgs a) {
  constexpr int BATCH = ROWS > 1 ? ROWS : kReadBatch, CHUNKS = BATCH / ROWS;
  const int l = threadIdx.x & 7, q_chunks = a.c.dim_q >> 7, width = a.c.dim_q + a.c.dim_raw;
  const int c0 = blockIdx.z * CHUNKS;
  int s[ROWS], page[ROWS];
  rows_to_read<ROWS>(a, s, page);
  uint4 w[BATCH][2];                           // 8 codes in half of one, or 8 bf16 values
  float sc[BATCH];
#pragma unroll
  for (int k = 0; k < BATCH; ++k) {
    const int r = k / CHUNKS, c = c0 + k % CHUNKS;
    const int at = s[r] & ((1 << a.c.page_shift) - 1);
    w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
    sc[k] = 1.f;
    if (page[r] < 0) continue;
    const int64_t p = page[r];
    if (c < q_chunks) {
      const uint8_t* from = a.c.codes + p * a.c.codes_ps + (int64_t)at * a.c.dim_q + c * 128 + l * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 u = *reinterpret_cast<const uint2*>(from + h * 64);
        w[k][h].x = u.x;
        w[k][h].y = u.y;
      }
      sc[k] = a.c.scale[p * a.c.scale_ps + at * q_chunks + c];
    } else {
      const __nv_bfloat16* from = a.c.raw + p * a.c.raw_ps + (int64_t)at * a.c.dim_raw;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int d = (c - q_chunks) * 128 + h * 64 + l * 8;
        if (d < a.c.dim_raw) w[k][h] = *reinterpret_cast<const uint4*>(from + d);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < BATCH; ++k) {
    const int r = k / CHUNKS, c = c0 + k % CHUNKS;
    if (page[r] == -1) continue;
    T* out = reinterpret_cast<T*>(a.out) + ((int64_t)blockIdx.y * a.n_k + s[r]) * width;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = c * 128 + h * 64 + l * 8;
      if (d >= width) continue;
      float v[8];
      if (c < q_chunks) {
        e4m3x4_values(w[k][h].x, sc[k], v);
        e4m3x4_values(w[k][h].y, sc[k], v + 4);
      } else {
        RowType<__nv_bfloat16>::unpack(w[k][h], v);
      }
      store8(out + d, v);
    }
  }
}

// Codes and scales as they stand (the operands of the indexer's e4m3 scan).  Measured
// (B200): 32 sequences of 16384 keys of 128 codes 23.8 us, 5.8 TB/s; of up to 16384, 270
// thousand keys, 14.7 us.
template <int ROWS>
__global__ void __launch_bounds__(kCacheThreads) cache_read_codes_kernel(const CacheReadArgs a) {
  constexpr int CHUNKS = kCacheBatch / ROWS;
  const int l = threadIdx.x & 7, q_chunks = a.c.dim_q >> 7;
  int s[ROWS], page[ROWS];
  rows_to_read<ROWS>(a, s, page);
  const int c0 = blockIdx.z * CHUNKS;
  uint4 w[kCacheBatch];
  float sc[kCacheBatch];
#pragma unroll
  for (int k = 0; k < kCacheBatch; ++k) {
    const int r = k / CHUNKS, c = c0 + k % CHUNKS;
    w[k] = make_uint4(0, 0, 0, 0);
    sc[k] = 1.f;
    if (page[r] >= 0 && c < q_chunks) {
      const int at = s[r] & ((1 << a.c.page_shift) - 1);
      w[k] = *reinterpret_cast<const uint4*>(a.c.codes + page[r] * a.c.codes_ps +
                                             (int64_t)at * a.c.dim_q + c * 128 + l * 16);
      sc[k] = a.c.scale[page[r] * a.c.scale_ps + at * q_chunks + c];
    }
  }
#pragma unroll
  for (int k = 0; k < kCacheBatch; ++k) {
    const int r = k / CHUNKS, c = c0 + k % CHUNKS;
    if (page[r] == -1 || c >= q_chunks) continue;
    const int64_t to = (int64_t)blockIdx.y * a.n_k + s[r];
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a.out) + to * a.c.dim_q + c * 128 +
                              l * 16) = w[k];
    if (l == 0) a.out_scale[to * q_chunks + c] = sc[k];
  }
}

}  // namespace dsa
