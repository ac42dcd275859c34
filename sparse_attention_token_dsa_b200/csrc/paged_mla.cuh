// paged_mla.cuh — latent attention over a paged cache: every cached position of a
// sequence, one query token, a few, or a chunk of a prompt.
//
// For query token t of sequence b at position p = k_len[b] - q_len[b] + t, with absorbed
// query heads q_h (512 latent + 64 rope values) and the cached rows kv_s, s <= p:
//     x_s = scale q_h . kv_s,  o_h = sum_s softmax(x)_s kv_s[0:512],  lse_h = log sum_s exp(x_s).
//
// What bounds it.  A cached row is 1152 bytes in bf16 and costs 2 (576 + 512) FLOP a head:
// with 128 heads 242 FLOP a byte, just under the ratio of the tensor cores' rate to the
// memory's, so one query token needs both nearly in full: each cached row must come from
// memory once, and both products must run on the tensor cores without recomputing one.
//
// Layout.  The (token, head) pairs of a sequence are rows; 128 rows make a tile, and two
// CTAs (a cluster) share one: the matrix instructions of the pair have M = 128 rows, 64
// from each CTA.  So a CTA holds 64 rows of q (72 KB), 64 rows of the output in TMEM (256
// columns, both lane halves), and half of each B operand:
//     S = Q K^T   N = 128 positions, of which the CTA brings 64 (all 576 values)
//     O += P V    N = 2 x 256 values, of which the CTA brings 256 (of all 128 positions)
// A single CTA would have to hold 128 x 512 outputs, all of TMEM, with no place for S.
// A tile of 128 positions runs through rings of operand slots: 3 of 64 positions x 192
// values (K) and 4 of 32 positions x 256 values (V, read in place as an MN-major operand).
//
// Work split.  The tiles of all (sequence, row tile) pairs form one line, cut into equal
// shares, one for each cluster; a pair that more than one cluster meets leaves partial
// (maximum, denominator, output) in the workspace, joined by a second kernel.  So long and
// short sequences, few rows and many use the whole GPU, and the lengths stay on the device.
// Going from one pair to the next drains the pipeline and costs about two tiles' time, so
// in long shares a pair counts as two tiles more than it has (24 ragged sequences with a
// few short ones among them: 119 -> 115 us; three or four tiles do as well).
//
// Softmax: fp32, one thread for a row's 64 of 128 positions; the running maximum is raised
// lazily (by more than 2^8), P is rounded to bf16 for the second product (the matrix
// instructions take both operands in one type), the denominator sums the unrounded values.
// Rows of the cache behind k_len hold anything, also NaN: their scores are replaced and
// their V rows zeroed, as 0 x NaN would not vanish in the product.
//
// Measured (B200, warm and back to back, on several boxes; a copy runs at 6545 GB/s there, the
// library's large bf16 product at 1658 TFLOP/s in a burst and at 1394 for seconds):
//   one token of 128 heads over 32 x 131072 positions   1.17 to 1.33 ms, 3.6 to 4.1 TB/s and
//     880 to 1000 TFLOP/s at once, at the chip's 1000 W with the SM clock at 1.05 of 1.97 GHz
//     (3000 clocks a tile).  Calls 60 ms apart, which run at 1.97 GHz and 270 W, 1.03 ms, 4.7
//     TB/s: 4600 clocks a tile, so then it is the rows' way from memory through a ring of one
//     tile that bounds it.  Alone the bytes would take 0.74 ms, the products 0.84 at the
//     sustained rate.
//   512 tokens of 128 heads behind 8192 positions   0.97 to 1.00 ms, 1200 to 1240 TFLOP/s (0.86
//     to 0.89 of the sustained rate), at the power limit, 1.46 GHz; 60 ms apart 0.86 ms.  Over
//     e4m3 rows 1.35 to 1.40 ms.
//   4 tokens of 64 heads over 24 sequences of 16384 e4m3 positions   0.285 to 0.30 ms, 750
//     TFLOP/s (bf16 rows 0.256), at the power limit, 1.67 GHz: a tile's rows are written and
//     read as codes, written and read as bf16 in shared memory.  Up to 4 tokens and 16001
//     113 to 120 us; one token of 128 heads over the same 87.
//   one token of 16 heads over 1000 positions   14 us replayed, 16 called: two launches, a plan
//     and a join.
#pragma once
#include "cache.cuh"
#include "pair.cuh"

namespace dsa {

constexpr int kPmDqk = 576;
constexpr int kPmDv = 512;
constexpr int kPmRows = 128;            // rows of a tile (64 a CTA)
constexpr int kPmKeys = 128;            // positions of a tile
constexpr int kPmChunk = 64 * 128;      // 64 positions (or rows) x 64 values in bf16
constexpr int kPmSlice = 4 * 32 * 128;  // 32 positions x 256 values
// Rings of operand slots, a tile's worth.  bf16 rows are copied into them; e4m3 rows are
// copied into the upper half of where their values go (a chunk of K, half a slice of V) and
// converted in place, the lower half first.
template <bool CODES>
struct PmRing {
  static constexpr int kKSlots = CODES ? 9 : 3;      // of K
  static constexpr int kChunks = CODES ? 1 : 3;      // in a slot of K
  static constexpr int kVSlots = 4;                  // slices of V
  static constexpr int kKBytes = kChunks * kPmChunk;
  // Chunk of q that meets the k-th chunk of K: in e4m3 the bf16 chunk comes first, as it
  // needs no conversion.
  __device__ __forceinline__ static int q_chunk(int k) { return CODES ? (k == 0 ? 8 : k - 1) : k; }
};
constexpr int kPmQBytes = 9 * 64 * 128;
constexpr int kPmPBytes = 2 * 64 * 128;
constexpr int kPmClusters = 74;         // one CTA an SM
constexpr int kPmSwitch = 2;            // tiles' worth of time to go to another pair
constexpr int kPmLongShare = 16;        // shares (in tiles) where that is reckoned
constexpr float kPmLazy = 8.f;          // log2 headroom before the maximum is raised
constexpr int kPmLoaders = 4;           // warps that convert e4m3 rows, for K and for V
constexpr int kPmThreadsRaw = 32 * 10;  // softmax 4, S, PV, K, V, relays of K and V
constexpr int kPmThreadsCodes = 32 * (8 + 2 * kPmLoaders);   // 8 as above, converting K 4, V 4
constexpr long long kPmGraceCycles = 200000;         // about 0.1 ms
constexpr int kPmJoinThreads = 128;
constexpr int kPmJoinBlocks = 148 * 8;  // of the join, resident at once

struct PagedMlaArgs {
  CachePlanes c;
  const int32_t* table;    // [batch][max_pages]
  const int32_t* k_len;    // [batch]
  const int32_t* q_len;    // [batch] or null
  int32_t batch, n_q, heads, max_pages;
  int32_t row_tiles;       // row tiles of a sequence of n_q tokens
  int32_t pairs;           // batch * row_tiles
  int32_t clusters;
  int32_t join_rows;       // rows that a block of the join takes
  int32_t wait_kilocycles; // limit of a wait
  int32_t stall;           // DSA_FLAG_TEST_STALL: in the first cluster CTA 1 loads V (bf16
                           // rows), or CTA 0 K (e4m3), for one tile only
  float scale_log2;        // softmax scale * log2(e)
  uint16_t* out;           // [batch][n_q][heads][512] bf16
  float* lse;              // [batch][n_q][heads] or null
  int32_t* status;         // of the call (written by the join)
  int32_t* states;         // [clusters][2]: status of a cluster, and the wait that gave up
  int32_t* plan;           // [0]: units of a share; [1 + pair]: place of the pair's first tile
  float* part_o;           // [clusters][later part, first part of a pair][128][512]
  float2* part_ml;         // [2 * clusters][128] maximum (log2 units), denominator
};

struct PagedMlaTail {
  uint64_t q_full, q_empty, q_ready, o_empty, p_full, pv_done, drain[2];
  uint64_t k_full[9], k_ready[9], k_empty[9];
  uint64_t v_full[4], v_ready[4], v_empty[4];
  uint64_t s_full[2], s_empty[2];
  float peer[2][128];      // maxima (and at the end denominators) of a row's two threads
  int32_t start_pair, start_off, count, share, extra;
  uint32_t tmem_base;
  WaitLimit limit;
};

constexpr size_t paged_mla_smem_bytes() {
  return 1024 + kPmQBytes + PmRing<false>::kKSlots * PmRing<false>::kKBytes +
         PmRing<false>::kVSlots * kPmSlice + kPmPBytes + sizeof(PagedMlaTail);
}
static_assert(paged_mla_smem_bytes() <= 227 * 1024, "shared memory of one CTA");
static_assert(PmRing<true>::kKSlots * PmRing<true>::kKBytes ==
                  PmRing<false>::kKSlots * PmRing<false>::kKBytes,
              "both forms fill the same space");

// ------------------------------------------------------------------- work --
struct PmPair {
  int b, row0, rows;       // sequence, first row, rows of the tile
  int kl, ql;              // cached positions, query tokens
  int tiles;               // tiles of positions that some row sees
};

__device__ __forceinline__ PmPair pm_pair(const PagedMlaArgs& a, int p) {
  PmPair r;
  r.b = p / a.row_tiles;
  r.row0 = (p - r.b * a.row_tiles) * kPmRows;
  const int most = a.max_pages << a.c.page_shift;
  r.kl = min(max(a.k_len[r.b], 0), most);
  r.ql = a.q_len ? min(max(a.q_len[r.b], 0), a.n_q) : a.n_q;
  r.rows = min(kPmRows, r.ql * a.heads - r.row0);
  r.tiles = 0;
  if (r.rows > 0) {
    const int last = r.kl - r.ql + (r.row0 + r.rows - 1) / a.heads;   // last row's position
    if (last >= 0) r.tiles = last / kPmKeys + 1;
  }
  return r;
}

// A cluster's place in its share of the line.  A pair stands there as `extra` units and
// then its tiles: the units are what it costs a cluster to go from one pair to the next.
struct PmWalk {
  int p, off, left;        // pair, units of it done, units left
  int at;                  // place on the line
  int extra, slot;
};
struct PmSegment {
  PmPair pair;
  int p, t0, n, slot;
  int first;               // place of the pair's first tile
  bool whole;
};

// The next run of tiles of one pair in a cluster's share (out of line: every role calls it,
// and only between its loops).
__device__ __noinline__ bool pm_next_far(const PagedMlaArgs& a, PmWalk* walk, PmSegment* seg) {
  PmWalk w = *walk;
  PmSegment s;
  if (w.left <= 0) return false;
  while (w.p < a.pairs) {
    s.pair = pm_pair(a, w.p);
    if (s.pair.tiles > 0) break;
    // behind a sequence's last token there are only empty row tiles
    w.p = s.pair.rows > 0 ? w.p + 1 : (s.pair.b + 1) * a.row_tiles;
  }
  if (w.p >= a.pairs) return false;
  // (a share may end among a pair's extra units, with no tile of it)
  const int cost = s.pair.tiles + w.extra, take = min(w.left, cost - w.off), to = w.off + take;
  if (to <= w.extra) return false;
  s.p = w.p;
  s.first = w.at - w.off + w.extra;
  s.t0 = max(w.off - w.extra, 0);
  s.n = to - w.extra - s.t0;
  s.whole = s.n == s.pair.tiles;
  s.slot = w.slot + (s.t0 == 0 ? 1 : 0);             // of a part: a pair's first, or a later one
  w.left -= take;
  w.off = to;
  w.at += take;
  if (to == cost) {
    w.off = 0;
    ++w.p;
  }
  *walk = w;
  *seg = s;
  return true;
}

// The same with the segment in a variable whose address nobody has.
__device__ __forceinline__ bool pm_next(const PagedMlaArgs& a, PmWalk& w, PmSegment& s) {
  PmWalk w1 = w;
  PmSegment s1;
  const bool more = pm_next_far(a, &w1, &s1);
  if (more) {
    w = w1;
    s = s1;
  }
  return more;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values side by side.
__device__ __forceinline__ uint64_t pack2u(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return pack2u(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

// 32 lanes x 8 columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// 16 e4m3 codes times a scale as bf16.  A code's exponent and mantissa, moved to where
// bf16 has its own, are the value times 2^-120 (also for e4m3's subnormal codes, which
// become bf16's), so one packed product with 2^120 scale gives two values, exactly, where
// the scale is a power of two of at most 2^7: four instructions for two codes, none of
// them a conversion (those run at a quarter of the rate).  `sel` spreads two bytes over
// halves with their signs above them, so a shift by 4 leaves the sign at bit 15 and its
// copies, masked away, below it.
__device__ __forceinline__ uint32_t two_codes(uint32_t w, uint32_t sel, uint32_t mul) {
  uint32_t t, r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(w), "r"(sel));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"((t << 4) & 0x87f087f0u), "r"(mul));
  return r;
}
__device__ __forceinline__ void codes_to_bf16(const uint4& w, uint32_t mul, uint4& lo, uint4& hi) {
  lo = make_uint4(two_codes(w.x, 0x9180, mul), two_codes(w.x, 0xb3a2, mul),
                  two_codes(w.y, 0x9180, mul), two_codes(w.y, 0xb3a2, mul));
  hi = make_uint4(two_codes(w.z, 0x9180, mul), two_codes(w.z, 0xb3a2, mul),
                  two_codes(w.w, 0x9180, mul), two_codes(w.w, 0xb3a2, mul));
}
// 2^120 scale in both halves; 0 where the short way does not hold.
__device__ __forceinline__ uint32_t code_factor(float scale) {
  const uint32_t u = __float_as_uint(scale);
  if ((u & 0x807fffffu) != 0u || u < 0x00800000u || scale > 128.f) return 0u;
  const uint32_t h = (u >> 16) + (120u << 7);
  return h | (h << 16);
}
// Any scale: four units, in fp32, rounded to bf16 once (out of line, for scales that
// dsa_cache_write does not make).
__device__ __noinline__ void four_units_any(const uint4* codes, uint8_t* const* to_lo,
                                            uint8_t* const* to_hi, float scale) {
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const uint4 w = codes[u];
    float v[16];
    e4m3x4_values(w.x, scale, v);
    e4m3x4_values(w.y, scale, v + 4);
    e4m3x4_values(w.z, scale, v + 8);
    e4m3x4_values(w.w, scale, v + 12);
    if (scale == 0.f) {                              // a row past the end: also NaN codes
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
    *reinterpret_cast<uint4*>(to_lo[u]) =
        make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
    *reinterpret_cast<uint4*>(to_hi[u]) = make_uint4(
        bf16x2(v[8], v[9]), bf16x2(v[10], v[11]), bf16x2(v[12], v[13]), bf16x2(v[14], v[15]));
  }
}
// Whether one of 8 codes is a NaN (0x7f, 0xff): its lower seven bits carry into the eighth.
__device__ __forceinline__ uint32_t nan_codes(uint32_t a, uint32_t b, uint32_t so_far) {
  return so_far | ((a & 0x7f7f7f7fu) + 0x01010101u) | ((b & 0x7f7f7f7fu) + 0x01010101u);
}
// Four units of 16 codes in shared memory a lane, from(u) to to(u, 0) and to(u, 1).  The
// warp has read all of them before it writes the first, as values may take codes' places.
// NANS: a lane that holds a NaN code takes the way of any scale, as the short one would make
// 480 times the scale of it (the look costs the e4m3 batch 2 %).  K is looked at and V is not: a
// NaN logit makes all outputs of the tokens that see its position NaN, and those of the others
// need V finite.
template <bool NANS, typename From, typename To>
__device__ __forceinline__ void four_units(bool exact, uint32_t f, float scale, From from, To to) {
  uint4 w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = *reinterpret_cast<const uint4*>(from(u));
  __syncwarp();
  if (NANS) {
    uint32_t nan = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) nan = nan_codes(w[u].z, w[u].w, nan_codes(w[u].x, w[u].y, nan));
    exact = exact && (nan & 0x80808080u) == 0;
  }
  if (exact) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint4 lo, hi;
      codes_to_bf16(w[u], f, lo, hi);
      *reinterpret_cast<uint4*>(to(u, 0)) = lo;
      *reinterpret_cast<uint4*>(to(u, 1)) = hi;
    }
  } else {
    uint4 a[4];
    uint8_t *b[4], *c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      a[u] = w[u];
      b[u] = to(u, 0);
      c[u] = to(u, 1);
    }
    four_units_any(a, b, c, scale);
  }
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// A slice of V: 4 blocks of 64 values of 32 positions, or, where a page has 16, twice 4
// blocks of 16 (so that a page is still one copy).
struct VLayout {
  uint32_t block, half;    // bytes from block to block, from 16 positions to the next 16
  __device__ __forceinline__ explicit VLayout(bool halves)
      : block(halves ? 2048 : 4096), half(halves ? 8192 : 2048) {}
  __device__ __forceinline__ uint32_t row(int r) const { return (r >> 4) * half + (r & 15) * 128; }
};

// Abort path: let a slot's last copies land.  `n` tiles were begun; the slot's last fill
// belongs to the n-th or, where the loader gave up before it, to the one before, which
// the wait's limit then covers.
__device__ __forceinline__ void drain_slot(uint64_t* full, uint32_t n, volatile WaitLimit* limit) {
  mbar_wait_drain(full, (n & 1) ^ 1, min(wait_cycles(limit), kWaitCycles / 64));
}

template <bool CODES>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(CODES ? kPmThreadsCodes : kPmThreadsRaw, 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ CUtensorMap rmap, const PagedMlaArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;                                // [9][64 rows x 128 B]
  using Ring = PmRing<CODES>;
  uint8_t* Ks = Qs + kPmQBytes;                      // [slots][chunks][64 positions x 128 B]
  uint8_t* Vs = Ks + Ring::kKSlots * Ring::kKBytes;  // [slots][4 blocks][32 positions x 128 B]
  uint8_t* Ps = Vs + Ring::kVSlots * kPmSlice;       // [2][64 rows x 128 B]
  PagedMlaTail* T = reinterpret_cast<PagedMlaTail*>(Ps + kPmPBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int cl = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  int32_t* const state = a.states + 2 * cl;

  if (threadIdx.x == 0) {
    mbar_init(&T->q_full, 1);
    mbar_init(&T->q_empty, 1);
    mbar_init(&T->q_ready, 2);
    mbar_init(&T->o_empty, 8);
    mbar_init(&T->p_full, 8);
    mbar_init(&T->pv_done, 1);
    for (int i = 0; i < 9; ++i) {
      mbar_init(&T->k_full[i], 1);
      mbar_init(&T->k_ready[i], 2);
      mbar_init(&T->k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&T->v_full[i], 1);
      mbar_init(&T->v_ready[i], CODES ? 4 : 2);
      mbar_init(&T->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T->s_full[i], 1);
      mbar_init(&T->s_empty[i], 8);
      mbar_init(&T->drain[i], 1);
    }
    T->limit.abort = 0;
    T->limit.kilocycles = a.wait_kilocycles;
    if (rank == 0) state[0] = DSA_OK;
    fence_barrier_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    if (CODES) prefetch_tmap(&rmap);
  }
  if (warp == 4) pair_tmem_alloc(&T->tmem_base, 512);
  if (warp == 5) {
    // this cluster's share of the line of tiles
    const bool few = a.pairs <= 32;                  // a lane each: looked at once
    const int mine = lane < a.pairs ? pm_pair(a, lane).tiles : 0;
    int total = 0, live = 0;                         // tiles, pairs that have some
    for (int p0 = 0; p0 < a.pairs; p0 += 32) {
      const int p = p0 + lane;
      const int n = few ? mine : (p < a.pairs ? pm_pair(a, p).tiles : 0);
      total += __reduce_add_sync(0xffffffffu, n);
      live += __popc(__ballot_sync(0xffffffffu, n > 0));
    }
    // (not in short shares, where it would only unbalance them)
    const int extra = total / clusters >= kPmLongShare ? kPmSwitch : 0;
    total += extra * live;
    const int share = max(1, (total + clusters - 1) / clusters);
    const int begin = (int)min((long long)cl * share, (long long)total);
    int before = 0, found = -1, off = 0;
    for (int p0 = 0; p0 < a.pairs && found < 0 && begin < total; p0 += 32) {
      const int p = p0 + lane;
      int n = few ? mine : (p < a.pairs ? pm_pair(a, p).tiles : 0);
      n += n > 0 ? extra : 0;
      int upto = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += v;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + upto > begin);
      if (hit) {
        const int l = __ffs(hit) - 1;
        found = p0 + l;
        off = begin - before - __shfl_sync(0xffffffffu, upto - n, l);
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) {
      T->start_pair = found;
      T->start_off = off;
      T->count = found < 0 ? 0 : min(share, total - begin);
      T->share = share;
      T->extra = extra;
      if (cl == 0 && rank == 0) a.plan[0] = share;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = T->tmem_base;
  volatile WaitLimit* limit = &T->limit;
  // tiles that a loader stops after (tests of the timeout path; else none)
  const uint32_t stop = a.stall && cl == 0 && rank == (CODES ? 0 : 1) ? 1u : 0xffffffffu;
  PmWalk walk{T->start_pair, T->start_off, T->count, cl * T->share, T->extra, 2 * cl};
  PmSegment s;

  auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return mbar_wait_far(bar, parity, limit, state, where);
  };
  // The matrix warps' waits, on barriers where both CTAs arrive (pair_acquire follows where
  // they announce shared memory).  A slot's barrier is looked at (`seen`) before the matrix
  // instructions of the slot before it are issued.
  auto wait_pair = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
    return mbar_wait_far<true>(bar, parity, limit, state, where);
  };
  auto wait_seen = [&](bool seen, uint64_t* bar, uint32_t parity, int where) -> bool {
    return seen || mbar_poll<true>(bar, parity, limit, state, where);
  };

  // The roles of warps 4 and up (but for the conversion of codes) run in one lane.
  if (warp == 4) {
    // ------------------------------------------------------- Q, and S = Q K^T --
    // Each CTA loads its 64 rows of q; CTA 0's warp issues the products of both.  S and
    // O += P V have a warp each, so neither waits for the other's operands.
    if (elect_one()) {
      const uint32_t idesc = make_idesc<MmaKind::BF16>(kPmKeys);
      const uint64_t q_desc = make_sdesc(smem_u32(Qs)), k_desc = make_sdesc(smem_u32(Ks));
      const uint32_t q_ready = in_cta(&T->q_ready, 0);
      uint32_t sc = 0, qc = 0;                       // tiles, segments so far
      int slot = 0, parity = 0;                      // of the next K slot
      bool ok = true;
      while (ok && pm_next(a, walk, s)) {
        ok = wait(&T->q_empty, (qc & 1) ^ 1, 57);
        if (!ok) break;
        mbar_arrive_expect_tx(&T->q_full, kPmQBytes);
        const int row = s.pair.b * a.n_q * a.heads + s.pair.row0 + 64 * rank;
        for (int c = 0; c < 9; ++c)
          tma_load_2d(Qs + c * kPmChunk, &qmap, &T->q_full, c * 64, row);
        ok = wait(&T->q_full, qc & 1, 58);
        if (!ok) mbar_wait_drain(&T->q_full, qc & 1);
        else pair_publish(q_ready);
        if (rank == 0) {
          ok = ok && wait_pair(&T->q_ready, qc & 1, 53);
          pair_acquire();
          for (int i = 0; i < s.n && ok; ++i, ++sc) {
            const int b = sc & 1;
            bool seen = mbar_seen(&T->k_ready[slot], parity);
            ok = wait_pair(&T->s_empty[b], ((sc >> 1) & 1) ^ 1, 51);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + 256 + b * 64;
#pragma unroll 1
            for (int k = 0; k < 9; k += Ring::kChunks) {
              ok = ok && wait_seen(seen, &T->k_ready[slot], parity, 52);
              if (!ok) break;
              pair_acquire();
              const int cur = slot;
              if (++slot == Ring::kKSlots) {
                slot = 0;
                parity ^= 1;
              }
              seen = mbar_seen(&T->k_ready[slot], parity);
#pragma unroll
              for (int c = 0; c < Ring::kChunks; ++c)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)       // 16 values
                  pair_mma_bf16(d, q_desc + ((Ring::q_chunk(k + c) * kPmChunk + kk * 32) >> 4),
                                k_desc + ((cur * Ring::kKBytes + c * kPmChunk + kk * 32) >> 4),
                                idesc, (k | c | kk) != 0);
              pair_commit(&T->k_empty[cur]);
            }
            if (!ok) break;
            pair_commit(&T->s_full[b]);
            if (i == s.n - 1) pair_commit(&T->q_empty);
          }
        }
        ++qc;
      }
      // the last arrival from the MMAs has come before the CTA may end
      if (ok && qc) wait(&T->q_empty, (qc & 1) ^ 1, 70);
      if (!ok && rank == 0) {
        // abort path: the MMAs already issued must end before TMEM is freed
        pair_commit(&T->drain[0]);
        mbar_wait_drain(&T->drain[0], 0);
      }
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- O += P V --
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = make_idesc<MmaKind::BF16>(256) | (1u << 16);   // B MN-major
      const VLayout at(!CODES && a.c.page_shift == 4);
      const uint64_t p_desc = make_sdesc(smem_u32(Ps));
      const uint64_t v_desc = make_sdesc_mn(smem_u32(Vs), at.block);
      uint32_t pc = 0, qc = 0;
      int slot = 0, parity = 0;                      // of the next V slot
      bool ok = true;
      while (ok && pm_next(a, walk, s)) {
        ok = wait_pair(&T->o_empty, (qc & 1) ^ 1, 54);
        for (int i = 0; i < s.n && ok; ++i, ++pc) {
          ok = wait_pair(&T->p_full, pc & 1, 55);
          if (!ok) break;
          bool seen = mbar_seen(&T->v_ready[slot], parity);
          tc_fence_after();
#pragma unroll 1
          for (int v = 0; v < 4; ++v) {
            ok = ok && wait_seen(seen, &T->v_ready[slot], parity, 56);
            if (!ok) break;
            pair_acquire();                          // (also for P, before the first slot)
            const int cur = slot;
            if (++slot == Ring::kVSlots) {
              slot = 0;
              parity ^= 1;
            }
            seen = mbar_seen(&T->v_ready[slot], parity);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {         // 16 positions
              const int k16 = v * 2 + kk;
              const uint64_t ad = p_desc + (((k16 >> 2) * kPmChunk + (k16 & 3) * 32) >> 4);
#pragma unroll
              for (int h = 0; h < 2; ++h)            // 128 values of each CTA
                pair_mma_bf16(tmem + h * 128, ad,
                              v_desc + ((cur * kPmSlice + h * 2 * at.block + kk * at.half) >> 4), idesc,
                              (i | k16) != 0);
            }
            pair_commit(&T->v_empty[cur]);
          }
          if (ok) pair_commit(&T->pv_done);
        }
        ++qc;
      }
      if (!ok) {
        pair_commit(&T->drain[1]);
        mbar_wait_drain(&T->drain[1], 0);
      }
    }
  } else if (warp >= 6) {
    // --------------------------------------------------------------- loaders --
    // K and V have loaders of their own: a V slot comes free half a tile later than the K
    // slots beside it, and one loader for both would hold the K copies back.
    uint32_t n = 0;                                  // tiles so far
    bool ok = true;
    const int shift = a.c.page_shift, mask = (1 << shift) - 1;
    const int32_t* table = nullptr;                  // of the sequence
    // page of a position; past the end (and where the table is wrong) one that TMA reads
    // as zeros
    auto page_at = [&](int key) -> int {
      if (key >= s.pair.kl) return a.c.n_pages;
      const int p = page_of(table, key, shift, a.c.n_pages);
      if (p < 0) set_status(state, DSA_ERR_INVALID, 61);
      return p < 0 ? a.c.n_pages : p;
    };
    if constexpr (!CODES) {
      if (warp == 6 && elect_one()) {
        const int rows = min(1 << shift, 64);        // of a copy
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
#pragma unroll 1
          for (int i = s.t0; i < s.t0 + s.n && ok; ++i, ++n) {
            // pages of the tile, looked up before its slots are free
            const int key = i * kPmKeys + 64 * rank;
            const int z0 = page_at(key), z1 = rows < 64 ? page_at(key + rows) : 0;
            const int z2 = rows < 32 ? page_at(key + 32) : 0, z3 = rows < 32 ? page_at(key + 48) : 0;
#pragma unroll 1
            for (int k = 0; k < Ring::kKSlots; ++k) {
              ok = wait(&T->k_empty[k], (n & 1) ^ 1, 62);
              if (!ok) break;
              mbar_arrive_expect_tx(&T->k_full[k], Ring::kKBytes);
              uint8_t* dst = Ks + k * Ring::kKBytes;
              if (rows == 64) {
                tma_load_4d(dst, &kmap, &T->k_full[k], 0, key & mask, 3 * k, z0);
              } else {                               // chunk by chunk, pages below one another
#pragma unroll 1
                for (int c = 0; c < 3; ++c) {
                  uint8_t* to = dst + c * kPmChunk;
                  tma_load_4d(to, &kmap, &T->k_full[k], 0, 0, 3 * k + c, z0);
                  tma_load_4d(to + rows * 128, &kmap, &T->k_full[k], 0, 0, 3 * k + c, z1);
                  if (rows < 32) {
                    tma_load_4d(to + 32 * 128, &kmap, &T->k_full[k], 0, 0, 3 * k + c, z2);
                    tma_load_4d(to + 48 * 128, &kmap, &T->k_full[k], 0, 0, 3 * k + c, z3);
                  }
                }
              }
            }
          }
        }
        // the last copies have landed (also on the abort path) and the last arrivals from
        // the MMAs have come before the CTA may end
        for (int k = 0; k < Ring::kKSlots && n; ++k)
          if (ok) wait(&T->k_empty[k], (n & 1) ^ 1, 64);
          else drain_slot(&T->k_full[k], n, limit);
      } else if (warp == 7 && elect_one()) {
        const int rows = min(1 << shift, 32);
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
#pragma unroll 1
          for (int i = s.t0; i < s.t0 + s.n && ok; ++i, ++n) {
            if (n == stop) {
              ok = false;
              break;
            }
#pragma unroll 1
            for (int v = 0; v < Ring::kVSlots; ++v) {
              const int key = i * kPmKeys + v * 32;
              const int page = page_at(key);
              ok = wait(&T->v_empty[v], (n & 1) ^ 1, 63);
              if (!ok) break;
              mbar_arrive_expect_tx(&T->v_full[v], kPmSlice);
              uint8_t* dst = Vs + v * kPmSlice;
              tma_load_4d(dst, &vmap, &T->v_full[v], 0, key & mask, rank * 4, page);
              if (rows == 16)
                tma_load_4d(dst + 8192, &vmap, &T->v_full[v], 0, 0, rank * 4, page_at(key + 16));
            }
          }
        }
        for (int v = 0; v < Ring::kVSlots && n; ++v)
          if (ok) wait(&T->v_empty[v], (n & 1) ^ 1, 65);
          else drain_slot(&T->v_full[v], n, limit);
      } else if (warp == 8 && elect_one()) {
        // K slots to the matrix warp (in CTA 0).  The slots' own barriers stay in the CTA
        // that issued the copies, so either CTA can wait for its own before it ends.
        const uint32_t k_ready = in_cta(&T->k_ready[0], 0);
        while (ok && pm_next(a, walk, s))
          for (int i = 0; i < s.n && ok; ++i, ++n)
            for (int k = 0; k < Ring::kKSlots && ok; ++k) {
              ok = wait(&T->k_full[k], n & 1, 59);
              if (ok) pair_publish(k_ready + k * 8);
            }
      } else if (warp == 9) {
        // V slots to the matrix warp, after zeroing the rows behind k_len
        const uint32_t v_ready = in_cta(&T->v_ready[0], 0);
        const VLayout at(shift == 4);
        while (ok && pm_next(a, walk, s)) {
          for (int i = s.t0; i < s.t0 + s.n && ok; ++i, ++n) {
            for (int v = 0; v < Ring::kVSlots; ++v) {
              ok = wait(&T->v_full[v], n & 1, 60);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const int live = s.pair.kl - (i * kPmKeys + v * 32);
              if (live < 32) {
                const int from = max(live, 0);
                for (int u = lane; u < (32 - from) * 32; u += 32) {
                  const int r = from + (u >> 5), blk = (u >> 3) & 3, k = u & 7;
                  *reinterpret_cast<uint4*>(Vs + v * kPmSlice + blk * at.block + at.row(r) + k * 16) =
                      make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              if (lane == 0) pair_publish(v_ready + v * 8);
            }
          }
        }
      }
    } else if (warp == 6) {
      // e4m3: the bf16 chunk of K, and its codes in chunks of 64
      if (elect_one()) {
        const int rows = min(1 << shift, 64);        // of a copy
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
#pragma unroll 1
          for (int i = s.t0; i < s.t0 + s.n && ok; ++i, ++n) {
            if (n == stop) {
              ok = false;
              break;
            }
            const int key = i * kPmKeys + 64 * rank;
            const int z0 = page_at(key), z1 = rows < 64 ? page_at(key + rows) : 0;
            const int z2 = rows < 32 ? page_at(key + 32) : 0, z3 = rows < 32 ? page_at(key + 48) : 0;
#pragma unroll 1
            for (int k = 0; k < Ring::kKSlots; ++k) {
              ok = wait(&T->k_empty[k], (n & 1) ^ 1, 62);
              if (!ok) break;
              const bool tail = k == 0;
              mbar_arrive_expect_tx(&T->k_full[k], tail ? kPmChunk : kPmChunk / 2);
              uint8_t* dst = Ks + k * kPmChunk + (tail ? 0 : kPmChunk / 2);
              const CUtensorMap* map = tail ? &rmap : &kmap;
              const int x = tail ? 0 : (k - 1) * 64, step = rows * (tail ? 128 : 64);
              tma_load_3d(dst, map, &T->k_full[k], x, key & mask, z0);
              if (rows < 64) {                       // pages below one another
                tma_load_3d(dst + step, map, &T->k_full[k], x, 0, z1);
                if (rows < 32) {
                  tma_load_3d(dst + 2 * step, map, &T->k_full[k], x, 0, z2);
                  tma_load_3d(dst + 3 * step, map, &T->k_full[k], x, 0, z3);
                }
              }
            }
          }
        }
        for (int k = 0; k < Ring::kKSlots && n; ++k)
          if (ok) wait(&T->k_empty[k], (n & 1) ^ 1, 64);
          else drain_slot(&T->k_full[k], n, limit);
      }
    } else if (warp == 7) {
      // the codes of V, in slices of 32 positions
      if (elect_one()) {
        const int rows = min(1 << shift, 32);
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
#pragma unroll 1
          for (int i = s.t0; i < s.t0 + s.n && ok; ++i, ++n) {
#pragma unroll 1
            for (int v = 0; v < Ring::kVSlots; ++v) {
              const int key = i * kPmKeys + v * 32;
              const int z0 = page_at(key), z1 = rows < 32 ? page_at(key + 16) : 0;
              ok = wait(&T->v_empty[v], (n & 1) ^ 1, 63);
              if (!ok) break;
              mbar_arrive_expect_tx(&T->v_full[v], kPmSlice / 2);
#pragma unroll 1
              for (int b = 0; b < 2; ++b) {          // groups of 128 values
                uint8_t* dst = Vs + v * kPmSlice + b * 8192 + 4096;
                const int x = rank * 256 + b * 128;
                tma_load_3d(dst, &vmap, &T->v_full[v], x, key & mask, z0);
                if (rows < 32) tma_load_3d(dst + 2048, &vmap, &T->v_full[v], x, 0, z1);
              }
            }
          }
        }
        for (int v = 0; v < Ring::kVSlots && n; ++v)
          if (ok) wait(&T->v_empty[v], (n & 1) ^ 1, 65);
          else drain_slot(&T->v_full[v], n, limit);
      }
    } else {
      // Conversion of codes in their slots.  Scales are loaded a tile ahead and their rows'
      // pages looked up a tile before that.
      const float* const scale0 = a.c.scale;
      auto scales = [&](int page, int key) {         // of a row
        const int64_t p = (uint32_t)page < (uint32_t)a.c.n_pages ? page : 0;
        return scale0 + p * a.c.scale_ps + (int64_t)(key & mask) * 4;
      };
      // page of a row to come, as the table has it: used a tile later, so that nobody waits
      // for it (a wrong entry has no live rows; the warps that copy record it)
      auto entry_of = [&](int key) { return key < s.pair.kl ? table[key >> shift] : -1; };
      auto ready = [&](uint32_t bar) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) pair_publish(bar);
      };
      if (warp < 8 + kPmLoaders) {
        // K: a warp takes every fourth chunk, a lane two of its rows
        const int w = warp - 8;
        const uint32_t k_ready = in_cta(&T->k_ready[0], 0);
        int page[2];
        float next[2][2];                            // [row][chunk w, w + 4]
        uint32_t live = 0;                           // bit: the row of `next` is one
        auto look = [&](int tile) {
#pragma unroll
          for (int h = 0; h < 2; ++h) page[h] = entry_of(tile * kPmKeys + 64 * rank + h * 32 + lane);
        };
        auto load = [&](int tile) {
          live = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float* sc = scales(page[h], tile * kPmKeys + 64 * rank + h * 32 + lane);
            next[h][0] = sc[w >> 1];
            next[h][1] = sc[(w >> 1) + 2];
            live |= ((uint32_t)page[h] < (uint32_t)a.c.n_pages ? 1u : 0u) << h;
          }
        };
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
          look(s.t0);
          load(s.t0);
          if (s.n > 1) look(s.t0 + 1);
#pragma unroll 1
          for (int i = 0; i < s.n && ok; ++i, ++n) {
            float now[2][2];
            const uint32_t on = live;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              now[h][0] = on >> h & 1 ? next[h][0] : 0.f;
              now[h][1] = on >> h & 1 ? next[h][1] : 0.f;
            }
            if (i + 1 < s.n) load(s.t0 + i + 1);
            if (i + 2 < s.n) look(s.t0 + i + 2);
            if (w == 0) {                            // the tile's bf16 chunk has landed
              ok = wait(&T->k_full[0], n & 1, 60);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              if (lane == 0) pair_publish(k_ready);
            }
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              const int slot = 1 + w + 4 * j;
              const float s0 = j ? now[0][1] : now[0][0], s1 = j ? now[1][1] : now[1][0];
              const uint32_t f0 = code_factor(s0), f1 = code_factor(s1);
              const bool exact =
                  __all_sync(0xffffffffu, (f0 != 0 || !(on & 1)) && (f1 != 0 || !(on & 2)));
              ok = ok && wait(&T->k_full[slot], n & 1, 59);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {          // row h * 32 + lane
                uint8_t* to = Ks + slot * kPmChunk + (h * 32 + lane) * 128;
                const uint8_t* from = Ks + slot * kPmChunk + kPmChunk / 2 + (h * 32 + lane) * 64;
                four_units<true>(
                    exact, h ? f1 : f0, h ? s1 : s0,
                    [&](int u) { return from + ((u ^ (lane >> 1 & 3)) << 4); },
                    [&](int u, int e) { return to + (((2 * u + e) ^ (lane & 7)) << 4); });
              }
              ready(k_ready + slot * 8);
            }
          }
        }
      } else {
        // V: two warps take every second slice, one its first group of 128 values and one its
        // second, a lane a row (so that neither the loads nor the stores meet in a bank)
        const int w = warp - 8 - kPmLoaders, odd = w >> 1, b = w & 1;
        const uint32_t v_ready = in_cta(&T->v_ready[0], 0);
        int page[2];
        float next[2];                               // of slices odd, odd + 2
        uint32_t live = 0;                           // bit: the row of `next` is one
        auto look = [&](int tile) {
#pragma unroll
          for (int j = 0; j < 2; ++j) page[j] = entry_of(tile * kPmKeys + (odd + 2 * j) * 32 + lane);
        };
        auto load = [&](int tile) {
          live = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            next[j] = scales(page[j], tile * kPmKeys + (odd + 2 * j) * 32 + lane)[rank * 2 + b];
            live |= ((uint32_t)page[j] < (uint32_t)a.c.n_pages ? 1u : 0u) << j;
          }
        };
        while (ok && pm_next(a, walk, s)) {
          table = a.table + (int64_t)s.pair.b * a.max_pages;
          look(s.t0);
          load(s.t0);
          if (s.n > 1) look(s.t0 + 1);
#pragma unroll 1
          for (int i = 0; i < s.n && ok; ++i, ++n) {
            const float now[2] = {live & 1 ? next[0] : 0.f, live & 2 ? next[1] : 0.f};
            const uint32_t on = live;
            if (i + 1 < s.n) load(s.t0 + i + 1);
            if (i + 2 < s.n) look(s.t0 + i + 2);
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              const int v = odd + 2 * j;
              const float sc = j ? now[1] : now[0];
              const uint32_t f = code_factor(sc);
              const bool exact = __all_sync(0xffffffffu, f != 0 || !(on >> j & 1));
              ok = ok && wait(&T->v_full[v], n & 1, 60);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {          // block of 64 values
                const uint8_t* from = Vs + v * kPmSlice + b * 8192 + 4096 + lane * 128;
                uint8_t* to = Vs + v * kPmSlice + b * 8192 + h * 4096 + lane * 128;
                four_units<false>(
                    exact, f, sc, [&](int u) { return from + (((4 * h + u) ^ (lane & 7)) << 4); },
                    [&](int u, int e) { return to + (((2 * u + e) ^ (lane & 7)) << 4); });
              }
              ready(v_ready + v * 8);
            }
          }
        }
      }
    }
  } else {
    // --------------------------------------------------- softmax and output --
    // Thread t of 128 = TMEM lane t: row t & 63 of this CTA, positions (or values) of
    // half t >> 6.  Warps w and w + 2 hold the two halves of the same rows and exchange
    // their maxima over a named barrier; a warp whose wait has run out goes on to meet its
    // mate there (with nothing else to wait for), so neither is left behind.
    // This is the longest chain of a tile, and it is short code on purpose: the roles of a
    // CTA share its instruction cache, and unrolled masks and rescales made every role
    // wait for instructions (42 % of all stalls, and the 128K batch above took 1.63 ms).
    const int t = threadIdx.x, half = t >> 6, row = t & 63;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float inf = __int_as_float(0x7f800000);
    const uint32_t p_full = in_cta(&T->p_full, 0), o_empty = in_cta(&T->o_empty, 0);
    const uint32_t s_empty = in_cta(&T->s_empty[0], 0);
    uint32_t sc = 0;                                 // tiles so far
    bool ok = true;
    auto exchange = [&](float v, int at) -> float {
      T->peer[at][t] = v;
      named_bar_sync(1 + (warp & 1), 64);
      return T->peer[at][t ^ 64];
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity, int where) {
      if (ok) ok = mbar_wait_far(bar, parity, limit, state, where);
      ok = __all_sync(0xffffffffu, ok);
    };
    while (pm_next(a, walk, s)) {
      const int r = s.pair.row0 + rank * 64 + row;   // row of the sequence
      const bool mine = rank * 64 + row < s.pair.rows;
      // positions this row sees: [0, lim); rows past the last are not looked at again
      const int lim = mine ? s.pair.kl - s.pair.ql + r / a.heads + 1 : 0x7fffffff;
      float m_run = -inf, l_run = 0.f;
#pragma unroll 1
      for (int i = 0; i < s.n; ++i, ++sc) {
        wait_all(&T->s_full[sc & 1], (sc >> 1) & 1, 66);
        tc_fence_after();
        const uint32_t at = tmem + lane_off + 256 + (sc & 1) * 64;
        const int seen = lim - ((s.t0 + i) * kPmKeys + half * 64);   // of these 64
        if (!__all_sync(0xffffffffu, seen >= 64)) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 8) {
            uint32_t v[8];
            tmem_ld8(at + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j >= seen) v[j] = 0xff800000u;
            tmem_st8(at + c, v);
          }
          tmem_st_wait();
        }
        uint32_t x[2][32];
        tmem_ld32(at, x[0]);
        tmem_ld32(at + 32, x[1]);
        tmem_ld_wait(x[0]);
        tmem_ld_wait(x[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(s_empty + (sc & 1) * 8);
        float top[4] = {-inf, -inf, -inf, -inf};
#pragma unroll
        for (int j = 0; j < 64; ++j)
          top[j & 3] = fmaxf(top[j & 3], __uint_as_float(x[j >> 5][j & 31]));
        float mt = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        mt = fmaxf(mt, exchange(mt, sc & 1)) * a.scale_log2;
        float f = 1.f;
        if (mt > m_run + kPmLazy) {
          if (m_run > -inf) {
            f = ex2(m_run - mt);
            l_run *= f;
          }
          m_run = mt;
        }
        // positions the row does not see weigh 0, also while its maximum is still -inf
        const float m_sub = m_run == -inf ? 0.f : -m_run;
        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), m2 = pack2(m_sub, m_sub);
        uint64_t l2 = 0;
        uint32_t w[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const uint64_t e = fma2(pack2u(x[j >> 4][2 * (j & 15)], x[j >> 4][2 * (j & 15) + 1]),
                                  scale2, m2);
          const float p0 = ex2(lo2(e)), p1 = ex2(hi2(e));
          l2 = add2(l2, pack2(p0, p1));
          w[j] = bf16x2(p0, p1);
        }
        l_run += lo2(l2) + hi2(l2);
        // P and O are free once the previous PV is complete
        if (i > 0) {
          wait_all(&T->pv_done, (sc - 1) & 1, 67);
          tc_fence_after();
          if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int c0 = 0; c0 < 256; c0 += 32) {
              uint32_t ov[32];
              tmem_ld32(tmem + lane_off + c0, ov);
              tmem_ld_wait(ov);
#pragma unroll
              for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * f);
              tmem_st32(tmem + lane_off + c0, ov);
            }
            tmem_st_wait();
          }
        }
        uint8_t* prow = Ps + half * kPmChunk + row * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(prow + ((c ^ (row & 7)) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) pair_publish(p_full);
      }
      wait_all(&T->pv_done, (sc - 1) & 1, 68);
      tc_fence_after();
      l_run += exchange(l_run, sc & 1);
      named_bar_sync(1 + (warp & 1), 64);            // the next tile writes the same place
      if (!ok) continue;
      const int64_t grow = (int64_t)s.pair.b * a.n_q * a.heads + r;
      const int64_t prow = (int64_t)s.slot * kPmRows + rank * 64 + row;
      if (mine && half == 0) {
        if (!s.whole) a.part_ml[prow] = make_float2(m_run, l_run);
        else if (a.lse)
          a.lse[grow] = l_run == 0.f ? -inf : (m_run + log2f(l_run)) * 0.6931471805599453f;
        if (rank == 0 && row == 0 && s.t0 == 0)
          a.plan[1 + s.p] = s.first;
      }
      // O goes out through the warp's own part of P (32 rows x 128 bytes, free now), so that
      // a store covers whole lines of four rows (stores of each lane's own row, 32 lines an
      // instruction, took 12000 clocks a tile of rows where this takes 8000).
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      uint8_t* stage = Ps + warp * 4096;
      const int first = rank * 64 + (warp & 1) * 32; // row of the tile of lane 0
      const int step = s.whole ? 64 : 32;            // values in 128 bytes
      uint8_t* to = s.whole ? reinterpret_cast<uint8_t*>(
                                  a.out + ((int64_t)s.pair.b * a.n_q * a.heads + s.pair.row0 + first) * kPmDv +
                                  half * 256)
                            : reinterpret_cast<uint8_t*>(
                                  a.part_o + ((int64_t)s.slot * kPmRows + first) * kPmDv + half * 256);
      const int pitch = kPmDv * (s.whole ? 2 : 4);
      const int live = s.pair.rows - first - (lane >> 3);   // rows from this lane's first
      to += (lane >> 3) * pitch + (lane & 7) * 16;
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += step, to += 128) {
#pragma unroll 1
        for (int h = 0; h < step; h += 32) {
          uint32_t ov[32];
          tmem_ld32(tmem + lane_off + c0 + h, ov);
          tmem_ld_wait(ov);
          if (s.whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w4[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w4[u] = bf16x2(__uint_as_float(ov[j + 2 * u]) * inv,
                               __uint_as_float(ov[j + 2 * u + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((h + j) / 8 ^ (lane & 7)) << 4)) =
                  make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(stage + lane * 128 + ((j / 4 ^ (lane & 7)) << 4)) =
                  make_uint4(ov[j], ov[j + 1], ov[j + 2], ov[j + 3]);
          }
        }
        __syncwarp();
        uint4 line[8];                               // of rows 4 i + lane / 8
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          line[i] = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane ^ r) & 7) << 4));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i * 4 < live) *reinterpret_cast<uint4*>(to + (size_t)(i * 4 * pitch)) = line[i];
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(o_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;");   // the join may be set up meanwhile
  // a CTA that gave up lets its last arrivals in the other one land before either ends
  // (otherwise that one has waited for all of them)
  if (limit->abort) {
    const long long t0 = clock64();
    while (clock64() - t0 < kPmGraceCycles) {}
  }
  __syncwarp();
  cluster_sync();
  if (warp == 4) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 512);
  }
}

// Rows whose positions more than one cluster read: o = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^(m_i - max m); rows that see nothing: o = 0, lse = -inf.  A warp takes a quarter of
// the values of ROWS rows at once and holds the weights of their parts, a lane a part, so
// no warp waits for another; either form has eight loads of O in flight a lane, of four rows
// or, where there are few rows, of eight parts of one.  A block takes several rows of a pair
// where there are many pairs (most pairs of a large call were read by one cluster, and
// their blocks only find that out).
template <int ROWS>
__global__ void __launch_bounds__(kPmJoinThreads) paged_mla_join_kernel(const PagedMlaArgs a) {
  constexpr int kHeld = (kPmClusters + 31) / 32, kAhead = 8 / ROWS;
  const int p = blockIdx.x, t = threadIdx.x, lane = t & 31;
  const PmPair pr = pm_pair(a, p);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // all of the attention kernel is done
  if (p == 0 && blockIdx.y == 0 && t < 32) {         // status of the call: the first cluster's
    int code = DSA_OK, where = 0;
    for (int c = t; c < a.clusters && code == DSA_OK; c += 32) {
      code = a.states[2 * c];
      if (code != DSA_OK) where = a.states[2 * c + 1];
    }
    const uint32_t bad = __ballot_sync(0xffffffffu, code != DSA_OK);
    if (bad ? t == __ffs(bad) - 1 : t == 0) {
      a.status[0] = code;
      a.status[1] = where;
    }
  }
  const int first_row = blockIdx.y * a.join_rows;
  const int last_row = min(pr.rows, first_row + a.join_rows);
  if (first_row >= last_row) return;
  const float inf = __int_as_float(0x7f800000);
  const int share = pr.tiles ? a.plan[0] : 1, first = pr.tiles ? a.plan[1 + p] : 0;
  const int c0 = first / share, c1 = (int)(((long long)first + pr.tiles - 1) / share);
  if (pr.tiles && c0 == c1) return;                  // written whole
  // a cluster whose wait ran out leaves its pair's place unwritten
  if (pr.tiles && (first < 0 || c0 >= c1 || c1 >= a.clusters)) return;
  const int n = pr.tiles ? c1 - c0 + 1 : 0;
  for (int row0 = first_row; row0 < last_row; row0 += ROWS) {
    float w[ROWS][kHeld], m[ROWS], l[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int row = min(row0 + r, last_row - 1);
      float2 ml[kHeld];
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        const int i = h * 32 + lane;
        ml[h] = make_float2(-inf, 0.f);
        if (i < n) ml[h] = a.part_ml[(int64_t)(2 * (c0 + i) + (i == 0)) * kPmRows + row];
      }
      m[r] = -inf;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) m[r] = fmaxf(m[r], ml[h].x);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], d));
      l[r] = 0.f;
#pragma unroll
      for (int h = 0; h < kHeld; ++h) {
        w[r][h] = ml[h].x == -inf ? 0.f : ex2(ml[h].x - m[r]);
        l[r] = fmaf(w[r][h], ml[h].y, l[r]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
    }
    float4 o[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4* part = reinterpret_cast<const float4*>(a.part_o) + t;   // 4 values a thread
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
#pragma unroll 1
      for (int i = 32 * h; i < min(n, 32 * h + 32); i += kAhead) {
        float4 v[kAhead][ROWS];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const int c = min(i + k, n - 1), row = min(row0 + r, last_row - 1);
            const int64_t at = (int64_t)(2 * (c0 + c) + (c == 0)) * kPmRows + row;
            v[k][r] = part[at * (kPmDv / 4)];
          }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const float held = __shfl_sync(0xffffffffu, w[r][h], (i + k) & 31);
            const float wi = i + k < n ? held : 0.f;
            o[r].x = fmaf(wi, v[k][r].x, o[r].x);
            o[r].y = fmaf(wi, v[k][r].y, o[r].y);
            o[r].z = fmaf(wi, v[k][r].z, o[r].z);
            o[r].w = fmaf(wi, v[k][r].w, o[r].w);
          }
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (row0 + r >= last_row) break;
      const int64_t grow = (int64_t)pr.b * a.n_q * a.heads + pr.row0 + row0 + r;
      const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
      *(reinterpret_cast<uint2*>(a.out + grow * kPmDv) + t) =
          make_uint2(bf16x2(o[r].x * inv, o[r].y * inv), bf16x2(o[r].z * inv, o[r].w * inv));
      if (t == 0 && a.lse)
        a.lse[grow] = l[r] == 0.f ? -inf : (m[r] + log2f(l[r])) * 0.6931471805599453f;
    }
  }
}

}  // namespace dsa
