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
// A tile of 128 positions runs through rings of operand slots: 9 of 64 positions x 64
// values (K) and 4 of 32 positions x 256 values (V, read in place as an MN-major operand).
//
// Work split.  The tiles of all (sequence, row tile) pairs form one line, cut into equal
// shares, one for each cluster; a pair that more than one cluster meets leaves partial
// (maximum, denominator, output) in the workspace, joined by a second kernel.  So long and
// short sequences, few rows and many use the whole GPU, and the lengths stay on the device.
//
// Softmax: fp32, one thread for a row's 64 of 128 positions; the running maximum is raised
// lazily (by more than 2^8), P is rounded to bf16 for the second product (the matrix
// instructions take both operands in one type), the denominator sums the unrounded values.
// Rows of the cache behind k_len hold anything, also NaN: their scores are replaced and
// their V rows zeroed, as 0 x NaN would not vanish in the product.
#pragma once
#include "cache.cuh"
#include "pair.cuh"

namespace dsa {

constexpr int kPmDqk = 576;
constexpr int kPmDv = 512;
constexpr int kPmRows = 128;            // rows of a tile (64 a CTA)
constexpr int kPmKeys = 128;            // positions of a tile
constexpr int kPmKSlots = 9;            // K chunks of 64 values: one tile
constexpr int kPmVSlots = 4;            // V slices of 32 positions: one tile
constexpr int kPmKBytes = 64 * 128;
constexpr int kPmVBytes = 4 * 32 * 128;
constexpr int kPmQBytes = 9 * 64 * 128;
constexpr int kPmPBytes = 2 * 64 * 128;
constexpr int kPmClusters = 74;         // one CTA an SM
constexpr float kPmLazy = 8.f;          // log2 headroom before the maximum is raised
constexpr int kPmLoaders = 8;           // warps that convert e4m3 rows
constexpr int kPmThreadsRaw = 32 * 7;   // softmax 4, MMA, Q and relay, TMA
constexpr int kPmThreadsCodes = 32 * (6 + kPmLoaders);
constexpr int kPmJoinThreads = 128;

struct PagedMlaArgs {
  CachePlanes c;
  const int32_t* table;    // [batch][max_pages]
  const int32_t* k_len;    // [batch]
  const int32_t* q_len;    // [batch] or null
  int32_t batch, n_q, heads, max_pages;
  int32_t row_tiles;       // row tiles of a sequence of n_q tokens
  int32_t pairs;           // batch * row_tiles
  float scale_log2;        // softmax scale * log2(e)
  uint16_t* out;           // [batch][n_q][heads][512] bf16
  float* lse;              // [batch][n_q][heads] or null
  int32_t* status;
  int32_t* plan;           // [0]: tiles of a share; [1 + pair]: the pair's first tile
  float* part_o;           // [2 * clusters][128][512]
  float2* part_ml;         // [2 * clusters][128] maximum (log2 units), denominator
};

struct PagedMlaTail {
  uint64_t q_full, q_empty, q_ready, o_empty, p_full, pv_done, drain;
  uint64_t k_full[kPmKSlots], k_ready[kPmKSlots], k_empty[kPmKSlots];
  uint64_t v_full[kPmVSlots], v_ready[kPmVSlots], v_empty[kPmVSlots];
  uint64_t s_full[2], s_empty[2];
  uint64_t mates[2];       // the two warps that hold the same 32 rows
  float peer[2][128];      // maxima (and at the end denominators) of a row's two threads
  int32_t start_pair, start_off, count, share;
  uint32_t tmem_base;
  int32_t abort;
};

constexpr size_t paged_mla_smem_bytes() {
  return 1024 + kPmQBytes + kPmKSlots * kPmKBytes + kPmVSlots * kPmVBytes + kPmPBytes +
         sizeof(PagedMlaTail);
}
static_assert(paged_mla_smem_bytes() <= 227 * 1024, "shared memory of one CTA");

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

struct PmWalk {
  int p, off, left, slot;
};
struct PmSegment {
  PmPair pair;
  int p, t0, n, slot;
  bool whole;
};

// The next run of tiles of one pair in a cluster's share.
__device__ __forceinline__ bool pm_next(const PagedMlaArgs& a, PmWalk& w, PmSegment& s) {
  if (w.left <= 0) return false;
  while (w.p < a.pairs) {
    s.pair = pm_pair(a, w.p);
    if (s.pair.tiles > 0) break;
    ++w.p;
  }
  if (w.p >= a.pairs) return false;
  s.p = w.p;
  s.t0 = w.off;
  s.n = min(w.left, s.pair.tiles - w.off);
  s.whole = s.n == s.pair.tiles;
  s.slot = w.slot;
  w.slot |= 1;
  w.left -= s.n;
  w.off += s.n;
  if (w.off == s.pair.tiles) {
    w.off = 0;
    ++w.p;
  }
  return true;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 e4m3 codes times a scale as bf16 (exact where the scale is a power of two).
__device__ __forceinline__ void codes_to_bf16(const uint4& w, float s, uint4& lo, uint4& hi) {
  float v[16];
  e4m3x4_values(w.x, s, v);
  e4m3x4_values(w.y, s, v + 4);
  e4m3x4_values(w.z, s, v + 8);
  e4m3x4_values(w.w, s, v + 12);
  lo = make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
  hi = make_uint4(bf16x2(v[8], v[9]), bf16x2(v[10], v[11]), bf16x2(v[12], v[13]),
                  bf16x2(v[14], v[15]));
}

template <bool CODES>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(CODES ? kPmThreadsCodes : kPmThreadsRaw, 1)
    paged_mla_kernel(const __grid_constant__ CUtensorMap qmap,
                     const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const PagedMlaArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* Qs = smem;                                // [9][64 rows x 128 B]
  uint8_t* Ks = Qs + kPmQBytes;                      // [9][64 positions x 128 B]
  uint8_t* Vs = Ks + kPmKSlots * kPmKBytes;          // [4][4 blocks][32 positions x 128 B]
  uint8_t* Ps = Vs + kPmVSlots * kPmVBytes;          // [2][64 rows x 128 B]
  PagedMlaTail* T = reinterpret_cast<PagedMlaTail*>(Ps + kPmPBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int cl = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  constexpr uint32_t kReady = CODES ? 2 * kPmLoaders : 2;

  if (threadIdx.x == 0) {
    mbar_init(&T->q_full, 1);
    mbar_init(&T->q_empty, 1);
    mbar_init(&T->q_ready, 2);
    mbar_init(&T->o_empty, 8);
    mbar_init(&T->p_full, 8);
    mbar_init(&T->pv_done, 1);
    mbar_init(&T->drain, 1);
    for (int i = 0; i < kPmKSlots; ++i) {
      mbar_init(&T->k_full[i], 1);
      mbar_init(&T->k_ready[i], kReady);
      mbar_init(&T->k_empty[i], 1);
    }
    for (int i = 0; i < kPmVSlots; ++i) {
      mbar_init(&T->v_full[i], 1);
      mbar_init(&T->v_ready[i], kReady);
      mbar_init(&T->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T->s_full[i], 1);
      mbar_init(&T->s_empty[i], 8);
      mbar_init(&T->mates[i], 2);
    }
    T->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&qmap);
    if (!CODES) {
      prefetch_tmap(&kmap);
      prefetch_tmap(&vmap);
    }
  }
  if (warp == 4) pair_tmem_alloc(&T->tmem_base, 512);
  if (warp == 5) {
    // this cluster's share of the line of tiles
    int total = 0;
    for (int p0 = 0; p0 < a.pairs; p0 += 32) {
      const int p = p0 + lane;
      total += __reduce_add_sync(0xffffffffu, p < a.pairs ? pm_pair(a, p).tiles : 0);
    }
    const int share = max(1, (total + clusters - 1) / clusters);
    const int begin = (int)min((long long)cl * share, (long long)total);
    int before = 0, found = -1, off = 0;
    for (int p0 = 0; p0 < a.pairs && found < 0 && begin < total; p0 += 32) {
      const int p = p0 + lane;
      const int n = p < a.pairs ? pm_pair(a, p).tiles : 0;
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
      if (cl == 0 && rank == 0) a.plan[0] = share;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = T->tmem_base;
  volatile int* abort = &T->abort;
  PmWalk walk{T->start_pair, T->start_off, T->count, 2 * cl};
  PmSegment s;

  if (warp == 4) {
    // ----------------------------------------------------------------- MMA --
    // The whole warp waits, one lane issues.
    if (rank == 0) {
      const uint32_t idesc_s = make_idesc<MmaKind::BF16>(kPmKeys);
      const uint32_t idesc_pv = make_idesc<MmaKind::BF16>(256) | (1u << 16);   // B MN-major
      const uint64_t q_desc = make_sdesc(smem_u32(Qs)), k_desc = make_sdesc(smem_u32(Ks));
      const uint64_t p_desc = make_sdesc(smem_u32(Ps)), v_desc = make_sdesc_mn(smem_u32(Vs), 4096);
      uint32_t sc = 0, pc = 0, qc = 0;               // S tiles, PV tiles, segments so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, int where) -> bool {
        const bool w = mbar_wait(bar, parity, abort, a.status, where);
        return __all_sync(0xffffffffu, w);
      };
      auto issue_s = [&]() -> bool {
        const int b = sc & 1;
        if (!wait(&T->s_empty[b], ((sc >> 1) & 1) ^ 1, 51)) return false;
        tc_fence_after();
        const uint32_t d = tmem + 256 + b * 64;
        for (int c = 0; c < kPmKSlots; ++c) {
          if (!wait(&T->k_ready[c], sc & 1, 52)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)           // 16 values
              pair_mma_bf16(d, q_desc + ((c * kPmKBytes + kk * 32) >> 4),
                            k_desc + ((c * kPmKBytes + kk * 32) >> 4), idesc_s, (c | kk) != 0);
            pair_commit(&T->k_empty[c]);
          }
          __syncwarp();
        }
        if (elect_one()) pair_commit(&T->s_full[b]);
        __syncwarp();
        ++sc;
        return true;
      };
      while (ok && pm_next(a, walk, s)) {
        ok = wait(&T->q_ready, qc & 1, 53) && issue_s();
        for (int i = 0; i < s.n && ok; ++i) {
          if (i + 1 < s.n) {
            ok = issue_s();
          } else if (elect_one()) {
            pair_commit(&T->q_empty);
          }
          __syncwarp();
          if (ok && i == 0) ok = wait(&T->o_empty, (qc & 1) ^ 1, 54);
          ok = ok && wait(&T->p_full, pc & 1, 55);
          if (!ok) break;
          tc_fence_after();
          for (int v = 0; v < kPmVSlots && ok; ++v) {
            ok = wait(&T->v_ready[v], pc & 1, 56);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {       // 16 positions
                const int k16 = v * 2 + kk;
                const uint64_t ad =
                    p_desc + (((k16 >> 2) * kPmKBytes + (k16 & 3) * 32) >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h)          // 128 values of each CTA
                  pair_mma_bf16(tmem + h * 128, ad,
                                v_desc + ((v * kPmVBytes + h * 8192 + kk * 2048) >> 4), idesc_pv,
                                (i | k16) != 0);
              }
              pair_commit(&T->v_empty[v]);
              if (v == kPmVSlots - 1) pair_commit(&T->pv_done);
            }
            __syncwarp();
          }
          ++pc;
        }
        ++qc;
      }
      if (!ok) {
        // abort path: the MMAs already issued must end before TMEM is freed
        if (elect_one()) pair_commit(&T->drain);
        __syncwarp();
        mbar_wait_drain(&T->drain, 0);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------- Q, and relay to the MMA --
    // Loads this CTA's 64 rows of q, and tells the MMA thread (in CTA 0) of each
    // operand slot that TMA has filled here, after zeroing V rows behind k_len.
    const uint32_t q_ready = in_cta(&T->q_ready, 0);
    uint32_t kc = 0, vc = 0, qc = 0;
    bool ok = true;
    while (ok && pm_next(a, walk, s)) {
      if (lane == 0) {
        ok = mbar_wait(&T->q_empty, (qc & 1) ^ 1, abort, a.status, 57);
        if (ok) {
          mbar_arrive_expect_tx(&T->q_full, kPmQBytes);
          const int row = s.pair.b * a.n_q * a.heads + s.pair.row0 + 64 * rank;
          for (int c = 0; c < 9; ++c)
            tma_load_2d(Qs + c * kPmKBytes, &qmap, &T->q_full, c * 64, row);
          ok = mbar_wait(&T->q_full, qc & 1, abort, a.status, 58);
          if (ok) mbar_arrive_cluster(q_ready);
          else mbar_wait_drain(&T->q_full, qc & 1);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++qc;
      if constexpr (!CODES) {
        for (int i = -1; i < s.n && ok; ++i) {
          if (i + 1 < s.n) {
            for (int c = 0; c < kPmKSlots && ok; ++c) {
              ok = mbar_wait(&T->k_full[c], kc & 1, abort, a.status, 59);
              ok = __all_sync(0xffffffffu, ok);
              if (ok && lane == 0) mbar_arrive_cluster(in_cta(&T->k_ready[c], 0));
            }
            ++kc;
          }
          if (i >= 0) {
            for (int v = 0; v < kPmVSlots && ok; ++v) {
              ok = mbar_wait(&T->v_full[v], vc & 1, abort, a.status, 60);
              ok = __all_sync(0xffffffffu, ok);
              const int live = s.pair.kl - ((s.t0 + i) * kPmKeys + v * 32);
              if (ok && live < 32) {
                const int from = max(live, 0);
                for (int u = lane; u < (32 - from) * 32; u += 32) {
                  const int r = from + (u >> 5), blk = (u >> 3) & 3, k = u & 7;
                  *reinterpret_cast<uint4*>(Vs + v * kPmVBytes + blk * 4096 + r * 128 + k * 16) =
                      make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
              if (ok && lane == 0) mbar_arrive_cluster(in_cta(&T->v_ready[v], 0));
            }
            ++vc;
          }
        }
      }
    }
    // the last arrival from the MMAs has come before the CTA may end
    if (ok && lane == 0 && qc) mbar_wait(&T->q_empty, (qc & 1) ^ 1, abort, a.status, 70);
  } else if (warp >= 6) {
    // --------------------------------------------------------------- loaders --
    uint32_t kc = 0, vc = 0;                         // tiles of K and V so far
    bool ok = true;
    const int shift = a.c.page_shift;
    if constexpr (!CODES) {
      // one warp: the boxes of each slot, spread over its lanes
      const int kb = min(1 << shift, 64), vb = min(1 << shift, 32);   // rows of a box
      auto pages = [&](int tile) -> int {            // lane j: page of the tile's j-th run
        const int key = tile * kPmKeys + (lane << shift);
        int z = a.c.n_pages;                         // past the end: reads as zeros
        if ((lane << shift) < kPmKeys && key < s.pair.kl) {
          const int p = page_of(a.table + (int64_t)s.pair.b * a.max_pages, key, shift, a.c.n_pages);
          if (p >= 0) z = p;
          else set_status(a.status, DSA_ERR_INVALID, 61);
        }
        return z;
      };
      const int mask = (1 << shift) - 1;
      auto load_k = [&](int tile) {
        const int z0 = pages(tile);
        const int o = 64 * rank + lane * kb;         // lane j < 64 / kb: box j
        const int z = __shfl_sync(0xffffffffu, z0, (o >> shift) & 31);
        const int row = (tile * kPmKeys + o) & mask;
        for (int c = 0; c < kPmKSlots && ok; ++c) {
          if (lane == 0) {
            ok = mbar_wait(&T->k_empty[c], (kc & 1) ^ 1, abort, a.status, 62);
            if (ok) mbar_arrive_expect_tx(&T->k_full[c], kPmKBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok && lane * kb < 64)
            tma_load_3d(Ks + c * kPmKBytes + lane * kb * 128, &kmap, &T->k_full[c], c * 64, row, z);
        }
        ++kc;
      };
      auto load_v = [&](int tile) {
        const int z0 = pages(tile);
        const int per = 32 / vb;                     // boxes of a block
        const int blk = lane / per, j = lane - blk * per;
        for (int v = 0; v < kPmVSlots && ok; ++v) {
          const int o = v * 32 + j * vb;
          const int z = __shfl_sync(0xffffffffu, z0, (o >> shift) & 31);
          if (lane == 0) {
            ok = mbar_wait(&T->v_empty[v], (vc & 1) ^ 1, abort, a.status, 63);
            if (ok) mbar_arrive_expect_tx(&T->v_full[v], kPmVBytes);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok && blk < 4)
            tma_load_3d(Vs + v * kPmVBytes + blk * 4096 + j * vb * 128, &vmap, &T->v_full[v],
                        rank * 256 + blk * 64, (tile * kPmKeys + o) & mask, z);
        }
        ++vc;
      };
      while (ok && pm_next(a, walk, s)) {
        load_k(s.t0);
        for (int i = 0; i < s.n && ok; ++i) {
          if (i + 1 < s.n) load_k(s.t0 + i + 1);
          if (ok) load_v(s.t0 + i);
        }
      }
      if (lane == 0) {
        // the last copies have landed (also on the abort path), and the last arrivals
        // from the MMAs have come, before the CTA may end
        for (int c = 0; c < kPmKSlots && kc; ++c)
          if (ok) mbar_wait(&T->k_empty[c], (kc & 1) ^ 1, abort, a.status, 64);
          else mbar_wait_drain(&T->k_full[c], (kc & 1) ^ 1, kWaitCycles / 64);
        for (int v = 0; v < kPmVSlots && vc; ++v)
          if (ok) mbar_wait(&T->v_empty[v], (vc & 1) ^ 1, abort, a.status, 65);
          else mbar_wait_drain(&T->v_full[v], (vc & 1) ^ 1, kWaitCycles / 64);
      }
    } else {
      // eight warps: 16 codes a thread and load, converted on the way to the slots
      const int c = threadIdx.x - 192;
      const int krow = c >> 2, ku = c & 3;           // K chunk: row, run of 16 values
      const int vrow = c >> 3, vu = c & 7;           // V slice: row, runs vu and vu + 8
      uint4 kreg[8], rreg[2], vreg[8];
      float ksc[4], vsc[8];
      auto load_k = [&](int tile) {
        const int key = tile * kPmKeys + 64 * rank + krow;
        int page = -1;
        if (key < s.pair.kl) {
          page = page_of(a.table + (int64_t)s.pair.b * a.max_pages, key, shift, a.c.n_pages);
          if (page < 0) set_status(a.status, DSA_ERR_INVALID, 61);
        }
        const int row = key & ((1 << shift) - 1);
        const uint8_t* codes = a.c.codes + page * a.c.codes_ps + row * kPmDv + ku * 16;
        const float* sc = a.c.scale + page * a.c.scale_ps + row * 4;
        const __nv_bfloat16* raw = a.c.raw + page * a.c.raw_ps + row * 64 + ku * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          kreg[i] = page >= 0 ? *reinterpret_cast<const uint4*>(codes + i * 64) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rreg[i] = page >= 0 ? *reinterpret_cast<const uint4*>(raw + i * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) ksc[i] = page >= 0 ? sc[i] : 0.f;
      };
      auto load_v = [&](int tile) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int key = tile * kPmKeys + v * 32 + vrow;
          int page = -1;
          if (key < s.pair.kl)
            page = page_of(a.table + (int64_t)s.pair.b * a.max_pages, key, shift, a.c.n_pages);
          const int row = key & ((1 << shift) - 1);
          const uint8_t* codes = a.c.codes + page * a.c.codes_ps + row * kPmDv + rank * 256 + vu * 16;
          const float* sc = a.c.scale + page * a.c.scale_ps + row * 4 + rank * 2;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            vreg[2 * v + h] = page >= 0 ? *reinterpret_cast<const uint4*>(codes + h * 128)
                                        : make_uint4(0, 0, 0, 0);
            vsc[2 * v + h] = page >= 0 ? sc[h] : 0.f;
          }
        }
      };
      auto ready = [&](uint64_t* bar) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(in_cta(bar, 0));
      };
      auto fill_k = [&]() {
#pragma unroll
        for (int i = 0; i < kPmKSlots; ++i) {
          if (ok) ok = mbar_wait(&T->k_empty[i], (kc & 1) ^ 1, abort, a.status, 62);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint4 lo, hi;
          if (i < 8) {
            codes_to_bf16(kreg[i & 7], ksc[(i & 7) >> 1], lo, hi);
          } else {
            lo = rreg[0];
            hi = rreg[1];
          }
          uint8_t* dst = Ks + i * kPmKBytes + krow * 128;
          *reinterpret_cast<uint4*>(dst + (((2 * ku) ^ (krow & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(dst + (((2 * ku + 1) ^ (krow & 7)) << 4)) = hi;
          ready(&T->k_ready[i]);
        }
        ++kc;
      };
      auto fill_v = [&]() {
#pragma unroll
        for (int v = 0; v < kPmVSlots; ++v) {
          if (ok) ok = mbar_wait(&T->v_empty[v], (vc & 1) ^ 1, abort, a.status, 63);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int u = vu + 8 * h;                // 16 values of the CTA's 256
            uint4 lo, hi;
            codes_to_bf16(vreg[2 * v + h], vsc[2 * v + h], lo, hi);
            uint8_t* dst = Vs + v * kPmVBytes + (u >> 2) * 4096 + vrow * 128;
            const int k = 2 * (u & 3);
            *reinterpret_cast<uint4*>(dst + ((k ^ (vrow & 7)) << 4)) = lo;
            *reinterpret_cast<uint4*>(dst + (((k + 1) ^ (vrow & 7)) << 4)) = hi;
          }
          ready(&T->v_ready[v]);
        }
        ++vc;
      };
      while (ok && pm_next(a, walk, s)) {
        load_k(s.t0);
        for (int i = -1; i < s.n && ok; ++i) {
          if (i >= 0) load_v(s.t0 + i);
          if (i + 1 < s.n) fill_k();
          if (i + 2 < s.n) load_k(s.t0 + i + 2);
          if (i >= 0 && ok) fill_v();
        }
      }
      if (ok && threadIdx.x == 192) {
        for (int i = 0; i < kPmKSlots && kc; ++i)
          mbar_wait(&T->k_empty[i], (kc & 1) ^ 1, abort, a.status, 64);
        for (int v = 0; v < kPmVSlots && vc; ++v)
          mbar_wait(&T->v_empty[v], (vc & 1) ^ 1, abort, a.status, 65);
      }
    }
  } else {
    // --------------------------------------------------- softmax and output --
    // Thread t of 128 = TMEM lane t: row t & 63 of this CTA, positions (or values) of
    // half t >> 6.  Warps w and w + 2 hold the two halves of the same rows.
    const int t = threadIdx.x, half = t >> 6, row = t & 63;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const float inf = __int_as_float(0x7f800000);
    const uint32_t p_full = in_cta(&T->p_full, 0), o_empty = in_cta(&T->o_empty, 0);
    const uint32_t s_empty[2] = {in_cta(&T->s_empty[0], 0), in_cta(&T->s_empty[1], 0)};
    uint32_t sc = 0, xc = 0;                         // tiles, exchanges so far
    bool ok = true;
    // v of this thread and its mate (bounded, as every wait: the mate may have given up)
    auto exchange = [&](float v) -> float {
      T->peer[xc & 1][t] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&T->mates[warp & 1]);
      ok = mbar_wait(&T->mates[warp & 1], xc & 1, abort, a.status, 69);
      ok = __all_sync(0xffffffffu, ok);
      return T->peer[xc++ & 1][t ^ 64];
    };
    while (ok && pm_next(a, walk, s)) {
      const int r = s.pair.row0 + rank * 64 + row;   // row of the sequence
      const bool mine = rank * 64 + row < s.pair.rows;
      // positions this row sees: [0, lim)
      const int lim = mine ? max(0, s.pair.kl - s.pair.ql + r / a.heads + 1) : 0;
      float m_run = -inf, l_run = 0.f;
      for (int i = 0; i < s.n; ++i, ++sc) {
        ok = mbar_wait(&T->s_full[sc & 1], (sc >> 1) & 1, abort, a.status, 66);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        float x[64];
        {
          uint32_t sv[2][32];
          const uint32_t at = tmem + lane_off + 256 + (sc & 1) * 64;
          tmem_ld32(at, sv[0]);
          tmem_ld32(at + 32, sv[1]);
          tmem_ld_wait(sv[0]);
          tmem_ld_wait(sv[1]);
#pragma unroll
          for (int j = 0; j < 64; ++j) x[j] = __uint_as_float(sv[j >> 5][j & 31]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(s_empty[sc & 1]);
        const int seen = lim - ((s.t0 + i) * kPmKeys + half * 64);   // of these 64
        float mt = -inf;
        if (__all_sync(0xffffffffu, seen >= 64)) {
#pragma unroll
          for (int j = 0; j < 64; ++j) mt = fmaxf(mt, x[j] * a.scale_log2);
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) {
            if (j >= seen) x[j] = -inf;
            else mt = fmaxf(mt, x[j] * a.scale_log2);
          }
        }
        mt = fmaxf(mt, exchange(mt));
        if (!ok) break;
        // P and O are free once the previous PV is complete
        if (i > 0) {
          ok = mbar_wait(&T->pv_done, (sc - 1) & 1, abort, a.status, 67);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        float f = 1.f;
        if (mt > m_run + kPmLazy || (m_run == -inf && mt > -inf)) {
          if (m_run > -inf) {
            f = ex2(m_run - mt);
            l_run *= f;
          }
          m_run = mt;
        }
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
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
        // positions the row does not see weigh 0, also while its maximum is still -inf
        const float m_sub = m_run == -inf ? 0.f : m_run;
        uint8_t* prow = Ps + half * kPmKBytes + row * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t w4[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int j = c * 8 + u * 2;
            const float p0 = ex2(fmaf(x[j], a.scale_log2, -m_sub));
            const float p1 = ex2(fmaf(x[j + 1], a.scale_log2, -m_sub));
            l_run += p0 + p1;
            w4[u] = bf16x2(p0, p1);
          }
          *reinterpret_cast<uint4*>(prow + ((c ^ (row & 7)) << 4)) =
              make_uint4(w4[0], w4[1], w4[2], w4[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(p_full);
      }
      if (!ok) break;
      ok = mbar_wait(&T->pv_done, (sc - 1) & 1, abort, a.status, 68);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      l_run += exchange(l_run);
      if (!ok) break;
      const int64_t grow = (int64_t)s.pair.b * a.n_q * a.heads + r;
      const int64_t prow = (int64_t)s.slot * kPmRows + rank * 64 + row;
      if (mine && half == 0) {
        if (!s.whole) a.part_ml[prow] = make_float2(m_run, l_run);
        else if (a.lse)
          a.lse[grow] = l_run == 0.f ? -inf : (m_run + log2f(l_run)) * 0.6931471805599453f;
        if (rank == 0 && row == 0 && s.t0 == 0) a.plan[1 + s.p] = cl * T->share + (T->count - walk.left - s.n);
      }
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t ov[32];
        tmem_ld32(tmem + lane_off + c0, ov);
        tmem_ld_wait(ov);
        if (mine) {
          if (s.whole) {
            uint16_t* dst = a.out + grow * kPmDv + half * 256 + c0;
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w4[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w4[u] = bf16x2(__uint_as_float(ov[j + 2 * u]) * inv,
                               __uint_as_float(ov[j + 2 * u + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + j) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          } else {
            float* dst = a.part_o + prow * kPmDv + half * 256 + c0;
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(dst + j) = make_uint4(ov[j], ov[j + 1], ov[j + 2], ov[j + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(o_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  __syncwarp();
  cluster_sync();
  if (warp == 4) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, 512);
  }
}

// Rows whose positions more than one cluster read: o = sum_i w_i O_i / sum_i w_i l_i with
// w_i = 2^(m_i - max m); rows that see nothing: o = 0, lse = -inf.  One block a row.
__global__ void __launch_bounds__(kPmJoinThreads) paged_mla_join_kernel(const PagedMlaArgs a) {
  __shared__ float w[2 * kPmClusters];
  __shared__ float red[2][kPmJoinThreads / 32];
  const int p = blockIdx.x, row = blockIdx.y, t = threadIdx.x;
  const PmPair pr = pm_pair(a, p);
  if (row >= pr.rows) return;
  const int64_t grow = (int64_t)pr.b * a.n_q * a.heads + pr.row0 + row;
  uint2* out = reinterpret_cast<uint2*>(a.out + grow * kPmDv) + t;
  const float inf = __int_as_float(0x7f800000);
  if (pr.tiles == 0) {
    *out = make_uint2(0, 0);
    if (t == 0 && a.lse) a.lse[grow] = -inf;
    return;
  }
  const int share = a.plan[0], first = a.plan[1 + p];
  const int c0 = first / share, c1 = (first + pr.tiles - 1) / share;
  if (c0 == c1) return;                              // written whole
  const int n = c1 - c0 + 1;
  // the pair's run in cluster c is that cluster's first unless it starts inside its share
  const int head = first > c0 * share ? 1 : 0;
  float m = -inf;
  float2 ml = make_float2(-inf, 0.f);
  if (t < n) {
    const int slot = 2 * (c0 + t) + (t == 0 ? head : 0);
    ml = a.part_ml[(int64_t)slot * kPmRows + row];
    m = ml.x;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((t & 31) == 0) red[0][t >> 5] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float wt = ml.x == -inf ? 0.f : ex2(ml.x - m);
  float l = wt * ml.y;
  if (t < n) w[t] = wt;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if ((t & 31) == 0) red[1][t >> 5] = l;
  __syncthreads();
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const int slot = 2 * (c0 + i) + (i == 0 ? head : 0);
    const float4 v =
        *(reinterpret_cast<const float4*>(a.part_o + ((int64_t)slot * kPmRows + row) * kPmDv) + t);
    const float wi = w[i];
    o.x = fmaf(wi, v.x, o.x);
    o.y = fmaf(wi, v.y, o.y);
    o.z = fmaf(wi, v.z, o.z);
    o.w = fmaf(wi, v.w, o.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *out = make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
  if (t == 0 && a.lse) a.lse[grow] = l == 0.f ? -inf : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace dsa
