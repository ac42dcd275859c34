// layer.cu — C ABI of the steps around a cached DSA layer (see include/dsaidx.h):
// rotary positions, the paged cache and latent attention over it.  Host code here
// only validates arguments, plans the launch and launches the kernels.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dsaidx.h"
#include "cache.cuh"
#include "common.cuh"
#include "host.cuh"
#include "paged_mla.cuh"

using namespace dsa;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launch_status() { return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

// ---------------------------------------------------------- rotary positions --
// Whether the places t * ts + h * hs + d of a [tokens][heads][dim] array are distinct.
bool distinct(int64_t tokens, int64_t heads, int64_t dim, int64_t ts, int64_t hs) {
  if (ts < 0 || hs < 0) return false;
  if (tokens == 1 && heads == 1) return true;
  if (tokens == 1) return hs >= dim;
  if (heads == 1) return ts >= dim;
  const bool heads_inside = hs >= dim && ts >= (heads - 1) * hs + dim;
  const bool tokens_inside = ts >= dim && hs >= (tokens - 1) * ts + dim;
  return heads_inside || tokens_inside;
}

template <typename T>
int launch_rope(RopeArgs& a, int dim, bool vec, bool inter, bool in_place, cudaStream_t st) {
  const int n = vec ? RowType<T>::kVec : 1;
  a.pairs = vec && inter ? a.rot / n : a.rot / 2 / n;
  a.units = a.pairs + (in_place ? 0 : (dim - a.rot) / n);
  // r / units as the upper word of r ceil(2^32 / units): exact while r units < 2^32
  if ((uint64_t)a.heads * a.units >= 1ull << 31) return DSA_ERR_UNSUPPORTED;
  a.per_unit = a.units > 1 && (uint64_t)a.heads * a.units * a.units < 1ull << 32
                   ? (uint32_t)(((1ull << 32) + a.units - 1) / a.units)
                   : 0;
  // a block takes about 768 units (three a thread): several tokens of few heads, or a
  // part of one token's heads
  const int64_t per_token = (int64_t)a.heads * a.units;
  const int64_t target = kRopeThreads * kRopeBatch;
  int64_t tpb = target / per_token;
  tpb = tpb < 1 ? 1 : (tpb > 32 ? 32 : tpb);
  int64_t parts = tpb > 1 ? 1 : (per_token + target - 1) / target;
  if (parts > 65535) parts = 65535;
  a.tpb = (int32_t)tpb;
  a.span = (int32_t)((per_token + parts - 1) / parts);
  const int64_t blocks = (a.n_tokens + tpb - 1) / tpb;
  if (blocks > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)parts);
  const size_t smem = (size_t)tpb * (a.rot / 2) * sizeof(float2);   // <= 64 KB
  void (*kern)(const RopeArgs) =
      vec ? (inter ? rope_kernel<T, true, true> : rope_kernel<T, true, false>)
          : (inter ? rope_kernel<T, false, true> : rope_kernel<T, false, false>);
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return DSA_ERR_CUDA;
  kern<<<grid, kRopeThreads, smem, st>>>(a);
  return launch_status();
}

// -------------------------------------------------------------- paged cache --
int page_shift(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

int validate_cache(const dsa_cache* c) {
  if (!c) return DSA_ERR_INVALID;
  if (c->n_pages < 1 || c->dim_q < 0 || c->dim_raw < 0 || c->dim_q + (int64_t)c->dim_raw < 1)
    return DSA_ERR_INVALID;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) ||
      c->dim_q % 128 || c->dim_raw % 8 || c->dim_q > 4096 || c->dim_raw > 4096)
    return DSA_ERR_UNSUPPORTED;
  if (c->dim_q) {
    if (!c->codes || !c->scale) return DSA_ERR_INVALID;
    if (!aligned16(c->codes) || !aligned(c->scale, 4) || c->codes_page_stride % 16)
      return DSA_ERR_INVALID;
    if (c->codes_page_stride < (int64_t)c->page_size * c->dim_q ||
        c->scale_page_stride < (int64_t)c->page_size * (c->dim_q / 128))
      return DSA_ERR_INVALID;
  } else if (c->codes || c->scale) {
    return DSA_ERR_INVALID;
  }
  if (c->dim_raw) {
    if (!c->raw || !aligned16(c->raw) || c->raw_page_stride % 8 ||
        c->raw_page_stride < (int64_t)c->page_size * c->dim_raw)
      return DSA_ERR_INVALID;
  } else if (c->raw) {
    return DSA_ERR_INVALID;
  }
  return DSA_OK;
}

CachePlanes planes(const dsa_cache* c) {
  CachePlanes p{};
  p.codes = reinterpret_cast<uint8_t*>(c->codes);
  p.scale = c->scale;
  p.raw = reinterpret_cast<__nv_bfloat16*>(c->raw);
  p.codes_ps = c->codes_page_stride;
  p.scale_ps = c->scale_page_stride;
  p.raw_ps = c->raw_page_stride;
  p.n_pages = c->n_pages;
  p.page_shift = page_shift(c->page_size);
  p.dim_q = c->dim_q;
  p.dim_raw = c->dim_raw;
  return p;
}

int chunks_of(const dsa_cache* c) { return c->dim_q / 128 + (c->dim_raw + 127) / 128; }

// Whether 8 lanes hold chunks of several rows at once and not several of one.
bool few_chunks(int chunks) { return chunks < 4; }
unsigned row_blocks(int64_t rows, int at_once) {
  const int span = kCacheUnits * at_once;
  return (unsigned)((rows + span - 1) / span);
}

typedef void (*WriteKernel)(const CacheWriteArgs);
template <typename T>
WriteKernel write_kernel(bool vec, bool turn, bool few) {
  if (few)
    return vec ? (turn ? cache_write_kernel<T, true, true, 2> : cache_write_kernel<T, true, false, 2>)
               : (turn ? cache_write_kernel<T, false, true, 2> : cache_write_kernel<T, false, false, 2>);
  return vec ? (turn ? cache_write_kernel<T, true, true, 1> : cache_write_kernel<T, true, false, 1>)
             : (turn ? cache_write_kernel<T, false, true, 1> : cache_write_kernel<T, false, false, 1>);
}

// Arguments shared by the two reads; *grid: x is 0 where there is nothing to read, z
// counts the threads' runs of chunks.
int read_args(const dsa_cache* c, const int32_t* table, int32_t batch, int32_t max_pages,
              int32_t n_k, const int32_t* k_len, void* out, bool few, int at_once,
              CacheReadArgs* a, dim3* grid) {
  const int v = validate_cache(c);
  if (v != DSA_OK) return v;
  if (batch < 1 || n_k < 0 || max_pages < 0) return DSA_ERR_INVALID;
  if ((int64_t)max_pages * c->page_size < n_k) return DSA_ERR_INVALID;
  if (batch > 65535 || n_k > (1 << 30)) return DSA_ERR_UNSUPPORTED;
  *grid = dim3(row_blocks(n_k, few ? 4 : 1), (unsigned)batch,
               few ? chunks_of(c) : (chunks_of(c) + at_once - 1) / at_once);
  if (n_k == 0) return DSA_OK;                       // (nothing to read has no address)
  if (!table || !out) return DSA_ERR_INVALID;
  if (!aligned(table, 4) || !aligned(k_len, 4) || !aligned16(out)) return DSA_ERR_INVALID;
  a->c = planes(c);
  a->table = table;
  a->k_len = k_len;
  a->batch = batch;
  a->max_pages = max_pages;
  a->n_k = n_k;
  a->out = out;
  return DSA_OK;
}

// -------------------------------------------------------- latent attention --
// 2-D map over the query rows [rows][576] bf16: box of 64 values x 64 rows, 128-byte
// swizzle; rows past the end read as zeros.
bool map_query(CUtensorMap* m, const void* base, uint64_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kPmDqk, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kPmDqk * 2};
  cuuint32_t box[2] = {64, 64};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D map over the bf16 plane [pages][page][9 chunks of 64 values]: box of 64 values x
// box_rows x box_chunks x one page, so a copy lands as whole chunks one after another; a
// page past the end reads as zeros.
bool map_pages(CUtensorMap* m, const dsa_cache* c, uint32_t box_rows, uint32_t box_chunks) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)c->page_size, (cuuint64_t)(kPmDqk / 64),
                        (cuuint64_t)c->n_pages};
  cuuint64_t strides[3] = {(cuuint64_t)kPmDqk * 2, 128, (cuuint64_t)c->raw_page_stride * 2};
  cuuint32_t box[4] = {64, box_rows, box_chunks, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, c->raw, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map over rows of a plane [pages][page][width bytes or words]: box of 64 or 128 bytes x
// box_rows x one page, swizzled over as many; a page past the end reads as zeros.
bool map_rows(CUtensorMap* m, const dsa_cache* c, bool codes, uint32_t box_bytes,
              uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t esz = codes ? 1 : 2, width = codes ? kPmDv : kPmDqk - kPmDv;
  const uint64_t stride = (uint64_t)(codes ? c->codes_page_stride : c->raw_page_stride);
  cuuint64_t dims[3] = {width, (cuuint64_t)c->page_size, (cuuint64_t)c->n_pages};
  cuuint64_t strides[2] = {width * esz, stride * esz};
  cuuint32_t box[3] = {(cuuint32_t)(box_bytes / esz), box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            codes ? c->codes : c->raw, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct PagedMlaPlan {
  int row_tiles, clusters;
  int64_t pairs;
  size_t off_states, off_plan, off_ml, off_o, bytes;
};

int plan_paged_mla(const dsa_paged_mla_problem* p, PagedMlaPlan* pl) {
  if (!p) return DSA_ERR_INVALID;
  if (p->batch < 1 || p->n_q < 1 || p->heads < 1 || p->max_pages < 1 || p->page_size < 1)
    return DSA_ERR_INVALID;
  if (p->heads > 128 || p->dim_qk != kPmDqk || p->dim_v != kPmDv || p->page_size > 4096 ||
      (int64_t)p->max_pages * p->page_size > (1ll << 24))
    return DSA_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)p->n_q * p->heads;
  const int64_t row_tiles = (rows + kPmRows - 1) / kPmRows;
  pl->pairs = row_tiles * p->batch;
  const int64_t key_tiles = ((int64_t)p->max_pages * p->page_size + kPmKeys - 1) / kPmKeys;
  if (rows * p->batch > 0x7fffffffll || pl->pairs * key_tiles >= 1 << 28)
    return DSA_ERR_UNSUPPORTED;
  pl->row_tiles = (int)row_tiles;
  const int64_t tiles = pl->pairs * key_tiles;
  pl->clusters = tiles < kPmClusters ? (int)tiles : kPmClusters;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  pl->off_states = kWsHeaderBytes;
  pl->off_plan = pl->off_states + up((size_t)pl->clusters * 2 * sizeof(int32_t));
  pl->off_ml = pl->off_plan + up((size_t)(1 + pl->pairs) * sizeof(int32_t));
  pl->off_o = pl->off_ml + up((size_t)2 * pl->clusters * kPmRows * sizeof(float2));
  pl->bytes = pl->off_o + (size_t)2 * pl->clusters * kPmRows * kPmDv * sizeof(float);
  return DSA_OK;
}

}  // namespace

extern "C" {

int dsa_rope_frequencies(int32_t rot_dim, double base, int32_t scaling, double factor,
                         double original_len, double beta_fast, double beta_slow, double* out) {
  if (!out || rot_dim < 2 || !(base > 1.0) || !isfinite(base)) return DSA_ERR_INVALID;
  if ((rot_dim & 1) || rot_dim > 512 || scaling < DSA_ROPE_PLAIN || scaling > DSA_ROPE_YARN)
    return DSA_ERR_UNSUPPORTED;
  if (scaling != DSA_ROPE_PLAIN && (!(factor > 0.0) || !isfinite(factor))) return DSA_ERR_INVALID;
  double lo = 0, hi = 0;
  if (scaling == DSA_ROPE_YARN) {
    if (!(original_len > 0.0) || !isfinite(original_len) || !(beta_fast > 0.0) ||
        !(beta_slow > 0.0) || !isfinite(beta_fast) || !isfinite(beta_slow))
      return DSA_ERR_INVALID;
    const double two_pi = 6.283185307179586477;
    lo = floor(rot_dim * log(original_len / (two_pi * beta_fast)) / (2.0 * log(base)));
    hi = ceil(rot_dim * log(original_len / (two_pi * beta_slow)) / (2.0 * log(base)));
    lo = lo < 0 ? 0 : lo;
    hi = hi > rot_dim - 1 ? rot_dim - 1 : hi;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot_dim);
    double g = scaling == DSA_ROPE_LINEAR ? 1.0 : 0.0;
    if (scaling == DSA_ROPE_YARN) {
      g = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      g = g < 0 ? 0 : (g > 1 ? 1 : g);
    }
    out[i] = scaling == DSA_ROPE_PLAIN ? f : f * (g / factor + 1.0 - g);
  }
  return DSA_OK;
}

int dsa_rope(const dsa_rope_problem* p, const void* x, const int32_t* pos, const double* freq,
             void* out, void* stream) {
  if (!p || p->n_tokens < 0 || p->heads < 1 || p->dim < 1 || p->offset < 0 || p->rot_dim < 2)
    return DSA_ERR_INVALID;
  if (p->dtype != DSA_BF16 && p->dtype != DSA_F32) return DSA_ERR_UNSUPPORTED;
  if ((p->rot_dim & 1) || p->rot_dim > 512 || p->dim > 65536 || p->heads > 65536)
    return DSA_ERR_UNSUPPORTED;
  if ((int64_t)p->offset + p->rot_dim > p->dim || !isfinite(p->mscale)) return DSA_ERR_INVALID;
  if (p->n_tokens == 0) return DSA_OK;
  if (!x || !pos || !freq || !out) return DSA_ERR_INVALID;
  const size_t esz = p->dtype == DSA_BF16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(out, esz) || !aligned(pos, 4) || !aligned(freq, 8))
    return DSA_ERR_INVALID;
  if (!distinct(p->n_tokens, p->heads, p->dim, p->out_token_stride, p->out_head_stride))
    return DSA_ERR_INVALID;
  const bool same = p->x_token_stride == p->out_token_stride &&
                    p->x_head_stride == p->out_head_stride;
  if (x == out && !same) return DSA_ERR_INVALID;
  RopeArgs a{};
  a.x = x;
  a.out = out;
  a.pos = pos;
  a.freq = freq;
  a.n_tokens = p->n_tokens;
  a.x_ts = p->x_token_stride;
  a.x_hs = p->x_head_stride;
  a.o_ts = p->out_token_stride;
  a.o_hs = p->out_head_stride;
  a.heads = p->heads;
  a.offset = p->offset;
  a.rot = p->rot_dim;
  a.mscale = p->mscale;
  a.sign = p->flags & DSA_FLAG_INVERSE ? -1.f : 1.f;
  const bool inter = (p->flags & DSA_FLAG_INTERLEAVED) != 0;
  // 16-byte vectors where every head's row, the rotated part and (halves) its middle
  // start on one
  const int n = (int)(16 / esz);
  const bool vec = aligned16(x) && aligned16(out) && p->dim % n == 0 && p->offset % n == 0 &&
                   (inter ? p->rot_dim % n == 0 : p->rot_dim % (2 * n) == 0) &&
                   a.x_ts % n == 0 && a.x_hs % n == 0 && a.o_ts % n == 0 && a.o_hs % n == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == DSA_BF16 ? launch_rope<__nv_bfloat16>(a, p->dim, vec, inter, x == out, st)
                              : launch_rope<float>(a, p->dim, vec, inter, x == out, st);
}

int dsa_cache_write(const dsa_cache* c, const void* x, int32_t x_dtype, int64_t x_stride,
                    int64_t n_tokens, const int64_t* slots, const dsa_rope_problem* rope,
                    const int32_t* pos, const double* freq, uint32_t flags, void* stream) {
  const int v = validate_cache(c);
  if (v != DSA_OK) return v;
  if (n_tokens < 0 || x_stride < 0) return DSA_ERR_INVALID;
  if (x_dtype != DSA_BF16 && x_dtype != DSA_F32) return DSA_ERR_UNSUPPORTED;
  if (rope) {
    if (rope->offset < 0 || rope->rot_dim < 2 ||
        (int64_t)rope->offset + rope->rot_dim > c->dim_q + c->dim_raw || !isfinite(rope->mscale))
      return DSA_ERR_INVALID;
    if (rope->offset % 8 || rope->rot_dim % 16 || rope->rot_dim > 512) return DSA_ERR_UNSUPPORTED;
    if (n_tokens && (!pos || !freq)) return DSA_ERR_INVALID;
  } else if (pos || freq) {
    return DSA_ERR_INVALID;
  }
  if (n_tokens == 0) return DSA_OK;
  const size_t esz = x_dtype == DSA_BF16 ? 2 : 4;
  if (!x || !slots || !aligned(x, esz) || !aligned(slots, 8) || !aligned(pos, 4) ||
      !aligned(freq, 8))
    return DSA_ERR_INVALID;
  CacheWriteArgs a{};
  a.c = planes(c);
  a.x = x;
  a.x_ts = x_stride;
  a.slots = slots;
  a.n_tokens = n_tokens;
  if (rope) {
    a.pos = pos;
    a.freq = freq;
    a.offset = rope->offset;
    a.rot = rope->rot_dim;
    a.inter = (rope->flags & DSA_FLAG_INTERLEAVED) != 0;
    a.mscale = rope->mscale;
    a.sign = rope->flags & DSA_FLAG_INVERSE ? -1.f : 1.f;
  }
  a.pow2 = (flags & DSA_FLAG_POW2_SCALE) != 0;
  if (n_tokens > 0x7fffffffll) return DSA_ERR_UNSUPPORTED;
  a.items = chunks_of(c);
  const bool few = few_chunks(a.items);
  const bool vec = aligned16(x) && x_stride % (int64_t)(16 / esz) == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kern = x_dtype == DSA_BF16 ? write_kernel<__nv_bfloat16>(vec, rope != nullptr, few)
                                  : write_kernel<float>(vec, rope != nullptr, few);
  const dim3 grid(row_blocks(n_tokens, few ? 2 : 1),
                  few ? a.items : (a.items + kCacheBatch - 1) / kCacheBatch);
  kern<<<grid, kCacheThreads, 0, st>>>(a);
  return launch_status();
}

int dsa_cache_read(const dsa_cache* c, const int32_t* block_table, int32_t batch,
                   int32_t max_pages, int32_t n_k, const int32_t* k_len, void* out,
                   int32_t out_dtype, void* stream) {
  CacheReadArgs a{};
  dim3 blocks;
  const bool few = c && few_chunks(chunks_of(c));
  const int v = read_args(c, block_table, batch, max_pages, n_k, k_len, out, few, kReadBatch, &a,
                          &blocks);
  if (v != DSA_OK) return v;
  if (out_dtype != DSA_BF16 && out_dtype != DSA_F32) return DSA_ERR_UNSUPPORTED;
  if (blocks.x == 0) return DSA_OK;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto kern = out_dtype == DSA_BF16
                  ? (few ? cache_read_kernel<__nv_bfloat16, 4> : cache_read_kernel<__nv_bfloat16, 1>)
                  : (few ? cache_read_kernel<float, 4> : cache_read_kernel<float, 1>);
  kern<<<blocks, kCacheThreads, 0, st>>>(a);
  return launch_status();
}

int dsa_cache_read_codes(const dsa_cache* c, const int32_t* block_table, int32_t batch,
                         int32_t max_pages, int32_t n_k, const int32_t* k_len, void* out,
                         float* out_scale, void* stream) {
  CacheReadArgs a{};
  dim3 blocks;
  const bool few = c && few_chunks(chunks_of(c));
  const int v = read_args(c, block_table, batch, max_pages, n_k, k_len, out, few, kCacheBatch, &a,
                          &blocks);
  if (v != DSA_OK) return v;
  if (c->dim_q == 0) return DSA_ERR_INVALID;
  if (c->dim_raw) return DSA_ERR_UNSUPPORTED;
  if (blocks.x == 0) return DSA_OK;
  if (!out_scale || !aligned(out_scale, 4)) return DSA_ERR_INVALID;
  a.out_scale = out_scale;
  auto kern = few ? cache_read_codes_kernel<4> : cache_read_codes_kernel<1>;
  kern<<<blocks, kCacheThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return launch_status();
}

int dsa_paged_mla_workspace_size(const dsa_paged_mla_problem* p, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID;
  PagedMlaPlan pl{};
  const int v = plan_paged_mla(p, &pl);
  if (v != DSA_OK) return v;
  *bytes = pl.bytes;
  return DSA_OK;
}

int dsa_paged_mla(const dsa_paged_mla_problem* p, const dsa_cache* c, const void* q,
                  const int32_t* block_table, const int32_t* k_len, const int32_t* q_len,
                  void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                  void* stream) {
  PagedMlaPlan pl{};
  int v = plan_paged_mla(p, &pl);
  if (v != DSA_OK) return v;
  v = validate_cache(c);
  if (v != DSA_OK) return v;
  if (c->page_size != p->page_size) return DSA_ERR_INVALID;
  const bool codes = c->dim_q == kPmDv && c->dim_raw == kPmDqk - kPmDv;
  if (!codes && !(c->dim_q == 0 && c->dim_raw == kPmDqk)) return DSA_ERR_UNSUPPORTED;
  if (!q || !block_table || !k_len || !out) return DSA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(out) || !aligned(block_table, 4) || !aligned(k_len, 4) ||
      !aligned(q_len, 4) || !aligned(out_lse, 4))
    return DSA_ERR_INVALID;
  if (!(p->scale > 0.f) || !(p->scale < 1.0e38f)) return DSA_ERR_INVALID;
  if (!workspace || workspace_bytes < pl.bytes) return DSA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DSA_ERR_INVALID;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  CUtensorMap qm{}, km{}, vm{}, rm{};
  if (!map_query(&qm, q, (uint64_t)p->batch * p->n_q * p->heads)) return DSA_ERR_CUDA;
  const uint32_t page = (uint32_t)c->page_size;
  if (codes) {
    if (!map_rows(&km, c, true, 64, page < 64 ? page : 64) ||
        !map_rows(&vm, c, true, 128, page < 32 ? page : 32) ||
        !map_rows(&rm, c, false, 128, page < 64 ? page : 64))
      return DSA_ERR_CUDA;
  } else {
    // K: one copy a slot where a page holds its rows, else one a page and chunk; V: one a page
    if (!map_pages(&km, c, page < 64 ? page : 64, page < 64 ? 1 : 3) ||
        !map_pages(&vm, c, page < 32 ? page : 32, 4))
      return DSA_ERR_CUDA;
  }
  PagedMlaArgs a{};
  a.c = planes(c);
  a.table = block_table;
  a.k_len = k_len;
  a.q_len = q_len;
  a.batch = p->batch;
  a.n_q = p->n_q;
  a.heads = p->heads;
  a.max_pages = p->max_pages;
  a.row_tiles = pl.row_tiles;
  a.pairs = (int32_t)pl.pairs;
  a.scale_log2 = p->scale * 1.4426950408889634f;
  a.out = reinterpret_cast<uint16_t*>(out);
  a.lse = out_lse;
  a.status = reinterpret_cast<int32_t*>(ws);
  a.states = reinterpret_cast<int32_t*>(ws + pl.off_states);
  a.clusters = pl.clusters;
  a.plan = reinterpret_cast<int32_t*>(ws + pl.off_plan);
  const bool stall = (p->flags & DSA_FLAG_TEST_STALL) != 0;
  a.wait_kilocycles = (int32_t)((stall ? kTestWaitCycles : kWaitCycles) >> 10);
  a.stall = stall;
  a.part_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.off_o);
  const int smem = (int)paged_mla_smem_bytes();
  auto kern = codes ? paged_mla_kernel<true> : paged_mla_kernel<false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return DSA_ERR_CUDA;
  kern<<<(unsigned)(2 * pl.clusters), codes ? kPmThreadsCodes : kPmThreadsRaw, smem, st>>>(
      qm, km, vm, rm, a);
  if (launch_status() != DSA_OK) return DSA_ERR_CUDA;
  const int64_t rows = (int64_t)p->n_q * p->heads;
  // the join is launched while the attention kernel drains, and waits for its end itself
  cudaLaunchConfig_t join{};
  const int64_t most = rows < kPmRows ? rows : kPmRows;
  const bool many = pl.pairs * most > kPmJoinBlocks;   // more rows than the GPU holds blocks
  // Rows a block: with few pairs one, as the GPU holds a block for each row; with many pairs
  // more, as most pairs were read by one cluster and their blocks only find that out.  Within
  // 4 % of the best of 1 to 64 (graph replays, us: 4 pairs 24 with 1, 27 with 4, 68 with 32; 32
  // pairs 64 with 4, 74 with 1 or 32; 100 pairs 125 with 4 or 8, 131 with 32, 145 with 1; 512
  // pairs 154 with 8 or 32, 158 with 4, 210 with 1).
  a.join_rows = pl.pairs >= 256 ? 32 : (pl.pairs >= 64 ? 8 : (many ? 4 : 1));
  join.gridDim = dim3((unsigned)pl.pairs, (unsigned)((most + a.join_rows - 1) / a.join_rows));
  join.blockDim = dim3(kPmJoinThreads);
  join.stream = st;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  join.attrs = &early;
  join.numAttrs = 1;
  if (cudaLaunchKernelEx(&join, many ? paged_mla_join_kernel<4> : paged_mla_join_kernel<1>, a) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (p->flags & DSA_FLAG_CHECK) return dsa_read_status(workspace, stream);
  return DSA_OK;
}

}  // extern "C"
