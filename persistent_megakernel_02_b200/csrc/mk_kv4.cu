// mk_kv4.cu -- the 4-bit KV cache: quantising rows as they are written, reading them
// back, and the host side of these calls.  Layout and quantisation: mk_kv4.cuh.
#include <cuda_runtime.h>

#include <cmath>

#include "mk_kv4.cuh"
#include "mk_kv4.h"

namespace mk {
namespace {

// Where the rows of a call are in memory.
struct BatchRows {  // the caller's tensors
  const char* base[2];
  long long row[2], head[2];  // strides in bytes
};
struct SlotRows {  // a handle's paged cache
  char* kv;        // [layer][physical page][kv head][K, V][PL][D] 16-bit values
  const int* table;
  int n_phys_pages, PL;
};

template <int D, class T>
__device__ __forceinline__ char* row_ptr(const BatchRows& b, int which, int, int row, int, int head, int) {
  return const_cast<char*>(b.base[which]) + row * b.row[which] + head * b.head[which];
}
template <int D, class T>
__device__ __forceinline__ char* row_ptr(const SlotRows& s, int which, int layer, int, int pos, int head, int heads) {
  const long long page = (long long)layer * s.n_phys_pages + s.table[pos / s.PL];
  return s.kv + (((page * heads + head) * 2 + which) * s.PL + pos % s.PL) * (long long)(D * sizeof(T));
}

// What a CTA works on: one tile of one sequence and kv head.
struct TileJob {
  int tile, first, end;  // tile index; its positions first .. end - 1 are concerned
  int row0;              // batch row of position `first`
  int layer;
  const int32_t* table;
  bool ok;
};

// Slots: sequence i owns slots cu[i] / 16 + 2 i onwards, enough for every tile its
// span touches (a span of n rows touches at most (n - 1) / 16 + 2 tiles), so a flat
// grid of n_rows / 16 + 2 n_seqs slots covers any batch.
__device__ __forceinline__ TileJob tile_job(const mk_kv4_cache& c, const mk_kv4_batch& b, int layer, int slot) {
  TileJob j{};
  int lo = 0, hi = b.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.cu[mid] / kKv4Tile + 2 * mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  const Kv4Seq s = kv4_seq(b, lo);
  const int start = s.len - s.n;
  if (!s.ok || start < 0) {
    if (threadIdx.x == 0) atomicOr(c.status, KV4_BAD_BATCH);
    return j;
  }
  const int t = start / kKv4Tile + slot - (s.row0 / kKv4Tile + 2 * lo);
  j.tile = t;
  j.first = max(start, t * kKv4Tile);
  j.end = min(s.len, (t + 1) * kKv4Tile);
  j.row0 = s.row0 + j.first - start;
  j.layer = layer;
  j.table = b.block_table + (size_t)lo * b.max_pages;
  j.ok = j.first < j.end && slot >= s.row0 / kKv4Tile + 2 * lo;
  return j;
}

constexpr int kRowThreads = 128;

// One CTA quantises one tile of one kv head.  A thread takes 8 neighbouring values of
// a row (its 4 neighbours share a group).  A tile that is written whole is put
// together in shared memory and stored with 16-byte stores; one that is not (a single
// new token) goes out value by value, leaving the other rows as they are.
template <int D, class T, class Rows>
__device__ __forceinline__ void quantise_tile(const mk_kv4_cache& c, const TileJob& j, const Rows& rows, int head) {
  using L = Kv4<D>;
  __shared__ __align__(16) uint8_t image[L::kBytes];
  uint8_t* out = kv4_tile<D>(c, j.table, j.layer, head, j.tile);
  if (!out) {
    if (threadIdx.x == 0) atomicOr(c.status, KV4_BAD_PAGE);
    return;
  }
  const bool whole = j.end - j.first == kKv4Tile;
  uint8_t* dst = whole ? image : out;
  constexpr int kChunks = D / 8, kItems = 2 * kKv4Tile * kChunks;
#pragma unroll
  for (int e0 = 0; e0 < kItems; e0 += kRowThreads) {
    const int e = e0 + threadIdx.x;
    const int which = e / (kKv4Tile * kChunks), r = e / kChunks % kKv4Tile, w = e % kChunks;
    const int pos = j.tile * kKv4Tile + r;
    const bool in = pos >= j.first && pos < j.end;
    float x[8];
    if (in) {
      load8<T>(row_ptr<D, T>(rows, which, j.layer, j.row0 + pos - j.first, pos, head, c.n_kv_heads) +
                   w * 8 * sizeof(T), x);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    __half s, z;
    const uint32_t codes = kv4_quantise(x, s, z);
    if (!in) continue;
    if (which == 0) {
      *reinterpret_cast<uint32_t*>(dst + L::k_word(r, w)) = codes;
    } else {
      *reinterpret_cast<uint16_t*>(dst + L::v_unit(r, 2 * w)) = (uint16_t)codes;
      *reinterpret_cast<uint16_t*>(dst + L::v_unit(r, 2 * w + 1)) = (uint16_t)(codes >> 16);
    }
    if (w % 4 == 0) {
      *reinterpret_cast<__half*>(dst + (which ? L::kVs : L::kKs) + L::scale(r, w / 4)) = s;
      *reinterpret_cast<__half*>(dst + (which ? L::v_min(r, w / 4) : L::k_min(r, w / 4))) = z;
    }
  }
  if (!whole) return;
  __syncthreads();
  for (int e = threadIdx.x; e < L::kBytes / 16; e += kRowThreads)
    reinterpret_cast<uint4*>(out)[e] = reinterpret_cast<const uint4*>(image)[e];
}

// One CTA reads one tile of one kv head: the tile comes in with 16-byte loads, and a
// thread puts out 8 neighbouring values of a row.
template <int D, class T, class Rows>
__device__ __forceinline__ void read_tile(const mk_kv4_cache& c, const TileJob& j, const Rows& rows, int head) {
  using L = Kv4<D>;
  __shared__ __align__(16) uint8_t image[L::kBytes];
  const uint8_t* src = kv4_tile<D>(c, j.table, j.layer, head, j.tile);
  if (!src) {
    if (threadIdx.x == 0) atomicOr(c.status, KV4_BAD_PAGE);
    return;
  }
  for (int e = threadIdx.x; e < L::kBytes / 16; e += kRowThreads)
    reinterpret_cast<uint4*>(image)[e] = reinterpret_cast<const uint4*>(src)[e];
  __syncthreads();
  constexpr int kChunks = D / 8, kItems = 2 * kKv4Tile * kChunks;
#pragma unroll
  for (int e0 = 0; e0 < kItems; e0 += kRowThreads) {
    const int e = e0 + threadIdx.x;
    const int which = e / (kKv4Tile * kChunks), r = e / kChunks % kKv4Tile, w = e % kChunks;
    const int pos = j.tile * kKv4Tile + r;
    if (pos < j.first || pos >= j.end) continue;
    uint32_t codes;
    if (which == 0) {
      codes = *reinterpret_cast<const uint32_t*>(image + L::k_word(r, w));
    } else {
      codes = *reinterpret_cast<const uint16_t*>(image + L::v_unit(r, 2 * w)) |
              (uint32_t)*reinterpret_cast<const uint16_t*>(image + L::v_unit(r, 2 * w + 1)) << 16;
    }
    const float s = __half2float(*reinterpret_cast<const __half*>(image + (which ? L::kVs : L::kKs) + L::scale(r, w / 4)));
    const float z = __half2float(*reinterpret_cast<const __half*>(image + (which ? L::v_min(r, w / 4) : L::k_min(r, w / 4))));
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(s, (float)((codes >> (4 * i)) & 15u), z);
    store8<T>(row_ptr<D, T>(rows, which, j.layer, j.row0 + pos - j.first, pos, head, c.n_kv_heads) + w * 8 * sizeof(T), x);
  }
}

template <int D, class T, bool WRITE>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(mk_kv4_cache c, int layer, mk_kv4_batch b, BatchRows rows) {
  const TileJob j = tile_job(c, b, layer, blockIdx.x);
  if (!j.ok) return;
  if (WRITE) quantise_tile<D, T>(c, j, rows, blockIdx.y);
  else read_tile<D, T>(c, j, rows, blockIdx.y);
}

// Positions start .. start + n - 1 of a handle's slot, every layer: grid (tiles, kv heads, layers).
template <int D, class T, bool WRITE>
__global__ void __launch_bounds__(kRowThreads)
    slot_kernel(mk_kv4_cache c, SlotRows rows, const int32_t* table_row, int start, int n) {
  TileJob j;
  j.tile = start / kKv4Tile + blockIdx.x;
  j.first = max(start, j.tile * kKv4Tile);
  j.end = min(start + n, (j.tile + 1) * kKv4Tile);
  j.row0 = 0;
  j.layer = blockIdx.z;
  j.table = table_row;
  if (WRITE) quantise_tile<D, T>(c, j, rows, blockIdx.y);
  else read_tile<D, T>(c, j, rows, blockIdx.y);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

mk_status launched() { return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA; }

template <bool WRITE>
mk_status run_rows(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, const mk_kv4_rows* k,
                   const mk_kv4_rows* v, int32_t dtype, void* stream) {
  mk_status st = kv4_check(c, layer, b, dtype);
  if (st != MK_OK) return st;
  if (b->n_rows == 0) return MK_OK;
  st = kv4_check_rows(k, dtype, b->n_rows, c->n_kv_heads, c->head_dim, !WRITE);
  if (st == MK_OK) st = kv4_check_rows(v, dtype, b->n_rows, c->n_kv_heads, c->head_dim, !WRITE);
  if (st != MK_OK) return st;
  const int size = dtype == 2 ? 4 : 2;
  BatchRows rows;
  const mk_kv4_rows* kv[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    rows.base[i] = static_cast<const char*>(kv[i]->p);
    rows.row[i] = kv[i]->row_stride * size;
    rows.head[i] = kv[i]->head_stride * size;
  }
  const long long slots = b->n_rows / kKv4Tile + 2ll * b->n_seqs;
  if (slots > 0x7FFFFFFF) return MK_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)slots, c->n_kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
#define MK_KV4_ROWS(D, T) rows_kernel<D, T, WRITE><<<grid, kRowThreads, 0, s>>>(*c, layer, *b, rows)
  if (c->head_dim == 64) {
    if (dtype == 0) MK_KV4_ROWS(64, __nv_bfloat16);
    else if (dtype == 1) MK_KV4_ROWS(64, __half);
    else MK_KV4_ROWS(64, float);
  } else {
    if (dtype == 0) MK_KV4_ROWS(128, __nv_bfloat16);
    else if (dtype == 1) MK_KV4_ROWS(128, __half);
    else MK_KV4_ROWS(128, float);
  }
#undef MK_KV4_ROWS
  return launched();
}

}  // namespace

mk_status kv4_check_cache(const mk_kv4_cache* c) {
  if (!c || !c->pool || !c->status || !aligned16(c->pool) || ((uintptr_t)c->status & 3u)) return MK_ERR_INVALID_ARG;
  if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1) return MK_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return MK_ERR_UNSUPPORTED;
  if (c->n_kv_heads > 65535) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

mk_status kv4_check(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, int32_t dtype) {
  const mk_status st = kv4_check_cache(c);
  if (st != MK_OK) return st;
  if (layer < 0 || layer >= c->n_layers) return MK_ERR_INVALID_ARG;
  if (!b || !b->block_table || !b->cu || !b->kv_lens) return MK_ERR_INVALID_ARG;
  if (b->n_seqs < 1 || b->max_pages < 1 || b->n_rows < 0 || b->max_new < 0 || b->max_len < 0) return MK_ERR_INVALID_ARG;
  if ((long long)b->max_len > (long long)MK_KV4_PAGE * b->max_pages) return MK_ERR_INVALID_ARG;
  if (dtype < 0 || dtype > 2) return MK_ERR_INVALID_ARG;
  if (b->n_seqs > 65535) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

mk_status kv4_check_rows(const mk_kv4_rows* r, int32_t dtype, int64_t rows, int32_t heads, int32_t d, bool written) {
  if (!r || !r->p || !aligned16(r->p)) return MK_ERR_INVALID_ARG;
  const int per16 = dtype == 2 ? 4 : 8;
  const int64_t rs = r->row_stride, hs = r->head_stride;
  if (rs < 0 || hs < 0 || (rows > 1 && rs % per16) || (heads > 1 && hs % per16)) return MK_ERR_INVALID_ARG;
  if (!written) return MK_OK;
  // rows that are written must not overlap: heads inside a row, or rows inside a head
  const bool by_row = (heads == 1 || hs >= d) && (rows == 1 || rs >= (heads - 1) * hs + d);
  const bool by_head = (rows == 1 || rs >= d) && (heads == 1 || hs >= (rows - 1) * rs + d);
  return by_row || by_head ? MK_OK : MK_ERR_INVALID_ARG;
}

mk_status kv4_slot(bool write, const mk_kv4_cache* c, void* kv, const int* slot_table, int n_phys_pages, int PL,
                   bool fp16, const int32_t* table_row, int start, int n, cudaStream_t s) {
  const SlotRows rows{static_cast<char*>(kv), slot_table, n_phys_pages, PL};
  const dim3 grid((start + n - 1) / kKv4Tile - start / kKv4Tile + 1, c->n_kv_heads, c->n_layers);
#define MK_KV4_SLOT(D, T)                                                                          \
  (write ? slot_kernel<D, T, true><<<grid, kRowThreads, 0, s>>>(*c, rows, table_row, start, n)     \
         : slot_kernel<D, T, false><<<grid, kRowThreads, 0, s>>>(*c, rows, table_row, start, n))
  if (c->head_dim == 64) {
    if (fp16) MK_KV4_SLOT(64, __half);
    else MK_KV4_SLOT(64, __nv_bfloat16);
  } else {
    if (fp16) MK_KV4_SLOT(128, __half);
    else MK_KV4_SLOT(128, __nv_bfloat16);
  }
#undef MK_KV4_SLOT
  return launched();
}

}  // namespace mk

using namespace mk;

extern "C" int64_t mk_kv4_page_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? (int64_t)kKv4Tiles * 20 * head_dim : 0;
}

extern "C" mk_status mk_kv4_append(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                   const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype, void* stream) {
  return run_rows<true>(cache, layer, batch, k, v, dtype, stream);
}

extern "C" mk_status mk_kv4_read(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                 const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype, void* stream) {
  return run_rows<false>(cache, layer, batch, k, v, dtype, stream);
}
