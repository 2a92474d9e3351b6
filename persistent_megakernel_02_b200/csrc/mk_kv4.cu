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

// Row 0 of a tile and the distance to the next, of K or V (`which`) of a kv head: the tile's
// rows are evenly spaced in both (a handle's page holds 32 or 64 positions, so a tile never
// crosses one).  (Indexing by `which` would put the block in local memory.)
template <int D, class T>
__device__ __forceinline__ char* tile_rows(const BatchRows& b, int which, int, int row0, int, int head, int,
                                           long long* step) {
  *step = which ? b.row[1] : b.row[0];
  return const_cast<char*>(which ? b.base[1] : b.base[0]) + row0 * *step + head * (which ? b.head[1] : b.head[0]);
}
template <int D, class T>
__device__ __forceinline__ char* tile_rows(const SlotRows& s, int which, int layer, int, int pos0, int head, int heads,
                                           long long* step) {
  const long long page = (long long)layer * s.n_phys_pages + s.table[pos0 / s.PL];
  *step = D * (long long)sizeof(T);
  return s.kv + (((page * heads + head) * 2 + which) * s.PL + pos0 % s.PL) * *step;
}

// What a warp works on: one tile of one sequence and kv head.
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
  const int owner = kv4_owner(b, slot, 4, 2), lo = max(owner, 0);
  static_assert(kKv4Tile == 1 << 4, "");
  const Kv4Seq s = kv4_seq(b, lo);
  const int start = s.len - s.n;
  if (owner < 0 || !s.ok || start < 0) {
    if ((threadIdx.x & 31) == 0) atomicOr(c.status, KV4_BAD_BATCH);
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

constexpr int kRowWarps = 4;  // warps per CTA, each with work of its own

// A warp takes one tile of one kv head, K and then V: a lane has 8 neighbouring values of a
// row (4 neighbouring lanes share a group), and a warp-wide access covers kStep rows.  The
// place of row r0 + rl in the tile is that of r0 plus that of rl, so only the part of rl
// is computed at run time.
template <int D, class T, class Rows>
__device__ __forceinline__ void quantise_tile(const mk_kv4_cache& c, const TileJob& j, const Rows& rows, int head,
                                              uint8_t* image) {
  using L = Kv4<D>;
  constexpr int kChunks = D / 8, kStep = 32 / kChunks, kItems = kKv4Tile / kStep;
  const int lane = threadIdx.x & 31, w = lane % kChunks, rl = lane / kChunks;
  uint8_t* out = kv4_tile<D>(c, j.table, j.layer, head, j.tile);
  if (!out) {
    if (lane == 0) atomicOr(c.status, KV4_BAD_PAGE);
    return;
  }
  const bool whole = j.end - j.first == kKv4Tile;
  const int skip = j.first - j.tile * kKv4Tile, stop = skip + j.end - j.first;  // the tile's rows concerned
  // A whole tile's codes and parameters are put together in shared memory and stored with
  // 16-byte stores: codes of K or of V, 8 D bytes, then scales and minima, 2 D bytes.
  // Part of a tile (a new token) goes out value by value; the other rows stay as they are.
  auto load = [&](Raw8<T> (&raw)[4], int b0) {  // accesses b0 .. b0 + 3: K has 0 .. kItems - 1, V the next
    const int which = b0 >= kItems, r0 = (b0 - which * kItems) * kStep + rl;
    long long step;
    const char* p = tile_rows<D, T>(rows, which, j.layer, j.row0 - skip, j.tile * kKv4Tile, head, c.n_kv_heads, &step) +
                    r0 * step + w * 8 * sizeof(T);
#pragma unroll
    for (int i = 0; i < 4; ++i, p += kStep * step) {
      const int r = r0 + i * kStep;
      raw[i] = Raw8<T>{};
      if (r >= skip && r < stop) raw[i] = load_raw8<T>(p);
    }
  };
  Raw8<T> next[4];
  load(next, 0);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    uint8_t* codes_base = whole ? image : out + (which ? L::kV : 0);
    uint8_t* param_base = whole ? image + 8 * D : out + (which ? L::kVs : L::kKs);
    uint8_t* codes_at = codes_base + (which ? L::v_unit(rl, 2 * w) - L::kV : L::k_word(rl, w));
#pragma unroll 1
    for (int b0 = 0; b0 < kItems; b0 += 4) {  // four accesses at a time, the next four on their way
      Raw8<T> raw[4];
      float2 e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[i] = next[i];
      if (which * kItems + b0 + 4 < 2 * kItems) load(next, which * kItems + b0 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = extent8(raw[i]);
      // lane k of a group's quad has the parameters of access k
      const float lo = quad_scatter_min(e[0].x, e[1].x, e[2].x, e[3].x, lane);
      const float hi = -quad_scatter_min(e[0].y, e[1].y, e[2].y, e[3].y, lane);
      const uint32_t mine = kv4_params(lo, hi);
      const float s = h_lo(mine), inv_mine = s > 0.f ? __frcp_rn(s) : 0.f;
      {
        const int r = (b0 + (lane & 3)) * kStep + rl, g = w / 4;
        if (r >= skip && r < stop) {
          *reinterpret_cast<uint16_t*>(param_base + L::scale(r, g)) = (uint16_t)mine;
          *reinterpret_cast<uint16_t*>(param_base + (which ? L::v_min(r, g) - L::kVs : L::k_min(r, g) - L::kKs)) =
              (uint16_t)(mine >> 16);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t params = __shfl_sync(0xFFFFFFFFu, mine, (lane & ~3) | i);
        const float inv = __shfl_sync(0xFFFFFFFFu, inv_mine, (lane & ~3) | i);
        float x[8];
        unpack8(raw[i], x);
        const uint32_t codes = kv4_codes(x, params, inv);
        const int r0 = (b0 + i) * kStep, r = r0 + rl;
        if (r < skip || r >= stop) continue;
        if (which == 0) {
          *reinterpret_cast<uint32_t*>(codes_at + L::k_word(r0, 0)) = codes;
        } else {
          constexpr int kNext = L::v_unit(0, 1) - L::v_unit(0, 0);
          uint8_t* at = codes_at + (L::v_unit(r0, 0) - L::kV);
          *reinterpret_cast<uint16_t*>(at) = (uint16_t)codes;
          *reinterpret_cast<uint16_t*>(at + kNext) = (uint16_t)(codes >> 16);
        }
      }
    }
    if (!whole) continue;
    __syncwarp();
#pragma unroll
    for (int e = lane; e < 8 * D / 16; e += 32)
      reinterpret_cast<uint4*>(out + (which ? L::kV : 0))[e] = reinterpret_cast<const uint4*>(image)[e];
    if (lane < 2 * D / 16)
      reinterpret_cast<uint4*>(out + (which ? L::kVs : L::kKs))[lane] =
          reinterpret_cast<const uint4*>(image + 8 * D)[lane];
    __syncwarp();
  }
}

// The way back: the tile comes in with 16-byte loads, and a lane puts out 8 neighbouring
// values of a row.  32-bit rows are twice as long to write, so a warp writes K or V only
// (eight sequences of 517 to 1420 rows, 8 heads of 128: 18.0 us, both 20.1; 16-bit rows
// gain by both, 8192 rows of 64 6.5 -> 5.1 us).
template <class T>
constexpr int kReadParts = sizeof(T) == 4 ? 2 : 1;
template <int D, class T, class Rows>
__device__ __forceinline__ void read_tile(const mk_kv4_cache& c, const TileJob& j, const Rows& rows, int head,
                                          int part_of, uint8_t* image) {
  using L = Kv4<D>;
  constexpr int kChunks = D / 8, kStep = 32 / kChunks, kItems = kKv4Tile / kStep;
  const int lane = threadIdx.x & 31, w = lane % kChunks, rl = lane / kChunks;
  const uint8_t* src = kv4_tile<D>(c, j.table, j.layer, head, j.tile);
  if (!src) {
    if (lane == 0) atomicOr(c.status, KV4_BAD_PAGE);
    return;
  }
  uint4 part[(L::kBytes / 16 + 31) / 32];
#pragma unroll
  for (int i = 0; i * 32 < L::kBytes / 16; ++i)
    if (lane + 32 * i < L::kBytes / 16) part[i] = reinterpret_cast<const uint4*>(src)[lane + 32 * i];
#pragma unroll
  for (int i = 0; i * 32 < L::kBytes / 16; ++i)
    if (lane + 32 * i < L::kBytes / 16) reinterpret_cast<uint4*>(image)[lane + 32 * i] = part[i];
  __syncwarp();
  const int skip = j.first - j.tile * kKv4Tile, stop = skip + j.end - j.first;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (kReadParts<T> == 2 && which != part_of) continue;
    long long step;
    char* p = tile_rows<D, T>(rows, which, j.layer, j.row0 - skip, j.tile * kKv4Tile, head, c.n_kv_heads, &step) +
              rl * step + w * 8 * sizeof(T);
    const uint8_t* codes_at = image + (which ? L::v_unit(rl, 2 * w) : L::k_word(rl, w));
    const uint8_t* scale_at = image + (which ? L::kVs : L::kKs) + L::scale(rl, w / 4);
    const uint8_t* min_at = image + (which ? L::v_min(rl, w / 4) : L::k_min(rl, w / 4));
#pragma unroll
    for (int i = 0; i < kItems; ++i, p += kStep * step) {
      const int r = i * kStep + rl;
      uint32_t codes;
      if (which == 0) {
        codes = *reinterpret_cast<const uint32_t*>(codes_at + L::k_word(i * kStep, 0));
      } else {
        constexpr int kNext = L::v_unit(0, 1) - L::v_unit(0, 0);
        const uint8_t* at = codes_at + (L::v_unit(i * kStep, 0) - L::kV);
        codes = *reinterpret_cast<const uint16_t*>(at) | (uint32_t)*reinterpret_cast<const uint16_t*>(at + kNext) << 16;
      }
      const uint32_t params =
          *reinterpret_cast<const uint16_t*>(scale_at + L::scale(i * kStep, 0)) |
          (uint32_t)*reinterpret_cast<const uint16_t*>(
              min_at + (which ? L::v_min(i * kStep, 0) - L::kVz : L::k_min(i * kStep, 0) - L::kKz)) << 16;
      float x[8];
      kv4_values(codes, h_lo(params), h_hi(params), x);
      if (r >= skip && r < stop) store8<T>(p, x);
    }
  }
}

template <int D, class T, bool WRITE, class Rows>
__device__ __forceinline__ void do_tile(const mk_kv4_cache& c, const TileJob& j, const Rows& rows, int head, int part) {
  __shared__ __align__(16) uint8_t image[kRowWarps][WRITE ? 10 * D : 20 * D];
  if (WRITE) quantise_tile<D, T>(c, j, rows, head, image[threadIdx.x >> 5]);
  else read_tile<D, T>(c, j, rows, head, part, image[threadIdx.x >> 5]);
}

// Warp g of the grid: kv head g % n_kv_heads, then K or V where they are apart, then the
// slot, so neighbouring warps are at neighbouring heads of the same rows.
template <int D, class T, bool WRITE>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 4 ? 5 : 7)
    rows_kernel(mk_kv4_cache c, int layer, mk_kv4_batch b, BatchRows rows, int n_slots) {
  const long long g = (long long)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  constexpr int kParts = WRITE ? 1 : kReadParts<T>;
  const int head = (int)(g % c.n_kv_heads), part = (int)(g / c.n_kv_heads % kParts);
  const int slot = (int)(g / (c.n_kv_heads * kParts));
  if (slot >= n_slots) return;
  const TileJob j = tile_job(c, b, layer, slot);
  if (j.ok) do_tile<D, T, WRITE>(c, j, rows, head, part);
  if ((threadIdx.x & 31) == 0) kv4_report_order(c, b, g);  // (two slots or more to a sequence)
}

// Positions start .. start + n - 1 of a handle's slot: warps over (tile, kv head), grid.y
// over the layers.
template <int D, class T, bool WRITE>
__global__ void __launch_bounds__(32 * kRowWarps, sizeof(T) == 4 ? 5 : 7)
    slot_kernel(mk_kv4_cache c, SlotRows rows, const int32_t* table_row, int start, int n, int n_tiles) {
  const int g = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int head = g % c.n_kv_heads, t = g / c.n_kv_heads;
  if (t >= n_tiles) return;
  TileJob j;
  j.tile = start / kKv4Tile + t;
  j.first = max(start, j.tile * kKv4Tile);
  j.end = min(start + n, (j.tile + 1) * kKv4Tile);
  j.row0 = 0;
  j.layer = blockIdx.y;
  j.table = table_row;
  do_tile<D, T, WRITE>(c, j, rows, head, 0);
}

__global__ void take_status_kernel(uint32_t* status, uint32_t* bits) { *bits = atomicExch(status, 0u); }

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

cudaLaunchConfig_t rows_launch(dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kRowWarps);
  cfg.stream = s;
  return cfg;
}

template <bool WRITE>
mk_status run_rows(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, const mk_kv4_rows* k,
                   const mk_kv4_rows* v, int32_t dtype, void* stream) {
  mk_status st = kv4_check(c, layer, b, dtype);
  if (st != MK_OK) return st;
  if (b->n_rows == 0) return MK_OK;
  st = kv4_check_rows(k, dtype, b->n_rows, c->n_kv_heads, c->head_dim, !WRITE);
  if (st == MK_OK) st = kv4_check_rows(v, dtype, b->n_rows, c->n_kv_heads, c->head_dim, !WRITE);
  if (st != MK_OK) return st;
  if (!WRITE && k->p == v->p) return MK_ERR_INVALID_ARG;  // one output for both
  const int size = dtype == 2 ? 4 : 2;
  BatchRows rows;
  const mk_kv4_rows* kv[2] = {k, v};
  for (int i = 0; i < 2; ++i) {
    rows.base[i] = static_cast<const char*>(kv[i]->p);
    rows.row[i] = kv[i]->row_stride * size;
    rows.head[i] = kv[i]->head_stride * size;
  }
  const long long slots = b->n_rows / kKv4Tile + 2ll * b->n_seqs;
  const int parts = WRITE || dtype != 2 ? 1 : kReadParts<float>;
  const long long ctas = (slots * c->n_kv_heads * parts + kRowWarps - 1) / kRowWarps;
  if (ctas > 0x7FFFFFFF) return MK_ERR_UNSUPPORTED;
  if (kv4_error_pending()) return MK_ERR_CUDA;
  const cudaLaunchConfig_t cfg = rows_launch(dim3((unsigned)ctas), static_cast<cudaStream_t>(stream));
  cudaError_t e;
#define MK_KV4_ROWS(D, T) e = cudaLaunchKernelEx(&cfg, rows_kernel<D, T, WRITE>, *c, layer, *b, rows, (int)slots)
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
  return kv4_status(e);
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
  if (b->n_seqs > 65535 || b->max_new > (1 << 27)) return MK_ERR_UNSUPPORTED;  // (row indexes times 8 query heads)
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
  const int n_tiles = (start + n - 1) / kKv4Tile - start / kKv4Tile + 1;
  const long long ctas = ((long long)n_tiles * c->n_kv_heads + kRowWarps - 1) / kRowWarps;
  if (ctas * kRowWarps > 0x7FFFFFFF || c->n_layers > 65535) return MK_ERR_UNSUPPORTED;
  const cudaLaunchConfig_t cfg = rows_launch(dim3((unsigned)ctas, c->n_layers), s);
  cudaError_t e;
#define MK_KV4_SLOT(D, T)                                                                                      \
  e = write ? cudaLaunchKernelEx(&cfg, slot_kernel<D, T, true>, *c, rows, table_row, start, n, n_tiles)        \
            : cudaLaunchKernelEx(&cfg, slot_kernel<D, T, false>, *c, rows, table_row, start, n, n_tiles)
  if (c->head_dim == 64) {
    if (fp16) MK_KV4_SLOT(64, __half);
    else MK_KV4_SLOT(64, __nv_bfloat16);
  } else {
    if (fp16) MK_KV4_SLOT(128, __half);
    else MK_KV4_SLOT(128, __nv_bfloat16);
  }
#undef MK_KV4_SLOT
  return kv4_status(e);
}

}  // namespace mk

using namespace mk;

extern "C" int64_t mk_kv4_page_bytes(int32_t head_dim) {
  return head_dim == 64 || head_dim == 128 ? (int64_t)kKv4Tiles * 20 * head_dim : 0;
}

extern "C" mk_status mk_kv4_take_status(const mk_kv4_cache* cache, uint32_t* bits, void* stream) {
  const mk_status st = kv4_check_cache(cache);
  if (st != MK_OK) return st;
  if (!bits || ((uintptr_t)bits & 3u)) return MK_ERR_INVALID_ARG;
  if (kv4_error_pending()) return MK_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = cfg.blockDim = dim3(1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  return kv4_status(cudaLaunchKernelEx(&cfg, take_status_kernel, cache->status, bits));
}

extern "C" mk_status mk_kv4_append(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                   const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype, void* stream) {
  return run_rows<true>(cache, layer, batch, k, v, dtype, stream);
}

extern "C" mk_status mk_kv4_read(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                 const mk_kv4_rows* k, const mk_kv4_rows* v, int32_t dtype, void* stream) {
  return run_rows<false>(cache, layer, batch, k, v, dtype, stream);
}
