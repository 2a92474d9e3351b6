// mk_kv4_prompt.cu -- causal attention over the 4-bit KV cache for many query rows of
// 16-bit types (prompts), on the tcgen05 tensor cores.
//
// A CTA has 256 query rows (tokens x the rep query heads of one kv head) as two tiles of
// 128, and walks the positions it sees in tiles of 128.  Roles:
//   warps 0-3, 4-7  softmax of query tile 0, 1: one thread per row
//   warps 8-11      dequantise: codes to fp16 K and V in the swizzled shared-memory layout
//   warp 12         issues the matrix instructions
// Per tile: S = Q K^T into tensor memory (128 x 128 fp32); the row's thread reads S twice
// (maximum, then weights) and writes the weights back over S as fp16, from where they are
// the A operand of O += W V, which stays in tensor memory.  The two query tiles alternate:
// while one is in its softmax, the tensor cores work for the other.
//
// K and V are z + s c rounded once to fp16 (one HFMA2 for two values), queries are scaled
// by a power of two per row, which is exact in fp16 but for values 2^-24 below the row's
// largest.  The order of values inside 8 and of positions inside 32 is the one the codes
// come in: queries are permuted alike, and S, W and V share the order of positions.
// O is rescaled only when a score passes the row's reference by more than 16x.
//
// Bound: one exponential per score and the two products; 128 x 128 x D scores cost the
// tensor cores 128 D / 32 cycles... see the figures at the launch.
#include <cuda_runtime.h>

#include <atomic>

#include "mk_kv4.cuh"
#include "mk_kv4.h"
#include "mk_tc.cuh"

namespace mk {
namespace {

constexpr int kPThreads = 13 * 32;
constexpr int kPTile = 128;  // positions per tile, and rows per query tile
constexpr int kPHead = 4;    // log2 of what a weight may pass the reference by
constexpr int kPLift = 10;   // weights are 2^(score - m + kPLift), at most 2^14
constexpr unsigned long long kPWaitNs = 1000000000ull;

template <int D>
struct PSmem {
  static constexpr int kQ = 2 * kPTile * D * 2;   // both query tiles
  static constexpr int kKV = kPTile * D * 2;      // one K or V tile
  static constexpr int kBytes = 1024 + kQ + 4 * kKV;
};

struct PShared {
  uint64_t q_full, kv_full[2], kv_empty[2], s_full[2], w_full[2], o_full[2], drained;
  uint32_t tmem;
  // what a tile needs special care for: bits 0-3 blocks of 32 positions whose page is
  // out of range, bit 4 + w block w holds NaN values
  uint32_t special[2][4];
  uint8_t nan_groups[2][kPTile];  // groups of V that are NaN, by position (valid where bit 4 + w is set)
};

// instruction descriptor: D fp32, A and B fp16, both K-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= A[tmem] * B[bdesc]^T: A's rows are tensor-memory lanes, two fp16 per column
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t acc) {
  const uint32_t z = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(z), "r"(z), "r"(z), "r"(z));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// loads that wait for their data in the same statement, so that no use can move before the wait
__device__ __forceinline__ void tmem_get16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_get32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float pex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The 8 values of a code word as four pairs (nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7),
// each z + s c rounded once: a code or'ed into the mantissa of 1024 and taken back out.
__device__ __forceinline__ void dequant8(uint32_t x, uint32_t s2, uint32_t z2, uint32_t (&v)[4]) {
  const uint32_t y = x >> 8;
  v[0] = hfma2(hadd2((x & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s2, z2);               // - 1024
  v[1] = hfma2(hfma2((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s2, z2);  // / 16 - 64
  v[2] = hfma2(hadd2((y & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s2, z2);
  v[3] = hfma2(hfma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s2, z2);
}
__device__ __forceinline__ uint32_t both(uint32_t pair, int which) {  // one half of a pair, twice
  return __byte_perm(pair, 0u, which ? 0x3232 : 0x1010);
}
__device__ __forceinline__ bool nan_half(uint32_t h) { return (h & 0x7FFFu) > 0x7C00u; }

__device__ __forceinline__ bool pwait(uint64_t* bar, uint32_t parity, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait_hint(bar, parity, 1000)) {
    if (globaltimer_ns() - t0 > kPWaitNs) {
      atomicOr(status, KV4_TIMEOUT);
      return false;
    }
  }
  return true;
}

// 16-byte chunk c (0..7) of row r in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// position (in a tile of 128) that column c of S holds: within 32 columns, column
// 8 tig + 4 u + 2 hf + e is row 8 hf + 2 tig + e of the block's tile u
__host__ __device__ constexpr int column_position(int c) {
  return (c & ~31) + 16 * ((c >> 2) & 1) + 8 * ((c >> 1) & 1) + 2 * ((c >> 3) & 3) + (c & 1);
}

template <int D, class T>
__global__ void __launch_bounds__(kPThreads, 1) attn_prompt(const Kv4Attn a, int n_blocks) {
  using L = Kv4<D>;
  constexpr int G = L::G;
  constexpr uint32_t kIdQK = idesc_f16(128, kPTile), kIdWV = idesc_f16(128, D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ PShared sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;                    // [2][D / 64][128 rows][128 bytes]
  uint8_t* skv = smem + PSmem<D>::kQ;    // [2 buffers][K, V]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int idx = blockIdx.x;
  const int blk = n_blocks - 1 - idx / (a.c.n_kv_heads * a.b.n_seqs);  // the blocks that see most come first
  idx %= a.c.n_kv_heads * a.b.n_seqs;
  const int head = idx % a.c.n_kv_heads, si = idx / a.c.n_kv_heads;
  const Kv4Seq seq = kv4_seq(a.b, si);
  if (!seq.ok) {
    if (tid == 0) atomicOr(a.c.status, KV4_BAD_BATCH);
    return;
  }
  const int n_rows = seq.n * a.rep, row0 = blk * 2 * kPTile;
  if (row0 >= n_rows) return;
  const int start = seq.len - seq.n;  // position of the first query token (may be negative)
  int n_tiles[2], n_max = 0;          // tiles of positions each query tile sees
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = row0 + t * kPTile, last = min(n_rows, first + kPTile) - 1;
    n_tiles[t] = first < n_rows ? (max(0, start + last / a.rep + 1) + kPTile - 1) / kPTile : 0;
    n_max = max(n_max, n_tiles[t]);
  }

  if (tid == 0) {
    mbar_init(&sh.q_full, 2 * kPTile);
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.kv_full[i], kPTile);
      mbar_init(&sh.kv_empty[i], 1);
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.w_full[i], kPTile);
      mbar_init(&sh.o_full[i], 1);
    }
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;  // S0, S1: 128 columns each; O0, O1: D each

  if (warp < 8) {
    // ---------------- softmax: one thread per row ----------------
    const int t = warp >> 2, r_in = tid & 127, row = row0 + t * kPTile + r_in;
    const bool live = row < n_rows;
    float kscale;
    {
      float mx = 0.f;
      const char* src = a.q + (long long)(seq.row0 + row / a.rep) * a.q_row +
                        (long long)(head * a.rep + row % a.rep) * a.q_head;
      Raw8<T> raw[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        raw[c] = Raw8<T>{};
        if (live) raw[c] = load_raw8<T>(src + c * 16);
        float x[8];
        unpack8(raw[c], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
      }
      // power of two that brings the row's largest to 2^12 .. 2^13 (rows of zeros and rows
      // with an infinity keep theirs); the sign of the scale goes to the queries, so that
      // the maximum of the accumulated scores is the maximum of the scores
      const int e = mx > 0.f && mx < INFINITY ? min(100, 12 + 127 - (int)(__float_as_uint(mx) >> 23)) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23), sup = a.scale_log2 < 0.f ? -up : up;
      kscale = fmaxf(fabsf(a.scale_log2) / up, 1e-37f);  // (never zero: it multiplies the -inf of masked positions)
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float x[8];
        unpack8(raw[c], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= sup;
        *reinterpret_cast<uint4*>(sq + (t * (D / 64) + c / 8) * 16384 + chunk_at(r_in, c % 8)) =
            make_uint4(pack_h(x[0], x[4]), pack_h(x[1], x[5]), pack_h(x[2], x[6]), pack_h(x[3], x[7]));
      }
    }
    fence_proxy_async_smem();
    mbar_arrive(&sh.q_full);

    const int lim = live ? start + row / a.rep + 1 : 0;               // positions this row sees
    const int lim_warp = start + (row0 + t * kPTile + (r_in & ~31)) / a.rep + 1;  // the warp's rows all see these
    const bool whole = row0 + t * kPTile + (r_in | 31) < n_rows;      // no row of the warp is past the end
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lane_base + (uint32_t)(t * 128), to = lane_base + (uint32_t)(256 + t * D);
    float m = -INFINITY, ref = 0.f, sum = 0.f;
    uint32_t nan_out = 0;  // groups of the output that a NaN value reaches
    const int n = n_tiles[t];
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = __all_sync(0xFFFFFFFFu, pwait(&sh.s_full[t], j & 1, a.c.status));
      if (!ok) break;
      tc_fence_after();
      const int base = j * kPTile, left = lim - base;  // columns with position < left are seen
      uint32_t special = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) special |= sh.special[j & 1][w];
      const bool plain = whole && base + kPTile <= lim_warp && special == 0;
      auto masked = [&](int c) {  // column c
        return column_position(c) >= left || (special >> (c >> 5) & 1u);
      };
      // maximum
      float mx = -INFINITY;
#pragma unroll
      for (int c0 = 0; c0 < kPTile; c0 += 32) {
        uint32_t s[32];
        tmem_get32(ts + c0, s);
        if (plain) {
          float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            q[(i >> 1) & 3] = fmaxf(q[(i >> 1) & 3], fmaxf(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
          mx = fmaxf(mx, fmaxf(fmaxf(q[0], q[1]), fmaxf(q[2], q[3])));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = masked(c0 + i) ? mx : fmaxf(mx, __uint_as_float(s[i]));
        }
      }
      mx *= kscale;
      if (__any_sync(0xFFFFFFFFu, mx > m + (float)kPHead)) {
        const bool first = m == -INFINITY;  // nothing kept so far (but a NaN, which stays one)
        m = fmaxf(m, mx);
        const float r = (m == -INFINITY ? 0.f : m) - (float)kPLift, corr = first ? 0.f : pex2(ref - r);
        ref = r;
        sum *= corr;
        if (j > 0) {  // O is complete up to the tile before: its product came before this S
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t o[16];
            tmem_get16(to + c0, o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tmem_st16(to + c0, o);
          }
        }
      }
      // weights, over the scores already read
      float2 part = make_float2(0.f, 0.f);
      const float2 k2 = make_float2(kscale, kscale), r2 = make_float2(-ref, -ref);
#pragma unroll
      for (int c0 = 0; c0 < kPTile; c0 += 32) {
        uint32_t s[32], w[16];
        tmem_get32(ts + c0, s);
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          float2 x = make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          if (!plain) {
            if (masked(c0 + i)) x.x = -INFINITY;
            if (masked(c0 + i + 1)) x.y = -INFINITY;
          }
          x = __ffma2_rn(x, k2, r2);
          x.x = pex2(x.x);
          x.y = pex2(x.y);
          part = __fadd2_rn(part, x);
          w[i / 2] = pack_h(x.x, x.y);
        }
        tmem_st16(ts + c0 / 2, w);
      }
      sum += part.x + part.y;
      if (special >> 4) {  // NaN values among this tile's V: zero there, and remembered here
        for (int c = 0; c < kPTile; ++c) {
          const int p = column_position(c);
          if ((sh.special[j & 1][p >> 5] >> (4 + (p >> 5)) & 1u) && !masked(c)) nan_out |= sh.nan_groups[j & 1][p];
        }
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&sh.w_full[t]);
    }
    if (n > 0 && ok) ok = __all_sync(0xFFFFFFFFu, pwait(&sh.o_full[t], 0, a.c.status));
    if (ok) {
      tc_fence_after();
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // 0: the row sees nothing
      char* dst = a.out + (long long)(seq.row0 + row / a.rep) * a.o_row +
                  (long long)(head * a.rep + row % a.rep) * a.o_head;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t o[16];
        if (n > 0) {
          tmem_get16(to + c0, o);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = n > 0 && sum != 0.f ? __uint_as_float(o[8 * h + i]) * inv : 0.f;
            if (nan_out >> (c0 / 32) & 1u) x[i] = __uint_as_float(0x7FFFFFFFu);
          }
          if (live) store8<T>(dst + (c0 + 8 * h) * sizeof(T), x);
        }
      }
    }
  } else if (warp < 12) {
    // ---------------- dequantise: warp w has positions 32 w .. 32 w + 31 of a tile ----------------
    const int w = warp - 8, gid = lane >> 2, tig = lane & 3;
    const int32_t* table = a.b.block_table + (size_t)si * a.b.max_pages;
    const int see = min(seq.len, n_max * kPTile);  // positions behind are left out (zero)
    // raw operands of this warp's two 16-position tiles
    uint4 kc[2][2 * G / 4] = {}, vc[2][2 * G / 4] = {}, vs[2][2 * G / 4] = {}, ks[2][2] = {};
    uint2 kz[2][2] = {};
    uint32_t vz[2][G][2] = {};
    int page = 0, page_next = 0;
    auto look = [&](int j) {  // page id of tile j, one tile ahead of its loads
      const int p = j * kPTile + 32 * w;
      page_next = p < see ? table[p / MK_KV4_PAGE] : -2;  // -2: nothing there
    };
    auto load = [&](int j) {
      page = page_next;
      if ((unsigned)page < (unsigned)a.c.n_pages) {
        const size_t at = (((size_t)a.layer * a.c.n_pages + page) * a.c.n_kv_heads + head) * kKv4Tiles + 2 * (w & 1);
        const uint8_t* tile = static_cast<const uint8_t*>(a.c.pool) + at * L::kBytes;
#pragma unroll
        for (int u = 0; u < 2; ++u, tile += L::kBytes) {
#pragma unroll
          for (int v = 0; v < 2 * G / 4; ++v) {
            kc[u][v] = ldnc16(tile + v * 512 + lane * 16);
            vc[u][v] = ldnc16(tile + L::kV + v * 512 + lane * 16);
            vs[u][v] = ldnc16(tile + L::kVs + v * 64 + tig * 16);
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            // scales of the groups of rows 2 (gid / 2), + 1 (+ 8 n): a pair per group
            if constexpr (G == 4) {
              ks[u][n] = ldnc16(tile + L::kKs + n * 64 + (gid >> 1) * 16);
              kz[u][n] = __ldg(reinterpret_cast<const uint2*>(tile + L::kKz + (8 * n + gid) * 8));
            } else {
              const uint2 s = __ldg(reinterpret_cast<const uint2*>(tile + L::kKs + (gid >> 1) * 16 + n * 8));
              ks[u][n] = make_uint4(s.x, s.y, 0u, 0u);
              kz[u][n] = make_uint2(__ldg(reinterpret_cast<const uint32_t*>(tile + L::kKz + (8 * n + gid) * 4)), 0u);
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
              vz[u][g][n] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::kVz + g * 32 + n * 16 + tig * 4));
          }
        }
      } else if (page != -2 && lane == 0) {
        atomicOr(a.c.status, KV4_BAD_PAGE);
      }
      if (j + 1 < n_max) look(j + 1);
    };
    look(0);
    if (n_max > 0) load(0);
    bool ok = true;
    for (int j = 0; j < n_max; ++j) {
      const int buf = j & 1;
      if (j >= 2) ok = __all_sync(0xFFFFFFFFu, pwait(&sh.kv_empty[buf], ((j >> 1) - 1) & 1, a.c.status));
      if (!ok) break;
      uint8_t* sk = skv + buf * 2 * PSmem<D>::kKV;
      uint8_t* sv = sk + PSmem<D>::kKV;
      const bool have = (unsigned)page < (unsigned)a.c.n_pages;
      const int left = have ? see - (j * kPTile + 32 * w) : 0;  // positions of the block that exist
      bool nan_any = false;
      if (left < 32) {  // the end of the sequence (or a missing page): V is zero there, K may be anything
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int p = 16 * u + 8 * n + 2 * tig;
            const uint32_t keep = (p < left ? 0xFFFFu : 0u) | (p + 1 < left ? 0xFFFF0000u : 0u);
            uint32_t* s = reinterpret_cast<uint32_t*>(vs[u]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              vz[u][g][n] &= keep;
              s[n * G + g] &= keep;
            }
          }
      }
      // NaN values of V become zeros here; the rows that see them learn of it through nan_groups
      uint32_t bits = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t z = vz[u][g][n];
            bits |= nan_half(z) || nan_half(z >> 16) ? 1u : 0u;
          }
      nan_any = __any_sync(0xFFFFFFFFu, bits != 0);
      if (nan_any) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t lo = 0, hi = 0;
            uint32_t* s = reinterpret_cast<uint32_t*>(vs[u]);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t z = vz[u][g][n];
              const uint32_t drop = (nan_half(z) ? 0xFFFFu : 0u) | (nan_half(z >> 16) ? 0xFFFF0000u : 0u);
              lo |= (nan_half(z) ? 1u : 0u) << g;
              hi |= (nan_half(z >> 16) ? 1u : 0u) << g;
              vz[u][g][n] &= ~drop;
              s[n * G + g] &= ~drop;
            }
            if (gid == 0) {
              sh.nan_groups[buf][32 * w + 16 * u + 8 * n + 2 * tig] = (uint8_t)lo;
              sh.nan_groups[buf][32 * w + 16 * u + 8 * n + 2 * tig + 1] = (uint8_t)hi;
            }
          }
      }
      if (lane == 0) sh.special[buf][w] = (page != -2 && !have ? 1u << w : 0u) | (nan_any ? 16u << w : 0u);
      // K: row of position 16 u + 8 n + gid of the block (column order), 16 bytes per word
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = 32 * w + 8 * (gid >> 1) + 4 * u + 2 * n + (gid & 1);
          const uint32_t* c = reinterpret_cast<const uint32_t*>(kc[u]);
          const uint32_t* s = reinterpret_cast<const uint32_t*>(&ks[u][n]);
          const uint32_t* z = reinterpret_cast<const uint32_t*>(&kz[u][n]);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            uint32_t v[4];
            dequant8(c[n * G + g], both(s[g], gid & 1), both(z[g / 2], g & 1), v);
            const int word = 4 * g + tig;
            *reinterpret_cast<uint4*>(sk + (word >> 3) * 16384 + chunk_at(r, word & 7)) = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      // V transposed: row of value 32 g + 4 gid + i, 8 positions (16 bytes) per lane
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t v[4][4];  // [2 u + hf][value]
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            dequant8(reinterpret_cast<const uint32_t*>(vc[u])[2 * g + n],
                     reinterpret_cast<const uint32_t*>(vs[u])[n * G + g], vz[u][g][n], v[2 * u + n]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = 32 * g + 4 * gid + i;
          *reinterpret_cast<uint4*>(sv + (w >> 1) * (D * 128) + chunk_at(d, 4 * (w & 1) + tig)) =
              make_uint4(v[0][i], v[1][i], v[2][i], v[3][i]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.kv_full[buf]);
      if (j + 1 < n_max) load(j + 1);
    }
  } else if (lane == 0 && n_max > 0) {
    // ---------------- matrix instructions ----------------
    bool ok = pwait(&sh.q_full, 0, a.c.status);
    auto qk = [&](int t, int j) {
      const uint32_t q = smem_u32(sq) + t * (D / 64) * 16384, k = smem_u32(skv) + (j & 1) * 2 * PSmem<D>::kKV;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        umma_f16(tmem + t * 128, sw128_desc(q + (i / 4) * 16384 + (i % 4) * 32),
                 sw128_desc(k + (i / 4) * 16384 + (i % 4) * 32), kIdQK, i ? 1u : 0u);
      umma_commit(&sh.s_full[t]);
    };
    auto wv = [&](int t, int j) {
      const uint32_t v = smem_u32(skv) + (j & 1) * 2 * PSmem<D>::kKV + PSmem<D>::kKV;
#pragma unroll
      for (int i = 0; i < kPTile / 16; ++i)
        umma_f16_ts(tmem + 256 + t * D, tmem + t * 128 + 8 * i, sw128_desc(v + (i / 4) * (D * 128) + (i % 4) * 32), kIdWV,
                    j || i ? 1u : 0u);
    };
    ok = ok && pwait(&sh.kv_full[0], 0, a.c.status);
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (n_tiles[t] > 0) qk(t, 0);
    }
    for (int j = 0; j < n_max && ok; ++j) {
      bool next = false;  // tile j + 1 has been waited for
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (j >= n_tiles[t] || !ok) continue;
        ok = pwait(&sh.w_full[t], j & 1, a.c.status);
        if (!ok) break;
        tc_fence_after();
        wv(t, j);
        if (j + 1 == n_tiles[t]) umma_commit(&sh.o_full[t]);
        if (t == 1 || n_tiles[1] <= j) umma_commit(&sh.kv_empty[j & 1]);  // the last product of this tile
        if (j + 1 < n_tiles[t]) {
          if (!next) ok = pwait(&sh.kv_full[(j + 1) & 1], ((j + 1) >> 1) & 1, a.c.status);
          next = true;
          if (!ok) break;
          tc_fence_after();
          qk(t, j + 1);
        }
      }
    }
    if (!ok) {  // let what was issued finish before the memory goes
      umma_commit(&sh.drained);
      pwait(&sh.drained, 0, a.c.status);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  __syncwarp();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

}  // namespace

template <int D, class T>
static mk_status launch(const Kv4Attn& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  if (!kv4_allow_smem(reinterpret_cast<const void*>(attn_prompt<D, T>), PSmem<D>::kBytes, &ready)) return MK_ERR_CUDA;
  const long long n_blocks = ((long long)a.b.max_new * a.rep + 2 * kPTile - 1) / (2 * kPTile);
  const long long ctas = n_blocks * a.c.n_kv_heads * a.b.n_seqs;
  if (ctas > 0x7FFFFFFF) return MK_ERR_UNSUPPORTED;
  attn_prompt<D, T><<<(unsigned)ctas, kPThreads, PSmem<D>::kBytes, s>>>(a, (int)n_blocks);
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status kv4_prompt(const Kv4Attn& a, int32_t dtype, cudaStream_t s) {
  if (a.c.head_dim == 64) return dtype == 0 ? launch<64, __nv_bfloat16>(a, s) : launch<64, __half>(a, s);
  return dtype == 0 ? launch<128, __nv_bfloat16>(a, s) : launch<128, __half>(a, s);
}

}  // namespace mk
