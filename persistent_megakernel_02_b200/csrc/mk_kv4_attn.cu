// mk_kv4_attn.cu -- causal attention over the 4-bit KV cache for few query rows: single
// new tokens, a few at a time, and every 32-bit call.
//
// Mathematics.  With K = z + s c per group g of 32 values, a score is
//   q . K = sum_g s_g (q_g . c_g) + sum_g z_g (sum of q_g),
// so the codes enter the matrix instructions (mma.m16n8k16) as they are: a 4-bit code in
// the low bits of an fp16 word is the subnormal c 2^-24 (or 16 c 2^-24 from the next
// nibble, with the query divided by 16 instead).  One AND turns 32 bits of codes into two
// operand values, and only the sums over 32 values are multiplied by a scale.  The second
// sum is one more mma over the groups.  (32-bit calls take one addition more, see low().)
// Values the same way: O = sum_p w_p V_p = sum_g c (w s)_g + z_g w, the weights of a
// position times its scale are the operand, and one mma holds the z part of all groups.
// The softmax runs in one pass with a running maximum and sum per row; the operand w s
// is kept in fp16's range by a power of two that follows the largest scale met so far.
//
// Bytes bound it for long contexts: 20 D bytes per 16 positions and kv head, read once.
// A warp takes whole stages of 5120 bytes (4 tiles of 64-value heads, 2 of 128) through
// a ring of bulk copies of its own, so no barrier is met until the warps' states are
// merged.  64 sequences of 823 to 16384 positions x 8 kv heads x 128: 149 us, 4.7 TB/s,
// 0.71 of the copy rate; the copies alone take 117 (64-value heads: 24 sequences 58 us for 32
// of bytes).  Fewer registers for a fifth CTA on the SM spill and lose (267 us).  Splits along
// the positions, where rows are few, are joined in the cluster's shared memory or by a second
// small kernel.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "mk_kv4.cuh"
#include "mk_kv4.h"

namespace mk {
namespace {

constexpr int kWarps = 4;
constexpr int kThreadsA = 32 * kWarps;
constexpr int kStageBytes = 5120;
constexpr int kStages = 2;  // ring depth per warp
constexpr int kHead = 4;    // log2 of what a weight may pass the peak's by

using AttnArgs = Kv4AttnSplit;

// c += A B (16 x 16 by 16 x 8), and the same from zero
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two codes of a word as operands, c and c' of one half each: their bits as they are, the
// subnormals c 2^-24 (16 c 2^-24 from the second nibbles), or NORMAL numbers c (16 c).  The
// matrix unit aligns products by the exponents of their operands, and a subnormal's is the
// smallest normal one, so up to ten bits go where a code is small: enough bits are left for
// 16-bit outputs, but not for 32-bit ones (8 lanes of about 1000 positions: 4e-5 off in the
// 2-norm, one of 16384 1.2e-4).
template <bool NORMAL>
__device__ __forceinline__ uint32_t low(uint32_t x) {
  return NORMAL ? hadd2((x & 0x000F000Fu) | 0x64006400u, 0xE400E400u) : x & 0x000F000Fu;
}
template <bool NORMAL>
__device__ __forceinline__ uint32_t high(uint32_t x) {
  return NORMAL ? hadd2((x & 0x00F000F0u) | 0x64006400u, 0xE400E400u) : x & 0x00F000F0u;
}
// The same for values: in 32-bit calls (c - 7.5) 2^-9, from the subnormal by one multiply-add,
// exactly and a normal number whatever c.
template <bool CENTRE>
__device__ __forceinline__ uint32_t low_v(uint32_t x) {
  x &= 0x000F000Fu;
  return CENTRE ? hfma2(x, 0x78007800u, 0xA380A380u) : x;
}
template <bool CENTRE>
__device__ __forceinline__ uint32_t high_v(uint32_t x) {
  x &= 0x00F000F0u;
  return CENTRE ? hfma2(x, 0x68006800u, 0xA380A380u) : x;
}
// Sums over more than 32 positions are kept out of the matrix unit: it cuts its sums off
// instead of rounding them, the codes' sums all grow in one direction, and the minima's part
// largely takes them back (fp16, 150 sequences of 16384 positions with even weights: results
// 4.5e-3 off in the 2-norm with the sums kept there, of 131072 4.4e-2).
__device__ __forceinline__ void add4(float (&a)[4], const float (&b)[4]) {
  const float2 x = __fadd2_rn(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
  const float2 y = __fadd2_rn(make_float2(a[2], a[3]), make_float2(b[2], b[3]));
  a[0] = x.x; a[1] = x.y; a[2] = y.x; a[3] = y.y;
}
__device__ __forceinline__ uint4 lds_u4(const uint8_t* p) { return lds128(smem_u32(p)); }
__device__ __forceinline__ uint32_t lds_u1(const uint8_t* p) { return lds32(smem_u32(p)); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {  // a NaN loses
  const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// a pair of halves with each one cleared that is infinite or NaN
__device__ __forceinline__ uint32_t finite2(uint32_t a) {
  if ((a & 0x7C00u) == 0x7C00u) a &= 0xFFFF0000u;
  if ((a & 0x7C000000u) == 0x7C000000u) a &= 0xFFFFu;
  return a;
}
// two fp16 parts of a pair of floats: x ~= hi + lo with 22 bits
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_h(x, y);
  lo = pack_h(x - h_lo(hi), y - h_hi(hi));
}

// One CTA: the rows of a row tile (8 NT rows: query tokens x the rep heads of one kv
// head) over one split of the positions, its stages dealt to the warps in turn.
// Registers per lane (gid = lane / 4, tig = lane % 4), NT row tiles of 8:
//   scores   row gid, positions 2 tig, 2 tig + 1 of each 8
//   outputs  value 32 g + 4 gid + 2 j + {0, 1} of rows 2 tig, 2 tig + 1
// 32-bit calls split queries and weights into two fp16 parts: the queries' low parts
// are rows 8..15 of the same mma, the weights' take a second one.
template <int D, class T, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kThreadsA, NT == 1 ? 4 : 2) attn_few(const AttnArgs a) {
  using L = Kv4<D>;
  constexpr int G = L::G;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr float kCode = kF32 ? 1.f : 16777216.f;  // a code's value over its operand's
  // weight * scale as two fp16 parts, exactly: the codes' part of a value and the minimum's
  // largely cancel, and then see the same weight.  (With one rounding more, fp16 outputs
  // are 5.1e-4 off instead of their own rounding's 2.1e-4; bf16's is 1.7e-3.)
  constexpr bool kExact = kF32 || std::is_same<T, __half>::value;
  // Values as (z + 7.5 s) + s (c - 7.5): neither part has a mean of its own, so that long sums do
  // not grow only to cancel (1024 sums of 32 positions added in 32 bits, 131072 positions: 4e-4 off
  // in the 2-norm without).  It costs little where codes are made normal numbers anyway: the sum
  // over a tile of w s is in rows 8..15 of the minima's product, which would be idle.  16-bit calls
  // bound the sum's length instead (all types so: 64 long sequences 153 -> 170 us).
  constexpr bool kCentre = kF32;
  constexpr float kLow = kCentre ? 512.f : 16777216.f, kHigh = kCentre ? 512.f : 1048576.f;  // a value's code over its operand's
  constexpr int MT = kF32 ? NT : (NT + 1) / 2;          // 16-row operands of the queries
  constexpr int kTilesPerStage = kStageBytes / L::kBytes;
  constexpr int kStagePos = kTilesPerStage * kKv4Tile;  // positions of a stage
  constexpr int kStagesPerPage = MK_KV4_PAGE / kStagePos;
  constexpr int SUB = 2;                                // tiles per softmax step
  constexpr int kRows = 8 * NT;

  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int slot_bad[kWarps][kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);

  int idx = blockIdx.x;
  const int split = idx % a.n_split;
  idx /= a.n_split;
  const int rt = a.n_rt - 1 - idx % a.n_rt;  // the tiles that see most come first
  idx /= a.n_rt;
  const int head = idx % a.c.n_kv_heads, si = idx / a.c.n_kv_heads;
  asm volatile("griddepcontrol.launch_dependents;");
  // the first page ids are loaded together with the lengths, which only bound them
  const int p0 = split * a.split_len, s0 = p0 / kStagePos;
  const int32_t* table = a.b.block_table + (size_t)si * a.b.max_pages;
  int page_id = 0;  // lane i: page of this warp's stage (32 k + i)
  {
    const int page = (s0 + warp + kWarps * lane) / kStagesPerPage;
    if (page < a.b.max_pages && kWarps * lane * kStagePos < a.split_len) page_id = table[page];
  }
  const Kv4Seq seq = kv4_seq(a.b, si);
  if (!seq.ok) {
    if (threadIdx.x == 0) atomicOr(a.c.status, KV4_BAD_BATCH);
    return;
  }
  const int n_rows = seq.n * a.rep, row0 = rt * kRows;
  if (row0 >= n_rows) return;
  const int start = seq.len - seq.n;  // position of the first query token (may be negative)
  const int last_row = min(n_rows, row0 + kRows) - 1;
  const int see_all = start + row0 / a.rep + 1;                // positions every row of the tile sees
  const int see_any = max(0, start + last_row / a.rep + 1);    // positions some row sees
  const int p1 = min(see_any, p0 + a.split_len);
  if (!CLUSTER && p0 >= p1 && split > 0) return;  // the join takes only the splits that hold something

  // ---- ring of bulk copies: this warp's stage i is stage s0 + warp + kWarps i ----
  const int n_stages = p0 < p1 ? (p1 - 1) / kStagePos - s0 + 1 : 0;
  const int mine = n_stages > warp ? (n_stages - warp - 1) / kWarps + 1 : 0;
  const int first = s0 + warp, last = s0 + n_stages - 1;
  const uint32_t last_bytes = (uint32_t)((p1 - last * kStagePos + kKv4Tile - 1) / kKv4Tile) * L::kBytes;
  const uint64_t page_stride = (uint64_t)a.c.n_kv_heads * (kKv4Tiles * L::kBytes);
  const uint8_t* base = static_cast<const uint8_t*>(a.c.pool) + (uint64_t)a.layer * a.c.n_pages * page_stride +
                        (uint64_t)head * (kKv4Tiles * L::kBytes);
  auto issue = [&](int i, int slot) {  // every lane calls
    if (i > 0 && (i & 31) == 0) {
      const int j = i + lane;
      page_id = j < mine ? table[(first + kWarps * j) / kStagesPerPage] : 0;
    }
    const int page = __shfl_sync(0xFFFFFFFFu, page_id, i & 31);
    if (lane == 0) {
      const int s = first + kWarps * i;
      const bool bad = (unsigned)page >= (unsigned)a.c.n_pages;
      slot_bad[warp][slot] = bad;
      if (bad) {
        atomicOr(a.c.status, KV4_BAD_PAGE);
        mbar_arrive(&full[warp][slot]);
      } else {
        const uint32_t bytes = s == last ? last_bytes : (uint32_t)kStageBytes;
        mbar_arrive_expect_tx(&full[warp][slot], bytes);
        bulk_g2s_plain(ring + slot * kStageBytes, base + (uint64_t)(uint32_t)page * page_stride + (s % kStagesPerPage) * kStageBytes,
                       bytes, &full[warp][slot]);
      }
    }
  };
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[warp][i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  for (int i = 0; i < kStages && i < mine; ++i) issue(i, i);

  // ---- queries: operand order of the codes, scaled by a power of two per row ----
  // [16 rows][group][k16 step][a0..a3].  With 8 rows of 16-bit queries rows 8..15 of the
  // operand would be idle: there it holds both steps, step 0 in rows 0..7 and step 1 in
  // rows 8..15, each product taken from its own half (half the registers, and no zeros to
  // be moved into place).
  constexpr bool kBoth = !kF32 && NT == 1;
  uint32_t qa[MT][G][kBoth ? 1 : 2][4];
  uint32_t qz[MT][4];        // sums over the groups, for the minima
  float kscale[NT];          // score = kscale * accumulated
  int lim[NT];               // positions the row sees
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 4; ++h) qz[m][h] = 0u;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = row0 + 8 * t + gid;
    const bool live = r < n_rows;
    float x[G][8];
    float mx = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (live) {
        load8<T>(a.q + (seq.row0 + r / a.rep) * a.q_row + (head * a.rep + r % a.rep) * a.q_head +
                     (32 * g + 8 * tig) * (int)sizeof(T),
                 x[g]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[g][i]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
    // power of two that brings the largest to 2^12 .. 2^13 (rows of zeros and rows
    // with an infinity keep theirs)
    const int e = mx > 0.f && mx < INFINITY ? min(126, 12 + 127 - (int)(__float_as_uint(mx) >> 23)) : 0;
    const float up = __uint_as_float((uint32_t)(127 + max(e, -126)) << 23);
    const float signed_up = a.scale_log2 < 0.f ? -up : up;
    kscale[t] = kv4_score_scale(fabsf(a.scale_log2) / up * kCode);
    lim[t] = live ? start + r / a.rep + 1 : 0;
    float sums[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[g][i] *= signed_up;
        sum += x[g][i];
      }
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
      sums[g] = sum * 0.015625f;  // 2^-6: at most 2^12
      // nibble i of a word is value 8 w + i; steps pair (0, 4), (1, 5) and (2, 6), (3, 7)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        uint32_t h0, l0, h1, l1;
        split2(x[g][2 * st], x[g][2 * st + 4], h0, l0);
        split2(x[g][2 * st + 1] * 0.0625f, x[g][2 * st + 5] * 0.0625f, h1, l1);
        if constexpr (kF32) {
          qa[t][g][st][0] = h0;
          qa[t][g][st][1] = l0;
          qa[t][g][st][2] = h1;
          qa[t][g][st][3] = l1;
        } else if constexpr (kBoth) {
          qa[0][g][0][st] = h0;
          qa[0][g][0][2 + st] = h1;
        } else {
          qa[t / 2][g][st][t & 1] = h0;
          qa[t / 2][g][st][2 + (t & 1)] = h1;
        }
      }
    }
    // k index of the minima's mma: groups 2 tig, 2 tig + 1 (high parts), + 8 (low parts)
    float s_lo = 0.f, s_hi = 0.f;
#pragma unroll
    for (int g = 0; g < G; g += 2)
      if (tig == g / 2) { s_lo = sums[g]; s_hi = sums[g + 1]; }
    uint32_t zh, zl;
    split2(s_lo, s_hi, zh, zl);
    if constexpr (kF32) {
      qz[t][0] = zh;
      qz[t][2] = zl;
    } else {
      qz[t / 2][t & 1] = zh;
      qz[t / 2][2 + (t & 1)] = zl;
    }
    if constexpr (kBoth) qz[0][1] = zh, qz[0][3] = zl;  // idle rows
  }

  // oz: row g the minima's part of group g, row G (operand of ones) the sum of the weights
  float o[NT][G][2][4], oz[NT][2];
  // Weights are 2^((score - peak) kscale + lift) of the accumulated scores: peak is the row's
  // largest when it was last moved (0: none so far), which happens when one passes `bound`.
  // lift: 14 - kHead, or less where scales are large; cap: the largest scale it allows (a pair of
  // halves).  Where all scales so far are below 2^-11, small weights times small scales would
  // leave fp16's range (values of 1e-6 under weights 2^12 apart: bf16 results 7e-3 off, fp32 6.8e-2):
  // the tiles' scales are made 2^boost as large in shared memory (below 2), at every step, for
  // which cap is 0.  That takes 15 % longer, so not for larger ones, which lose nothing.
  float peak[NT], bound[NT];
  int lift = 14 - kHead, boost = 15;
  uint32_t cap = 0u;
  [[maybe_unused]] float middle = 7.5f;  // ... of a group, in steps of the scales as they are taken
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    bound[t] = -INFINITY;
    peak[t] = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) oz[t][i] = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][g][j][i] = 0.f;
  }

  // SUB tiles at `tiles`, the first at position `pos`
  auto step = [&](const uint8_t* tiles, int pos, auto masked_tag) {
    constexpr bool kMasked = decltype(masked_tag)::value;
    float s[NT][SUB][4];
    uint32_t top = 0;  // largest V scale
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const uint8_t* tile = tiles + u * L::kBytes;
      uint32_t kc[2 * G], ks[2 * G], kz[2];
#pragma unroll
      for (int v = 0; v < 2 * G / 4; ++v) {
        const uint4 x = lds_u4(tile + v * 512 + lane * 16), y = lds_u4(tile + L::kKs + v * 64 + tig * 16);
        const uint4 w = lds_u4(tile + L::kVs + v * 64 + tig * 16);
        kc[4 * v] = x.x; kc[4 * v + 1] = x.y; kc[4 * v + 2] = x.z; kc[4 * v + 3] = x.w;
        ks[4 * v] = y.x; ks[4 * v + 1] = y.y; ks[4 * v + 2] = y.z; ks[4 * v + 3] = y.w;
        uint32_t w4[4] = {w.x, w.y, w.z, w.w};
        if constexpr (kMasked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = pos + 16 * u + 8 * ((4 * v + i) / G) + 2 * tig;
            w4[i] = finite2(w4[i]);
            if (p >= p1) w4[i] &= 0xFFFF0000u;
            if (p + 1 >= p1) w4[i] &= 0xFFFFu;
          }
        }
        top = hmax2(top, hmax2(hmax2(w4[0], w4[1]), hmax2(w4[2], w4[3])));
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) kz[n] = tig < G / 2 ? lds_u1(tile + L::kKz + (8 * n + gid) * (2 * G) + 4 * tig) : 0u;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float c[4];
          mma16816_zero(c, qz[mt][0], qz[mt][1], qz[mt][2], qz[mt][3], kz[n], kz[n]);
          const float2 unit = make_float2(64.f / kCode, 64.f / kCode);
          float2 acc0 = __fmul2_rn(make_float2(c[0], c[1]), unit), acc1;  // rows 0..7, 8..15
          if constexpr (!kF32 && NT > 1) acc1 = __fmul2_rn(make_float2(c[2], c[3]), unit);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t w = kc[n * G + g], w8 = w >> 8;
            const float2 sc = make_float2(h_lo(ks[n * G + g]), h_hi(ks[n * G + g]));
            float d[4];
            mma16816_zero(d, qa[mt][g][0][0], qa[mt][g][0][1], qa[mt][g][0][2], qa[mt][g][0][3], low<kF32>(w),
                          high<kF32>(w));
            float2 d0, d1;
            if constexpr (kBoth) {
              float e[4];
              mma16816_zero(e, qa[mt][g][0][0], qa[mt][g][0][1], qa[mt][g][0][2], qa[mt][g][0][3], low<kF32>(w8),
                            high<kF32>(w8));
              d0 = __fadd2_rn(make_float2(d[0], d[1]), make_float2(e[2], e[3]));
            } else {
              mma16816(d, qa[mt][g][1][0], qa[mt][g][1][1], qa[mt][g][1][2], qa[mt][g][1][3], low<kF32>(w8),
                       high<kF32>(w8));
              d0 = make_float2(d[0], d[1]);
              d1 = make_float2(d[2], d[3]);
              if constexpr (kF32) d0 = __fadd2_rn(d0, d1);
            }
            acc0 = __ffma2_rn(d0, sc, acc0);
            if constexpr (!kF32 && NT > 1) acc1 = __ffma2_rn(d1, sc, acc1);
          }
          const int t0 = kF32 ? mt : 2 * mt;
          s[t0][u][2 * n] = acc0.x;
          s[t0][u][2 * n + 1] = acc0.y;
          if constexpr (!kF32 && NT > 1) {
            s[t0 + 1][u][2 * n] = acc1.x;
            s[t0 + 1][u][2 * n + 1] = acc1.y;
          }
        }
      }
    }
    // The peak moves only when a score passes it by more than kHead (or a scale the largest
    // one allowed so far), so most steps need one vote and no shuffle.
    bool over = hmax2(top, cap) != cap;
    float mx[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float r[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        if constexpr (kMasked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int p = pos + 16 * u + 8 * (i / 2) + 2 * tig + (i & 1);
            if (p >= lim[t] || p >= p1) s[t][u][i] = -INFINITY;
          }
        }
        r[u] = max3(fmaxf(s[t][u][0], s[t][u][1]), s[t][u][2], s[t][u][3]);
      }
#pragma unroll
      for (int u = 1; u < SUB; ++u) r[0] = fmaxf(r[0], r[u]);
      mx[t] = r[0];
      over |= r[0] > bound[t];
    }
    if (__any_sync(0xFFFFFFFFu, over)) {
      top = hmax2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = hmax2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      top = max(top & 0xFFFFu, top >> 16);
      const int before = lift, exponent = (int)(top >> 10), boosted = boost;  // top < 2^(exponent - 14)
      lift = min(lift, 29 - kHead - exponent);  // weight * scale < 2^15
      boost = min(boost, exponent < 4 ? 15 - exponent : 0);
      const float less = __uint_as_float((uint32_t)(127 + boost - boosted) << 23);
      cap = boost > 0 ? 0u : (((uint32_t)(30 - kHead - lift) << 10) - 1u) * 0x00010001u;
      if (boost > 0) {
        if constexpr (kCentre) middle = 7.5f * __uint_as_float((uint32_t)(127 - boost) << 23);
#pragma unroll 1
        for (int e = lane; e < SUB * D / 4; e += 32) {  // D bytes of scales a tile
          const uint32_t at = smem_u32(tiles) + e / (D / 4) * L::kBytes + L::kVs + e % (D / 4) * 4;
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(hmul2(lds32(at), (uint32_t)(15 + boost) * 0x04000400u)));
        }
        fence_proxy_async_smem();  // (the next copy into these bytes comes behind)
        __syncwarp();
      } else if constexpr (kCentre) {
        middle = 7.5f;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mx[t] = fmaxf(mx[t], __shfl_xor_sync(0xFFFFFFFFu, mx[t], 1));
        mx[t] = fmaxf(mx[t], __shfl_xor_sync(0xFFFFFFFFu, mx[t], 2));
        const bool first = bound[t] == -INFINITY;  // nothing kept so far (but a NaN, which stays one)
        const float now = first ? mx[t] : fmaxf(peak[t], mx[t]);
        const float b = now == -INFINITY ? 0.f : now;
        const float corr = first ? 0.f : ex2(fmaf(peak[t] - b, kscale[t], (float)(lift - before)));
        peak[t] = b;
        bound[t] = __fadd_rd(now, kHead / kscale[t]);  // (never more than kHead above)
        const float c0 = __shfl_sync(0xFFFFFFFFu, corr, 8 * tig), c1 = __shfl_sync(0xFFFFFFFFu, corr, 8 * tig + 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) oz[t][i] *= i ? c1 : c0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][g][j][i] *= ((i & 1) ? c1 : c0) * less;
      }
    }
    // weights, and the minima's product
    uint32_t vs[SUB][2 * G], wp[SUB][NT][2];  // weights of positions 2 tig, 2 tig + 1 (+ 8)
    [[maybe_unused]] float w[SUB][NT][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      const uint8_t* tile = tiles + u * L::kBytes;
      uint32_t vz[2], sz[2];  // sz: scales of group gid, as rows 8..15 of the minima's operand
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        vz[n] = gid < G ? lds_u1(tile + L::kVz + gid * 32 + n * 16 + tig * 4) : gid == G ? 0x3C003C00u : 0u;
        sz[n] = kCentre && gid < G ? lds_u1(tile + L::kVs + (n * G + gid) / 4 * 64 + tig * 16 + (n * G + gid) % 4 * 4) : 0u;
        if constexpr (kMasked) {
          const int p = pos + 16 * u + 8 * n + 2 * tig;
          const uint32_t keep = gid >= G ? ~0u : (p < p1 ? 0xFFFFu : 0u) | (p + 1 < p1 ? 0xFFFF0000u : 0u);
          vz[n] = finite2(vz[n]) & keep;
          sz[n] = finite2(sz[n]) & keep;
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float x[4];
        uint32_t wl[2];  // low parts
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          // (the difference first: scores far from zero keep their order, and equal ones their weights)
          const float2 e = __ffma2_rn(__fadd2_rn(make_float2(s[t][u][i], s[t][u][i + 1]), make_float2(-peak[t], -peak[t])),
                                      make_float2(kscale[t], kscale[t]), make_float2((float)lift, (float)lift));
          x[i] = ex2(e.x);
          x[i + 1] = ex2(e.y);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          if constexpr (kF32) split2(x[2 * n], x[2 * n + 1], wp[u][t][n], wl[n]);
          else wp[u][t][n] = pack_h(x[2 * n], x[2 * n + 1]);
        }
        if constexpr (kF32) w[u][t][0] = x[0], w[u][t][1] = x[1], w[u][t][2] = x[2], w[u][t][3] = x[3];
        float z[4];
        if constexpr (kF32) {
          mma16816_zero(z, vz[0], sz[0], vz[1], sz[1], wl[0], wl[1]);
          mma16816(z, vz[0], sz[0], vz[1], sz[1], wp[u][t][0], wp[u][t][1]);
        } else {
          mma16816_zero(z, vz[0], sz[0], vz[1], sz[1], wp[u][t][0], wp[u][t][1]);
        }
        oz[t][0] += kCentre ? fmaf(middle, z[2], z[0]) : z[0];
        oz[t][1] += kCentre ? fmaf(middle, z[3], z[1]) : z[1];
      }
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int v = 0; v < 2 * G / 4; ++v) {
        const uint4 y = lds_u4(tiles + u * L::kBytes + L::kVs + v * 64 + tig * 16);
        vs[u][4 * v] = y.x; vs[u][4 * v + 1] = y.y; vs[u][4 * v + 2] = y.z; vs[u][4 * v + 3] = y.w;
      }
    // values, a group of both tiles at a time
#pragma unroll
    for (int g2 = 0; g2 < G; g2 += 2) {
      uint4 vc[SUB];
#pragma unroll
      for (int u = 0; u < SUB; ++u) vc[u] = lds_u4(tiles + u * L::kBytes + L::kV + g2 / 2 * 512 + lane * 16);
#pragma unroll
      for (int g = g2; g < g2 + 2; ++g) {
        float y0[NT][4], y1[NT][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const uint32_t x0 = g & 1 ? vc[u].z : vc[u].x, x1 = g & 1 ? vc[u].w : vc[u].y, x2 = x0 >> 8, x3 = x1 >> 8;
          const uint32_t a0 = low_v<kCentre>(x0), a1 = high_v<kCentre>(x0), a2 = low_v<kCentre>(x1), a3 = high_v<kCentre>(x1);
          const uint32_t b0 = low_v<kCentre>(x2), b1 = high_v<kCentre>(x2), b2 = low_v<kCentre>(x3), b3 = high_v<kCentre>(x3);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            uint32_t p[2], q[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const uint32_t sc = vs[u][n * G + g];
              if constexpr (kF32) split2(w[u][t][2 * n] * h_lo(sc), w[u][t][2 * n + 1] * h_hi(sc), p[n], q[n]);
              else if constexpr (kExact) split2(h_lo(wp[u][t][n]) * h_lo(sc), h_hi(wp[u][t][n]) * h_hi(sc), p[n], q[n]);
              else p[n] = hmul2(wp[u][t][n], sc);
              if constexpr (kMasked) {  // a scale behind the mask may be anything
                const int at = pos + 16 * u + 8 * n + 2 * tig;
                const uint32_t keep = (at < lim[t] && at < p1 ? 0xFFFFu : 0u) | (at + 1 < lim[t] && at + 1 < p1 ? 0xFFFF0000u : 0u);
                p[n] &= keep;
                if constexpr (kExact) q[n] &= keep;
              }
            }
            if constexpr (kExact) {
              if (u == 0) {
                mma16816_zero(y0[t], a0, a1, a2, a3, q[0], q[1]);
                mma16816_zero(y1[t], b0, b1, b2, b3, q[0], q[1]);
              } else {
                mma16816(y0[t], a0, a1, a2, a3, q[0], q[1]);
                mma16816(y1[t], b0, b1, b2, b3, q[0], q[1]);
              }
              mma16816(y0[t], a0, a1, a2, a3, p[0], p[1]);
              mma16816(y1[t], b0, b1, b2, b3, p[0], p[1]);
            } else if (u == 0) {
              mma16816_zero(y0[t], a0, a1, a2, a3, p[0], p[1]);
              mma16816_zero(y1[t], b0, b1, b2, b3, p[0], p[1]);
            } else {
              mma16816(y0[t], a0, a1, a2, a3, p[0], p[1]);
              mma16816(y1[t], b0, b1, b2, b3, p[0], p[1]);
            }
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          add4(o[t][g][0], y0[t]);
          add4(o[t][g][1], y1[t]);
        }
      }
    }
  };

  bool alive = true;
  const int clear = min(see_all, p1);  // positions that need no mask
  int slot = 0;
  uint32_t parity = 0;
  for (int i = 0; i < mine; ++i) {
    alive = __all_sync(0xFFFFFFFFu, kv4_wait(&full[warp][slot], parity, a.c.status));
    if (!alive) break;
    if (!slot_bad[warp][slot]) {
      const uint8_t* tiles = ring + slot * kStageBytes;
      int at = (first + kWarps * i) * kStagePos;
      const int end = min(p1, at + kStagePos);
#pragma unroll 1
      for (; at < end; at += 16 * SUB, tiles += SUB * L::kBytes) {
        if (at + 16 * SUB <= clear) step(tiles, at, std::false_type{});
        else step(tiles, at, std::true_type{});
      }
    }
    __syncwarp();
    if (i + kStages < mine) issue(i + kStages, slot);
    if (++slot == kStages) {
      slot = 0;
      parity ^= 1u;
    }
  }
  if (!alive) {  // copies still in flight must land before the CTA's shared memory goes
    for (int i = 0; i < kStages; ++i) kv4_wait(&full[warp][i], 0, a.c.status), kv4_wait(&full[warp][i], 1, a.c.status);
  }

  // ---- merge of the warps' states, in the ring's memory ----
  __syncthreads();
  float* ob = reinterpret_cast<float*>(smem);            // [warp][row][D]
  float* ml = ob + kWarps * kRows * D;                   // [warp][row][2]
  float* own = ml + kWarps * kRows * 2;                  // [row][D + 4], of a cluster's CTA
  // without the lift, which a reference far from zero would swallow
  const float down = __uint_as_float((uint32_t)(127 - lift) << 23), unboost = __uint_as_float((uint32_t)(127 - boost) << 23),
              c_low = kLow * down * unboost, c_high = kHigh * down * unboost;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (tig == 0) ml[(warp * kRows + 8 * t + gid) * 2] = peak[t] * kscale[t];
    oz[t][0] *= down;
    oz[t][1] *= down;
    if (gid == G) {  // the row of ones has the sums of the weights
      ml[(warp * kRows + 8 * t + 2 * tig) * 2 + 1] = oz[t][0];
      ml[(warp * kRows + 8 * t + 2 * tig + 1) * 2 + 1] = oz[t][1];
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // the minima's part of group g is in the lanes with gid = g
      const float z0 = __shfl_sync(0xFFFFFFFFu, oz[t][0], 4 * g + tig), z1 = __shfl_sync(0xFFFFFFFFu, oz[t][1], 4 * g + tig);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* d0 = ob + (warp * kRows + 8 * t + 2 * tig) * D + 32 * g + 4 * gid + 2 * j;
        *reinterpret_cast<float2*>(d0) =
            make_float2(fmaf(o[t][g][j][0], c_low, z0), fmaf(o[t][g][j][2], c_high, z0));
        *reinterpret_cast<float2*>(d0 + D) =
            make_float2(fmaf(o[t][g][j][1], c_low, z1), fmaf(o[t][g][j][3], c_high, z1));
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kRows * (D / 8); e += kThreadsA) {
    const int r = e / (D / 8), w8 = e % (D / 8), row = row0 + r;
    if (row > last_row) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)  // a sum of zero: this warp had nothing for the row
      top = fmaxf(top, ml[(w * kRows + r) * 2 + 1] == 0.f ? -INFINITY : ml[(w * kRows + r) * 2]);
    float sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ml[(w * kRows + r) * 2 + 1] == 0.f ? 0.f : ex2(ml[(w * kRows + r) * 2] - top);
      sum = fmaf(f, ml[(w * kRows + r) * 2 + 1], sum);
      const float* src = ob + (w * kRows + r) * D + 8 * w8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(f, src[i], x[i]);
    }
    if (a.n_split > 1) {
      // for the join: in the workspace, or in this CTA's shared memory for its cluster
      float* dst = CLUSTER ? own + r * (D + 4) : a.part + ((size_t)blockIdx.x * kRows + r) * (D + 4);
      store8<float>(dst + 4 + 8 * w8, x);
      if (w8 == 0) *reinterpret_cast<float2*>(dst) = make_float2(top, sum);
    } else {
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // 0: the row sees nothing
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      store8<T>(a.out + (seq.row0 + row / a.rep) * a.o_row + (head * a.rep + row % a.rep) * a.o_head + 8 * w8 * sizeof(T), x);
    }
  }
  if constexpr (CLUSTER) {
    // the cluster's CTAs are the splits: each joins a share of the rows out of all their
    // shared memories
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int e = threadIdx.x * a.n_split + split; e < kRows * (D / 8); e += kThreadsA * a.n_split) {
      const int r = e / (D / 8), w8 = e % (D / 8), row = row0 + r;
      if (row > last_row) break;
      float top = -INFINITY;
      for (int q = 0; q < a.n_split; ++q) top = fmaxf(top, cluster.map_shared_rank(own, q)[r * (D + 4)]);
      float sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int q = 0; q < a.n_split; ++q) {
        const float* p = cluster.map_shared_rank(own, q) + r * (D + 4);
        const float2 ml = *reinterpret_cast<const float2*>(p);
        const float4 u = *reinterpret_cast<const float4*>(p + 4 + 8 * w8), v = *reinterpret_cast<const float4*>(p + 8 + 8 * w8);
        const float f = top == -INFINITY ? 0.f : ex2(ml.x - top);
        const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        sum = fmaf(f, ml.y, sum);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(f, y[i], x[i]);
      }
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv;
      store8<T>(a.out + (seq.row0 + row / a.rep) * a.o_row + (head * a.rep + row % a.rep) * a.o_head + 8 * w8 * sizeof(T), x);
    }
    cluster.sync();  // no CTA leaves while another reads its memory
  }
}

// Joins the splits of a row, a CTA per row: a warp's lanes look at the splits' references
// and sums together, then D / 4 threads per split sum the values, all loads independent.
template <int D, class T, int ROWS>
__global__ void __launch_bounds__(128) attn_join(const AttnArgs a) {
  constexpr int kRows = ROWS, kPer = D / 4, kGroups = 128 / kPer;
  __shared__ float4 red[kGroups][kPer];
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x % kRows, tile = blockIdx.x / kRows;
  int idx = tile;
  const int rt = a.n_rt - 1 - idx % a.n_rt;
  idx /= a.n_rt;
  const int head = idx % a.c.n_kv_heads, si = idx / a.c.n_kv_heads;
  const Kv4Seq seq = kv4_seq(a.b, si);
  const int n_rows = seq.n * a.rep, row0 = rt * kRows, last_row = min(n_rows, row0 + kRows) - 1, row = row0 + r;
  const int see_any = max(0, seq.len - seq.n + last_row / a.rep + 1);
  const int n = max(1, min(a.n_split, (see_any + a.split_len - 1) / a.split_len));
  const float* part = a.part + ((size_t)tile * a.n_split * kRows + r) * (D + 4);
  const size_t stride = (size_t)kRows * (D + 4);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the splits' kernel is done and its writes are seen
  if (!seq.ok || row > last_row) return;
  float top = -INFINITY;
  for (int s = lane; s < n; s += 32) top = fmaxf(top, __ldcg(part + s * stride));
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const int g = threadIdx.x / kPer, w = threadIdx.x % kPer;
  float sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = g; s < n; s += kGroups) {
    const float* p = part + s * stride;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p));
    const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 4 + 4 * w));
    const float f = top == -INFINITY ? 0.f : ex2(ml.x - top);
    sum = fmaf(f, ml.y, sum);
    x.x = fmaf(f, y.x, x.x);
    x.y = fmaf(f, y.y, x.y);
    x.z = fmaf(f, y.z, x.z);
    x.w = fmaf(f, y.w, x.w);
  }
  __shared__ float sums[kGroups];
  red[g][w] = x;
  if (w == 0) sums[g] = sum;
  __syncthreads();
  if (threadIdx.x >= D / 8) return;
  float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const float4 u = red[i][2 * threadIdx.x], v = red[i][2 * threadIdx.x + 1];
    y[0] += u.x; y[1] += u.y; y[2] += u.z; y[3] += u.w;
    y[4] += v.x; y[5] += v.y; y[6] += v.z; y[7] += v.w;
    sum += sums[i];
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] *= inv;
  store8<T>(a.out + (seq.row0 + row / a.rep) * a.o_row + (head * a.rep + row % a.rep) * a.o_head + 8 * threadIdx.x * sizeof(T), y);
}

// The same for a prompt's tiles, many rows of few splits: D / 8 threads per row, one split
// after another (a CTA per row took 16 us for 64 tiles of 256 rows).
template <int D, class T>
__global__ void __launch_bounds__(128) attn_join_prompt(const AttnArgs a) {
  constexpr int kRows = kKv4PromptRows, kPer = D / 8, kStep = 128 / kPer, kCtas = kRows / kStep;
  const int w8 = threadIdx.x % kPer, r = blockIdx.x % kCtas * kStep + threadIdx.x / kPer, tile = blockIdx.x / kCtas;
  const Kv4Block block = kv4_block(a, tile);
  const int head = block.head;
  const Kv4Seq seq = kv4_seq(a.b, max(block.seq, 0));
  const int n_rows = seq.n * a.rep;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (block.seq < 0 || !seq.ok || block.tile < 0 || block.tile >= (n_rows + kRows - 1) / kRows) return;
  const int row0 = block.tile * kRows, last_row = min(n_rows, row0 + kRows) - 1, row = row0 + r;
  const int see_any = max(0, seq.len - seq.n + last_row / a.rep + 1);
  const int n = max(1, min(a.n_split, (see_any + a.split_len - 1) / a.split_len));
  if (row > last_row) return;
  const float* part = a.part + ((size_t)tile * a.n_split * kRows + r) * (D + 4);
  const size_t stride = (size_t)kRows * (D + 4);
  float top = -INFINITY, sum = 0.f, x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = 0; s < n; ++s) top = fmaxf(top, __ldcg(part + s * stride));
#pragma unroll 4
  for (int s = 0; s < n; ++s) {
    const float* p = part + s * stride;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p));
    const float4 u = __ldcg(reinterpret_cast<const float4*>(p + 4 + 8 * w8)), v = __ldcg(reinterpret_cast<const float4*>(p + 8 + 8 * w8));
    const float f = top == -INFINITY ? 0.f : ex2(ml.x - top), y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    sum = fmaf(f, ml.y, sum);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(f, y[i], x[i]);
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= inv;
  store8<T>(a.out + (seq.row0 + row / a.rep) * a.o_row + (head * a.rep + row % a.rep) * a.o_head + 8 * w8 * sizeof(T), x);
}

struct Plan {
  bool prompt;  // many rows of 16-bit queries: the tcgen05 kernel
  int nt, n_rt, n_split, split_len;
  int n_blocks, row_shift;  // see Kv4AttnSplit
  bool cluster;  // the splits of a row tile are a cluster and join in shared memory
  long long ctas;
  int64_t part_bytes;
};

// SMs of the current device (looked up once per device), 0 on an error.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (kv4_status(cudaGetDevice(&dev)) != MK_OK) return 0;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (kv4_status(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != MK_OK) return 0;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// How a call is cut up, from its bounds alone.
mk_status plan_few(const mk_kv4_cache* c, const mk_kv4_batch* b, int rep, int dtype, Plan* p) {
  const int sms = sm_count();
  if (sms <= 0) return MK_ERR_CUDA;
  const long long rows = std::max<long long>(b->max_new, 1) * rep;  // 0: still looks at the spans
  // Many rows of 16-bit types: 256-row tiles on tcgen05, where that is expected to be
  // faster.  Measured (one B200, us, 64- / 128-value heads): there a tile of 128 positions takes
  // 1.85 / 2.2 (fp16 2.15 / 2.75) and a CTA 6 more, one CTA on an SM, and a join 5 and 0.35 per split; here
  // 16 rows x 16 positions take 0.00033 / 0.00062 of the whole GPU, and a call 10 more.  E.g.
  // 8 kv heads x 4 query heads over 16384 positions, 64 values: 16 new tokens 24 here, 27
  // there; 128 tokens 106 here, 243 there unsplit, 45 split; 512 tokens 334, 248, 134.
  // Sequences of unequal spans: a batch of n_rows rows has at most n_rows * rep / 256 + n_seqs row tiles,
  // by which the times go.  Where that is less than half of what it is with as many for every sequence
  // as for the longest, so do the grid and the workspace (64 sequences, one of 8192 new tokens, 131072
  // positions: 35 GB without, 0.8).  Looking for a tile's sequence takes longer than an idle CTA: eight
  // prompts of 517 to 1420 tokens, 129 tiles of 184, 187 us so, 195 by the batch's.
  const long long seq_heads = (long long)b->n_seqs * c->n_kv_heads, all_rows = (long long)b->n_rows * rep;
  const auto row_tiles = [&](long long of) { return std::min(b->n_seqs * ((rows + of - 1) / of), all_rows / of + b->n_seqs); };
  p->prompt = false;
  p->n_blocks = p->row_shift = 0;
  if (dtype != 2 && rows > 16) {
    const bool wide = c->head_dim == 128;
    const long long n_rt = (rows + kKv4PromptRows - 1) / kKv4PromptRows, blocks = row_tiles(kKv4PromptRows);
    const bool packed = 2 * blocks < n_rt * b->n_seqs;
    const long long base = blocks * c->n_kv_heads, grid = packed ? base : n_rt * seq_heads;
    const long long tiles = (b->max_len + 127) / 128;
    // splits of at least four tiles, as many as keep one CTA per SM; and of at most 256, since
    // sums in tensor memory are cut off, not rounded: 0.7e-8 a position, measured (131072
    // positions in one split: results 9e-4 too small)
    const long long n_split = std::max({1ll, std::min(sms / std::max(base, 1ll), tiles / 4), (tiles + 255) / 256});
    const long long per = std::max(1ll, (tiles + n_split - 1) / n_split);
    const double here = 10 + (double)c->n_kv_heads * row_tiles(16) * ((b->max_len + 15) / 16) * (wide ? 0.00062 : 0.00033);
    const double tile = dtype == 0 ? (wide ? 2.2 : 1.85) : wide ? 2.75 : 2.15;
    const double there = (double)((base * n_split + sms - 1) / sms) * (6 + per * tile) + (n_split > 1 ? 5 + 0.35 * n_split : 0);
    if (there < here) {
      p->prompt = true;
      p->cluster = false;
      p->nt = 0;
      p->n_rt = (int)n_rt;
      if (packed) {
        p->n_blocks = (int)blocks;
        for (p->row_shift = 8; kKv4PromptRows >> p->row_shift < rep;) --p->row_shift;  // 256 / rep rows
      }
      p->n_split = (int)((tiles + per - 1) / std::max(per, 1ll));
      if (p->n_split < 1) p->n_split = 1;
      p->split_len = (int)std::min<long long>(per * 128, 0x7FFFFF80);
      p->ctas = grid * p->n_split;
      static_assert(kKv4PromptRows == 1 << 8, "");
      if (p->ctas > 0x7FFFFFFF / kKv4PromptRows) return MK_ERR_UNSUPPORTED;
      p->part_bytes = p->n_split > 1 ? p->ctas * kKv4PromptRows * (c->head_dim + 4) * (int64_t)sizeof(float) : 0;
      return MK_OK;
    }
  }
  p->nt = rows <= 8 ? 1 : 2;
  const long long n_rt = (rows + 8 * p->nt - 1) / (8 * p->nt);
  const long long base = seq_heads * n_rt;
  const int unit = MK_KV4_PAGE;
  const long long pages = (b->max_len + unit - 1) / unit;
  // Splits: enough that every SM has about two CTAs, in pieces of at least a page per warp
  // (one sequence of 8200 positions, 8 kv heads of 64: 15.9 us with 4 splits, 9.1 with 32);
  // and where there are more, up to eight CTAs per SM in pieces of 32 pages, so that
  // sequences of unequal length fill the SMs evenly (64 of up to 16384 positions, kv heads
  // of 128: 190 us unsplit, 149 so; 64 of about 2000 lose by a split, 55 to 65 us).
  // A sum of 32 bits that a warp keeps over more than 4096 positions shows in 16-bit results, whose
  // codes' and minima's parts cancel: at most 16384 to a split in any case.
  const long long least = dtype == 2 ? 1 : std::max(1ll, (pages + 255) / 256);
  long long n_split = least;
  if (base > 0)
    n_split = std::max({n_split, std::min(2ll * sms / base, pages / kWarps), std::min(8ll * sms / base, pages / 32)});
  // Where the splits fill the SMs about once, up to 16 of them are a cluster (a power of
  // two): no workspace and no second launch (eight lanes of about 1000 positions in fp32:
  // 9.6 -> 8.3 us).  Longer grids lose by it, a cluster's CTAs being placed together (64
  // sequences of up to 16384 positions: 152 -> 204 us).
  p->cluster = n_split > 1 && n_split <= 16 && base * n_split <= 2ll * sms;
  if (p->cluster) {
    long long c = 2;
    while (2 * c <= std::min(n_split, 16ll) || c < least) c *= 2;
    n_split = c;
  }
  const long long per = std::max(1ll, (pages + n_split - 1) / n_split);
  if (!p->cluster) n_split = std::max(1ll, (pages + per - 1) / per);
  p->n_rt = (int)n_rt;
  p->n_split = (int)n_split;
  p->split_len = (int)std::min<long long>(per * unit, 0x7FFFFFC0);
  p->ctas = base * n_split;
  if (p->ctas > 0x7FFFFFFF / 64) return MK_ERR_UNSUPPORTED;
  p->part_bytes = n_split > 1 && !p->cluster ? p->ctas * 8 * p->nt * (c->head_dim + 4) * (int64_t)sizeof(float) : 0;
  return MK_OK;
}

// A join, launched while the splits run (its first loads wait for them).
template <int D, class T, int ROWS>
mk_status launch_join(const AttnArgs& a, const Plan& p, cudaStream_t s) {
  constexpr bool kPrompt = ROWS == kKv4PromptRows;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.gridDim = dim3((unsigned)(p.ctas / p.n_split * (kPrompt ? ROWS / (128 / (D / 8)) : ROWS)));
  cfg.blockDim = dim3(128);
  cfg.stream = s;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e;
  if constexpr (kPrompt) e = cudaLaunchKernelEx(&cfg, attn_join_prompt<D, T>, a);
  else e = cudaLaunchKernelEx(&cfg, attn_join<D, T, ROWS>, a);
  return kv4_status(e);
}

template <int D, class T, int NT>
mk_status launch_few(const AttnArgs& a, const Plan& p, cudaStream_t s) {
  constexpr int kMerge = 8 * NT * (kWarps * (D + 2) + D + 4) * 4;
  constexpr int kSmem = kMerge > kWarps * kStages * kStageBytes ? kMerge : kWarps * kStages * kStageBytes;
  static std::atomic<uint64_t> ready{0}, ready_cluster{0};  // devices whose attributes are set
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  cfg.blockDim = dim3(kThreadsA);
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  if (p.cluster) {
    const void* kernel = reinterpret_cast<const void*>(attn_few<D, T, NT, true>);
    if (!kv4_allow_smem(kernel, kSmem, &ready_cluster, true)) return MK_ERR_CUDA;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.n_split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return kv4_status(cudaLaunchKernelEx(&cfg, attn_few<D, T, NT, true>, a));
  }
  if (!kv4_allow_smem(reinterpret_cast<const void*>(attn_few<D, T, NT, false>), kSmem, &ready, false)) return MK_ERR_CUDA;
  const mk_status st = kv4_status(cudaLaunchKernelEx(&cfg, attn_few<D, T, NT, false>, a));
  return st == MK_OK && p.n_split > 1 ? launch_join<D, T, 8 * NT>(a, p, s) : st;
}

template <int D, class T>
mk_status launch_few(const AttnArgs& a, const Plan& p, cudaStream_t s) {
  if (p.nt == 1) return launch_few<D, T, 1>(a, p, s);
  return launch_few<D, T, 2>(a, p, s);
}

mk_status check_attention(const mk_kv4_cache* c, int32_t layer, const mk_kv4_batch* b, int32_t n_heads, int32_t dtype) {
  const mk_status st = kv4_check(c, layer, b, dtype);
  if (st != MK_OK) return st;
  if (n_heads < 1 || n_heads % c->n_kv_heads) return MK_ERR_INVALID_ARG;
  const int rep = n_heads / c->n_kv_heads;
  if (rep != 1 && rep != 2 && rep != 4 && rep != 8) return MK_ERR_UNSUPPORTED;
  return MK_OK;
}

}  // namespace

bool kv4_allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* ready, bool large_cluster) {
  int dev = 0;
  if (kv4_status(cudaGetDevice(&dev)) != MK_OK) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready->load(std::memory_order_relaxed) & bit) return true;
  if (kv4_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != MK_OK) return false;
  if (large_cluster && kv4_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != MK_OK)
    return false;
  ready->fetch_or(bit, std::memory_order_relaxed);
  return true;
}

}  // namespace mk

using namespace mk;

extern "C" mk_status mk_kv4_attention_workspace(const mk_kv4_cache* cache, const mk_kv4_batch* batch, int32_t n_heads,
                                                int32_t dtype, int64_t* bytes) {
  if (!bytes) return MK_ERR_INVALID_ARG;
  mk_status st = check_attention(cache, 0, batch, n_heads, dtype);
  if (st != MK_OK) return st;
  *bytes = 0;
  if (batch->n_rows == 0) return MK_OK;
  Plan p;
  st = plan_few(cache, batch, n_heads / cache->n_kv_heads, dtype, &p);
  if (st == MK_OK) *bytes = p.part_bytes;
  return st;
}

extern "C" mk_status mk_kv4_attention(const mk_kv4_cache* cache, int32_t layer, const mk_kv4_batch* batch,
                                      const mk_kv4_rows* q, const mk_kv4_rows* out, int32_t n_heads, int32_t dtype,
                                      float scale, void* workspace, int64_t workspace_bytes, void* stream) {
  mk_status st = check_attention(cache, layer, batch, n_heads, dtype);
  if (st != MK_OK) return st;
  if (!std::isfinite(scale * 1.44269504088896341f)) return MK_ERR_INVALID_ARG;
  if (batch->n_rows == 0) return MK_OK;
  st = kv4_check_rows(q, dtype, batch->n_rows, n_heads, cache->head_dim, false);
  if (st == MK_OK) st = kv4_check_rows(out, dtype, batch->n_rows, n_heads, cache->head_dim, true);
  if (st != MK_OK) return st;
  if (kv4_error_pending()) return MK_ERR_CUDA;
  const int rep = n_heads / cache->n_kv_heads;
  Plan p;
  st = plan_few(cache, batch, rep, dtype, &p);
  if (st != MK_OK) return st;
  if (p.part_bytes > 0 && (!workspace || ((uintptr_t)workspace & 15u) || workspace_bytes < p.part_bytes))
    return MK_ERR_INVALID_ARG;
  const int size = dtype == 2 ? 4 : 2;
  const AttnArgs a{{*cache, *batch, static_cast<const char*>(q->p), static_cast<char*>(out->p), q->row_stride * size,
              q->head_stride * size, out->row_stride * size, out->head_stride * size, layer, rep,
              scale * 1.44269504088896341f},
             p.n_split, p.split_len, p.n_rt, p.n_blocks, p.row_shift, static_cast<float*>(workspace)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.prompt) {
    st = kv4_prompt(a, dtype, s);
    if (st != MK_OK || p.n_split == 1) return st;
    if (cache->head_dim == 64)
      return dtype == 0 ? launch_join<64, __nv_bfloat16, kKv4PromptRows>(a, p, s)
                        : launch_join<64, __half, kKv4PromptRows>(a, p, s);
    return dtype == 0 ? launch_join<128, __nv_bfloat16, kKv4PromptRows>(a, p, s)
                      : launch_join<128, __half, kKv4PromptRows>(a, p, s);
  }
  if (cache->head_dim == 64) {
    if (dtype == 0) return launch_few<64, __nv_bfloat16>(a, p, s);
    if (dtype == 1) return launch_few<64, __half>(a, p, s);
    return launch_few<64, float>(a, p, s);
  }
  if (dtype == 0) return launch_few<128, __nv_bfloat16>(a, p, s);
  if (dtype == 1) return launch_few<128, __half>(a, p, s);
  return launch_few<128, float>(a, p, s);
}
