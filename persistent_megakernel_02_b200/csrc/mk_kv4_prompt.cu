// mk_kv4_prompt.cu -- causal attention over the 4-bit KV cache for many query rows of
// 16-bit types (prompts), on the tcgen05 tensor cores.
//
// A CTA has 256 query rows (tokens x the rep query heads of one kv head) as two tiles of
// 128, and walks the positions it sees in tiles of 128.  Roles:
//   warps 0-3, 4-7  softmax of query tile 0, 1: one thread per row
//   warps 8-11      dequantise: codes to fp16 K and V in the swizzled shared-memory layout
//   warps 12, 13    issue the matrix instructions of query tile 0, 1
// Scores S = Q K^T of a half tile (64 positions) go into 64 columns of tensor memory; the
// row's thread reads them once (maximum, weights) and writes the weights over them as fp16,
// from where they are the A operand of O += W V, which stays in tensor memory.  The next
// half's scores are under way meanwhile, K's buffers are freed apart from V's, and each
// query tile has an issuing warp of its own, so that neither waits for the other.
//
// For bf16 calls K and V are z + s c rounded once to fp16.  V's rounding, 2^-11, is an eighth of
// the output's own.  K's moves a score by up to 2^-11 of its largest products, so it grows with
// the keys: in the 2-norm 1.7e-3 off, as single tokens are, where no channel of all keys is more
// than 30 from zero, 2.4e-3 at 100, 8.9e-3 at 300 (two parts as below: 1.7e-3 throughout, but
// 2048 tokens of 128-value heads take 70 us instead of 58).  For fp16 calls both would show:
// there K, and V of 64-value heads, are two fp16 parts, good to 2^-17 together, and take two
// products.  Errors in the 2-norm, 2048 tokens over 8192 positions: 7.2e-4 rounded, 2.8e-4 so,
// the output's own rounding 2.1e-4; 260 us for bf16's 223, with 128-value heads 376 for 296 (V
// in two parts too: 572).  Queries are scaled by a power of two per row, which is exact in fp16
// but for values 2^-24 below the row's largest, weights are rounded to fp16.  The order of
// values inside 8 and of positions inside 32 is the one the codes come in: queries are permuted
// alike, and S, W and V share the order of positions.  O is rescaled only when a score passes
// the row's peak by more than 16x.
//
// Bound: with 64-value heads the exponentials, 16 per SM and cycle: 2048 cycles for the
// 256 x 128 scores of a tile, 1024 for its products.  A tile takes about 3500 (1.85 us), the
// warps' instructions in between: 2048 bf16 tokens x 32 heads over 8192 positions 223 us, 540
// TFLOP/s; 2048 tokens of 128-value heads, causal, 58 us, 590 TFLOP/s.  (Three or four
// query tiles, which would fill the exponential unit, do not fit tensor memory; sixteen
// softmax warps for the two, 32 columns each, measured 267 us for the former.)
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "mk_kv4.cuh"
#include "mk_kv4.h"
#include "mk_tc.cuh"

namespace mk {
namespace {

constexpr int kPThreads = 14 * 32;
constexpr int kPTile = 128;  // positions per tile, and rows per query tile
constexpr int kPHead = 4;    // log2 of what a weight may pass the peak's by
constexpr int kPLift = 10;   // log2 of the peak's weight: none is above 2^14

// K and V buffers: two of a tile; where K's or V's values have two parts they are of a half
// tile, and four of them with 64-value heads.  (With 128-value heads there is room for two
// halves of K and no more: with V in two parts as well the buffers wait for one another.)
template <int D, class T>
struct PSmem {
  static constexpr bool kK2 = std::is_same<T, __half>::value, kV2 = kK2 && D == 64;
  static constexpr int kQ = D == 64 ? 0 : 2 * kPTile * D * 2;  // both query tiles, if not in tensor memory
  static constexpr int kKV = kPTile * D * 2;      // one K or V buffer
  static constexpr int kBufs = kV2 ? 4 : 2;
  static constexpr int kBytes = 1024 + kQ + 2 * kBufs * kKV;
};

struct PShared {
  uint64_t q_full, k_full[4], k_empty[4], v_full[4], v_empty[4], s_full[2][2], w_full[2][2], wv_done[2], o_full[2], drained[2];
  uint32_t tmem;
  // Blocks of 32 positions whose page id is out of range.  By tile modulo 4: K's buffer is free
  // once the scores are computed, which is before they are masked, so that a tile's flags have
  // to outlive the next tile's but one (the one behind that starts after they have been read).
  uint32_t bad[4][4];
  // first position whose V is NaN, by group: it is zero in the product (0 x NaN would reach
  // rows that do not see it) and put into the rows that see it at the end
  int nan_first[4];
};

// instruction descriptor: D fp32, A and B fp16, both K-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// The issuing warp stays converged and one lane's predicate is inside the statement, so
// that descriptors live in uniform registers (from a branch of one lane each instruction
// took about 80 cycles to issue).
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one));
}
// A in tensor memory: its rows are the lanes, two fp16 values per column
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(one));
}
__device__ __forceinline__ void mma_commit(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
  return e;
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
__device__ __forceinline__ void tmem_get64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, "
      "%23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, "
      "%44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"
      "}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The 8 values of a code word as four pairs (nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7),
// each z + s c rounded once: a code or'ed into the mantissa of 1024 and taken back out.
__device__ __forceinline__ void dequant8(uint32_t x, uint32_t s2, uint32_t z2, uint32_t (&v)[4]) {
  const uint32_t y = x >> 8;
  v[0] = hfma2(hadd2((x & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s2, z2);               // - 1024
  v[1] = hfma2(hfma2((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s2, z2);  // / 16 - 64
  v[2] = hfma2(hadd2((y & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s2, z2);
  v[3] = hfma2(hfma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s2, z2);
}
// The same as two fp16 values: hi = z_a + s_hi c, exact, and lo = z_b + s_lo c, with s_hi and z_a
// the multiples of a grid nearest to s and z, and s_lo, z_b what is left.  With 2^e the leading
// bit of the group's largest value the grid is 2^(e - 8): hi is at most 2^9 + 8 of its steps,
// lo at most 8, where rounding it to fp16 is 2^-17 of the largest.  Rounding to the grid:
// adding 1.5 x 2^10 of its steps and taking them off again.
struct Params {
  uint32_t sh, za, sl, zb;
};
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) { return hadd2(a, b ^ 0x80008000u); }
__device__ __forceinline__ Params split_params(uint32_t s2, uint32_t z2) {
  const uint32_t end = hfma2(s2, 0x4B804B80u, z2) & 0x7FFF7FFFu, low = z2 & 0x7FFF7FFFu;  // |z + 15 s|, |z|
  const uint32_t top = __vmaxu2(end, low);  // (as integers: their order is that of the values)
  uint32_t big = (top & 0x7C007C00u) + 0x0A000A00u;
  big &= __vcmpleu2(big, 0x7A007A00u);  // (from 2^14 on, where the sum could overflow, hi is rounded once)
  const uint32_t bz = big | (~z2 & 0x80008000u);  // of the other sign than z: no overflow either
  Params p;
  p.sh = hsub2(hadd2(s2, big), big);
  p.sl = hsub2(s2, p.sh);
  p.za = hsub2(hadd2(z2, bz), bz);
  p.zb = hsub2(z2, p.za);
  return p;
}
__device__ __forceinline__ void dequant8(uint32_t x, const Params& p, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  const uint32_t y = x >> 8;
  const uint32_t c[4] = {hadd2((x & 0x000F000Fu) | 0x64006400u, 0xE400E400u),
                         hfma2((x & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u),
                         hadd2((y & 0x000F000Fu) | 0x64006400u, 0xE400E400u),
                         hfma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = hfma2(c[i], p.sh, p.za);
    lo[i] = hfma2(c[i], p.sl, p.zb);
  }
}
__device__ __forceinline__ uint32_t both(uint32_t pair, int which) {  // one half of a pair, twice
  return __byte_perm(pair, 0u, which ? 0x3232 : 0x1010);
}
__device__ __forceinline__ bool nan_half(uint32_t h) { return (h & 0x7FFFu) > 0x7C00u; }

// 16-byte chunk c (0..7) of row r in a tile of 128-byte rows, 128-byte swizzle
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// position (in a tile of 128) that column c of S holds: within 32 columns, column
// 8 tig + 4 u + 2 hf + e is row 8 hf + 2 tig + e of the block's tile u
__host__ __device__ constexpr int column_position(int c) {
  return (c & ~31) + 16 * ((c >> 2) & 1) + 8 * ((c >> 1) & 1) + 2 * ((c >> 3) & 3) + (c & 1);
}

template <int D, class T>
__global__ void __launch_bounds__(kPThreads, 1) attn_prompt(const Kv4AttnSplit a) {
  using L = Kv4<D>;
  constexpr int G = L::G;
  constexpr uint32_t kPart = D * 128;  // bytes of a half, or of a part of one
  using M = PSmem<D, T>;
  constexpr bool kK2 = M::kK2, kV2 = M::kV2;  // values in two parts
  constexpr int kBufs = M::kBufs;
  constexpr uint32_t kIdQK = idesc_f16(128, 64), kIdWV = idesc_f16(128, D);
  extern __shared__ uint8_t smem_raw[];
  __shared__ PShared sh;
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* sq = smem;                    // [2][D / 64][128 rows][128 bytes]
  // [buffers][K, V]: a tile each (K [D / 64][128 rows][128 bytes], V [2 halves][D rows][128
  // bytes]), or where there are two parts a half of 64 positions each (K [hi, lo][D / 64][64
  // rows][128 bytes], V [hi, lo][D rows][128 bytes])
  uint8_t* skv = smem + M::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const int split = blockIdx.x % a.n_split;
  const Kv4Block block = kv4_block(a, blockIdx.x / a.n_split);
  if (a.n_blocks && tid == 0) kv4_report_order(a.c, a.b, blockIdx.x);  // (a row tile or more to a sequence)
  const int head = block.head, si = max(block.seq, 0);
  const Kv4Seq seq = kv4_seq(a.b, si);
  if (block.seq < 0 || !seq.ok) {
    if (tid == 0) atomicOr(a.c.status, KV4_BAD_BATCH);
    return;
  }
  const int n_rows = seq.n * a.rep;
  if (block.tile < 0 || block.tile >= (n_rows + 2 * kPTile - 1) / (2 * kPTile)) return;
  const int row0 = block.tile * 2 * kPTile;
  const int start = seq.len - seq.n;  // position of the first query token (may be negative)
  const int p0 = split * a.split_len;  // this split's positions: p0 .. p0 + split_len - 1
  int n_half[2], n_max = 0;            // halves of 64 positions each query tile sees of them; tiles of 128
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int first = row0 + t * kPTile, last = min(n_rows, first + kPTile) - 1;
    n_half[t] = first < n_rows ? (max(0, min(start + last / a.rep + 1 - p0, a.split_len)) + 63) / 64 : 0;
    n_max = max(n_max, (n_half[t] + 1) / 2);
  }
  if (n_max == 0 && split > 0) return;  // the join takes only the splits that hold something

  if (tid < 4) sh.nan_first[tid] = 0x7FFFFFFF;
  if (tid == 0) {
    mbar_init(&sh.q_full, 2 * kPTile);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sh.k_full[i], kK2 ? kPTile / 2 : kPTile);
      mbar_init(&sh.k_empty[i], 2);
      mbar_init(&sh.v_full[i], kV2 ? kPTile / 2 : kPTile);
      mbar_init(&sh.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh.s_full[i][h], 1);
        mbar_init(&sh.w_full[i][h], 4);
      }
      mbar_init(&sh.wv_done[i], 1);
      mbar_init(&sh.o_full[i], 1);
      mbar_init(&sh.drained[i], 1);
    }
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Columns: S0, S1 128 each (two halves of 64 positions), O0, O1 D each.  The weights of a
  // half, 32 columns, lie over the scores of that half.
  const uint32_t tmem = sh.tmem;
  // 64-value queries, 32 columns a tile, are behind them (from shared memory their reads hold
  // up the products: fp16 275 us there for 2048 tokens over 8192 positions, 258 here).
  constexpr uint32_t kO = 256, kQ = 384;
  constexpr bool kQT = D == 64;

  if (warp < 8) {
    // ---------------- softmax: one thread per row ----------------
    const int t = warp >> 2, r_in = tid & 127, row = row0 + t * kPTile + r_in;
    const bool live = row < n_rows;
    float kscale;
    {
      const char* src = a.q + (long long)(seq.row0 + row / a.rep) * a.q_row +
                        (long long)(head * a.rep + row % a.rep) * a.q_head;
      Raw8<T> raw[D / 8];
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        raw[c] = Raw8<T>{};
        if (live) raw[c] = load_raw8<T>(src + c * 16);
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float x[8];
        unpack8(raw[c], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[i]));
      }
      // power of two that brings the row's largest to 2^12 .. 2^13 (rows of zeros and rows
      // with an infinity keep theirs); the sign of the scale goes to the queries, so that
      // the maximum of the accumulated scores is the maximum of the scores
      const int e = mx > 0.f && mx < INFINITY ? min(126, 12 + 127 - (int)(__float_as_uint(mx) >> 23)) : 0;
      const float up = __uint_as_float((uint32_t)(127 + e) << 23), sup = a.scale_log2 < 0.f ? -up : up;
      [[maybe_unused]] uint32_t qt[16];
      kscale = kv4_score_scale(fabsf(a.scale_log2) / up);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        float x[8];
        unpack8(raw[c], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= sup;
        if constexpr (kQT) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qt[4 * (c & 3) + i] = pack_h(x[i], x[i + 4]);
          if ((c & 3) == 3) tmem_st16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kQ + t * 32 + 4 * (c - 3), qt);
        } else {
          *reinterpret_cast<uint4*>(sq + (t * (D / 64) + c / 8) * 16384 + chunk_at(r_in, c % 8)) =
              make_uint4(pack_h(x[0], x[4]), pack_h(x[1], x[5]), pack_h(x[2], x[6]), pack_h(x[3], x[7]));
        }
      }
    }
    if constexpr (kQT) {
      tmem_st_wait();
      tc_fence_before();
    } else {
      fence_proxy_async_smem();
    }
    mbar_arrive(&sh.q_full);

    const int lim = live ? start + row / a.rep + 1 : 0;               // positions this row sees
    const int lim_warp = start + (row0 + t * kPTile + (r_in & ~31)) / a.rep + 1;  // the warp's rows all see these
    const bool whole = row0 + t * kPTile + (r_in | 31) < n_rows;      // no row of the warp is past the end
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t ts = lane_base + (uint32_t)(t * 128), to = lane_base + kO + (uint32_t)(t * D);
    // weights are 2^((score - peak) kscale + kPLift), peak the largest accumulated score when it was
    // last moved (0: none so far), which happens when one passes `bound`
    float peak = 0.f, bound = -INFINITY, sum = 0.f;
    const int n = n_half[t];
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int h = i & 1, buf = (i >> 1) & 1;
      ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.s_full[t][h], buf, a.c.status));
      if (!ok) break;
      tc_fence_after();
      uint32_t s[64];
      tmem_get64(ts + 64 * h, s);
      const int pos = p0 + i * 64, left = lim - pos;  // columns with position < left are seen
      const uint32_t bad0 = sh.bad[(i >> 1) & 3][2 * h], bad1 = sh.bad[(i >> 1) & 3][2 * h + 1];
      float mx;
      if (whole && pos + 64 <= lim_warp && (bad0 | bad1) == 0) {
        float q[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          q[(c >> 1) & 3] = max3(q[(c >> 1) & 3], __uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        mx = fmaxf(max3(q[0], q[1], q[2]), q[3]);
      } else {  // (with a maximum of its own: a mask in the common code is paid by every tile)
        mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          if (column_position(c) >= left || (c < 32 ? bad0 : bad1)) s[c] = 0xFF800000u;
          mx = fmaxf(mx, __uint_as_float(s[c]));
        }
      }
      if (__any_sync(0xFFFFFFFFu, mx > bound)) {  // the peak moves: seldom
        const bool first = bound == -INFINITY;  // nothing kept so far (but a NaN, which stays one)
        const float now = first ? mx : fmaxf(peak, mx), b = now == -INFINITY ? 0.f : now;
        const float corr = first ? 0.f : ex2((peak - b) * kscale);
        peak = b;
        bound = __fadd_rd(now, kPHead / kscale);  // (never more than kPHead above)
        sum *= corr;
        if (i > 0) {  // O, once the product of the half before is in it
          ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.wv_done[t], (i - 1) & 1, a.c.status));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int d0 = 0; d0 < D; d0 += 16) {
            uint32_t o[16];
            tmem_get16(to + d0, o);
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * corr);
            tmem_st16(to + d0, o);
          }
        }
      }
      float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      const float2 k2 = make_float2(kscale, kscale), b2 = make_float2(-peak, -peak), lift2 = make_float2(kPLift, kPLift);
#pragma unroll
      for (int c0 = 0; c0 < 64; c0 += 32) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          // (the difference first: scores far from zero keep their order, and equal ones their weights)
          float2 x = __ffma2_rn(__fadd2_rn(make_float2(__uint_as_float(s[c0 + c]), __uint_as_float(s[c0 + c + 1])), b2), k2, lift2);
          x.x = ex2(x.x);
          x.y = ex2(x.y);
          part[(c >> 1) & 1] = __fadd2_rn(part[(c >> 1) & 1], x);
          w[c / 2] = pack_h(x.x, x.y);
        }
        tmem_st16(ts + 64 * h + c0 / 2, w);  // (over scores that are in registers)
      }
      sum += (part[0].x + part[0].y) + (part[1].x + part[1].y);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.w_full[t][h]);
    }
    // (a barrier of its own: the phases of wv_done may be two ahead by now, which a parity
    // would take for none)
    if (n > 0 && ok) ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.o_full[t], 0, a.c.status));
    if (ok) {
      tc_fence_after();
      // splits are joined later: the sums as they are, after the reference and the weights' sum
      const float inv = sum == 0.f ? 0.f : a.n_split > 1 ? 1.0f : 1.0f / sum;  // 0: the row sees nothing
      float* part = a.part + ((size_t)blockIdx.x * (2 * kPTile) + t * kPTile + r_in) * (D + 4);
      if (a.n_split > 1 && live) *reinterpret_cast<float2*>(part) = make_float2(sum == 0.f ? -INFINITY : peak * kscale, sum);
      char* dst = a.out + (long long)(seq.row0 + row / a.rep) * a.o_row +
                  (long long)(head * a.rep + row % a.rep) * a.o_head;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t o[16];
        if (n > 0) tmem_get16(to + c0, o);
        const bool nan = n > 0 && sh.nan_first[c0 / 32] < lim;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[i] = n > 0 && sum != 0.f ? __uint_as_float(o[8 * hh + i]) * inv : 0.f;
            if (nan) x[i] = __uint_as_float(0x7FFFFFFFu);
          }
          if (!live) continue;
          if (a.n_split > 1) store8<float>(part + 4 + c0 + 8 * hh, x);
          else store8<T>(dst + (c0 + 8 * hh) * sizeof(T), x);
        }
      }
    }
  } else if (warp < 12) {
    // ---------------- dequantise: warp 8 + w has positions 32 w .. 32 w + 31 of a tile ----------------
    const int w = warp - 8, gid = lane >> 2, tig = lane & 3;
    const int32_t* table = a.b.block_table + (size_t)si * a.b.max_pages;
    const int see = min(seq.len, p0 + n_max * kPTile);  // positions behind are left out (zero)
    // raw operands of this warp's two 16-position tiles
    uint4 kc[2][2 * G / 4] = {}, vc[2][2 * G / 4] = {}, vs[2][2 * G / 4] = {}, ks[2][2] = {};
    uint2 kz[2][2] = {};
    uint32_t vz[2][G][2] = {};
    // page id of tile j, looked up a tile ahead of its loads (-1 where there is no position)
    auto look = [&](int j) {
      const int p = p0 + j * kPTile + 32 * w;
      return j < n_max && p < see ? table[p / MK_KV4_PAGE] : -1;
    };
    auto tile_at = [&](int page) {
      const size_t at = (((size_t)a.layer * a.c.n_pages + page) * a.c.n_kv_heads + head) * kKv4Tiles + 2 * (w & 1);
      return static_cast<const uint8_t*>(a.c.pool) + at * L::kBytes;
    };
    auto load_k = [&](int page) {
      if ((unsigned)page >= (unsigned)a.c.n_pages) return;
      const uint8_t* tile = tile_at(page);
#pragma unroll
      for (int u = 0; u < 2; ++u, tile += L::kBytes) {
#pragma unroll
        for (int v = 0; v < 2 * G / 4; ++v) kc[u][v] = ldnc16(tile + v * 512 + lane * 16);
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
        }
      }
    };
    auto load_v = [&](int page) {
      if ((unsigned)page >= (unsigned)a.c.n_pages) return;
      const uint8_t* tile = tile_at(page);
#pragma unroll
      for (int u = 0; u < 2; ++u, tile += L::kBytes) {
#pragma unroll
        for (int v = 0; v < 2 * G / 4; ++v) {
          vc[u][v] = ldnc16(tile + L::kV + v * 512 + lane * 16);
          vs[u][v] = ldnc16(tile + L::kVs + v * 64 + tig * 16);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int g = 0; g < G; ++g)
            vz[u][g][n] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::kVz + g * 32 + n * 16 + tig * 4));
      }
    };
    bool ok = true;
    // K of tile j: row of position 16 u + 8 n + gid of the block (column order), 16 bytes per word
    auto put_k = [&](int j, int page) {
      const int b = kK2 ? 2 * j + (w >> 1) : j, buf = b % kBufs, before = b / kBufs - 1;  // its use before
      if (before >= 0) ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.k_empty[buf], before & 1, a.c.status));
      if (!ok) return;
      uint8_t* sk = skv + buf * 2 * M::kKV;
      if (lane == 0) {
        const bool bad = p0 + j * kPTile + 32 * w < see && (unsigned)page >= (unsigned)a.c.n_pages;
        sh.bad[j & 3][w] = bad;
        if (bad) atomicOr(a.c.status, KV4_BAD_PAGE);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int r = 32 * (kK2 ? w & 1 : w) + 8 * (gid >> 1) + 4 * u + 2 * n + (gid & 1);
          const uint32_t* c = reinterpret_cast<const uint32_t*>(kc[u]);
          const uint32_t* s = reinterpret_cast<const uint32_t*>(&ks[u][n]);
          const uint32_t* z = reinterpret_cast<const uint32_t*>(&kz[u][n]);
          [[maybe_unused]] Params pp;  // of groups g, g + 1
#pragma unroll
          for (int g = 0; g < G; ++g) {
            uint32_t v[4];
            const int word = 4 * g + tig;
            if constexpr (kK2) {
              if (g % 2 == 0) pp = split_params(__byte_perm(s[g], s[g + 1], gid & 1 ? 0x7632 : 0x5410), z[g / 2]);
              const Params p{both(pp.sh, g & 1), both(pp.za, g & 1), both(pp.sl, g & 1), both(pp.zb, g & 1)};
              uint32_t lo[4];
              uint8_t* to = sk + (word >> 3) * 8192 + chunk_at(r, word & 7);
              dequant8(c[n * G + g], p, v, lo);
              *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(to + kPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            } else {
              dequant8(c[n * G + g], both(s[g], gid & 1), both(z[g / 2], g & 1), v);
              *reinterpret_cast<uint4*>(sk + (word >> 3) * 16384 + chunk_at(r, word & 7)) =
                  make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        }
      fence_proxy_async_smem();
      mbar_arrive(&sh.k_full[buf]);
    };
    // V of tile j transposed: row of value 32 g + 4 gid + i, 8 positions (16 bytes) per lane
    auto put_v = [&](int j, int page) {
      const int b = kV2 ? 2 * j + (w >> 1) : j, buf = b % kBufs, before = b / kBufs - 1;
      const int first = p0 + j * kPTile + 32 * w;
      const int left = (unsigned)page < (unsigned)a.c.n_pages ? see - first : 0;  // positions of the block that exist
      uint32_t odd = 0;  // a NaN among the parameters
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int p = 16 * u + 8 * n + 2 * tig;
          uint32_t* s = reinterpret_cast<uint32_t*>(vs[u]);
          if (left < 32) {  // the end of the sequence (or a missing page): zeros
            const uint32_t keep = (p < left ? 0xFFFFu : 0u) | (p + 1 < left ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              vz[u][g][n] &= keep;
              s[n * G + g] &= keep;
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) odd |= (uint32_t)(nan_half(vz[u][g][n]) || nan_half(vz[u][g][n] >> 16));
        }
      if (__any_sync(0xFFFFFFFFu, odd != 0)) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t z = vz[u][g][n];
              const int p = first + 16 * u + 8 * n + 2 * tig;
              if (nan_half(z) || nan_half(z >> 16)) atomicMin(&sh.nan_first[g], nan_half(z) ? p : p + 1);
              const uint32_t keep = (nan_half(z) ? 0u : 0xFFFFu) | (nan_half(z >> 16) ? 0u : 0xFFFF0000u);
              vz[u][g][n] &= keep;
              reinterpret_cast<uint32_t*>(vs[u])[n * G + g] &= keep;
            }
      }
      if (before >= 0) ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.v_empty[buf], before & 1, a.c.status));
      if (!ok) return;
      uint8_t* sv = skv + buf * 2 * M::kKV + M::kKV;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t v[4][4];  // [2 u + hf][value]
        [[maybe_unused]] uint32_t lo[4][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t c = reinterpret_cast<const uint32_t*>(vc[u])[2 * g + n];
            const uint32_t s = reinterpret_cast<const uint32_t*>(vs[u])[n * G + g], z = vz[u][g][n];
            if constexpr (kV2) dequant8(c, split_params(s, z), v[2 * u + n], lo[2 * u + n]);
            else dequant8(c, s, z, v[2 * u + n]);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint8_t* to = sv + (kV2 ? 0 : (w >> 1) * kPart) + chunk_at(32 * g + 4 * gid + i, 4 * (w & 1) + tig);
          *reinterpret_cast<uint4*>(to) = make_uint4(v[0][i], v[1][i], v[2][i], v[3][i]);
          if constexpr (kV2) *reinterpret_cast<uint4*>(to + kPart) = make_uint4(lo[0][i], lo[1][i], lo[2][i], lo[3][i]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.v_full[buf]);
    };
    // K runs a tile ahead of V (its buffer is free as soon as the scores are done), but not
    // where its buffers are two halves
    constexpr int kAhead = kK2 && kBufs == 2 ? 0 : 1;
    int page_k = look(0), page_v = page_k, page_next = look(1);
    load_k(page_k);
    load_v(page_v);
    for (int j = -kAhead; j < n_max && ok; ++j) {
      if (j + kAhead < n_max) {
        put_k(j + kAhead, page_k);
        page_k = page_next;
        load_k(page_k);
        page_next = look(j + kAhead + 2);
      }
      if (j >= 0 && ok) {
        put_v(j, page_v);
        page_v = look(j + 1);
        load_v(page_v);
      }
    }
  } else if (n_max > 0) {
    // ---------------- matrix instructions (the warp converged, one lane issues) ----------------
    const int t = warp - 12, n = n_half[t];
    const uint32_t one = elect_one();
    const uint64_t dq = sw128_desc(smem_u32(sq) + t * (D / 64) * 16384), dk = sw128_desc(smem_u32(skv)),
                   dv = sw128_desc(smem_u32(skv) + M::kKV);
    constexpr uint32_t kBuf = 2 * M::kKV / 16;  // a buffer further, in the descriptor's 16-byte units
    const uint32_t tms = tmem + t * 128, tmo = tmem + kO + t * D;
    auto score = [&](int i, int c, uint64_t k, bool first) {  // 16 of the queries' values
      if constexpr (kQT) mma_ts(one, tms + (i & 1) * 64, tmem + kQ + t * 32 + 8 * c, k, kIdQK, first ? 0u : 1u);
      else mma_ss(one, tms + (i & 1) * 64, dq + (c / 4) * 1024 + (c % 4) * 2, k, kIdQK, first ? 0u : 1u);
    };
    // scores of half i, and the product of its weights
    auto qk = [&](int i) {
      if constexpr (kK2) {
        const uint64_t k = dk + (uint32_t)(i % kBufs) * kBuf;
#pragma unroll
        for (int c = 0; c < 2 * (D / 16); ++c) {  // the parts in turn
          const int q = c / 2;
          score(i, q, k + (c & 1) * (kPart / 16) + (q / 4) * 512 + (q % 4) * 2, c == 0);
        }
        mma_commit(one, &sh.s_full[t][i & 1]);
        mma_commit(one, &sh.k_empty[i % kBufs]);
        return;
      }
      const uint64_t k = dk + (uint32_t)(i >> 1 & 1) * kBuf + (uint32_t)(i & 1) * 512;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        score(i, c, k + (c / 4) * 1024 + (c % 4) * 2, c == 0);
      mma_commit(one, &sh.s_full[t][i & 1]);
      if (i & 1 || i + 1 == n) mma_commit(one, &sh.k_empty[i >> 1 & 1]);  // the tile's last scores
    };
    auto wv = [&](int i) {
      if constexpr (kV2) {
        const uint64_t v = dv + (uint32_t)(i % kBufs) * kBuf;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          mma_ts(one, tmo, tms + (i & 1) * 64 + 8 * (c / 2), v + (c & 1) * (kPart / 16) + (c / 2) * 2, kIdWV, i || c ? 1u : 0u);
        mma_commit(one, &sh.wv_done[t]);
        mma_commit(one, &sh.v_empty[i % kBufs]);
        if (i + 1 == n) mma_commit(one, &sh.o_full[t]);
        return;
      }
      const uint64_t v = dv + (uint32_t)(i >> 1 & 1) * kBuf + (uint32_t)(i & 1) * (D * 8);
#pragma unroll
      for (int c = 0; c < 4; ++c) mma_ts(one, tmo, tms + (i & 1) * 64 + 8 * c, v + c * 2, kIdWV, i || c ? 1u : 0u);
      mma_commit(one, &sh.wv_done[t]);
      if (i & 1 || i + 1 == n) mma_commit(one, &sh.v_empty[i >> 1 & 1]);
      if (i + 1 == n) mma_commit(one, &sh.o_full[t]);
    };
    auto ready = [&](uint64_t* bar, int j, int bufs) {
      const bool r = __all_sync(0xFFFFFFFFu, kv4_wait(bar + j % bufs, (j / bufs) & 1, a.c.status));
      tc_fence_after();
      return r;
    };
    bool ok = __all_sync(0xFFFFFFFFu, kv4_wait(&sh.q_full, 0, a.c.status));
    tc_fence_after();
    if (n > 0) {
      ok = ok && ready(sh.k_full, 0, kBufs);
      if (ok) {
        qk(0);
        if (kK2 && n > 1) ok = ready(sh.k_full, 1, kBufs);
        if (n > 1 && ok) qk(1);
      }
      for (int i = 0; i < n && ok; ++i) {
        if (kV2) ok = ready(sh.v_full, i, kBufs);
        else if (!(i & 1)) ok = ready(sh.v_full, i >> 1, kBufs);
        if (ok) ok = ready(sh.w_full[t], i, 2);
        if (!ok) break;
        wv(i);
        if (i + 2 < n) {
          if (kK2) ok = ready(sh.k_full, i + 2, kBufs);
          else if (!(i & 1)) ok = ready(sh.k_full, (i + 2) >> 1, kBufs);
          if (ok) qk(i + 2);
        }
      }
    }
    // tiles (or halves) that only the other query tile sees, if any: this one lets go of them as they come
    for (int i = n; i < 2 * n_max && ok; ++i) {
      const int k = kK2 ? i : i >> 1, v = kV2 ? i : i >> 1;
      if (kK2 || !(i & 1)) {
        ok = ready(sh.k_full, k, kBufs);
        if (ok && lane == 0) mbar_arrive(&sh.k_empty[k % kBufs]);
      }
      if (ok && (kV2 || !(i & 1))) {
        ok = ready(sh.v_full, v, kBufs);
        if (ok && lane == 0) mbar_arrive(&sh.v_empty[v % kBufs]);
      }
      __syncwarp();
    }
    if (!ok) {  // let what was issued finish before the memory goes
      mma_commit(one, &sh.drained[t]);
      kv4_wait(&sh.drained[t], 0, a.c.status);
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
static mk_status launch(const Kv4AttnSplit& a, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  constexpr int kSmem = PSmem<D, T>::kBytes;
  if (!kv4_allow_smem(reinterpret_cast<const void*>(attn_prompt<D, T>), kSmem, &ready)) return MK_ERR_CUDA;
  const long long ctas = (a.n_blocks ? a.n_blocks : (long long)a.n_rt * a.b.n_seqs) * a.c.n_kv_heads * a.n_split;
  if (ctas > 0x7FFFFFFF) return MK_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  return kv4_status(cudaLaunchKernelEx(&cfg, attn_prompt<D, T>, a));
}

mk_status kv4_prompt(const Kv4AttnSplit& a, int32_t dtype, cudaStream_t s) {
  if (a.c.head_dim == 64) return dtype == 0 ? launch<64, __nv_bfloat16>(a, s) : launch<64, __half>(a, s);
  return dtype == 0 ? launch<128, __nv_bfloat16>(a, s) : launch<128, __half>(a, s);
}

}  // namespace mk
