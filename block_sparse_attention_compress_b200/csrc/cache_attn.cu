// Attention of the newest tokens over a paged cache in bf16 or 4 bits.  Bound: the cache's bytes.
//
// Per KV head the query rows (n_new tokens x G heads) stand as the MMA's N (tiles of 8) and 16
// cached tokens as its M, so that a group of 8 heads wastes nothing:
//   S[key, row]  = K Q^T      A = K as it lies in memory: a lane takes its quad's share of a key
//                             row, and the queries' dims are permuted to match;
//   O^T[d, row] += V^T P^T    A = V^T: a register pairs two tokens of one dim (byte permutes), and
//                             the tile's dims are permuted to match.  S's C fragment becomes
//                             P^T's B fragment by movmatrix.
// The operands come from registers (warp-level MMA): in 4 bits a tcgen05 form would have to write
// every widened value to shared memory and read it back, 640 bytes a token against the 200 that
// are stored, about 210 cycles of an SM's shared memory for 16 tokens of (192, 128); HBM takes 120.  In bf16 that reason holds
// up to 16 rows a head, where HBM bounds the call; more rows read each tile again (64 rows: 275 us where HBM takes 84).
//
// Keys in 4 bits: w & 0x000f000f and w & 0x00f000f0 are pairs of f16 subnormals c 2^-24 and
// c 2^-20, which the tensor cores multiply exactly: no conversion.  The queries of the latter are
// divided by 16, and every query row is scaled by a power of two so that f16 holds it.  (The e4m3
// MMA would take the nibbles as they are too, but on sm_100 it is carried out as conversions and
// 16-bit MMAs: 781 us instead of 571 for 32 sequences of 64K tokens in the kernel's first form.)  A group's (s, z) come in behind
// the product: S = sum_g s_g (sum c q) + (z_g - 8 s_g) sum_g q, the second sum as more MMAs with
// the stored pairs as A and the groups' query sums (three bf16 terms: 24 bits) as B.
//
// Values in 4 bits: nibbles become s 2^k (c - 8) in f16, pairs of two tokens of a dim, exactly (at most 11 bits):
// three instructions a pair (mask on the exponent of 1024, subtract, multiply), the same for every row.  k by group
// from the largest s met so far: full digits down to scales 2^-28 of the largest, nothing below 2^-36 of it.  Weights
// are two f16 terms (2^-22, and down to 2^-32 of the largest), P z is summed in fp32.  P s 2^k as one f16, against codes as
// subnormals, was 10% (one row a head) to 15% (16 rows) faster, but made outputs differ from 32-bit arithmetic by 1.3e-3 of
// their size instead of 1e-4.
//
// The tensor cores cut off sums instead of rounding them, always towards zero (as the MMA's C, an accumulator lost 2^-18 of
// the mean value over 3,200 tiles), so a step's products are summed by themselves and join the accumulators rounded: 5%
// of the time at 16 rows in 4 bits, nothing with fewer.
//
// Every warp copies its own tiles of 16 tokens into a ring in shared memory (cp.async, no block-wide
// waits).  The tiles of all sequences and heads are laid end to end and cut into equal runs, one
// per block, so unequal lengths and head counts fill the GPU alike; a sequence cut into several runs
// leaves a part in each block's slots and a second small kernel joins the parts by their maxima and
// sums, in a fixed order.
//
// Measured (B200): 32 x 16K tokens in bf16, 64 query heads on 4, (192, 128): 225-232 us, 5.8-6.0 TB/s.  32 x 64K tokens
// in 4 bits, same heads: 579 us, 2.9 TB/s; 32 heads of one query over 128K tokens in 4 bits, (128, 128): 171 us, 3.9
// TB/s.  In 4 bits the issue slots bound it, not HBM: logic at half rate, MMAs and fp32 products compete for the same
// slots (4 MMAs, 16 logic and 16 fma instructions take 58 cycles, not 32).
#include <algorithm>

#include "cache.cuh"

namespace nsa {
namespace {

constexpr int kTile = 16;         // tokens of an MMA's M
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D = A B
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  mma16816(d, a, b0, b1);
}
// transpose of an 8 x 8 tile of 16-bit values held as an MMA fragment
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// (x, y) += (a, b) * f and (x, y) * f for a lane's J columns: two as one packed instruction
template <int J>
__device__ __forceinline__ void fma_columns(float& x, float& y, float a, float b, float f) {
  if constexpr (J == 1) {
    x = fmaf(a, f, x);
  } else {
    const float2 r = f2_unpack(f2_fma(f2_pack(a, b), f2_pack(f, f), f2_pack(x, y)));
    x = r.x;
    y = r.y;
  }
}
// o += y, rounded
__device__ __forceinline__ void add_to(float (&o)[4], const float (&y)[4]) {
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float2 r = f2_unpack(f2_add(f2_pack(o[e], o[e + 1]), f2_pack(y[e], y[e + 1])));
    o[e] = r.x;
    o[e + 1] = r.y;
  }
}
// x cut to the 11 bits that f16 holds of it
__device__ __forceinline__ float leading11(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }
// s (c - 8) of the codes c in bits 0..3 (4..7) of each half of w, s f16: 1024 + c (1024 + 16 c) is the code below f16's
// exponent of 2^10; the rest is exact (4 bits times 8 are at most 11: 8 s is s shifted)
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t low_values(uint32_t w, uint32_t s) {
  const __half2 c = __hsub2(as_half2((w & 0x000f000fu) | 0x64006400u), as_half2(0x64086408u));
  const __half2 v = __hmul2(c, as_half2(s));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t high_values(uint32_t w, uint32_t s) {
  const __half2 c = __hfma2(as_half2((w & 0x00f000f0u) | 0x64006400u), as_half2(0x2c002c00u), as_half2(0xd480d480u));   // / 16 - 72
  const __half2 v = __hmul2(c, as_half2(s));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float inverse_pow2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }   // of a normal one
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126 <= e <= 127

// copies of 8 or 16 bytes into shared memory; `on` false: zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
  const int n = on ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}
// N 32-bit words from shared memory, as wide as 8-byte alignment (16 for multiples of 4) allows
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const char* p) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + 16 * i);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 u = *reinterpret_cast<const uint2*>(p + 8 * i);
      w[2 * i] = u.x; w[2 * i + 1] = u.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
}

// cap tanh(x / cap): 1 - 2 / (e^2t + 1), and for small t, where that loses the digits of t, the
// series t - t^3/3 + 2 t^5/15 - 17 t^7/315 + 62 t^9/2835 (the next term is below 1e-8 t at t = 1/4).
__device__ __forceinline__ float capped(float x, float cap, float inv_cap) {
  const float t = x * inv_cap, t2 = t * t;
  const float big = 1.f - __fdividef(2.f, ex2(t * (2.f * kLog2e)) + 1.f);
  float p = fmaf(t2, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(t2, p, 2.f / 15.f);
  p = fmaf(t2, p, -1.f / 3.f);
  return cap * (fabsf(t) < 0.25f ? fmaf(t * t2, p, t) : big);
}

// A column's running maximum before any token: below every finite score, and finite, so that
// 2^(-inf - kNone) is 0 (a masked token) and 2^(NaN - kNone) a NaN (an attended one).
constexpr float kNone = -3.0e38f;

// How a call is cut.  whole: one block per (sequence, head, tile of rows).  Else `blocks` blocks share
// the tiles of all of them in equal runs of at least min_tiles.
struct Plan {
  int row_tiles, tile_rows;   // row tiles per head and rows of one
  int blocks, min_tiles, row_groups;
  int per_g;                  // r / G = r per_g >> 16 for the rows r < 256 of a call
  int first[4], last[4];      // of each row tile: the first and the last new token it has rows of
  bool whole, small;          // small: the tiles of all items count in 32 bits
};
__device__ __forceinline__ int row_token(const Plan& p, int r) { return r * p.per_g >> 16; }

// A block that holds the first part of an item cut over blocks says here which blocks hold the rest.
struct Cut {
  int b, head_tile, last, rows;   // last < 0: nothing to join
};

// The keys a tile of rows attends to, of one sequence: [lo, hi), in `tiles` tiles from base on.
struct Span {
  int p0, lo, hi, base, tiles;
};
template <int STEP>
__device__ __forceinline__ Span span_of(const CacheAttnArgs& a, const Plan& p, int b, int rt) {
  Span s;
  s.p0 = min(max(__ldg(a.seqlens + b), 0), a.max_seqlen) - a.n_new;
  s.hi = max(0, s.p0 + p.last[rt] + 1);
  s.lo = a.window > 0 ? max(0, s.p0 + p.first[rt] - a.window + 1) : 0;
  s.base = s.lo & ~(kTile - 1);
  s.tiles = max(1, (s.hi - s.base + STEP - 1) / STEP);
  return s;
}
// a / b for counts: 64-bit division is a hundred instructions
__device__ __forceinline__ int runs_before(long long a, long long b) {
  return ((a | b) >> 31) == 0 ? (int)((uint32_t)a / (uint32_t)b) : (int)(a / b);
}

__device__ __forceinline__ void check_length(const CacheArgs& c, const CacheAttnArgs& a, int b) {
  const int len = __ldg(a.seqlens + b);
  if (len < 0 || len > a.max_seqlen) cache::report(c.status);
}

// One tile of 16 tokens as a stage of the ring holds it.  4 bits: key codes, value codes, (s, z) pairs of
// keys and of values; rows of values lie with their 16-byte units turned by the row, so that the
// lanes' loads spread over the banks.  bf16: key rows, value rows, units turned likewise.
template <bool INT4, int DK, int DV>
struct Stage {
  static constexpr int kRowK = INT4 ? DK / 2 : DK * 2, kRowV = INT4 ? DV / 2 : DV * 2;
  static constexpr int kRowKs = INT4 ? DK / 8 : 0, kRowVs = INT4 ? DV / 8 : 0;
  static constexpr int kV = kTile * kRowK, kKs = kV + kTile * kRowV, kVs = kKs + kTile * kRowKs;
  static constexpr int kBytes = kVs + kTile * kRowVs;
  __device__ static int key_unit(int row, int u) { return u ^ ((row & 1) << 2); }   // bf16
  __device__ static int value_unit(int row, int u) {
    if constexpr (INT4) return DV == 128 ? u ^ ((row >> 1) & 3) : u;
    return u ^ (((row >> 1) & 3) << 1);
  }
};

// Tile copies are unrolled where all 16 rows exist (FULL), and short loops where some do not: code that
// runs once a tile at most has to be fetched too, and a single token's call is mostly that.
constexpr int copy_steps(bool full, int units) { return full ? (units + 31) / 32 : 1; }

// 16 rows of ROW bytes that lie one behind the other, from the lane's place `src` on, to `at`(x) for unit x
template <int ROW, bool FULL, class At>
__device__ __forceinline__ void copy_run(const char* src, int lane, int lo, int hi, At at) {
  constexpr int kBytes = ROW % 16 == 0 ? 16 : 8, kAll = kTile * ROW / kBytes;
#pragma unroll copy_steps(FULL, kAll)
  for (int i = 0; i < (kAll + 31) / 32; ++i) {
    const int x = lane + 32 * i, row = x * kBytes / ROW;
    if (kAll % 32 == 0 || x < kAll) copy_async<kBytes>(at(x), src + 32 * i * kBytes, FULL || (row >= lo && row < hi));
  }
}

// rows [0, 16) of ROW bytes, `stride` apart in memory
template <int ROW, bool FULL, class Unit>
__device__ __forceinline__ void copy_rows(uint32_t dst, const char* src, size_t stride, int lane, int lo, int hi, Unit unit) {
  constexpr int kUnits = ROW / 16, kAll = kTile * kUnits;
#pragma unroll copy_steps(FULL, kAll)
  for (int i = 0; i < kAll / 32; ++i) {
    const int x = lane + 32 * i, row = x / kUnits, u = x % kUnits;
    copy_async<16>(dst + row * ROW + unit(row, u) * 16, src + row * stride + u * 16, FULL || (row >= lo && row < hi));
  }
}

// Where the tiles of one head lie in memory, walked from tile to tile (4 bits: a lane's own places, so that a
// copy is an instruction of its own and little else).
template <bool INT4, int DK, int DV>
struct Walk {
  using T = Stage<INT4, DK, DV>;
  const char *k, *v, *ks, *vs;
  __device__ __forceinline__ void go(const CacheArgs& c, int page, int off, int h, int lane) {
    if constexpr (INT4) {
      const size_t row = ((size_t)page * c.h_kv + h) * c.page_size + off;
      k = static_cast<const char*>(c.k) + row * T::kRowK + lane * 16;
      v = static_cast<const char*>(c.v) + row * T::kRowV + lane * 16;
      ks = static_cast<const char*>(c.k_scale) + row * T::kRowKs + lane * (T::kRowKs % 16 ? 8 : 16);
      vs = static_cast<const char*>(c.v_scale) + row * T::kRowVs + lane * (T::kRowVs % 16 ? 8 : 16);
    } else {
      const size_t row = ((size_t)page * c.page_size + off) * c.h_kv + h;
      k = static_cast<const char*>(c.k) + row * T::kRowK;
      v = static_cast<const char*>(c.v) + row * T::kRowV;
    }
  }
  __device__ __forceinline__ void next(const CacheArgs& c) {   // the next 16 tokens of the page
    const int n = INT4 ? kTile : kTile * c.h_kv;
    k += (size_t)n * T::kRowK;
    v += (size_t)n * T::kRowV;
    if constexpr (INT4) {
      ks += n * T::kRowKs;
      vs += n * T::kRowVs;
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void copy(const CacheArgs& c, uint32_t dst, int lane, int lo, int hi) const {
    if constexpr (INT4) {
      copy_run<T::kRowK, FULL>(k, lane, lo, hi, [&](int x) { return dst + x * 16; });
      copy_run<T::kRowV, FULL>(v, lane, lo, hi, [&](int x) {
        constexpr int kUnits = T::kRowV / 16;
        return dst + T::kV + (x / kUnits * kUnits + T::value_unit(x / kUnits, x % kUnits)) * 16;
      });
      copy_run<T::kRowKs, FULL>(ks, lane, lo, hi, [&](int x) { return dst + T::kKs + x * (T::kRowKs % 16 ? 8 : 16); });
      copy_run<T::kRowVs, FULL>(vs, lane, lo, hi, [&](int x) { return dst + T::kVs + x * (T::kRowVs % 16 ? 8 : 16); });
    } else {
      copy_rows<T::kRowK, FULL>(dst, k, (size_t)c.h_kv * T::kRowK, lane, lo, hi, [](int r, int u) { return T::key_unit(r, u); });
      copy_rows<T::kRowV, FULL>(dst + T::kV, v, (size_t)c.h_kv * T::kRowV, lane, lo, hi, [](int r, int u) { return T::value_unit(r, u); });
    }
  }
};

// Zeros for the tokens of a step with a value that is not finite (4 bits: a scale or an offset): their bits
template <class T, bool INT4, int DV, int U>
__device__ __forceinline__ uint32_t drop_odd_values(char* step, int lane) {
  const auto odd2 = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
  // tokens of a step, lanes of a token, and bytes of a lane
  constexpr int kTokens = U * kTile, kLanes = 32 / kTokens, kRow = INT4 ? T::kRowVs : T::kRowV, kBytes = kRow / kLanes;
  const int tok = lane / kLanes;
  char* row = step + tok / kTile * T::kBytes + (INT4 ? T::kVs : T::kV) + tok % kTile * kRow + lane % kLanes * kBytes;
  bool odd = false;
#pragma unroll 1
  for (int i = 0; i < kBytes; i += 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + i);
    odd |= odd2(w.x) || odd2(w.y);
  }
  uint32_t lanes = __ballot_sync(0xffffffffu, odd), tokens = lanes;
  if (lanes == 0) return 0;
  if constexpr (kLanes == 2) {
    tokens = 0;
    for (int i = 0; i < kTokens; ++i) tokens |= (lanes >> (2 * i) & 3u) ? 1u << i : 0u;
  }
  if (tokens >> tok & 1) {
#pragma unroll 1
    for (int i = 0; i < kBytes; i += 8) *reinterpret_cast<uint2*>(row + i) = make_uint2(0, 0);
  }
  __syncwarp();
  return tokens;
}

// Shared memory of a block: a ring (and later the joined rows) per warp, then in 4 bits the queries of
// each row group: per tile of 8 rows the B fragments [DK / 32][32 lanes] x 16 bytes, the group sums'
// [32 lanes] x (16 + 8) bytes and the rows' factors.
template <bool INT4, int DV, int U>
constexpr int scale_smem() {
  return INT4 ? U * kTile * (DV / 32) * 2 : 0;
}
template <bool INT4, int DK, int DV, int NT, int U, int S>
constexpr int warp_smem() {
  return std::max(S * U * Stage<INT4, DK, DV>::kBytes + scale_smem<INT4, DV, U>(), NT * 8 * (DV + 4 + 2) * 4);
}
template <bool INT4, int DK, int NT>
constexpr int query_smem() {
  return INT4 ? NT * ((DK / 32 + 1) * 512 + 256 + 8 * 4) : 0;
}

template <bool INT4, int DK, int DV, int NT, int J, int W, int MINB, int U, int S, bool EXT>
__global__ void __launch_bounds__(W * 32, MINB)
cache_attn_kernel(const CacheArgs c, const CacheAttnArgs a, const Plan pl, Cut* __restrict__ cuts, float2* __restrict__ part_ml,
                  float* __restrict__ part_o) {
  using T = Stage<INT4, DK, DV>;
  constexpr int NG = DK / 32, NH = DV / 32, MT = DV / 16, KS = DK / 16;
  // 4 bits: the reference lies 2^7 below the maximum, so that f16 holds weights down to 2^-32 of it (and the largest, 2^15)
  constexpr float kAbove = INT4 ? 7.f : 0.f;
  // a warp's rows: J of a lane's two columns hold one
  constexpr int kCols = NT * 4 * J, kRow = DV + 4;
  const auto row_of = [](int nt, int column) { return J == 2 ? nt * 8 + column : column >> 1; };
  constexpr int kWarpBytes = warp_smem<INT4, DK, DV, NT, U, S>(), kStep = kTile * U, kQ = query_smem<INT4, DK, NT>();
  extern __shared__ __align__(128) char smem[];
  __shared__ long long s_scan[W];
  __shared__ long long s_off;
  __shared__ int s_b, s_h;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, q4 = lane & 3;
  const int rg = warp % pl.row_groups, streams = W / pl.row_groups, ts = warp / pl.row_groups;
  const int R = a.n_new * a.G;
  char* ring = smem + warp * kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);
  char* sq = smem + W * kWarpBytes + rg * kQ;                     // this row group's queries
  char* sq_last = sq + NT * (NG + 1) * 512;
  float* sq_sc = reinterpret_cast<float*>(sq_last + NT * 256);

  // ---- which tiles are this block's: `left` of them from tile t of item (b, h, rt) on
  asm volatile("griddepcontrol.launch_dependents;");   // the join may be set up; it waits before it reads
  // a step of all streams is 1.3 us (4 bits), a part's start and end about 5
  const int extra = 4 * streams;
  int b, h, rt, t = 0;
  long long left, pos0 = 0, per = 0;   // pos0: index of the first among all tiles
  if (pl.whole) {
    int id = blockIdx.x;
    rt = id % pl.row_tiles; id /= pl.row_tiles;
    h = id % c.h_kv;
    b = id / c.h_kv;
    left = (long long)span_of<kStep>(a, pl, b, rt).tiles + extra;
    if (h == 0 && rt == 0 && threadIdx.x == 0) check_length(c, a, b);
  } else {
    const auto cut_work = [&](auto zero) {   // false: nothing is left for this block
      using N = decltype(zero);              // 32 bits wherever the count of tiles allows it
      const auto quotient = [](N x, N y) { return sizeof(N) == 4 ? (N)((uint32_t)x / (uint32_t)y) : (N)(x / y); };
      const int strip = (c.batch + W * 32 - 1) / (W * 32);
      const int b0 = min(c.batch, (int)threadIdx.x * strip), b1 = min(c.batch, b0 + strip);
      // a thread with one sequence of one row tile looks its length up once
      const bool single = strip == 1 && pl.row_tiles == 1;
      const int own = single && b0 < b1 ? span_of<kStep>(a, pl, b0, 0).tiles : 0;
      // An item's share of the work: its tiles and, before them, what its start costs in tiles.  And that of a head, in all
      // row tiles.
      const auto units = [&](int bb, int x) -> N { return span_of<kStep>(a, pl, bb, x).tiles + extra; };
      const auto head_units = [&](int bb) {
        if (single) return (N)(own + extra);
        N w = 0;
        for (int x = 0; x < pl.row_tiles; ++x) w += units(bb, x);
        return w;
      };
      // the strips' sums: of those before this thread's, and of all
      const auto scan = [&](N mine, N& total) {
        N upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const N y = __shfl_up_sync(0xffffffffu, upto, d);
          if (lane >= d) upto += y;
        }
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const N y = (N)s_scan[w];
          if (w < warp) upto += y;
          total += y;
        }
        return (N)(upto - mine);
      };
      N mine = 0, total;
      for (int x = b0; x < b1; ++x) {
        mine += head_units(x) * c.h_kv;
        if (blockIdx.x == 0) check_length(c, a, x);
      }
      // (Runs that end with their items, for many short ones, spare a block the end of one item and the start of the next, but
      // their ends cost more: 64 items of 1100 tokens in 4 bits, 8 rows, 13.0 us so and 14.4 that way, 64 of 2400 with 16
      // rows 21.5 and 25.6; of 200 sizes four were quicker that way, by 2 us at most.)
      const N before = scan(mine, total), run = max((N)pl.min_tiles, quotient(total + gridDim.x - 1, gridDim.x));
      const N pos = run * (N)blockIdx.x;
      if (pos >= total) return false;
      if (before <= pos && pos < before + mine) {
        N off = pos - before, head;
        int x = b0;
        for (; off >= (head = head_units(x)) * c.h_kv; ++x) off -= head * c.h_kv;
        const N skip = quotient(off, head);
        s_b = x;
        s_h = (int)skip;
        s_off = off - skip * head;
      }
      __syncthreads();
      b = s_b;
      h = s_h;
      N at = (N)s_off;
      rt = 0;
      if (pl.row_tiles > 1)
        for (N n; at >= (n = units(b, rt)); ++rt) at -= n;
      t = (int)at;
      left = min(run, (N)(total - pos));
      pos0 = pos;
      per = run;
      return true;
    };
    if (!(pl.small ? cut_work(0) : cut_work(0ll))) {
      if (threadIdx.x == 0) cuts[blockIdx.x] = Cut{0, 0, -1, 0};
      return;
    }
  }

  Cut cut{0, 0, -1, 0};
  while (left > 0) {
    const Span sp = span_of<kStep>(a, pl, b, rt);
    // the block's part of the item's share, [t, t + part), and its tiles in that
    const int part = (int)min(left, (long long)(sp.tiles + extra - t)), first = max(0, t - extra);
    const int take = max(0, t + part - extra) - first;
    const int r0 = rt * pl.tile_rows + rg * kCols;   // this warp's first row (maybe behind the last)
    const auto next_item = [&] {
      left -= part;
      pos0 += part;
      t = 0;
      if (++rt == pl.row_tiles) {
        rt = 0;
        if (++h == c.h_kv) {
          h = 0;
          ++b;
        }
      }
    };
    const int tile_rows = min(R - rt * pl.tile_rows, pl.tile_rows);
    const auto out_row = [&](int r) {   // of the item's row r, among all
      const int i = row_token(pl, r);
      return ((size_t)b * a.n_new + i) * a.h_q + h * a.G + (r - i * a.G);
    };
    if (take == 0) break;   // the run ends before the item's first tile
    if (sp.hi == 0) {       // an empty sequence
      for (int x = threadIdx.x; x < tile_rows * (DV / 4); x += W * 32) {
        const size_t row = out_row(rt * pl.tile_rows + x / (DV / 4));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + (x % (DV / 4)) * 4) = make_uint2(0, 0);
        if (a.lse && x % (DV / 4) == 0) a.lse[row] = -INFINITY;
      }
      next_item();
      continue;
    }
    if (first == 0 && take < sp.tiles) {
      cut.b = b;
      cut.head_tile = h * pl.row_tiles + rt;
      cut.last = runs_before(pos0 - t + extra + sp.tiles - 1, per);
      cut.rows = tile_rows;
    }

    // ---- queries on their way: row n = lane / 4 of each tile of 8
    uint4 qraw[NT][NG];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = min(r0 + row_of(nt, g8), R - 1), i = row_token(pl, r), g = r - i * a.G;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + (((size_t)b * a.n_new + i) * a.h_q + h * a.G + g) * DK;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) qraw[nt][gr] = __ldg(reinterpret_cast<const uint4*>(qr + 32 * gr + 8 * q4));
    }

    // ---- this warp's run of tiles, [ta, tb) of the item
    const int each = (take + streams - 1) / streams;
    const int ta = first + min(take, ts * each), tb = first + min(take, (ts + 1) * each);
    // steps inside [all_lo, all_hi) are seen whole by every row of the block
    const int all_lo = a.window > 0 ? max(0, sp.p0 + pl.last[rt] - a.window + 1) : 0, all_hi = sp.p0 + pl.first[rt] + 1;

    // the next tile to copy: its place in its page, and the page after that one, fetched ahead
    int cp_u = sp.base + ta * kStep, cp_j = 0, cp_off = 0, ahead = 0;
    const int cp_end = sp.base + tb * kStep;
    bool here = false;      // the page is valid
    uint32_t missing = 0;   // bit stage * U + x: tile x of that stage has no valid page
    const int32_t* pages = c.page_table + (size_t)b * c.max_pages;
    Walk<INT4, DK, DV> walk;
    const auto open_page = [&](int page) {
      here = page >= 0 && page < c.n_pages;
      walk.go(c, here ? page : 0, cp_off, h, lane);
      if (!here && lane == 0) cache::report(c.status);
      // pages behind the last token are not looked up
      const long long next = (long long)(cp_j + 1) * c.page_size;
      ahead = next < min(sp.hi, cp_end) ? __ldg(pages + cp_j + 1) : -1;
    };
    if (ta < tb) {
      cp_j = cp_u / c.page_size;
      cp_off = cp_u - cp_j * c.page_size;
      open_page(__ldg(pages + cp_j));
    } else {
      walk.go(c, 0, 0, h, lane);
    }
    const auto copy_next = [&](int stage) {
      if (cp_u < cp_end) {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const uint32_t dst = ring_u + (stage * U + x) * T::kBytes, bit = 1u << (stage * U + x);
          if (here && cp_u >= sp.lo && cp_u + kTile <= sp.hi) {
            walk.template copy<true>(c, dst, lane, 0, kTile);
            missing &= ~bit;
          } else {   // rows that do not exist are zeros, and masked
            const bool some = here && cp_u < sp.hi;
            walk.template copy<false>(c, dst, lane, some ? sp.lo - cp_u : 0, some ? sp.hi - cp_u : 0);
            missing = some ? missing & ~bit : missing | bit;
          }
          cp_u += kTile;
          cp_off += kTile;
          if (cp_off < c.page_size) {
            walk.next(c);
          } else if (cp_u < min(sp.hi, cp_end)) {
            cp_off = 0;
            ++cp_j;
            open_page(ahead);
          } else {
            here = false;
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) copy_next(s);

    // ---- queries as B fragments: row n = lane / 4 of each tile of 8.  4 bits: through shared memory
    uint32_t qf[INT4 ? 1 : NT][INT4 ? 1 : KS][2];
    float sc[NT][J];                    // what a column's raw score is multiplied by (natural units)
    int pos[NT][J];                     // the columns' positions
    float slope[EXT ? NT : 1][J];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (!INT4) {
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const uint4 u = qraw[nt][gr];
          qf[nt][2 * gr][0] = u.x;
          qf[nt][2 * gr][1] = u.y;
          qf[nt][2 * gr + 1][0] = u.z;
          qf[nt][2 * gr + 1][1] = u.w;
        }
      } else {
        const uint4(&u)[NG] = qraw[nt];
        uint32_t top = 0;   // the largest |q| as bf16 bits, in both halves
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const uint32_t w[4] = {u[gr].x, u[gr].y, u[gr].z, u[gr].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // a power of two that takes the row's largest query into [2^13, 2^14)
        const int e2 = min(max(13 - ((int)(top >> 7) - 127), -120), 120);
        const float up = pow2(e2);
        uint4* frag = reinterpret_cast<uint4*>(sq) + nt * (NG + 1) * 32 + lane;
        uint32_t* sums = reinterpret_cast<uint32_t*>(frag + NG * 32);
        uint32_t* last = reinterpret_cast<uint32_t*>(sq_last + (nt * 32 + lane) * 8);
        // (-8 sum, sum) of the groups' queries, each in three terms.  An MMA's K holds eight pairs: a term of
        // up to eight groups (words 2 i, 2 i + 1: term i of groups q4, q4 + 4), or two terms of up to four
        // (word i: term i); zeros where there is no group
        if (ts == 0) {
          if (NG <= 4) sums[3] = 0u;
          if (NG < 4 && q4 >= NG) sums[0] = sums[1] = sums[2] = 0u;
          if (NG > 4 && q4 + 4 >= NG) sums[1] = sums[3] = last[1] = 0u;
          // a query that is not finite, or so large that its factor leaves fp32, makes its row NaN
          const float factor = a.scale * pow2(-e2) * 0x1p24f;
          if (q4 == 0) sq_sc[nt * 8 + g8] = top >= 0x7f80u || !(factor <= 1e38f) ? NAN : factor;
        }
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          if (gr % streams != ts) continue;   // the warps of a row group share the groups out
          const uint32_t w[4] = {u[gr].x, u[gr].y, u[gr].z, u[gr].w};
          float x[8], sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[2 * e] = cache::bf16_lo(w[e]) * up;
            x[2 * e + 1] = cache::bf16_hi(w[e]) * up;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += x[e];
          frag[gr * 32] = make_uint4(pack_f16(x[0], x[4]), pack_f16(x[1] * 0.0625f, x[5] * 0.0625f), pack_f16(x[2], x[6]),
                                     pack_f16(x[3] * 0.0625f, x[7] * 0.0625f));
          sum = warp_sum4(sum) * 0x1p-24f;   // the products carry 2^-24: so do the sums beside them
          if (gr % 4 == q4) {
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              const float x = __bfloat162float(__float2bfloat16_rn(sum));
              sum -= x;
              (NG > 4 && term == 2 ? last : sums + (NG <= 4 ? term : 2 * term))[gr / 4] = pack_bf16(-8.f * x, x);
            }
          }
        }
      }
    }
    if constexpr (INT4) __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int rc = min(r0 + row_of(nt, 2 * q4 + j), R - 1), ic = row_token(pl, rc);
        sc[nt][j] = INT4 ? sq_sc[nt * 8 + 2 * q4 + j] : a.scale;
        pos[nt][j] = sp.p0 + ic;
        if constexpr (EXT) slope[nt][j] = a.slopes ? __ldg(a.slopes + h * a.G + rc - ic * a.G) * kLog2e : 0.f;
        else sc[nt][j] *= kLog2e;
      }

    float o[MT][NT][4];
    float m[NT][J], l[NT][J], zacc[INT4 ? NT : 1][NH][J];
    float top_s[INT4 ? NH : 1];   // 2^k of each group's weights
    uint32_t max_s[INT4 ? NH : 1];   // the largest s that k allows, as bf16 bits
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        m[nt][j] = kNone;
        l[nt][j] = 0.f;
        if constexpr (INT4) {
#pragma unroll
          for (int gr = 0; gr < NH; ++gr) zacc[nt][gr][j] = 0.f;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }
    if constexpr (INT4) {
#pragma unroll
      for (int gr = 0; gr < NH; ++gr) {
        top_s[gr] = 0x1p100f;
        max_s[gr] = 0;
      }
    }

    int stage = 0;
    for (int tile = ta; tile < tb; ++tile) {
      cp_async_wait<S - 2>();
      __syncwarp();
      const uint32_t gone = missing >> (stage * U) & ((1u << U) - 1);
      copy_next(stage == 0 ? S - 1 : stage - 1);
      char* st = ring + stage * U * T::kBytes;
      stage = stage == S - 1 ? 0 : stage + 1;
      const int u0 = sp.base + tile * kStep;

      // ---- S = K Q^T
      float s[U][NT][4];
      if constexpr (INT4) {
        uint4 q[NT];
        uint2 qlast[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          q[nt] = *reinterpret_cast<const uint4*>(sq + (nt * (NG + 1) + NG) * 512 + lane * 16);
          if constexpr (NG > 4) qlast[nt] = *reinterpret_cast<const uint2*>(sq_last + (nt * 32 + lane) * 8);
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
          uint32_t kz[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const char* row = st + x * T::kBytes + T::kKs + (g8 + 8 * j) * T::kRowKs + q4 * 4;
            kz[j] = NG >= 4 || q4 < NG ? *reinterpret_cast<const uint32_t*>(row) : 0u;
            if constexpr (NG > 4) kz[j + 2] = q4 + 4 < NG ? *reinterpret_cast<const uint32_t*>(row + 16) : 0u;
            else kz[j + 2] = kz[j];
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_first(s[x][nt], kz[0], kz[1], kz[2], kz[3], q[nt].x, q[nt].y);
            mma_bf16(s[x][nt], kz[0], kz[1], kz[2], kz[3], q[nt].z, q[nt].w);
            if constexpr (NG > 4) mma_bf16(s[x][nt], kz[0], kz[1], kz[2], kz[3], qlast[nt].x, qlast[nt].y);
          }
        }
        constexpr int GC = NG == 4 ? 4 : 2;   // groups whose words a lane loads at once
#pragma unroll
        for (int gc = 0; gc < NG; gc += GC) {
          uint32_t kw[U][2][GC], ks[U][2][GC];
#pragma unroll
          for (int x = 0; x < U; ++x)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              lds_words<GC>(kw[x][j], st + x * T::kBytes + (g8 + 8 * j) * T::kRowK + q4 * (NG * 4) + gc * 4);
              lds_words<GC>(ks[x][j], st + x * T::kBytes + T::kKs + (g8 + 8 * j) * T::kRowKs + gc * 4);
            }
#pragma unroll
          for (int gr = 0; gr < GC; ++gr) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) q[nt] = *reinterpret_cast<const uint4*>(sq + (nt * (NG + 1) + gc + gr) * 512 + lane * 16);
#pragma unroll
            for (int x = 0; x < U; ++x) {
              const uint32_t w0 = kw[x][0][gr], w1 = kw[x][1][gr], x0 = w0 >> 8, x1 = w1 >> 8;
              const float s0 = cache::bf16_lo(ks[x][0][gr]), s1 = cache::bf16_lo(ks[x][1][gr]);
              float acc[NT][4];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_first(acc[nt], w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, q[nt].x, q[nt].y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(acc[nt], x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, q[nt].z, q[nt].w);
                fma_columns<J>(s[x][nt][0], s[x][nt][1], acc[nt][0], acc[nt][1], s0);
                fma_columns<J>(s[x][nt][2], s[x][nt][3], acc[nt][2], acc[nt][3], s1);
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < U; ++x)
#pragma unroll
          for (int i = 0; i < DK / 32; ++i) {
            const char* row = st + x * T::kBytes + g8 * T::kRowK + T::key_unit(g8, 4 * i + q4) * 16;   // g8 and g8 + 8 turn alike
            const uint4 k0 = *reinterpret_cast<const uint4*>(row), k1 = *reinterpret_cast<const uint4*>(row + 8 * T::kRowK);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (i == 0) mma_bf16_first(s[x][nt], k0.x, k1.x, k0.y, k1.y, qf[nt][0][0], qf[nt][0][1]);
              else mma_bf16(s[x][nt], k0.x, k1.x, k0.y, k1.y, qf[nt][2 * i][0], qf[nt][2 * i][1]);
              mma_bf16(s[x][nt], k0.z, k1.z, k0.w, k1.w, qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
            }
          }
      }

      // ---- a value that is not finite, in a step that some rows see more of than others: no MMA may meet it, since 0 times it
      // is a NaN.  Zeros take its token's place, and the rows that attend the token are NaN from here on
      const bool edge = gone || u0 < all_lo || u0 + kStep > all_hi;
      if (edge && pl.first[rt] != pl.last[rt]) {
        if (const uint32_t odd = drop_odd_values<T, INT4, DV, U>(st, lane)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              bool met = false;
              for (uint32_t left_odd = odd; left_odd; left_odd &= left_odd - 1) {
                const int u = u0 + __ffs(left_odd) - 1, p = pos[nt][j];
                met |= u <= p && !(a.window > 0 && u <= p - a.window);
              }
              const float spoil = met ? NAN : 0.f;
              if constexpr (INT4) {
#pragma unroll
                for (int gr = 0; gr < NH; ++gr) zacc[nt][gr][j] += spoil;
              } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int e = j; e < 4; e += 2) o[mt][nt][e] += spoil;
              }
            }
        }
      }

      // ---- softmax: scores in log2 units, the reference moved only when a score passes it by 8
      uint32_t sv[INT4 ? NH : 1];   // 4 bits: the scales of the values of token `lane` of the step
      bool move = false;
      if constexpr (INT4) {
        const int tok = lane % kStep;
        lds_words<NH>(sv, st + (tok / kTile) * T::kBytes + T::kVs + (tok % kTile) * T::kRowVs);
#pragma unroll
        for (int gr = 0; gr < NH; ++gr) move |= (sv[gr] & 0xffffu) > max_s[gr];
      }
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; e += 3 - J) {
            float y = s[x][nt][e] * sc[nt][e & 1];
            if constexpr (EXT) {
              if (a.softcap > 0.f) y = capped(y, a.softcap, a.inv_softcap);
              y = fmaf(y, kLog2e, slope[nt][e & 1] * (float)(u0 + x * kTile + g8 + 8 * (e >> 1) - pos[nt][e & 1]));
            }
            s[x][nt][e] = y;
          }
      if (edge) {
#pragma unroll
        for (int x = 0; x < U; ++x)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; e += 3 - J) {
              const int u = u0 + x * kTile + g8 + 8 * (e >> 1), p = pos[nt][e & 1];
              if ((gone >> x & 1) || u > p || u < sp.lo || (a.window > 0 && u <= p - a.window)) s[x][nt][e] = -INFINITY;
            }
      }
      float top[NT][J];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          top[nt][j] = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
          for (int x = 1; x < U; ++x) top[nt][j] = fmaxf(top[nt][j], fmaxf(s[x][nt][j], s[x][nt][j + 2]));
          move |= top[nt][j] > m[nt][j] + (8.f + kAbove);
        }
      if (__any_sync(0xffffffffu, move)) {
        float grow[INT4 ? NH : 1];
        if constexpr (INT4) {
#pragma unroll
          for (int gr = 0; gr < NH; ++gr) {
            uint32_t x = sv[gr] & 0xffffu;
            x = __reduce_max_sync(0xffffffffu, x < 0x7f80u ? x : 0u);   // a NaN shows in its products
            x = max(x, max_s[gr]);
            x = x ? x | 0x7fu : 0u;             // all of the binade
            // s 2^k < 2^12, so that 8 s 2^k is an f16: k = 11 - (exponent of s)
            const float to = pow2(x ? min(11 - ((int)(x >> 7) - 127), 100) : 100);
            grow[gr] = to * inverse_pow2(top_s[gr]);
            top_s[gr] = to;
            max_s[gr] = x;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            float x = top[nt][j];
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            x = fmaxf(x - kAbove, m[nt][j]);
            const float k = ex2(m[nt][j] - x);
            m[nt][j] = x;
            l[nt][j] *= k;
            if constexpr (INT4) {
#pragma unroll
              for (int gr = 0; gr < NH; ++gr) zacc[nt][gr][j] *= k;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const float f = INT4 ? k * grow[INT4 ? mt / 2 : 0] : k;
#pragma unroll
              for (int e = j; e < 4; e += J) o[mt][nt][e] *= f;   // one row to two columns: both
            }
          }
      }
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; e += 3 - J) {
            const float p = ex2(s[x][nt][e] - m[nt][e & 1]);
            s[x][nt][e] = p;
            l[nt][e & 1] += p;
          }

      // ---- O^T += V^T P^T
      if constexpr (INT4) {
        // the step's scales times their 2^k as f16 pairs of neighbouring tokens
        __half* scales = reinterpret_cast<__half*>(ring + S * U * T::kBytes);
        const int tok = lane % kStep;
#pragma unroll
        for (int gr = 0; gr < NH; ++gr)
          scales[((tok >> 1) * NH + gr) * 2 + (tok & 1)] = __float2half_rn(cache::bf16_lo(sv[gr]) * top_s[gr]);
        __syncwarp();
        // the offsets' sum; the weights as two f16 terms: MMAs of their own, or (one row to two columns) the row's other column
        uint32_t ph[U][NT][2], pl[J == 2 ? U : 1][NT][2];
#pragma unroll
        for (int x = 0; x < U; ++x) {
          uint32_t vs[2][NH];   // rows g8, g8 + 8
#pragma unroll
          for (int j = 0; j < 2; ++j) lds_words<NH>(vs[j], st + x * T::kBytes + T::kVs + (g8 + 8 * j) * T::kRowVs);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float(&p)[4] = s[x][nt];
#pragma unroll
            for (int gr = 0; gr < NH; ++gr) {
              fma_columns<J>(zacc[nt][gr][0], zacc[nt][gr][J - 1], p[0], p[1], cache::bf16_hi(vs[0][gr]));
              fma_columns<J>(zacc[nt][gr][0], zacc[nt][gr][J - 1], p[2], p[3], cache::bf16_hi(vs[1][gr]));
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float h0 = leading11(p[2 * e]);
              if constexpr (J == 2) {
                const float h1 = leading11(p[2 * e + 1]);
                const float2 rest = f2_unpack(f2_fma(f2_pack(h0, h1), f2_pack(-1.f, -1.f), f2_pack(p[2 * e], p[2 * e + 1])));
                ph[x][nt][e] = movmatrix(pack_f16(h0, h1));
                pl[x][nt][e] = movmatrix(pack_f16(rest.x, rest.y));
              } else {
                ph[x][nt][e] = movmatrix(pack_f16(h0, p[2 * e] - h0));
              }
            }
          }
        }
        uint32_t vw[U][4][NH / 2];   // tokens 2q, 2q+1, 2q+8, 2q+9
#pragma unroll
        for (int x = 0; x < U; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 2 * q4 + (j & 1) + 8 * (j >> 1), at = g8 * (NH * 2);
            lds_words<NH / 2>(vw[x][j], st + x * T::kBytes + T::kV + row * T::kRowV + T::value_unit(row, at / 16) * 16 + at % 16);
          }
#pragma unroll
        for (int gr = 0; gr < NH; ++gr) {
          float y[2][NT][4];   // the step's own sum
#pragma unroll
          for (int x = 0; x < U; ++x) {
            const uint32_t* pair = reinterpret_cast<const uint32_t*>(scales) + (8 * x + q4) * NH + gr;
            const uint32_t s01 = pair[0], s89 = pair[4 * NH], sel = (gr & 1) ? 0x7632u : 0x5410u;
            const uint32_t lo = __byte_perm(vw[x][0][gr / 2], vw[x][1][gr / 2], sel);
            const uint32_t hi = __byte_perm(vw[x][2][gr / 2], vw[x][3][gr / 2], sel);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t wl = lo >> (8 * e), wh = hi >> (8 * e);
              const uint32_t a0 = low_values(wl, s01), a1 = high_values(wl, s01), a2 = low_values(wh, s89), a3 = high_values(wh, s89);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (J == 2) {
                  if (x == 0) mma_f16_first(y[e][nt], a0, a1, a2, a3, pl[x][nt][0], pl[x][nt][1]);
                  else mma_f16(y[e][nt], a0, a1, a2, a3, pl[x][nt][0], pl[x][nt][1]);
                }
                if (J == 1 && x == 0) mma_f16_first(y[e][nt], a0, a1, a2, a3, ph[x][nt][0], ph[x][nt][1]);
                else mma_f16(y[e][nt], a0, a1, a2, a3, ph[x][nt][0], ph[x][nt][1]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) add_to(o[2 * gr + e][nt], y[e][nt]);
        }
      } else {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          // the weights as two bf16 terms (2^-18): one alone made outputs 1.4 times as far off as their own rounding does.
          // And every tile's sum is added to the accumulators by itself, rounded: as the MMA's C they lost 2^-18 of the mean
          // value over 3,200 tiles.  1 or 2% while HBM bounds the call; rows beyond 16 a head, which the MMAs bound, pay (16 x
          // 16,800 tokens of 4 heads): the second term 110 -> 134 us for 32 rows, 207 -> 254 for 64; the sums another 5%
          uint32_t pb[NT][2], rest[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float p0 = s[x][nt][2 * e], p1 = s[x][nt][2 * e + 1];
              const uint32_t w = pack_bf16(p0, p1);
              pb[nt][e] = movmatrix(w);
              rest[nt][e] = movmatrix(pack_bf16(p0 - cache::bf16_lo(w), p1 - cache::bf16_hi(w)));
            }
          const char* vrow = st + x * T::kBytes + T::kV + 2 * q4 * T::kRowV;
#pragma unroll
          for (int i = 0; i < DV / 64; ++i) {
            const int at = T::value_unit(2 * q4, 8 * i + g8) * 16;   // the lane's four rows turn alike
            const uint4 v0 = *reinterpret_cast<const uint4*>(vrow + at), v1 = *reinterpret_cast<const uint4*>(vrow + T::kRowV + at);
            const uint4 v2 = *reinterpret_cast<const uint4*>(vrow + 8 * T::kRowV + at);
            const uint4 v3 = *reinterpret_cast<const uint4*>(vrow + 9 * T::kRowV + at);
            const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
            const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // word e holds dims 2 e and 2 e + 1 of the lane's eight
              const uint32_t a0 = __byte_perm(w0[e], w1[e], 0x5410), a1 = __byte_perm(w0[e], w1[e], 0x7632);
              const uint32_t a2 = __byte_perm(w2[e], w3[e], 0x5410), a3 = __byte_perm(w2[e], w3[e], 0x7632);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4];   // the tile's own sum: the MMA cuts off what the accumulator's last place does not hold
                mma_bf16_first(y, a0, a1, a2, a3, rest[nt][0], rest[nt][1]);
                mma_bf16(y, a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                add_to(o[4 * i + e][nt], y);
              }
            }
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();

    // ---- join the warps of a row group, in the ring's place: sums over the lanes of a column, then over
    // the warps
    float* s_o = reinterpret_cast<float*>(ring);   // [kCols][kRow], then maxima and sums
    float* s_m = s_o + kCols * kRow;
    float* s_l = s_m + kCols;
    if (ta >= tb) {   // no tiles: its sums are not read
      if (lane < kCols) {
        s_m[lane] = kNone;
        s_l[lane] = 0.f;
      }
    } else
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int col = row_of(nt, 2 * q4 + j);
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
        if (g8 == 0) {
          s_m[col] = m[nt][j];
          s_l[col] = l[nt][j];
        }
        float* row = s_o + col * kRow;
        if constexpr (INT4) {
#pragma unroll
          for (int gr = 0; gr < NH; ++gr) {
            float z = zacc[nt][gr][j];
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            const float down = inverse_pow2(top_s[gr]);
            const auto sum = [&](const float(&y)[4], int e) { return J == 2 ? y[e + j] : y[e] + y[e + 1]; };
            *reinterpret_cast<float4*>(row + 32 * gr + 4 * g8) =
                make_float4(fmaf(sum(o[2 * gr][nt], 0), down, z), fmaf(sum(o[2 * gr][nt], 2), down, z),
                            fmaf(sum(o[2 * gr + 1][nt], 0), down, z), fmaf(sum(o[2 * gr + 1][nt], 2), down, z));
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; mt += 2)
            *reinterpret_cast<float4*>(row + 64 * (mt / 4) + 8 * g8 + 2 * (mt % 4)) =
                make_float4(o[mt][nt][j], o[mt][nt][j + 2], o[mt + 1][nt][j], o[mt + 1][nt][j + 2]);
        }
      }
    __syncthreads();
    const bool alone = take == sp.tiles;   // else: to the slot of a run that begins (1) or continues (0) the item
    const size_t slot = (size_t)blockIdx.x * 2 + (first == 0);
    for (int x = threadIdx.x; x < tile_rows * (DV / 4); x += W * 32) {
      const int rr = x / (DV / 4), d = (x % (DV / 4)) * 4, col = rr % kCols, r = rt * pl.tile_rows + rr;
      const char* base = smem + (rr / kCols) * kWarpBytes;   // the first warp of the row's group
      const size_t step = (size_t)pl.row_groups * kWarpBytes;
      float mw[W], lw[W], mm = kNone, ll = 0.f;   // all streams' loads side by side
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float* f = reinterpret_cast<const float*>(base + w * step) + kCols * kRow + col;
        mw[w] = w < streams ? f[0] : kNone;
        lw[w] = w < streams ? f[kCols] : 0.f;
      }
      float4 y[W], acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        mm = fmaxf(mm, mw[w]);
        y[w] = lw[w] == 0.f ? acc : *reinterpret_cast<const float4*>(base + w * step + (col * kRow + d) * 4);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float k = ex2(mw[w] - mm);
        ll += k * lw[w];
        acc.x += k * y[w].x; acc.y += k * y[w].y; acc.z += k * y[w].z; acc.w += k * y[w].w;
      }
      if (alone) {
        const size_t row = out_row(r);
        const float inv = ll > 0.f ? 1.f / ll : ll;   // a NaN stays one; nothing attended: zeros
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + d) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if (a.lse && d == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      } else {
        const size_t row = slot * pl.tile_rows + rr;
        *reinterpret_cast<float4*>(part_o + row * DV + d) = acc;
        if (d == 0) part_ml[row] = make_float2(mm, ll);
      }
    }
    next_item();
    if (left > 0) __syncthreads();   // the next item's copies reuse the ring
  }
  if (!pl.whole && threadIdx.x == 0) cuts[blockIdx.x] = cut;
}

// Joins the parts of the items that were cut: block (x, y) those of the item whose first part block x
// has, WPR warps per row, the row's parts shared out to them and their sums joined in order.
constexpr int kJoinWarps = 8;
template <int DV, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32)
cache_join_kernel(const CacheArgs c, const CacheAttnArgs a, const Plan pl, const Cut* cuts, const float2* part_ml,
                  const float* part_o) {
  constexpr int kPer = DV / 32;
  __shared__ float s_acc[WPR > 1 ? kJoinWarps : 1][DV];
  __shared__ float2 s_ml[WPR > 1 ? kJoinWarps : 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // every thread, also of blocks with nothing to join
  const Cut cut = cuts[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int rr = blockIdx.y * (kJoinWarps / WPR) + warp / WPR;
  if (cut.last < 0 || rr >= cut.rows) return;   // WPR > 1: the whole block
  const int n = cut.last - (int)blockIdx.x + 1;   // parts: slot 1 of this block, slot 0 of the next ones
  const auto at = [&](int i) { return ((size_t)(blockIdx.x + i) * 2 + (i == 0)) * pl.tile_rows + rr; };
  const auto fetch = [&](int i, float (&v)[kPer]) {
    const float* y = part_o + at(i) * DV + lane * kPer;
    if constexpr (kPer == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(y);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(y);
  };
  constexpr int kAhead = 4;   // parts of this warp on their way at once; the first before the maxima are known
  float v[kAhead][kPer];
#pragma unroll
  for (int x = 0; x < kAhead; ++x)
    if (sub + x * WPR < n) fetch(sub + x * WPR, v[x]);
  float mm = kNone;
  for (int i = lane; i < n; i += 32) mm = fmaxf(mm, part_ml[at(i)].x);
#pragma unroll
  for (int d = 1; d <= 16; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
  float ll = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int i0 = sub; i0 < n; i0 += kAhead * WPR) {
    if (i0 != sub) {
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (i0 + x * WPR < n) fetch(i0 + x * WPR, v[x]);
    }
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (i0 + x * WPR >= n) break;
      const float2 ml = part_ml[at(i0 + x * WPR)];
      const float k = ex2(ml.x - mm);
      ll += k * ml.y;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += k * v[x][e];
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) s_acc[warp][lane * kPer + e] = acc[e];
    if (lane == 0) s_ml[warp] = make_float2(0.f, ll);
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      ll += s_ml[warp + w].y;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += s_acc[warp + w][lane * kPer + e];
    }
  }
  const int h = cut.head_tile / pl.row_tiles, r = cut.head_tile % pl.row_tiles * pl.tile_rows + rr, i = row_token(pl, r);
  const size_t row = ((size_t)cut.b * a.n_new + i) * a.h_q + h * a.G + (r - i * a.G);
  const float inv = ll > 0.f ? 1.f / ll : ll;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + lane * kPer);
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) dst[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// Warps per block, blocks per SM, tiles of 16 tokens per step.  4 bits: eight warps an SM of up to 255 registers (with 16
// rows and (128, 128) or (192, 128) 32 to 47 words of a thread spill, in bf16 18 to 45); twelve of 168 spill far more (16
// rows, 8 x 64K tokens: 208 us instead of 157), and one tile a step leaves a warp too little that is independent (169).
// bf16: the ring needs the shared memory.
template <bool INT4, int NT, int J>
struct Shape {
  static constexpr bool kInt4 = INT4;
  static constexpr int kNT = NT, kJ = J, kRows = NT * 4 * J;
  static constexpr int W = INT4 ? 4 : 8;
  static constexpr int B = INT4 ? 2 : 1;
  static constexpr int U = INT4 ? 2 : 1;
};
// Stages of the ring: as many as fit beside the other blocks of the SM, at most 4 (4 bits: 3).
template <bool INT4, int DK, int DV, int NT, int J>
constexpr int stages() {
  using H = Shape<INT4, NT, J>;
  constexpr int room = 227 * 1024 / H::B - 1024 - 1024 - query_smem<INT4, DK, NT>() - H::W * scale_smem<INT4, DV, H::U>();
  return std::min(INT4 ? 3 : 4, room / (H::W * H::U * Stage<INT4, DK, DV>::kBytes));
}
// f of the shape a call's rows take: up to 16 of a head, its queries times its new tokens.  Four at most
// use one of a lane's columns (4 bits, 32 heads of one query over 64K tokens: 93 us instead of 99); a bf16
// cache waits for memory either way.
template <class F>
auto with_shape(bool int4, int rows, F f) {
  if (!int4) return rows > 8 ? f(Shape<false, 2, 2>()) : f(Shape<false, 1, 2>());
  return rows > 8 ? f(Shape<true, 2, 2>()) : rows > 4 ? f(Shape<true, 1, 2>()) : f(Shape<true, 1, 1>());
}

constexpr int kSms = 148;
// A warp's share of items that are not cut: the second kernel and the parts cost 2 to 5 us, so does a share of 128 tokens
// (8 rows, 32 items of 500 tokens: whole 7.5 us in bf16 and 9.1 in 4 bits, cut 9.2 and 10.8; of twice that, 13.0 and 13.4
// against 10.5 and 11.2).  Twice as much where the items alone fill the SMs, from 64 on: there it is about even (1,500
// tokens in bf16 13.1 and 13.0, 1,000 in 4 bits 13.6 and 12.8), at 128 items 14.4 against 19.1 and 13.9 against 17.6.
constexpr int kWholeTokens = 128, kManyItems = 64;

Plan plan_of(const CacheArgs& c, const CacheAttnArgs& a) {
  Plan p{};
  const int R = a.n_new * a.G;
  int W = 0, step = 0, resident = 0, rows = 0;
  with_shape(c.int4, R, [&](auto h) { W = h.W; step = kTile * h.U; resident = h.B; rows = h.kRows; });
  p.row_groups = R <= 16 ? 1 : R <= 32 ? 2 : 4;
  p.tile_rows = rows * p.row_groups;
  p.row_tiles = (R + p.tile_rows - 1) / p.tile_rows;
  p.per_g = (65536 + a.G - 1) / a.G;
  for (int rt = 0; rt < p.row_tiles; ++rt) {   // R <= 256: at most four tiles, of 64 rows
    p.first[rt] = rt * p.tile_rows / a.G;
    p.last[rt] = (std::min(R, (rt + 1) * p.tile_rows) - 1) / a.G;
  }
  // the most tiles an item can have
  long long range = a.max_seqlen;
  if (a.window > 0) range = std::min<long long>(range, (long long)a.window + a.n_new + kTile);
  const long long tiles = (range + step - 1) / step, items = (long long)c.batch * c.h_kv * p.row_tiles;
  p.min_tiles = 2 * (W / p.row_groups);
  p.small = items * (tiles + 4 * W) < (1 << 30);
  p.whole = range <= kWholeTokens * (W / p.row_groups) * (items >= kManyItems ? 2 : 1);
  const long long most = (long long)kSms * resident;
  // items <= 2^31 (cache_attn_fits), tiles <= 2^26
  p.blocks = (int)(p.whole ? std::min<long long>(items, INT32_MAX) : std::min(most, (items * tiles + p.min_tiles - 1) / p.min_tiles));
  return p;
}

struct Parts {
  size_t cuts, ml, o, bytes;
};
Parts parts_of(const CacheArgs& c, const Plan& p) {
  Parts x{};
  if (p.whole) return x;
  const size_t rows = (size_t)p.blocks * 2 * p.tile_rows;
  x.ml = (size_t)p.blocks * sizeof(Cut);                    // multiples of 16 bytes throughout
  x.o = x.ml + rows * sizeof(float2);
  x.bytes = x.o + rows * c.dv * sizeof(float);
  return x;
}

// The join waits on the device for the blocks that it reads from, so that its launch is behind it by then.
template <int DV, int WPR>
cudaError_t launch_join(const CacheArgs& c, const CacheAttnArgs& a, const Plan& p, const Cut* cuts, const float2* ml,
                        const float* o, cudaStream_t st) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.blocks, (p.tile_rows * WPR + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_join_kernel<DV, WPR>, c, a, p, cuts, ml, o);
}

template <class H, bool INT4, int DK, int DV, bool EXT>
cudaError_t launch_variant(const CacheArgs& c, const CacheAttnArgs& a, const Plan& p, cudaStream_t st) {
  constexpr int NT = H::kNT, J = H::kJ, S = stages<INT4, DK, DV, NT, J>();
  constexpr int kRing = H::W * warp_smem<INT4, DK, DV, NT, H::U, S>(), kQ = query_smem<INT4, DK, NT>();
  static_assert(S >= 2 && (kRing + kQ + 2048) * H::B <= 228 * 1024, "the rings of the resident blocks fit an SM");
  static_assert(kRing + 4 * kQ <= 227 * 1024, "a block's shared memory");
  static PerDevice set;
  auto* f = cache_attn_kernel<INT4, DK, DV, NT, J, H::W, H::B, H::U, S, EXT>;
  cudaError_t e = set.once([&] { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 4 * kQ); });
  if (e != cudaSuccess) return e;
  const Parts x = parts_of(c, p);
  char* ws = static_cast<char*>(a.workspace);
  Cut* cuts = reinterpret_cast<Cut*>(ws);
  float2* ml = reinterpret_cast<float2*>(ws + x.ml);
  float* o = reinterpret_cast<float*>(ws + x.o);
  f<<<p.blocks, H::W * 32, kRing + p.row_groups * kQ, st>>>(c, a, p, cuts, ml, o);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  // few items, many parts each: a block per row; else a warp per row
  const long long items = (long long)c.batch * c.h_kv * p.row_tiles;
  if (items * 16 <= p.blocks) return launch_join<DV, kJoinWarps>(c, a, p, cuts, ml, o, st);
  return launch_join<DV, 1>(c, a, p, cuts, ml, o, st);
}

template <int DK, int DV>
cudaError_t launch_dims(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t st) {
  const Plan p = plan_of(c, a);
  const bool ext = a.softcap > 0.f || a.slopes;
  return with_shape(c.int4, a.n_new * a.G, [&](auto h) {
    using H = decltype(h);
    return ext ? launch_variant<H, H::kInt4, DK, DV, true>(c, a, p, st) : launch_variant<H, H::kInt4, DK, DV, false>(c, a, p, st);
  });
}

}  // namespace

size_t cache_attn_workspace(const CacheArgs& c, const CacheAttnArgs& a) { return parts_of(c, plan_of(c, a)).bytes; }

bool cache_attn_fits(const CacheArgs& c, const CacheAttnArgs& a) {
  return (long long)c.batch * c.h_kv * plan_of(c, a).row_tiles <= INT32_MAX;
}

cudaError_t launch_cache_attn(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t st) {
  if (c.dk == 64) return launch_dims<64, 64>(c, a, st);
  if (c.dk == 128) return launch_dims<128, 128>(c, a, st);
  return launch_dims<192, 128>(c, a, st);
}

}  // namespace nsa
