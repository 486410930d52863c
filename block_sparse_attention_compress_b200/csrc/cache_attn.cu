// Attention of the newest tokens over a paged cache in bf16 or 4 bits.
//
// Per KV head the query rows (n_new tokens x G heads) stand as the MMA's N (tiles of 8) and 16
// cached tokens as its M, so that a group of 8 heads wastes nothing:
//   S[key, row]  = K Q^T      A = K as it lies in memory: a lane takes its quad's share of a key
//                             row, and the queries' dims are permuted to match;
//   O^T[d, row] += V^T P^T    A = V^T: a register pairs two tokens of one dim (byte permutes), and
//                             the tile's dims are permuted to match.  S's C fragment becomes
//                             P^T's B fragment by movmatrix.
// Keys in 4 bits: (w >> 8 i) & 0x000f000f and & 0x00f000f0 are pairs of f16 subnormals c 2^-24 and
// c 2^-20, which the tensor cores multiply exactly: no conversion.  The queries of the latter are
// divided by 16, and every query row is scaled by a power of two so that f16 holds it.  The
// group's (s, z) come in behind the product: S = sum_g s_g (sum c q) + (z_g - 8 s_g) sum_g q.
// Values in 4 bits: codes become the bf16 integers c - 8 and P is scaled by the token's s (one
// rounding); P z is summed in fp32.
// The keys of a sequence are split over blocks, a block's over its warps; the parts are joined
// by their maxima and sums in a fixed order.  Bound: the cache's bytes.
#include <algorithm>

#include "cache.cuh"

namespace nsa {
namespace {

constexpr int kWarps = 8;
constexpr int kTile = 16;   // tokens per step of a warp
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// N 32-bit words from global memory, as wide as 8-byte alignment (16 for N = 4) allows
template <int N>
__device__ __forceinline__ void ld_words(uint32_t (&w)[N], const void* p) {
  if constexpr (N == 4) {
    const uint4 u = __ldg(static_cast<const uint4*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const uint2 u = __ldg(static_cast<const uint2*>(p) + i);
      w[2 * i] = u.x; w[2 * i + 1] = u.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(static_cast<const uint32_t*>(p) + i);
  }
}

// cap tanh(x / cap): 1 - 2 / (e^2t + 1), and for small t, where that loses the digits of t, the
// series t - t^3/3 + 2 t^5/15 - 17 t^7/315 + 62 t^9/2835 (the next term is below 1e-8 t at t = 1/4).
__device__ __forceinline__ float capped(float x, float cap) {
  const float t = x / cap, t2 = t * t;
  const float big = 1.f - __fdividef(2.f, ex2(t * (2.f * kLog2e)) + 1.f);
  float p = fmaf(t2, 62.f / 2835.f, -17.f / 315.f);
  p = fmaf(t2, p, 2.f / 15.f);
  p = fmaf(t2, p, -1.f / 3.f);
  return cap * (fabsf(t) < 0.25f ? fmaf(t * t2, p, t) : big);
}

// A column's running maximum before any token: below every finite score, and finite, so that
// 2^(-inf - kNone) is 0 (a masked token) and 2^(NaN - kNone) a NaN (an attended one).
constexpr float kNone = -3.0e38f;

// The keys a tile of rows attends to, of one sequence: [lo, hi), cut into n parts of `chunk` from
// base on; rows see [p - window + 1, p] with p = p0 + (row's token).
struct Span {
  int p0, lo, hi, base, n;
};
__device__ __forceinline__ Span span_of(int len, int n_new, int i0, int i1, int window, int chunk) {
  Span s;
  s.p0 = len - n_new;
  s.hi = max(0, s.p0 + i1 + 1);
  s.lo = window > 0 ? max(0, s.p0 + i0 - window + 1) : 0;
  s.base = s.lo & ~(kTile - 1);
  s.n = s.hi > s.base ? (s.hi - s.base + chunk - 1) / chunk : 1;
  return s;
}

__device__ __forceinline__ int seq_len_clamped(const CacheArgs& c, const CacheAttnArgs& a, int b, bool tell) {
  const int n = __ldg(a.seqlens + b);
  if (tell && (n < 0 || n > a.max_seqlen)) cache::report(c.status);
  return min(max(n, 0), a.max_seqlen);
}

template <bool INT4, int DK, int DV, int NT>
struct Frag {   // registers of one 16-token tile
  static constexpr int NG = DK / 32, NH = DV / 32;
  uint32_t k[2][INT4 ? NG : DK / 8];    // rows lane / 4 and lane / 4 + 8
  uint32_t v[4][INT4 ? NH / 2 : DV / 16];   // tokens 2q, 2q+1, 2q+8, 2q+9 (q = lane % 4)
  uint32_t ks[2][INT4 ? NG : 1], vs[2][INT4 ? NH : 1];
};

template <bool INT4, int DK, int DV, int NT, bool EXT>
__global__ void __launch_bounds__(kWarps * 32)
cache_attn_kernel(const CacheArgs c, const CacheAttnArgs a, int chunk, int splits, int row_tiles,
                  float* __restrict__ part_o, float2* __restrict__ part_ml) {
  constexpr int NG = DK / 32, NH = DV / 32, MT = DV / 16, KS = DK / 16;
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, q4 = lane & 3;
  int bid = blockIdx.x;
  const int rt = bid % row_tiles; bid /= row_tiles;
  const int h = bid % c.h_kv; bid /= c.h_kv;
  const int split = bid % splits, b = bid / splits;
  const int R = a.n_new * a.G, r0 = rt * NT * 8, r1 = min(R, r0 + NT * 8);
  const int i0 = r0 / a.G, i1 = (r1 - 1) / a.G;
  const int len = seq_len_clamped(c, a, b, threadIdx.x == 0 && split == 0 && h == 0 && rt == 0);
  const Span sp = span_of(len, a.n_new, i0, i1, a.window, chunk);
  if (split >= sp.n) return;

  // ---- queries as B fragments: row n = lane / 4 of each tile of 8
  uint32_t qf[NT][KS][2];
  float qz[INT4 ? NT : 1][NG][2];   // 4 bits: the sum of each group's queries, for columns 2q, 2q+1
  float sc[NT][2];                  // what a column's raw score is multiplied by (natural units)
  int pos[NT][2];                   // the columns' positions
  float slope[EXT ? NT : 1][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = min(r0 + nt * 8 + g8, R - 1), i = r / a.G, g = r - i * a.G;
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + (((size_t)b * a.n_new + i) * a.h_q + h * a.G + g) * DK;
    if constexpr (!INT4) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(qr + 32 * (ks >> 1) + 8 * q4 + 4 * (ks & 1)));
        qf[nt][ks][0] = u.x;
        qf[nt][ks][1] = u.y;
      }
      sc[nt][0] = sc[nt][1] = a.scale;
    } else {
      uint4 u[NG];
      float amax = 0.f;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        u[gr] = __ldg(reinterpret_cast<const uint4*>(qr + 32 * gr + 8 * q4));
        const uint32_t w[4] = {u[gr].x, u[gr].y, u[gr].z, u[gr].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(cache::bf16_lo(w[e])), fabsf(cache::bf16_hi(w[e]))));
      }
      amax = warp_max4(amax);
      // a power of two that takes the row's largest query into [2^13, 2^14)
      int e2 = (int)((__float_as_uint(amax) >> 23) & 255u);
      e2 = (e2 == 0 || e2 == 255) ? 0 : 13 - (e2 - 127);
      e2 = min(max(e2, -120), 120);
      const float up = __uint_as_float((uint32_t)(e2 + 127) << 23), down = __uint_as_float((uint32_t)(127 - e2) << 23);
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const uint32_t w[4] = {u[gr].x, u[gr].y, u[gr].z, u[gr].w};
        float x[8], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = cache::bf16_lo(w[e]) * up;
          x[2 * e + 1] = cache::bf16_hi(w[e]) * up;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += x[e];
        const __half2 b00 = __floats2half2_rn(x[0], x[4]), b01 = __floats2half2_rn(x[1] * 0.0625f, x[5] * 0.0625f);
        const __half2 b10 = __floats2half2_rn(x[2], x[6]), b11 = __floats2half2_rn(x[3] * 0.0625f, x[7] * 0.0625f);
        qf[nt][2 * gr][0] = *reinterpret_cast<const uint32_t*>(&b00);
        qf[nt][2 * gr][1] = *reinterpret_cast<const uint32_t*>(&b01);
        qf[nt][2 * gr + 1][0] = *reinterpret_cast<const uint32_t*>(&b10);
        qf[nt][2 * gr + 1][1] = *reinterpret_cast<const uint32_t*>(&b11);
        sum = warp_sum4(sum);
        // the products carry 2^-24 (the subnormals): so does the sum beside them
        sum *= 0x1p-24f;
        qz[nt][gr][0] = __shfl_sync(0xffffffffu, sum, 8 * q4);
        qz[nt][gr][1] = __shfl_sync(0xffffffffu, sum, 8 * q4 + 4);
      }
      const float f = a.scale * down;
      sc[nt][0] = __shfl_sync(0xffffffffu, f, 8 * q4);
      sc[nt][1] = __shfl_sync(0xffffffffu, f, 8 * q4 + 4);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int rc = min(r0 + nt * 8 + 2 * q4 + j, R - 1), ic = rc / a.G;
      pos[nt][j] = sp.p0 + ic;
      if constexpr (EXT) slope[nt][j] = a.slopes ? __ldg(a.slopes + h * a.G + rc - ic * a.G) * kLog2e : 0.f;
    }
  }

  float o[MT][NT][4];
  float m[NT][2], l[NT][2], zacc[INT4 ? NT : 1][NH][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
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

  // ---- this warp's run of tiles
  const int start = sp.base + split * chunk, stop = min(sp.hi, start + chunk);
  const int tiles = (max(0, stop - start) + kTile - 1) / kTile, per = (tiles + kWarps - 1) / kWarps;
  const int t1 = min(tiles, (warp + 1) * per);
  // tiles inside [all_lo, all_hi) are seen whole by every row
  const int all_lo = a.window > 0 ? sp.p0 + i1 - a.window + 1 : 0, all_hi = sp.p0 + i0 + 1;

  for (int t = warp * per; t < t1; ++t) {
    const int u0 = start + t * kTile;
    const int pj = u0 / c.page_size;
    const int page = __ldg(c.page_table + (size_t)b * c.max_pages + pj);
    if (page < 0 || page >= c.n_pages) {
      if (lane == 0) cache::report(c.status);
      continue;
    }
    const int off = u0 - pj * c.page_size;   // place of the tile's first token
    // places of this lane's tokens; those outside [lo, hi) are masked, and load a row inside
    const int c_lo = max(0, sp.lo - u0), c_hi = min(kTile, sp.hi - u0) - 1;
    Frag<INT4, DK, DV, NT> f;
    const size_t head_row = ((size_t)page * c.h_kv + h) * c.page_size + off;   // 4 bits
    const size_t tok_row = ((size_t)page * c.page_size + off) * c.h_kv + h;    // bf16
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int x = min(max(g8 + 8 * j, c_lo), c_hi);
      if constexpr (INT4) {
        ld_words<NG>(f.k[j], static_cast<const uint8_t*>(c.k) + (head_row + x) * (DK / 2) + q4 * (NG * 4));
        ld_words<NG>(f.ks[j], static_cast<const uint8_t*>(c.k_scale) + (head_row + x) * (NG * 4));
        ld_words<NH>(f.vs[j], static_cast<const uint8_t*>(c.v_scale) + (head_row + x) * (NH * 4));
      } else {
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.k) + (tok_row + (size_t)x * c.h_kv) * DK);
#pragma unroll
        for (int i = 0; i < DK / 32; ++i) {
          const uint4 u = __ldg(row + 4 * i + q4);
          f.k[j][4 * i] = u.x; f.k[j][4 * i + 1] = u.y; f.k[j][4 * i + 2] = u.z; f.k[j][4 * i + 3] = u.w;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = min(max(2 * q4 + (j & 1) + 8 * (j >> 1), c_lo), c_hi);
      if constexpr (INT4) {
        ld_words<NH / 2>(f.v[j], static_cast<const uint8_t*>(c.v) + (head_row + x) * (DV / 2) + g8 * (NH * 2));
      } else {
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(c.v) + (tok_row + (size_t)x * c.h_kv) * DV);
#pragma unroll
        for (int i = 0; i < DV / 64; ++i) {
          const uint4 u = __ldg(row + 8 * i + g8);
          f.v[j][4 * i] = u.x; f.v[j][4 * i + 1] = u.y; f.v[j][4 * i + 2] = u.z; f.v[j][4 * i + 3] = u.w;
        }
      }
    }

    // ---- S = K Q^T
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
    if constexpr (INT4) {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const uint32_t w0 = f.k[0][gr], w1 = f.k[1][gr], x0 = w0 >> 8, x1 = w1 >> 8;
        const float s0 = cache::bf16_lo(f.ks[0][gr]), s1 = cache::bf16_lo(f.ks[1][gr]);
        const float z0 = fmaf(-8.f, s0, cache::bf16_hi(f.ks[0][gr])), z1 = fmaf(-8.f, s1, cache::bf16_hi(f.ks[1][gr]));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(acc, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, qf[nt][2 * gr][0],
                  qf[nt][2 * gr][1]);
          mma_f16(acc, x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u, qf[nt][2 * gr + 1][0],
                  qf[nt][2 * gr + 1][1]);
          s[nt][0] += s0 * acc[0] + z0 * qz[nt][gr][0];
          s[nt][1] += s0 * acc[1] + z0 * qz[nt][gr][1];
          s[nt][2] += s1 * acc[2] + z1 * qz[nt][gr][0];
          s[nt][3] += s1 * acc[3] + z1 * qz[nt][gr][1];
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_bf16(s[nt], f.k[0][2 * ks], f.k[1][2 * ks], f.k[0][2 * ks + 1], f.k[1][2 * ks + 1], qf[nt][ks][0],
                   qf[nt][ks][1]);
    }

    // ---- softmax: scores in log2 units, the reference moved only when a score passes it by 8
    const bool inner = u0 >= all_lo && u0 + kTile <= all_hi;
    bool move = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e & 1, u = u0 + g8 + 8 * (e >> 1);
        float x = s[nt][e] * sc[nt][j];
        if constexpr (INT4) x *= 0x1p24f;
        if constexpr (EXT) {
          if (a.softcap > 0.f) x = capped(x, a.softcap);
          x = fmaf(x, kLog2e, slope[nt][j] * (float)(u - pos[nt][j]));
        } else {
          x *= kLog2e;
        }
        if (!inner) {
          const int p = pos[nt][j];
          if (u > p || u < sp.lo || (a.window > 0 && u <= p - a.window)) x = -INFINITY;
        }
        s[nt][e] = x;
        move |= x > m[nt][j] + 8.f;
      }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(s[nt][j], s[nt][j + 2]);
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
          x = fmaxf(x, m[nt][j]);
          const float k = ex2(m[nt][j] - x);
          m[nt][j] = x;
          l[nt][j] *= k;
          if constexpr (INT4) {
#pragma unroll
            for (int gr = 0; gr < NH; ++gr) zacc[nt][gr][j] *= k;
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[mt][nt][j] *= k;
            o[mt][nt][j + 2] *= k;
          }
        }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float p = ex2(s[nt][e] - m[nt][e & 1]);
        s[nt][e] = p;
        l[nt][e & 1] += p;
      }

    // ---- O^T += V^T P^T
    if constexpr (INT4) {
#pragma unroll
      for (int gr = 0; gr < NH; ++gr) {
        uint32_t pb[NT][2];
        const float s0 = cache::bf16_lo(f.vs[0][gr]), s1 = cache::bf16_lo(f.vs[1][gr]);
        const float z0 = cache::bf16_hi(f.vs[0][gr]), z1 = cache::bf16_hi(f.vs[1][gr]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = movmatrix(pack_bf16(s[nt][0] * s0, s[nt][1] * s0));
          pb[nt][1] = movmatrix(pack_bf16(s[nt][2] * s1, s[nt][3] * s1));
          zacc[nt][gr][0] += s[nt][0] * z0 + s[nt][2] * z1;
          zacc[nt][gr][1] += s[nt][1] * z0 + s[nt][3] * z1;
        }
        const uint32_t sel = (gr & 1) ? 0x7632u : 0x5410u;
        const uint32_t lo = __byte_perm(f.v[0][gr / 2], f.v[1][gr / 2], sel);
        const uint32_t hi = __byte_perm(f.v[2][gr / 2], f.v[3][gr / 2], sel);
        uint32_t al[4], ah[4];
        const uint32_t magic = 0x43004300u, off8 = 0x43084308u;   // 128 + c and 136 in bf16
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint32_t x = ((lo >> (4 * n)) & 0x000f000fu) | magic, y = ((hi >> (4 * n)) & 0x000f000fu) | magic;
          const __nv_bfloat162 e = *reinterpret_cast<const __nv_bfloat162*>(&off8);
          const __nv_bfloat162 dx = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), e);
          const __nv_bfloat162 dy = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&y), e);
          al[n] = *reinterpret_cast<const uint32_t*>(&dx);
          ah[n] = *reinterpret_cast<const uint32_t*>(&dy);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_bf16(o[2 * gr][nt], al[0], al[1], ah[0], ah[1], pb[nt][0], pb[nt][1]);
          mma_bf16(o[2 * gr + 1][nt], al[2], al[3], ah[2], ah[3], pb[nt][0], pb[nt][1]);
        }
      }
    } else {
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        pb[nt][0] = movmatrix(pack_bf16(s[nt][0], s[nt][1]));
        pb[nt][1] = movmatrix(pack_bf16(s[nt][2], s[nt][3]));
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {   // word mt holds dims 2 mt and 2 mt + 1 of the lane's eight
        const uint32_t a0 = __byte_perm(f.v[0][mt], f.v[1][mt], 0x5410), a1 = __byte_perm(f.v[0][mt], f.v[1][mt], 0x7632);
        const uint32_t a2 = __byte_perm(f.v[2][mt], f.v[3][mt], 0x5410), a3 = __byte_perm(f.v[2][mt], f.v[3][mt], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16(o[mt][nt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }
  }

  // ---- join the warps: sums over the lanes of a column, then over the warps through shared memory
  constexpr int kCols = NT * 8, kRow = DV + 4;
  float* s_o = smem;                                  // [kWarps][kCols][kRow]
  float* s_m = smem + kWarps * kCols * kRow;          // [kWarps][kCols]
  float* s_l = s_m + kWarps * kCols;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = nt * 8 + 2 * q4 + j;
#pragma unroll
      for (int d = 4; d <= 16; d <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], d);
      if (g8 == 0) {
        s_m[warp * kCols + col] = m[nt][j];
        s_l[warp * kCols + col] = l[nt][j];
      }
      float* row = s_o + (warp * kCols + col) * kRow;
      if constexpr (INT4) {
#pragma unroll
        for (int gr = 0; gr < NH; ++gr) {
          float z = zacc[nt][gr][j];
#pragma unroll
          for (int d = 4; d <= 16; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
          *reinterpret_cast<float4*>(row + 32 * gr + 4 * g8) =
              make_float4(o[2 * gr][nt][j] + z, o[2 * gr][nt][j + 2] + z, o[2 * gr + 1][nt][j] + z, o[2 * gr + 1][nt][j + 2] + z);
        }
      } else {
#pragma unroll
        for (int mt = 0; mt < MT; mt += 2)
          *reinterpret_cast<float4*>(row + 64 * (mt / 4) + 8 * g8 + 2 * (mt % 4)) =
              make_float4(o[mt][nt][j], o[mt][nt][j + 2], o[mt + 1][nt][j], o[mt + 1][nt][j + 2]);
      }
    }
  __syncthreads();
  for (int x = threadIdx.x; x < (r1 - r0) * (DV / 4); x += kWarps * 32) {
    const int col = x / (DV / 4), d = (x % (DV / 4)) * 4, r = r0 + col;
    float mm = kNone;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * kCols + col]);
    float ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float k = ex2(s_m[w * kCols + col] - mm);
      const float4 y = *reinterpret_cast<const float4*>(s_o + (w * kCols + col) * kRow + d);
      ll += k * s_l[w * kCols + col];
      acc.x += k * y.x; acc.y += k * y.y; acc.z += k * y.z; acc.w += k * y.w;
    }
    if (sp.n == 1) {
      const int i = r / a.G;
      const size_t row = ((size_t)b * a.n_new + i) * a.h_q + h * a.G + (r - i * a.G);
      const float inv = ll > 0.f ? 1.f / ll : ll;   // a NaN stays one; nothing attended: zeros
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + d) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      if (a.lse && d == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    } else {
      const size_t row = (((size_t)b * c.h_kv + h) * R + r) * splits + split;
      *reinterpret_cast<float4*>(part_o + row * DV + d) = acc;
      if (d == 0) part_ml[row] = make_float2(mm, ll);
    }
  }
}

// Joins the parts of a row: one warp per row, in the order of the parts.
template <int DV>
__global__ void cache_join_kernel(const CacheArgs c, const CacheAttnArgs a, int chunk, int splits, int tile_rows,
                                  const float* __restrict__ part_o, const float2* __restrict__ part_ml) {
  constexpr int kPer = DV / 32;
  const int lane = threadIdx.x & 31, R = a.n_new * a.G;
  const long long id = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (id >= (long long)c.batch * c.h_kv * R) return;
  const int r = (int)(id % R), h = (int)(id / R % c.h_kv), b = (int)(id / R / c.h_kv);
  const int r0 = r / tile_rows * tile_rows, r1 = min(R, r0 + tile_rows);
  const Span sp = span_of(seq_len_clamped(c, a, b, false), a.n_new, r0 / a.G, (r1 - 1) / a.G, a.window, chunk);
  if (sp.n == 1) return;   // written by the block itself
  const size_t base = (size_t)id * splits;
  float mm = kNone;
  for (int s = lane; s < sp.n; s += 32) mm = fmaxf(mm, part_ml[base + s].x);
#pragma unroll
  for (int d = 1; d <= 16; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
  float ll = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int s = 0; s < sp.n; ++s) {
    const float2 ml = part_ml[base + s];
    const float k = ex2(ml.x - mm);
    ll += k * ml.y;
    const float* y = part_o + (base + s) * DV + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += k * y[e];
  }
  const int i = r / a.G;
  const size_t row = ((size_t)b * a.n_new + i) * a.h_q + h * a.G + (r - i * a.G);
  const float inv = ll > 0.f ? 1.f / ll : ll;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * DV + lane * kPer);
#pragma unroll
  for (int e = 0; e < kPer / 2; ++e) dst[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// How a call is cut: rows per block, tokens per block, parts per sequence.
struct Plan {
  int nt, row_tiles, chunk, splits;
  size_t rows;   // parts of rows kept in the workspace
};

Plan plan_of(const CacheArgs& c, const CacheAttnArgs& a) {
  Plan p;
  const int R = a.n_new * a.G;
  p.nt = R <= 8 ? 1 : 2;
  p.row_tiles = (R + p.nt * 8 - 1) / (p.nt * 8);
  // the longest range of keys a block's rows can have, from its first tile on
  long long range = a.max_seqlen;
  if (a.window > 0) range = std::min<long long>(range, (long long)a.window + a.n_new + kTile);
  const long long items = (long long)c.batch * c.h_kv * p.row_tiles;
  const long long slots = 148 * 2;
  const long long want = std::max<long long>(1, (2 * slots + items - 1) / items);
  long long chunk = (range + want - 1) / want;
  chunk = std::max<long long>(kWarps * kTile, (chunk + kWarps * kTile - 1) / (kWarps * kTile) * (kWarps * kTile));
  p.chunk = (int)chunk;
  p.splits = (int)((range + chunk - 1) / chunk);
  p.rows = p.splits > 1 ? (size_t)c.batch * c.h_kv * R * p.splits : 0;
  return p;
}

template <bool INT4, int DK, int DV, int NT, bool EXT>
cudaError_t launch_variant(const CacheArgs& c, const CacheAttnArgs& a, const Plan& p, float* po, float2* pml, cudaStream_t st) {
  constexpr int kSmem = kWarps * NT * 8 * (DV + 4 + 2) * 4;
  static PerDevice set;
  auto* f = cache_attn_kernel<INT4, DK, DV, NT, EXT>;
  cudaError_t e = set.once([&] { return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)c.batch * p.splits * c.h_kv * p.row_tiles;   // cache_attn_fits
  f<<<grid, kWarps * 32, kSmem, st>>>(c, a, p.chunk, p.splits, p.row_tiles, po, pml);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t launch_dims(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t st) {
  const Plan p = plan_of(c, a);
  float2* pml = static_cast<float2*>(a.workspace);
  float* po = reinterpret_cast<float*>(pml + (p.rows + 1) / 2 * 2);
  const bool ext = a.softcap > 0.f || a.slopes;
  cudaError_t e;
#define NSA_VARIANT(I, N, X) launch_variant<I, DK, DV, N, X>(c, a, p, po, pml, st)
  if (c.int4)
    e = p.nt == 1 ? (ext ? NSA_VARIANT(true, 1, true) : NSA_VARIANT(true, 1, false))
                  : (ext ? NSA_VARIANT(true, 2, true) : NSA_VARIANT(true, 2, false));
  else
    e = p.nt == 1 ? (ext ? NSA_VARIANT(false, 1, true) : NSA_VARIANT(false, 1, false))
                  : (ext ? NSA_VARIANT(false, 2, true) : NSA_VARIANT(false, 2, false));
#undef NSA_VARIANT
  if (e != cudaSuccess || p.splits == 1) return e;
  const long long rows = (long long)c.batch * c.h_kv * a.n_new * a.G;
  cache_join_kernel<DV><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(c, a, p.chunk, p.splits, p.nt * 8, po, pml);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attn_workspace(const CacheArgs& c, const CacheAttnArgs& a) {
  const Plan p = plan_of(c, a);
  return p.rows ? ((p.rows + 1) / 2 * 2) * sizeof(float2) + p.rows * c.dv * sizeof(float) : 0;
}

bool cache_attn_fits(const CacheArgs& c, const CacheAttnArgs& a) {
  const Plan p = plan_of(c, a);
  return (long long)c.batch * c.h_kv * std::max(p.splits * p.row_tiles, a.n_new * a.G) <= INT32_MAX;
}

cudaError_t launch_cache_attn(const CacheArgs& c, const CacheAttnArgs& a, cudaStream_t st) {
  if (c.dk == 64) return launch_dims<64, 64>(c, a, st);
  if (c.dk == 128) return launch_dims<128, 128>(c, a, st);
  return launch_dims<192, 128>(c, a, st);
}

}  // namespace nsa
