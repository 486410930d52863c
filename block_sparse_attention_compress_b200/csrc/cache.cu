// Writing new tokens into a paged cache (keys rotated on the way, 4-bit codes formed from the
// rounded rows) and reading rows back.  Both move every byte once and compute little: HBM bounds
// a prompt, the launch and a chain of dependent loads (length, page, angles) a single token.  A
// block takes several tokens of a prompt: their places are looked up side by side, and every thread has
// several rows' loads in flight.
#include <algorithm>

#include "cache.cuh"

namespace nsa {
namespace {

using cache::Row;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = cache::bf16_lo(w[i]);
    x[2 * i + 1] = cache::bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// Dims d0 .. d0 + 7 of a head at `head`, the pairs (j, j + rot / 2) rotated by the table row cs (cosines,
// then sines): (a, b) -> (a cos - b sin, b cos + a sin).  Products and sums are rounded one by one (no
// contraction), so that the result is the same wherever it is computed.
__device__ __forceinline__ uint4 rotated_chunk(const __nv_bfloat16* head, int d0, const float* cs, int rot) {
  const uint4 own = __ldg(reinterpret_cast<const uint4*>(head + d0));
  if (d0 >= rot) return own;
  const int half = rot >> 1;
  float x[8], y[8];
  unpack8(own, x);
  const bool first = d0 < half;   // which member of its pairs this chunk holds
  const int j = first ? d0 : d0 - half;
  float o[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>(head + (first ? d0 + half : d0 - half))), o);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + j + 4 * h));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + j + 4 * h));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xc = __fmul_rn(x[4 * h + i], cc[i]), os = __fmul_rn(o[4 * h + i], ss[i]);
      y[4 * h + i] = first ? __fsub_rn(xc, os) : __fadd_rn(xc, os);
    }
  }
  return pack8(y);
}

// Least and largest of 8 values, and NaN as soon as one of them is not finite.
struct Range {
  float lo, hi, odd;
};
__device__ __forceinline__ Range range_of(const float (&x)[8]) {
  Range r{x[0], x[0], 0.f};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.lo = fminf(r.lo, x[i]);
    r.hi = fmaxf(r.hi, x[i]);
    r.odd = __fmaf_rn(x[i], 0.f, r.odd);
  }
  return r;
}
__device__ __forceinline__ Range both(const Range& a, const Range& b) {
  return Range{fminf(a.lo, b.lo), fmaxf(a.hi, b.hi), a.odd + b.odd};
}
__device__ __forceinline__ Range across(const Range& r, int lanes, uint32_t mask) {
  return both(r, Range{__shfl_xor_sync(mask, r.lo, lanes), __shfl_xor_sync(mask, r.hi, lanes), __shfl_xor_sync(mask, r.odd, lanes)});
}

// Codes of 8 consecutive values of a row (one 32-bit word, low nibble first) and the (s, z) of their
// group, whose range is r.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], const Range& r, uint32_t& sz) {
  const float lo = r.lo, hi = r.hi, odd = r.odd;
  const float span = __fsub_rn(hi, lo);
  if (!(span < INFINITY) || odd != 0.f || isnan(odd)) {
    sz = 0x7fc07fc0u;
    return 0x88888888u;
  }
  // 1/15 as a product: the definition's own rounding
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(span, 1.f / 15.f)));
  if (s < 0x1p-100f) s = 0.f;
  const float z = __bfloat162float(__float2bfloat16_rn(__fmaf_rn(8.f, s, lo)));
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // in [-8, 7] and on top of 1.5 * 2^23 the sum's rounding (nearest, even) is the integer's
    const float c = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], z), inv), -8.f), 7.f);
    w |= (__float_as_uint(__fadd_rn(c, 12582920.f)) & 15u) << (4 * i);
  }
  sz = pack_bf16(s, z);
  return w;
}
// The same where the four lanes of a quad hold the four chunks of one group of 32.
__device__ __forceinline__ uint32_t quantise_chunk(const uint4& u, uint32_t& sz) {
  float x[8];
  unpack8(u, x);
  const uint32_t quad = 0xfu << (threadIdx.x & 28);
  return codes_of(x, across(across(range_of(x), 1, quad), 2, quad), sz);
}

// Stores the word of values 8 n .. 8 n + 7 of a row of DIM values at its place in the stored order.
template <int DIM, bool KEY>
__device__ __forceinline__ void store_codes(uint8_t* row, int n, uint32_t w) {
  constexpr int kGroups = DIM / 32;
  if constexpr (KEY) {
    reinterpret_cast<uint32_t*>(row)[(n & 3) * kGroups + (n >> 2)] = w;
  } else {   // halves 2 n and 2 n + 1: half 8 g + i goes to i * groups + g
    uint16_t* h = reinterpret_cast<uint16_t*>(row);
    const int g = n >> 2, i = (2 * n) & 7;
    h[i * kGroups + g] = (uint16_t)w;
    h[(i + 1) * kGroups + g] = (uint16_t)(w >> 16);
  }
}
template <int DIM, bool KEY>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* row, int n) {
  constexpr int kGroups = DIM / 32;
  if constexpr (KEY) {
    return __ldg(reinterpret_cast<const uint32_t*>(row) + (n & 3) * kGroups + (n >> 2));
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
    const int g = n >> 2, i = (2 * n) & 7;
    return __ldg(h + i * kGroups + g) | (uint32_t)__ldg(h + (i + 1) * kGroups + g) << 16;
  }
}

// One chunk (8 values) of a new key or value row into the cache.
template <int DIM, bool KEY>
__device__ __forceinline__ void put_codes(const CacheArgs& c, const Row& w, int h, int n, uint32_t codes, uint32_t sz) {
  const size_t row = ((size_t)w.page * c.h_kv + h) * c.page_size + w.place;
  store_codes<DIM, KEY>(static_cast<uint8_t*>(KEY ? c.k : c.v) + row * (DIM / 2), n, codes);
  if ((n & 3) == 0) reinterpret_cast<uint32_t*>(KEY ? c.k_scale : c.v_scale)[row * (DIM / 32) + (n >> 2)] = sz;
}
template <int DIM, bool KEY, bool INT4>
__device__ __forceinline__ void put_chunk(const CacheArgs& c, const Row& w, int h, int n, const uint4& u) {
  void* pool = KEY ? c.k : c.v;
  if constexpr (INT4) {
    uint32_t sz;
    const uint32_t codes = quantise_chunk(u, sz);
    put_codes<DIM, KEY>(c, w, h, n, codes, sz);
  } else {
    const size_t row = ((size_t)w.page * c.page_size + w.place) * c.h_kv + h;
    reinterpret_cast<uint4*>(pool)[row * (DIM / 8) + n] = u;
  }
}

// A block's tokens, looked up by its first threads.
// kFlight: heads (kReadFlight: units of 16 values) a thread has in flight.  Append with 2 at 4 blocks an SM
// moves 64K tokens of (64, 4) heads in 625 us (3.44 GB, 5.5 TB/s), with 2 at 3 blocks in 739, with 4 in 817 (its rows
// spill), with 1 in 746; read with 2 gives back 128K tokens of 4 heads in 88 us, with 1 in 90, with 4 in 98.
constexpr int kThreads = 256, kMaxTokens = 16, kFlight = 2, kReadFlight = 2;
struct Place : Row {
  bool live;   // written (append) or there (read)
};

// The chunks (of 8 or 16 values) of a block's tokens, `per` each, end to end: a thread's own ones, kThreads apart.
struct Chunks {
  int tok, y, dtok, dy;
  __device__ __forceinline__ Chunks(int tid, int per) : tok(tid / per), y(tid % per), dtok(kThreads / per), dy(kThreads % per) {}
  __device__ __forceinline__ void next(int per) {
    tok += dtok;
    y += dy;
    if (y >= per) {
      y -= per;
      ++tok;
    }
  }
};

// Sixteen values of a head, in two chunks of 8: the pairs of angles 8 u .. 8 u + 7.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void turn(uint4& lo, uint4& hi, const Angles& t, bool interleaved) {
  float a[8], b[8], x[8], y[8];
  unpack8(lo, a);
  unpack8(hi, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // interleaved: pair i is (2 i, 2 i + 1) of the sixteen
    const float p = interleaved ? (i < 4 ? a[2 * i % 8] : b[2 * i % 8]) : a[i];
    const float q = interleaved ? (i < 4 ? a[2 * i % 8 + 1] : b[2 * i % 8 + 1]) : b[i];
    x[i] = __fsub_rn(__fmul_rn(p, t.c[i]), __fmul_rn(q, t.s[i]));
    y[i] = __fadd_rn(__fmul_rn(q, t.c[i]), __fmul_rn(p, t.s[i]));
  }
  if (interleaved) {
    lo = make_uint4(pack_bf16(x[0], y[0]), pack_bf16(x[1], y[1]), pack_bf16(x[2], y[2]), pack_bf16(x[3], y[3]));
    hi = make_uint4(pack_bf16(x[4], y[4]), pack_bf16(x[5], y[5]), pack_bf16(x[6], y[6]), pack_bf16(x[7], y[7]));
  } else {
    lo = pack8(x);
    hi = pack8(y);
  }
}

template <int DK, int DV, bool INT4>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const CacheArgs c, const RowsArgs r, const AppendArgs a, int tokens) {
  __shared__ Place s_place[kMaxTokens];
  const int i0 = blockIdx.x * tokens, n = min(tokens, r.rows - i0), tid = threadIdx.x;
  if (tid < n) {
    Place p;
    static_cast<Row&>(p) = cache::find_row(c, r, i0 + tid);
    p.live = p.pos >= 0 && p.page >= 0 && (a.cos_sin == nullptr || p.pos < a.n_positions);
    if (p.pos >= 0 && !p.live) cache::report(c.status);
    s_place[tid] = p;
  }
  __syncthreads();

  // queries and keys: sixteen values a thread, the same ones of every head, so that a thread loads its
  // angles once a token.  4 bits: the chunks of a group of 32 are then those of a quad of threads (pairs (j, j + rot / 2),
  // rot a multiple of 64) or both chunks of two threads (interleaved pairs); other rotations take the
  // keys chunk by chunk below.
  constexpr int kUnits = DK / 16, kSlots = kThreads / kUnits;
  const int u = tid % kUnits, slot = tid / kUnits;
  const int rot = a.cos_sin ? a.rot : 0, nq = a.q ? a.h_q : 0;
  const bool by_chunk = INT4 && !a.interleaved && rot % 64;
  const int heads = nq + (by_chunk ? 0 : c.h_kv);
  const bool turned = u < rot / 16;
  // chunks (of 8 values) of the unit
  const int c0 = a.interleaved ? 2 * u : turned ? u : rot / 16 + u;
  const int c1 = a.interleaved ? 2 * u + 1 : turned ? u + rot / 16 : u + DK / 16;
  for (int x = 0; x < n && slot < kSlots; ++x) {
    const Place p = s_place[x];
    if (p.seq < 0) continue;
    const size_t i = (size_t)i0 + x;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + i * a.q_stride);
    const uint4* k = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.k) + i * a.k_stride);
    uint4* qo = static_cast<uint4*>(a.q_out) + i * nq * (DK / 8);
    uint4* ko = static_cast<uint4*>(c.k) + (INT4 || !p.live ? 0 : ((size_t)p.page * c.page_size + p.place) * c.h_kv * (DK / 8));
    Angles t;
    if (turned && p.live) {
      const float4* cs = reinterpret_cast<const float4*>(a.cos_sin + (size_t)p.pos * a.rot + 8 * u);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        reinterpret_cast<float4*>(t.c)[e] = __ldg(cs + e);
        reinterpret_cast<float4*>(t.s)[e] = __ldg(cs + a.rot / 8 + e);
      }
    }
    const int end = p.live ? heads : nq;
    for (int h0 = slot; h0 < end; h0 += kFlight * kSlots) {
      uint4 lo[kFlight], hi[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int h = h0 + f * kSlots;
        if (h >= end) break;
        const uint4* src = h < nq ? q + h * (DK / 8) : k + (h - nq) * (DK / 8);
        lo[f] = p.live ? __ldg(src + c0) : make_uint4(0, 0, 0, 0);
        hi[f] = p.live ? __ldg(src + c1) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int h = h0 + f * kSlots;
        if (h >= end) break;
        if (turned && p.live) turn(lo[f], hi[f], t, a.interleaved);
        if (INT4 && h >= nq) {
          float x[2][8];
          unpack8(lo[f], x[0]);
          unpack8(hi[f], x[1]);
          Range g[2] = {range_of(x[0]), range_of(x[1])};
          const uint32_t quad = 0xfu << (tid & 28);   // all of a head
          if (a.interleaved) {
            g[0] = g[1] = across(both(g[0], g[1]), 1, quad);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) g[e] = across(across(g[e], 1, quad), 2, quad);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t sz;
            const uint32_t codes = codes_of(x[e], g[e], sz);
            put_codes<DK, true>(c, p, h - nq, e ? c1 : c0, codes, sz);
          }
          continue;
        }
        uint4* dst = h < nq ? qo + h * (DK / 8) : ko + (h - nq) * (DK / 8);
        dst[c0] = lo[f];
        dst[c1] = hi[f];
      }
    }
  }

  // values (and keys by chunks): a chunk of 8 values a thread, the tokens' chunks end to end
  const int nk = by_chunk ? c.h_kv * (DK / 8) : 0, nv = c.h_kv * (DV / 8), per = nk + nv;
  Chunks at(tid, per);
  for (int x0 = tid; x0 < n * per; x0 += kFlight * kThreads) {
    uint4 v[kFlight];
    int tok[kFlight], y[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      tok[f] = at.tok;
      y[f] = at.y;
      at.next(per);
      if (tok[f] >= n || !s_place[tok[f]].live) continue;
      const size_t i = (size_t)i0 + tok[f];
      if (INT4 && y[f] < nk)
        v[f] = rotated_chunk(static_cast<const __nv_bfloat16*>(a.k) + i * a.k_stride + y[f] / (DK / 8) * DK, y[f] % (DK / 8) * 8,
                             a.cos_sin + (size_t)s_place[tok[f]].pos * rot, rot);   // by_chunk: there is a table
      else
        v[f] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + i * a.v_stride) + (y[f] - nk));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (tok[f] >= n || !s_place[tok[f]].live) continue;   // per is a multiple of 4: a quad's threads stay together
      const int z = y[f] - nk;
      if (INT4 && z < 0) put_chunk<DK, true, INT4>(c, s_place[tok[f]], y[f] / (DK / 8), y[f] % (DK / 8), v[f]);
      else put_chunk<DV, false, INT4>(c, s_place[tok[f]], z / (DV / 8), z % (DV / 8), v[f]);
    }
  }
}

// Sixteen values of a row, chunks u and u + DIM / 16 (the threads of a warp then read and write 16 bytes next to
// one another): the row itself (bf16), or two words of codes and their groups' (s, z).
struct Sixteen {
  uint4 a, b;
};
template <int DIM, bool KEY, bool INT4>
__device__ __forceinline__ Sixteen fetch(const CacheArgs& c, const Row& w, int h, int u) {
  const void* pool = KEY ? c.k : c.v;
  Sixteen r;
  if constexpr (!INT4) {
    const size_t row = ((size_t)w.page * c.page_size + w.place) * c.h_kv + h;
    const uint4* src = reinterpret_cast<const uint4*>(pool) + row * (DIM / 8) + u;
    r.a = __ldg(src);
    r.b = __ldg(src + DIM / 16);
  } else {
    const size_t row = ((size_t)w.page * c.h_kv + h) * c.page_size + w.place;
    const uint8_t* src = static_cast<const uint8_t*>(pool) + row * (DIM / 2);
    const uint32_t* sz = reinterpret_cast<const uint32_t*>(KEY ? c.k_scale : c.v_scale) + row * (DIM / 32);
    r.a.x = load_codes<DIM, KEY>(src, u);
    r.a.y = load_codes<DIM, KEY>(src, u + DIM / 16);
    r.a.z = __ldg(sz + (u >> 2));
    r.a.w = __ldg(sz + ((u + DIM / 16) >> 2));
  }
  return r;
}
// The values of a word of codes.  128 + c is a bf16 with c as its last bits; less 136, times s, plus z in one
// fma: the value rounded once.
__device__ __forceinline__ uint4 values_of(uint32_t w, uint32_t sz) {
  const __nv_bfloat162 pair = *reinterpret_cast<const __nv_bfloat162*>(&sz);
  const __nv_bfloat162 s = __low2bfloat162(pair), z = __high2bfloat162(pair);
  uint32_t v[4];   // values j and j + 4
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u, o = 0x43084308u;
    const __nv_bfloat162 c = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&o));
    const __nv_bfloat162 y = __hfma2(s, c, z);
    v[j] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                    __byte_perm(v[2], v[3], 0x7632));
}

template <int DK, int DV, bool INT4>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheArgs c, const RowsArgs r, uint4* __restrict__ k_out,
                                                        uint4* __restrict__ v_out, int tokens) {
  __shared__ Place s_place[kMaxTokens];
  const int i0 = blockIdx.x * tokens, n = min(tokens, r.rows - i0), tid = threadIdx.x;
  if (tid < n) {
    Place p;
    static_cast<Row&>(p) = cache::find_row(c, r, i0 + tid);
    p.live = p.page >= 0;
    if (p.pos >= 0 && !p.live) cache::report(c.status);
    s_place[tid] = p;
  }
  __syncthreads();
  const int nk = c.h_kv * (DK / 16), nv = c.h_kv * (DV / 16), per = nk + nv;
  Chunks at(tid, per);
  for (int x0 = tid; x0 < n * per; x0 += kReadFlight * kThreads) {
    Sixteen v[kReadFlight];
    int tok[kReadFlight], y[kReadFlight];
#pragma unroll
    for (int f = 0; f < kReadFlight; ++f) {
      tok[f] = at.tok;
      y[f] = at.y;
      at.next(per);
      if (tok[f] >= n || !s_place[tok[f]].live) continue;
      const int z = y[f] - nk;
      v[f] = z < 0 ? fetch<DK, true, INT4>(c, s_place[tok[f]], y[f] / (DK / 16), y[f] % (DK / 16))
                   : fetch<DV, false, INT4>(c, s_place[tok[f]], z / (DV / 16), z % (DV / 16));
    }
#pragma unroll
    for (int f = 0; f < kReadFlight; ++f) {
      if (tok[f] >= n || s_place[tok[f]].seq < 0) continue;
      const size_t i = (size_t)i0 + tok[f];
      const int z = y[f] - nk;
      uint4* dst = z < 0 ? k_out + 2 * i * nk + y[f] / (DK / 16) * (DK / 8) + y[f] % (DK / 16)
                         : v_out + 2 * i * nv + z / (DV / 16) * (DV / 8) + z % (DV / 16);
      if (!s_place[tok[f]].live) v[f].a = v[f].b = make_uint4(0, 0, 0, 0);
      else if (INT4) v[f] = Sixteen{values_of(v[f].a.x, v[f].a.z), values_of(v[f].a.y, v[f].a.w)};
      dst[0] = v[f].a;
      dst[z < 0 ? DK / 16 : DV / 16] = v[f].b;
    }
  }
}

// Tokens a block takes: one while there are few of them, up to `most` once the blocks fill the GPU.
int tokens_per_block(int rows, int most) { return std::max(1, std::min(most, rows / (148 * 8))); }

template <int DK, int DV>
cudaError_t append_dims(const CacheArgs& c, const RowsArgs& r, const AppendArgs& a, cudaStream_t st) {
  // eight; fewer with many heads of values, so that a block is not long in one phase (8K tokens of 32 heads in bf16: 78 us with four, 82 with eight; 64K of 4 in 4 bits: 637 with four, 625 with eight)
  const int n = tokens_per_block(r.rows, std::min(8, 2048 / (c.h_kv * DV / 8))), grid = (r.rows + n - 1) / n;
  if (c.int4) append_kernel<DK, DV, true><<<grid, kThreads, 0, st>>>(c, r, a, n);
  else append_kernel<DK, DV, false><<<grid, kThreads, 0, st>>>(c, r, a, n);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t read_dims(const CacheArgs& c, const RowsArgs& r, void* k_out, void* v_out, cudaStream_t st) {
  // about four units a thread: 12 tokens of 4 heads (128K of them 88 us; 6 tokens 96), 2 of 32 (16K: 64; 8 tokens 70)
  const int n = tokens_per_block(r.rows, std::min(kMaxTokens, 1024 / (c.h_kv * (DK + DV) / 16))), grid = (r.rows + n - 1) / n;
  uint4 *k = static_cast<uint4*>(k_out), *v = static_cast<uint4*>(v_out);
  if (c.int4) read_kernel<DK, DV, true><<<grid, kThreads, 0, st>>>(c, r, k, v, n);
  else read_kernel<DK, DV, false><<<grid, kThreads, 0, st>>>(c, r, k, v, n);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& c, const RowsArgs& r, const AppendArgs& a, cudaStream_t st) {
  if (c.dk == 64) return append_dims<64, 64>(c, r, a, st);
  if (c.dk == 128) return append_dims<128, 128>(c, r, a, st);
  return append_dims<192, 128>(c, r, a, st);
}

cudaError_t launch_cache_read(const CacheArgs& c, const RowsArgs& r, void* k_out, void* v_out, cudaStream_t st) {
  if (c.dk == 64) return read_dims<64, 64>(c, r, k_out, v_out, st);
  if (c.dk == 128) return read_dims<128, 128>(c, r, k_out, v_out, st);
  return read_dims<192, 128>(c, r, k_out, v_out, st);
}

}  // namespace nsa
