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

// Dims d0 .. d0 + 7 of a head at `head`, rotated by the table row cs (cosines, then sines):
// (a, b) -> (a cos - b sin, b cos + a sin).  Products and sums are rounded one by one (no
// contraction), so that the result is the same wherever it is computed.
__device__ __forceinline__ uint4 rotated_chunk(const __nv_bfloat16* head, int d0, const float* cs, int rot,
                                               int interleaved) {
  const uint4 own = __ldg(reinterpret_cast<const uint4*>(head + d0));
  if (cs == nullptr || d0 >= rot) return own;
  const int half = rot >> 1;
  float x[8], y[8];
  unpack8(own, x);
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(cs + (d0 >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(cs + half + (d0 >> 1)));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], cc[i]), __fmul_rn(x[2 * i + 1], ss[i]));
      y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], cc[i]), __fmul_rn(x[2 * i], ss[i]));
    }
    return pack8(y);
  }
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

// Codes of 8 consecutive values of a row (one 32-bit word, low nibble first) and the group's
// (s, z).  The four lanes of a quad hold the four chunks of one group of 32.
__device__ __forceinline__ uint32_t quantise_chunk(const uint4& u, uint32_t& sz) {
  float x[8];
  unpack8(u, x);
  float lo = x[0], hi = x[0], odd = 0.f;   // odd: NaN as soon as one value is not finite
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    odd = __fmaf_rn(x[i], 0.f, odd);
  }
  const uint32_t quad = 0xfu << (threadIdx.x & 28);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(quad, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(quad, hi, o));
    odd += __shfl_xor_sync(quad, odd, o);
  }
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
    const float c = fminf(fmaxf(__fadd_rn(rintf(__fmul_rn(__fsub_rn(x[i], z), inv)), 8.f), 0.f), 15.f);
    w |= (uint32_t)(int)c << (4 * i);
  }
  sz = pack_bf16(s, z);
  return w;
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
template <int DIM, bool KEY, bool INT4>
__device__ __forceinline__ void put_chunk(const CacheArgs& c, const Row& w, int h, int n, const uint4& u) {
  void* pool = KEY ? c.k : c.v;
  if constexpr (INT4) {
    uint32_t sz;
    const uint32_t codes = quantise_chunk(u, sz);
    const size_t row = ((size_t)w.page * c.h_kv + h) * c.page_size + w.place;
    store_codes<DIM, KEY>(static_cast<uint8_t*>(pool) + row * (DIM / 2), n, codes);
    if ((n & 3) == 0)
      reinterpret_cast<uint32_t*>(KEY ? c.k_scale : c.v_scale)[row * (DIM / 32) + (n >> 2)] = sz;
  } else {
    const size_t row = ((size_t)w.page * c.page_size + w.place) * c.h_kv + h;
    reinterpret_cast<uint4*>(pool)[row * (DIM / 8) + n] = u;
  }
}

// A block's tokens, looked up by its first threads.
constexpr int kThreads = 256, kMaxTokens = 8, kFlight = 4;   // kFlight: rows of a thread in flight
struct Place : Row {
  bool live;   // written (append) or there (read)
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
__global__ void __launch_bounds__(kThreads) append_kernel(const CacheArgs c, const RowsArgs r, const AppendArgs a, int tokens) {
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

  // queries, and keys of a bf16 cache: sixteen values a thread, the same ones of every head, so that a
  // thread loads its angles once a token
  constexpr int kUnits = DK / 16, kSlots = kThreads / kUnits;
  const int u = tid % kUnits, slot = tid / kUnits;
  const int nq = a.q ? a.h_q : 0, heads = nq + (INT4 ? 0 : c.h_kv);
  const bool turned = a.cos_sin != nullptr && u < a.rot / 16;
  // chunks (of 8 values) of the unit
  const int c0 = turned && !a.interleaved ? u : 2 * u, c1 = turned && !a.interleaved ? u + a.rot / 16 : 2 * u + 1;
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
        uint4* dst = h < nq ? qo + h * (DK / 8) : ko + (h - nq) * (DK / 8);
        dst[c0] = lo[f];
        dst[c1] = hi[f];
      }
    }
  }

  // keys of a 4-bit cache and values: a chunk of 8 values a thread, the tokens' chunks end to end
  const int nk = INT4 ? c.h_kv * (DK / 8) : 0, nv = c.h_kv * (DV / 8), per = nk + nv;
  for (int x0 = tid; x0 < n * per; x0 += kFlight * kThreads) {
    uint4 v[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int x = x0 + f * kThreads, tok = x / per, y = x - tok * per;
      if (x >= n * per) break;
      const Place& p = s_place[tok];
      if (!p.live) continue;
      const size_t i = (size_t)i0 + tok;
      if (INT4 && y < nk)
        v[f] = rotated_chunk(static_cast<const __nv_bfloat16*>(a.k) + i * a.k_stride + y / (DK / 8) * DK, y % (DK / 8) * 8,
                             a.cos_sin ? a.cos_sin + (size_t)p.pos * a.rot : nullptr, a.rot, a.interleaved);
      else
        v[f] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) + i * a.v_stride) + (y - nk));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int x = x0 + f * kThreads, tok = x / per, y = x - tok * per;
      if (x >= n * per) break;
      const Place& p = s_place[tok];
      if (!p.live) continue;   // per is a multiple of 4: a quad's threads stay together
      if (INT4 && y < nk) put_chunk<DK, true, INT4>(c, p, y / (DK / 8), y % (DK / 8), v[f]);
      else put_chunk<DV, false, INT4>(c, p, (y - nk) / (DV / 8), (y - nk) % (DV / 8), v[f]);
    }
  }
}

// What a chunk of 8 values is made from: the row itself (bf16), or the codes' word and the group's (s, z).
template <int DIM, bool KEY, bool INT4>
__device__ __forceinline__ uint4 fetch_chunk(const CacheArgs& c, const Row& w, int h, int n) {
  const void* pool = KEY ? c.k : c.v;
  if constexpr (!INT4) {
    const size_t row = ((size_t)w.page * c.page_size + w.place) * c.h_kv + h;
    return __ldg(reinterpret_cast<const uint4*>(pool) + row * (DIM / 8) + n);
  } else {
    const size_t row = ((size_t)w.page * c.h_kv + h) * c.page_size + w.place;
    const uint32_t codes = load_codes<DIM, KEY>(static_cast<const uint8_t*>(pool) + row * (DIM / 2), n);
    const uint32_t* sz = reinterpret_cast<const uint32_t*>(KEY ? c.k_scale : c.v_scale) + row * (DIM / 32) + (n >> 2);
    return make_uint4(codes, __ldg(sz), 0, 0);
  }
}
template <bool INT4>
__device__ __forceinline__ uint4 chunk_value(const uint4& u) {
  if constexpr (!INT4) return u;
  const float s = cache::bf16_lo(u.y), z = cache::bf16_hi(u.y);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __fmaf_rn(s, (float)((int)(u.x >> (4 * j) & 15u) - 8), z);   // s (c - 8) is exact
  return pack8(x);
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
  const int nk = c.h_kv * (DK / 8), nv = c.h_kv * (DV / 8), per = nk + nv;
  for (int x0 = tid; x0 < n * per; x0 += kFlight * kThreads) {
    uint4 u[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int x = x0 + f * kThreads, tok = x / per, y = x - tok * per;
      if (x >= n * per) break;
      const Place& p = s_place[tok];
      if (!p.live) continue;
      u[f] = y < nk ? fetch_chunk<DK, true, INT4>(c, p, y / (DK / 8), y % (DK / 8))
                    : fetch_chunk<DV, false, INT4>(c, p, (y - nk) / (DV / 8), (y - nk) % (DV / 8));
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int x = x0 + f * kThreads, tok = x / per, y = x - tok * per;
      if (x >= n * per) break;
      const Place& p = s_place[tok];
      if (p.seq < 0) continue;
      const size_t i = (size_t)i0 + tok;
      const uint4 o = p.live ? chunk_value<INT4>(u[f]) : make_uint4(0, 0, 0, 0);
      if (y < nk) k_out[i * nk + y] = o;
      else v_out[i * nv + y - nk] = o;
    }
  }
}

// Tokens a block takes: one while there are few of them, more once the blocks fill the GPU.
int tokens_per_block(int rows) { return std::max(1, std::min(kMaxTokens, rows / (148 * 8))); }

template <int DK, int DV>
cudaError_t append_dims(const CacheArgs& c, const RowsArgs& r, const AppendArgs& a, cudaStream_t st) {
  const int n = tokens_per_block(r.rows), grid = (r.rows + n - 1) / n;
  if (c.int4) append_kernel<DK, DV, true><<<grid, kThreads, 0, st>>>(c, r, a, n);
  else append_kernel<DK, DV, false><<<grid, kThreads, 0, st>>>(c, r, a, n);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t read_dims(const CacheArgs& c, const RowsArgs& r, void* k_out, void* v_out, cudaStream_t st) {
  const int n = tokens_per_block(r.rows), grid = (r.rows + n - 1) / n;
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
