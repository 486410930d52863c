// Writing new tokens into a paged cache (keys rotated on the way, 4-bit codes formed from the
// rounded rows) and reading rows back.  Both move every byte once and compute little: HBM bounds
// a prompt, the launch a single token.
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
template <int DIM, bool KEY>
__device__ __forceinline__ void put_chunk(const CacheArgs& c, const Row& w, int h, int n, const uint4& u) {
  void* pool = KEY ? c.k : c.v;
  if (c.int4) {
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

// One block per token; its threads walk the token's chunks of 8 values: keys, values, queries.
template <int DK, int DV>
__global__ void append_kernel(const CacheArgs c, const RowsArgs r, const AppendArgs a) {
  const int i = blockIdx.x;
  const Row w = cache::find_row(c, r, i);
  if (w.seq < 0) return;
  const bool in_table = a.cos_sin == nullptr || w.pos < a.n_positions;
  const bool live = w.pos >= 0 && w.page >= 0 && in_table;
  if (w.pos >= 0 && !live && threadIdx.x == 0) cache::report(c.status);
  const float* cs = a.cos_sin && live ? a.cos_sin + (size_t)w.pos * a.rot : nullptr;
  const int nk = c.h_kv * (DK / 8), nv = c.h_kv * (DV / 8), nq = a.q ? a.h_q * (DK / 8) : 0;
  const auto* kr = static_cast<const __nv_bfloat16*>(a.k) + (size_t)i * a.k_stride;
  const auto* vr = static_cast<const __nv_bfloat16*>(a.v) + (size_t)i * a.v_stride;
  const auto* qr = static_cast<const __nv_bfloat16*>(a.q) + (size_t)i * a.q_stride;
  for (int t = live ? threadIdx.x : nk + nv + threadIdx.x; t < nk + nv + nq; t += blockDim.x) {
    if (t < nk) {
      const int h = t / (DK / 8), n = t % (DK / 8);
      put_chunk<DK, true>(c, w, h, n, rotated_chunk(kr + h * DK, 8 * n, cs, a.rot, a.interleaved));
    } else if (t < nk + nv) {
      const int h = (t - nk) / (DV / 8), n = (t - nk) % (DV / 8);
      put_chunk<DV, false>(c, w, h, n, __ldg(reinterpret_cast<const uint4*>(vr + h * DV) + n));
    } else {
      const int x = t - nk - nv, h = x / (DK / 8), n = x % (DK / 8);
      const uint4 u = live ? rotated_chunk(qr + (size_t)h * DK, 8 * n, cs, a.rot, a.interleaved) : make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(a.q_out)[(size_t)i * nq + x] = u;
    }
  }
}

template <int DIM, bool KEY>
__device__ __forceinline__ uint4 get_chunk(const CacheArgs& c, const Row& w, int h, int n) {
  const void* pool = KEY ? c.k : c.v;
  if (!c.int4) {
    const size_t row = ((size_t)w.page * c.page_size + w.place) * c.h_kv + h;
    return __ldg(reinterpret_cast<const uint4*>(pool) + row * (DIM / 8) + n);
  }
  const size_t row = ((size_t)w.page * c.h_kv + h) * c.page_size + w.place;
  const uint32_t codes = load_codes<DIM, KEY>(static_cast<const uint8_t*>(pool) + row * (DIM / 2), n);
  const uint32_t sz =
      __ldg(reinterpret_cast<const uint32_t*>(KEY ? c.k_scale : c.v_scale) + row * (DIM / 32) + (n >> 2));
  const float s = cache::bf16_lo(sz), z = cache::bf16_hi(sz);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = __fmaf_rn(s, (float)((int)(codes >> (4 * j) & 15u) - 8), z);   // s (c - 8) is exact
  return pack8(x);
}

template <int DK, int DV>
__global__ void read_kernel(const CacheArgs c, const RowsArgs r, uint4* __restrict__ k_out, uint4* __restrict__ v_out) {
  const int i = blockIdx.x;
  const Row w = cache::find_row(c, r, i);
  if (w.seq < 0) return;
  if (w.pos >= 0 && w.page < 0 && threadIdx.x == 0) cache::report(c.status);
  const int nk = c.h_kv * (DK / 8), nv = c.h_kv * (DV / 8);
  for (int t = threadIdx.x; t < nk + nv; t += blockDim.x) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (t < nk) {
      if (w.page >= 0) u = get_chunk<DK, true>(c, w, t / (DK / 8), t % (DK / 8));
      k_out[(size_t)i * nk + t] = u;
    } else {
      if (w.page >= 0) u = get_chunk<DV, false>(c, w, (t - nk) / (DV / 8), (t - nk) % (DV / 8));
      v_out[(size_t)i * nv + t - nk] = u;
    }
  }
}

template <int DK, int DV>
cudaError_t append_dims(const CacheArgs& c, const RowsArgs& r, const AppendArgs& a, cudaStream_t st) {
  append_kernel<DK, DV><<<r.rows, 256, 0, st>>>(c, r, a);
  return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t read_dims(const CacheArgs& c, const RowsArgs& r, void* k_out, void* v_out, cudaStream_t st) {
  read_kernel<DK, DV><<<r.rows, 256, 0, st>>>(c, r, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out));
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
