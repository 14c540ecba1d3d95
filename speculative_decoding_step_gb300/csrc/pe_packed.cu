// Packing key and value rows into a 4-bit paged cache, and reading entries back.
// The format is in pe_packed.cuh.
#include <algorithm>

#include "pe_internal.h"
#include "pe_packed.cuh"

namespace pe {

namespace {

constexpr int kPackThreads = 256;

template <typename T>
PE_DEV void load16(const T* p, float (&x)[16]);
template <>
PE_DEV void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(p) + k);
    x[4 * k] = t.x; x[4 * k + 1] = t.y; x[4 * k + 2] = t.z; x[4 * k + 3] = t.w;
  }
}
template <>
PE_DEV void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p) + k);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[8 * k + 2 * e] = __uint_as_float(w[e] << 16);
      x[8 * k + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}

// The scale byte of a block whose largest finite magnitude is amax: the smallest c with
// 7 s(c) >= amax.  amax/7, cut to three mantissa bits, is at most two steps short (the rounding
// of 1/7 and of the product, then the cut); 7 s has seven significant bits, so the comparisons
// that find the rest are exact.
PE_DEV uint32_t scale_code(float amax) {
  uint32_t b = __float_as_uint(amax * 0.142857149f) >> 20;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (7.f * __uint_as_float(b << 20) < amax) ++b;
  const int c = (int)b - 108 * 8;
  return (uint32_t)min(max(c, 0), 255);
}

// Rounds a block of 16 entries: nibbles n[e] = code + 8 and the scale byte.  Returns whether
// an entry was NaN (kept as 0) or infinite (kept as +-7 s).
template <typename T>
PE_DEV bool quantise_block(float (&x)[16], uint32_t (&n)[16], uint32_t& code) {
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float m = fabsf(x[e]);
    bad |= !(m < INFINITY);
    amax = m < INFINITY ? fmaxf(amax, m) : amax;
  }
  code = scale_code(amax);
  const float s = packed_scale(code);
  if (bad || amax > 7.f * s) {  // entries beyond the largest scale's range keep its largest code
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = x[e] != x[e] ? 0.f : fminf(fmaxf(x[e], -7.f * s), 7.f * s);
  }
  // round(x / s), halves away from zero, as x times the float above 1/s plus 1.5 * 2^23 + 8 in one
  // fused operation: the sum's low mantissa bits are the nibble.  The factor is at most two
  // rounding steps above 1/s, so an exact half goes away from zero; a bf16 x over a scale of
  // four bits is never nearer to a half than 2^-10 without being one.
  const float inv = __uint_as_float(__float_as_uint(1.f / s) + 1);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    n[e] = __float_as_uint(fmaf(x[e], inv, 12582920.f)) & 15u;
    if (sizeof(T) == 4) {
      // fp32 entries can be nearer to a half than that: the halves themselves decide (exact
      // products of four-bit numbers)
      const float m = fabsf(x[e]), c = fabsf((float)((int)n[e] - 8));
      const int off = m < (c - 0.5f) * s ? -1 : m >= (c + 0.5f) * s ? 1 : 0;
      n[e] += x[e] < 0.f ? -off : off;
    }
  }
  return bad;
}

// One thread per (row, head, block of 16); blockIdx.y: keys or values.  The four threads of 64
// entries exchange nibbles so that each stores whole words of the row.
template <typename T, int HD>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a) {
  using L = PackedLayout<HD>;
  constexpr int NB = HD / 16;  // blocks per head row
  pdl_wait();
  pdl_trigger();
  const bool is_v = blockIdx.y != 0;
  const int n_rows = a.n_dev != nullptr ? min(max(__ldcg(a.n_dev), 0), a.n_rows) : a.n_rows;
  const long long per_row = (long long)a.n_kv * NB;
  const long long idx = (long long)blockIdx.x * kPackThreads + threadIdx.x;
  const bool live = idx < n_rows * per_row;  // the same for the four threads of 64 entries
  const long long row = live ? idx / per_row : 0;
  const int rest = live ? (int)(idx - row * per_row) : 0;
  const int head = rest / NB, j = rest - (rest / NB) * NB;
  const int q = threadIdx.x & 3;  // = j & 3
  long long slot = -1;
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.f;
  if (live) {
    slot = __ldcg(reinterpret_cast<const long long*>(a.slots) + row);
    if (slot < -1 || slot >= (long long)a.num_pages * kPackedPage) {
      set_err(a.err, PE_DEV_BAD_PAGE);
      slot = -1;
    }
    if (slot >= 0) {
      const T* src = static_cast<const T*>(is_v ? a.v : a.k) + row * (is_v ? a.v_stride : a.k_stride) + head * HD + j * 16;
      load16<T>(src, x);
    }
  }
  uint32_t n[16], code;
  if (quantise_block<T>(x, n, code)) set_err(a.err, PE_DEV_NONFINITE);
  const long long page = slot >= 0 ? slot / kPackedPage : 0;
  const int off = slot >= 0 ? (int)(slot % kPackedPage) : 0;
  uint8_t* rec = a.pool + ((size_t)page * a.n_kv + head) * L::kRecord;
  if (!is_v) {
    // word (t, u): entries 4t..4t+3 of blocks 2u and 2u+1, a byte of each half from either block
    uint32_t w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      w[t] = (n[4 * t] | n[4 * t + 2] << 4 | n[4 * t + 1] << 16 | n[4 * t + 3] << 20) << (8 * (q & 1));
    const bool hi = q & 1;  // the even block's thread keeps t = 0, 1 and the odd one's t = 2, 3
    uint32_t o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t give = hi ? w[k] : w[2 + k];
      o[k] = (hi ? w[2 + k] : w[k]) | __shfl_xor_sync(0xFFFFFFFFu, give, 1);
    }
    if (slot >= 0) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(rec + L::kK + off * L::kRow);
#pragma unroll
      for (int k = 0; k < 2; ++k) dst[((hi ? 2 : 0) + k) * (HD / 32) + (j >> 1)] = o[k];
      rec[L::kKs + off * L::kScaleRow + j] = (uint8_t)code;
    }
  } else {
    // word (g, h): a byte from each of the four blocks of 64 entries (entries g and g + 8 of the block)
    uint32_t w[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) w[g] = (n[g] | n[g + 8] << 4) << (8 * q);
    const bool b0 = q & 1, b1 = q & 2;
    uint32_t m[4], o[2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t give = b0 ? w[k] : w[4 + k];
      m[k] = (b0 ? w[4 + k] : w[k]) | __shfl_xor_sync(0xFFFFFFFFu, give, 1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t give = b1 ? m[k] : m[2 + k];
      o[k] = (b1 ? m[2 + k] : m[k]) | __shfl_xor_sync(0xFFFFFFFFu, give, 2);
    }
    if (slot >= 0) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(rec + L::kV + off * L::kRow);
      const int g0 = (b0 ? 4 : 0) + (b1 ? 2 : 0);
#pragma unroll
      for (int k = 0; k < 2; ++k) dst[(g0 + k) * (HD / 64) + (j >> 2)] = o[k];
      rec[L::kVs + off * L::kScaleRow + j] = (uint8_t)code;
    }
  }
}

template <typename T>
PE_DEV void store8(T* p, const float (&x)[8]);
template <>
PE_DEV void store8<float>(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
PE_DEV void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread per (row, head, eight entries); blockIdx.y: keys or values.
template <typename T, int HD>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const UnpackArgs a) {
  using L = PackedLayout<HD>;
  constexpr int NE = HD / 8;
  pdl_wait();
  pdl_trigger();
  const bool is_v = blockIdx.y != 0;
  const long long per_row = (long long)a.n_kv * NE;
  const long long idx = (long long)blockIdx.x * kPackThreads + threadIdx.x;
  if (idx >= a.n_rows * per_row) return;
  const long long row = idx / per_row;
  const int rest = (int)(idx - row * per_row);
  const int head = rest / NE, e8 = rest - (rest / NE) * NE;
  const long long slot = __ldcg(reinterpret_cast<const long long*>(a.slots) + row);
  if (slot < 0 || slot >= (long long)a.num_pages * kPackedPage) {
    if (slot != -1) set_err(a.err, PE_DEV_BAD_PAGE);
    return;
  }
  const int off = (int)(slot % kPackedPage);
  const uint8_t* rec = a.pool + ((size_t)(slot / kPackedPage) * a.n_kv + head) * L::kRecord;
  const int j = e8 >> 1, h8 = e8 & 1;  // block, and which half of it
  float x[8];
  if (!is_v) {
    const float s = packed_scale(__ldcg(rec + L::kKs + off * L::kScaleRow + j));
    const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + L::kK + off * L::kRow);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w = __ldcg(src + (2 * h8 + k) * (HD / 32) + (j >> 1)) >> (8 * (j & 1));
      x[4 * k] = s * (float)((int)(w & 15u) - 8);
      x[4 * k + 1] = s * (float)((int)((w >> 16) & 15u) - 8);
      x[4 * k + 2] = s * (float)((int)((w >> 4) & 15u) - 8);
      x[4 * k + 3] = s * (float)((int)((w >> 20) & 15u) - 8);
    }
  } else {
    const float s = packed_scale(__ldcg(rec + L::kVs + off * L::kScaleRow + j));
    const uint32_t* src = reinterpret_cast<const uint32_t*>(rec + L::kV + off * L::kRow);
    const int sh = 8 * (j & 3) + 4 * h8;
#pragma unroll
    for (int g = 0; g < 8; ++g)
      x[g] = s * (float)((int)((__ldcg(src + g * (HD / 64) + (j >> 2)) >> sh) & 15u) - 8);
  }
  T* dst = static_cast<T*>(is_v ? a.v_out : a.k_out) + row * (is_v ? a.v_stride : a.k_stride) + head * HD + e8 * 8;
  store8<T>(dst, x);
}

template <typename T, int HD>
cudaError_t pack_typed(const PackArgs& a, cudaStream_t s) {
  const long long n = (long long)a.n_rows * a.n_kv * (HD / 16);
  return launch_pdl(pack_kernel<T, HD>, dim3((unsigned)((n + kPackThreads - 1) / kPackThreads), 2), dim3(kPackThreads),
                    0, s, a);
}
template <typename T, int HD>
cudaError_t unpack_typed(const UnpackArgs& a, cudaStream_t s) {
  const long long n = (long long)a.n_rows * a.n_kv * (HD / 8);
  return launch_pdl(unpack_kernel<T, HD>, dim3((unsigned)((n + kPackThreads - 1) / kPackThreads), 2),
                    dim3(kPackThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_pack(const PackArgs& a, pe_dtype dt, cudaStream_t s) {
  if (a.n_rows == 0) return cudaSuccess;
  if (a.head_dim == 64)
    return dt == PE_BF16 ? pack_typed<__nv_bfloat16, 64>(a, s) : pack_typed<float, 64>(a, s);
  return dt == PE_BF16 ? pack_typed<__nv_bfloat16, 128>(a, s) : pack_typed<float, 128>(a, s);
}

cudaError_t launch_unpack(const UnpackArgs& a, pe_dtype dt, cudaStream_t s) {
  if (a.n_rows == 0) return cudaSuccess;
  if (a.head_dim == 64)
    return dt == PE_BF16 ? unpack_typed<__nv_bfloat16, 64>(a, s) : unpack_typed<float, 64>(a, s);
  return dt == PE_BF16 ? unpack_typed<__nv_bfloat16, 128>(a, s) : unpack_typed<float, 128>(a, s);
}

}  // namespace pe
