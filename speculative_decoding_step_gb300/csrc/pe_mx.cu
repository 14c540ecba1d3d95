// Microscaled (MX) 4-bit matrices: rounding rows and reading them back.  The format is in pe_mx.cuh.
#include <cuda_fp16.h>

#include <algorithm>

#include "pe_internal.h"
#include "pe_mx.cuh"

namespace pe {

namespace {

constexpr int kMxThreads = 256;

// 32 entries of a row from p on, the ones from `left` on as zeros.  VEC: 16-byte loads (p aligned, all 32 there).
template <typename T>
PE_DEV void load32(const T* p, int left, bool vec, float (&x)[32]);
template <>
PE_DEV void load32<float>(const float* p, int left, bool vec, float (&x)[32]) {
  if (vec && left >= 32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = t.x; x[4 * i + 1] = t.y; x[4 * i + 2] = t.z; x[4 * i + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i < left ? __ldcg(p + i) : 0.f;
  }
}
template <>
PE_DEV void load32<__nv_bfloat16>(const __nv_bfloat16* p, int left, bool vec, float (&x)[32]) {
  if (vec && left >= 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p) + i);
      const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[8 * i + 2 * e] = __uint_as_float(w[e] << 16);
        x[8 * i + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = i < left ? to_float<__nv_bfloat16>(p[i]) : 0.f;
  }
}

// Rounds a block: its codes and its scale byte.  The scale is 2^(floor(log2 amax) - 2): the exponent field of amax less
// two.  Returns whether an entry was NaN (kept as 0) or infinite (kept as +-6 of the scale of the finite ones).
PE_DEV bool mx_round(float (&x)[32], uint4& codes, uint32_t& scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  const bool bad = top >= 0x7F800000u;
  if (bad) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t m = __float_as_uint(x[i]) & 0x7FFFFFFFu;
      if (m < 0x7F800000u) top = max(top, m);
      if (m > 0x7F800000u) x[i] = 0.f;
    }
  }
  // fields 0..2 (below 2^-124) have the smallest scale, 2^-127
  scale = (uint32_t)max((int)(top >> 23) - 2, 0);
  const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale): 2^127 down to 2^-125, exact products
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[8 * i + e] * inv;
    w[i] = mx_encode8(v);
  }
  codes = make_uint4(w[0], w[1], w[2], w[3]);
  return bad;
}

// A thread a block; a warp takes eight rows of a piece: 512 bytes of codes one after another.
template <typename T>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const MxRowsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int pieces = (a.width + kMxPiece - 1) / kMxPiece;
  const int groups = (a.n_rows + 7) / 8;
  const long long unit = (long long)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)groups * pieces) return;
  const int lane = threadIdx.x & 31, b = lane & 3;
  const int piece = (int)(unit % pieces);
  const long long row = (unit / pieces) * 8 + (lane >> 2);
  const int at = piece * kMxPiece + b * kMxBlock;
  const bool live = row < a.n_rows;
  uint4 codes = make_uint4(0, 0, 0, 0);
  uint32_t scale = 0;
  if (live && at < a.width) {
    float x[32];
    load32<T>(static_cast<const T*>(a.x) + row * a.stride + at, a.width - at, a.vec != 0, x);
    if (mx_round(x, codes, scale)) set_err(a.err, PE_DEV_NONFINITE);
  }
  uint32_t s4 = scale << (8 * b);
  s4 |= __shfl_xor_sync(0xFFFFFFFFu, s4, 1);
  s4 |= __shfl_xor_sync(0xFFFFFFFFu, s4, 2);
  if (!live) return;
  const int r = (int)(row % kMxPiece);
  uint8_t* rec = a.mx + ((size_t)(row / kMxPiece) * pieces + piece) * kMxRecord;
  *reinterpret_cast<uint4*>(rec + mx_code_at(r, b)) = codes;
  if (b == 0) *reinterpret_cast<uint32_t*>(rec + mx_scale_at(r, 0)) = s4;
}

PE_DEV void store_pair(float* p, float x, float y, bool both) {
  p[0] = x;
  if (both) p[1] = y;
}
PE_DEV void store_pair(__nv_bfloat16* p, float x, float y, bool both) {
  p[0] = __float2bfloat16_rn(x);
  if (both) p[1] = __float2bfloat16_rn(y);
}

template <typename T>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const MxRowsArgs a) {
  pdl_wait();
  pdl_trigger();
  const int pieces = (a.width + kMxPiece - 1) / kMxPiece;
  const int groups = (a.n_rows + 7) / 8;
  const long long unit = (long long)blockIdx.x * (kMxThreads / 32) + (threadIdx.x >> 5);
  if (unit >= (long long)groups * pieces) return;
  const int lane = threadIdx.x & 31, b = lane & 3;
  const int piece = (int)(unit % pieces);
  const long long row = (unit / pieces) * 8 + (lane >> 2);
  const int at = piece * kMxPiece + b * kMxBlock;
  if (row >= a.n_rows || at >= a.width) return;
  const int r = (int)(row % kMxPiece), left = a.width - at;
  const uint8_t* rec = a.mx + ((size_t)(row / kMxPiece) * pieces + piece) * kMxRecord;
  const uint4 codes = __ldcg(reinterpret_cast<const uint4*>(rec + mx_code_at(r, b)));
  const float s = mx_scale(__ldcg(rec + mx_scale_at(r, b)));
  T* out = static_cast<T*>(a.out) + row * a.stride + at;
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t h[4];
    mx_decode8(w[i], h);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
      const int j = 8 * i + 2 * e;
      if (j < left) store_pair(out + j, f.x * s, f.y * s, j + 1 < left);
    }
  }
}

}  // namespace

static unsigned mx_grid(long long units) { return (unsigned)((units + kMxThreads / 32 - 1) / (kMxThreads / 32)); }

cudaError_t launch_mx_quantize(const MxRowsArgs& a, pe_dtype dt, cudaStream_t s) {
  const long long units = (long long)((a.n_rows + 7) / 8) * ((a.width + kMxPiece - 1) / kMxPiece);
  const dim3 grid(mx_grid(units)), block(kMxThreads);
  return dt == PE_BF16 ? launch_pdl(mx_quantize_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                       : launch_pdl(mx_quantize_kernel<float>, grid, block, 0, s, a);
}

cudaError_t launch_mx_dequantize(const MxRowsArgs& a, pe_dtype dt, cudaStream_t s) {
  const long long units = (long long)((a.n_rows + 7) / 8) * ((a.width + kMxPiece - 1) / kMxPiece);
  const dim3 grid(mx_grid(units)), block(kMxThreads);
  return dt == PE_BF16 ? launch_pdl(mx_dequantize_kernel<__nv_bfloat16>, grid, block, 0, s, a)
                       : launch_pdl(mx_dequantize_kernel<float>, grid, block, 0, s, a);
}

}  // namespace pe
