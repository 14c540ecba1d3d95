// Rotary positions applied to query and key rows on their way to the attention and into a paged KV cache.
//
// Pair i of a head, entries (i, i + hd/2), turns by positions[axis(i)] * theta^(-2i/hd).  The angle is kept in turns as
// a 64-bit fraction: the pair's turns per position, mod 1, times 2^64 as a whole number (made on the host in double),
// times the position, mod 2^64.  That product is exact, so an angle is off by what the frequency is (2^-53 relative) and
// by the rounding of the fraction to fp32, at any position.
#include <algorithm>

#include "pe_append.cuh"
#include "pe_internal.h"

namespace pe {

namespace {

constexpr int kAppendThreads = 128;

template <typename T>
PE_DEV void load8(const T* p, float (&x)[8]);
template <>
PE_DEV void load8<float>(const float* p, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 t = __ldcg(reinterpret_cast<const float4*>(p) + k);
    x[4 * k] = t.x; x[4 * k + 1] = t.y; x[4 * k + 2] = t.z; x[4 * k + 3] = t.w;
  }
}
template <>
PE_DEV void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
PE_DEV void store8(float* p, const float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    reinterpret_cast<float4*>(p)[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
}
PE_DEV void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA a row.  A thread has eight pairs of a head (the sines and cosines of one chunk serve every head that it takes);
// value rows are copied as two eights the same way.
template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr int C = HD / 16, HALF = HD / 2;  // chunks of eight pairs
  pdl_wait();
  pdl_trigger();
  const long long row = blockIdx.x;
  const int c = threadIdx.x % C;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) rope_angle(a.rope, __ldcg(a.positions + (long long)a.rope.axis[8 * c + j] * a.n_rows + row), 8 * c + j, cs[j], sn[j]);
  int64_t slot = -1;
  bool put = false;
  if (a.k != nullptr) {
    slot = __ldcg(reinterpret_cast<const long long*>(a.slots) + row);
    put = (uint64_t)slot < (uint64_t)a.num_pages * 16;
    if (!put && slot != -1 && threadIdx.x == 0) set_err(a.err, PE_DEV_BAD_PAGE);
  }
  const int n_q = a.q != nullptr ? a.n_q : 0, n_kv = put ? a.n_kv : 0;
  for (int h = threadIdx.x / C; h < n_q + 2 * n_kv; h += kAppendThreads / C) {
    const T* src;
    T* dst;
    if (h < n_q) {
      src = static_cast<const T*>(a.q) + row * a.q_stride + (long long)h * HD;
      dst = static_cast<T*>(a.q_out) + row * a.q_out_stride + (long long)h * HD;
    } else {
      const bool key = h < n_q + n_kv;
      const int g = h - n_q - (key ? 0 : n_kv);
      src = static_cast<const T*>(key ? a.k : a.v) + row * (key ? a.k_stride : a.v_stride) + (long long)g * HD;
      dst = static_cast<T*>(key ? a.k_cache : a.v_cache) + (slot * a.n_kv + g) * HD;
    }
    float x1[8], x2[8];
    load8<T>(src + 8 * c, x1);
    load8<T>(src + 8 * c + HALF, x2);
    if (h < n_q + n_kv)
#pragma unroll
      for (int j = 0; j < 8; ++j) rope_turn(x1[j], x2[j], cs[j], sn[j]);
    store8(dst + 8 * c, x1);
    store8(dst + 8 * c + HALF, x2);
  }
}

template <typename T, int HD>
cudaError_t append_typed(const AppendArgs& a, cudaStream_t s) {
  return launch_pdl(append_kernel<T, HD>, dim3((unsigned)a.n_rows), dim3(kAppendThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int head_dim, pe_dtype dt, cudaStream_t s) {
  if (head_dim == 64) return dt == PE_BF16 ? append_typed<__nv_bfloat16, 64>(a, s) : append_typed<float, 64>(a, s);
  return dt == PE_BF16 ? append_typed<__nv_bfloat16, 128>(a, s) : append_typed<float, 128>(a, s);
}

}  // namespace pe
