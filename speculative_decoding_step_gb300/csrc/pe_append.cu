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
constexpr int kAppendDepth = 3;

// Sixteen entries on their way, as they were read: eight of a head's first half and the eight they are paired with.
template <typename T>
struct Pairs;
template <>
struct Pairs<__nv_bfloat16> {
  uint4 a, b;
  PE_DEV void load(const __nv_bfloat16* p, int half) {
    a = __ldcg(reinterpret_cast<const uint4*>(p));
    b = __ldcg(reinterpret_cast<const uint4*>(p + half));
  }
  PE_DEV void store(__nv_bfloat16* p, int half) const {
    *reinterpret_cast<uint4*>(p) = a;
    *reinterpret_cast<uint4*>(p + half) = b;
  }
  PE_DEV static void turn(uint32_t& x, uint32_t& y, const float2 (&t)[2]) {
    float x0 = __uint_as_float(x << 16), x1 = __uint_as_float(x & 0xFFFF0000u);
    float y0 = __uint_as_float(y << 16), y1 = __uint_as_float(y & 0xFFFF0000u);
    rope_turn(x0, y0, t[0].x, t[0].y);
    rope_turn(x1, y1, t[1].x, t[1].y);
    const __nv_bfloat162 u = __floats2bfloat162_rn(x0, x1), v = __floats2bfloat162_rn(y0, y1);
    x = *reinterpret_cast<const uint32_t*>(&u);
    y = *reinterpret_cast<const uint32_t*>(&v);
  }
  PE_DEV void turn(const float2 (&t)[4][2]) {
    turn(a.x, b.x, t[0]);
    turn(a.y, b.y, t[1]);
    turn(a.z, b.z, t[2]);
    turn(a.w, b.w, t[3]);
  }
};
template <>
struct Pairs<float> {
  float4 a[2], b[2];
  PE_DEV void load(const float* p, int half) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      a[k] = __ldcg(reinterpret_cast<const float4*>(p) + k);
      b[k] = __ldcg(reinterpret_cast<const float4*>(p + half) + k);
    }
  }
  PE_DEV void store(float* p, int half) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      reinterpret_cast<float4*>(p)[k] = a[k];
      reinterpret_cast<float4*>(p + half)[k] = b[k];
    }
  }
  PE_DEV void turn(const float2 (&t)[4][2]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      rope_turn(a[k].x, b[k].x, t[2 * k][0].x, t[2 * k][0].y);
      rope_turn(a[k].y, b[k].y, t[2 * k][1].x, t[2 * k][1].y);
      rope_turn(a[k].z, b[k].z, t[2 * k + 1][0].x, t[2 * k + 1][0].y);
      rope_turn(a[k].w, b[k].w, t[2 * k + 1][1].x, t[2 * k + 1][1].y);
    }
  }
};

// A CTA a row.  Its heads' loads go out first (kAppendDepth of each thread at a time); meanwhile a thread a pair finds the
// sines and cosines, which all heads share.  Bound by memory at many rows.
template <typename T, int HD>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  constexpr int C = HD / 16, HALF = HD / 2;  // a head's chunks of eight pairs
  __shared__ __align__(16) float2 turns[HALF];
  pdl_wait();
  pdl_trigger();
  const long long row = blockIdx.x;
  const int c = threadIdx.x % C, n_q = a.q != nullptr ? a.n_q : 0, n_kv = a.k != nullptr ? a.n_kv : 0;
  const int heads = n_q + 2 * n_kv;
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride;
  const T* k = static_cast<const T*>(a.k) + row * a.k_stride;
  const T* v = static_cast<const T*>(a.v) + row * a.v_stride;
  Pairs<T> x[kAppendDepth];
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kAppendDepth; ++j) {
      const int h = h0 + j * (kAppendThreads / C);
      if (h < n_q)
        x[j].load(q + (long long)h * HD + 8 * c, HALF);
      else if (h < n_q + n_kv)
        x[j].load(k + (long long)(h - n_q) * HD + 8 * c, HALF);
      else if (h < heads)
        x[j].load(v + (long long)(h - n_q - n_kv) * HD + 8 * c, HALF);
    }
  };
  load(threadIdx.x / C);
  const int64_t slot = n_kv > 0 ? __ldcg(reinterpret_cast<const long long*>(a.slots) + row) : -1;
  if (threadIdx.x < HALF) {
    const int i = threadIdx.x;
    rope_angle(a.rope, __ldcg(a.positions + (long long)a.rope.axis[i] * a.n_rows + row), i, turns[i].x, turns[i].y);
  }
  __syncthreads();
  float2 t[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 w = *reinterpret_cast<const float4*>(&turns[8 * c + 2 * j]);
    t[j][0] = make_float2(w.x, w.y);
    t[j][1] = make_float2(w.z, w.w);
  }
  const bool put = (uint64_t)slot < (uint64_t)a.num_pages * 16;
  if (!put && slot != -1 && threadIdx.x == 0) set_err(a.err, PE_DEV_BAD_PAGE);
  T* qo = static_cast<T*>(a.q_out) + row * a.q_out_stride;
  T* kc = static_cast<T*>(a.k_cache) + (put ? slot * a.n_kv * HD : 0);
  T* vc = static_cast<T*>(a.v_cache) + (put ? slot * a.n_kv * HD : 0);
  for (int h0 = threadIdx.x / C;;) {
#pragma unroll
    for (int j = 0; j < kAppendDepth; ++j) {
      const int h = h0 + j * (kAppendThreads / C);
      if (h < n_q + n_kv) x[j].turn(t);
      if (h < n_q)
        x[j].store(qo + (long long)h * HD + 8 * c, HALF);
      else if (put && h < n_q + n_kv)
        x[j].store(kc + (long long)(h - n_q) * HD + 8 * c, HALF);
      else if (put && h < heads)
        x[j].store(vc + (long long)(h - n_q - n_kv) * HD + 8 * c, HALF);
    }
    h0 += kAppendDepth * (kAppendThreads / C);
    if (h0 >= heads) break;
    load(h0);
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
