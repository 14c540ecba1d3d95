// Grouped-query attention of ragged query rows over a packed (4-bit) paged cache.
// The cache's format is in pe_packed.cuh.
//
// Row r of sequence b (rows row_start[b] .. row_start[b+1] - 1) at position p attends to the
// cache positions 0..p of its sequence:
//   out[r][h] = sum_{x <= p} w_x v_x / sum_{x <= p} w_x,  w_x = exp(q[r][h] . k_x / sqrt(hd) - max)
// with keys and values of head h / (n_q / n_kv).  A row at position -1 sees nothing: zeros.
#include <algorithm>

#include "pe_internal.h"
#include "pe_packed.cuh"

namespace pe {

namespace {

// One warp per (row, query head): lanes stride over the positions with an online softmax each,
// then merge.
template <typename T, int HD>
__global__ void __launch_bounds__(256) attend_kernel(const PackedAttnArgs a) {
  using L = PackedLayout<HD>;
  pdl_wait();
  pdl_trigger();
  const long long gw = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = (int)(gw / a.n_q), h = (int)(gw - (long long)row * a.n_q);
  if (row >= a.n_rows) return;
  int lo = 0, hi = a.B;  // the sequence whose rows hold `row`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.row_start + mid) <= row) lo = mid;
    else hi = mid;
  }
  const int b = lo, r0 = __ldcg(a.row_start + b), r1 = a.row_len ? r0 + __ldcg(a.row_len + b) : __ldcg(a.row_start + b + 1);
  if (r0 < 0 || r1 < r0 || r1 > a.n_rows || r1 - r0 > a.max_rows) {
    if (lane == 0) set_err(a.err, PE_DEV_BAD_ROW);
    return;
  }
  if (row < r0 || row >= r1) return;
  int p = __ldcg(a.positions + row);
  if (p < -1 || p >= a.max_pages * kPackedPage) {
    if (lane == 0) set_err(a.err, PE_DEV_BAD_POSITION);
    p = -1;
  }
  const int G = a.n_q / a.n_kv, g = h / G;
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride + (long long)h * HD;
  float qr[HD], o[HD];
#pragma unroll
  for (int e = 0; e < HD; ++e) {
    qr[e] = to_float<T>(q[e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int pos = lane; pos <= p; pos += 32) {
    const int page = __ldcg(a.block_table + (size_t)b * a.max_pages + pos / kPackedPage);
    const bool ok = page >= 0 && page < a.num_pages;
    if (!ok) set_err(a.err, PE_DEV_BAD_PAGE);  // such a page's keys and values read as zeros
    const uint8_t* rec = a.pool + ((size_t)(ok ? page : 0) * a.n_kv + g) * L::kRecord;
    const int off = pos % kPackedPage;
    const uint32_t* kw = reinterpret_cast<const uint32_t*>(rec + L::kK + off * L::kRow);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(rec + L::kV + off * L::kRow);
    float dot[HD / 16];
#pragma unroll
    for (int j = 0; j < HD / 16; ++j) dot[j] = 0.f;
#pragma unroll
    for (int w = 0; w < HD / 8; ++w) {
      const uint32_t c = __ldg(kw + w);
      const int t = w / (HD / 32), u = w % (HD / 32);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = 2 * u + (i & 3) / 2, e = 16 * j + 4 * t + 2 * (i & 1) + i / 4;
        dot[j] += qr[e] * (float)((int)((c >> (4 * i)) & 15u) - 8);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < HD / 16; ++j) s += dot[j] * packed_scale(rec[L::kKs + off * L::kScaleRow + j]);
    s = ok ? s * a.scale : 0.f;
    const float m_new = fmaxf(m, s);
    const float c = m == -INFINITY ? 0.f : expf(m - m_new);
    const float w = expf(s - m_new);
    l = l * c + w;
    float ws[HD / 16];
#pragma unroll
    for (int j = 0; j < HD / 16; ++j) ws[j] = ok ? w * packed_scale(rec[L::kVs + off * L::kScaleRow + j]) : 0.f;
#pragma unroll
    for (int wd = 0; wd < HD / 8; ++wd) {
      const uint32_t cd = __ldg(vw + wd);
      const int gg = wd / (HD / 64), hh = wd % (HD / 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int j = 4 * hh + i / 2, e = 16 * j + gg + 8 * (i & 1);
        o[e] = o[e] * c + ws[j] * (float)((int)((cd >> (4 * i)) & 15u) - 8);
      }
    }
    m = m_new;
  }
  float M = m;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, s));
  const float f = m == -INFINITY ? 0.f : expf(m - M);
  float sum = l * f;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
  T* out = static_cast<T*>(a.out) + row * a.out_stride + (long long)h * HD;
#pragma unroll
  for (int e = 0; e < HD; ++e) {
    float v = o[e] * f;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
    if (lane == (e & 31)) out[e] = from_float<T>(sum > 0.f ? v / sum : 0.f);
  }
}

template <typename T, int HD>
cudaError_t attend_typed(const PackedAttnArgs& a, cudaStream_t s) {
  const long long warps = (long long)a.n_rows * a.n_q;
  return launch_pdl(attend_kernel<T, HD>, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, s, a);
}

}  // namespace

size_t packed_attn_workspace_bytes(int, pe_dtype, int) { return 256; }

cudaError_t launch_attend_packed(const PackedAttnArgs& a, pe_dtype dt, int, cudaStream_t s) {
  if (a.n_rows == 0) return cudaSuccess;
  if (a.head_dim == 64) return dt == PE_BF16 ? attend_typed<__nv_bfloat16, 64>(a, s) : attend_typed<float, 64>(a, s);
  return dt == PE_BF16 ? attend_typed<__nv_bfloat16, 128>(a, s) : attend_typed<float, 128>(a, s);
}

}  // namespace pe
