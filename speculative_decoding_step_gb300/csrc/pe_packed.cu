// Packing key and value rows into a 4-bit paged cache, and reading entries back.
// The format is in pe_packed.cuh.
#include <algorithm>

#include "pe_internal.h"
#include "pe_packed.cuh"

namespace pe {

namespace {

constexpr int kPackThreads = 128;  // (256: 0 to 2 us more for both kernels)

// Eight entries at a 16-byte boundary: their values, and the bits of the largest magnitude as fp32 (at least
// kInfBits: one is infinite or NaN).  Magnitudes compare as whole numbers, bf16 two at a time.
constexpr uint32_t kInfBits = 0x7F800000u;
struct Eight {
  float x[8];
  uint32_t top;
  PE_DEV void load(const float* p) {
    top = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(p) + k);
      x[4 * k] = t.x; x[4 * k + 1] = t.y; x[4 * k + 2] = t.z; x[4 * k + 3] = t.w;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  }
  PE_DEV void load(const __nv_bfloat16* p) {
    const uint4 t = __ldcg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(w[e] & 0x7FFF7FFFu));
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    top = max(m << 16, m & 0xFFFF0000u);
  }
};
// Eight entries given as bf16 pairs.
PE_DEV void store8(__nv_bfloat16* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
PE_DEV void store8(float* p, const uint32_t (&w)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    reinterpret_cast<float4*>(p)[k] =
        make_float4(__uint_as_float(w[2 * k] << 16), __uint_as_float(w[2 * k] & 0xFFFF0000u),
                    __uint_as_float(w[2 * k + 1] << 16), __uint_as_float(w[2 * k + 1] & 0xFFFF0000u));
}

// Both kernels give a head's row of keys and of values to HD/8 lanes.  A lane holds word w (its number) of
// either code row, and the eight entries whose codes come together from the words of a few lanes:
//   keys    w = t*(HD/32) + u.  Lanes t and t^1 hold, byte by byte, blocks 2u and 2u+1: they exchange half a word, and
//           lane (t, u) has entries 8(t/2)..+7 of block 2u + t%2.
//   values  w = g*(HD/64) + h, a nibble for each of eight pieces of eight entries: an 8 x 8 transpose of nibbles
//           over the lanes g, in three exchanges of half a word; lane (g, h) has entries 64h + 8i..+7, i = g with
//           its bits 0, 2, 1 as bits 2, 1, 0 (which leaves pairs of entries 16 bits apart, as for the keys).
// An exchange turns a bit of the lane's number into a bit of the place of a field in the word, and that bit into it:
// the lane keeps one half of its word's fields and swaps the other for its partner's.
template <int SH, uint32_t MASK>
struct Exchange {
  uint32_t keep;
  int away;  // where the partner's half goes
  PE_DEV explicit Exchange(bool upper) : keep(upper ? MASK << SH : MASK), away(upper ? 0 : SH) {}
  PE_DEV uint32_t operator()(uint32_t x, int by) const {
    return (x & keep) | __shfl_xor_sync(0xFFFFFFFFu, (x >> away) & MASK, by) << away;
  }
};
template <int HD>
struct Lane {
  static constexpr int N = HD / 8, KU = HD / 32, VU = HD / 64;
  int w, key, value;  // word; first entry of its eight of the keys and of the values
  Exchange<8, 0x00FF00FFu> kx, v1;
  Exchange<16, 0x0000FFFFu> v0;
  Exchange<4, 0x0F0F0F0Fu> v2;
  PE_DEV explicit Lane(int lane)
      : w(lane % N), kx((w / KU) & 1), v1((w / VU) & 4), v0((w / VU) & 1), v2((w / VU) & 2) {
    const int t = w / KU, g = w / VU;
    key = 16 * (2 * (w % KU) + (t & 1)) + 8 * (t >> 1);
    value = 64 * (w % VU) + 8 * ((g & 1) << 2 | (g >> 2 & 1) << 1 | (g >> 1 & 1));
  }
  // Words from codes and codes from words: eight nibbles, the pairs of entries 16 bits apart.  The keys' entries
  // 0..3 stand in bytes 0 and 2, entries 4..7 in bytes 1 and 3; the values' in nibble order.
  PE_DEV uint32_t keys(uint32_t x) const { return kx(x, KU); }
  PE_DEV uint32_t values(uint32_t x) const { return v2(v1(v0(x, VU), 4 * VU), 2 * VU); }
};

// How a launch deals out rows and heads: a CTA has `heads` groups of lanes side by side for `rows` rows at a
// time, `steps` times, and again for the heads that are left.  Addresses then advance by additions, and there
// are eight CTAs an SM (four: a third more time, the loads of a step wait for the one before; sixteen: the same), all
// resident at once but for packing fp32, whose registers leave six.  With a CTA per 128 lanes' rows, the
// instructions that found each lane's place were half of all.
struct Deal {
  int heads, rows, steps, n_kv;
  Div by_heads;
};
constexpr int kPackCtas = 152 * 8;
template <int HD>
Deal deal(int n_rows, int n_kv, unsigned* grid, unsigned* threads) {
  constexpr int N = Lane<HD>::N, groups = kPackThreads / N;
  Deal d{};
  const int passes = (n_kv + groups - 1) / groups;
  d.heads = (n_kv + passes - 1) / passes;
  d.rows = groups / d.heads;
  d.steps = (int)((n_rows + (long long)d.rows * kPackCtas - 1) / ((long long)d.rows * kPackCtas));
  d.n_kv = n_kv;
  d.by_heads = make_div(d.heads);
  const long long per = (long long)d.rows * d.steps;
  *grid = (unsigned)((n_rows + per - 1) / per);
  *threads = (unsigned)((d.heads * d.rows * N + 31) / 32 * 32);
  return d;
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

// Rounds eight entries of a block of 16, whose other half the lane `by` away has: the nibbles code + 8 of
// pairs of entries 16 bits apart (entry 2i in bits 4i, 2i + 1 in bits 16 + 4i), and the block's scale
// byte.  Returns whether one of the eight was NaN (kept as 0) or infinite (kept as +-7 s).
template <typename T>
PE_DEV bool quantise(Eight& h, int by, uint32_t& nibbles, uint32_t& code) {
  const bool bad = h.top >= kInfBits;
  if (bad) {
    h.top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = __float_as_uint(h.x[e]) & 0x7FFFFFFFu;
      if (m < kInfBits) h.top = max(h.top, m);
      if (m > kInfBits) h.x[e] = 0.f;
    }
  }
  const float amax = __uint_as_float(max(h.top, __shfl_xor_sync(0xFFFFFFFFu, h.top, by)));
  code = scale_code(amax);
  const float s = packed_scale(code);
  if (bad || amax > 7.f * s) {  // entries beyond the largest scale's range keep its largest code
#pragma unroll
    for (int e = 0; e < 8; ++e) h.x[e] = fminf(fmaxf(h.x[e], -7.f * s), 7.f * s);
  }
  // round(x / s), halves away from zero, as x times a float above 1/s plus 1.5 * 2^23 + 8 in one
  // fused operation: the sum's mantissa bits are 2^22 + the nibble.  The factor is at most two
  // rounding steps above 1/s, so an exact half goes away from zero; a bf16 x over a scale of
  // four bits is never nearer to a half than 2^-10 without being one.  (A scale has
  // eight mantissas, so the tests have seen every factor that there is.)
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));  // off by at most one step
  inv = __uint_as_float(__float_as_uint(inv) + 1);
  constexpr uint32_t kSum = 0x4B400000u;  // of 1.5 * 2^23; eight of them shifted are taken off at once
  nibbles = 0u - kSum * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t n = __float_as_uint(fmaf(h.x[e], inv, 12582920.f));
    if (sizeof(T) == 4) {
      // fp32 entries can be nearer to a half than that: the halves themselves decide (exact
      // products of four-bit numbers)
      const float m = fabsf(h.x[e]), c = fabsf((float)((int)(n & 15u) - 8));
      const int off = m < (c - 0.5f) * s ? -1 : m >= (c + 0.5f) * s ? 1 : 0;
      n += h.x[e] < 0.f ? -off : off;
    }
    nibbles += n << (4 * (e >> 1) + 16 * (e & 1));
  }
  return bad;
}

// Packing and reading back are bound by memory in principle: bytes of the rows and of their packed form, once
// each.  Measured, 12,026 rows of 4 heads of 128 entries in bf16 (56 MB both ways) are packed and read back in
// 17.4 us (20.7 as a graph), 24,586 rows of 8 heads of 64 read back (65 MB) in 16.1 us (18.6): 3.2 and 4.0 TB/s.  A lane
// takes five and eleven steps there, one after the other, each a chain of dependent loads (the slot, then, reading
// back, the entries) and stores; no unit is full (schedulers 45 to 64 % busy, integer pipe 42 to 54 %, DRAM below
// 27 %).  Loading one step ahead of its use did not change the times (21.6 and 17.7 us against 21 and 18 then), nor did
// longer rows per lane.

// HD/8 lanes per (row, head), eight keys and eight values each.
template <typename T, int HD>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a, const Deal d) {
  using L = PackedLayout<HD>;
  const Lane<HD> ln(threadIdx.x);
  const int group = threadIdx.x / Lane<HD>::N, r = (int)((uint32_t)group / d.by_heads);
  const uint64_t n_slots = (uint64_t)a.num_pages * kPackedPage;
  const uint32_t page_bytes = (uint32_t)d.n_kv * L::kRecord;
  const long long row0 = (long long)blockIdx.x * d.rows * d.steps + r;
  pdl_wait();
  pdl_trigger();
  const int n_rows = a.n_dev != nullptr ? min(max(__ldcg(a.n_dev), 0), a.n_rows) : a.n_rows;
  for (int h0 = 0; h0 < d.n_kv; h0 += d.heads) {
    const int head = h0 + group - r * d.heads;
    const bool mine = r < d.rows && head < d.n_kv;
    const int64_t* slots = a.slots + row0;
    const T* k_row = static_cast<const T*>(a.k) + row0 * a.k_stride + (long long)head * HD + ln.key;
    const T* v_row = static_cast<const T*>(a.v) + row0 * a.v_stride + (long long)head * HD + ln.value;
    uint8_t* pool = a.pool + (size_t)head * L::kRecord;
    for (int i = 0; i < d.steps; ++i) {
      int64_t slot = -1;
      Eight k{}, v{};
      if (mine && row0 + (long long)i * d.rows < n_rows) {
        slot = __ldcg(reinterpret_cast<const long long*>(slots));
        k.load(k_row);
        v.load(v_row);
      }
      slots += d.rows;
      k_row += d.rows * a.k_stride;
      v_row += d.rows * a.v_stride;
      uint32_t kw, vw, kc, vc;
      bool bad = quantise<T>(k, 2 * Lane<HD>::KU, kw, kc);
      bad |= quantise<T>(v, 2 * Lane<HD>::VU, vw, vc);
      kw = ln.keys(kw);
      vw = ln.values(vw);
      if ((uint64_t)slot >= n_slots) {
        if (slot != -1) set_err(a.err, PE_DEV_BAD_PAGE);
        continue;
      }
      if (bad) set_err(a.err, PE_DEV_NONFINITE);
      const int off = (int)slot & (kPackedPage - 1);
      uint8_t* rec = pool + (uint64_t)(uint32_t)(slot / kPackedPage) * page_bytes;
      reinterpret_cast<uint32_t*>(rec + L::kK + off * L::kRow)[ln.w] = kw;
      reinterpret_cast<uint32_t*>(rec + L::kV + off * L::kRow)[ln.w] = vw;
      if ((ln.key & 8) == 0) rec[L::kKs + off * L::kScaleRow + ln.key / kPackedBlock] = (uint8_t)kc;
      if ((ln.value & 8) == 0) rec[L::kVs + off * L::kScaleRow + ln.value / kPackedBlock] = (uint8_t)vc;
    }
  }
}

// HD/8 lanes per (row, head), eight keys and eight values each.
template <typename T, int HD>
__global__ void __launch_bounds__(kPackThreads) unpack_kernel(const UnpackArgs a, const Deal d) {
  using L = PackedLayout<HD>;
  const Lane<HD> ln(threadIdx.x);
  const PairBits bits;
  const int group = threadIdx.x / Lane<HD>::N, r = (int)((uint32_t)group / d.by_heads);
  const uint64_t n_slots = (uint64_t)a.num_pages * kPackedPage;
  const uint32_t page_bytes = (uint32_t)d.n_kv * L::kRecord;
  const long long row0 = (long long)blockIdx.x * d.rows * d.steps + r;
  pdl_wait();
  pdl_trigger();
  for (int h0 = 0; h0 < d.n_kv; h0 += d.heads) {
    const int head = h0 + group - r * d.heads;
    const bool mine = r < d.rows && head < d.n_kv;
    const int64_t* slots = a.slots + row0;
    T* k_row = static_cast<T*>(a.k_out) + row0 * a.k_stride + (long long)head * HD + ln.key;
    T* v_row = static_cast<T*>(a.v_out) + row0 * a.v_stride + (long long)head * HD + ln.value;
    const uint8_t* pool = a.pool + (size_t)head * L::kRecord;
    for (int i = 0; i < d.steps; ++i) {
      const bool live = mine && row0 + (long long)i * d.rows < a.n_rows;
      const int64_t slot = live ? __ldcg(reinterpret_cast<const long long*>(slots)) : -1;
      const bool good = (uint64_t)slot < n_slots;
      if (!good && slot != -1) set_err(a.err, PE_DEV_BAD_PAGE);
      uint32_t kw = 0, vw = 0, ks = 0, vs = 0;
      if (good) {
        const int off = (int)slot & (kPackedPage - 1);
        const uint8_t* rec = pool + (uint64_t)(uint32_t)(slot / kPackedPage) * page_bytes;
        kw = __ldcg(reinterpret_cast<const uint32_t*>(rec + L::kK + off * L::kRow) + ln.w);
        vw = __ldcg(reinterpret_cast<const uint32_t*>(rec + L::kV + off * L::kRow) + ln.w);
        ks = __ldcg(rec + L::kKs + off * L::kScaleRow + ln.key / kPackedBlock);
        vs = __ldcg(rec + L::kVs + off * L::kScaleRow + ln.value / kPackedBlock);
      }
      const uint32_t x = ln.keys(kw), y = x >> 8, z = ln.values(vw);
      if (good) {
        const uint32_t sk = packed_scale_pair(ks), sv = packed_scale_pair(vs);
        const uint32_t bk = bf16x2_mul(sk, kMinus136), bv = bf16x2_mul(sv, kMinus136);
        const uint32_t k4[4] = {bf16x2_fma(bits.pair<0>(x), sk, bk), bf16x2_fma(bits.pair<1>(x), sk, bk),
                                bf16x2_fma(bits.pair<0>(y), sk, bk), bf16x2_fma(bits.pair<1>(y), sk, bk)};
        const uint32_t v4[4] = {bf16x2_fma(bits.pair<0>(z), sv, bv), bf16x2_fma(bits.pair<1>(z), sv, bv),
                                bf16x2_fma(bits.pair<2>(z), sv, bv), bf16x2_fma(bits.pair<3>(z), sv, bv)};
        store8(k_row, k4);
        store8(v_row, v4);
      }
      slots += d.rows;
      k_row += d.rows * a.k_stride;
      v_row += d.rows * a.v_stride;
    }
  }
}

template <typename T, int HD>
cudaError_t pack_typed(const PackArgs& a, cudaStream_t s) {
  unsigned grid, threads;
  const Deal d = deal<HD>(a.n_rows, a.n_kv, &grid, &threads);
  return launch_pdl(pack_kernel<T, HD>, dim3(grid), dim3(threads), 0, s, a, d);
}
template <typename T, int HD>
cudaError_t unpack_typed(const UnpackArgs& a, cudaStream_t s) {
  unsigned grid, threads;
  const Deal d = deal<HD>(a.n_rows, a.n_kv, &grid, &threads);
  return launch_pdl(unpack_kernel<T, HD>, dim3(grid), dim3(threads), 0, s, a, d);
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
