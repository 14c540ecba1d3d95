// What the two kernels of the 4-bit product share (pe_mx_gemm.cu has the mathematics): instructions, and what becomes of
// the sums.
#pragma once

#include <type_traits>

#include "pe_internal.h"
#include "pe_mx.cuh"

namespace pe {

constexpr uint32_t kMxgSeen = 1024;            // shared memory of barriers, tensor-memory slot and flags, then
constexpr uint32_t kMxgCtrl = kMxgSeen + 2048;  // mx_seen's numbers of two units

// Shared-memory descriptor of a K-major operand in core matrices: lbo bytes to the next 16-byte column, sbo to the next
// eight rows.
PE_DEV uint64_t sdesc_core(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}
// Instruction descriptor of kind::mxf4: both operands e2m1, K-major, scales ue8m0, fp32 accumulators.  The scales' place in
// their 32-bit columns (0: the first two blocks, 2: the other two) goes into bits 4 and 29.
PE_DEV uint32_t idesc_mxf4(int M, int N) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
constexpr uint32_t kScaleUpper = (2u << 4) | (2u << 29);

PE_DEV void tc_mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t a_scale, uint32_t b_scale,
                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}
// 512 bytes of scales into four columns of all 128 lanes (in order before MMAs issued later by this thread).
PE_DEV void tc_copy_scales(uint32_t dst, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(sdesc) : "memory");
}
// mbar_wait by a whole warp, which stays together; false too where another role gave up.  (One lane's question and a shuffle take 80 ns longer.)
PE_DEV bool mbar_wait_warp(uint32_t bar, uint32_t parity, const MxMatmulArgs& a, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, a.err, abort, a.wait_ns) && !*abort);
}

// What is added to 16 columns (rows t0.. of y) of feature f, as it is read: widened where it is used, so that nothing waits
// for it before.  Rows and features beyond the last read the last one's, and do not use it: loads under a condition wait for
// each other (158 rows to 23494 features, bf16: 21 us).
template <typename T>
PE_DEV void mx_addend(const MxMatmulArgs& a, int f, int t0, uint32_t (&old)[16]) {
  using Bits = typename std::conditional<sizeof(T) == 2, unsigned short, uint32_t>::type;
  const Bits* add = static_cast<const Bits*>(a.add) + min(f, a.n_out - 1);
#pragma unroll
  for (int j = 0; j < 16; ++j) old[j] = add[(long long)min(t0 + j, a.n_rows - 1) * a.add_stride];
}
template <typename T>
PE_DEV void mx_store(const MxMatmulArgs& a, int f, int t0, const float (&v)[16]) {
  if (f >= a.n_out) return;
  T* y = static_cast<T*>(a.y) + (long long)t0 * a.y_stride + f;
  const int n = a.n_rows - t0;
  if (n >= 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) y[(long long)j * a.y_stride] = from_float<T>(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) y[(long long)j * a.y_stride] = from_float<T>(v[j]);
  }
}

// Type of the output where the rows' largest sums are looked for instead (MxHeadArgs).
struct MxArgmax {};

// Largest sums that the rows of a unit (from row0 on) had so far, out of their keys, into shared memory: row `thread`'s.
// NaN: none yet; rows beyond the last: infinite.  On barrier 1, by all `threads` threads that write results.
PE_DEV void mx_seen(const MxMatmulArgs& a, int row0, float* seen, int thread, int threads) {
  const int t = row0 + thread;
  uint32_t bits = 0x7F800000u;
  if (t < a.n_rows) {
    const uint32_t ord = (uint32_t)(__ldcg(a.head.keys + t) >> 32);
    bits = ord ^ ((uint32_t)((int32_t)~ord >> 31) | 0x80000000u);
  }
  seen[thread] = __uint_as_float(bits);
  named_bar_sync(1, threads);
}
// 16 rows of x (from t0 on) of 32 features, a feature f a lane: the warp's largest sum of each row joins the row's key.  Few
// of a row's tiles raise its maximum; where none of the 16 x 32 sums reaches what its row had, or is no number, that is all.
// Otherwise a reduction and a vote of the warp a row find the largest and the lowest feature that has it, lane j row j's.
// (448 rows to 201088 logits, with quantising: 117 us; the reductions for every tile 150, of 64-bit keys 230.)
PE_DEV void mx_argmax(const MxMatmulArgs& a, int f, int t0, const float (&v)[16], const float* seen, int lane) {
  const int rows = min(16, a.n_rows - t0);
  const bool live = f < a.n_out;
  if (a.head.logits != nullptr && live) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < rows) a.head.logits[(size_t)(t0 + j) * a.n_out + f] = v[j];
  }
  bool raise = false;
  float size = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    raise |= !(v[j] < seen[j]);
    size = fmaxf(size, fabsf(v[j]));
  }
  if (!__any_sync(0xFFFFFFFFu, live && (raise || !(size < __uint_as_float(0x7F800000u))))) return;
  uint32_t top = 0, who = 0, largest = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t bits = __float_as_uint(v[j] + 0.0f);  // -0 -> +0, so equal values compare equal
    const uint32_t ord = live ? bits ^ ((uint32_t)((int32_t)bits >> 31) | 0x80000000u) : 0u;
    if (j < rows) largest = max(largest, bits & 0x7FFFFFFFu);
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, ord);
    const uint32_t w = __ballot_sync(0xFFFFFFFFu, live && ord == m);
    if (lane == j) {
      top = m;
      who = w;
    }
  }
  if (live && largest >= 0x7F800000u) set_err(a.err, PE_DEV_NONFINITE);
  const uint32_t first = (uint32_t)(f - lane + __ffs(who) - 1);
  const unsigned long long key = (unsigned long long)top << 32 | (unsigned long long)~first;
  if (lane < rows && who != 0 && key > __ldcg(a.head.keys + t0 + lane)) atomicMax(a.head.keys + t0 + lane, key);
}

// The rows' largest keys become draft tokens, by the CTA that finishes last (`threads` threads on barrier 1), which
// verifies them as well.
PE_DEV void mx_head_finish(const MxMatmulArgs& a, volatile int* last_flag, int thread, int threads) {
  __threadfence();
  named_bar_sync(1, threads);
  if (thread == 0) *last_flag = atomicAdd(a.head.done, 1) == (int)gridDim.x - 1;
  named_bar_sync(1, threads);
  if (!*last_flag) return;
  __threadfence();
  for (int t = thread; t < a.n_rows; t += threads) a.head.drafts[t] = argmax_key_index(__ldcg(a.head.keys + t));
  if (thread == 0) *a.head.done = 0;
  if (a.head.has_verify) {
    named_bar_sync(1, threads);
    for (int b = thread; b < a.head.verify.B; b += threads) verify_seq(a.head.verify, b);
  }
}

// While the MMAs run: what is added to the warp's chunks of 16 rows n = h, h + stride, ... comes to L2; row_of(n) is a
// chunk's first row, f0 the warp's first feature.
template <typename T, typename RowOf>
PE_DEV void mx_prefetch_addend(const MxMatmulArgs& a, int f0, int lane, int h, int chunks, int stride, RowOf row_of) {
  if (f0 >= a.n_out) return;
  for (int n = h; n < chunks; n += stride) {
    const int t = row_of(n) + (lane & 15);
    if (t < a.n_rows)
      prefetch_l2(static_cast<const T*>(a.add) + (long long)t * a.add_stride + min(f0 + (lane & 16), a.n_out - 1));
  }
}

// A feature's sums on their way out, chunk by chunk of 16 rows; what a chunk is added to is loaded while the one before it
// is stored.
template <typename T>
struct MxOut {
  const MxMatmulArgs& a;
  int f, lane;
  uint32_t old[16];
  PE_DEV MxOut(const MxMatmulArgs& args, int feature, int t0, const float*)
      : a(args), f(feature), lane(threadIdx.x & 31) {
    if (a.add != nullptr) mx_addend<T>(a, f, t0, old);
  }
  // Rows t0.. of the sums v (some: there are any); the next chunk's rows are t_next.. (-1: it is the last).
  PE_DEV void put(int t0, int t_next, bool some, float (&v)[16]) {
    uint32_t next[16];
    if (a.add != nullptr && t_next >= 0) mx_addend<T>(a, f, t_next, next);
    if (some) {
      if (a.add != nullptr)
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(sizeof(T) == 2 ? old[j] << 16 : old[j]);
      mx_store<T>(a, f, t0, v);
    }
    if (a.add != nullptr)
#pragma unroll
      for (int j = 0; j < 16; ++j) old[j] = next[j];
  }
};
template <>
struct MxOut<MxArgmax> {
  const MxMatmulArgs& a;
  int f, lane, row0;
  const float* seen;  // mx_seen's
  PE_DEV MxOut(const MxMatmulArgs& args, int feature, int first_row, const float* s)
      : a(args), f(feature), lane(threadIdx.x & 31), row0(first_row), seen(s) {}
  PE_DEV void put(int t0, int, bool some, float (&v)[16]) {
    if (some) mx_argmax(a, f, t0, v, seen + (t0 - row0), lane);
  }
};

}  // namespace pe
