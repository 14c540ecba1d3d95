// The product of two microscaled (MX) 4-bit matrices on the 5th-generation tensor cores:
//   y[r][f] = add[r][f] + sum_k x[r][k] w[f][k]
// with tcgen05.mma kind::mxf4: 4-bit operands in shared memory, their scales in tensor memory, fp32 accumulators.
//
// Weights sit on the MMA's M side (128 rows of w, one record high), rows of x on its N side, so that a few rows read
// every weight byte once.  The records of pe_mx.cuh are what a stage of the pipeline holds as it is: a stage's weights are
// one contiguous copy of `ka` records, codes in core-matrix order (K-major, no swizzle: 128 bytes from one 16-byte
// column of eight rows to the next, 512 to the next eight rows) and scales in the order in which tcgen05.cp spreads them
// over tensor memory (32 lanes x 4 columns for the 128 rows' four blocks each, repeated in every lane quarter).
//
// Many rows: tiles of 128 x 256, whose MMAs read a stage's weights from shared memory once for both halves (4099 x 2048 to
// 12288 features 76.8 -> 52.9 us; pairs of CTAs on 256 x 256 took 66, a stage's hand-over between them half a microsecond).
//
// With fewer tiles than SMs a cluster of CTAs shares a tile: each takes an equal part of its pieces along k, and the
// partial sums meet in shared memory over the cluster, each CTA summing its share of the columns in rank order, so the
// result does not depend on scheduling, and the call needs no workspace and no second kernel.
#include <algorithm>
#include <type_traits>

#include "pe_internal.h"
#include "pe_mx.cuh"

namespace pe {

namespace {

constexpr uint32_t kMxgCtrl = 1024;  // barriers, tensor-memory slot, flags
constexpr int kMxgThreads = 32 * 12;

// Where a tile's rows of x come from: with each stage, as records beside the weights' (128 rows or, wide, 256); or once,
// into shared memory for all of a CTA's tiles, as they are in 4 bits or quantised there from rows of bf16 or fp32.
enum MxSrc : int { SRC_STAGES = 0, SRC_WIDE = 1, SRC_RECORDS = 2, SRC_BF16 = 3, SRC_F32 = 4 };

// Pieces of a stage.  A copy takes the thread that issues it 40 ns and a stage's round trip through the ring about a
// microsecond, so stages are large and weights, x, and either half of a wide x have a thread each.
template <int SRC>
constexpr int kMxgKa = SRC == SRC_WIDE ? 2 : 4;

// Tensor memory: two accumulators, the stages' scales, and the scales of x where it is kept (four columns a piece).
// Wide: two accumulators of 256 columns that share 96, and four stages' scales (12 columns a piece) at the end; the
// epilogue empties the shared columns first, after which the next unit's MMAs may start.
struct MxPlan {
  int pieces, n_f, n_t, bn, cluster, stages, grid, src;
  int acc_stride, scale_col, x_col;
  uint32_t x_piece, stage_bytes, ring_bytes, x_bytes;
  size_t smem;
};
constexpr int kMxgKeepRows = 64;             // rows of x that are kept at most (accumulators of 64 columns)
constexpr int kMxgKeepPieces = 64;           // pieces of x that are kept at most (256 columns of scales)
constexpr uint32_t kMxgKeepBytes = 96 * 1024;
constexpr uint32_t kMxgCodes = 16 * kMxGroup;  // a record's codes
constexpr int kWideStages = 4;
constexpr int kWideShared = kWideStages * 2 * 12;  // columns that wide accumulators share
constexpr int kWideOdd = 512 - kWideShared - 256;  // first column of odd units' accumulator
static_assert(kWideOdd + kWideShared == 256 && kWideShared % 16 == 0, "whole chunks are shared");

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
PE_DEV void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

struct MxUnit {
  int tile_f, tile_t, row0, cols;
};
template <int SRC>
PE_DEV MxUnit mx_unit(const MxMatmulArgs& a, const MxPlan& p, int u) {
  MxUnit w;
  w.tile_t = u % p.n_t;  // a weight tile's row tiles run side by side (its records come from L2)
  w.tile_f = u / p.n_t;
  w.row0 = w.tile_t * (SRC == SRC_WIDE ? 2 : 1) * kMxPiece;
  w.cols = min(p.bn, (a.n_rows - w.row0 + 15) & ~15);
  return w;
}

// Rows of x into shared memory in 4 bits: pieces p0..p1 - 1 of all bn rows, x_piece bytes each (a record's scales and its
// first rows), by `warps` warps of which this is the w-th.  Rows beyond the last become zeros.
PE_DEV void keep_records(const MxMatmulArgs& a, const MxPlan& p, uint8_t* xs, int p0, int p1, int w, int warps, int lane) {
  const uint32_t chunks = p.x_piece / 16;
  for (int k = p0 + w; k < p1; k += warps) {
    const uint8_t* src = a.x + (size_t)k * kMxRecord;
    const uint32_t dst = smem_u32(xs + (size_t)(k - p0) * p.x_piece);
    for (uint32_t c = lane; c < chunks; c += 32)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * c), "l"(src + 16 * c) : "memory");
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}
template <typename T>
PE_DEV void keep_rows(const MxMatmulArgs& a, const MxPlan& p, uint8_t* xs, int p0, int p1, int w, int warps, int lane) {
  constexpr int N = sizeof(T) == 2 ? 2 : 1;  // units of eight rows of a piece whose loads a warp has in flight
  const int groups = p.bn / 8, units = groups * (p1 - p0), quarter = lane & 3;
  bool bad = false;
  for (int u0 = w; u0 < units; u0 += N * warps) {
    float x[N][4][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = u0 + i * warps, g = u % groups, k = p0 + u / groups, row = g * 8 + (lane >> 2);
      const bool live = u < units && row < a.n_rows;
      const T* src = static_cast<const T*>(a.rows) + (long long)row * a.rows_stride + k * kMxPiece + quarter * 8;
      const int left = a.width - k * kMxPiece - quarter * 8;
      if (live && left >= kMxPiece - quarter * 8) {
#pragma unroll
        for (int b = 0; b < 4; ++b) get8(src + b * kMxBlock, x[i][b]);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            x[i][b][e] = live && b * kMxBlock + e < left ? to_float<T>(src[b * kMxBlock + e]) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = u0 + i * warps;
      if (u >= units) break;
      const int g = u % groups, r = g * 8 + (lane >> 2);
      uint8_t* out = xs + (size_t)(u / groups) * p.x_piece;
      uint32_t s4 = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t codes, scale;
        bad |= mx_round8(x[i][b], codes, scale);
        s4 |= scale << (8 * b);
        reinterpret_cast<uint32_t*>(out + mx_code_at(r, b))[quarter] = codes;
      }
      if (quarter == 0) *reinterpret_cast<uint32_t*>(out + mx_scale_at(r, 0)) = s4;
    }
  }
  if (bad) set_err(a.err, PE_DEV_NONFINITE);
}

// What is added to 16 columns (rows t0.. of y) of feature f.
template <typename T>
PE_DEV void mx_addend(const MxMatmulArgs& a, int f, int t0, float (&old)[16]) {
  const T* add = static_cast<const T*>(a.add) + (long long)t0 * a.add_stride + f;
  const int n = f < a.n_out ? a.n_rows - t0 : 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) old[j] = j < n ? to_float<T>(add[(long long)j * a.add_stride]) : 0.f;
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

// 16 rows of x (from t0 on) of feature f: the warp's largest keys join the rows' own.
PE_DEV void mx_argmax(const MxMatmulArgs& a, int f, int t0, const float (&v)[16], int lane) {
  const int t = t0 + (lane >> 1);
  const bool mine = (lane & 1) == 0 && t < a.n_rows;
  // an older key at worst: few of a row's tiles raise its maximum, and the rest need no atomic
  const unsigned long long seen = mine ? __ldcg(a.head.keys + t) : 0ull;
  unsigned long long k[16];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const bool live = f < a.n_out && t0 + j < a.n_rows;
    bad |= live && !isfinite(v[j]);
    k[j] = live ? argmax_key(v[j], (uint32_t)f) : 0ull;
  }
  if (bad) set_err(a.err, PE_DEV_NONFINITE);
  if (a.head.logits != nullptr) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (f < a.n_out && t0 + j < a.n_rows) a.head.logits[(size_t)(t0 + j) * a.n_out + f] = v[j];
  }
  const unsigned long long top = argmax_reduce16(k, lane);
  if (mine && top > seen) atomicMax(a.head.keys + t, top);
}

// Roles: one thread copies weights (warp 0), one or two x (warps 2 and 3), one issues the MMAs (warp 1); the other warps
// bring in x where it is kept and write results.
template <typename T, int SRC>
__global__ void __launch_bounds__(kMxgThreads, 1) mx_gemm_kernel(const MxMatmulArgs a, const MxPlan p) {
  constexpr bool KEEP = SRC >= SRC_RECORDS, WIDE = SRC == SRC_WIDE, ARGMAX = std::is_same<T, MxArgmax>::value;
  constexpr int EW = kMxgThreads / 32 - 4, KA = kMxgKa<SRC>;
  // a stage: weight records, then x: records, or (wide) the codes of both halves of each piece and their scales
  constexpr uint32_t X_OFF = KA * kMxRecord, X_PIECE = WIDE ? 2 * kMxgCodes : kMxRecord;
  constexpr uint32_t X_SCALES = WIDE ? X_OFF + KA * X_PIECE : X_OFF, X_SCALE_PIECE = WIDE ? 2 * kMxScales : kMxRecord;
  // columns of a piece's scales, and of a stage's
  constexpr int PIECE_COLS = KEEP ? 4 : WIDE ? 12 : 8, STAGE_COLS = KA * PIECE_COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.stages;
  uint8_t* xs = smem + p.ring_bytes;  // x where it is kept
  uint8_t* ctrl = xs + p.x_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint64_t* kept = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kept + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued_max = abort_flag + 1;  // [4], by warp
  volatile int* last_flag = issued_max + 4;
  float* recv = reinterpret_cast<float*>(smem);  // clusters, after the MMAs: [rank][columns of this CTA][128]

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), KEEP ? 1 : WIDE ? 3 : 2);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(tfull + b), 1);
      mbar_init(smem_u32(tempty + b), EW);
    }
    mbar_init(smem_u32(kept), EW);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_trigger();

  const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / p.cluster, step = (int)gridDim.x / p.cluster, units = p.n_f * p.n_t;
  const int p0 = (int)((long long)p.pieces * rank / p.cluster), p1 = (int)((long long)p.pieces * (rank + 1) / p.cluster);
  const int drop = blockIdx.x == 0 ? a.drop_stage : -1;
  int issued = 0;  // stages that this thread began to fill

  if (warp == 0) {
    if (lane == 0) {
      // weights of a call whose x is kept are read once (a tile's only unit)
      const uint64_t pol = KEEP ? l2_policy_evict_first() : l2_policy_evict_last();
      fence_proxy_async_global();
      auto start = [&](int st, const uint8_t* src, int k) {
        const uint32_t bytes = (uint32_t)min(KA, p1 - k) * kMxRecord;
        mbar_expect_tx(smem_u32(full + st), bytes);
        bulk_g2s_hint(smem_u32(smem + (size_t)st * p.stage_bytes), src + (size_t)(k - p0) * kMxRecord, bytes,
                      smem_u32(full + st), pol);
      };
      auto tile = [&](int u) { return a.w + ((size_t)(u / p.n_t) * p.pieces + p0) * kMxRecord; };
      int s = 0, it = 0, npre = 0;
      uint32_t ph = 0;
      if (a.w_ready && first < units)  // the first unit's weights, where they are known to be there already
        for (int k = p0; k < p1 && npre < S; k += KA, ++npre)
          if (npre != drop) start(npre, tile(first), k);
      pdl_wait();
      fence_proxy_async_global();
      bool stop = false;
      for (int u = first; u < units && !stop; u += step) {
        const uint8_t* src = tile(u);
        for (int k = p0; k < p1; k += KA, ++it) {
          if (it >= S && !mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns)) {
            stop = true;
            break;
          }
          if (it >= npre && it != drop) start(s, src, k);
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      issued = it;
    }
  } else if (warp == 2 || warp == 3) {
    if (!KEEP && (warp == 2 || WIDE) && lane == 0) {
      const uint64_t pol = l2_policy_evict_last();
      const int half = warp - 2;
      pdl_wait();
      fence_proxy_async_global();
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool stop = false;
      for (int u = first; u < units && !stop; u += step) {
        const int row0 = mx_unit<SRC>(a, p, u).row0 + half * kMxPiece;
        const uint8_t* src = a.x + ((size_t)(row0 / kMxPiece) * p.pieces + p0) * kMxRecord;
        for (int k = p0; k < p1; k += KA, ++it) {
          if (it >= S && !mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns)) {
            stop = true;
            break;
          }
          const int n = min(KA, p1 - k);
          const uint32_t fb = smem_u32(full + s), dst = smem_u32(smem + (size_t)s * p.stage_bytes);
          const uint8_t* rec = src + (size_t)(k - p0) * kMxRecord;
          if (!WIDE) {
            // whole records: rows beyond the tile's columns come along unused
            mbar_expect_tx(fb, (uint32_t)n * kMxRecord);
            bulk_g2s_hint(dst + X_OFF, rec, (uint32_t)n * kMxRecord, fb, pol);
          } else if (row0 < a.n_rows) {
            mbar_expect_tx(fb, (uint32_t)n * kMxRecord);
#pragma unroll
            for (int j = 0; j < KA; ++j)
              if (j < n) {
                bulk_g2s_hint(dst + X_OFF + (uint32_t)(2 * j + half) * kMxgCodes, rec + j * kMxRecord + kMxScales, kMxgCodes,
                              fb, pol);
                bulk_g2s_hint(dst + X_SCALES + (uint32_t)(2 * j + half) * kMxScales, rec + j * kMxRecord, kMxScales, fb, pol);
              }
          } else {
            mbar_arrive(fb);  // no second half: the unit has 128 columns at most
          }
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      issued = it;
    }
  } else if (warp == 1) {
    // The warp stays together and one elected lane issues, with descriptors that advance by additions: operands of
    // these instructions are uniform, and made by one lane of a diverged warp they take twice the time of an MMA.
    pdl_wait();
    const uint32_t s0 = smem_u32(smem);
    const uint64_t w_codes = sdesc_core(s0 + kMxScales, 128, kMxGroup), w_scales = sdesc_core(s0, 16, 128);
    const uint64_t x_codes = sdesc_core(KEEP ? smem_u32(xs) + kMxScales : s0 + X_OFF + (WIDE ? 0 : kMxScales), 128, kMxGroup);
    const uint64_t x_scales = sdesc_core(KEEP ? smem_u32(xs) : s0 + X_SCALES, 16, 128);
    const uint32_t stage16 = p.stage_bytes >> 4, piece16 = KEEP ? p.x_piece >> 4 : X_PIECE / 16;
    int s = 0, i = 0;
    uint32_t ph = 0;
    bool stop = false;
    if (KEEP) {
      const bool ok = mbar_wait(smem_u32(kept), 0, a.err, abort_flag, a.wait_ns);
      stop = !__shfl_sync(0xFFFFFFFFu, ok, 0);
      tc_fence_after();
      if (!stop && elect_one())
        for (int k = 0; k < p1 - p0; ++k)
          tc_copy_scales(tmem + (uint32_t)(p.x_col + 4 * k), x_scales + (uint32_t)k * piece16);
      __syncwarp();
    }
    for (int u = first; u < units && !stop; u += step, ++i) {
      const int cols = mx_unit<SRC>(a, p, u).cols;
      const uint32_t idesc = idesc_mxf4(kMxPiece, cols);
      const int buf = i & 1;
      if (WIDE ? i >= 1 : i >= 2) {
        const bool ok = WIDE ? mbar_wait(smem_u32(tempty), (uint32_t)(i - 1) & 1u, a.err, abort_flag, a.wait_ns)
                             : mbar_wait(smem_u32(tempty + buf), (uint32_t)((i >> 1) - 1) & 1u, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(buf * p.acc_stride);
      for (int k = p0; k < p1; k += KA) {
        const bool ok = mbar_wait(smem_u32(full + s), ph, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const int n = p1 - k;  // pieces left
          const uint32_t at = (uint32_t)s * stage16;
          const uint64_t wc = w_codes + at, ws = w_scales + at;
          const uint64_t xc = x_codes + (KEEP ? (uint32_t)(k - p0) * piece16 : at), xsc = x_scales + at;
          const uint32_t sa = tmem + (uint32_t)(p.scale_col + s * STAGE_COLS);
          const uint32_t sb = KEEP ? tmem + (uint32_t)(p.x_col + 4 * (k - p0)) : sa + 4;
          constexpr int SB_PIECE = KEEP ? 4 : PIECE_COLS;
#pragma unroll
          for (int j = 0; j < KA; ++j)
            if (j < n) {
              tc_copy_scales(sa + j * PIECE_COLS, ws + j * (kMxRecord / 16));
              if (!KEEP) tc_copy_scales(sb + j * SB_PIECE, xsc + j * (X_SCALE_PIECE / 16));
              if (WIDE && cols > kMxPiece) tc_copy_scales(sb + j * SB_PIECE + 4, xsc + (j * X_SCALE_PIECE + kMxScales) / 16);
            }
#pragma unroll
          for (int j = 0; j < KA; ++j)
            if (j < n) {
              const uint64_t da = wc + j * (kMxRecord / 16), db = xc + (uint32_t)j * piece16;
              // 64 entries: two 16-byte columns, 256 bytes on
              tc_mma_mxf4(d, da, db, idesc, sa + j * PIECE_COLS, sb + j * SB_PIECE, (k > p0 || j > 0) ? 1u : 0u);
              tc_mma_mxf4(d, da + 16, db + 16, idesc | kScaleUpper, sa + j * PIECE_COLS, sb + j * SB_PIECE, 1u);
            }
          tc_commit(smem_u32(empty + s));
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (elect_one()) tc_commit(smem_u32(tfull + buf));
      __syncwarp();
    }
    // after a wait gave up: every MMA issued completes before the tensor memory is freed
    if (stop && i > 0)
      mbar_wait(smem_u32(tfull + ((i - 1) & 1)), (uint32_t)((i - 1) >> 1) & 1u, a.err, nullptr, a.wait_ns);
  } else {
    pdl_wait();
    if (KEEP) {
      if (SRC == SRC_RECORDS) keep_records(a, p, xs, p0, p1, warp - 4, EW, lane);
      if (SRC == SRC_BF16) keep_rows<__nv_bfloat16>(a, p, xs, p0, p1, warp - 4, EW, lane);
      if (SRC == SRC_F32) keep_rows<float>(a, p, xs, p0, p1, warp - 4, EW, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(kept));
    }
    const int q = warp & 3, h = (warp - 4) >> 2;
    const int r = q * 32 + lane;
    if (p.cluster == 1) {
      int i = 0;
      for (int u = first; u < units; u += step, ++i) {
        const MxUnit w = mx_unit<SRC>(a, p, u);
        const int buf = i & 1, f = w.tile_f * kMxPiece + r, chunks = w.cols / 16;
        // wide: the shared columns first, the last chunks of an even unit, the first of an odd one
        constexpr int ALL = WIDE ? 16 : 8, SHARED = kWideShared / 16;
        const int turn = WIDE && !buf ? ALL - SHARED : 0;
        auto row_of = [&](int n) { return w.row0 + ((n + turn) & (ALL - 1)) * 16; };
        if constexpr (!ARGMAX) {
          if (a.add != nullptr && f - lane < a.n_out)  // while the MMAs run: what is added comes to L2
            for (int n = h; n < ALL; n += EW / 4) {
              const int t = row_of(n) + (lane & 15);
              if (t < a.n_rows)
                prefetch_l2(static_cast<const T*>(a.add) + (long long)t * a.add_stride + min(f - lane + (lane & 16), a.n_out - 1));
            }
        }
        const bool ok =
            mbar_wait(smem_u32(tfull + buf), (uint32_t)(i >> 1) & 1u, a.err, abort_flag, a.wait_ns) && !*abort_flag;
        tc_fence_after();
        const uint32_t tl = tmem + (uint32_t)(buf * p.acc_stride) + ((uint32_t)(q * 32) << 16);
        float old[16];
        if constexpr (!ARGMAX) {
          if (a.add != nullptr && ok) mx_addend<T>(a, f, row_of(h), old);
        }
        for (int n = h; n < ALL; n += EW / 4) {
          if (WIDE && n >= SHARED && n - EW / 4 < SHARED) {  // this warp's shared chunks have left tensor memory
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(tempty));
          }
          const int c = (n + turn) & (ALL - 1), t0 = w.row0 + c * 16;
          float v[16];
          if constexpr (ARGMAX) {
            if (ok && c < chunks) {
              tmem_load16(tl + (uint32_t)(c * 16), v);
              mx_argmax(a, f, t0, v, lane);
            }
          } else {
            float next[16];
            if (a.add != nullptr && ok && n + EW / 4 < ALL) mx_addend<T>(a, f, row_of(n + EW / 4), next);
            if (ok && c < chunks) {
              tmem_load16(tl + (uint32_t)(c * 16), v);
              if (a.add != nullptr)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += old[j];
              mx_store<T>(a, f, t0, v);
            }
            if (a.add != nullptr)
#pragma unroll
              for (int j = 0; j < 16; ++j) old[j] = next[j];
          }
        }
        if (!WIDE) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(tempty + buf));
        }
      }
      if constexpr (ARGMAX) {
        const int thread = threadIdx.x - 128;
        __threadfence();
        named_bar_sync(1, 32 * EW);
        if (thread == 0) *last_flag = atomicAdd(a.head.done, 1) == (int)gridDim.x - 1;
        named_bar_sync(1, 32 * EW);
        if (*last_flag) {
          __threadfence();
          for (int t = thread; t < a.n_rows; t += 32 * EW) a.head.drafts[t] = argmax_key_index(__ldcg(a.head.keys + t));
          if (thread == 0) *a.head.done = 0;
          if (a.head.has_verify) {
            named_bar_sync(1, 32 * EW);
            for (int b = thread; b < a.head.verify.B; b += 32 * EW) verify_seq(a.head.verify, b);
          }
        }
      }
    } else {
      mbar_wait(smem_u32(tfull), 0, a.err, abort_flag, a.wait_ns);
      tc_fence_after();
    }
  }

  if constexpr (!ARGMAX)
  if (p.cluster > 1) {
    // the cluster's one unit: every CTA's MMAs are done (or given up), so the stages' memory takes the partial sums
    const MxUnit w = mx_unit<SRC>(a, p, first);
    const int share = w.cols / p.cluster;  // columns that each CTA sums
    __syncthreads();
    cluster_sync();
    if (warp >= 4 && !*abort_flag) {
      const int q = warp & 3, h = (warp - 4) >> 2, r = q * 32 + lane;
      const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
      for (int c = h; c < w.cols / 16; c += EW / 4) {
        float v[16];
        tmem_load16(tl + (uint32_t)(c * 16), v);
        int owner = c * 16 / share, col = c * 16 - owner * share;  // and on from there column by column
        uint32_t at = mapa_shared(smem_u32(recv + (size_t)(rank * share) * kMxPiece + r), (uint32_t)owner);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          st_cluster_f32(at + (uint32_t)(col * kMxPiece * 4), v[j]);
          if (++col == share) {
            col = 0;
            if (++owner < p.cluster)
              at = mapa_shared(smem_u32(recv + (size_t)(rank * share) * kMxPiece + r), (uint32_t)owner);
          }
        }
      }
      tc_fence_before();
    }
    __syncwarp();
    cluster_sync();  // every partial sum is where it is summed
    if (warp >= 4 && !*abort_flag) {
      const int r = (warp & 3) * 32 + lane, h = (warp - 4) >> 2;
      const int f = w.tile_f * kMxPiece + r, t0 = w.row0 + rank * share;
      if (f < a.n_out)
        for (int c = h; c < share && t0 + c < a.n_rows; c += EW / 4) {
          float part[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            part[k] = k < p.cluster ? recv[(size_t)(k * share + c) * kMxPiece + r] : 0.f;
          float v = part[0];
#pragma unroll
          for (int k = 1; k < 8; ++k)
            if (k < p.cluster) v += part[k];
          if (a.add != nullptr)
            v += to_float<T>(static_cast<const T*>(a.add)[(long long)(t0 + c) * a.add_stride + f]);
          static_cast<T*>(a.y)[(long long)(t0 + c) * a.y_stride + f] = from_float<T>(v);
        }
    }
  }

  __syncthreads();
  if (*abort_flag) {
    // After a wait gave up no copy may stay in flight into this CTA's shared memory: threads that stopped earlier than
    // others arrive, without a copy, for the stages they left out, so that every stage begun completes.
    const bool copier = lane == 0 && (warp == 0 || (!KEEP && (warp == 2 || (WIDE && warp == 3))));
    if (copier) issued_max[warp] = issued;
    __syncthreads();
    const int last = KEEP ? issued_max[0] : max(issued_max[0], max(issued_max[2], WIDE ? issued_max[3] : 0));
    if (copier) {
      if (warp == 0 && drop >= 0 && drop < issued) mbar_arrive(smem_u32(full + drop % S));
      for (int i = issued; i < last; ++i) mbar_arrive(smem_u32(full + i % S));
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = max(last - S, 0); i < last; ++i)
        mbar_wait(smem_u32(full + (i % S)), (uint32_t)(i / S) & 1u, a.err, nullptr, a.wait_ns);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Whether x can be kept in shared memory with its scales in tensor memory: one row tile, few rows, `pieces` of a CTA.
bool keeps_x(int n_rows, int pieces) {
  const int bn = (n_rows + 15) & ~15;
  return bn <= kMxgKeepRows && pieces <= kMxgKeepPieces &&
         (size_t)pieces * (kMxScales + 64u * (uint32_t)bn) <= kMxgKeepBytes;
}

MxPlan plan_mx(const MxMatmulArgs& a, int sms) {
  MxPlan p{};
  p.pieces = (a.width + kMxPiece - 1) / kMxPiece;
  p.n_f = (a.n_out + kMxPiece - 1) / kMxPiece;
  p.n_t = (a.n_rows + kMxPiece - 1) / kMxPiece;
  p.bn = std::min(kMxPiece, (a.n_rows + 15) & ~15);
  long long units = (long long)p.n_f * p.n_t;
  p.cluster = 1;
  // (the LM head's sums are looked at as they are: no shares)
  while (a.head.keys == nullptr && p.cluster < 8 && units * p.cluster * 2 <= sms && p.pieces >= p.cluster * 4) p.cluster *= 2;
  const int part = (p.pieces + p.cluster - 1) / p.cluster;
  const bool keep = keeps_x(a.n_rows, part);
  // a wide tile takes in 3 records a piece for the 4 of two tiles, and reads its weights from shared memory once: about
  // three quarters of their time
  const long long wide_units = (long long)p.n_f * ((p.n_t + 1) / 2);
  const bool wide = !keep && p.n_t > 1 && (wide_units + sms - 1) / sms * p.pieces * 3 < (units + sms - 1) / sms * part * 2;
  p.src = wide ? SRC_WIDE : !keep ? SRC_STAGES : a.rows == nullptr ? SRC_RECORDS : a.rows_type == PE_BF16 ? SRC_BF16 : SRC_F32;
  if (wide) {
    p.cluster = 1;
    p.n_t = (p.n_t + 1) / 2;
    p.bn = 2 * kMxPiece;
    units = wide_units;
  }
  const int ka = wide ? kMxgKa<SRC_WIDE> : kMxgKa<SRC_STAGES>;
  p.x_piece = keep ? kMxScales + 64u * (uint32_t)p.bn : kMxRecord;
  p.x_bytes = keep ? (uint32_t)part * p.x_piece : 0;
  p.stage_bytes = (uint32_t)ka * (keep ? 1 : wide ? 3 : 2) * kMxRecord;
  p.stages = wide ? kWideStages : (int)((kTcSmemOptIn - 128 - (long long)kMxgCtrl - p.x_bytes) / p.stage_bytes);
  if (p.cluster > 1) p.stages = std::min(p.stages, (part + ka - 1) / ka);
  p.ring_bytes = (uint32_t)p.stages * p.stage_bytes;
  if (p.cluster > 1) p.ring_bytes = std::max(p.ring_bytes, (uint32_t)p.bn * kMxPiece * 4u);
  p.acc_stride = wide ? kWideOdd : keep ? kMxgKeepRows : kMxPiece;
  p.scale_col = wide ? 512 - kWideShared : 2 * p.acc_stride;
  p.x_col = 256;
  p.grid = p.cluster * (int)std::min<long long>(units, p.cluster > 1 ? units : sms);
  p.smem = 128 + (size_t)p.ring_bytes + p.x_bytes + kMxgCtrl;
  return p;
}

template <typename T, int SRC>
cudaError_t launch_src(const MxMatmulArgs& a, const MxPlan& p, cudaStream_t s) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(mx_gemm_kernel<T, SRC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOptIn);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kMxgThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T, SRC>, a, p);
}

template <typename T>
cudaError_t launch_typed(const MxMatmulArgs& a, int sms, cudaStream_t s) {
  const MxPlan p = plan_mx(a, sms);
  switch (p.src) {
    case SRC_STAGES: return launch_src<T, SRC_STAGES>(a, p, s);
    case SRC_WIDE: return launch_src<T, SRC_WIDE>(a, p, s);
    case SRC_RECORDS: return launch_src<T, SRC_RECORDS>(a, p, s);
    case SRC_BF16: return launch_src<T, SRC_BF16>(a, p, s);
    case SRC_F32: return launch_src<T, SRC_F32>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Where a CTA has no more than 12,288 entries of x: it rounds them in less than a launch before the product takes (8 rows
// of 256: 3.7 against 4.6 us; 14 rows of 2880: 12.5 against 9.5 us).
bool mx_matmul_quantises(int n_rows, int n_out, int width, bool head, int sms) {
  MxMatmulArgs a{};
  unsigned long long key;
  a.head.keys = head ? &key : nullptr;
  a.n_rows = n_rows; a.n_out = n_out; a.width = width;
  const MxPlan p = plan_mx(a, sms);
  return p.src == SRC_RECORDS && (long long)p.bn * ((p.pieces + p.cluster - 1) / p.cluster) * kMxPiece <= 12288;
}

cudaError_t launch_mx_matmul(const MxMatmulArgs& a, pe_dtype dt, int sms, cudaStream_t s) {
  if (a.head.keys != nullptr) return launch_typed<MxArgmax>(a, sms, s);
  return dt == PE_BF16 ? launch_typed<__nv_bfloat16>(a, sms, s) : launch_typed<float>(a, sms, s);
}

}  // namespace pe
