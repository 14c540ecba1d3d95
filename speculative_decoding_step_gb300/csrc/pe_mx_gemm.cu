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
// With fewer tiles than SMs a cluster of CTAs shares a tile: each takes an equal part of its pieces along k, and the
// partial sums meet in shared memory over the cluster, each CTA summing its share of the columns in rank order, so the
// result does not depend on scheduling, and the call needs no workspace and no second kernel.
#include <algorithm>

#include "pe_internal.h"
#include "pe_mx.cuh"

namespace pe {

namespace {

constexpr uint32_t kMxgCtrl = 1024;  // barriers, tensor-memory slot, flags
constexpr int kMxgThreads = 64 + 32 * 8;

// Where a tile's rows of x come from: with each stage, as whole records beside the weights'; or once, into shared memory
// for all of a CTA's tiles, as they are in 4 bits or quantised there from rows of bf16 or fp32.
enum MxSrc : int { SRC_STAGES = 0, SRC_RECORDS = 1, SRC_BF16 = 2, SRC_F32 = 3 };

// An SM's bulk copies run one after another at about 90 ns + 4.2 ns a KB (measured: 107 GB/s an SM with copies of two
// records, 148 with four), so a stage is one copy of four weight records, and one of four x records where x is not kept.
constexpr int kMxgKa = 4;

// Tensor memory: two accumulators, the stages' scales, and the scales of x where it is kept (four columns a piece).
struct MxPlan {
  int pieces, n_f, n_t, bn, cluster, stages, grid, src;
  int acc_stride, scale_col, scale_stage, x_col;
  uint32_t x_piece, x_off, stage_bytes, ring_bytes, x_bytes;
  size_t smem;
};
constexpr int kMxgKeepRows = 64;             // rows of x that are kept at most (accumulators of 64 columns)
constexpr int kMxgKeepPieces = 64;           // pieces of x that are kept at most (256 columns of scales)
constexpr uint32_t kMxgKeepBytes = 96 * 1024;

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
PE_DEV void tc_copy_scales(uint32_t dst, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(sdesc_core(saddr, 16, 128))
               : "memory");
}
PE_DEV void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

struct MxUnit {
  int tile_f, tile_t, cols;
};
PE_DEV MxUnit mx_unit(const MxMatmulArgs& a, const MxPlan& p, int u) {
  MxUnit w;
  w.tile_t = u % p.n_t;  // a weight tile's row tiles run side by side (its records come from L2)
  w.tile_f = u / p.n_t;
  w.cols = min(p.bn, (a.n_rows - w.tile_t * kMxPiece + 15) & ~15);
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

// Adds and stores up to 16 columns (rows t0.. of y) of feature f.
template <typename T>
PE_DEV void mx_store(const MxMatmulArgs& a, int f, int t0, int n, const float (&v)[16]) {
  if (f >= a.n_out) return;
  T* y = static_cast<T*>(a.y) + (long long)t0 * a.y_stride + f;
  if (a.add != nullptr) {
    const T* add = static_cast<const T*>(a.add) + (long long)t0 * a.add_stride + f;
    float old[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) old[j] = j < n ? to_float<T>(add[(long long)j * a.add_stride]) : 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) y[(long long)j * a.y_stride] = from_float<T>(v[j] + old[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) y[(long long)j * a.y_stride] = from_float<T>(v[j]);
  }
}

// Roles: warp 0 copies (one elected lane issues), warp 1 issues the MMAs, the others bring in x where it is kept and write
// results.
template <typename T, int SRC>
__global__ void __launch_bounds__(kMxgThreads, 1) mx_gemm_kernel(const MxMatmulArgs a, const MxPlan p) {
  constexpr bool KEEP = SRC != SRC_STAGES;
  constexpr int EW = kMxgThreads / 32 - 2;
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
  float* recv = reinterpret_cast<float*>(smem);  // clusters, after the MMAs: [rank][columns of this CTA][128]

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
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
  int issued = 0;  // stages that the copying warp issued

  if (warp == 0) {
    // weights of a call whose x is kept are read once (a tile's only unit)
    const uint64_t pol_w = KEEP ? l2_policy_evict_first() : l2_policy_evict_last(), pol_x = l2_policy_evict_last();
    fence_proxy_async_global();
    int s = 0, it = 0, npre = 0;
    uint32_t ph = 0;
    auto start_w = [&](int st, int tile_f, int k) {
      const uint32_t n = (uint32_t)min(kMxgKa, p1 - k);
      mbar_expect_tx(smem_u32(full + st), n * kMxRecord * (KEEP ? 1u : 2u));
      bulk_g2s_hint(smem_u32(smem + (size_t)st * p.stage_bytes), a.w + ((size_t)tile_f * p.pieces + k) * kMxRecord,
                    n * kMxRecord, smem_u32(full + st), pol_w);
    };
    if (a.w_ready && first < units) {  // the first unit's weights, where they are known to be there already
      const MxUnit w = mx_unit(a, p, first);
      for (int k = p0; k < p1 && npre < S; k += kMxgKa, ++npre)
        if (npre != drop && elect_one()) start_w(npre, w.tile_f, k);
    }
    __syncwarp();
    pdl_wait();
    fence_proxy_async_global();
    bool stop = false;
    for (int u = first; u < units && !stop; u += step) {
      const MxUnit w = mx_unit(a, p, u);
      for (int k = p0; k < p1; k += kMxgKa, ++it) {
        if (it >= S) {
          const bool ok = mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns);
          if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
            stop = true;
            break;
          }
        }
        if (it != drop && elect_one()) {
          if (it >= npre) start_w(s, w.tile_f, k);
          if (!KEEP)  // whole records: rows beyond the tile's columns come along unused
            bulk_g2s_hint(smem_u32(smem + (size_t)s * p.stage_bytes) + p.x_off,
                          a.x + ((size_t)w.tile_t * p.pieces + k) * kMxRecord, (uint32_t)min(kMxgKa, p1 - k) * kMxRecord,
                          smem_u32(full + s), pol_x);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    issued = it;
  } else if (warp == 1) {
    pdl_wait();
    int s = 0, i = 0;
    uint32_t ph = 0;
    bool stop = false;
    if (KEEP) {
      const bool ok = mbar_wait(smem_u32(kept), 0, a.err, abort_flag, a.wait_ns);
      stop = !__shfl_sync(0xFFFFFFFFu, ok, 0);
      tc_fence_after();
      if (!stop && elect_one())
        for (int k = 0; k < p1 - p0; ++k)
          tc_copy_scales(tmem + (uint32_t)(p.x_col + 4 * k), smem_u32(xs + (size_t)k * p.x_piece));
      __syncwarp();
    }
    for (int u = first; u < units && !stop; u += step, ++i) {
      const MxUnit w = mx_unit(a, p, u);
      const uint32_t idesc = idesc_mxf4(kMxPiece, w.cols);
      const int buf = i & 1;
      if (i >= 2) {
        const bool ok = mbar_wait(smem_u32(tempty + buf), (uint32_t)((i >> 1) - 1) & 1u, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(buf * p.acc_stride);
      for (int k = p0; k < p1; k += kMxgKa) {
        const bool ok = mbar_wait(smem_u32(full + s), ph, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const int n = min(kMxgKa, p1 - k);
          const uint32_t sw = smem_u32(smem + (size_t)s * p.stage_bytes);
          const uint32_t sx = KEEP ? smem_u32(xs + (size_t)(k - p0) * p.x_piece) : sw + p.x_off;
          const uint32_t sc = tmem + (uint32_t)(p.scale_col + s * p.scale_stage);
          for (int j = 0; j < n; ++j) {
            tc_copy_scales(sc + (uint32_t)(4 * j), sw + (uint32_t)j * kMxRecord);
            if (!KEEP) tc_copy_scales(sc + (uint32_t)(4 * kMxgKa + 4 * j), sx + (uint32_t)j * p.x_piece);
          }
          for (int j = 0; j < n; ++j) {
            const uint64_t da = sdesc_core(sw + (uint32_t)j * kMxRecord + kMxScales, 128, kMxGroup);
            const uint64_t db = sdesc_core(sx + (uint32_t)j * p.x_piece + kMxScales, 128, kMxGroup);
            const uint32_t sa = sc + (uint32_t)(4 * j);
            const uint32_t sb = KEEP ? tmem + (uint32_t)(p.x_col + 4 * (k - p0 + j)) : sa + 4 * kMxgKa;
            // 64 entries: two 16-byte columns, 256 bytes on
            tc_mma_mxf4(d, da, db, idesc, sa, sb, (k > p0 || j > 0) ? 1u : 0u);
            tc_mma_mxf4(d, da + 16, db + 16, idesc | kScaleUpper, sa, sb, 1u);
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
      if (SRC == SRC_RECORDS) keep_records(a, p, xs, p0, p1, warp - 2, EW, lane);
      if (SRC == SRC_BF16) keep_rows<__nv_bfloat16>(a, p, xs, p0, p1, warp - 2, EW, lane);
      if (SRC == SRC_F32) keep_rows<float>(a, p, xs, p0, p1, warp - 2, EW, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(kept));
    }
    const int q = warp & 3, h = (warp - 2) >> 2;
    const int r = q * 32 + lane;
    if (p.cluster == 1) {
      int i = 0;
      for (int u = first; u < units; u += step, ++i) {
        const MxUnit w = mx_unit(a, p, u);
        const int buf = i & 1;
        const bool ok =
            mbar_wait(smem_u32(tfull + buf), (uint32_t)(i >> 1) & 1u, a.err, abort_flag, a.wait_ns) && !*abort_flag;
        tc_fence_after();
        const uint32_t tl = tmem + (uint32_t)(buf * p.acc_stride) + ((uint32_t)(q * 32) << 16);
        if (ok)
          for (int c = h; c < w.cols / 16; c += EW / 4) {
            float v[16];
            tmem_load16(tl + (uint32_t)(c * 16), v);
            const int t0 = w.tile_t * kMxPiece + c * 16;
            mx_store<T>(a, w.tile_f * kMxPiece + r, t0, min(16, a.n_rows - t0), v);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(tempty + buf));
      }
    } else {
      mbar_wait(smem_u32(tfull), 0, a.err, abort_flag, a.wait_ns);
      tc_fence_after();
    }
  }

  if (p.cluster > 1) {
    // the cluster's one unit: every CTA's MMAs are done (or given up), so the stages' memory takes the partial sums
    const MxUnit w = mx_unit(a, p, first);
    const int share = w.cols / p.cluster;  // columns that each CTA sums
    __syncthreads();
    cluster_sync();
    if (warp >= 2 && !*abort_flag) {
      const int q = warp & 3, h = (warp - 2) >> 2, r = q * 32 + lane;
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
    if (warp >= 2 && !*abort_flag) {
      const int r = (warp & 3) * 32 + lane, h = (warp - 2) >> 2;
      const int f = w.tile_f * kMxPiece + r, t0 = w.tile_t * kMxPiece + rank * share;
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
  // after a wait gave up: no copy stays in flight into this CTA's shared memory
  if (warp == 0 && *abort_flag) {
    for (int i = issued > S ? issued - S : 0; i < issued; ++i)
      if (i != drop) mbar_wait(smem_u32(full + (i % S)), (uint32_t)(i / S) & 1u, a.err, nullptr, a.wait_ns);
    __syncwarp();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================================= CTA pairs
//
// Many rows: a pair of CTAs multiplies 256 weight rows by 256 rows of x in one MMA (cta_group::2), each CTA holding 128 rows
// of either and taking in half the bytes per flop of a CTA by itself.  Each CTA's copies complete on its own barrier; the
// peer's second warp passes each stage's completion on to the leader, which issues every MMA.  Scales of all 256 rows of x
// go to both CTAs' tensor memory.
//
// Tensor memory, 512 columns: two accumulators of 256 that share 48 columns, and four pieces' scales (12 columns each) at
// the end.  The epilogue empties the shared columns first, after which the next unit's MMAs may start.

constexpr int kPairRows = 2 * kMxPiece;
constexpr int kPairKa = 4;                                     // pieces per stage
constexpr uint32_t kPairHalf = kPairKa * kMxRecord;            // a stage's records of w, and of x
constexpr uint32_t kPairScale = 2 * kMxScales;                 // scales of a piece's 256 rows of x
constexpr uint32_t kPairStage = 2 * kPairHalf + kPairKa * kPairScale;
constexpr int kPairStages = (kTcSmemOptIn - 128 - (int)kMxgCtrl) / (int)kPairStage;
constexpr int kPairScaleCols = 12;                             // of a piece: four for w, eight for x
constexpr int kPairSlots = 2;                                  // stages whose scales have columns
constexpr int kPairShared = kPairSlots * kPairKa * kPairScaleCols;  // columns that the accumulators share
constexpr int kPairOdd = 512 - kPairShared - 256;              // first column of odd units' accumulator
constexpr int kPairThreads = 32 * 11;
static_assert(kPairStages >= 3 && kPairOdd + kPairShared == 256 && kPairShared % 16 == 0, "whole chunks are shared");

PE_DEV void tc_mma_mxf4_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t a_scale,
                             uint32_t b_scale, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(a_scale), "r"(b_scale), "r"(accumulate)
      : "memory");
}
// In both CTAs, each from its own shared memory.
PE_DEV void tc_copy_scales_pair(uint32_t dst, uint32_t saddr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(sdesc_core(saddr, 16, 128))
               : "memory");
}

struct MxPairPlan {
  int pieces, n_f, n_t, units;  // tiles of 256 x 256
  int blocks_f, blocks_t;       // records of 128 rows
};

// A record of x of unit u: piece k of the tile's first or second 128 rows.  Rows beyond the last block's stand in for
// themselves (their results are not stored).
PE_DEV const uint8_t* x_record(const MxMatmulArgs& a, const MxPairPlan& p, int u, int k, int half) {
  const int b = min(2 * (u % p.n_t) + half, p.blocks_t - 1);
  return a.x + ((size_t)b * p.pieces + k) * kMxRecord;
}

template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1) mx_gemm_pair_kernel(const MxMatmulArgs a, const MxPairPlan p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int S = kPairStages, EW = 8;
  uint8_t* ctrl = smem + (size_t)S * kPairStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);  // this CTA's copies
  uint64_t* peer = full + S;                           // leader: the other CTA's are there
  uint64_t* empty = peer + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;  // leader: the columns that the next unit needs are empty
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 2);  // the copies' and the scales'
      mbar_init(smem_u32(peer + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    mbar_init(smem_u32(tfull + 1), 1);
    mbar_init(smem_u32(tempty), 2 * EW);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_cg2(smem_u32(tmem_slot), 512);
    tmem_relinquish_cg2();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cluster_sync();  // both CTAs' barriers are initialised before any arrival crosses over
  pdl_trigger();

  const int first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;
  const int drop = blockIdx.x == 0 ? a.drop_stage : -1;
  int issued = 0;

  if (warp == 0) {
    const uint64_t pol = l2_policy_evict_last();
    fence_proxy_async_global();
    int s = 0, it = 0, npre = 0;
    uint32_t ph = 0;
    // records of this CTA; blocks beyond the last stand in for themselves (their results are not stored)
    auto w_at = [&](int u, int k) {
      const int b = min(2 * (u / p.n_t) + (int)rank, p.blocks_f - 1);
      return a.w + ((size_t)b * p.pieces + k) * kMxRecord;
    };
    auto x_at = [&](int u, int k, int half) { return x_record(a, p, u, k, half); };
    auto start_w = [&](int st, int u, int k) {
      const uint32_t n = (uint32_t)min(kPairKa, p.pieces - k);
      mbar_expect_tx(smem_u32(full + st), 2 * n * kMxRecord);
      bulk_g2s_hint(smem_u32(smem + (size_t)st * kPairStage), w_at(u, k), n * kMxRecord, smem_u32(full + st), pol);
    };
    if (a.w_ready && first < p.units)
      for (int k = 0; k < p.pieces && npre < S; k += kPairKa, ++npre)
        if (npre != drop && elect_one()) start_w(npre, first, k);
    __syncwarp();
    pdl_wait();
    fence_proxy_async_global();
    bool stop = false;
    for (int u = first; u < p.units && !stop; u += step)
      for (int k = 0; k < p.pieces; k += kPairKa, ++it) {
        if (it >= S) {
          const bool ok = mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns);
          if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
            stop = true;
            break;
          }
        }
        if (it != drop && elect_one()) {
          if (it >= npre) start_w(s, u, k);
          bulk_g2s_hint(smem_u32(smem + (size_t)s * kPairStage) + kPairHalf, x_at(u, k, (int)rank),
                        (uint32_t)min(kPairKa, p.pieces - k) * kMxRecord, smem_u32(full + s), pol);
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    issued = it;
  } else if (warp == 1) {
    pdl_wait();
    int s = 0, it = 0, i = 0;
    uint32_t ph = 0;
    bool stop = false;
    const uint32_t idesc = idesc_mxf4(2 * kMxPiece, kPairRows);
    for (int u = first; u < p.units && !stop; u += step, ++i) {
      if (rank == 0 && i >= 1) {
        const bool ok = mbar_wait_cluster(smem_u32(tempty), (uint32_t)(i - 1) & 1u, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
      }
      tc_fence_after();
      const uint32_t d = tmem + ((i & 1) ? (uint32_t)kPairOdd : 0u);
      for (int k = 0; k < p.pieces; k += kPairKa, ++it) {
        bool ok = mbar_wait(smem_u32(full + s), ph, a.err, abort_flag, a.wait_ns);
        if (rank == 0) {
          ok = ok && mbar_wait_cluster(smem_u32(peer + s), ph, a.err, abort_flag, a.wait_ns);
          // the scales go where those of two stages ago were: that stage's MMAs are done
          const int before = it - kPairSlots;
          if (before >= 0)
            ok = ok && mbar_wait(smem_u32(empty + before % S), (uint32_t)(before / S) & 1u, a.err, abort_flag, a.wait_ns);
        }
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
        if (rank != 0) {
          if (elect_one()) mbar_arrive_cluster(mapa_shared(smem_u32(peer + s), 0));
        } else {
          tc_fence_after();
          if (elect_one()) {
            const int n = min(kPairKa, p.pieces - k);
            const uint32_t sw = smem_u32(smem + (size_t)s * kPairStage), sx = sw + kPairHalf, ss = sx + kPairHalf;
            const uint32_t sc = tmem + 512 - kPairShared + (uint32_t)(it % kPairSlots * kPairKa * kPairScaleCols);
            for (int j = 0; j < n; ++j) {
              const uint32_t c = sc + (uint32_t)(j * kPairScaleCols);
              tc_copy_scales_pair(c, sw + (uint32_t)j * kMxRecord);
              tc_copy_scales_pair(c + 4, ss + (uint32_t)j * kPairScale);
              tc_copy_scales_pair(c + 8, ss + (uint32_t)j * kPairScale + kMxScales);
            }
            for (int j = 0; j < n; ++j) {
              const uint64_t da = sdesc_core(sw + (uint32_t)j * kMxRecord + kMxScales, 128, kMxGroup);
              const uint64_t db = sdesc_core(sx + (uint32_t)j * kMxRecord + kMxScales, 128, kMxGroup);
              const uint32_t c = sc + (uint32_t)(j * kPairScaleCols);
              tc_mma_mxf4_pair(d, da, db, idesc, c, c + 4, (k > 0 || j > 0) ? 1u : 0u);
              tc_mma_mxf4_pair(d, da + 16, db + 16, idesc | kScaleUpper, c, c + 4, 1u);
            }
            tc_commit_pair(smem_u32(empty + s));
          }
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (rank == 0 && elect_one()) tc_commit_pair(smem_u32(tfull + (i & 1)));
      __syncwarp();
    }
    // after a wait gave up: every MMA issued completes before the tensor memory is freed
    if (rank == 0 && stop && i > 0)
      mbar_wait(smem_u32(tfull + ((i - 1) & 1)), (uint32_t)((i - 1) >> 1) & 1u, a.err, nullptr, a.wait_ns);
  } else if (warp == 2) {
    // scales of x, 512 bytes of either half of a piece's rows: a 16-byte load a lane, a stage ahead of its use
    pdl_wait();
    uint4 next[kPairKa][2];
    auto load = [&](int u, int k) {
#pragma unroll
      for (int j = 0; j < kPairKa; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          if (k + j < p.pieces) next[j][half] = __ldcg(reinterpret_cast<const uint4*>(x_record(a, p, u, k + j, half)) + lane);
    };
    int s = 0, it = 0;
    uint32_t ph = 0;
    bool stop = false;
    if (first < p.units) load(first, 0);
    for (int u = first; u < p.units && !stop; u += step)
      for (int k = 0; k < p.pieces; k += kPairKa, ++it) {
        uint4 now[kPairKa][2];
#pragma unroll
        for (int j = 0; j < kPairKa; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) now[j][half] = next[j][half];
        if (k + kPairKa < p.pieces) load(u, k + kPairKa);
        else if (u + step < p.units) load(u + step, 0);
        if (it >= S) {
          const bool ok = mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns);
          if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
            stop = true;
            break;
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(smem + (size_t)s * kPairStage + 2 * kPairHalf) + lane;
#pragma unroll
        for (int j = 0; j < kPairKa; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            if (k + j < p.pieces) dst[(j * kPairScale + half * kMxScales) / 16] = now[j][half];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(full + s));
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
  } else {
    pdl_wait();
    const int q = warp & 3, h = (warp - 3) >> 2;
    const int r = q * 32 + lane;
    int i = 0;
    for (int u = first; u < p.units; u += step, ++i) {
      const int f = (2 * (u / p.n_t) + (int)rank) * kMxPiece + r, row0 = (u % p.n_t) * kPairRows;
      const bool ok =
          mbar_wait(smem_u32(tfull + (i & 1)), (uint32_t)(i >> 1) & 1u, a.err, abort_flag, a.wait_ns) && !*abort_flag;
      tc_fence_after();
      const uint32_t tl = tmem + ((i & 1) ? (uint32_t)kPairOdd : 0u) + ((uint32_t)(q * 32) << 16);
      // the shared columns first: the last chunks of an even unit, the first of an odd one
      constexpr int kChunks = kPairRows / 16, kFirst = kPairShared / 16;
      const int turn = (i & 1) ? 0 : kChunks - kFirst;
      for (int n = h; n < kChunks; n += 2) {
        if (n - 2 < kFirst && n >= kFirst) {  // this warp's shared chunks are in registers, or stored
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(tempty), 0));
        }
        const int c = (n + turn) & (kChunks - 1);
        const int t0 = row0 + c * 16;
        if (!ok || t0 >= a.n_rows) continue;
        float v[16];
        tmem_load16(tl + (uint32_t)(c * 16), v);
        mx_store<T>(a, f, t0, min(16, a.n_rows - t0), v);
      }
    }
  }

  __syncthreads();
  if (warp == 0 && *abort_flag) {
    for (int i = issued > S ? issued - S : 0; i < issued; ++i)
      if (i != drop) mbar_wait(smem_u32(full + (i % S)), (uint32_t)(i / S) & 1u, a.err, nullptr, a.wait_ns);
    __syncwarp();
  }
  __syncthreads();
  cluster_sync();  // neither CTA frees its tensor memory or exits while the pair works
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg2(tmem, 512);
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
  const long long units = (long long)p.n_f * p.n_t;
  p.cluster = 1;
  while (p.cluster < 8 && units * p.cluster * 2 <= sms && p.pieces >= p.cluster * 4) p.cluster *= 2;
  const int part = (p.pieces + p.cluster - 1) / p.cluster;
  const bool keep = keeps_x(a.n_rows, part);
  p.src = !keep ? SRC_STAGES : a.rows == nullptr ? SRC_RECORDS : a.rows_type == PE_BF16 ? SRC_BF16 : SRC_F32;
  p.x_piece = keep ? kMxScales + 64u * (uint32_t)p.bn : kMxRecord;
  p.x_bytes = keep ? (uint32_t)part * p.x_piece : 0;
  p.x_off = kMxgKa * kMxRecord;
  p.stage_bytes = (keep ? 1 : 2) * kMxgKa * kMxRecord;
  const int per_unit = (part + kMxgKa - 1) / kMxgKa;  // stages of a unit
  p.stages = (int)((kTcSmemOptIn - 128 - (long long)kMxgCtrl - p.x_bytes) / p.stage_bytes);
  if (p.cluster > 1) p.stages = std::min(p.stages, per_unit);
  p.ring_bytes = (uint32_t)p.stages * p.stage_bytes;
  if (p.cluster > 1) p.ring_bytes = std::max(p.ring_bytes, (uint32_t)p.bn * kMxPiece * 4u);
  p.acc_stride = keep ? kMxgKeepRows : kMxPiece;
  p.scale_col = 2 * p.acc_stride;
  p.scale_stage = (keep ? 4 : 8) * kMxgKa;
  p.x_col = 256;
  p.grid = p.cluster * (int)std::min<long long>(units, p.cluster > 1 ? units : sms);
  p.smem = 128 + (size_t)p.ring_bytes + p.x_bytes + kMxgCtrl;
  return p;
}

constexpr size_t kPairSmem = 128 + (size_t)kPairStages * kPairStage + kMxgCtrl;

MxPairPlan plan_pair(const MxMatmulArgs& a) {
  MxPairPlan p{};
  p.pieces = (a.width + kMxPiece - 1) / kMxPiece;
  p.blocks_f = (a.n_out + kMxPiece - 1) / kMxPiece;
  p.blocks_t = (a.n_rows + kMxPiece - 1) / kMxPiece;
  p.n_f = (p.blocks_f + 1) / 2;
  p.n_t = (p.blocks_t + 1) / 2;
  p.units = (int)std::min<long long>((long long)p.n_f * p.n_t, 1 << 30);
  return p;
}

// Both kernels are bound by what an SM takes in, so the one whose busiest CTA takes in less is chosen.
bool use_pairs(const MxMatmulArgs& a, const MxPlan& p, const MxPairPlan& pp, int sms, int pairs) {
  if (a.n_rows <= kMxPiece) return false;
  const long long one = ((long long)p.n_f * p.n_t + sms - 1) / sms * ((p.pieces + p.cluster - 1) / p.cluster);
  const long long two = ((long long)pp.n_f * pp.n_t + pairs - 1) / pairs * p.pieces;
  return two < one;
}

// Largest dynamic shared memory for both kernels, once per device; pairs: clusters of two of the pair kernel that fit on
// the GPU at once (fewer than half the SMs where a processing cluster has an odd number).
template <typename T>
cudaError_t prepare_device(int* pairs) {
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (known[dev] == 0) {
    cudaError_t e = cudaSuccess;
    for (auto* kernel : {mx_gemm_kernel<T, SRC_STAGES>, mx_gemm_kernel<T, SRC_RECORDS>, mx_gemm_kernel<T, SRC_BF16>,
                         mx_gemm_kernel<T, SRC_F32>})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOptIn);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mx_gemm_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOptIn);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = kPairSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if ((e = cudaOccupancyMaxActiveClusters(&n, mx_gemm_pair_kernel<T>, &cfg)) != cudaSuccess) return e;
    known[dev] = n > 0 ? n : 1;
  }
  *pairs = known[dev];
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_typed(const MxMatmulArgs& a, int sms, cudaStream_t s) {
  int pairs = 1;
  const cudaError_t e = prepare_device<T>(&pairs);
  if (e != cudaSuccess) return e;
  const MxPlan p = plan_mx(a, sms);
  const MxPairPlan pp = plan_pair(a);
  cudaLaunchConfig_t cfg = {};
  const bool pair = use_pairs(a, p, pp, sms, pairs);
  cfg.gridDim = dim3(pair ? 2u * (unsigned)std::min(pp.units, pairs) : (unsigned)p.grid);
  cfg.blockDim = dim3(pair ? kPairThreads : kMxgThreads);
  cfg.dynamicSmemBytes = pair ? kPairSmem : p.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = pair ? 2u : (unsigned)p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair || p.cluster > 1 ? 2 : 1;
  count_launch();
  if (pair) return cudaLaunchKernelEx(&cfg, mx_gemm_pair_kernel<T>, a, pp);
  switch (p.src) {
    case SRC_RECORDS: return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T, SRC_RECORDS>, a, p);
    case SRC_BF16: return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T, SRC_BF16>, a, p);
    case SRC_F32: return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T, SRC_F32>, a, p);
  }
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T, SRC_STAGES>, a, p);
}

}  // namespace

// Up to 32 rows: each CTA's own rounding of all of them takes less than a launch before the product.
bool mx_matmul_quantises(int n_rows, int n_out, int width, int sms) {
  if (n_rows > 32) return false;
  MxMatmulArgs a{};
  a.n_rows = n_rows; a.n_out = n_out; a.width = width;
  return plan_mx(a, sms).src != SRC_STAGES;
}

cudaError_t launch_mx_matmul(const MxMatmulArgs& a, pe_dtype dt, int sms, cudaStream_t s) {
  return dt == PE_BF16 ? launch_typed<__nv_bfloat16>(a, sms, s) : launch_typed<float>(a, sms, s);
}

}  // namespace pe
