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
// Many rows go to the kernel of pe_mx_pair.cu.
//
// With fewer tiles than SMs a cluster of CTAs shares a tile: each takes an equal part of its pieces along k, and the
// partial sums meet in shared memory over the cluster, each CTA summing its share of the columns in rank order, so the
// result does not depend on scheduling, and the call needs no workspace and no second kernel.
#include <algorithm>

#include "pe_internal.h"
#include "pe_mx_gemm.cuh"

namespace pe {

namespace {

constexpr int kMxgThreads = 32 * 12;

// Where a tile's rows of x come from: with each stage, as records beside the weights' (128 rows); or once, into shared
// memory for all of a CTA's tiles, as they are in 4 bits or quantised there from rows of bf16 or fp32.
enum MxSrc : int { SRC_STAGES = 0, SRC_RECORDS = 1, SRC_BF16 = 2, SRC_F32 = 3 };

// Pieces of a stage.  A copy takes the thread that issues it 40 ns and a stage's round trip through the ring about a
// microsecond, so stages are large and weights and x have a thread each.
constexpr int kMxgKa = 4;

// Tensor memory: two accumulators, the stages' scales, and the scales of x where it is kept (four columns a piece).
struct MxPlan {
  int pieces, n_f, n_t, bn, cluster, stages, grid, src;
  int acc_stride, scale_col, x_col;
  uint32_t x_piece, stage_bytes, ring_bytes, x_bytes;
  size_t smem;
};
constexpr int kMxgKeepRows = 64;             // rows of x that are kept at most (accumulators of 64 columns)
constexpr int kMxgKeepPieces = 64;           // pieces of x that are kept at most (256 columns of scales)
constexpr uint32_t kMxgKeepBytes = 96 * 1024;

// Shared memory that a CTA of a cluster asks for at least: more than half of an SM's (228 KB, with 1 KB of its own for every
// CTA), so that no SM has two of them.  Such a CTA holds all of its SM's tensor memory until its cluster has joined its
// parts, and an allocation waits without a limit: of two clusters (calls on two streams), each with a CTA that waits for
// tensor memory which a CTA of the other holds, neither would end.  (Pairs of CTAs, here and in the drafter's GEMMs, take
// nearly all of an SM's shared memory, so none fits beside one either.)
constexpr size_t kMxgClusterSmem = 116 * 1024;
static_assert(2 * (kMxgClusterSmem + 1024) > 228 * 1024, "two CTAs do not fit an SM");

PE_DEV void st_cluster_v4(uint32_t addr, float x, float y, float z, float w) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}

struct MxUnit {
  int tile_f, tile_t, row0, cols;
};
PE_DEV MxUnit mx_unit(const MxMatmulArgs& a, const MxPlan& p, int u) {
  MxUnit w;
  w.tile_t = u % p.n_t;  // a weight tile's row tiles run side by side (its records come from L2)
  w.tile_f = u / p.n_t;
  w.row0 = w.tile_t * kMxPiece;
  w.cols = min(p.bn, (a.n_rows - w.row0 + 15) & ~15);
  return w;
}

// Rows of x into shared memory in 4 bits: pieces p0..p1 - 1 of all bn rows, x_piece bytes each (a record's scales and its
// first rows), by `warps` warps of which this is the w-th.  Rows beyond the last are zeros, or (records) as they are.
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
  // a warp takes eight rows of a piece at a time, the pieces of the same rows side by side (so that rows beyond the last,
  // which wait for no load, come in a turn of their own)
  const int pieces = p1 - p0, units = p.bn / 8 * pieces, quarter = lane & 3;
  bool bad = false;
  for (int u = w; u < units; u += warps) {
    const int g = u / pieces, k = u - g * pieces, r = g * 8 + (lane >> 2);
    const bool live = r < a.n_rows;
    const T* src = static_cast<const T*>(a.rows) + (long long)r * a.rows_stride + (p0 + k) * kMxPiece + quarter * 8;
    const int left = a.width - (p0 + k) * kMxPiece - quarter * 8;
    float x[4][8];
    if (live && left >= kMxPiece - quarter * 8) {
#pragma unroll
      for (int b = 0; b < 4; ++b) get8(src + b * kMxBlock, x[b]);
    } else {
#pragma unroll
      for (int b = 0; b < 4; ++b) get8_of(src + b * kMxBlock, live ? left - b * kMxBlock : 0, x[b]);
    }
    uint8_t* out = xs + (size_t)k * p.x_piece;
    uint32_t s4 = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t codes, scale;
      bad |= mx_round8(x[b], codes, scale);
      s4 |= scale << (8 * b);
      reinterpret_cast<uint32_t*>(out + mx_code_at(r, b))[quarter] = codes;
    }
    if (quarter == 0) *reinterpret_cast<uint32_t*>(out + mx_scale_at(r, 0)) = s4;
  }
  if (bad) set_err(a.err, PE_DEV_NONFINITE);
}

// A cluster's one unit: its CTAs exchange their partial sums (through `recv`, in the place of the stages) and write their
// shares of the columns, quad by quad.
template <typename T>
PE_DEV void mx_join(const MxMatmulArgs& a, const MxPlan& p, const MxUnit& w, int rank, uint32_t tmem, uint8_t* recv,
                    volatile int* abort_flag) {
  constexpr int HALVES = (kMxgThreads / 32 - 4) / 4;  // warps of a lane quarter
  const int warp = threadIdx.x >> 5, r = threadIdx.x & 127, h = (warp - 4) >> 2;  // row of w, and which columns
  const int quads = w.cols / 4, share = (quads + p.cluster - 1) / p.cluster;
  __syncthreads();
  cluster_sync();
  if (warp >= 4 && !*abort_flag) {
    const uint32_t tl = tmem + ((uint32_t)(r & ~31) << 16);
    // to [rank][quad of the owner's][row of w], 16 bytes each
    const uint32_t mine = smem_u32(recv) + (uint32_t)(rank * share * kMxPiece + r) * 16;
    for (int c = h; c < w.cols / 16; c += HALVES) {
      float v[16];
      tmem_load16(tl + (uint32_t)(c * 16), v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int owner = (4 * c + j) / share, at = 4 * c + j - owner * share;
        st_cluster_v4(mapa_shared(mine + (uint32_t)(at * kMxPiece) * 16, (uint32_t)owner), v[4 * j], v[4 * j + 1],
                      v[4 * j + 2], v[4 * j + 3]);
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();  // every partial sum is where it is summed
  const int f = w.tile_f * kMxPiece + r, n = min(share, quads - rank * share);
  if (warp < 4 || *abort_flag || f >= a.n_out) return;
  const float4* part = reinterpret_cast<const float4*>(recv) + r;
  for (int c = h; c < n; c += HALVES) {
    const int t0 = w.row0 + 4 * (rank * share + c);
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < p.cluster) x[k] = part[(k * share + c) * kMxPiece];
    float old[4], v[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      old[j] = a.add == nullptr ? 0.f
                                : to_float<T>(static_cast<const T*>(
                                      a.add)[(long long)min(t0 + j, a.n_rows - 1) * a.add_stride + f]);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < p.cluster) {
        v[0] += x[k].x;
        v[1] += x[k].y;
        v[2] += x[k].z;
        v[3] += x[k].w;
      }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + j < a.n_rows) static_cast<T*>(a.y)[(long long)(t0 + j) * a.y_stride + f] = from_float<T>(v[j] + old[j]);
  }
}

// Roles: one thread copies weights (warp 0), one x (warp 2), one issues the MMAs (warp 1); the other warps
// bring in x where it is kept and write results.
template <typename T, int SRC>
__global__ void __launch_bounds__(kMxgThreads, 1) mx_gemm_kernel(const MxMatmulArgs a, const MxPlan p) {
  constexpr bool KEEP = SRC >= SRC_RECORDS, ARGMAX = std::is_same<T, MxArgmax>::value;
  constexpr int EW = kMxgThreads / 32 - 4, KA = kMxgKa;
  constexpr uint32_t X_OFF = KA * kMxRecord;  // a stage: weight records, then those of x
  constexpr int PIECE_COLS = KEEP ? 4 : 8, STAGE_COLS = KA * PIECE_COLS;  // columns of a piece's scales, and of a stage's
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

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), KEEP ? 1 : 2);
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
    if (!KEEP && warp == 2 && lane == 0) {
      const uint64_t pol = l2_policy_evict_last();
      pdl_wait();
      fence_proxy_async_global();
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool stop = false;
      for (int u = first; u < units && !stop; u += step) {
        const uint8_t* src = a.x + ((size_t)mx_unit(a, p, u).tile_t * p.pieces + p0) * kMxRecord;
        for (int k = p0; k < p1; k += KA, ++it) {
          if (it >= S && !mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns)) {
            stop = true;
            break;
          }
          // whole records: rows beyond the tile's columns come along unused
          const uint32_t bytes = (uint32_t)min(KA, p1 - k) * kMxRecord;
          mbar_expect_tx(smem_u32(full + s), bytes);
          bulk_g2s_hint(smem_u32(smem + (size_t)s * p.stage_bytes) + X_OFF, src + (size_t)(k - p0) * kMxRecord, bytes,
                        smem_u32(full + s), pol);
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
    const uint64_t x_codes = sdesc_core((KEEP ? smem_u32(xs) : s0 + X_OFF) + kMxScales, 128, kMxGroup);
    const uint64_t x_scales = sdesc_core(KEEP ? smem_u32(xs) : s0 + X_OFF, 16, 128);
    const uint32_t stage16 = p.stage_bytes >> 4, piece16 = p.x_piece >> 4;
    int s = 0, i = 0;
    uint32_t ph = 0;
    bool stop = false;
    if (KEEP) {
      stop = !mbar_wait_warp(smem_u32(kept), 0, a, abort_flag);
      tc_fence_after();
      if (!stop && elect_one())
        for (int k = 0; k < p1 - p0; ++k)
          tc_copy_scales(tmem + (uint32_t)(p.x_col + 4 * k), x_scales + (uint32_t)k * piece16);
      __syncwarp();
    }
    for (int u = first; u < units && !stop; u += step, ++i) {
      const int cols = mx_unit(a, p, u).cols;
      const uint32_t idesc = idesc_mxf4(kMxPiece, cols);
      const int buf = i & 1;
      if (i >= 2) {
        if (!mbar_wait_warp(smem_u32(tempty + buf), (uint32_t)((i >> 1) - 1) & 1u, a, abort_flag)) {
          stop = true;
          break;
        }
      }
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(buf * p.acc_stride);
      for (int k = p0; k < p1; k += KA) {
        if (!mbar_wait_warp(smem_u32(full + s), ph, a, abort_flag)) {
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
              if (!KEEP) tc_copy_scales(sb + j * SB_PIECE, xsc + j * (kMxRecord / 16));
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
        const MxUnit w = mx_unit(a, p, u);
        const int buf = i & 1, f = w.tile_f * kMxPiece + r, chunks = w.cols / 16;
        auto row_of = [&](int n) { return w.row0 + n * 16; };
        if constexpr (!ARGMAX)
          if (a.add != nullptr) mx_prefetch_addend<T>(a, f - lane, lane, h, 8, EW / 4, row_of);
        float* seen = reinterpret_cast<float*>(ctrl + kMxgSeen) + buf * 32 * EW;
        if constexpr (ARGMAX) mx_seen(a, w.row0, seen, threadIdx.x - 128, 32 * EW);
        MxOut<T> out(a, f, ARGMAX ? w.row0 : row_of(h), seen);
        const bool ok = mbar_wait_warp(smem_u32(tfull + buf), (uint32_t)(i >> 1) & 1u, a, abort_flag);
        tc_fence_after();
        const uint32_t tl = tmem + (uint32_t)(buf * p.acc_stride) + ((uint32_t)(q * 32) << 16);
        for (int n = h; n < chunks; n += EW / 4) {
          float v[16];
          if (ok) tmem_load16(tl + (uint32_t)(n * 16), v);
          out.put(row_of(n), n + EW / 4 < chunks ? row_of(n + EW / 4) : -1, ok, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(tempty + buf));
      }
      if constexpr (ARGMAX) mx_head_finish(a, last_flag, threadIdx.x - 128, 32 * EW);
    } else {
      mbar_wait_warp(smem_u32(tfull), 0, a, abort_flag);
      tc_fence_after();
    }
  }

  if constexpr (!ARGMAX)
    if (p.cluster > 1)  // every CTA's MMAs are done (or given up), so the stages' memory takes the partial sums
      mx_join<T>(a, p, mx_unit(a, p, first), rank, tmem, smem, abort_flag);

  __syncthreads();
  if (*abort_flag) {
    // After a wait gave up no copy may stay in flight into this CTA's shared memory: threads that stopped earlier than
    // others arrive, without a copy, for the stages they left out, so that every stage begun completes.
    const bool copier = lane == 0 && (warp == 0 || (!KEEP && warp == 2));
    if (copier) issued_max[warp] = issued;
    __syncthreads();
    const int last = KEEP ? issued_max[0] : max(issued_max[0], issued_max[2]);
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

// Clusters of so many CTAs that fit on the GPU at once.  Without a device (host-only use of the plan): a quarter less than
// the SMs would hold.
int clusters_that_fit(int size, int sms) {
  static int known[64][9] = {{0}};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms * 3 / 4 / size;
  if (known[dev][size] == 0) {
    int n = 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kMxgThreads);
    cfg.dynamicSmemBytes = kTcSmemOptIn;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = mx_gemm_kernel<float, SRC_STAGES>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOptIn) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return sms * 3 / 4 / size;
    }
    known[dev][size] = n;
  }
  return known[dev][size];
}

// CTAs that share a tile along k.  A CTA takes about 0.107 us a piece where few are at work, and joining the parts 1 us and
// 0.02 a column (16 rows of 4096 to 128 features 5.8 us alone, 4.4 as eight; of 1024 3.4 and 4.2; 128 rows of 8192 10.1
// and 7.2, of 2048 5.1 and 6.4).
int cluster_of(long long units, int pieces, int bn, int sms) {
  int best = 1, gain = 0;  // ns
  for (int c = 2; c <= 8; c *= 2) {
    const int g = (pieces - (pieces + c - 1) / c) * 107 - (1000 + 20 * bn);
    if (g > gain && units <= clusters_that_fit(c, sms)) {
      best = c;
      gain = g;
    }
  }
  return best;
}

MxPlan plan_mx(const MxMatmulArgs& a, int sms) {
  MxPlan p{};
  p.pieces = (a.width + kMxPiece - 1) / kMxPiece;
  p.n_f = (a.n_out + kMxPiece - 1) / kMxPiece;
  p.n_t = (a.n_rows + kMxPiece - 1) / kMxPiece;
  p.bn = std::min(kMxPiece, (a.n_rows + 15) & ~15);
  const long long units = (long long)p.n_f * p.n_t;
  p.cluster = a.head.keys == nullptr ? cluster_of(units, p.pieces, p.bn, sms) : 1;  // (the LM head looks at its sums as they are)
  const int part = (p.pieces + p.cluster - 1) / p.cluster;
  const bool keep = keeps_x(a.n_rows, part);
  p.src = !keep ? SRC_STAGES : a.rows == nullptr ? SRC_RECORDS : a.rows_type == PE_BF16 ? SRC_BF16 : SRC_F32;
  const int ka = kMxgKa;
  p.x_piece = keep ? kMxScales + 64u * (uint32_t)p.bn : kMxRecord;
  p.x_bytes = keep ? (uint32_t)part * p.x_piece : 0;
  p.stage_bytes = (uint32_t)ka * (keep ? 1 : 2) * kMxRecord;
  p.stages = (int)((kTcSmemOptIn - 128 - (long long)kMxgCtrl - p.x_bytes) / p.stage_bytes);
  if (p.cluster > 1) p.stages = std::min(p.stages, (part + ka - 1) / ka);
  p.ring_bytes = (uint32_t)p.stages * p.stage_bytes;
  if (p.cluster > 1)  // the partial sums of a CTA's share
    p.ring_bytes = std::max(p.ring_bytes, (uint32_t)((p.bn / 4 + p.cluster - 1) / p.cluster * p.cluster) * kMxPiece * 16u);
  p.acc_stride = keep ? kMxgKeepRows : kMxPiece;
  p.scale_col = 2 * p.acc_stride;
  p.x_col = 256;
  p.grid = p.cluster * (int)std::min<long long>(units, p.cluster > 1 ? units : sms);
  p.smem = 128 + (size_t)p.ring_bytes + p.x_bytes + kMxgCtrl;
  if (p.cluster > 1) p.smem = std::max(p.smem, kMxgClusterSmem);
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
    case SRC_RECORDS: return launch_src<T, SRC_RECORDS>(a, p, s);
    case SRC_BF16: return launch_src<T, SRC_BF16>(a, p, s);
    case SRC_F32: return launch_src<T, SRC_F32>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Where a CTA has no more than 12,288 entries of x: it rounds them in less than a launch before the product takes (8 rows
// of 256: 3.4 against 4.7 us; 14 rows of 2880: 12.5 against 8.2 us).
bool mx_matmul_quantises(int n_rows, int n_out, int width, bool head, int sms) {
  MxMatmulArgs a{};
  unsigned long long key;
  a.n_rows = n_rows; a.n_out = n_out; a.width = width; a.head.keys = head ? &key : nullptr;
  const MxPlan p = plan_mx(a, sms);
  return p.src == SRC_RECORDS && (long long)p.bn * ((p.pieces + p.cluster - 1) / p.cluster) * kMxPiece <= 12288;
}

size_t mx_matmul_smem(int n_rows, int n_out, int width, int sms, int* cluster) {
  MxMatmulArgs a{};
  a.n_rows = n_rows; a.n_out = n_out; a.width = width;
  const MxPlan p = plan_mx(a, sms);
  *cluster = p.cluster;
  return p.smem;
}

// More than 128 rows go to pairs of CTAs where those are expected to take less: about 0.17 us a piece of their 256 x 256
// tiles against 0.12 of a CTA's 128 x 128 ones, and 1.7 us a call more (640 rows of 7680 to 4096 features: 17.5 us by CTAs,
// 15.5 by pairs; 256 of 2048 to 4096: 5.4 and 8.2; 1500 of 7680 to 12288: 62 and 48; 640 of 2880 to 5120: 9.7 and 9.8).  The
// results' way out, which nothing hides at one tile a pair, is in neither side: 896 rows of 7680 to 2880 features with fp32
// addends take 19.2 us by CTAs and 17.1 by pairs, where 14.4 and 11.9 are expected.
cudaError_t launch_mx_matmul(const MxMatmulArgs& a, pe_dtype dt, int sms, cudaStream_t s) {
  const MxPlan p = plan_mx(a, sms);
  if (a.n_rows > kMxPiece) {
    const int pairs = mx_pair_clusters(sms);
    const long long tiles = (long long)((a.n_out + 255) / 256) * ((a.n_rows + 255) / 256);
    const long long two = (tiles + pairs - 1) / pairs * p.pieces * 170 + 1700;
    const long long one = p.cluster > 1 ? (p.pieces + p.cluster - 1) / p.cluster * 107 + 1000 + 20 * p.bn
                                        : ((long long)p.n_f * p.n_t + sms - 1) / sms * p.pieces * 120;
    if (two < one) return launch_mx_pairs(a, dt, pairs, s);
  }
  if (a.head.keys != nullptr) return launch_typed<MxArgmax>(a, sms, s);
  return dt == PE_BF16 ? launch_typed<__nv_bfloat16>(a, sms, s) : launch_typed<float>(a, sms, s);
}

}  // namespace pe
