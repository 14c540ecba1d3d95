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

constexpr int kMxgMaxStages = 12;
constexpr uint32_t kMxgCtrl = 1024;  // barriers, tensor-memory slot, flags
constexpr int kMxgScaleCols = 8;     // tensor-memory columns of a piece's scales: four for w, four for x

struct MxPlan {
  int pieces, n_f, n_t, bn, cluster, ka, stages, threads, grid;
  uint32_t x_piece, stage_bytes, acc_stride, scale_col, recv_bytes;
  size_t smem;
};

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

// This CTA's units u = first, first + step, ... < end, and its part of their pieces.
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

// Roles: warp 0 copies (one elected lane issues), warp 1 issues the MMAs, the others write results.
template <typename T>
__global__ void __launch_bounds__(64 + 32 * 8, 1) mx_gemm_kernel(const MxMatmulArgs a, const MxPlan p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int EW = (int)(blockDim.x >> 5) - 2;
  const int S = p.stages;
  uint8_t* ctrl = smem + (size_t)S * p.stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* recv = reinterpret_cast<float*>(ctrl + kMxgCtrl);  // clusters: [rank][columns of this CTA][128]

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
      mbar_init(smem_u32(empty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(tfull + b), 1);
      mbar_init(smem_u32(tempty + b), EW);
    }
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
  if (p.cluster > 1) cluster_sync();  // every CTA of the cluster runs before another writes into its shared memory
  pdl_trigger();

  const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int first = (int)blockIdx.x / p.cluster, step = (int)gridDim.x / p.cluster, units = p.n_f * p.n_t;
  const int p0 = (int)((long long)p.pieces * rank / p.cluster), p1 = (int)((long long)p.pieces * (rank + 1) / p.cluster);
  const int drop = blockIdx.x == 0 ? a.drop_stage : -1;
  int issued = 0;  // stages that the copying warp issued

  if (warp == 0) {
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    int s = 0, it = 0, npre = 0;
    uint32_t ph = 0;
    // the first unit's weights, where they are known to be there already
    auto copy_w = [&](int st, int tile_f, int k) {
      const int n = min(p.ka, p1 - k);
      bulk_g2s_hint(smem_u32(smem + (size_t)st * p.stage_bytes), a.w + ((size_t)tile_f * p.pieces + k) * kMxRecord,
                    (uint32_t)n * kMxRecord, smem_u32(full + st), pol_w);
    };
    auto arm = [&](int st, int cols, int k) {
      const int n = min(p.ka, p1 - k);
      mbar_expect_tx(smem_u32(full + st), (uint32_t)n * (kMxRecord + kMxScales + 64u * (uint32_t)cols));
    };
    fence_proxy_async_global();
    if (a.w_ready && first < units) {
      const MxUnit w = mx_unit(a, p, first);
      for (int k = p0; k < p1 && npre < S; k += p.ka, ++npre)
        if (npre != drop && elect_one()) {
          arm(npre, w.cols, k);
          copy_w(npre, w.tile_f, k);
        }
    }
    __syncwarp();
    pdl_wait();
    fence_proxy_async_global();
    bool stop = false;
    for (int u = first; u < units && !stop; u += step) {
      const MxUnit w = mx_unit(a, p, u);
      for (int k = p0; k < p1; k += p.ka, ++it) {
        if (it >= S) {
          const bool ok = mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns);
          if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
            stop = true;
            break;
          }
        }
        if (it != drop && elect_one()) {
          if (it >= npre) {
            arm(s, w.cols, k);
            copy_w(s, w.tile_f, k);
          }
          const int n = min(p.ka, p1 - k);
          const uint8_t* src = a.x + ((size_t)w.tile_t * p.pieces + k) * kMxRecord;
          const uint32_t dst = smem_u32(smem + (size_t)s * p.stage_bytes) + (uint32_t)p.ka * kMxRecord;
          if (p.x_piece == kMxRecord && w.cols == kMxPiece) {
            bulk_g2s_hint(dst, src, (uint32_t)n * kMxRecord, smem_u32(full + s), pol_x);
          } else {
            for (int i = 0; i < n; ++i)
              bulk_g2s_hint(dst + (uint32_t)i * p.x_piece, src + (size_t)i * kMxRecord, kMxScales + 64u * (uint32_t)w.cols,
                            smem_u32(full + s), pol_x);
          }
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
      const uint32_t d = tmem + (uint32_t)buf * p.acc_stride;
      for (int k = p0; k < p1; k += p.ka) {
        const bool ok = mbar_wait(smem_u32(full + s), ph, a.err, abort_flag, a.wait_ns);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const int n = min(p.ka, p1 - k);
          const uint32_t sw = smem_u32(smem + (size_t)s * p.stage_bytes), sx = sw + (uint32_t)p.ka * kMxRecord;
          const uint32_t sc = tmem + p.scale_col + (uint32_t)(s * p.ka * kMxgScaleCols);
          for (int j = 0; j < n; ++j) {
            tc_copy_scales(sc + (uint32_t)(j * kMxgScaleCols), sw + (uint32_t)j * kMxRecord);
            tc_copy_scales(sc + (uint32_t)(j * kMxgScaleCols) + 4, sx + (uint32_t)j * p.x_piece);
          }
          for (int j = 0; j < n; ++j) {
            const uint64_t da = sdesc_core(sw + (uint32_t)j * kMxRecord + kMxScales, 128, kMxGroup);
            const uint64_t db = sdesc_core(sx + (uint32_t)j * p.x_piece + kMxScales, 128, kMxGroup);
            const uint32_t sa = sc + (uint32_t)(j * kMxgScaleCols);
            // 64 entries: two 16-byte columns, 256 bytes on
            tc_mma_mxf4(d, da, db, idesc, sa, sa + 4, (k > p0 || j > 0) ? 1u : 0u);
            tc_mma_mxf4(d, da + 16, db + 16, idesc | kScaleUpper, sa, sa + 4, 1u);
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
    if (stop) mbar_wait(smem_u32(tfull + ((i - 1) & 1)), (uint32_t)((i - 1) >> 1) & 1u, a.err, nullptr, a.wait_ns);
  } else {
    pdl_wait();
    const int q = warp & 3, h = (warp - 2) >> 2, hs = EW >> 2;
    const int r = q * 32 + lane;
    int i = 0;
    for (int u = first; u < units; u += step, ++i) {
      const MxUnit w = mx_unit(a, p, u);
      const int buf = i & 1;
      const bool ok =
          mbar_wait(smem_u32(tfull + buf), (uint32_t)(i >> 1) & 1u, a.err, abort_flag, a.wait_ns) && !*abort_flag;
      tc_fence_after();
      const uint32_t tl = tmem + (uint32_t)buf * p.acc_stride + ((uint32_t)(q * 32) << 16);
      if (ok)
        for (int c = h; c < w.cols / 16; c += hs) {
          float v[16];
          tmem_load16(tl + (uint32_t)(c * 16), v);
          const int t0 = w.tile_t * kMxPiece + c * 16;
          if (p.cluster == 1) {
            mx_store<T>(a, w.tile_f * kMxPiece + r, t0, min(16, a.n_rows - t0), v);
          } else {
            const int share = w.cols / p.cluster;  // columns that each CTA of the cluster sums
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int col = c * 16 + j, owner = col / share;
              st_cluster_f32(mapa_shared(smem_u32(recv + (size_t)(rank * share + col - owner * share) * kMxPiece + r),
                                         (uint32_t)owner),
                             v[j]);
            }
          }
        }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(tempty + buf));
    }
  }

  if (p.cluster > 1) {
    __syncwarp();
    cluster_sync();  // every partial sum is where it is summed
    if (warp >= 2 && first < units) {
      const MxUnit w = mx_unit(a, p, first);
      const int share = w.cols / p.cluster;
      const int r = threadIdx.x & 127, half = (threadIdx.x - 64) >> 7;
      const int f = w.tile_f * kMxPiece + r, t0 = w.tile_t * kMxPiece + rank * share;
      if (f < a.n_out && !*abort_flag)
        for (int c = half; c < share && t0 + c < a.n_rows; c += EW >> 2) {
          float v = 0.f;
          for (int k = 0; k < p.cluster; ++k) v += recv[(size_t)(k * share + c) * kMxPiece + r];
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

MxPlan plan_mx(const MxMatmulArgs& a, int sms) {
  MxPlan p{};
  p.pieces = (a.width + kMxPiece - 1) / kMxPiece;
  p.n_f = (a.n_out + kMxPiece - 1) / kMxPiece;
  p.n_t = (a.n_rows + kMxPiece - 1) / kMxPiece;
  p.bn = std::min(kMxPiece, (a.n_rows + 15) & ~15);
  const long long units = (long long)p.n_f * p.n_t;
  p.cluster = 1;
  while (p.cluster < 8 && units * p.cluster * 2 <= sms && p.pieces >= p.cluster * 4) p.cluster *= 2;
  p.x_piece = kMxScales + 64u * (uint32_t)p.bn;
  p.ka = 2;
  p.stage_bytes = (uint32_t)p.ka * (kMxRecord + p.x_piece);
  p.recv_bytes = p.cluster > 1 ? (uint32_t)p.bn * kMxPiece * 4 : 0;
  const long long avail = kTcSmemOptIn - 128 - (long long)kMxgCtrl - p.recv_bytes;
  p.stages = (int)std::min<long long>(kMxgMaxStages, avail / p.stage_bytes);
  p.stages = std::min(p.stages, 256 / (kMxgScaleCols * p.ka));
  p.acc_stride = kMxPiece;
  p.scale_col = 2 * kMxPiece;
  p.threads = p.bn >= 64 ? 64 + 32 * 8 : 64 + 32 * 4;
  p.grid = p.cluster * (int)std::min<long long>(units, p.cluster > 1 ? units : sms);
  p.smem = 128 + (size_t)p.stages * p.stage_bytes + kMxgCtrl + p.recv_bytes;
  return p;
}

template <typename T>
cudaError_t launch_typed(const MxMatmulArgs& a, const MxPlan& p, cudaStream_t s) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(mx_gemm_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOptIn);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3((unsigned)p.threads);
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
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<T>, a, p);
}

}  // namespace

cudaError_t launch_mx_matmul(const MxMatmulArgs& a, pe_dtype dt, int sms, cudaStream_t s) {
  const MxPlan p = plan_mx(a, sms);
  return dt == PE_BF16 ? launch_typed<__nv_bfloat16>(a, p, s) : launch_typed<float>(a, p, s);
}

}  // namespace pe
