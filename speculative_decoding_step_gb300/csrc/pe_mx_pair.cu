// The product of two microscaled (MX) 4-bit matrices for many rows (pe_mx_gemm.cu has the mathematics and the kernel for
// few), on pairs of CTAs: an MMA of cta_group::2 multiplies 256 rows of w by 256 of x, each CTA of the pair holding 128
// rows of either, so that an SM takes in two records a piece for its 128 x 256 sums.
//
// Bound by the MMAs and by what lies between units.  4099 rows of 2048 to 12288 features, 816 units of eight stages of 256
// entries for 76 pairs: 47 us, without copies and stores 36.8.  The tensor pipe is active 0.30 us a stage (26 of 50.6 us of
// a launch under the profiler; 0.19 would be the nominal rate of 4-bit products), and from a unit's last MMA until the
// columns that it shares with the next are empty takes about 1 us.  Copies, 66 bytes a ns into an SM, cost 2 us of it.
//
// Every copy of a stage, of either CTA, completes on the leader's barrier, and the leader issues every MMA; its commits
// free the stage in both.  (Copies that complete on their own CTA's barrier, whose completion the peer passes on, take
// half a microsecond more a round through the ring: 66 us for 4099 x 2048 to 12288 features.)  So they are tensor copies,
// of records as [records][34][256 bytes]: a stage takes w's records as they are, x's codes (32 of 34 rows), and the scales
// (2 of 34) of all 256 rows of x, which both CTAs' tensor memory holds.
//
// Tensor memory, 512 columns: two accumulators of 256 that share 96, and four stages' scales (12 columns a piece) at the
// end.  The epilogue empties the shared columns first, after which the next unit's MMAs may start.
#include "pe_mx_gemm.cuh"

namespace pe {

namespace {

constexpr int kPairTile = 2 * kMxPiece;
constexpr int kPairKa = 2;                                         // pieces of a stage
constexpr uint32_t kPairW = kPairKa * kMxRecord;                   // bytes of a stage's records of w,
constexpr uint32_t kPairX = kPairKa * (kMxRecord - kMxScales);     // codes of x,
constexpr uint32_t kPairXs = kPairKa * kMxScales;                  // and scales of either half of x
constexpr uint32_t kPairStage = kPairW + kPairX + 2 * kPairXs;
constexpr int kPairStages = (kTcSmemOptIn - 128 - (int)kMxgCtrl) / (int)kPairStage;
constexpr int kPairSlots = 4;                                      // stages whose scales have columns
constexpr int kPieceCols = 12;                                     // of a piece: four for w, eight for x
constexpr int kPairShared = kPairSlots * kPairKa * kPieceCols;     // columns that the accumulators share
constexpr int kPairOdd = 512 - kPairShared - 256;                  // first column of odd units' accumulator
constexpr int kPairThreads = 32 * 12;
constexpr size_t kPairSmem = 128 + (size_t)kPairStages * kPairStage + kMxgCtrl;
static_assert(kPairOdd + kPairShared == 256 && kPairShared % 16 == 0, "whole chunks are shared");
static_assert(kPairStage % 128 == 0 && kPairW % 128 == 0 && kPairX % 128 == 0 && kPairXs % 128 == 0, "copies' alignment");
static_assert(kPairStages >= kPairSlots, "a slot's stage was freed before the slot is used again");

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
PE_DEV void tc_copy_scales_pair(uint32_t dst, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(dst), "l"(sdesc) : "memory");
}
PE_DEV void st_cluster_s32(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Arrive on an mbarrier of either CTA.  Relaxed: what it says is that tensor memory was read, and a release would first see
// the thread's stores to y through (a microsecond).
PE_DEV void mbar_arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// N times 16 columns, `apart` columns on each.
template <int N>
PE_DEV void tmem_load16s(uint32_t taddr, uint32_t apart, float (&v)[N][16]) {
  uint32_t r[N][16];
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[i][0]), "=r"(r[i][1]), "=r"(r[i][2]), "=r"(r[i][3]), "=r"(r[i][4]), "=r"(r[i][5]), "=r"(r[i][6]),
          "=r"(r[i][7]), "=r"(r[i][8]), "=r"(r[i][9]), "=r"(r[i][10]), "=r"(r[i][11]), "=r"(r[i][12]), "=r"(r[i][13]),
          "=r"(r[i][14]), "=r"(r[i][15])
        : "r"(taddr + (uint32_t)i * apart)
        : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i)  // the registers are there after the wait: each is an operand of it
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[i][0]), "+r"(r[i][1]), "+r"(r[i][2]), "+r"(r[i][3]), "+r"(r[i][4]), "+r"(r[i][5]), "+r"(r[i][6]),
                   "+r"(r[i][7]), "+r"(r[i][8]), "+r"(r[i][9]), "+r"(r[i][10]), "+r"(r[i][11]), "+r"(r[i][12]),
                   "+r"(r[i][13]), "+r"(r[i][14]), "+r"(r[i][15])
                 :
                 : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) v[i][j] = __uint_as_float(r[i][j]);
}

struct MxPairPlan {
  int pieces, n_t, units;  // units: tiles of 256 x 256, those of the same weights side by side
};

// Roles: warps 0, 2 and 3 have a thread each that copies w, x's codes and x's scales; warp 1 of the leader issues the MMAs;
// warps 4 to 11 write results.
template <typename T>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_pair_kernel(const MxMatmulArgs a, const MxPairPlan p, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_xs) {
  constexpr bool ARGMAX = std::is_same<T, MxArgmax>::value;
  constexpr int S = kPairStages, EW = kPairThreads / 32 - 4, KA = kPairKa;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ctrl = smem + (size_t)S * kPairStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(ctrl);  // the leader's are used: both CTAs' copies
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* tempty = tfull + 2;  // the leader's is used: the columns that the next unit needs are empty
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = abort_flag + 1;
  volatile int* ends = last_flag + 1;  // [rank][warp]: stages that either CTA's copying threads began; [rank][1]: gave up
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(full + s), 1);
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
  const int per = (p.pieces + KA - 1) / KA;  // stages of a unit
  const int drop = blockIdx.x == 0 ? a.drop_stage : -1;
  const bool copier = warp != 1 && warp < 4 && lane == 0;
  const uint64_t pol = l2_policy_evict_last();
  const uint32_t leader_full = mapa_shared(smem_u32(full), 0);
  int issued = 0;  // stages that this thread began to fill

  // This thread's part of stage s: pieces k.. of unit u.  Pieces beyond a tile's last and tiles beyond the matrix come
  // as other records or as zeros, and are not used.
  auto copy = [&](int s, int u, int k) {
    const uint32_t dst = smem_u32(smem + (size_t)s * kPairStage), bar = leader_full + 8u * (uint32_t)s;
    const int tile_f = u / p.n_t, tile_t = u - tile_f * p.n_t;
    if (warp == 0) {
      if (rank == 0) mbar_expect_tx(smem_u32(full + s), 2 * kPairStage);
      tma_load_3d_pair(dst, &tm_w, bar, 0, 0, (2 * tile_f + (int)rank) * p.pieces + k, pol);
    } else if (warp == 2) {
      tma_load_3d_pair(dst + kPairW, &tm_x, bar, 0, (int)(kMxScales / 256), (2 * tile_t + (int)rank) * p.pieces + k, pol);
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half)
        tma_load_3d_pair(dst + kPairW + kPairX + (uint32_t)half * kPairXs, &tm_xs, bar, 0, 0,
                         (2 * tile_t + half) * p.pieces + k, pol);
    }
  };

  if (copier) {
    int s = 0, it = 0, npre = 0;
    uint32_t ph = 0;
    fence_proxy_async_global();
    if (warp == 0 && a.w_ready && first < p.units)  // the first unit's weights, where they are known to be there already
      for (; npre < S && npre < per; ++npre)
        if (npre != drop) copy(npre, first, npre * KA);
    pdl_wait();
    fence_proxy_async_global();
    bool stop = false;
    for (int u = first; u < p.units && !stop; u += step)
      for (int k = 0; k < p.pieces; k += KA, ++it) {
        if (it >= S && !mbar_wait(smem_u32(empty + s), ph ^ 1u, a.err, abort_flag, a.wait_ns)) {
          stop = true;
          break;
        }
        if (it >= npre && !(warp == 0 && it == drop)) copy(s, u, k);
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
      }
    issued = it;
  } else if (warp == 1 && rank == 0) {
    // The warp stays together and one elected lane issues: operands of these instructions are uniform, and made by one
    // lane of a diverged warp they take twice the time of an MMA.
    pdl_wait();
    const uint32_t s0 = smem_u32(smem);
    const uint64_t w_codes = sdesc_core(s0 + kMxScales, 128, kMxGroup), w_scales = sdesc_core(s0, 16, 128);
    const uint64_t x_codes = sdesc_core(s0 + kPairW, 128, kMxGroup), x_scales = sdesc_core(s0 + kPairW + kPairX, 16, 128);
    const uint32_t idesc = idesc_mxf4(2 * kMxPiece, kPairTile);
    int s = 0, i = 0, slot = 0;
    uint32_t ph = 0;
    int ahead = kPairSlots, bs = 0;  // stages until the scales' columns come round, and the stage that had them, with
    uint32_t bph = 0;                // its phase
    bool stop = false;
    for (int u = first; u < p.units && !stop; u += step, ++i) {
      if (i >= 1) {
        if (!mbar_wait_warp(smem_u32(tempty), (uint32_t)(i - 1) & 1u, a, abort_flag)) {
          stop = true;
          break;
        }
      }
      tc_fence_after();
      const uint32_t d = tmem + ((i & 1) ? (uint32_t)kPairOdd : 0u);
      for (int k = 0; k < p.pieces; k += KA) {
        // the scales go where those of four stages ago were: that stage's MMAs are done
        bool ok = mbar_wait(smem_u32(full + s), ph, a.err, abort_flag, a.wait_ns);
        if (ahead == 0)
          ok = ok && mbar_wait(smem_u32(empty + bs), bph, a.err, abort_flag, a.wait_ns);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t at = (uint32_t)s * (kPairStage / 16);
          const uint32_t sc = tmem + 512 - kPairShared + (uint32_t)(slot * KA * kPieceCols);
          const int n = p.pieces - k;  // pieces left
#pragma unroll
          for (int j = 0; j < KA; ++j)
            if (j < n) {
              const uint32_t c = sc + (uint32_t)(j * kPieceCols);
              tc_copy_scales_pair(c, w_scales + at + (uint32_t)j * (kMxRecord / 16));
              tc_copy_scales_pair(c + 4, x_scales + at + (uint32_t)j * (kMxScales / 16));
              tc_copy_scales_pair(c + 8, x_scales + at + (kPairXs + (uint32_t)j * kMxScales) / 16);
            }
#pragma unroll
          for (int j = 0; j < KA; ++j)
            if (j < n) {
              const uint32_t c = sc + (uint32_t)(j * kPieceCols);
              const uint64_t da = w_codes + at + (uint32_t)j * (kMxRecord / 16);
              const uint64_t db = x_codes + at + (uint32_t)j * ((kMxRecord - kMxScales) / 16);
              // 64 entries: two 16-byte columns, 256 bytes on
              tc_mma_mxf4_pair(d, da, db, idesc, c, c + 4, (k > 0 || j > 0) ? 1u : 0u);
              tc_mma_mxf4_pair(d, da + 16, db + 16, idesc | kScaleUpper, c, c + 4, 1u);
            }
          tc_commit_pair(smem_u32(empty + s));
        }
        __syncwarp();
        if (++s == S) {
          s = 0;
          ph ^= 1u;
        }
        if (++slot == kPairSlots) slot = 0;
        if (ahead > 0) {
          --ahead;
        } else if (++bs == S) {
          bs = 0;
          bph ^= 1u;
        }
      }
      if (elect_one()) tc_commit_pair(smem_u32(tfull + (i & 1)));
      __syncwarp();
    }
    // after a wait gave up: every MMA issued completes before the tensor memory is freed
    if (stop && i > 0)
      mbar_wait(smem_u32(tfull + ((i - 1) & 1)), (uint32_t)((i - 1) >> 1) & 1u, a.err, nullptr, a.wait_ns);
  } else if (warp >= 4) {
    pdl_wait();
    const int q = warp & 3, h = (warp - 4) >> 2, r = q * 32 + lane;
    const uint32_t leader_tempty = mapa_shared(smem_u32(tempty), 0);
    int i = 0;
    for (int u = first; u < p.units; u += step, ++i) {
      const int tile_f = u / p.n_t, row0 = (u - tile_f * p.n_t) * kPairTile;
      const int f = (2 * tile_f + (int)rank) * kMxPiece + r, buf = i & 1;
      // the shared columns' chunks first, the last of an even unit and the first of an odd one: all into registers
      constexpr int ALL = kPairTile / 16, SHARED = kPairShared / 16, MINE = SHARED / (EW / 4);
      static_assert(SHARED % (EW / 4) == 0, "the same number for every warp");
      const int turn = buf ? 0 : ALL - SHARED;
      auto column = [&](int n) { return ((n + turn) & (ALL - 1)) * 16; };
      auto row_of = [&](int n) { return row0 + column(n); };
      if constexpr (!ARGMAX)
        if (a.add != nullptr) mx_prefetch_addend<T>(a, f - lane, lane, h, ALL, EW / 4, row_of);
      float* seen = reinterpret_cast<float*>(ctrl + kMxgSeen) + buf * kPairTile;
      if constexpr (ARGMAX) mx_seen(a, row0, seen, threadIdx.x - 128, 32 * EW);
      MxOut<T> out(a, f, ARGMAX ? row0 : row_of(h), seen);
      const bool ok = mbar_wait_warp(smem_u32(tfull + buf), (uint32_t)(i >> 1) & 1u, a, abort_flag);
      tc_fence_after();
      const uint32_t tl = tmem + (buf ? (uint32_t)kPairOdd : 0u) + ((uint32_t)(q * 32) << 16);
      float first[MINE][16], v[16];
      if (ok) tmem_load16s<MINE>(tl + (uint32_t)column(h), (uint32_t)(EW / 4 * 16), first);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(leader_tempty);
#pragma unroll
      for (int j = 0; j < MINE; ++j) {
        const int n = h + j * (EW / 4);
        out.put(row_of(n), row_of(n + EW / 4), ok && row_of(n) < a.n_rows, first[j]);
      }
#pragma unroll 1
      for (int n = h + SHARED; n < ALL; n += EW / 4) {
        const bool some = ok && row_of(n) < a.n_rows;
        if (some) tmem_load16(tl + (uint32_t)column(n), v);
        out.put(row_of(n), n + EW / 4 < ALL ? row_of(n + EW / 4) : -1, some, v);
      }
    }
    if constexpr (ARGMAX) mx_head_finish(a, last_flag, threadIdx.x - 128, 32 * EW);
    tc_fence_before();
  }

  // Neither CTA frees its tensor memory or exits while the pair works.  After a wait gave up no copy may stay in flight:
  // threads that stopped earlier than others begin the stages they left out, and the leader sees all of them complete.
  __syncthreads();
  if (lane == 0 && warp < 4) {
    const uint32_t slot = smem_u32(const_cast<const int*>(ends + 4 * rank + warp));
    const int v = warp == 1 ? *abort_flag : issued;
    st_cluster_s32(mapa_shared(slot, 0), v);
    st_cluster_s32(mapa_shared(slot, 1), v);
  }
  __syncwarp();
  cluster_sync();
  if (ends[1] || ends[5]) {
    int last = 0;
    for (int j = 0; j < 8; ++j)
      if (j != 1 && j != 5) last = max(last, ends[j]);
    auto again = [&](int it) { copy(it % S, first + it / per * step, it % per * KA); };
    if (copier) {
      if (warp == 0 && drop >= 0 && drop < issued) again(drop);
      for (int it = issued; it < last; ++it) again(it);
    }
    if (threadIdx.x == 0 && rank == 0)
      for (int it = max(last - S, 0); it < last; ++it)
        mbar_wait(smem_u32(full + it % S), (uint32_t)(it / S) & 1u, a.err, nullptr, a.wait_ns);
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg2(tmem, 512);
  }
}

cudaLaunchConfig_t pair_config(unsigned pairs, cudaLaunchAttribute (&attr)[2], cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <typename T>
cudaError_t launch_typed(const MxMatmulArgs& a, const MxPairPlan& p, const CUtensorMap (&tm)[3], int pairs,
                         cudaStream_t s) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(mx_pair_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pair_config((unsigned)(p.units < pairs ? p.units : pairs), attr, s);
  count_launch();
  return cudaLaunchKernelEx(&cfg, mx_pair_kernel<T>, a, p, tm[0], tm[1], tm[2]);
}

}  // namespace

// Fewer than half the SMs where a processing cluster has an odd number of them.  Without a device (host-only use of the
// plan): half the SMs.
int mx_pair_clusters(int sms) {
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return sms / 2;
  if (known[dev] == 0) {
    int n = 0;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = pair_config(1, attr, nullptr);
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(mx_pair_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPairSmem) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, mx_pair_kernel<float>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      return sms / 2;
    }
    known[dev] = n < sms / 2 ? n : sms / 2;
  }
  return known[dev];
}

cudaError_t launch_mx_pairs(const MxMatmulArgs& a, pe_dtype dt, int pairs, cudaStream_t s) {
  MxPairPlan p{};
  p.pieces = (a.width + kMxPiece - 1) / kMxPiece;
  p.n_t = (a.n_rows + kPairTile - 1) / kPairTile;
  const long long units = (long long)((a.n_out + kPairTile - 1) / kPairTile) * p.n_t;
  if (units >= 1ll << 30) return cudaErrorInvalidValue;
  p.units = (int)units;
  const uint64_t w_records = (uint64_t)((a.n_out + kMxPiece - 1) / kMxPiece) * p.pieces;
  const uint64_t x_records = (uint64_t)((a.n_rows + kMxPiece - 1) / kMxPiece) * p.pieces;
  CUtensorMap tm[3];
  if (!tmap_mx(&tm[0], a.w, w_records, kMxRecord / 256) ||
      !tmap_mx(&tm[1], a.x, x_records, (kMxRecord - kMxScales) / 256) || !tmap_mx(&tm[2], a.x, x_records, kMxScales / 256))
    return cudaErrorInvalidValue;
  if (a.head.keys != nullptr) return launch_typed<MxArgmax>(a, p, tm, pairs, s);
  return dt == PE_BF16 ? launch_typed<__nv_bfloat16>(a, p, tm, pairs, s) : launch_typed<float>(a, p, tm, pairs, s);
}

}  // namespace pe
