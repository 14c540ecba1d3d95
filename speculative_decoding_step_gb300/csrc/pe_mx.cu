// Microscaled (MX) 4-bit matrices: rounding rows and reading them back.  The format is in pe_mx.cuh.
#include <cuda_fp16.h>

#include <algorithm>

#include "pe_internal.h"
#include "pe_mx.cuh"

namespace pe {

namespace {

constexpr int kMxThreads = 128;
constexpr int kMxWarps = kMxThreads / 32;
constexpr int kMxTileRow = kMxPiece + 4;  // floats from one row of a warp's tile to the next

// Which rows and pieces a warp takes: a CTA has `along` warps side by side over the pieces and 4 / along groups of
// eight rows; its warps take `steps` pieces each, `along` apart.  No divisions by sizes then, and a few rows spread over
// many CTAs.
struct MxDeal {
  int along_log2, steps, pieces;
};
MxDeal mx_deal(int n_rows, int width, dim3* grid) {
  MxDeal d{};
  d.pieces = (width + kMxPiece - 1) / kMxPiece;
  const long long groups = (n_rows + 7) / 8;
  while ((1 << d.along_log2) < std::min(kMxWarps, d.pieces)) ++d.along_log2;
  const int along = 1 << d.along_log2;
  const long long gx = (groups * along + kMxWarps - 1) / kMxWarps;
  // enough CTAs to fill the GPU, each warp four pieces at most
  d.steps = 1;
  while (d.steps < 4 && along * d.steps < d.pieces &&
         gx * ((d.pieces + along * d.steps - 1) / (along * d.steps)) > 2LL * 152 * 16)
    d.steps *= 2;
  *grid = dim3((unsigned)gx, (unsigned)((d.pieces + along * d.steps - 1) / (along * d.steps)));
  return d;
}

template <typename T>
struct BitsOf;
template <>
struct BitsOf<float> {
  using type = uint32_t;
};
template <>
struct BitsOf<__nv_bfloat16> {
  using type = uint16_t;
};
template <typename T>
PE_DEV float widen(uint32_t b) {
  return __uint_as_float(sizeof(T) == 2 ? b << 16 : b);
}

// Eight entries of each lane of a pair, the odd lane's after the even lane's.  fp32: the lanes exchange halves, so
// that either store of a pair fills 32 bytes (a lane its own 16 at a time: 75 us instead of 44 for 8209 x 7680).
PE_DEV void put8(float* p, const float (&v)[8]) {
  const bool odd = threadIdx.x & 1;
  float4 mine = odd ? make_float4(v[4], v[5], v[6], v[7]) : make_float4(v[0], v[1], v[2], v[3]);
  float4 away = odd ? make_float4(v[0], v[1], v[2], v[3]) : make_float4(v[4], v[5], v[6], v[7]);
  away.x = __shfl_xor_sync(0xFFFFFFFFu, away.x, 1);
  away.y = __shfl_xor_sync(0xFFFFFFFFu, away.y, 1);
  away.z = __shfl_xor_sync(0xFFFFFFFFu, away.z, 1);
  away.w = __shfl_xor_sync(0xFFFFFFFFu, away.w, 1);
  // even: its own first half, the odd lane's first half; odd: the even lane's second half, its own second half
  float4* q = reinterpret_cast<float4*>(odd ? p - 8 : p) + (odd ? 1 : 0);
  __stcs(q, odd ? away : mine);
  __stcs(q + 2, odd ? mine : away);
}
PE_DEV void put8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&t);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// A warp's place: eight rows (lane / 4 the row), pieces piece, piece + along, ... ; lane % 4 is the quarter of a block.
struct MxPlace {
  int warp, quarter, along, piece;
  long long row0, row;
  PE_DEV explicit MxPlace(const MxDeal& d) {
    warp = threadIdx.x >> 5;
    quarter = threadIdx.x & 3;
    along = 1 << d.along_log2;
    row0 = ((long long)blockIdx.x * (kMxWarps >> d.along_log2) + (warp >> d.along_log2)) * 8;
    row = row0 + ((threadIdx.x & 31) >> 2);
    piece = (int)blockIdx.y * along * d.steps + (warp & (along - 1));
  }
};

// Four lanes take a block, eight entries each, so that a warp's loads are 64 bytes or more side by side and its stores of
// codes 128 (a lane a block: half the sectors of every access unused, and twice the registers).
// VEC: rows start at 16-byte boundaries.  Otherwise the warp reads each row's 128 entries side by side into a tile in
// shared memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads) mx_quantize_kernel(const MxRowsArgs a, const MxDeal d) {
  __shared__ float tiles[VEC ? 1 : kMxWarps][VEC ? 1 : 8 * kMxTileRow];
  const MxPlace at(d);
  const bool live = at.row < a.n_rows;
  const int r = (int)(at.row & (kMxPiece - 1)), lane = threadIdx.x & 31;
  const T* src = static_cast<const T*>(a.x) + at.row * a.stride + at.quarter * 8;
  uint8_t* rec = a.mx + ((size_t)(at.row / kMxPiece) * d.pieces) * kMxRecord;
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  int piece = at.piece;
  for (int i = 0; i < d.steps && piece < d.pieces; ++i, piece += at.along) {
    const int left = a.width - piece * kMxPiece;
    float x[4][8];
    if constexpr (VEC) {
      const T* p = src + (size_t)piece * kMxPiece;
      if (live && left >= kMxPiece) {
#pragma unroll
        for (int b = 0; b < 4; ++b) get8(p + b * kMxBlock, x[b]);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          get8_of(p + b * kMxBlock, live ? left - b * kMxBlock - at.quarter * 8 : 0, x[b]);
      }
    } else {
      using Bits = typename BitsOf<T>::type;
      float* tile = tiles[at.warp];
      // Loaded together, each is a trip to memory: what is not there is read from another place, since loads under a
      // condition wait for each other (16-bit ones: 24.9 us for 2316 x 6919 instead of 12.2).  Plain loads: the kernel before
      // this one may still write x when this one starts, which the read-only path does not allow.
      Bits raw[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const long long row = min(at.row0 + j, (long long)a.n_rows - 1);
        const Bits* p = reinterpret_cast<const Bits*>(static_cast<const T*>(a.x) + row * a.stride + (size_t)piece * kMxPiece);
#pragma unroll
        for (int e = 0; e < 4; ++e) raw[j][e] = p[min(e * 32 + lane, left - 1)];
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          tile[j * kMxTileRow + e * 32 + lane] = e * 32 + lane < left ? widen<T>(raw[j][e]) : 0.f;
      __syncwarp();
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(tile + (lane >> 2) * kMxTileRow + b * kMxBlock +
                                                            at.quarter * 8 + 4 * k);
          x[b][4 * k] = v.x; x[b][4 * k + 1] = v.y; x[b][4 * k + 2] = v.z; x[b][4 * k + 3] = v.w;
        }
    }
    uint8_t* out = rec + (size_t)piece * kMxRecord;
    uint32_t s4 = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      uint32_t codes, scale;
      bad |= mx_round8(x[b], codes, scale);
      s4 |= scale << (8 * b);
      if (live) reinterpret_cast<uint32_t*>(out + mx_code_at(r, b))[at.quarter] = codes;
    }
    if (live && at.quarter == 0) *reinterpret_cast<uint32_t*>(out + mx_scale_at(r, 0)) = s4;
  }
  if (bad) set_err(a.err, PE_DEV_NONFINITE);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads) mx_dequantize_kernel(const MxRowsArgs a, const MxDeal d) {
  __shared__ float tiles[VEC ? 1 : kMxWarps][VEC ? 1 : 8 * kMxTileRow];
  const MxPlace at(d);
  const bool live = at.row < a.n_rows;
  const int r = (int)(at.row & (kMxPiece - 1)), lane = threadIdx.x & 31;
  const uint8_t* rec = a.mx + ((size_t)(at.row / kMxPiece) * d.pieces) * kMxRecord;
  T* dst = static_cast<T*>(a.out) + at.row * a.stride + at.quarter * 8;
  pdl_wait();
  pdl_trigger();
  int piece = at.piece;
  for (int i = 0; i < d.steps && piece < d.pieces; ++i, piece += at.along) {
    const int left = a.width - piece * kMxPiece;
    uint32_t w[4] = {}, s4 = 0;
    if (live) {
      const uint8_t* in = rec + (size_t)piece * kMxRecord;
      s4 = __ldcs(reinterpret_cast<const uint32_t*>(in + mx_scale_at(r, 0)));
#pragma unroll
      for (int b = 0; b < 4; ++b) w[b] = __ldcs(reinterpret_cast<const uint32_t*>(in + mx_code_at(r, b)) + at.quarter);
    }
    if (!VEC) __syncwarp();
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float s = mx_scale(s4 >> (8 * b) & 255u);
      uint32_t h[4];
      mx_decode8(w[b], h);
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[e]));
        v[2 * e] = f.x * s;
        v[2 * e + 1] = f.y * s;
      }
      if constexpr (VEC) {
        T* out = dst + (size_t)piece * kMxPiece + b * kMxBlock;
        const int n = left - b * kMxBlock - at.quarter * 8;
        if (at.row0 + 8 <= a.n_rows && left >= (b + 1) * kMxBlock) {  // whole warps
          put8(out, v);
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) out[e] = from_float<T>(v[e]);
        }
      } else {
        float4* tile = reinterpret_cast<float4*>(tiles[at.warp] + (lane >> 2) * kMxTileRow + b * kMxBlock + at.quarter * 8);
        tile[0] = make_float4(v[0], v[1], v[2], v[3]);
        tile[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    if constexpr (!VEC) {
      __syncwarp();
      for (int j = 0; j < 8 && at.row0 + j < a.n_rows; ++j) {
        T* p = static_cast<T*>(a.out) + (at.row0 + j) * a.stride + (size_t)piece * kMxPiece;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = e * 32 + lane;
          if (c < left) p[c] = from_float<T>(tiles[at.warp][j * kMxTileRow + c]);
        }
      }
    }
  }
}

template <typename T>
cudaError_t quantize_typed(const MxRowsArgs& a, cudaStream_t s) {
  dim3 grid;
  const MxDeal d = mx_deal(a.n_rows, a.width, &grid);
  return a.vec ? launch_pdl(mx_quantize_kernel<T, true>, grid, dim3(kMxThreads), 0, s, a, d)
               : launch_pdl(mx_quantize_kernel<T, false>, grid, dim3(kMxThreads), 0, s, a, d);
}
template <typename T>
cudaError_t dequantize_typed(const MxRowsArgs& a, cudaStream_t s) {
  dim3 grid;
  const MxDeal d = mx_deal(a.n_rows, a.width, &grid);
  return a.vec ? launch_pdl(mx_dequantize_kernel<T, true>, grid, dim3(kMxThreads), 0, s, a, d)
               : launch_pdl(mx_dequantize_kernel<T, false>, grid, dim3(kMxThreads), 0, s, a, d);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxRowsArgs& a, pe_dtype dt, cudaStream_t s) {
  return dt == PE_BF16 ? quantize_typed<__nv_bfloat16>(a, s) : quantize_typed<float>(a, s);
}

cudaError_t launch_mx_dequantize(const MxRowsArgs& a, pe_dtype dt, cudaStream_t s) {
  return dt == PE_BF16 ? dequantize_typed<__nv_bfloat16>(a, s) : dequantize_typed<float>(a, s);
}

}  // namespace pe
