// Grouped-query attention of ragged query rows over a packed (4-bit) paged cache.
// The cache's format is in pe_packed.cuh.
//
// Row r of sequence b (rows row_start[b] .. row_start[b+1] - 1) at position p attends to the
// cache positions 0..p of its sequence:
//   out[r][h] = sum_{x <= p} w_x v_x / sum_{x <= p} w_x,  w_x = exp(q[r][h] . k_x / sqrt(hd) - max)
// with keys and values of head h / (n_q / n_kv).  A row at position -1 sees nothing: zeros.
//
// Work.  The query vectors of a sequence and kv head (rows x G query heads, G = n_q / n_kv) are
// cut into tiles; a (tile, kv head) pair's range of positions is counted in units.  All ranges of
// the launch form one line (tile after tile, head after head, unit after unit), a range a little longer
// than its units, for what its start costs.  N CTAs divide the line into pieces of about one length, so
// ragged lengths leave no CTA idle; a unit belongs to the piece in which it starts.  A range that lies in
// one CTA's piece is finished there; one that is cut leaves a record per CTA (reference maximum,
// sum, unnormalised output) that the merge kernel joins in CTA order.  Every CTA works the line
// out for itself from row_start and positions (two dependent loads and a scan), which costs less
// than a launch and a round trip through memory for a kernel that would do it once.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "pe_internal.h"
#include "pe_packed.cuh"

namespace pe {

namespace {

constexpr int kPlanTiles = 1024;    // tiles per launch (their line is held in shared memory)
constexpr float kRescaleLog2 = 8.f; // a reference maximum moves when a score exceeds it by more (log2 units)

PE_DEV float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
PE_DEV uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
PE_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// A wait's outcome, made the same for the whole warp.
PE_DEV bool warp_ok(bool ok) { return __all_sync(0xFFFFFFFFu, ok); }

// r / d where the quotient is at most 2^16: the fp32 quotient is off by one at most.
PE_DEV uint32_t small_quotient(uint32_t r, uint32_t d) {
  uint32_t q = (uint32_t)__fdividef((float)r, (float)d);
  if ((uint64_t)q * d > r) --q;
  else if (r - q * d >= d) ++q;
  return q;
}

// The factor of a vector's output.  Without a positive sum of weights its row sees nothing (zeros), or its
// scores are NaN or infinite (NaN, as the formula gives).  Joins take the sums of parts without a maximum (-inf)
// as well: NaN where the scores were.
PE_DEV float normaliser(float sum, bool sees) {
  return sum > 0.f ? kPackedUnit / sum : sees ? __int_as_float(0x7FFFFFFF) : 0.f;
}

// ----------------------------------------------------------------------------- the line of work

struct Line {
  int tile0, n_tiles;  // this launch's tiles: b * tps + t
  Div tps;             // tiles per sequence (host bound)
  int n_tps;
  Div group, heads;    // query heads per kv head, kv heads
  Div grid;            // CTAs launched
  Div half;            // half of it (tile kernel)
  int older;           // CTAs that take the longer pieces, half the grid, or 0
  int G;
  int tile_rows;       // query vectors per tile, 2^rows_log2
  int rows_log2;
  int unit_pages;      // pages per unit
  int lanes;           // threads that look through one tile's rows (a power of two, at most 32)
  int whole;           // CTAs take whole ranges
  int sms;
  int pair_log2;       // pieces are at least 2^this long where there are more than SMs
  int range_cost;      // of a range's start, in units
  int* prefix;         // workspace [n_tiles + 1]: cost per head before each tile, for the merge
  float* part;         // workspace: records of cut ranges, two per CTA
  float* spill;        // workspace: a warp's piece of a range that began before it (small kernel)
};

struct TileRows {
  int r0, m0, M;  // first row of the sequence, first vector of the tile, vectors of the tile (0: none)
};

// The rows of tile `tile`, and whether its sequence's are out of bounds (then none).  Here and in
// row_limit errors are flagged, not reported: a report would hold the next loads back.
PE_DEV TileRows tile_rows(const PackedAttnArgs& a, const Line& ln, int tile, bool& bad) {
  const int b = (int)((uint32_t)tile / ln.tps), t = tile - b * ln.n_tps;
  const int r0 = __ldcg(a.row_start + b);
  const int next = __ldcg(a.row_len != nullptr ? a.row_len + b : a.row_start + b + 1);
  const int r1 = a.row_len != nullptr ? r0 + next : next;
  const bool out = r0 < 0 || r1 < r0 || r1 > a.n_rows || r1 - r0 > a.max_rows;
  bad |= out && r1 != r0;
  const int m0 = t * ln.tile_rows;
  return TileRows{out ? 0 : r0, m0, out ? 0 : max(0, min((r1 - r0) * ln.G - m0, ln.tile_rows))};
}

// A row's last visible position: -1 when it sees nothing or its position is out of range.
PE_DEV int row_limit(const PackedAttnArgs& a, int p, bool& bad) {
  const bool out = p < -1 || p / kPackedPage >= a.max_pages;
  bad |= out;
  return out ? -1 : p;
}

// Whether a row sees a position (for the few vectors without a sum of weights: a load each).
PE_DEV bool row_sees(const PackedAttnArgs& a, int row) {
  bool bad = false;  // reported by lay_out
  return row_limit(a, __ldcg(a.positions + row), bad) >= 0;
}

// The line in shared memory, each array of n_tiles (+ 1) entries.
struct Layout {
  int* prefix;  // cost per head before the tile
  int* last;    // largest position that the tile sees (-1: none)
  int* row0;    // its TileRows
  int* rows;
  static constexpr int kBytesPerTile = 16;
  PE_DEV Layout(void* smem, int n) : prefix(static_cast<int*>(smem)), last(prefix + n + 1), row0(last + n), rows(row0 + n) {}
  PE_DEV TileRows tile(const Line& ln, int k) const {
    const int tile = ln.tile0 + k;
    return TileRows{row0[k], (tile - (int)((uint32_t)tile / ln.tps) * ln.n_tps) * ln.tile_rows, rows[k]};
  }
};

PE_DEV int range_units(const Line& ln, int last) {  // at least one: a range that sees nothing has to be zeroed
  return max(1, (last / kPackedPage + ln.unit_pages) >> (ln.unit_pages == 2 ? 1 : 2));
}
PE_DEV int tile_cost(const Line& ln, const TileRows& t, int last) {
  return t.M == 0 ? 0 : range_units(ln, last) + ln.range_cost;
}

// Fills the line in.  Every thread of the CTA.
PE_DEV void lay_out(const PackedAttnArgs& a, const Line& ln, const Layout& lo, int* warp_sums) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  const int n = ln.n_tiles;
  constexpr int W = 4;  // tiles per lane
  bool bad_rows = false, bad_pos = false;
  if (n <= 32 * W && ln.lanes == 1) {
    // few tiles of few rows: every warp works the whole line out (the same values go to the same places), so
    // that none waits for another.  Two round trips: the rows of every tile, then their positions.
    TileRows t[W];
    int pos[W][4], mx[W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int k = lane + 32 * i;
      t[i] = TileRows{0, 0, 0};
      if (k < n) t[i] = tile_rows(a, ln, ln.tile0 + k, bad_rows);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int ra = t[i].r0 + (int)((uint32_t)t[i].m0 / ln.group);
      const int rb = t[i].r0 + (int)((uint32_t)(t[i].m0 + t[i].M - 1) / ln.group);
#pragma unroll
      for (int r = 0; r < 4; ++r) pos[i][r] = t[i].M > 0 && ra + r <= rb ? __ldcg(a.positions + ra + r) : -1;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      mx[i] = -1;
#pragma unroll
      for (int r = 0; r < 4; ++r) mx[i] = max(mx[i], row_limit(a, pos[i][r], bad_pos));
    }
    int before = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int k = lane + 32 * i;
      if (32 * i >= n) break;
      int inc = tile_cost(ln, t[i], mx[i]);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
      }
      inc += before;
      if (k < n) {
        lo.prefix[k + 1] = inc;
        lo.last[k] = mx[i];
        lo.row0[k] = t[i].r0;
        lo.rows[k] = t[i].M;
      }
      before = __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
    if (lane == 0) lo.prefix[0] = 0;
    __syncwarp();
    if (bad_rows) set_err(a.err, PE_DEV_BAD_ROW);
    if (bad_pos) set_err(a.err, PE_DEV_BAD_POSITION);
    return;
  }
  const int per = ln.lanes, sub = tid & (per - 1);
  for (int k0 = 0; k0 < n; k0 += nt / per) {  // the same trip count for every thread
    const int k = k0 + tid / per;
    int mx = -1;
    TileRows t{0, 0, 0};
    if (k < n) {
      t = tile_rows(a, ln, ln.tile0 + k, bad_rows);
      if (t.M > 0) {
        const int ra = t.r0 + (int)((uint32_t)t.m0 / ln.group);
        const int rb = t.r0 + (int)((uint32_t)(t.m0 + t.M - 1) / ln.group);
        for (int r = ra + sub; r <= rb; r += 4 * per) {
          int pos[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) pos[i] = r + i * per <= rb ? __ldcg(a.positions + r + i * per) : -1;
#pragma unroll
          for (int i = 0; i < 4; ++i) mx = max(mx, row_limit(a, pos[i], bad_pos));
        }
      }
    }
    for (int o = per >> 1; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    if (k < n && sub == 0) {
      lo.prefix[k + 1] = tile_cost(ln, t, mx);
      lo.last[k] = mx;
      lo.row0[k] = t.r0;
      lo.rows[k] = t.M;
    }
  }
  if (bad_rows) set_err(a.err, PE_DEV_BAD_ROW);
  if (bad_pos) set_err(a.err, PE_DEV_BAD_POSITION);
  __syncthreads();
  // inclusive scan of prefix[1..n]: a run of consecutive tiles per thread, then over threads
  const int run = (n + nt - 1) / nt, k0 = tid * run, k1 = min(n, k0 + run);
  int sum = 0;
  for (int k = k0; k < k1; ++k) sum += lo.prefix[k + 1];
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warp_sums[tid >> 5] = inc;
  __syncthreads();
  int before = inc - sum;
  for (int w = 0; w < (tid >> 5); ++w) before += warp_sums[w];
  if (tid == 0) lo.prefix[0] = 0;
  for (int k = k0; k < k1; ++k) {
    before += lo.prefix[k + 1];
    lo.prefix[k + 1] = before;
  }
  __syncthreads();
}

// A line of length T in n pieces: n is the grid, or less where that would leave a piece shorter than four units,
// or than 2^pair_log2 where there are more pieces than SMs (a piece's start and its records cost more than
// a CTA beside another saves).  Tiles: 14 rows of 8 heads over 4000 positions, 4 kv heads of 128, 16 us (20 with
// eight units throughout); four sequences of them, 8 kv heads, 25.6 us with 16 units (30.9 with eight).  Single
// tokens: 16 sequences over 4000 positions, 4 kv heads of 128, 18.6 us with eight units (19.4 with 16).
//
// Pieces are equal (the first of them one longer where it does not come out even), except that of the tile
// kernel's two CTAs an SM the older ones, the first half of the grid, take more than half of the line: schedulers
// prefer the older warps, and with equal halves the younger CTA ended 13 % later.  36 of 64 took draft blocks
// at B = 64 from 151 to 146 us (34: 148.5, 40: 151).  Single tokens, whose warps fill the SM's instruction
// slots alone as well as in pairs, gained nothing (66 us, 67 with 34).
constexpr int kLoneLog2 = 2;
constexpr int kOlderShare = 36;  // of 64
struct Cuts {
  uint32_t n, h, T1, q1, r1, q2, r2;  // the first h pieces: T1, each q1 and the first r1 of them one longer; the rest
  PE_DEV Cuts(const Line& ln, int grid, uint32_t T) {
    n = grid;
    h = (T >> 4) >= n ? ln.older : 0;  // (not for pieces of a few units)
    const uint32_t busy = ln.whole ? T : max(T >> ln.pair_log2, min(T >> kLoneLog2, (uint32_t)ln.sms));
    if (busy < n) {
      n = max(1u, busy);
      h = 0;
      q2 = small_quotient(T, n);
      r2 = T - q2 * n;
    } else if (h == 0) {
      q2 = T / ln.grid;
      r2 = T - q2 * n;
    }
    T1 = q1 = r1 = 0;
    if (h != 0) {  // as many younger as older ones
      T1 = (T >> 6) * kOlderShare;
      q1 = T1 / ln.half;
      r1 = T1 - q1 * h;
      q2 = (T - T1) / ln.half;
      r2 = T - T1 - q2 * h;
    }
  }
  PE_DEV uint32_t first(uint32_t c) const {
    return c < h ? q1 * c + min(c, r1) : T1 + q2 * (c - h) + min(c - h, r2);
  }
  PE_DEV uint32_t piece(uint32_t u) const {  // the one that holds u
    const bool young = u >= T1;
    const uint32_t q = young ? q2 : q1, r = young ? r2 : r1, longer = r * (q + 1);
    if (young) u -= T1;
    return (young ? h : 0) + (u < longer ? small_quotient(u, q + 1) : r + small_quotient(u - longer, q));
  }
};

// The part of a (tile, head) range that a piece of the line holds.
struct Segment {
  int k, g;          // tile (of this launch), kv head
  int page0, page1;  // its pages
  bool any;          // a unit starts in the piece
  bool from_start, to_end;
  uint32_t next;     // where the line goes on
};

struct Walk {
  const Line& ln;
  const Layout& lo;
  int n_kv;

  PE_DEV int tile_of(uint32_t u) const {  // the last tile that starts at or before u (the whole warp)
    int at = 0;
    for (int step = 1024; step > 0; step >>= 5) {  // 32 places at a time: the 1024 tiles of a launch in three rounds
      if (step > ln.n_tiles) continue;
      const int k = at + (int)(threadIdx.x & 31) * step;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, k < ln.n_tiles && (uint32_t)lo.prefix[min(k, ln.n_tiles)] * n_kv <= u);
      at += (31 - __clz(hit)) * step;
    }
    return at;
  }
  PE_DEV Segment at(int k, uint32_t u, uint32_t u1) const {
    Segment s;
    const uint32_t p0 = lo.prefix[k], len = lo.prefix[k + 1] - p0;
    uint32_t r = u - p0 * n_kv;
    s.k = k;
    s.g = (int)small_quotient(r, len);
    r -= s.g * len;
    const uint32_t end = min(len, r + (u1 - u));
    s.next = u + (end - r);
    // unit i starts at range_cost + i
    const int b0 = max(0, (int)r - ln.range_cost), b1 = max(0, (int)end - ln.range_cost);
    s.any = b1 > b0;
    s.from_start = b0 == 0;
    s.to_end = end == len;
    s.page0 = b0 * ln.unit_pages;
    s.page1 = min((lo.last[k] + kPackedPage) / kPackedPage, b1 * ln.unit_pages);
    return s;
  }
  // The first segment of [u, u1) with a unit, and the one behind `s`; false where there is none.
  PE_DEV bool skip_empty(Segment& s, uint32_t u1) const {
    while (!s.any)
      if (!step(s, u1)) return false;
    return true;
  }
  PE_DEV bool step(Segment& s, uint32_t u1) const {
    if (s.next >= u1) return false;
    int k = s.k;
    if (s.next >= (uint32_t)lo.prefix[k + 1] * n_kv)
      do ++k;
      while (lo.prefix[k + 1] == lo.prefix[k]);
    s = at(k, s.next, u1);
    return true;
  }
  PE_DEV bool first(Segment& s, uint32_t u, uint32_t u1) const {
    if (u >= u1) return false;
    s = at(tile_of(u), u, u1);
    return skip_empty(s, u1);
  }
  PE_DEV bool next(Segment& s, uint32_t u1) const { return step(s, u1) && skip_empty(s, u1); }
  // The start of the range that holds u (u < T).
  PE_DEV uint32_t range_start(uint32_t u) const {
    const int k = tile_of(u);
    const uint32_t p0 = lo.prefix[k], len = lo.prefix[k + 1] - p0, r = u - p0 * n_kv;
    return u - (r - small_quotient(r, len) * len);
  }
};

// The piece of this CTA: [u0, u1) of T.
PE_DEV void cta_piece(const Line& ln, const Walk& w, uint32_t T, uint32_t& u0, uint32_t& u1) {
  u0 = u1 = 0;
  const Cuts cuts(ln, gridDim.x, T);
  if (T == 0 || blockIdx.x >= cuts.n) return;
  u0 = cuts.first(blockIdx.x);
  u1 = cuts.first(blockIdx.x + 1);
  if (ln.whole) {
    u0 = w.range_start(u0);
    if (u1 < T) u1 = w.range_start(u1);
  }
}

// A record of a cut range: maximum and sum of each vector, then the outputs.
template <int HD>
PE_DEV float* part_record(const Line& ln, int cta, bool from_start) {
  return ln.part + (size_t)(2 * cta + (from_start ? 1 : 0)) * ln.tile_rows * (HD + 2);
}

// ----------------------------------------------------------------------------- few query vectors: warp MMAs
//
// A warp takes pairs of pages (32 positions), brought into its own ring of shared-memory stages by
// 16-byte asynchronous copies of its lanes (a bulk copy per page took longer to issue: the SM's copy
// unit saw a request per 1152 bytes): S^T = K Q^T and O^T += V^T P^T with
// 16 x 8 x 16 warp MMAs, positions (then entries) on the 16 side and 8 query vectors on the other, so one
// unpacked page serves NQ * 8 vectors and no row is padded beyond 8.
//   Scales: each lane turns a few of a page's scale bytes into bf16 pairs, into a small table that the
//   others read: a lane needs the scales of eight rows, and converting them all itself cost 36 of
//   400 instructions a page.
//   Values: two positions' words give pairs of positions; P is rounded to bf16 and transposed by
//   movmatrix into the other operand.
// bf16: P is rounded to bf16, as the queries and outputs are and as in attn_bf16_kernel (half a step, 2^-8 of a
// weight; a second term would double the products).
// fp32: q and P are each split into three bf16 terms (24 bits), three MMAs for one; keys and values
// are exact in bf16, so the products are those of fp32.  The tensor cores cut what they add to an accumulator
// instead of rounding it, so each page's PV starts at zero and is added to O in fp32: over 16,384 positions outputs
// are off by 8e-7 of the largest (1.6e-5, all towards zero, through one accumulator, for 3 to 12 % less time).  Against
// bf16's rounding the cut is nothing (1e-5 there).
// A CTA's piece of the line is divided once more, evenly, among its eight warps, each of which runs on its
// own over whole ranges, or parts, of its piece; at the end the parts of ranges that the warps
// share join in shared memory.  (Dividing every range among the eight warps instead, with a join
// after each, left SMs with many short ranges behind the others: an eighth more time at B = 64
// single tokens.)
//
// Bound: unpacking.  A page of one head is 1152 bytes at head_dim 64: an SM's share of the HBM rate
// brings it in about 50 cycles, in which it can issue about 200 instructions, half of them to the
// integer pipe; a page takes 267, in a chain (copies, tables, scores, softmax, values) that a warp goes through
// pair by pair, with 16 warps an SM to fill each other's waits.  B = 64 single tokens of 64 query heads over 8 kv heads of
// 64, up to 16384 positions (163 MB): 60 to 62 us, 2.7 TB/s, schedulers busy 60 % of the time and the integer pipe
// 54 %.  One token over 131,072 positions, 4 kv heads of 128 (75 MB): 34 us, 2.2 TB/s, 50 and 47 %.

constexpr int kSmallWarps = 8;
constexpr int kSmallRangeCost = 1;  // a range's start costs about as much as a pair of pages

// A warp's part of a range that it shares with its neighbours: [ROWS][OROW] outputs, [ROWS] maxima, [ROWS]
// sums, in its ring or (a part that began before the warp's piece, when more ranges follow) in the
// workspace.
enum : int { kFirst = 1, kFirstEnds = 2, kFirstSpilled = 4, kSecond = 8 };
struct Parts {
  int state;             // kFirst: a part of a range that began before the warp; kSecond: of one that begins in it
  int k[2], g[2], pad[3];  // their tiles and heads
};

template <typename T, int HD, int NQ>
struct Small {
  static constexpr int TERMS = sizeof(T) == 4 ? 3 : 1;
  static constexpr int STAGES = HD == 64 ? 3 : 2;  // pairs of pages in flight per warp
  static constexpr int ROWS = 8 * NQ;
  static constexpr int OROW = HD + 4;  // floats per vector of the joint buffer (no bank conflicts)
  static constexpr int CTAS = TERMS == 1 && (NQ == 1 || HD == 64) ? 2 : 1;  // per SM
  static constexpr int STAGE = 2 * PackedLayout<HD>::kRecord;
  static constexpr int RING = kSmallWarps * STAGES * STAGE;
  static constexpr int KTAB = HD * 4, VTAB = HD * 2, TAB = 2 * (KTAB + VTAB);  // scale tables of a warp (two pages)
  static constexpr int PIECE = ROWS * (OROW + 2);  // floats of a warp's part of a shared range
  static_assert(PIECE * 4 <= STAGES * STAGE, "it fits the warp's drained ring");
  static constexpr int FIXED = RING + kSmallWarps * TAB + 16 * 4 + kSmallWarps * (int)sizeof(Parts);
  static size_t smem(int n_tiles) { return 128 + FIXED + Layout::kBytesPerTile * (size_t)n_tiles + 4; }
};

PE_DEV void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
PE_DEV void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
PE_DEV void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

PE_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
PE_DEV uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Pairs (x0, x1) as `TERMS` bf16 pairs whose sums are x0 and x1 (one term: rounded to bf16).
template <int TERMS>
PE_DEV void split_pair(float x0, float x1, uint32_t (&t)[TERMS]) {
#pragma unroll
  for (int k = 0; k < TERMS; ++k) {
    t[k] = pack_bf16(x0, x1);
    if (k + 1 < TERMS) {
      x0 -= __uint_as_float(t[k] << 16);
      x1 -= __uint_as_float(t[k] & 0xFFFF0000u);
    }
  }
}

// The scale tables of one page.  ktab: [16 positions][HD/16 blocks] pairs (S, S); vtab:
// [position t][t + 8 or not][HD/16 blocks] pairs (S of position t or t + 8, S of the position 4 after it).
template <int HD>
PE_DEV void scale_tables(const uint8_t* rec, uint8_t* ktab, uint8_t* vtab, int lane) {
  using L = PackedLayout<HD>;
  constexpr int NB = HD / 16;
  {
    // NB/2 neighbouring bytes of a row per lane
    const int pos = lane >> 1, j0 = (lane & 1) * (NB / 2);
    uint32_t c;
    if constexpr (NB == 4) c = *reinterpret_cast<const uint16_t*>(rec + L::kKs + pos * NB + j0);
    else c = *reinterpret_cast<const uint32_t*>(rec + L::kKs + pos * NB + j0);
    const uint32_t s01[2] = {packed_scale_lo(__byte_perm(c, 0, 0x4040)), packed_scale_lo(__byte_perm(c, 0, 0x4141))};
    if constexpr (NB == 4) {
      *reinterpret_cast<uint2*>(ktab + (pos * NB + j0) * 4) = make_uint2(s01[0], s01[1]);
    } else {
      const uint32_t s23[2] = {packed_scale_lo(__byte_perm(c, 0, 0x4242)), packed_scale_lo(__byte_perm(c, 0, 0x4343))};
      *reinterpret_cast<uint4*>(ktab + (pos * NB + j0) * 4) = make_uint4(s01[0], s01[1], s23[0], s23[1]);
    }
  }
#pragma unroll
  for (int h = 0; h < NB / 4; ++h) {
    const int row = lane >> 2, j = (lane & 3) + 4 * h;  // row = 2 * t + (8 more)
    const int pos = (row >> 1) + 8 * (row & 1);
    const uint32_t c0 = rec[L::kVs + pos * NB + j], c1 = rec[L::kVs + (pos + 4) * NB + j];
    *reinterpret_cast<uint32_t*>(vtab + (row * NB + j) * 4) = packed_scale_lo(c0 | c1 << 16);
  }
}

template <typename T, int HD, int NQ>
__global__ void __launch_bounds__(kSmallWarps * 32, (Small<T, HD, NQ>::CTAS))
    attend_small_kernel(const PackedAttnArgs a, const Line ln) {
  using S = Small<T, HD, NQ>;
  using L = PackedLayout<HD>;
  constexpr int NB = HD / 16, TERMS = S::TERMS;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 127) & ~uintptr_t(127));
  uint8_t* tabs = sm + S::RING;
  int* scratch = reinterpret_cast<int*>(tabs + kSmallWarps * S::TAB);  // [16]
  Parts* parts = reinterpret_cast<Parts*>(scratch + 16);               // [warps]
  const Layout lo(parts + kSmallWarps, ln.n_tiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  uint8_t* my_ring = sm + warp * S::STAGES * S::STAGE;
  uint8_t* my_tab = tabs + warp * S::TAB;
  const int G = ln.G;
  const float sl2 = a.scale * 1.4426950408889634f * kPackedUnit;
  const PairBits bits;
  float* spill = ln.spill + (size_t)blockIdx.x * kSmallWarps * S::PIECE;
  if (lane == 0) parts[warp].state = 0;
  pdl_wait();
  pdl_trigger();
  lay_out(a, ln, lo, scratch);
  const Walk walk{ln, lo, a.n_kv};
  const uint32_t total = (uint32_t)lo.prefix[ln.n_tiles] * a.n_kv;
  if (blockIdx.x == 0 && !ln.whole)
    for (int k = tid; k <= ln.n_tiles; k += blockDim.x) ln.prefix[k] = lo.prefix[k];
  uint32_t u0, u1;
  cta_piece(ln, walk, total, u0, u1);
  if (u0 == u1) return;  // the whole CTA
  {
    const uint32_t n = u1 - u0;
    const uint32_t c0 = (n >> 3) * warp + min((uint32_t)warp, n & 7);
    const uint32_t c1 = (n >> 3) * (warp + 1) + min((uint32_t)warp + 1, n & 7);
    u1 = u0 + c1;
    u0 += c0;
  }
  static_assert(kSmallWarps == 8, "");

  // Two walks over the pairs of pages of the warp's units, the copies `STAGES` pairs ahead of the
  // products.  A unit is a pair, so a pair lacks its second page at a range's end only, where every
  // position of that page is masked.
  Segment ps{}, cs;
  const bool some = walk.first(ps, u0, u1);
  bool p_done = !some;
  cs = ps;
  int p_page = ps.page0;  // the next pair of the segment
  int ids = -1;           // page ids of the 16 pairs from p_page - p_id on, one per lane
  int p_id = 0;
  const uint32_t step = (uint32_t)a.n_kv * L::kRecord;
  const uint8_t* head = a.pool + (size_t)ps.g * L::kRecord + lane * 16;  // of the segment's head, in page 0
  uint32_t issued = 0, used = 0, stage_in = smem_u32(my_ring) + lane * 16;
  const uint32_t ring_end = stage_in + S::RING / kSmallWarps;
  auto issue = [&]() {
    while (p_page >= ps.page1) {
      if (!walk.next(ps, u1)) {
        p_done = true;
        return;
      }
      p_page = ps.page0;
      p_id = 0;
      head = a.pool + (size_t)ps.g * L::kRecord + lane * 16;
    }
    if (p_id == 0) {
      const int x = p_page + lane;
      ids = -1;
      if (x < ps.page1) {
        ids = __ldcg(a.block_table + (size_t)((uint32_t)(ln.tile0 + ps.k) / ln.tps) * a.max_pages + x);
        if (ids < 0 || ids >= a.num_pages) {
          set_err(a.err, PE_DEV_BAD_PAGE);
          ids = -1;
        }
      }
    }
    const int id0 = __shfl_sync(0xFFFFFFFFu, ids, p_id), id1 = __shfl_sync(0xFFFFFFFFu, ids, p_id + 1);
    if ((id0 | id1) >= 0) {
      const uint8_t* src0 = head + (uint64_t)(uint32_t)id0 * step;
      const uint8_t* src1 = head + (uint64_t)(uint32_t)id1 * step - L::kRecord;
#pragma unroll
      for (int i = 0; i < (S::STAGE + 511) / 512; ++i) {
        const int at = i * 512 + lane * 16;  // byte of the two records
        const bool first = i * 512 + 511 < L::kRecord || (i * 512 < L::kRecord && at < L::kRecord);
        if (i * 512 + 511 < S::STAGE || at < S::STAGE) copy16(stage_in + i * 512, (first ? src0 : src1) + i * 512);
      }
    } else {
      // a page outside the pool stands for zeros, every nibble 8; so may the page behind the range
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int id = h == 0 ? id0 : id1;
        for (int i = 0; i + lane * 16 < L::kRecord; i += 512) {
          const uint32_t d = stage_in + h * L::kRecord + i;
          if (id >= 0) copy16(d, head + (uint64_t)(uint32_t)id * step + i);
          else asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(d), "r"(0x88888888u) : "memory");
        }
      }
    }
    stage_in = stage_in + S::STAGE == ring_end ? ring_end - S::RING / kSmallWarps : stage_in + S::STAGE;
    p_page += 2;
    p_id = (p_id + 2) & 31;
  };
  const uint8_t* recs = my_ring;  // the stage to be used next

  // rows 0..7 of a product stand for positions 0, 4, 1, 5, 2, 6, 3, 7 and rows 8..15 for 8 more, so that
  // the transposed P pairs positions t and t + 4
  const int kpos = (gr >> 1) + 4 * (gr & 1);
  while (some) {
    const TileRows tr = lo.tile(ln, cs.k);
    // offset of vector m of the sequence in the rows of q or out
    auto row_of = [&](int m, int g, long long stride) {
      const int r = (int)((uint32_t)m / ln.group);
      return (tr.r0 + r) * stride + (g * G + m - r * G) * HD;
    };
    // queries: the operand of block j and vector gr is entries 4t..4t+3 of the block
    uint32_t qf[TERMS][NQ][NB][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int m = tr.m0 + n * 8 + gr;
      const bool live = n * 8 + gr < tr.M;
      const T* q = static_cast<const T*>(a.q) + (live ? row_of(m, cs.g, a.q_stride) : 0);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if constexpr (TERMS == 1) {
          const uint2 v = live ? __ldcg(reinterpret_cast<const uint2*>(q + 16 * j + 4 * t)) : make_uint2(0, 0);
          qf[0][n][j][0] = v.x;
          qf[0][n][j][1] = v.y;
        } else {
          const float4 v = live ? __ldcg(reinterpret_cast<const float4*>(q + 16 * j + 4 * t)) : make_float4(0, 0, 0, 0);
          uint32_t x[TERMS], y[TERMS];
          split_pair<TERMS>(v.x, v.y, x);
          split_pair<TERMS>(v.z, v.w, y);
#pragma unroll
          for (int k = 0; k < TERMS; ++k) {
            qf[k][n][j][0] = x[k];
            qf[k][n][j][1] = y[k];
          }
        }
      }
    }
    int lim[NQ][2], min_lim = INT_MAX;
    bool bad_pos = false;  // reported by lay_out
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int v = n * 8 + 2 * t + e;
        lim[n][e] = INT_MAX;
        if (v < tr.M)
          lim[n][e] = row_limit(a, __ldcg(a.positions + tr.r0 + (int)((uint32_t)(tr.m0 + v) / ln.group)), bad_pos);
        min_lim = min(min_lim, lim[n][e]);
      }
    min_lim = min(min_lim, __shfl_xor_sync(0xFFFFFFFFu, min_lim, 1));
    min_lim = min(min_lim, __shfl_xor_sync(0xFFFFFFFFu, min_lim, 2));

    float o[NB][NQ][4], nm[NQ][2], l[NQ][2];  // outputs, minus the reference maxima (+inf: none yet), sums
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      nm[n][0] = nm[n][1] = INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NB; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
    }
#pragma unroll 1
    for (int page = cs.page0; page < cs.page1; page += 2) {
      // a group of copies per step, empty behind the last pair, so that the oldest of STAGES is this step's
#pragma unroll 1
      for (; issued < used + S::STAGES; ++issued) {
        if (!p_done) issue();
        copy_commit();
      }
      copy_wait<S::STAGES - 1>();
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint8_t* tab = my_tab + h * (S::KTAB + S::VTAB);
        scale_tables<HD>(recs + h * L::kRecord, tab, tab + S::KTAB, lane);
      }
      __syncwarp();
      // ---- scores
      float sc[2][NQ][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* rec = recs + h * L::kRecord + L::kK;
        const uint8_t* ktab = my_tab + h * (S::KTAB + S::VTAB);
        uint32_t kw[2][HD / 32], ks[2][NB];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int pos = kpos + 8 * r;
          if constexpr (HD == 64) {
            const uint2 w = *reinterpret_cast<const uint2*>(rec + pos * L::kRow + t * 8);
            kw[r][0] = w.x; kw[r][1] = w.y;
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(rec + pos * L::kRow + t * 16);
            kw[r][0] = w.x; kw[r][1] = w.y; kw[r][2] = w.z; kw[r][3] = w.w;
          }
#pragma unroll
          for (int j = 0; j < NB; j += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(ktab + (pos * NB + j) * 4);
            ks[r][j] = w.x; ks[r][j + 1] = w.y; ks[r][j + 2] = w.z; ks[r][j + 3] = w.w;
          }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) sc[h][n][0] = sc[h][n][1] = sc[h][n][2] = sc[h][n][3] = 0.f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint32_t w0 = kw[0][j / 2], w1 = kw[1][j / 2], s0 = ks[0][j], s1 = ks[1][j];
          const uint32_t z0 = bf16x2_mul(s0, kMinus136), z1 = bf16x2_mul(s1, kMinus136);
          const bool odd = j & 1;
          const uint32_t af[4] = {bf16x2_fma(odd ? bits.pair<2>(w0) : bits.pair<0>(w0), s0, z0),
                                  bf16x2_fma(odd ? bits.pair<2>(w1) : bits.pair<0>(w1), s1, z1),
                                  bf16x2_fma(odd ? bits.pair<3>(w0) : bits.pair<1>(w0), s0, z0),
                                  bf16x2_fma(odd ? bits.pair<3>(w1) : bits.pair<1>(w1), s1, z1)};
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int k = TERMS - 1; k >= 0; --k) mma16816(sc[h][n], af, qf[k][n][j][0], qf[k][n][j][1]);
        }
      }
      // ---- softmax
      const bool edge = (page + 2) * kPackedPage > min_lim + 1;
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((page + h) * kPackedPage + kpos + 8 * (e >> 1) > lim[n][e & 1]) sc[h][n][e] = -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][c + 2]), fmaxf(sc[1][n][c], sc[1][n][c + 2]));
          // a vector without a reference yet needs one unless all is masked (-inf plus +inf is no number)
          top = fmaxf(top, mx == -INFINITY ? mx : fmaf(mx, sl2, nm[n][c]));
        }
      if (__any_sync(0xFFFFFFFFu, top > kRescaleLog2)) {
        // a new reference maximum for every vector: the largest score so far
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float mx = fmaxf(fmaxf(sc[0][n][c], sc[0][n][c + 2]), fmaxf(sc[1][n][c], sc[1][n][c + 2])) * sl2;
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
            mx = fmaxf(mx, -nm[n][c]);
            const float f = nm[n][c] == INFINITY ? 0.f : ex2_approx(-nm[n][c] - mx);
            nm[n][c] = -mx;
            l[n][c] *= f;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
              o[j][n][c] *= f;
              o[j][n][c + 2] *= f;
            }
          }
      }
      uint32_t pf[2][TERMS][NQ][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2_approx(fmaf(sc[h][n][e], sl2, nm[n][e & 1]));
            if (edge && sc[h][n][e] == -INFINITY) p[e] = 0.f;  // no number where a vector has seen nothing yet
            l[n][e & 1] += p[e];
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t x[TERMS];
            split_pair<TERMS>(p[2 * r], p[2 * r + 1], x);
#pragma unroll
            for (int k = 0; k < TERMS; ++k) pf[h][k][n][r] = transpose8(x[k]);
          }
        }
      // ---- values
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* rec = recs + h * L::kRecord + L::kV;
        const uint8_t* vtab = my_tab + h * (S::KTAB + S::VTAB) + S::KTAB;
        uint32_t vw[4][HD / 64], vs[2][NB];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (HD == 64) {
            vw[i][0] = *reinterpret_cast<const uint32_t*>(rec + (t + 4 * i) * L::kRow + gr * 4);
          } else {
            const uint2 w = *reinterpret_cast<const uint2*>(rec + (t + 4 * i) * L::kRow + gr * 8);
            vw[i][0] = w.x; vw[i][1] = w.y;
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < NB; j += 4) {
            const uint4 w = *reinterpret_cast<const uint4*>(vtab + ((2 * t + r) * NB + j) * 4);
            vs[r][j] = w.x; vs[r][j + 1] = w.y; vs[r][j + 2] = w.z; vs[r][j + 3] = w.w;
          }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          const uint32_t sel = (j & 2) ? 0x7632u : 0x5410u;  // blocks 0, 1 of 64 entries in the lower halves
          const uint32_t wa = __byte_perm(vw[0][j / 4], vw[1][j / 4], sel);
          const uint32_t wb = __byte_perm(vw[2][j / 4], vw[3][j / 4], sel);
          const uint32_t sa = vs[0][j], sb = vs[1][j];
          const uint32_t za = bf16x2_mul(sa, kMinus136), zb = bf16x2_mul(sb, kMinus136);
          const bool odd = j & 1;
          const uint32_t af[4] = {bf16x2_fma(odd ? bits.pair<2>(wa) : bits.pair<0>(wa), sa, za),
                                  bf16x2_fma(odd ? bits.pair<3>(wa) : bits.pair<1>(wa), sa, za),
                                  bf16x2_fma(odd ? bits.pair<2>(wb) : bits.pair<0>(wb), sb, zb),
                                  bf16x2_fma(odd ? bits.pair<3>(wb) : bits.pair<1>(wb), sb, zb)};
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            if constexpr (TERMS == 1) {
              mma16816(o[j][n], af, pf[h][0][n][0], pf[h][0][n][1]);
            } else {
              float d[4] = {0.f, 0.f, 0.f, 0.f};  // of this page
#pragma unroll
              for (int k = TERMS - 1; k >= 0; --k) mma16816(d, af, pf[h][k][n][0], pf[h][k][n][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[j][n][e] += d[e];
            }
          }
        }
      }
      __syncwarp();  // the stage and the tables are read
      ++used;
      recs = recs + S::STAGE == my_ring + S::RING / kSmallWarps ? my_ring : recs + S::STAGE;
    }
    // ---- the segment's end
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], w);
    const Segment at = cs;
    const bool ends = !walk.next(cs, u1);
    if (at.from_start && at.to_end) {
      // a whole range: its rows, through the tables' shared memory (vectors' entries side by side)
      float* buf = reinterpret_cast<float*>(my_tab);
      constexpr int COLS = 8;  // entries of all the vectors at a time
      static_assert(S::ROWS * COLS * 4 <= S::TAB, "");
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float inv = normaliser(l[n][c], lim[n][c] >= 0);
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            o[j][n][c] *= inv;
            o[j][n][c + 2] *= inv;
          }
        }
#pragma unroll
      for (int j8 = 0; j8 < 2 * NB; ++j8) {
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) buf[(n * 8 + 2 * t + c) * COLS + gr] = o[j8 / 2][n][c + 2 * (j8 & 1)];
        __syncwarp();
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const int v = n * 8 + gr;
          if (v < tr.M) {
            const float2 x = *reinterpret_cast<const float2*>(buf + v * COLS + 2 * t);
            const int m = tr.m0 + v;
            T* out = static_cast<T*>(a.out) + row_of(m, at.g, a.out_stride) + 8 * j8 + 2 * t;
            if constexpr (TERMS == 1) *reinterpret_cast<uint32_t*>(out) = pack_bf16(x.x, x.y);
            else *reinterpret_cast<float2*>(out) = x;
          }
        }
      }
      __syncwarp();
    } else {
      // part of a range: kept for the join
      float* dst = ends ? reinterpret_cast<float*>(my_ring) : spill + (size_t)warp * S::PIECE;
      if (ends) copy_wait<0>();
      __syncwarp();
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int v = n * 8 + 2 * t + c;
          if (gr == 0) {
            dst[S::ROWS * S::OROW + v] = -nm[n][c];
            dst[S::ROWS * (S::OROW + 1) + v] = l[n][c];
          }
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            dst[v * S::OROW + 16 * j + gr] = o[j][n][c];
            dst[v * S::OROW + 16 * j + 8 + gr] = o[j][n][c + 2];
          }
        }
      if (lane == 0) {
        Parts& p = parts[warp];
        const int second = at.from_start ? 1 : 0;
        p.state |= second ? kSecond : kFirst | (at.to_end ? kFirstEnds : 0) | (ends ? 0 : kFirstSpilled);
        p.k[second] = at.k;
        p.g[second] = at.g;
      }
    }
    if (ends) break;
  }
  // ---- ranges shared by warps: each is a run of parts, one per warp, the first of which may have
  // begun before this CTA and the last of which may go on behind it
  __syncthreads();
  uint32_t firsts = 0, lasts = 0, spilled = 0, seconds = 0;  // bit w: warp w
#pragma unroll
  for (int w = 0; w < kSmallWarps; ++w) {
    const int st = parts[w].state;
    firsts |= (st & kFirst) ? 1u << w : 0;
    lasts |= (st & kFirstEnds) ? 1u << w : 0;
    spilled |= (st & kFirstSpilled) ? 1u << w : 0;
    seconds |= (st & kSecond) ? 1u << w : 0;
  }
  // the first run may be a range that began before the CTA: it has first parts alone
  bool begins = firsts == 0 || (seconds != 0 && __ffs(seconds) < __ffs(firsts));
  uint32_t heads = seconds;
#pragma unroll 1
  while (!begins || heads != 0) {
    const int w0 = (begins ? __ffs(heads) : __ffs(firsts)) - 1;
    const uint32_t later = ~0u << (begins ? w0 + 1 : w0);  // warps whose first parts can be of this run
    const bool closed = (lasts & later) != 0;
    const int w1 = closed ? __ffs(lasts & later) - 1 : kSmallWarps - 1;
    const uint32_t in = firsts & later & ((2u << w1) - 1);
    const bool done = begins && closed;
    const TileRows tr = lo.tile(ln, parts[w0].k[begins ? 1 : 0]);
    const int g = parts[w0].g[begins ? 1 : 0];
    float* rec = done ? nullptr : part_record<HD>(ln, blockIdx.x, begins);
#pragma unroll 1
    for (int x4 = tid; x4 < tr.M * (HD / 4); x4 += kSmallWarps * 32) {
      const int v = x4 / (HD / 4), e = (x4 - v * (HD / 4)) * 4;
      // at most one part per warp, all of them loaded at once
      float m[kSmallWarps], l[kSmallWarps];
      float4 y[kSmallWarps];
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) {
        const bool second = begins && w == w0, has = second || (in >> w & 1);
        const float* d = !second && (spilled >> w & 1) ? spill + (size_t)w * S::PIECE
                                                       : reinterpret_cast<const float*>(sm + w * S::STAGES * S::STAGE);
        m[w] = has ? d[S::ROWS * S::OROW + v] : -INFINITY;
        l[w] = has ? d[S::ROWS * (S::OROW + 1) + v] : 0.f;
        y[w] = has ? *reinterpret_cast<const float4*>(d + v * S::OROW + e) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mx = -INFINITY, sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) mx = fmaxf(mx, m[w]);
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int w = 0; w < kSmallWarps; ++w) {
        const float f = ex2_approx(m[w] - ref);
        sum = fmaf(f, l[w], sum);
        x[0] = fmaf(f, y[w].x, x[0]); x[1] = fmaf(f, y[w].y, x[1]);
        x[2] = fmaf(f, y[w].z, x[2]); x[3] = fmaf(f, y[w].w, x[3]);
      }
      if (done) {
        const int mv = tr.m0 + v, r = (int)((uint32_t)mv / ln.group);
        const float inv = normaliser(sum, !(sum > 0.f) && row_sees(a, tr.r0 + r));
        T* out = static_cast<T*>(a.out) + (tr.r0 + r) * a.out_stride + (g * G + mv - r * G) * HD + e;
        if constexpr (TERMS == 1)
          *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv));
        else
          *reinterpret_cast<float4*>(out) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      } else {
        if (e == 0) {
          rec[v] = mx;
          rec[S::ROWS + v] = sum;
        }
        *reinterpret_cast<float4*>(rec + 2 * S::ROWS + v * HD + e) = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
    if (begins) heads &= heads - 1;
    begins = true;
  }
}

// ----------------------------------------------------------------------------- many query vectors: tcgen05
//
// A tile of up to 128 query vectors (bf16) against blocks of 64 positions: S = Q K^T and O += P V on
// the 5th-generation tensor core, S and O in tensor memory, P written over S as bf16.  One unpacked
// block serves all 128 vectors.  Roles of a CTA (two CTAs per SM where their lines fit, see tile_ctas):
//   one warp     issues the MMAs: a block's PV once P is there, then the S that reuses its buffer, two
//                or three blocks on.
//   three warps  unpack: each takes two pages of a block in turn, a row (position) per lane, from a ring
//                of its own that asynchronous copies fill ahead, into the K and V rings (128-byte
//                swizzle).  Entries stay in the order of the cache's words: K's is a permutation of the
//                contraction, given to Q as well; V's one of O's columns, undone on output.
//   four warps   do the softmax, one thread per query vector (TMEM lane).
// A vector's reference maximum only moves when a block exceeds it by 2^8; then O is rescaled in TMEM.
//
// Bound: the roles' work and its handover.  B = 64 draft blocks (7 to 14 rows of 64 query heads, 8 kv heads of 64,
// up to 16384 positions: 45,000 blocks, 217 MB) take 134 us, and 141 with equal pieces for an SM's CTAs: then 885 cycles
// of an SM per block, in which it issues 1770 warp instructions (442 cycles of its four schedulers) and computes 270
// cycles of products; HBM is a fifth busy, the exponent unit 23 %.  In a CTA a block takes the softmax warps 1000
// cycles and the unpacking warps 970 of the 1770 that it lasts; the rest they wait for each other's buffers.  Without
// the softmax call and merge take 126 us of 151, without the unpacking 125, without both 102, with no copies and
// products either 86: no one part bounds it.  Registers end it (eight warps of 128 in two CTAs are all there are):
// more unpacking warps spill.  Copies of whole pages by the SM's copy engine in place of the lanes' (fewer
// instructions) took 159 us of 151.
// head_dim 128, two chunks of 500 to 691 prompt rows: 85 us, 605 TFLOP/s, bound by the same; every tile unpacks its
// pages for itself.

constexpr int kTileRows = 128;
constexpr int kTileRangeCost = 6;  // a range's start (queries, filling the pipeline, output), in blocks
constexpr int kTileBlk = 64;
constexpr uint32_t kTileTmemCols = 256;  // S buffers, then O

template <int HD>
struct Tile {
  static constexpr bool JOINT = HD == 64;             // a block's keys and values are handed over together
  static constexpr int NB = HD == 64 ? 3 : 2;         // S buffers; O takes the rest of the tensor memory
  static constexpr int UNPACK = 3;                    // unpacking warps
  static constexpr int THREADS = 32 * (1 + UNPACK) + kTileRows;  // warp 0: MMA; 1..3: unpack; 4..7: softmax
  static constexpr int ST = HD == 64 ? 4 : 2;         // stages of keys and values
  static constexpr int RAW = HD == 64 ? 3 : 1;        // steps that an unpacking warp's copies are ahead
  static constexpr int STEP = 2 * PackedLayout<HD>::kRecord;  // two pages, half a block
  static constexpr uint32_t TO = NB * kTileBlk;       // first column of O
  static constexpr uint32_t Q = kTileRows * HD * 2, KV = kTileBlk * HD * 2;
  static constexpr uint32_t KRING = Q, VRING = KRING + ST * KV, RAWS = VRING + ST * KV;
  static constexpr uint32_t CTRL = (RAWS + UNPACK * RAW * STEP + 127) / 128 * 128;
  static constexpr uint32_t FIXED = CTRL + 256;
  static size_t smem(int n_tiles) { return 1024 + FIXED + Layout::kBytesPerTile * (size_t)n_tiles + 4; }
};

struct TileCtrl {
  uint64_t kfull[4], vfull[2];     // an arrival per step of the unpacking warps
  uint64_t vempty[4];              // the block's PV product has completed
  uint64_t s_full[3], p_full[3];   // S of a block is in its buffer (and its keys are read); P is (O rescaled where needed)
  uint64_t q_full;                 // the item's query tile is staged
  uint64_t pv_item, o_free;        // the item's last PV has completed; its O has been read
  uint64_t drain;
  int scratch[16];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(TileCtrl) <= 256, "");

// 16-byte unit c of row r of a shared-memory tile [HD/64][ROWS][64 bf16], 128-byte swizzle.
template <int ROWS>
PE_DEV uint32_t unit_addr(uint32_t base, int row, int c) {
  return base + (uint32_t)((c >> 3) * ROWS * 128 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}
PE_DEV void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// 8 bytes, or zeros where `bytes` is 0.
PE_DEV void copy8(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Two fp32 values in one 64-bit register, for the packed fp32 instructions.
struct F2 {
  uint64_t v;
  PE_DEV F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  PE_DEV explicit F2(uint64_t x) : v(x) {}
  PE_DEV float lo() const {
    float x;
    asm("mov.b64 {%0, _}, %1;" : "=f"(x) : "l"(v));
    return x;
  }
  PE_DEV float hi() const {
    float x;
    asm("mov.b64 {_, %0}, %1;" : "=f"(x) : "l"(v));
    return x;
  }
  static PE_DEV F2 fma(F2 a, F2 b, F2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a.v), "l"(b.v), "l"(c.v));
    return F2(d);
  }
  static PE_DEV F2 add(F2 a, F2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
    return F2(d);
  }
};

// 32 consecutive fp32 columns of this thread's TMEM lane, waited on.
PE_DEV void tmem_load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <int HD>
__global__ void __launch_bounds__(Tile<HD>::THREADS, 2) attend_tile_kernel(const PackedAttnArgs a, const Line ln) {
  using C = Tile<HD>;
  using L = PackedLayout<HD>;
  constexpr int H = HD / 64, CH = HD / 8, ST = C::ST;
  constexpr int NB = C::NB;
  extern __shared__ uint8_t sm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sQ = smem_u32(sm);
  TileCtrl* ctl = reinterpret_cast<TileCtrl*>(sm + C::CTRL);
  const Layout lo(sm + C::FIXED, ln.n_tiles);
  volatile int* abort_flag = &ctl->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_wait();
  lay_out(a, ln, lo, ctl->scratch);
  const Walk walk{ln, lo, a.n_kv};
  const uint32_t total = (uint32_t)lo.prefix[ln.n_tiles] * a.n_kv;
  if (blockIdx.x == 0 && !ln.whole)
    for (int k = tid; k <= ln.n_tiles; k += blockDim.x) ln.prefix[k] = lo.prefix[k];
  uint32_t u0, u1;
  cta_piece(ln, walk, total, u0, u1);
  if (u0 == u1) return;  // the whole CTA, before it holds anything
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(smem_u32(&ctl->kfull[s]), 2);
      if (!C::JOINT) mbar_init(smem_u32(&ctl->vfull[s]), 2);
      mbar_init(smem_u32(&ctl->vempty[s]), 1);
    }
    for (int b = 0; b < NB; ++b) {
      mbar_init(smem_u32(&ctl->s_full[b]), 1);
      mbar_init(smem_u32(&ctl->p_full[b]), 4);
    }
    mbar_init(smem_u32(&ctl->q_full), 4);
    mbar_init(smem_u32(&ctl->pv_item), 1);
    mbar_init(smem_u32(&ctl->o_free), 4);
    mbar_init(smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&ctl->tmem), kTileTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // The next kernel may be a GEMM, which allocates tensor memory and then waits for this one: it may start once every
  // CTA here has its own (or, above, has ended).
  pdl_trigger();
  auto blocks_of = [](const Segment& s) { return s.page1 > s.page0 ? (s.page1 - s.page0 + 3) >> 2 : 0; };
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    return warp_ok(mbar_wait(smem_u32(bar), phase & 1u, a.err, abort_flag, a.wait_ns));
  };
  auto arrive = [&](uint64_t* bar) {  // one arrival per warp
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
  };
  // Blocks are counted through the CTA's segments: block x uses stage x % ST and S buffer x % NB.
  Segment seg;
  const bool some = walk.first(seg, u0, u1);

  if (!some) {  // nothing starts here
  } else if (warp == 0) {
    // ------------------------------------------------------------------ MMA issuer (a converged warp)
    constexpr uint32_t kIdS = idesc_bf16(kTileRows, kTileBlk);               // N = positions
    constexpr uint32_t kIdO = idesc_bf16(kTileRows, HD) | kIdescTransposeB;  // V is MN-major
    const uint64_t dk = sdesc_k_sw128(sQ + C::KRING), dv = sdesc_mn_sw128(sQ + C::VRING, kTileBlk * 128);
    const uint64_t dq = sdesc_k_sw128(sQ);
    // The products run in the order of their issue: an S after the PV whose P it overwrites.
    auto issue_s = [&](int x) -> bool {
      const int s = x % ST;
      if (!wait(&ctl->kfull[s], (uint32_t)(x / ST))) return false;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t bk = dk + (uint64_t)((uint32_t)s * (C::KV >> 4));
        const uint32_t d = tmem + (uint32_t)((x % NB) * kTileBlk);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(d, dq + ((kk >> 2) * (kTileRows * 128 >> 4) + 2 * (kk & 3)),
                      bk + ((kk >> 2) * (kTileBlk * 128 >> 4) + 2 * (kk & 3)), kIdS, kk > 0 ? 1u : 0u);
        tc_commit(smem_u32(&ctl->s_full[x % NB]));
      }
      __syncwarp();
      return true;
    };
    int gi = 0, ii = 0;
    bool stop = false;
    do {
      const int nblk = blocks_of(seg);
      if (nblk == 0) continue;
      stop = !wait(&ctl->q_full, (uint32_t)ii);
      for (int j = 0; j < NB && j < nblk && !stop; ++j) stop = !issue_s(gi + j);
#pragma unroll 1
      for (int j = 0; j < nblk && !stop; ++j) {
        const int x = gi + j, s = x % ST, b = x % NB;
        // the item's first products overwrite O: the last item's has to have been read
        if ((!C::JOINT && !wait(&ctl->vfull[s], (uint32_t)(x / ST))) || !wait(&ctl->p_full[b], (uint32_t)(x / NB)) ||
            (j == 0 && ii > 0 && !wait(&ctl->o_free, (uint32_t)(ii - 1)))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t bv = dv + (uint64_t)((uint32_t)s * (C::KV >> 4));
          const uint32_t pa = tmem + (uint32_t)(b * kTileBlk);
#pragma unroll
          for (int kk = 0; kk < kTileBlk / 16; ++kk)
            tc_mma_bf16_tmem_a(tmem + C::TO, pa + 8u * kk, bv + kk * (2048 >> 4), kIdO, (j > 0 || kk > 0) ? 1u : 0u);
          if (j == nblk - 1) tc_commit(smem_u32(&ctl->pv_item));
          tc_commit(smem_u32(&ctl->vempty[s]));
        }
        __syncwarp();
        if (j + NB < nblk) stop = !issue_s(x + NB);
      }
      gi += nblk;
      ++ii;
    } while (!stop && walk.next(seg, u1));
    // TMEM is freed only after every MMA issued here has completed
    if (elect_one()) tc_commit(smem_u32(&ctl->drain));
    __syncwarp();
    mbar_wait(smem_u32(&ctl->drain), 0, a.err, nullptr, a.wait_ns);
  } else if (warp < 4) {
    // ------------------------------------------------------------------ unpack
    const PairBits bits;
    // Steps of two pages are counted through the CTA's blocks; step q belongs to warp q % UNPACK.  A row (position)
    // per lane.
    constexpr int PP = 2, PER = 2;  // pages of a step, steps of a block
    const int uw = warp - 1, row = lane;
    const uint32_t row_x = (uint32_t)(row & 7) << 4;
    const uint32_t step = (uint32_t)a.n_kv * L::kRecord;
    const uint32_t raw0 = sQ + C::RAWS + (uint32_t)uw * (C::RAW * C::STEP);
    int page = uw * PP, ids = -1, n_ids = 0;  // page: of the segment's blocks (the last may lack some)
    uint32_t raw_in = raw0 + lane * 16;
    bool more = true;
    // copies the pages of the warp's next step, over the segments; a group of copies each time, empty behind the last
    auto fetch = [&]() {
      if (more) {
        for (int n; page >= (n = 4 * blocks_of(seg));) {
          if (!walk.next(seg, u1)) {
            more = false;
            break;
          }
          page -= n;
          n_ids = 0;
        }
      }
      if (more) {
        if (n_ids == 0) {  // the ids of this warp's next 32 pages, one per lane
          const int x = seg.page0 + page + (lane / PP) * (C::UNPACK * PP) + lane % PP;
          ids = -1;
          if (x < seg.page1) {
            ids = __ldcg(a.block_table + (size_t)((uint32_t)(ln.tile0 + seg.k) / ln.tps) * a.max_pages + x);
            if (ids < 0 || ids >= a.num_pages) {
              set_err(a.err, PE_DEV_BAD_PAGE);
              ids = -1;
            }
          }
        }
        const uint8_t* head = a.pool + (size_t)seg.g * L::kRecord + lane * 16;
        const int id0 = __shfl_sync(0xFFFFFFFFu, ids, n_ids), id1 = __shfl_sync(0xFFFFFFFFu, ids, n_ids + 1);
        n_ids = (n_ids + PP) & 31;
        page += C::UNPACK * PP;
        const uint8_t* src0 = head + (uint64_t)(uint32_t)id0 * step;
        const uint8_t* src1 = head + (uint64_t)(uint32_t)id1 * step - L::kRecord;
        if ((id0 | id1) >= 0) {
#pragma unroll
          for (int i = 0; i < (C::STEP + 511) / 512; ++i) {
            const int at = i * 512 + lane * 16;  // byte of the records
            const bool first = i * 512 + 511 < L::kRecord || (i * 512 < L::kRecord && at < L::kRecord);
            if (i * 512 + 511 < C::STEP || at < C::STEP) copy16(raw_in + i * 512, (first ? src0 : src1) + i * 512);
          }
        } else {
          // a page behind the range or outside the pool stands for zeros, every nibble 8
#pragma unroll 1
          for (int i = 0; i + lane * 16 < C::STEP; i += 512) {
            const bool first = i + lane * 16 < L::kRecord;
            if ((first ? id0 : id1) >= 0) copy16(raw_in + i, (first ? src0 : src1) + i);
            else st_shared16(raw_in + i, 0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
          }
        }
        raw_in = raw_in + C::STEP == raw0 + lane * 16 + C::RAW * C::STEP ? raw0 + lane * 16 : raw_in + C::STEP;
      }
      copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < C::RAW; ++i) fetch();
    // how many steps there are: a second walk
    Segment cs;
    int steps = 0;
    if (walk.first(cs, u0, u1))
      do steps += PER * blocks_of(cs);
      while (walk.next(cs, u1));
    const uint8_t* raw = sm + C::RAWS + (size_t)uw * (C::RAW * C::STEP);
    int slot = 0;
#pragma unroll 1
    for (int q = uw; q < steps; q += C::UNPACK) {
      const int gi = q / PER, s = gi % ST;
      const uint32_t at = (uint32_t)(((q % PER) * PP * 16 + row) * 128);
      copy_wait<C::RAW - 1>();
      __syncwarp();
      uint4 k[2 * H], v[2 * H];
      uint32_t ks[H], vs[H];
      {
        const uint8_t* rec = raw + slot * C::STEP + (row >> 4) * L::kRecord;
        const int r16 = row & 15;
#pragma unroll
        for (int c = 0; c < 2 * H; ++c) {
          k[c] = *reinterpret_cast<const uint4*>(rec + L::kK + r16 * L::kRow + c * 16);
          v[c] = *reinterpret_cast<const uint4*>(rec + L::kV + r16 * L::kRow + c * 16);
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
          ks[h] = reinterpret_cast<const uint32_t*>(rec + L::kKs + r16 * L::kScaleRow)[h];
          vs[h] = reinterpret_cast<const uint32_t*>(rec + L::kVs + r16 * L::kScaleRow)[h];
        }
      }
      slot = slot + 1 == C::RAW ? 0 : slot + 1;
      __syncwarp();  // the pages are in registers
      fetch();
      // head_dim 64: the stage is free once its last PV has completed; 128: its keys once S has
      if (gi >= ST && !wait(C::JOINT ? &ctl->vempty[s] : &ctl->s_full[s], (uint32_t)(gi / ST) - 1u)) break;
      {
        const uint32_t base = sQ + C::KRING + (uint32_t)s * C::KV + at;
        // word w = t * HD/32 + u of the row: entries 4t..4t+3 of blocks 2u and 2u + 1, unit w of the tile's row
        uint32_t sp[4 * H], zp[4 * H];
#pragma unroll
        for (int i = 0; i < 4 * H; ++i) {
          sp[i] = packed_scale_lo(__byte_perm(ks[i / 4], 0, 0x4040 + 0x0101 * (i & 3)));
          zp[i] = bf16x2_mul(sp[i], kMinus136);
        }
#pragma unroll
        for (int c = 0; c < 2 * H; ++c) {
          const uint32_t w4[4] = {k[c].x, k[c].y, k[c].z, k[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = 4 * c + i, u = w % (HD / 32);
            st_shared16(base + (uint32_t)((w >> 3) * kTileBlk * 128) + (((uint32_t)(w & 7) << 4) ^ row_x),
                        bf16x2_fma(bits.pair<0>(w4[i]), sp[2 * u], zp[2 * u]),
                        bf16x2_fma(bits.pair<1>(w4[i]), sp[2 * u], zp[2 * u]),
                        bf16x2_fma(bits.pair<2>(w4[i]), sp[2 * u + 1], zp[2 * u + 1]),
                        bf16x2_fma(bits.pair<3>(w4[i]), sp[2 * u + 1], zp[2 * u + 1]));
          }
        }
      }
      if constexpr (!C::JOINT) {
        fence_proxy_async_smem();
        arrive(&ctl->kfull[s]);
        if (gi >= ST && !wait(&ctl->vempty[s], (uint32_t)(gi / ST) - 1u)) break;
      }
      {
        const uint32_t base = sQ + C::VRING + (uint32_t)s * C::KV + at;
        // word g * H + h: entries g and g + 8 of four blocks, pairs 32 entries apart; unit g of the h-th 64 columns
        uint32_t sp[H][2], zp[H][2];
#pragma unroll
        for (int h = 0; h < H; ++h) {
          sp[h][0] = packed_scale_lo(vs[h]);
          sp[h][1] = packed_scale_hi(vs[h]);
          zp[h][0] = bf16x2_mul(sp[h][0], kMinus136);
          zp[h][1] = bf16x2_mul(sp[h][1], kMinus136);
        }
#pragma unroll
        for (int c = 0; c < 2 * H; ++c) {
          const uint32_t w4[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int w = 4 * c + i, h = w % H;
            st_shared16(base + (uint32_t)(h * kTileBlk * 128) + (((uint32_t)(w / H) << 4) ^ row_x),
                        bf16x2_fma(bits.pair<0>(w4[i]), sp[h][0], zp[h][0]),
                        bf16x2_fma(bits.pair<1>(w4[i]), sp[h][0], zp[h][0]),
                        bf16x2_fma(bits.pair<2>(w4[i]), sp[h][1], zp[h][1]),
                        bf16x2_fma(bits.pair<3>(w4[i]), sp[h][1], zp[h][1]));
          }
        }
      }
      fence_proxy_async_smem();
      arrive(C::JOINT ? &ctl->kfull[s] : &ctl->vfull[s]);
    }
    copy_wait<0>();  // leave no copy in flight into this CTA's shared memory
  } else {
    // ------------------------------------------------------------------ softmax and output
    const int et = tid - 128;
    const int r = (warp & 3) * 32 + lane;  // query vector of the tile = TMEM lane
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sl2 = a.scale * 1.4426950408889634f * kPackedUnit;
    const __nv_bfloat16* qbuf = static_cast<const __nv_bfloat16*>(a.q);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
    auto row_of = [&](const TileRows& t, int v, int g, long long stride) {
      const int m = t.m0 + v, rr = (int)((uint32_t)m / ln.group);
      return (t.r0 + rr) * stride + (g * ln.G + m - rr * ln.G) * HD;
    };
    // the query tile, entries in the order of the key words: unit w = t * HD/32 + u holds entries 4t..4t+3 of
    // blocks 2u and 2u + 1; zeros behind the tile's vectors
    auto stage_q = [&](const Segment& sg) {
      const TileRows t = lo.tile(ln, sg.k);
#pragma unroll 1
      for (int idx = et; idx < kTileRows * CH; idx += kTileRows) {
        const int m = idx / CH, w = idx % CH;
        const __nv_bfloat16* src =
            qbuf + row_of(t, m < t.M ? m : 0, sg.g, a.q_stride) + 32 * (w % (HD / 32)) + 4 * (w / (HD / 32));
        const uint32_t dst = unit_addr<kTileRows>(sQ, m, w), bytes = m < t.M ? 8u : 0u;
        copy8(dst, src, bytes);
        copy8(dst + 8, src + 16, bytes);
      }
      copy_commit();
    };
    auto q_staged = [&] {
      copy_wait<0>();
      fence_proxy_async_smem();
      arrive(&ctl->q_full);
    };
    // the next segment with positions to see; rows of those without get zeros
    auto advance = [&](Segment& sg) -> bool {
      for (;;) {
        if (blocks_of(sg) > 0) return true;
        const TileRows t = lo.tile(ln, sg.k);
        if (r < t.M) {
          __nv_bfloat16* dst = out + row_of(t, r, sg.g, a.out_stride);
#pragma unroll
          for (int c = 0; c < CH; ++c) reinterpret_cast<uint4*>(dst)[c] = make_uint4(0, 0, 0, 0);
        }
        if (!walk.next(sg, u1)) return false;
      }
    };
    int gi = 0, ii = 0;
    bool more = advance(seg);
    if (more) stage_q(seg);
    while (more) {
      q_staged();
      const Segment cur = seg;
      more = walk.next(seg, u1) && advance(seg);
      const TileRows tr = lo.tile(ln, cur.k);
      const int nblk = blocks_of(cur);
      const bool valid = r < tr.M;
      // the vector's last visible position within the segment
      bool bad = false;  // reported by lay_out
      int lim = -1;
      if (valid) {
        const int pos = __ldcg(a.positions + tr.r0 + (int)((uint32_t)(tr.m0 + r) / ln.group));
        lim = min(row_limit(a, pos, bad), cur.page1 * kPackedPage - 1);
      }
      const bool warp_any = __any_sync(0xFFFFFFFFu, valid);
      int wmin = valid ? lim : INT_MAX;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wmin = min(wmin, __shfl_xor_sync(0xFFFFFFFFu, wmin, o));
      float m_ref = -INFINITY, l = 0.f;  // reference maximum (log2 units) and sum
      const uint32_t o_at = lanes + C::TO;
      bool stop = false;
#pragma unroll 1
      for (int j = 0; j < nblk; ++j) {
        const int x = gi + j, b = x % NB;
        if (!wait(&ctl->s_full[b], (uint32_t)(x / NB))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (warp_any) {
          const uint32_t sbuf = lanes + (uint32_t)(b * kTileBlk);
          const int kb0 = cur.page0 * kPackedPage + j * kTileBlk;
          float sc[kTileBlk], mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          tmem_load64(sbuf, sc);
          if (kb0 + kTileBlk - 1 > wmin) {  // some position is masked for some vector of the warp
#pragma unroll
            for (int c = 0; c < kTileBlk; ++c) sc[c] = (kb0 + c <= lim) ? sc[c] : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < kTileBlk; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx4[e] = max3(mx4[e], sc[c + e], sc[c + 4 + e]);
          const float bm = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          const bool fresh = m_ref == -INFINITY;
          const bool need = !fresh && bm > m_ref + kRescaleLog2;
          if (__any_sync(0xFFFFFFFFu, need)) {
            // O holds the PV products of the blocks before.  The PV of block x - 1 tells by its stage (at most one
            // phase short: S(x) was issued behind the PV of block x - NB, and there are as many stages).
            if (!wait(&ctl->vempty[(x - 1) % ST], (uint32_t)((x - 1) / ST))) {
              stop = true;
            } else {
              tc_fence_after();
              const float f = need ? ex2_approx(m_ref - bm) : 1.f;
#pragma unroll 1
              for (int c = 0; c < HD; c += 16) {
                float ov[16];
                tmem_load16(o_at + (uint32_t)c, ov);
#pragma unroll
                for (int e = 0; e < 16; ++e) ov[e] *= f;
                tmem_store16(o_at + (uint32_t)c, ov);
              }
              if (need) {
                l *= f;
                m_ref = bm;
              }
            }
          }
          if (fresh) m_ref = bm;
          // masked scores are -inf; a vector with nothing unmasked yet takes offset -inf, so P = 0 there too
          const float nmr = m_ref == -INFINITY ? -INFINITY : -m_ref;
          const F2 scale2(sl2, sl2), off2(nmr, nmr);
          F2 sum2[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
          uint32_t pk[kTileBlk / 2];
#pragma unroll
          for (int c = 0; c < kTileBlk / 2; ++c) {
            const F2 d = F2::fma(F2(sc[2 * c], sc[2 * c + 1]), scale2, off2);
            const float p0 = ex2_approx(d.lo()), p1 = ex2_approx(d.hi());
            sum2[c & 1] = F2::add(sum2[c & 1], F2(p0, p1));
            pk[c] = pack_bf16(p0, p1);
          }
          tmem_store32(sbuf, pk);  // over the first half of S's columns
          const F2 s2 = F2::add(sum2[0], sum2[1]);
          l += s2.lo() + s2.hi();
        }
        tc_fence_before();
        arrive(&ctl->p_full[b]);
        if (stop) break;
      }
      if (stop) break;
      gi += nblk;
      if (!wait(&ctl->pv_item, (uint32_t)ii)) break;
      tc_fence_after();
      if (more) stage_q(seg);  // every product of this item has completed
      const bool whole = cur.from_start && cur.to_end;
      if (warp_any) {
        const float inv = whole ? normaliser(l, lim >= 0) : 1.f;
        float* rec = whole ? nullptr : part_record<HD>(ln, blockIdx.x, cur.from_start);
        if (valid && !whole) {
          rec[r] = m_ref;
          rec[kTileRows + r] = l;
        }
        // column 8g + 2i + e of 64 holds entry 16 (i/2) + g + 8 (i%2) + 32 e: four entries (g or g + 4 on) at a time
        __nv_bfloat16* dst = out + row_of(tr, r, cur.g, a.out_stride);
        float* rdst = rec + 2 * kTileRows + r * HD;
#pragma unroll 1
        for (int h = 0; h < 2 * H; ++h) {
          float ov[32];
          tmem_load32(o_at + 32u * h, ov);
#pragma unroll
          for (int c = 0; c < 32; ++c) ov[c] *= inv;
          if (valid) {
            const int at = 64 * (h >> 1) + 4 * (h & 1);
#pragma unroll
            for (int c = 0; c < 8; ++c) {  // i = c % 4, e = c / 4
              const int col = 2 * (c & 3) + (c >> 2), e = at + 16 * ((c >> 1) & 1) + 8 * (c & 1) + 32 * (c >> 2);
              if (whole)
                *reinterpret_cast<uint2*>(dst + e) =
                    make_uint2(pack_bf16(ov[col], ov[8 + col]), pack_bf16(ov[16 + col], ov[24 + col]));
              else
                *reinterpret_cast<float4*>(rdst + e) = make_float4(ov[col], ov[8 + col], ov[16 + col], ov[24 + col]);
            }
          }
        }
      }
      tc_fence_before();
      arrive(&ctl->o_free);
      ++ii;
    }
    copy_wait<0>();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTileTmemCols);
  }
}

// ----------------------------------------------------------------------------- merge of cut ranges

constexpr int kMergeThreads = 256;

// A CTA per (tile, head), or one of `shares` (grid's y) that take its vectors in turn: it finds the CTAs that
// hold parts of the range, then its warps take the vectors, 16 bytes of a vector a lane and U vectors a lane at a
// time; `split` warps (a power of two, at most 8) share the records of the same vectors and join in shared
// memory.  Sums run in CTA order within a warp, then in warp order.  It is bound by the time of its loads
// (each range has few records), so what counts is how many a warp has under way.
template <typename T, int HD, int U>
__global__ void __launch_bounds__(kMergeThreads) attend_merge_kernel(const PackedAttnArgs a, const Line ln, int grid,
                                                                     int split) {
  constexpr int CB = 4 / U, LPV = HD / 4, VW = 32 / LPV;  // records at a time; lanes per vector, vectors per warp
  __shared__ float sh_m[8][U][VW], sh_l[8][U][VW];
  __shared__ float4 sh_o[8][U][32];
  pdl_wait();
  pdl_trigger();
  const int k = (int)(blockIdx.x / ln.heads), g = (int)blockIdx.x - k * a.n_kv;
  const int p0 = __ldcg(ln.prefix + k), p1 = __ldcg(ln.prefix + k + 1);
  const uint32_t tot = (uint32_t)__ldcg(ln.prefix + ln.n_tiles) * a.n_kv;
  bool bad = false;  // reported by the kernel before
  const TileRows tr = tile_rows(a, ln, ln.tile0 + k, bad);
  if (p1 == p0) return;
  const Cuts cuts(ln, grid, tot);
  const uint32_t len = p1 - p0, start = (uint32_t)p0 * a.n_kv + (uint32_t)g * len;
  // the pieces in which its first and its last unit start
  const int c0 = (int)cuts.piece(start + ln.range_cost), c1 = (int)cuts.piece(start + len - 1);
  if (c0 == c1) return;  // finished by its CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp & (split - 1), teams = 8 / split;
  const int vl = lane / LPV, el = lane % LPV * 4;  // the lane's vector of the warp's, its first entry
  const int per = teams * U * VW;                  // vectors at a time
  for (int v0 = blockIdx.y * per; v0 < tr.M; v0 += gridDim.y * per) {  // the same trip count for every warp
    const int va = v0 + warp / split * U * VW + vl;  // vector u of the lane: va + u * VW
    float mx[U], sum[U];
    float4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mx[u] = -INFINITY;
      sum[u] = 0.f;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c = c0 + sub; c <= c1; c += CB * split) {
      float m[U][CB], l[U][CB];
      float4 y[U][CB];
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        const int cc = c + i * split;
        const float* rec = part_record<HD>(ln, min(cc, c1), cc == c0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int v = va + u * VW;
          m[u][i] = -INFINITY;
          l[u][i] = 0.f;
          y[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (cc <= c1 && v < tr.M) {
            m[u][i] = __ldcg(rec + v);
            l[u][i] = __ldcg(rec + ln.tile_rows + v);
            y[u][i] = __ldcg(reinterpret_cast<const float4*>(rec + 2 * ln.tile_rows + (size_t)v * HD + el));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float nx = mx[u];
#pragma unroll
        for (int i = 0; i < CB; ++i) nx = fmaxf(nx, m[u][i]);
        if (nx == -INFINITY) {  // sums of 0, or NaN
#pragma unroll
          for (int i = 0; i < CB; ++i) sum[u] += l[u][i];
          continue;
        }
        const float f = ex2_approx(mx[u] - nx);
        sum[u] *= f;
        x[u].x *= f; x[u].y *= f; x[u].z *= f; x[u].w *= f;
#pragma unroll
        for (int i = 0; i < CB; ++i) {
          const float w = ex2_approx(m[u][i] - nx);
          sum[u] = fmaf(w, l[u][i], sum[u]);
          x[u].x = fmaf(w, y[u][i].x, x[u].x); x[u].y = fmaf(w, y[u][i].y, x[u].y);
          x[u].z = fmaf(w, y[u][i].z, x[u].z); x[u].w = fmaf(w, y[u][i].w, x[u].w);
        }
        mx[u] = nx;
      }
    }
    if (split > 1) {
      __syncthreads();  // the last vectors' values have been read
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (el == 0) {
          sh_m[warp][u][vl] = mx[u];
          sh_l[warp][u][vl] = sum[u];
        }
        sh_o[warp][u][lane] = x[u];
      }
      __syncthreads();
      if (sub == 0)
        for (int w = warp + 1; w < warp + split; ++w)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const float m = sh_m[w][u][vl], nx = fmaxf(mx[u], m);
            if (nx == -INFINITY) {
              sum[u] += sh_l[w][u][vl];
              continue;
            }
            const float f = ex2_approx(mx[u] - nx), q = ex2_approx(m - nx);
            const float4 y = sh_o[w][u][lane];
            sum[u] = sum[u] * f + q * sh_l[w][u][vl];
            x[u].x = x[u].x * f + q * y.x; x[u].y = x[u].y * f + q * y.y;
            x[u].z = x[u].z * f + q * y.z; x[u].w = x[u].w * f + q * y.w;
            mx[u] = nx;
          }
    }
    if (sub != 0) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = va + u * VW;
      if (v >= tr.M) continue;
      const int m = tr.m0 + v, r = (int)((uint32_t)m / ln.group);
      const float inv = normaliser(sum[u], !(sum[u] > 0.f) && row_sees(a, tr.r0 + r));
      T* out = static_cast<T*>(a.out) + (tr.r0 + r) * a.out_stride + (g * ln.G + m - r * ln.G) * HD + el;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(out) = make_float4(x[u].x * inv, x[u].y * inv, x[u].z * inv, x[u].w * inv);
      else
        *reinterpret_cast<uint2*>(out) =
            make_uint2(pack_bf16(x[u].x * inv, x[u].y * inv), pack_bf16(x[u].z * inv, x[u].w * inv));
    }
  }
}

// ----------------------------------------------------------------------------- launch

constexpr size_t kPrefixBytes = ((size_t)(kPlanTiles + 1) * 4 + 255) / 256 * 256;
constexpr int kMaxCtasPerSm = 2;

template <auto kernel>
cudaError_t allow_smem(size_t bytes) {
  static bool done[64] = {false};  // per kernel
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  return cudaSuccess;
}

template <typename T, int HD, int U>
cudaError_t launch_merge(const PackedAttnArgs& a, const Line& ln, int grid, int sms, cudaStream_t s) {
  // warps that the vectors leave idle share records, and so they do where few ranges are cut into many
  const long long ranges = (long long)ln.n_tiles * a.n_kv;
  const int per = 8 * U * (128 / HD);  // vectors that a CTA's warps take at a time when none share
  int split = 1;
  while (split < 8 && (per / split > ln.tile_rows || ranges * split * 8 < grid)) split *= 2;
  const long long shares = std::min<long long>(ln.tile_rows * split / per, (8LL * sms + ranges - 1) / ranges);
  return launch_pdl(attend_merge_kernel<T, HD, U>, dim3((unsigned)ranges, (unsigned)std::max(1LL, shares)),
                    dim3(kMergeThreads), 0, s, a, ln, grid, split);
}

// The longest that a range can be.
long long line_length(const PackedAttnArgs& a, const Line& ln) {
  return (long long)((a.max_pages + ln.unit_pages - 1) / ln.unit_pages) + ln.range_cost;
}

// Sequences of several tiles that give every SM a range: these even each other out, and twice as many pages stay
// whole (2 x 500 rows of 8 heads, 4 kv heads of 128, 1000 positions 48 -> 42 us; 500 rows, 8 kv heads of 64, 1500
// positions 39 -> 37 us).
bool filling(const Line& ln, long long ranges, int sms) { return ln.n_tps > 1 && ranges > sms; }

// The launch's line for tiles of `tile_rows` vectors and units of `unit_pages`, and how many of its tiles one
// launch takes (their units, counted in 32 bits, and kPlanTiles bound it).
Line make_line(const PackedAttnArgs& a, int tile_rows, int unit_pages, int pair_log2, int range_cost, int whole_pages,
               int sms, int* tiles_per_launch) {
  const int G = a.n_q / a.n_kv;
  const long long vectors = (long long)a.max_rows * G;
  Line ln{};
  ln.tile_rows = tile_rows;
  while ((1 << ln.rows_log2) < tile_rows) ++ln.rows_log2;
  ln.unit_pages = unit_pages;
  ln.n_tps = (int)((vectors + tile_rows - 1) / tile_rows);
  ln.tps = make_div(ln.n_tps);
  ln.group = make_div(G);
  ln.heads = make_div(a.n_kv);
  ln.G = G;
  const long long ranges = (long long)a.B * ln.n_tps * a.n_kv;
  ln.whole = a.max_pages <= (filling(ln, ranges, sms) ? 2 : 1) * whole_pages;
  ln.sms = sms;
  ln.pair_log2 = pair_log2;
  const int rows = std::min(a.max_rows, tile_rows / G + 2);
  ln.lanes = 1;
  while (ln.lanes < 32 && ln.lanes * 4 < rows) ln.lanes *= 2;
  ln.range_cost = range_cost;
  *tiles_per_launch = (int)std::min<long long>(kPlanTiles, std::max(1LL, ((1LL << 31) - 1) / (line_length(a, ln) * a.n_kv)));
  return ln;
}

// CTAs of a launch: no more than the tables' positions could keep busy (whole ranges: one each).
int line_grid(const PackedAttnArgs& a, const Line& ln, int most) {
  const long long ranges = (long long)ln.n_tiles * a.n_kv;
  return (int)std::min<long long>(most, std::max(1LL, ln.whole ? ranges : (ranges * line_length(a, ln)) >> kLoneLog2));
}

// Tables of at most so many pages: no range is cut between CTAs.  A CTA then works longer than its even part, by a
// range at most, but the merge's launch goes.  Sixteen tokens, 8 kv heads of 64, 700
// positions 14.2 -> 11.4 us; 32 x 14 rows of 8 heads, 8 kv heads of 64, 760 positions 31.9 -> 22.3 us (28.6 -> 24.0
// where lengths vary fivefold; 16 x 10 rows of such lengths 16.1 -> 18.0).  Pages take longer in tiles and at
// head_dim 128, so the limit is lower there: one sequence of 200 rows of 8 heads of 128 over 700 positions takes
// 23 us cut and 29 us whole.  The host knows the tables' width alone, so short contexts under wide tables are cut.
constexpr int whole_pages(int head_dim, bool tiles) { return head_dim == 64 ? (tiles ? 48 : 64) : 32; }

Line small_line(const PackedAttnArgs& a, int nq, int sms, int* per_launch) {
  return make_line(a, 8 * nq, 2, 3, kSmallRangeCost, whole_pages(a.head_dim, false), sms, per_launch);
}
Line tile_line(const PackedAttnArgs& a, int sms, int* per_launch) {
  return make_line(a, kTileRows, 4, 4, kTileRangeCost, whole_pages(a.head_dim, true), sms, per_launch);
}

template <typename T, int HD, int NQ>
cudaError_t launch_small(const PackedAttnArgs& a, int sms, cudaStream_t s) {
  using C = Small<T, HD, NQ>;
  int per_launch = 0;
  Line ln = small_line(a, NQ, sms, &per_launch);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  ln.prefix = reinterpret_cast<int*>(ws);
  ln.part = reinterpret_cast<float*>(ws + kPrefixBytes);
  ln.spill = ln.part + (size_t)sms * C::CTAS * 2 * C::ROWS * (HD + 2);
  cudaError_t e = allow_smem<attend_small_kernel<T, HD, NQ>>(C::smem(kPlanTiles));
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)a.B * ln.n_tps;
  for (long long t0 = 0; t0 < tiles; t0 += per_launch) {
    ln.tile0 = (int)t0;
    ln.n_tiles = (int)std::min<long long>(per_launch, tiles - t0);
    const int grid = line_grid(a, ln, sms * C::CTAS);
    ln.grid = make_div(grid);
    e = launch_pdl(attend_small_kernel<T, HD, NQ>, dim3(grid), dim3(kSmallWarps * 32), C::smem(ln.n_tiles), s, a, ln);
    if (e != cudaSuccess) return e;
    if (!ln.whole && grid > 1 && (e = launch_merge<T, HD, 1>(a, ln, grid, sms, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// CTAs of the tile kernel that an SM holds at once: two, until the line takes too much of its shared memory (16 bytes a
// tile: from 144 tiles a launch on at head_dim 128, 736 at 64).  Then one CTA an SM, and equal pieces: the others would
// only begin, and lay the line out once more, when the first have ended.  14 rows of 8 heads, 4 kv heads of
// 128, 1500 to 4000 positions: 143 sequences 153 us, 144 of them 194 us (205 with two CTAs launched for each SM).
constexpr size_t kSmemPerSm = 228 * 1024, kSmemReserved = 1024;  // of an SM; for each CTA
int tile_ctas(size_t smem) { return 2 * (smem + kSmemReserved) <= kSmemPerSm ? 2 : 1; }

template <int HD>
cudaError_t launch_tile(const PackedAttnArgs& a, int sms, cudaStream_t s) {
  using C = Tile<HD>;
  int per_launch = 0;
  Line ln = tile_line(a, sms, &per_launch);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  ln.prefix = reinterpret_cast<int*>(ws);
  ln.part = reinterpret_cast<float*>(ws + kPrefixBytes);
  cudaError_t e = allow_smem<attend_tile_kernel<HD>>(C::smem(kPlanTiles));
  if (e != cudaSuccess) return e;
  const long long tiles = (long long)a.B * ln.n_tps;
  for (long long t0 = 0; t0 < tiles; t0 += per_launch) {
    ln.tile0 = (int)t0;
    ln.n_tiles = (int)std::min<long long>(per_launch, tiles - t0);
    const int ctas = tile_ctas(C::smem(ln.n_tiles)), grid = line_grid(a, ln, sms * ctas);
    ln.grid = make_div(grid);
    ln.half = make_div(std::max(1, grid / 2));
    ln.older = ctas == 2 && grid == 2 * sms ? sms : 0;
    e = launch_pdl(attend_tile_kernel<HD>, dim3(grid), dim3(C::THREADS), C::smem(ln.n_tiles), s, a, ln);
    if (e != cudaSuccess) return e;
    if (!ln.whole && grid > 1 && (e = launch_merge<__nv_bfloat16, HD, 2>(a, ln, grid, sms, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// bf16: warp MMAs up to 16 query vectors per sequence and kv head, above them the tensor core's tiles.  B = 64 and
// 3000 positions, 8 kv heads of 64, 8 query heads each: rows of 16 vectors 59 us (tiles: 80), of 24 vectors
// 84 us (warp MMAs: 106); 4 kv heads of 128 likewise, 16 vectors 56 us (73) and 24 vectors 76 us (100).  Over a single
// sequence of 3900 positions the two are within 10 % of each other from 8 to 16 vectors.  fp32 has no exact form on the
// tensor core's tiles.
long long query_vectors(const PackedAttnArgs& a) { return (long long)a.max_rows * (a.n_q / a.n_kv); }
bool use_tiles(const PackedAttnArgs& a, pe_dtype dt) { return dt == PE_BF16 && query_vectors(a) > 16; }

template <typename T, int HD>
cudaError_t launch_attend_typed(const PackedAttnArgs& a, int sms, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (use_tiles(a, PE_BF16)) return launch_tile<HD>(a, sms, s);
  return query_vectors(a) <= 8 ? launch_small<T, HD, 1>(a, sms, s) : launch_small<T, HD, 2>(a, sms, s);
}

}  // namespace

size_t packed_attn_workspace_bytes(int head_dim, pe_dtype dt, int sms) {
  // small tiles: two records per CTA, and a part per warp, of up to 16 vectors; large ones (bf16): two records
  // of 128 vectors
  const size_t rec = (size_t)16 * (head_dim + 2) * 4, part = (size_t)16 * (head_dim + 6) * 4;
  const size_t small = 2 * rec + kSmallWarps * part, large = dt == PE_BF16 ? 2 * (size_t)kTileRows * (head_dim + 2) * 4 : 0;
  return kPrefixBytes + (size_t)sms * kMaxCtasPerSm * std::max(small, large);
}

long long packed_attn_launches(const PackedAttnArgs& a, pe_dtype dt) {
  if (a.n_rows == 0) return 0;
  int per_launch = 0;
  const Line ln =
      use_tiles(a, dt) ? tile_line(a, 1, &per_launch) : small_line(a, query_vectors(a) <= 8 ? 1 : 2, 1, &per_launch);
  return ((long long)a.B * ln.n_tps + per_launch - 1) / per_launch;
}

cudaError_t launch_attend_packed(const PackedAttnArgs& a, pe_dtype dt, int sms, cudaStream_t s) {
  if (a.n_rows == 0) return cudaSuccess;
  if (a.head_dim == 64)
    return dt == PE_BF16 ? launch_attend_typed<__nv_bfloat16, 64>(a, sms, s) : launch_attend_typed<float, 64>(a, sms, s);
  return dt == PE_BF16 ? launch_attend_typed<__nv_bfloat16, 128>(a, sms, s) : launch_attend_typed<float, 128>(a, sms, s);
}

}  // namespace pe
