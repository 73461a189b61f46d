// The experts' products on the received rows: the gated feed-forward's first half, the linear product
// behind it, and their backward passes.  One grid covers all experts; which rows an expert holds is read
// from the handle's counts on the device, so nothing waits for the host.
#include <cmath>

#include "ep_expert_dev.h"
#include "ep_internal.h"

namespace ep {
namespace expert {
namespace {

enum Kind { kLinear, kGated, kGatedGrad };

// ---------------------------------------------------------------------------
// Forward: out[r][n] = sum over k of x[r][k] w[e][n][k]; both operands lie along k
// ---------------------------------------------------------------------------

// Gated tiles hold half their columns' gate weights and then the same columns' up weights, and a wave the
// same columns of both, so that the product of the two is formed in its registers.  Rows past the expert's
// last one and columns past the last one are read as zeros and not stored.
template <class C, bool GATED>
struct AlongSrc {
  static constexpr int kCols = GATED ? C::BA / 2 : C::BA;
  static_assert(!GATED || kCols % (C::NW * C::ROWS) == 0, "a load holds rows of one matrix");
  const uint8_t *w0, *w1, *x, *sc;   // bases of the next step
  int offa[C::JA], offb[C::JB], offs;
  int left;                          // bytes of the contraction behind this lane's piece
  bool inside;

  static constexpr int wave_span_a() { return GATED ? C::TA / 2 : C::TA; }
  static __device__ __forceinline__ int frag_a_at(int fa, int i) {
    return GATED && i >= C::FA / 2 ? C::BA / 2 + fa + (i - C::FA / 2) * 16 : fa + i * 16;
  }
  static __device__ __forceinline__ bool second_scale(int fa, int i) {
    return GATED ? i >= C::FA / 2 : fa + i * 16 >= 128;
  }

  __device__ __forceinline__ AlongSrc(const AlongArgs& a, const Span& s, int n0, int m0) {
    const int w = wave_id(), piece = C::along_piece() * 16;
    const int row0 = first_row(a.rows, s, m0);
    w0 = a.w[0] + s.e * a.w_expert[0] + n0 * a.ld_w[0] - C::PIECE;
    w1 = GATED ? a.w[1] + s.e * a.w_expert[1] + n0 * a.ld_w[1] - C::PIECE : nullptr;
    x = a.x + row0 * a.ld_x - C::PIECE;
    left = static_cast<int>(a.k_bytes) - piece + C::PIECE;
#pragma unroll
    for (int j = 0; j < C::JA; ++j) {
      const int r = (j * C::NW + w) * C::ROWS + C::along_row();
      const bool second = GATED && j >= C::JA / 2;
      const int n = second ? r - kCols : r;
      offa[j] = n0 + n < a.N ? n * static_cast<int>(a.ld_w[second]) + piece : kOutside;
    }
#pragma unroll
    for (int j = 0; j < C::JB; ++j) {
      const int p = m0 + (j * C::NW + w) * C::ROWS + C::along_row();
      offb[j] = p < s.count ? (row_of(a.rows, s, p) - row0) * static_cast<int>(a.ld_x) + piece : kOutside;
    }
    if constexpr (C::F8) {
      const int t = threadIdx.x;
      if (w < C::WS / 64) {
        sc = a.x_scales + row0 * a.ld_xs - 4;
        offs = t < C::BB && m0 + t < s.count ? (row_of(a.rows, s, m0 + t) - row0) * static_cast<int>(a.ld_xs) : kOutside;
      } else {
        // the first weight scale: of the tile's first 128 columns; the second: of the second matrix, or of
        // the next 128 columns
        const int second = w > C::WS / 64, nb = (n0 >> 7) + (GATED ? 0 : second), at = GATED ? second : 0;
        sc = a.w_scales[at] + s.e * a.ws_expert[at] + nb * a.ld_ws[at] - 4;
        offs = w < C::WS / 64 + 2 && lane_id() == 0 && nb * 128 < a.N ? 0 : kOutside;
      }
    }
  }
  __device__ __forceinline__ void step() {
    w0 += C::PIECE;
    if (GATED) w1 += C::PIECE;
    x += C::PIECE;
    left -= C::PIECE;
    inside = left > 0;
    if (C::F8) sc += 4;
  }
  __device__ __forceinline__ Rsrc a_rsrc(int j) const { return rsrc(GATED && j >= C::JA / 2 ? w1 : w0, kExtent); }
  __device__ __forceinline__ Rsrc b_rsrc() const { return rsrc(x, kExtent); }
  __device__ __forceinline__ Rsrc scale_rsrc() const { return rsrc(sc, kExtent); }
  __device__ __forceinline__ int a(int j) const { return inside ? offa[j] : kOutside; }
  __device__ __forceinline__ int b(int j) const { return inside ? offb[j] : kOutside; }
  __device__ __forceinline__ int scale() const { return inside ? offs : kOutside; }
};

// Rounded to bf16: the results, and of kGatedGrad the gradients of both products, which are operands of the
// matrix unit next (all gradients together are then 0.0023 off in norm, 0.0017 with fp32 ones in between, of
// which the results' own rounding makes the most); all else stays fp32.
// The 256 x 256 tile of kGatedGrad puts 16 registers a lane aside behind its main loop, beside 128 accumulators; with
// the gradients of all the wave's rows at a time it was 32, and 64 experts of 7168 x 2048, 512 rows each, took 1 % more
// in all (6.24 ms, 6.17 so).  The FP8 gated one spills one.
// Measured, 256 experts of 7168 x 2048:
//   32768 rows, none to several hundred an expert: gated bf16 2.28 ms, 840 TFLOP/s, 11.1 GB read beyond the L2 (8.1
//   needed: an expert's row tiles drift apart); gated FP8 1.34 ms, 1440 TFLOP/s; linear bf16 1.21 ms, 800 TFLOP/s.
//   13 % of the multiplied fragments are padding (37568 rows of them); the rest of the distance is the kernels' own
//   rate without padding.
//   4 rows each, FP8: gated 1.19 ms, 6.3 TB/s, bound by the weights' bytes.  Two workgroups a CU need
//   FP8 stages of 21 KiB, three each: linear of 8 rows each in 64 experts 170 us so, 200 with one and four stages.
template <class C, int KIND, int ACT>
__global__ __launch_bounds__(C::NT) void along_kernel(AlongArgs a) {
  constexpr bool GATED = KIND != kLinear;
  constexpr int cols = GATED ? C::BA / 2 : C::BA;
  const int col_tiles = (a.N + cols - 1) / cols;
  const Span s = find_span<C::BB>(a.rows, blockIdx.x, col_tiles);
  if (s.e < 0) return;
  if (s.count < s.all && s.m == 0 && s.n == 0 && threadIdx.x == 0) atomicOr(a.rows.err, EP_DEVERR_ROW_RANGE);
  const int m0 = s.m * C::BB, n0 = s.n * cols;
  if (m0 >= s.count) return;

  typename C::Acc acc = {};
  AlongSrc<C, GATED> src(a, s, n0, m0);
  C::run(One<AlongSrc<C, GATED>>{src}, static_cast<int>((a.k_bytes + C::PIECE - 1) / C::PIECE), s.count - m0, acc);

  constexpr int CF = GATED ? C::FA / 2 : C::FA;
  const int first = n0 + (wave_id() % C::WA) * src.wave_span_a();   // the wave's first column
  const int bytes = (a.N - first) * 2;
  auto row = [&](int r) {
    const int p = m0 + C::wave_row(r);
    return p < s.count ? static_cast<int64_t>(row_of(a.rows, s, p)) : -1;
  };
  if constexpr (KIND == kGatedGrad) {
    auto grad_row = [&](int r) {
      const int64_t at = row(r);
      return at < 0 ? nullptr : reinterpret_cast<const uint8_t*>(a.grad + at * a.ld_grad + first);
    };
    C::template for_rows<CF>(bytes, grad_row, [&](int j, const uint2 (&d)[CF]) {
#pragma unroll
      for (int i = 0; i < CF; ++i) {
        const uint2 b = d[i];
        const f32x4 dh = {from_bf16(b.x & 0xffff), from_bf16(b.x >> 16), from_bf16(b.y & 0xffff), from_bf16(b.y >> 16)};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f, df;
          activate<ACT>(acc[i][j][k], &f, &df);
          acc[i][j][k] = df * dh[k] * acc[i + CF][j][k];
          acc[i + CF][j][k] = f * dh[k];
        }
      }
    });
  } else if constexpr (KIND == kGated) {
#pragma unroll
    for (int i = 0; i < CF; ++i)
#pragma unroll
      for (int j = 0; j < C::FB; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f, df;
          activate<ACT>(acc[i][j][k], &f, &df);
          acc[i][j][k] = f * acc[i + CF][j][k];
        }
  }
  // The gradients of the two products are kept in bf16: they are operands of the matrix unit next.
#pragma unroll
  for (int o = 0; o < (KIND == kGatedGrad ? 2 : 1); ++o) {
    auto out_row = [&](int r) {
      const int64_t at = row(r);
      return at < 0 ? nullptr : reinterpret_cast<uint8_t*>(a.out[o] + at * a.ld_out[o] + first);
    };
    C::template store_rows<CF, 2>(acc, o * CF, bytes, out_row);
  }
}

// ---------------------------------------------------------------------------
// Gradient of the rows: dx[r][h] = sum over i of dy[r][i] w[e][i][h], for one or two (dy, w)
// ---------------------------------------------------------------------------

template <class C>
struct RowGradSrc {
  const uint8_t *w, *dy;      // bases of the step
  int64_t ld_w;
  int offa[C::JA], offb[C::JB];
  int left;                   // contracted rows from the step on

  static constexpr int wave_span_a() { return C::TA; }
  static __device__ __forceinline__ int frag_a_at(int fa, int i) { return fa + i * 16; }

  __device__ __forceinline__ RowGradSrc(const RowGradArgs& g, const Span& s, int n0, int m0, int part) {
    const int v = wave_id(), row0 = first_row(g.rows, s, m0);
    ld_w = g.ld_w[part];
    const int64_t ld_dy = g.ld_dy[part];
#pragma unroll
    for (int j = 0; j < C::JA; ++j) {
      const int l = j * C::NW + v, n = n0 + C::template across_col<C::BA>(l);
      offa[j] = n < g.N ? C::template across_row<C::BA>(l) * static_cast<int>(ld_w) + n * 2 : kOutside;
    }
#pragma unroll
    for (int j = 0; j < C::JB; ++j) {
      const int p = m0 + (j * C::NW + v) * C::ROWS + C::along_row();
      offb[j] = p < s.count ? (row_of(g.rows, s, p) - row0) * static_cast<int>(ld_dy) + C::along_piece() * 16 : kOutside;
    }
    w = g.w[part] + s.e * g.w_expert[part] - ld_w * C::KROWS;
    dy = g.dy[part] + row0 * ld_dy - C::PIECE;
    left = g.I + C::KROWS;
  }
  __device__ __forceinline__ void step() {
    left -= C::KROWS;
    w += ld_w * C::KROWS;
    dy += C::PIECE;
  }
  // contracted rows past the last one lie behind the extent
  __device__ __forceinline__ Rsrc a_rsrc(int) const { return rsrc(w, extent_of(left * ld_w)); }
  __device__ __forceinline__ Rsrc b_rsrc() const { return rsrc(dy, kExtent); }
  __device__ __forceinline__ int a(int j) const { return offa[j]; }
  __device__ __forceinline__ int b(int j) const { return C::along_piece() * 8 < left ? offb[j] : kOutside; }
};

template <class C>
struct RowGradPlan {
  const RowGradArgs& g;
  const Span& s;
  int n0, m0;
  __device__ __forceinline__ int parts() const { return g.parts; }
  __device__ __forceinline__ RowGradSrc<C> source(int p) const { return RowGradSrc<C>(g, s, n0, m0, p); }
};

// The parts are summed in the same registers: one rounding, one write.  Two waves a SIMD at least: without the
// bound the compiler takes over 256 registers where four waves make a workgroup.
// 64 experts of 7168 x 2048, 512 rows each: gated 2.1 ms, 910 TFLOP/s; one part, 256 rows each: 0.82 ms, of which
// the weights' 1.9 GB alone take 0.31.  Bound by the matrix unit (59% busy) and by the loads of its tiles.
template <class C>
__global__ __launch_bounds__(C::NT, 2) void row_grad_kernel(RowGradArgs g) {
  const int col_tiles = (g.N + C::BA - 1) / C::BA;
  const Span s = find_span<C::BB>(g.rows, blockIdx.x, col_tiles);
  if (s.e < 0) return;
  if (s.count < s.all && s.m == 0 && s.n == 0 && threadIdx.x == 0) atomicOr(g.rows.err, EP_DEVERR_ROW_RANGE);
  const int m0 = s.m * C::BB, n0 = s.n * C::BA;
  if (m0 >= s.count) return;

  typename C::Acc acc = {};
  C::run(RowGradPlan<C>{g, s, n0, m0}, (g.I + C::KROWS - 1) / C::KROWS, s.count - m0, acc);

  const int first = n0 + (wave_id() % C::WA) * C::TA;
  C::template store_rows<C::FA, 2>(acc, 0, (g.N - first) * 2, [&](int r) -> uint8_t* {
    const int p = m0 + C::wave_row(r);
    if (p >= s.count) return nullptr;
    return reinterpret_cast<uint8_t*>(g.dx + row_of(g.rows, s, p) * g.ld_dx + first);
  });
}

// ---------------------------------------------------------------------------
// Gradient of the weights: dw[e][i][h] = sum over the expert's rows r of dy[r][i] x[r][h]
// ---------------------------------------------------------------------------

// LIST: the rows are looked up step by step (an expert's rows in several runs: LL, several sources); else they
// follow each other.  Rows past the expert's last one are zeros in both operands.
template <class C, bool LIST>
struct WeightGradSrc {
  const WeightGradArgs* args;
  Span s;
  const uint8_t *x, *dy;      // bases of the step; else the expert's first slot
  int64_t ld_dy;
  int offa[C::JA], offb[C::JB];
  int h0, i0, left;

  static constexpr int wave_span_a() { return C::TA; }
  static __device__ __forceinline__ int frag_a_at(int fa, int i) { return fa + i * 16; }

  __device__ __forceinline__ WeightGradSrc(const WeightGradArgs& g_, const Span& s_, int which, int h0_, int i0_)
      : args(&g_), s(s_), ld_dy(g_.ld_dy[which]), h0(h0_), i0(i0_) {
    const WeightGradArgs& g = g_;
    const int v = wave_id(), back = LIST ? 0 : C::KROWS;
    x = g.x + (s.first - back) * g.ld_x;
    dy = g.dy[which] + (s.first - back) * ld_dy;
    left = s.count + C::KROWS;
    if constexpr (!LIST) {
#pragma unroll
      for (int j = 0; j < C::JA; ++j) offa[j] = offset_a(j, C::template across_row<C::BA>(j * C::NW + v));
#pragma unroll
      for (int j = 0; j < C::JB; ++j) offb[j] = offset_b(j, C::template across_row<C::BB>(j * C::NW + v));
    }
  }
  __device__ __forceinline__ int offset_a(int j, int row) const {
    const WeightGradArgs& g = *args;
    const int h = h0 + C::template across_col<C::BA>(j * C::NW + wave_id());
    return h < g.H ? row * static_cast<int>(g.ld_x) + h * 2 : kOutside;
  }
  __device__ __forceinline__ int offset_b(int j, int row) const {
    const WeightGradArgs& g = *args;
    const int i = i0 + C::template across_col<C::BB>(j * C::NW + wave_id());
    return i < g.I ? row * static_cast<int>(ld_dy) + i * 2 : kOutside;
  }
  __device__ __forceinline__ void step() {
    const WeightGradArgs& g = *args;
    left -= C::KROWS;
    if constexpr (!LIST) {
      x += g.ld_x * C::KROWS;
      dy += ld_dy * C::KROWS;
    } else {
#pragma unroll
      for (int j = 0; j < C::JA; ++j) {
        const int r = C::template across_row<C::BA>(j * C::NW + wave_id());
        offa[j] = r < left ? offset_a(j, row_of(g.rows, s, s.count - left + r) - s.first) : kOutside;
      }
#pragma unroll
      for (int j = 0; j < C::JB; ++j) {
        const int r = C::template across_row<C::BB>(j * C::NW + wave_id());
        offb[j] = r < left ? offset_b(j, row_of(g.rows, s, s.count - left + r) - s.first) : kOutside;
      }
    }
  }
  __device__ __forceinline__ Rsrc a_rsrc(int) const { return rsrc(x, LIST ? kExtent : extent_of(left * args->ld_x)); }
  __device__ __forceinline__ Rsrc b_rsrc() const { return rsrc(dy, LIST ? kExtent : extent_of(left * ld_dy)); }
  __device__ __forceinline__ int a(int j) const { return offa[j]; }
  __device__ __forceinline__ int b(int j) const { return offb[j]; }
};

// An expert without rows gets zeros.  Both operands lie across the contraction: they reach the matrix unit by
// transposing LDS reads.
// 64 experts of 7168 x 2048, 256 rows each, F32: 1.1 ms, 3.5 TB/s written.  The two bounds add up: the stores of a
// tile (256 KiB; without rows 0.62 ms in all, 6.0 TB/s) and the short contraction (256 rows more: 0.335 ms, the
// library's 1440 TFLOP/s).  Two workgroups a CU of 256 x 128 or 128 x 128 gain no overlap and take more loads (a linear
// backward of 1.7 ms takes 1.9 and 2.2), nor do staggered starts.  Another order of the tiles that reads a quarter of
// the bytes beyond the L2 changes nothing.
template <class C, bool F32, bool LIST>
__global__ __launch_bounds__(C::NT, 2) void weight_grad_kernel(WeightGradArgs g) {
  const int ht = (g.H + C::BA - 1) / C::BA, it = (g.I + C::BB - 1) / C::BB;
  const int per = ht * it * g.parts;
  const int tile = xcd_tile(blockIdx.x, per * g.rows.E);
  if (tile < 0) return;
  const int e = tile / per, local = tile - e * per;
  const Span s = find_span<0>(g.rows, e, 0);
  if (s.count < s.all && local == 0 && threadIdx.x == 0) atomicOr(g.rows.err, EP_DEVERR_ROW_RANGE);
  const int which = local / (ht * it), at = local - which * ht * it, i0 = at / ht * C::BB, h0 = at % ht * C::BA;

  typename C::Acc acc = {};
  WeightGradSrc<C, LIST> src(g, s, which, h0, i0);
  C::run(One<WeightGradSrc<C, LIST>>{src}, (s.count + C::KROWS - 1) / C::KROWS, g.I - i0, acc);

  constexpr int ES = F32 ? 4 : 2;
  const int first = h0 + (wave_id() % C::WA) * C::TA;
  C::template store_rows<C::FA, ES>(acc, 0, (g.H - first) * ES, [&](int r) -> uint8_t* {
    const int i = i0 + C::wave_row(r);
    return i < g.I ? g.dw[which] + e * g.dw_expert[which] + i * g.ld_dw[which] + first * ES : nullptr;
  });
}

// The same, bf16 gradients, with one workgroup a CU that takes tile after tile: while a tile's results are stored the
// next one's first loads run, and nothing is looked up again.  64 experts of 7168 x 2048, 512 rows each, both gated
// gradients: 2.53 ms by a workgroup a tile, 2.28 so; one bf16 gradient, skewed rows: 1.25 and 1.19.  F32 gradients do
// not gain (256 rows each: 1.76 ms with the gradient of the rows, 1.81 so): twice the stores stand between the loads.
// Letting the stores run on behind the next tile's first two steps took registers from the main loop (6.2 ms in all
// became 6.7).
// An expert's tiles take as long as it has rows: a tile without any as long as kTileRows rows (512 rows: 20 us, of
// which 256 are 6).  The XCDs share the tiles by that measure; by their number alone, skewed rows made the fullest XCD
// late (64 experts of 7168 x 2048, 512 rows each on average, one gradient and that of the rows: 2.32 ms, 2.13 so).
// Below eight turns of all workgroups equal numbers do (24 experts of 1152 x 712, gated: 102.4 us, by rows 103.9).
constexpr int kTileRows = 320, kTurns = 8;

// The first tile behind the share `t` of all that the experts take; before[e]: rows of the experts before e.
__device__ __forceinline__ int tile_behind(const int* before, int experts, int per, int64_t t) {
  auto cost = [&](int e) { return before[e] + static_cast<int64_t>(kTileRows) * e; };   // of the experts before e
  int e = -1;   // the last one that begins at t or before it
  for (int e0 = 0; e0 < experts; e0 += 64) e += __popcll(__ballot(e0 + lane_id() < experts && cost(e0 + lane_id()) <= t));
  if (cost(experts) <= t) return experts * per;
  return e * per + static_cast<int>((t - cost(e)) * per / (cost(e + 1) - cost(e)));
}

template <class C, bool LIST>
__global__ __launch_bounds__(C::NT, 2) void weight_grads_kernel(WeightGradArgs g) {
  __shared__ int before[kMaxExperts + 1];   // rows of the experts before each
  const int ht = (g.H + C::BA - 1) / C::BA, it = (g.I + C::BB - 1) / C::BB;
  const int per = ht * it * g.parts;
  if (wave_id() == 0) {
    int at = 0;
    for (int e0 = 0; e0 < g.rows.E; e0 += 64) {
      const int n = e0 + lane_id() < g.rows.E ? rows_of(g.rows, e0 + lane_id()) : 0, to = scan64(n);
      if (e0 + lane_id() < g.rows.E) before[e0 + lane_id()] = at + to - n;
      at += __builtin_amdgcn_readlane(to, 63);
    }
    if (lane_id() == 0) before[g.rows.E] = at;
  }
  __syncthreads();
  // An XCD's workgroups take its tiles in turn.
  const int64_t all = before[g.rows.E] + static_cast<int64_t>(kTileRows) * g.rows.E;
  const int turn = gridDim.x >> 3;
  auto border = [&](int xcd) {
    const int total = per * g.rows.E, part = (total + 7) >> 3;
    if (total < kTurns * 8 * turn) return xcd * part < total ? xcd * part : total;
    // at whole turns, or XCDs with a few tiles more would take a turn more
    const int t = (tile_behind(before, g.rows.E, per, all * xcd / 8) + turn / 2) / turn * turn;
    return __builtin_amdgcn_readfirstlane(xcd == 8 || t > total ? total : t);   // the last turn may be a part of one
  };
  int tile = border(blockIdx.x & 7) + (blockIdx.x >> 3);
  const int end = border((blockIdx.x & 7) + 1);
  if (tile >= end) return;

  int e, which, i0, h0;
  auto take = [&]() {
    e = tile / per;
    const int local = tile - e * per;
    which = local / (ht * it);
    const int at = local - which * ht * it;
    i0 = at / ht * C::BB;
    h0 = at % ht * C::BA;
    Span s;
    s.e = e;
    s.before = __builtin_amdgcn_readfirstlane(before[e]);
    s.all = s.count = __builtin_amdgcn_readfirstlane(before[e + 1]) - s.before;
    s.first = g.rows.stride > 0 ? e * g.rows.stride : s.before;
    keep_limit(g.rows, &s);
    if (s.count < s.all && local == 0 && threadIdx.x == 0) atomicOr(g.rows.err, EP_DEVERR_ROW_RANGE);
    return s;
  };
  Span s = take();
  WeightGradSrc<C, LIST> src(g, s, which, h0, i0);
  C::start(src);
  for (;;) {
    typename C::Acc acc = {};
    C::finish(src, (s.count + C::KROWS - 1) / C::KROWS, g.I - i0, acc);

    const int first = h0 + (wave_id() % C::WA) * C::TA, from = i0, bytes = (g.H - first) * 2;
    uint8_t* const to = g.dw[which] + e * g.dw_expert[which] + first * 2;
    const int64_t ld = g.ld_dw[which];
    const bool more = tile + turn < end;
    if (more) {
      tile += turn;
      s = take();
      src = WeightGradSrc<C, LIST>(g, s, which, h0, i0);
      C::start(src);
    }
    C::template store_rows<C::FA, 2, typename C::LastStage>(acc, 0, bytes, [&](int r) -> uint8_t* {
      const int i = from + C::wave_row(r);
      return i < g.I ? to + i * ld : nullptr;
    });
    if (!more) break;
  }
}

// ---------------------------------------------------------------------------
// Rows per expert where several sources fill their own slots (LL)
// ---------------------------------------------------------------------------

// One workgroup (256 threads) per expert: its rows (e*S + s)*T_max + slot for all sources in order, at the sum of the
// counts before it.  Each workgroup sums those counts itself: E*S of them at most, from the L2.  64 experts with 4
// sources: 3 us, the launch.
__device__ __forceinline__ void list_rows(const int32_t* counts, int e, int S, int slots, int32_t* total, int32_t* list) {
  __shared__ int part[4];
  int sum = 0;
  for (int i = threadIdx.x; i < e * S; i += 256) sum += counts[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
  if (lane_id() == 0) part[wave_id()] = sum;
  __syncthreads();
  int at = part[0] + part[1] + part[2] + part[3];
  const int first = at;
  for (int s0 = 0; s0 < S; s0 += 64) {
    const int c = s0 + lane_id() < S ? counts[e * S + s0 + lane_id()] : 0;
    const int to = scan64(c);
    const int here = S - s0 < 64 ? S - s0 : 64;
    for (int q = wave_id(); q < here; q += 4) {
      const int n = __builtin_amdgcn_readlane(c, q), from = at + __builtin_amdgcn_readlane(to, q) - n;
      for (int i = lane_id(); i < n; i += 64) list[from + i] = (e * S + s0 + q) * slots + i;
    }
    at += __builtin_amdgcn_readlane(to, 63);
  }
  if (threadIdx.x == 0) total[e] = at - first;
}
__global__ __launch_bounds__(256) void list_rows_kernel(const int32_t* counts, int S, int slots, int32_t* total,
                                                        int32_t* list) {
  list_rows(counts, blockIdx.x, S, slots, total, list);
}

// ---------------------------------------------------------------------------
// Rows kept in 8 bits, back in bf16
// ---------------------------------------------------------------------------

// out = bf16_rne(code * scale) on the experts' rows.  The product has up to 28 bits, an operand of the matrix unit 8: the
// rounding is ep_dequantize_rows' own, so that gradients from kept codes have the bits of those from kept bf16 rows.  The
// gated gradients are 0.0033 of their norm off 64 bits so, 0.0023 with rows that bf16 holds, 0.0017 with their own
// rounding alone; the scales cannot be applied behind the products instead, as those of the weights sum over rows.
// Memory bounds it (32768 rows of 7168: 104 us, 6.9 TB/s; 2997 of 1152: 5.5 us).  A wave takes 2048 codes of a row, eight
// a lane and load, so that a store instruction writes one run.  HT: the rows are the first ones, as many as the counts
// sum up to.  LL: entry by entry, its tile's prefix and its rank in the tile.  A grid by experts' tiles, each finding its
// span as the products do: 14 us more at those 2997 rows on 24 experts, 500 us at the 32768.  The products behind it read
// the rows again: plain stores.  Where they need the rows' list too, the first workgroups make it: a launch less (linear
// backward of 64 experts, 4 sources of 64 tokens: 53.8 us, 56.5 with two).
constexpr int kDecodeChunks = 4;   // eight codes of a lane

template <bool FIRST>
__global__ __launch_bounds__(256) void decode_kernel(DecodeArgs a, int W) {
  typedef __attribute__((ext_vector_type(2))) float f32x2;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  typedef __attribute__((ext_vector_type(2))) int i32x2;
  int block = blockIdx.x, blocks = gridDim.x;
  if constexpr (!FIRST) {
    if (a.list) {
      if (block < a.E) {
        list_rows(a.ll_count, block, a.S, a.slots, a.total, a.list);
        return;
      }
      block -= a.E;
      blocks -= a.E;
    }
  }
  const int C = a.C / 8;
  const int64_t waves = static_cast<int64_t>(blocks) * 4;
  const int64_t first = static_cast<int64_t>(block) * 4 + wave_id();
  int64_t total = a.n * W;
  if constexpr (FIRST) {
    int sum = 0;
    for (int e0 = 0; e0 < a.E; e0 += 256) {
#pragma unroll
      for (int e = 0; e < 256; e += 64) sum += e0 + e + lane_id() < a.E ? a.count[e0 + e + lane_id()] : 0;
    }
    int64_t n = __builtin_amdgcn_readlane(scan64(sum), 63);
    if (n > a.rows) {
      n = a.rows;
      if (first == 0 && lane_id() == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
    }
    total = n * W;
  }
  for (int64_t at = first; at < total; at += waves) {
    int64_t row = at / W;
    const int c0 = static_cast<int>(at - row * W) * kDecodeChunks * 64 + lane_id();
    if constexpr (!FIRST) {
      const uint32_t token = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.K);
      const uint32_t s = token / static_cast<uint32_t>(a.T), t = token - s * static_cast<uint32_t>(a.T);
      const int e = a.topk[row], rank = a.rank_e[row];
      if (rank < 0 || static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) continue;
      const int slot = a.hist_e[(static_cast<int64_t>(s) * a.tps + t / kLayoutTile) * a.E + e] + rank;
      if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(a.slots)) continue;
      row = (static_cast<int64_t>(e) * a.S + s) * a.slots + slot;
    }
    i32x2 q[kDecodeChunks];
    float scale[kDecodeChunks];
#pragma unroll
    for (int v = 0; v < kDecodeChunks; ++v) {
      const int c = c0 + v * 64;
      q[v] = c < C ? __builtin_nontemporal_load(reinterpret_cast<const i32x2*>(a.x + row * a.ld_x + 8 * c)) : i32x2{0, 0};
      scale[v] = c < C ? a.scales[row * a.ld_s + (c >> 4)] : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < kDecodeChunks; ++v) {
      const int c = c0 + v * 64;
      if (c >= C) continue;
      i32x4 o;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[v][w], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[v][w], true);
        o[2 * w] = __builtin_bit_cast(int, __builtin_convertvector(f32x2{lo[0] * scale[v], lo[1] * scale[v]}, bf16x2));
        o[2 * w + 1] = __builtin_bit_cast(int, __builtin_convertvector(f32x2{hi[0] * scale[v], hi[1] * scale[v]}, bf16x2));
      }
      *reinterpret_cast<i32x4*>(a.out + row * a.ld_out + 8 * c) = o;
    }
  }
}

// Blocks for at most `rows` rows in all and `per_expert` in one.
template <int BM>
int64_t row_tiles(const ExpertRows& r, int64_t rows, int64_t per_expert) {
  const int64_t by_rows = (rows + static_cast<int64_t>(r.E) * (BM - 1)) / BM;
  const int64_t by_expert = r.E * ((per_expert + BM - 1) / BM);
  return by_rows < by_expert ? by_rows : by_expert;
}

constexpr int64_t kMaxBlocks = INT32_MAX / 512;
constexpr int kCus = 256;

template <class C, int KIND, int ACT>
hipError_t launch_along_as(const AlongArgs& a, hipStream_t stream, bool check) {
  const int cols = KIND == kLinear ? C::BA : C::BA / 2;
  const int64_t tiles = row_tiles<C::BB>(a.rows, a.rows_max, a.per_expert_max) * ((a.N + cols - 1) / cols);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (tiles == 0 || check) return hipSuccess;
  along_kernel<C, KIND, ACT><<<static_cast<int>((tiles + 7) / 8 * 8), C::NT, 0, stream>>>(a);
  return hipGetLastError();
}

// Which tile a product over the rows takes, by the average rows of an expert (the counts themselves are only
// on the device) and by how many 256 x 256 tiles there are for the 256 CUs.  Measured, 64 experts of 2048 x 1408,
// rows spread evenly at random, us (small / middle / big):
//   rows an expert    linear bf16         gradient of the rows    gated FP8
//         16          74 /  78 /  87       74 /  80 /  85          78 /  82 /  99
//         24          80 /  78 /  87       74 /  75 /  86          79 /  82 / 101
//         32          83 /  79 /  88       85 /  77 /  87          91 /  86 / 101
//         48          96 /  81 /  90       90 /  80 /  91         107 /  91 / 104
//         96         128 /  90 /  96      124 / 114 / 101         153 / 111 / 112
//        128         153 / 114 / 101      148 / 121 / 110         184 / 141 / 123
// Both borders lie where the forward products' times cross; the gradient of the rows would take the big tile from
// 64 rows on (98 / 94).  The gated bf16 product's times move by a tenth from run to run: 24: 146 / 157 / 177, 32: 157
// / 150 to 171 / 181, 48: 177 / 153 to 182 / 170 to 198, 96: 243 / 170 / 182 to 202, 128: 290 / 220 / 190 to 220.
// From 24 rows on the small tile's 32 rows are often two tiles, which read the weights twice.  Rows spread over
// the experts as a router leaves them make many tiles of the average's multiple: at 128 rows on average (256
// experts of 7168 x 2048, bf16) the big tile takes 2.35 ms, the middle one 2.67.
// Few big tiles leave CUs idle: 88 of them (8 experts, 256 rows each) take 48 us, middle ones 37.
// No more middle tiles than CUs, as a random routing leaves the rows: each has a CU's LDS to itself, and a ring of four
// stages keeps three of them in flight instead of one.  bf16, 8 experts of 1024 x 768, us, two stages / four: gated
// 15.1 / 11.1 of 32 rows each, 17.2 / 14.4 of 128; linear 10.3 / 9.7 and 14.9 / 13.0.  With more tiles two workgroups
// share a CU, which four stages leave no room for: 24 experts of 1152 x 712, 48 rows each, gated 19.9 / 25.8.  With 128
// rows each on average half of the experts have two row tiles: 16 of 1024 x 768, gated, 21.6 / 26.5.
enum Size { kSmall, kMiddle, kMiddleDeep, kBig };
Size tile_size(const ExpertRows& r, int64_t rows, int64_t col_tiles, int64_t middle_col_tiles) {
  const int64_t each = rows / r.E;
  if (each <= 24) return kSmall;
  if (each > 96 && r.E * ((each + 255) / 256) * col_tiles >= 256) return kBig;
  // an expert's row tiles on average, its rows being spread by the square root of their number
  auto more_than = [&](int64_t n) { return 0.5 * std::erfc((n - each) / std::sqrt(2.0 * each)); };
  const int64_t least = (each - 1) / 128;
  const double row_tiles = least + more_than(128 * least) + more_than(128 * (least + 1));
  return r.E * row_tiles * middle_col_tiles <= kCus ? kMiddleDeep : kMiddle;
}

template <bool F8, int KIND, int ACT>
hipError_t launch_along_kind(const AlongArgs& a, hipStream_t stream, bool check) {
  const int cols = KIND == kLinear ? 256 : 128;
  switch (tile_size(a.rows, a.rows_max, (a.N + cols - 1) / cols, (a.N + cols / 2 - 1) / (cols / 2))) {
    case kSmall: return launch_along_as<Core<128, 32, 4, 1, false, false, F8, F8 ? 3 : 4, 128>, KIND, ACT>(a, stream, check);
    case kMiddleDeep:
      if constexpr (!F8) return launch_along_as<Core<128, 128, 2, 2, false, false, F8, 4, 128>, KIND, ACT>(a, stream, check);
      [[fallthrough]];
    case kMiddle: return launch_along_as<Core<128, 128, 2, 2, false, false, F8, 2, 128>, KIND, ACT>(a, stream, check);
    default: return launch_along_as<Core<256, 256, 2, 4, false, false, F8, 2, 128>, KIND, ACT>(a, stream, check);
  }
}

template <bool F8>
hipError_t launch_along_type(const AlongArgs& a, int kind, int act, hipStream_t stream, bool check) {
  if (kind == kLinear) return launch_along_kind<F8, kLinear, kSilu>(a, stream, check);
  return act == kSilu ? launch_along_kind<F8, kGated, kSilu>(a, stream, check)
                      : launch_along_kind<F8, kGated, kGeluTanh>(a, stream, check);
}

}  // namespace

hipError_t launch_list_rows(const int32_t* counts, int E, int S, int slots, int32_t* total, int32_t* list,
                            hipStream_t stream) {
  list_rows_kernel<<<E, 256, 0, stream>>>(counts, S, slots, total, list);
  return hipGetLastError();
}

hipError_t launch_linear(const AlongArgs& a, bool fp8, hipStream_t stream, bool check) {
  return fp8 ? launch_along_type<true>(a, kLinear, 0, stream, check) : launch_along_type<false>(a, kLinear, 0, stream, check);
}

hipError_t launch_gated(const AlongArgs& a, bool fp8, int act, hipStream_t stream, bool check) {
  return fp8 ? launch_along_type<true>(a, kGated, act, stream, check) : launch_along_type<false>(a, kGated, act, stream, check);
}

hipError_t launch_gated_grad(const AlongArgs& a, int act, hipStream_t stream, bool check) {
  return act == kSilu ? launch_along_kind<false, kGatedGrad, kSilu>(a, stream, check)
                      : launch_along_kind<false, kGatedGrad, kGeluTanh>(a, stream, check);
}

namespace {

template <class C>
hipError_t launch_row_grad_as(const RowGradArgs& g, hipStream_t stream, bool check) {
  const int64_t tiles = row_tiles<C::BB>(g.rows, g.rows_max, g.per_expert_max) * ((g.N + C::BA - 1) / C::BA);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (tiles == 0 || check) return hipSuccess;
  row_grad_kernel<C><<<static_cast<int>((tiles + 7) / 8 * 8), C::NT, 0, stream>>>(g);
  return hipGetLastError();
}

// One workgroup a CU: an eighth of them on each XCD.
template <class C>
hipError_t launch_weight_grads_as(const WeightGradArgs& g, hipStream_t stream, bool check) {
  const int64_t tiles = static_cast<int64_t>(g.rows.E) * g.parts * ((g.H + C::BA - 1) / C::BA) *
                        ((g.I + C::BB - 1) / C::BB);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  if (scattered(g.rows)) weight_grads_kernel<C, true><<<kCus, C::NT, 0, stream>>>(g);
  else weight_grads_kernel<C, false><<<kCus, C::NT, 0, stream>>>(g);
  return hipGetLastError();
}

template <class C, bool F32>
hipError_t launch_weight_grad_as(const WeightGradArgs& g, hipStream_t stream, bool check) {
  const int64_t tiles = static_cast<int64_t>(g.rows.E) * g.parts * ((g.H + C::BA - 1) / C::BA) *
                        ((g.I + C::BB - 1) / C::BB);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  const int blocks = static_cast<int>((tiles + 7) / 8 * 8);
  if (scattered(g.rows)) weight_grad_kernel<C, F32, true><<<blocks, C::NT, 0, stream>>>(g);
  else weight_grad_kernel<C, F32, false><<<blocks, C::NT, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_decode(const DecodeArgs& a, hipStream_t stream) {
  const int W = (a.C / 8 + 64 * kDecodeChunks - 1) / (64 * kDecodeChunks);
  const dim3 grid(grid_blocks((a.n * W + 3) / 4 + (a.list ? a.E : 0), 256)), block(256);
  if (a.count) decode_kernel<true><<<grid, block, 0, stream>>>(a, W);
  else decode_kernel<false><<<grid, block, 0, stream>>>(a, W);
  return hipGetLastError();
}

hipError_t launch_row_grad(const RowGradArgs& g, hipStream_t stream, bool check) {
  switch (tile_size(g.rows, g.rows_max, (g.N + 255) / 256, (g.N + 127) / 128)) {
    case kSmall: return launch_row_grad_as<Core<128, 32, 4, 1, true, false, false, 4, 128>>(g, stream, check);
    case kMiddleDeep:
    case kMiddle: return launch_row_grad_as<Core<128, 128, 2, 2, true, false, false, 4, 64>>(g, stream, check);
    default: return launch_row_grad_as<Core<256, 256, 2, 4, true, false, false, 4, 64>>(g, stream, check);
  }
}

// F32 gradients, a workgroup a tile: with fewer than two 256 x 256 tiles a CU the smaller ones fill the chip.  128 rows an
// expert, us, small tiles and big ones, by the number of big ones:
//     96 (8 experts of 1024 x 768)     16   21       640 (40 of 1024 x 1024)    50   53
//    256 (16 of 1024 x 1024)           26   25      1024 (64 of 1024 x 1024)    77   72
//    384 (24 of 1024 x 1024)           34   37      1536 (96 of 1024 x 1024)   117  102
//    512 (32 of 1024 x 1024)           42   40      2048 (128 of 1024 x 1024)  163  145
// Near the border the big ones win where they fill the CUs a whole number of times (256, 512).
// bf16 gradients, big tiles one after the other: the smaller ones win as long as all of them run at once, two a CU.
// Linear backward of 4 / 32 / 128 / 384 rows an expert, us, by the number of small tiles:
//    384 (8 experts of 1024 x 768)    small 15.1 19.4 25.2 27.9   big 16.0 20.5 27.2 31.7
//    480 (10)                               15.8 19.5 24.8 29.2       16.8 21.2 27.2 32.0
//    576 (12)                               20.4 23.7 29.6 35.9       17.4 21.3 27.0 32.2
//   1296 (24 of 1152 x 712, odd)            31.7 34.0 42.0 61.6       27.8 30.9 39.5 60.1
//   1408 (8 of 2048 x 1408)                 30.1 37.3 46.6 69.2       27.0 34.5 43.8 67.0
//   1920 (40 of 1024 x 768)                 36.5 39.2 52.7 83.9       30.2 33.0 45.8 77.3
hipError_t launch_weight_grad(const WeightGradArgs& g, bool f32, hipStream_t stream, bool check) {
  using Small = Core<128, 128, 2, 2, true, true, false, 4, 64>;
  using Big = Core<256, 256, 2, 4, true, true, false, 4, 64>;
  const int64_t matrices = static_cast<int64_t>(g.rows.E) * g.parts;
  const int64_t small = matrices * ((g.H + 127) / 128) * ((g.I + 127) / 128);
  const int64_t big = matrices * ((g.H + 255) / 256) * ((g.I + 255) / 256);
  if (f32) {
    return big < 2 * kCus ? launch_weight_grad_as<Small, true>(g, stream, check)
                          : launch_weight_grad_as<Big, true>(g, stream, check);
  }
  return small <= 2 * kCus ? launch_weight_grad_as<Small, false>(g, stream, check)
                           : launch_weight_grads_as<Big>(g, stream, check);
}

}  // namespace expert
}  // namespace ep
