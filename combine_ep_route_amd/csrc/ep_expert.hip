// The experts' products on the received rows: the gated feed-forward's first half, the linear product
// behind it, and their backward passes.  One grid covers all experts; which rows an expert holds is read
// from the handle's counts on the device, so nothing waits for the host.
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
// same columns of both, so that the product of the two is formed in its registers.
template <class C, bool GATED>
struct AlongSrc {
  const uint8_t* pa[C::JA];
  const uint8_t* pb[C::JB];
  const uint8_t* ps;
  int limit;
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
    constexpr int cols = GATED ? C::BA / 2 : C::BA;
    limit = static_cast<int>(a.k_bytes) - piece;
#pragma unroll
    for (int j = 0; j < C::JA; ++j) {
      const int r = (j * C::NW + w) * 8 + C::along_row();
      const bool second = GATED && r >= cols;
      int n = n0 + (second ? r - cols : r);
      n = n < a.N ? n : a.N - 1;   // columns past the last one are not stored
      pa[j] = (second ? a.w[1] + s.e * a.w_expert[1] + n * a.ld_w[1] : a.w[0] + s.e * a.w_expert[0] + n * a.ld_w[0]) + piece;
    }
#pragma unroll
    for (int j = 0; j < C::JB; ++j) pb[j] = a.x + row(a, s, m0 + (j * C::NW + w) * 8 + C::along_row()) * a.ld_x + piece;
    if constexpr (C::F8) {
      const int t = threadIdx.x;
      if (t < C::BB) {
        ps = a.x_scales + row(a, s, m0 + t) * a.ld_xs;
      } else {
        // thread BB: the scale of the tile's first 128 columns; BB + 1: of the second matrix or 128 columns
        const int second = t == C::BB + 1, last = (a.N - 1) >> 7;
        int nb = (n0 >> 7) + (GATED ? 0 : second);
        nb = nb < last ? nb : last;
        const int at = GATED ? second : 0;
        ps = a.w_scales[at] + s.e * a.ws_expert[at] + nb * a.ld_ws[at];
      }
    }
  }
  // rows past the expert's last one are read as its last row, and not stored
  static __device__ __forceinline__ int64_t row(const AlongArgs& a, const Span& s, int p) {
    return row_of(a.rows, s, p < s.count ? p : s.count - 1);
  }
  __device__ __forceinline__ void step(int t) { inside = t * kPiece < limit; }
  __device__ __forceinline__ const uint8_t* a(int j, int t) const { return inside ? pa[j] + t * kPiece : zeros(); }
  __device__ __forceinline__ const uint8_t* b(int j, int t) const { return inside ? pb[j] + t * kPiece : zeros(); }
  __device__ __forceinline__ const uint8_t* scale(int t) const { return inside ? ps + t * 4 : zeros(); }
};

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
  C::run(src, static_cast<int>((a.k_bytes + kPiece - 1) / kPiece), s.count - m0, acc);

  const int l = lane_id(), w = wave_id();
  const int fa = (w % C::WA) * src.wave_span_a();
#pragma unroll
  for (int j = 0; j < C::FB; ++j) {
    const int p = m0 + C::from_b(j) + (l & 15);
    if (p >= s.count) continue;
    const int64_t r = row_of(a.rows, s, p);
#pragma unroll
    for (int i = 0; i < (GATED ? C::FA / 2 : C::FA); ++i) {
      const int n = n0 + fa + i * 16 + (l >> 4) * 4;
      if (n >= a.N) continue;
      if constexpr (KIND == kLinear) {
        *reinterpret_cast<uint2*>(a.out[0] + r * a.ld_out[0] + n) = bf16x4(acc[i][j]);
      } else {
        const f32x4 g = acc[i][j], u = acc[i + C::FA / 2][j];
        f32x4 f, df;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float v, d;
          activate<ACT>(g[k], &v, &d);
          f[k] = v;
          df[k] = d;
        }
        if constexpr (KIND == kGated) {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] *= u[k];
          *reinterpret_cast<uint2*>(a.out[0] + r * a.ld_out[0] + n) = bf16x4(f);
        } else {
          // The gradients of the two products are kept in bf16: they are operands of the matrix unit next.
          const uint2 d = *reinterpret_cast<const uint2*>(a.grad + r * a.ld_grad + n);
          const f32x4 dh = {from_bf16(d.x & 0xffff), from_bf16(d.x >> 16), from_bf16(d.y & 0xffff), from_bf16(d.y >> 16)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            df[k] *= dh[k] * u[k];
            f[k] *= dh[k];
          }
          *reinterpret_cast<uint2*>(a.out[0] + r * a.ld_out[0] + n) = bf16x4(df);
          *reinterpret_cast<uint2*>(a.out[1] + r * a.ld_out[1] + n) = bf16x4(f);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient of the rows: dx[r][h] = sum over i of dy[r][i] w[e][i][h], for one or two (dy, w)
// ---------------------------------------------------------------------------

template <class C>
struct RowGradSrc {
  const RowGradArgs& g;
  const Span& s;
  const uint8_t* pa[C::JA];   // advanced step by step
  const uint8_t* pb[C::JB];
  int64_t advance;
  int n0, m0, steps, part, left;

  static constexpr int wave_span_a() { return C::TA; }
  static __device__ __forceinline__ int frag_a_at(int fa, int i) { return fa + i * 16; }

  __device__ __forceinline__ RowGradSrc(const RowGradArgs& g_, const Span& s_, int n0_, int m0_)
      : g(g_), s(s_), n0(n0_), m0(m0_), steps((g_.I + kStepRows - 1) / kStepRows), part(-1) {}

  __device__ __forceinline__ void begin(int which) {
    const int w = wave_id();
#pragma unroll
    for (int j = 0; j < C::JA; ++j) {
      const int at = j * C::NW + w;
      int n = n0 + C::template across_col<C::BA>(at);
      n = n < g.N ? n : 0;   // columns past the last one are not stored
      pa[j] = g.w[which] + s.e * g.w_expert[which] + C::template across_row<C::BA>(at) * g.ld_w[which] + n * 2;
    }
#pragma unroll
    for (int j = 0; j < C::JB; ++j) {
      const int p = m0 + (j * C::NW + w) * 8 + C::along_row();
      pb[j] = g.dy[which] + static_cast<int64_t>(row_of(g.rows, s, p < s.count ? p : s.count - 1)) * g.ld_dy[which] +
              C::along_piece() * 16;
    }
    advance = g.ld_w[which] * kStepRows;
    part = which;
    left = g.I;
  }
  // the core asks for every step once, in order
  __device__ __forceinline__ void step(int t) {
    const int which = g.parts == 2 && t >= steps;
    if (which != part) {
      begin(which);
      return;
    }
    left -= kStepRows;
#pragma unroll
    for (int j = 0; j < C::JA; ++j) pa[j] += advance;
#pragma unroll
    for (int j = 0; j < C::JB; ++j) pb[j] += kPiece;
  }
  __device__ __forceinline__ const uint8_t* a(int j, int) const {
    return C::template across_row<C::BA>(j * C::NW + wave_id()) < left ? pa[j] : zeros();
  }
  __device__ __forceinline__ const uint8_t* b(int j, int) const {
    return C::along_piece() * 8 < left ? pb[j] : zeros();
  }
};

template <class C>
__global__ __launch_bounds__(C::NT) void row_grad_kernel(RowGradArgs g) {
  const int col_tiles = (g.N + C::BA - 1) / C::BA;
  const Span s = find_span<C::BB>(g.rows, blockIdx.x, col_tiles);
  if (s.e < 0) return;
  if (s.count < s.all && s.m == 0 && s.n == 0 && threadIdx.x == 0) atomicOr(g.rows.err, EP_DEVERR_ROW_RANGE);
  const int m0 = s.m * C::BB, n0 = s.n * C::BA;
  if (m0 >= s.count) return;

  typename C::Acc acc = {};
  RowGradSrc<C> src(g, s, n0, m0);
  C::run(src, src.steps * g.parts, s.count - m0, acc);

  const int l = lane_id(), w = wave_id();
#pragma unroll
  for (int j = 0; j < C::FB; ++j) {
    const int p = m0 + C::from_b(j) + (l & 15);
    if (p >= s.count) continue;
    const int64_t r = row_of(g.rows, s, p);
#pragma unroll
    for (int i = 0; i < C::FA; ++i) {
      const int n = n0 + (w % C::WA) * C::TA + i * 16 + (l >> 4) * 4;
      if (n < g.N) *reinterpret_cast<uint2*>(g.dx + r * g.ld_dx + n) = bf16x4(acc[i][j]);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weights: dw[e][i][h] = sum over the expert's rows r of dy[r][i] x[r][h]
// ---------------------------------------------------------------------------

template <class C>
struct WeightGradSrc {
  const WeightGradArgs& g;
  const Span& s;
  const uint8_t* dy;
  int64_t ld_dy;
  int h0, i0;

  static constexpr int wave_span_a() { return C::TA; }
  static __device__ __forceinline__ int frag_a_at(int fa, int i) { return fa + i * 16; }
  __device__ __forceinline__ void step(int) {}
  // rows past the expert's last one are zeros in both operands; columns past the last one are not stored
  __device__ __forceinline__ const uint8_t* a(int j, int t) const {
    const int at = j * C::NW + wave_id(), p = t * kStepRows + C::template across_row<C::BA>(at);
    const int h = h0 + C::template across_col<C::BA>(at);
    return p < s.count ? g.x + static_cast<int64_t>(row_of(g.rows, s, p)) * g.ld_x + (h < g.H ? h : 0) * 2 : zeros();
  }
  __device__ __forceinline__ const uint8_t* b(int j, int t) const {
    const int at = j * C::NW + wave_id(), p = t * kStepRows + C::template across_row<C::BB>(at);
    const int i = i0 + C::template across_col<C::BB>(at);
    return p < s.count ? dy + static_cast<int64_t>(row_of(g.rows, s, p)) * ld_dy + (i < g.I ? i : 0) * 2 : zeros();
  }
};

template <class C, bool F32>
__global__ __launch_bounds__(C::NT) void weight_grad_kernel(WeightGradArgs g) {
  const int ht = (g.H + C::BA - 1) / C::BA, it = (g.I + C::BB - 1) / C::BB;
  const int per = ht * it * g.parts;
  const int tile = xcd_tile(blockIdx.x, per * g.rows.E);
  if (tile < 0) return;
  const int e = tile / per, local = tile - e * per;
  const Span s = find_span<0>(g.rows, e, 0);
  if (s.count < s.all && local == 0 && threadIdx.x == 0) atomicOr(g.rows.err, EP_DEVERR_ROW_RANGE);
  const int which = local / (ht * it), at = local - which * ht * it, i0 = at / ht * C::BB, h0 = at % ht * C::BA;

  typename C::Acc acc = {};
  WeightGradSrc<C> src{g, s, g.dy[which], g.ld_dy[which], h0, i0};
  C::run(src, (s.count + kStepRows - 1) / kStepRows, g.I - i0, acc);

  const int l = lane_id(), w = wave_id();
#pragma unroll
  for (int j = 0; j < C::FB; ++j) {
    const int i = i0 + C::from_b(j) + (l & 15);
    if (i >= g.I) continue;
#pragma unroll
    for (int f = 0; f < C::FA; ++f) {
      const int h = h0 + (w % C::WA) * C::TA + f * 16 + (l >> 4) * 4;
      if (h >= g.H) continue;
      uint8_t* p = g.dw[which] + e * g.dw_expert[which] + i * g.ld_dw[which];
      if constexpr (F32) *reinterpret_cast<f32x4*>(p + h * 4) = acc[f][j];
      else *reinterpret_cast<uint2*>(p + h * 2) = bf16x4(acc[f][j]);
    }
  }
}

// ---------------------------------------------------------------------------
// Rows per expert where several sources fill their own slots (LL)
// ---------------------------------------------------------------------------

// One workgroup per expert: its rows (e*S + s)*T_max + slot for all sources in order, at the sum of the
// counts before it.  Each workgroup sums those counts itself: E*S of them at most, from the L2.
__global__ __launch_bounds__(256) void list_rows_kernel(const int32_t* counts, int S, int slots, int32_t* total,
                                                        int32_t* list) {
  __shared__ int part[4];
  const int e = blockIdx.x;
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

// Blocks for at most `rows` rows in all and `per_expert` in one.
template <int BM>
int64_t row_tiles(const ExpertRows& r, int64_t rows, int64_t per_expert) {
  const int64_t by_rows = (rows + static_cast<int64_t>(r.E) * (BM - 1)) / BM;
  const int64_t by_expert = r.E * ((per_expert + BM - 1) / BM);
  return by_rows < by_expert ? by_rows : by_expert;
}

constexpr int64_t kMaxBlocks = INT32_MAX / 512;

template <class C, int KIND, int ACT>
hipError_t launch_along_as(const AlongArgs& a, hipStream_t stream, bool check) {
  const int cols = KIND == kLinear ? C::BA : C::BA / 2;
  const int64_t tiles = row_tiles<C::BB>(a.rows, a.rows_max, a.per_expert_max) * ((a.N + cols - 1) / cols);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (tiles == 0 || check) return hipSuccess;
  along_kernel<C, KIND, ACT><<<static_cast<int>((tiles + 7) / 8 * 8), C::NT, 0, stream>>>(a);
  return hipGetLastError();
}

template <bool F8, int KIND, int ACT>
hipError_t launch_along_kind(const AlongArgs& a, hipStream_t stream, bool check) {
  if (a.rows_max <= static_cast<int64_t>(a.rows.E) * 32)
    return launch_along_as<Core<128, 32, 4, 1, false, false, F8, 4>, KIND, ACT>(a, stream, check);
  return launch_along_as<Core<256, 256, 2, 4, false, false, F8, 2>, KIND, ACT>(a, stream, check);
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

hipError_t launch_row_grad(const RowGradArgs& g, hipStream_t stream, bool check) {
  using C = Core<256, 256, 2, 4, true, false, false, 2>;
  const int64_t tiles = row_tiles<C::BB>(g.rows, g.rows_max, g.per_expert_max) * ((g.N + C::BA - 1) / C::BA);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (tiles == 0 || check) return hipSuccess;
  row_grad_kernel<C><<<static_cast<int>((tiles + 7) / 8 * 8), C::NT, 0, stream>>>(g);
  return hipGetLastError();
}

hipError_t launch_weight_grad(const WeightGradArgs& g, bool f32, hipStream_t stream, bool check) {
  using C = Core<256, 256, 2, 4, true, true, false, 2>;
  const int64_t tiles = static_cast<int64_t>(g.rows.E) * g.parts * ((g.H + C::BA - 1) / C::BA) *
                        ((g.I + C::BB - 1) / C::BB);
  if (tiles > kMaxBlocks) return hipErrorInvalidConfiguration;
  if (check) return hipSuccess;
  const int blocks = static_cast<int>((tiles + 7) / 8 * 8);
  if (f32) weight_grad_kernel<C, true><<<blocks, C::NT, 0, stream>>>(g);
  else weight_grad_kernel<C, false><<<blocks, C::NT, 0, stream>>>(g);
  return hipGetLastError();
}

}  // namespace expert
}  // namespace ep
