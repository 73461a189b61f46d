// The norms around the block, fused with its gate and the residual stream: what stands between a
// combine and the next router.  One pass over the rows; every sum in fp32.
#include <algorithm>

#include "ep_internal.h"

namespace ep {
namespace norm {
namespace {

constexpr int kMaxThreads = 1024;

enum Gate { kNone, kChannel, kToken };

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xf, false));
}
// The sum over a wave, in lane 63: pairs, quads, halves and whole rows of 16 lanes, then the rows.
__device__ __forceinline__ float add_wave(float v) {
  v = add_dpp<0xb1, 0xf>(v);    // lanes 1 0 3 2 of each quad
  v = add_dpp<0x4e, 0xf>(v);    // lanes 2 3 0 1
  v = add_dpp<0x141, 0xf>(v);   // half rows mirrored
  v = add_dpp<0x140, 0xf>(v);   // rows mirrored
  v = add_dpp<0x142, 0xa>(v);   // each row's last lane to the next row
  return add_dpp<0x143, 0xc>(v);   // lane 31 to the upper rows
}

// Sums over the workgroup's waves, in a fixed order.  Consecutive calls take turns between two buffers: a wave
// that writes one again has passed the barrier of the call between, before which all waves have read it.
struct BlockSum {
  float (*part)[3 * 16];
  int turn = 0;

  // once per workgroup: entries of waves that it does not have stay zeros
  __device__ __forceinline__ BlockSum(float (*p)[3 * 16]) : part(p) {
    for (int i = threadIdx.x; i < 2 * 3 * 16; i += blockDim.x) part[i / 48][i % 48] = 0.0f;
    __syncthreads();
  }
  template <int N>
  __device__ __forceinline__ void add(float (&v)[N]) {
    float* p = part[turn];
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = add_wave(v[i]);
      if (lane_id() == 63) p[i * 16 + (threadIdx.x >> 6)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4* q = reinterpret_cast<const float4*>(p + i * 16);
      const float4 a = q[0], b = q[1], c = q[2], d = q[3];
      v[i] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w)) + ((c.x + c.y) + (c.z + c.w)) +
             ((d.x + d.y) + (d.z + d.w));
    }
  }
};

struct V8 {
  float v[8];
};

__device__ __forceinline__ float lo(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }
__device__ __forceinline__ V8 unpack(uint4 u) {
  return {{lo(u.x), hi(u.x), lo(u.y), hi(u.y), lo(u.z), hi(u.z), lo(u.w), hi(u.w)}};
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const uint32_t l = __builtin_bit_cast(uint16_t, static_cast<__bf16>(a));
  return l | static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}
__device__ __forceinline__ uint4 pack(const V8& a) {
  return {pack2(a.v[0], a.v[1]), pack2(a.v[2], a.v[3]), pack2(a.v[4], a.v[5]), pack2(a.v[6], a.v[7])};
}
// (written in place instead, the backward pass's loads ahead are waited for early: 94 us instead of 84)
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ V8 load8(const uint16_t* p) { return unpack(load16(p)); }
// eight weights from column c, F32 or BF16
__device__ __forceinline__ V8 weights8(const void* w, bool f32, int c) {
  if (!f32) return load8(static_cast<const uint16_t*>(w) + c);
  const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c);
  const float4 a = p[0], b = p[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(float* p, const V8& a) {
  reinterpret_cast<float4*>(p)[0] = {a.v[0], a.v[1], a.v[2], a.v[3]};
  reinterpret_cast<float4*>(p)[1] = {a.v[4], a.v[5], a.v[6], a.v[7]};
}

// Streaming accesses: a row is read once and its results are not read again here.
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
__device__ __forceinline__ V8 load8_once(const uint16_t* p) {
  const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return unpack({u.x, u.y, u.z, u.w});
}
__device__ __forceinline__ void store8_once(uint16_t* p, uint4 u) {
  __builtin_nontemporal_store(u32x4{u.x, u.y, u.z, u.w}, reinterpret_cast<u32x4*>(p));
}

// x' = a x + b gate y w_post / rms(y), n = x' w_pre / rms(x'), rms(v) = sqrt(mean v^2 + eps).
// One workgroup a row, CPT pieces of 8 columns a thread: a row is read once, both norms' sums are formed
// from registers.  Bound by memory: 2 reads and 2 writes a value; the two sums wait for one another, which
// other rows' workgroups on the CU cover.  16384 x 7168 with a channel gate: 183 us, 5.13 TB/s (a copy of that
// size: 4.9); plain stores 188, plain loads and stores 191.  128 rows of 7168: 4 us in a graph, the launch and two
// round trips to memory.
template <int CPT, bool POST, int GATE>
__global__ __launch_bounds__(kMaxThreads) void residual_norm_kernel(NormArgs a) {
  __shared__ __attribute__((aligned(16))) float part[2][3 * 16];
  BlockSum sum(part);
  const int64_t r = blockIdx.x;
  V8 y[CPT], x[CPT];
  float ss[1] = {0.0f};
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    const bool in = c < a.H;
    y[p] = in ? load8_once(a.y + r * a.ld_y + c) : V8{};
    x[p] = in ? load8_once(a.x + r * a.ld_x + c) : V8{};
  }
  float ry = 1.0f;
  if constexpr (POST) {
#pragma unroll
    for (int p = 0; p < CPT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] += y[p].v[i] * y[p].v[i];
    sum.add<1>(ss);
    ry = 1.0f / sqrtf(ss[0] / a.H + a.eps);
    ss[0] = 0.0f;
  }
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    if (c >= a.H) continue;
    V8 w, g;
    if constexpr (POST) w = weights8(a.w_post, a.post_f32, c);
    if constexpr (GATE != kNone) g = load8(a.gate + (GATE == kToken ? r * a.ld_gate : 0) + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float t = y[p].v[i];
      if constexpr (POST) t = t * ry * w.v[i];
      if constexpr (GATE != kNone) t *= g.v[i];
      x[p].v[i] = a.a * x[p].v[i] + a.b * t;
    }
    const uint4 u = pack(x[p]);
    store8_once(a.out_x + r * a.ld_out_x + c, u);
    // the next norm reads the stream as it is kept, so that the backward pass, which is given the stream,
    // differentiates at the same values
    x[p] = unpack(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] += x[p].v[i] * x[p].v[i];
  }
  sum.add<1>(ss);
  const float rx = 1.0f / sqrtf(ss[0] / a.H + a.eps);
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    if (c >= a.H) continue;
    const V8 w = weights8(a.w_pre, a.pre_f32, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[p].v[i] = x[p].v[i] * rx * w.v[i];
    store8_once(a.out_n + r * a.ld_out_n + c, pack(x[p]));
  }
}

// With xh = x r, r = (mean x^2 + eps)^-1/2 and v = g_norm w_pre:
//   d = g_res + r (v - xh mean(v xh));  residual: a d;  gate: b d t;
//   y: with q = b gate d w_post, yh = y ry: ry (q - yh mean(q yh)); without a post norm b gate d itself.
// Column sums: w_pre of g_norm xh; and one more, of s = b d yh (yh = y without a post norm; times a token's
// gate): w_post's is gate times it, a channel gate's is w_post times it.
// A workgroup takes rows blockIdx, blockIdx + blocks, ... and keeps the weights and its share of the column
// sums in registers, of which 1024 threads have 128 each; the workgroups' shares are added in order by
// sum_columns_kernel.  What a row waits for is the loads and two sums over the workgroup, one after the other: the
// next row's loads are started first.
// 4096 x 7168 with a channel gate: 84 us with the column sums, 4.2 TB/s of 352 MB (this kernel 72 us, 4.9 TB/s;
// with separate sums for w_post and the gate, wave sums by shuffles and no loads ahead 142 us).
// Streaming stores gain 2.5 us, streaming loads lose 6.
// One piece a thread (up to 8192 columns) keeps all of that in registers but for the token gate with a post norm
// (21 a lane go to scratch: 118 us, 4.0 TB/s at 4096 x 7168).  Two pieces do not: 123 to 139 go to scratch with a post
// norm (4096 x 16384: 400 us, 2.0 TB/s; token gate 580, 1.9), 76 with a channel gate alone (223 us, 3.6 TB/s), 16
// with a token gate alone (209 us, 5.1 TB/s).
template <int CPT, bool POST, int GATE>
__global__ __launch_bounds__(kMaxThreads) void residual_norm_backward_kernel(NormGradArgs a) {
  __shared__ __attribute__((aligned(16))) float part[2][3 * 16];
  BlockSum sum(part);
  constexpr bool Y = POST || GATE != kNone;
  struct Row {
    uint4 x[CPT], g[CPT], r[CPT], y[CPT], t[CPT];
  };
  auto column = [&](int p) { return static_cast<int>(p * blockDim.x + threadIdx.x) * 8; };
  auto load = [&](int64_t r, Row& v) {
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const int c = column(p);
      v.x[p] = v.g[p] = v.r[p] = v.y[p] = v.t[p] = uint4{0, 0, 0, 0};
      if (c >= a.H || r >= a.n) continue;
      v.x[p] = load16(a.x + r * a.ld_x + c);
      v.g[p] = load16(a.g_norm + r * a.ld_g_norm + c);
      if (Y) v.y[p] = load16(a.y + r * a.ld_y + c);
      if (a.g_res) v.r[p] = load16(a.g_res + r * a.ld_g_res + c);
      if (GATE == kToken) v.t[p] = load16(a.gate + r * a.ld_gate + c);
    }
  };
  // scale: b, times a channel's gate, times w_post
  V8 w_pre[CPT] = {}, scale[CPT], s_pre[CPT] = {}, s_two[CPT] = {};
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = column(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) scale[p].v[i] = a.b;
    if (c >= a.H) continue;
    w_pre[p] = weights8(a.w_pre, a.pre_f32, c);
    V8 w, g;
    if constexpr (POST) w = weights8(a.w_post, a.post_f32, c);
    if constexpr (GATE == kChannel) g = load8(a.gate + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (POST) scale[p].v[i] *= w.v[i];
      if constexpr (GATE == kChannel) scale[p].v[i] *= g.v[i];
    }
  }
  const float inv = 1.0f / a.H;
  constexpr bool AHEAD = CPT == 1;   // two pieces a thread leave no registers for another row
  Row now, next;
  if (AHEAD) load(blockIdx.x, now);
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    if constexpr (AHEAD) load(r + gridDim.x, next);
    else load(r, now);
    float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const V8 x = unpack(now.x[p]), g = unpack(now.g[p]), y = unpack(now.y[p]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[0] += x.v[i] * x.v[i];
        v[1] += g.v[i] * w_pre[p].v[i] * x.v[i];
        if constexpr (POST) v[2] += y.v[i] * y.v[i];
      }
    }
    sum.add<3>(v);
    const float rx = 1.0f / sqrtf(v[0] * inv + a.eps);
    const float kx = v[1] * rx * inv * rx * rx;   // r^2 mean(v xh)
    const float ry = POST ? 1.0f / sqrtf(v[2] * inv + a.eps) : 1.0f;
    float m[1] = {0.0f};
    V8 q[CPT];
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const V8 x = unpack(now.x[p]), g = unpack(now.g[p]), y = unpack(now.y[p]), gr = unpack(now.r[p]);
      const V8 gt = unpack(now.t[p]);
      V8 dx, dg;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = gr.v[i] + rx * (g.v[i] * w_pre[p].v[i]) - kx * x.v[i];
        s_pre[p].v[i] += g.v[i] * x.v[i] * rx;
        dx.v[i] = a.a * d;
        q[p].v[i] = d * scale[p].v[i];
        const float yh = POST ? y.v[i] * ry : y.v[i];
        if constexpr (GATE == kToken) {
          dg.v[i] = q[p].v[i] * yh;
          q[p].v[i] *= gt.v[i];
        }
        if constexpr (Y && (POST || GATE == kChannel)) {
          const float e = a.b * d * (GATE == kToken ? gt.v[i] : 1.0f);
          s_two[p].v[i] += e * yh;
        }
        if constexpr (POST) m[0] += q[p].v[i] * yh;
      }
      const int c = column(p);
      if (c >= a.H) continue;
      store8_once(a.dres + r * a.ld_dres + c, pack(dx));
      if constexpr (GATE == kToken) {
        if (a.dgate_token) store8_once(a.dgate_token + r * a.ld_dgate + c, pack(dg));
      }
    }
    if constexpr (POST) sum.add<1>(m);
    const float ky = m[0] * inv * ry * ry;
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const int c = column(p);
      if (c >= a.H) continue;
      if constexpr (POST) {
        const V8 y = unpack(now.y[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[p].v[i] = ry * q[p].v[i] - ky * y.v[i];
      }
      store8_once(a.dy + r * a.ld_dy + c, pack(q[p]));
    }
    if constexpr (AHEAD) now = next;
  }
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = column(p);
    if (c >= a.H) continue;
    float* at = a.work + static_cast<int64_t>(blockIdx.x) * a.H + c;
    store8(at, s_pre[p]);
    if (POST || GATE == kChannel) store8(at + static_cast<int64_t>(gridDim.x) * a.H, s_two[p]);
  }
}

__device__ __forceinline__ float weight_at(const void* w, bool f32, int c) {
  return f32 ? static_cast<const float*>(w)[c] : lo(static_cast<const uint16_t*>(w)[c]);
}

// Column sums of the workgroups' shares: 64 columns a workgroup, 16 threads a column.  blockIdx.y 0: w_pre's;
// 1: the second sum, of which w_post's and a channel gate's are multiples.  The order is fixed, so the sums are the
// same bits every time.  256 x 2 x 7168: 7 us, 15 MB of reads and the launch.
__global__ __launch_bounds__(1024) void sum_columns_kernel(NormGradArgs a, int blocks) {
  __shared__ float part[16][64];
  const int c = blockIdx.x * 64 + lane_id(), q = threadIdx.x >> 6;
  const float* w = a.work + static_cast<int64_t>(blockIdx.y) * blocks * a.H;
  float s = 0.0f;
  if (c < a.H)
    for (int b = q; b < blocks; b += 16) s += w[static_cast<int64_t>(b) * a.H + c];
  part[q][lane_id()] = s;
  __syncthreads();
  if (q != 0 || c >= a.H) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += part[i][lane_id()];
  if (blockIdx.y == 0) {
    a.dw_pre[c] = s;
    return;
  }
  const bool channel = a.gate && !a.gate_rows;
  if (a.dw_post) a.dw_post[c] = channel ? s * lo(a.gate[c]) : s;
  if (a.dgate_channel) a.dgate_channel[c] = a.w_post ? s * weight_at(a.w_post, a.post_f32, c) : s;
}

inline int pieces(int H) { return H / 8 > kMaxThreads ? 2 : 1; }
inline int threads(int H) { return ((H / 8 + pieces(H) - 1) / pieces(H) + 63) / 64 * 64; }

template <int CPT, bool POST>
void run_forward(const NormArgs& a, int gate, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.n)), block(threads(a.H));
  if (gate == kNone) residual_norm_kernel<CPT, POST, kNone><<<grid, block, 0, s>>>(a);
  else if (gate == kChannel) residual_norm_kernel<CPT, POST, kChannel><<<grid, block, 0, s>>>(a);
  else residual_norm_kernel<CPT, POST, kToken><<<grid, block, 0, s>>>(a);
}

template <int CPT, bool POST>
void run_backward(const NormGradArgs& a, int gate, int blocks, hipStream_t s) {
  const dim3 grid(blocks), block(threads(a.H));
  if (gate == kNone) residual_norm_backward_kernel<CPT, POST, kNone><<<grid, block, 0, s>>>(a);
  else if (gate == kChannel) residual_norm_backward_kernel<CPT, POST, kChannel><<<grid, block, 0, s>>>(a);
  else residual_norm_backward_kernel<CPT, POST, kToken><<<grid, block, 0, s>>>(a);
}

}  // namespace

// One workgroup per CU when it fills one (16 waves at 128 registers); of smaller ones as many as fit, while
// each has eight rows for its share of the column sums (4096 x 7168: 256 workgroups).
int grad_blocks(int64_t n, int H) {
  const int64_t fit = kNormCus * std::max(1, 16 / (threads(H) / 64));
  return static_cast<int>(std::min(n, std::max<int64_t>(kNormCus, std::min(fit, n / 8))));
}

// One workgroup a row: more rows than a grid holds take several launches.
hipError_t launch_residual_norm(const NormArgs& args, hipStream_t s) {
  const int gate = !args.gate ? kNone : args.gate_rows ? kToken : kChannel;
  NormArgs a = args;
  for (int64_t left = args.n; left > 0; left -= a.n) {
    a.n = grid_blocks(left, threads(a.H));
    if (pieces(a.H) == 1) a.w_post ? run_forward<1, true>(a, gate, s) : run_forward<1, false>(a, gate, s);
    else a.w_post ? run_forward<2, true>(a, gate, s) : run_forward<2, false>(a, gate, s);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    a.y += a.n * a.ld_y;
    a.x += a.n * a.ld_x;
    if (gate == kToken) a.gate += a.n * a.ld_gate;
    a.out_x += a.n * a.ld_out_x;
    a.out_n += a.n * a.ld_out_n;
  }
  return hipSuccess;
}

hipError_t launch_residual_norm_backward(const NormGradArgs& a, hipStream_t s) {
  const int gate = !a.gate ? kNone : a.gate_rows ? kToken : kChannel, blocks = grad_blocks(a.n, a.H);
  if (blocks > 0) {
    if (pieces(a.H) == 1)
      a.w_post ? run_backward<1, true>(a, gate, blocks, s) : run_backward<1, false>(a, gate, blocks, s);
    else
      a.w_post ? run_backward<2, true>(a, gate, blocks, s) : run_backward<2, false>(a, gate, blocks, s);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const int sums = a.dw_post || a.dgate_channel ? 2 : 1;
  sum_columns_kernel<<<dim3((a.H + 63) / 64, sums), 1024, 0, s>>>(a, blocks);
  return hipGetLastError();
}

}  // namespace norm
}  // namespace ep
