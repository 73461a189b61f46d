// The norms around the block, fused with its gate and the residual stream: what stands between a
// combine and the next router.  One pass over the rows; every sum in fp32.
#include "ep_internal.h"

namespace ep {
namespace norm {
namespace {

constexpr int kMaxThreads = 1024;

enum Gate { kNone, kChannel, kToken };

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// Sums of N values over the workgroup, in a fixed order; all threads get them.  `part` holds 16 N floats
// and is free again once every thread has passed the second barrier of the next call.
template <int N>
__device__ __forceinline__ void sum_block(float (&v)[N], float* part) {
  const int w = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v[i] += __shfl_xor(v[i], d);
    if (lane_id() == 0) part[i * 16 + w] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = 0.0f;
    for (int q = 0; q < waves; ++q) s += part[i * 16 + q];
    v[i] = s;
  }
  __syncthreads();
}

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
__device__ __forceinline__ V8 load8(const uint16_t* p) { return unpack(*reinterpret_cast<const uint4*>(p)); }
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

// One workgroup a row, CPT pieces of 8 columns a thread: a row is read once, both norms' sums are formed
// from registers.
template <int CPT, bool POST, int GATE>
__global__ void residual_norm_kernel(NormArgs a) {
  __shared__ float part[16];
  const int64_t r = blockIdx.x;
  V8 y[CPT], x[CPT];
  float ss[1] = {0.0f};
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    const bool in = c < a.H;
    y[p] = in ? load8(a.y + r * a.ld_y + c) : V8{};
    x[p] = in ? load8(a.x + r * a.ld_x + c) : V8{};
  }
  float ry = 1.0f;
  if constexpr (POST) {
#pragma unroll
    for (int p = 0; p < CPT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] += y[p].v[i] * y[p].v[i];
    sum_block<1>(ss, part);
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
    *reinterpret_cast<uint4*>(a.out_x + r * a.ld_out_x + c) = u;
    // the next norm reads the stream as it is kept, so that the backward pass, which is given the stream,
    // differentiates at the same values
    x[p] = unpack(u);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss[0] += x[p].v[i] * x[p].v[i];
  }
  sum_block<1>(ss, part);
  const float rx = 1.0f / sqrtf(ss[0] / a.H + a.eps);
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    if (c >= a.H) continue;
    const V8 w = weights8(a.w_pre, a.pre_f32, c);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[p].v[i] = x[p].v[i] * rx * w.v[i];
    *reinterpret_cast<uint4*>(a.out_n + r * a.ld_out_n + c) = pack(x[p]);
  }
}

// With xh = x r, r = (mean x^2 + eps)^-1/2 and v = g_norm w_pre:
//   dx = g_res + r (v - xh mean(v xh));  residual: a dx;  dt = b gate dx;  gate: b dx t;
//   y: with q = dt w_post, yh = y ry: ry (q - yh mean(q yh)); without a post norm dt itself.
// A workgroup takes rows blockIdx, blockIdx + blocks, ... and keeps its share of the column sums in
// registers; the workgroups' shares are added in order by sum_columns_kernel.
template <int CPT, bool POST, int GATE>
__global__ void residual_norm_backward_kernel(NormGradArgs a) {
  __shared__ float part[3 * 16];
  V8 s_pre[CPT] = {}, s_post[CPT] = {}, s_gate[CPT] = {};
  const float inv = 1.0f / a.H;
  for (int64_t r = blockIdx.x; r < a.n; r += gridDim.x) {
    V8 x[CPT], g[CPT], y[CPT];
    float v[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const int c = (p * blockDim.x + threadIdx.x) * 8;
      const bool in = c < a.H;
      x[p] = in ? load8(a.x + r * a.ld_x + c) : V8{};
      g[p] = in ? load8(a.g_norm + r * a.ld_g_norm + c) : V8{};
      if (POST || GATE != kNone) y[p] = in ? load8(a.y + r * a.ld_y + c) : V8{};
      const V8 w = in ? weights8(a.w_pre, a.pre_f32, c) : V8{};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[0] += x[p].v[i] * x[p].v[i];
        v[1] += g[p].v[i] * w.v[i] * x[p].v[i];
        if constexpr (POST) v[2] += y[p].v[i] * y[p].v[i];
      }
    }
    sum_block<3>(v, part);
    const float rx = 1.0f / sqrtf(v[0] * inv + a.eps);
    const float mx = v[1] * rx * inv;   // mean of v xh
    const float ry = POST ? 1.0f / sqrtf(v[2] * inv + a.eps) : 1.0f;
    float q[1] = {0.0f};
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const int c = (p * blockDim.x + threadIdx.x) * 8;
      if (c >= a.H) continue;
      const V8 w = weights8(a.w_pre, a.pre_f32, c);
      V8 gr{}, wp, gt, dx, dg;
      if (a.g_res) gr = load8(a.g_res + r * a.ld_g_res + c);
      if constexpr (POST) wp = weights8(a.w_post, a.post_f32, c);
      if constexpr (GATE != kNone) gt = load8(a.gate + (GATE == kToken ? r * a.ld_gate : 0) + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xh = x[p].v[i] * rx, yh = POST ? y[p].v[i] * ry : 0.0f;
        const float d = gr.v[i] + rx * (g[p].v[i] * w.v[i] - xh * mx);
        s_pre[p].v[i] += g[p].v[i] * xh;
        dx.v[i] = a.a * d;
        float dt = a.b * d;
        if constexpr (GATE != kNone) {
          const float t = POST ? yh * wp.v[i] : y[p].v[i];
          dg.v[i] = dt * t;
          if constexpr (GATE == kChannel) s_gate[p].v[i] += dg.v[i];
          dt *= gt.v[i];
        }
        if constexpr (POST) {
          s_post[p].v[i] += dt * yh;
          dt *= wp.v[i];
          q[0] += dt * yh;
        }
        g[p].v[i] = dt;
      }
      *reinterpret_cast<uint4*>(a.dres + r * a.ld_dres + c) = pack(dx);
      if constexpr (GATE == kToken) {
        if (a.dgate_token) *reinterpret_cast<uint4*>(a.dgate_token + r * a.ld_dgate + c) = pack(dg);
      }
    }
    float my = 0.0f;
    if constexpr (POST) {
      sum_block<1>(q, part);
      my = q[0] * inv;
    }
#pragma unroll
    for (int p = 0; p < CPT; ++p) {
      const int c = (p * blockDim.x + threadIdx.x) * 8;
      if (c >= a.H) continue;
      V8 dy;
#pragma unroll
      for (int i = 0; i < 8; ++i) dy.v[i] = POST ? ry * (g[p].v[i] - y[p].v[i] * ry * my) : g[p].v[i];
      *reinterpret_cast<uint4*>(a.dy + r * a.ld_dy + c) = pack(dy);
    }
  }
#pragma unroll
  for (int p = 0; p < CPT; ++p) {
    const int c = (p * blockDim.x + threadIdx.x) * 8;
    if (c >= a.H) continue;
    float* at = a.work + static_cast<int64_t>(blockIdx.x) * a.H + c;
    const int64_t next = static_cast<int64_t>(gridDim.x) * a.H;
    store8(at, s_pre[p]);
    if (POST) store8(at += next, s_post[p]);
    if (GATE == kChannel) store8(at += next, s_gate[p]);
  }
}

// Column sums of `blocks` rows: 64 columns a workgroup, 16 threads a column; blockIdx.y picks the sum.
__global__ __launch_bounds__(1024) void sum_columns_kernel(const float* work, int blocks, int H, float* o0, float* o1,
                                                           float* o2) {
  __shared__ float part[16][64];
  float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
  const int c = blockIdx.x * 64 + lane_id(), q = threadIdx.x >> 6;
  const float* w = work + static_cast<int64_t>(blockIdx.y) * blocks * H;
  float s = 0.0f;
  if (c < H)
    for (int b = q; b < blocks; b += 16) s += w[static_cast<int64_t>(b) * H + c];
  part[q][lane_id()] = s;
  __syncthreads();
  if (q != 0 || c >= H || !out) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) s += part[i][lane_id()];
  out[c] = s;
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

int grad_blocks(int64_t n) { return static_cast<int>(n < kGradBlocks ? n : kGradBlocks); }

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const int gate = !a.gate ? kNone : a.gate_rows ? kToken : kChannel;
  if (pieces(a.H) == 1) a.w_post ? run_forward<1, true>(a, gate, s) : run_forward<1, false>(a, gate, s);
  else a.w_post ? run_forward<2, true>(a, gate, s) : run_forward<2, false>(a, gate, s);
  return hipGetLastError();
}

hipError_t launch_residual_norm_backward(const NormGradArgs& a, hipStream_t s) {
  const int gate = !a.gate ? kNone : a.gate_rows ? kToken : kChannel, blocks = grad_blocks(a.n);
  if (blocks > 0) {
    if (pieces(a.H) == 1)
      a.w_post ? run_backward<1, true>(a, gate, blocks, s) : run_backward<1, false>(a, gate, blocks, s);
    else
      a.w_post ? run_backward<2, true>(a, gate, blocks, s) : run_backward<2, false>(a, gate, blocks, s);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  float* sums[3] = {a.dw_pre, nullptr, nullptr};
  int count = 1;
  if (a.w_post) sums[count++] = a.dw_post;
  if (gate == kChannel) sums[count++] = a.dgate_channel;
  sum_columns_kernel<<<dim3((a.H + 63) / 64, count), 1024, 0, s>>>(a.work, blocks, a.H, sums[0], sums[1], sums[2]);
  return hipGetLastError();
}

}  // namespace norm
}  // namespace ep
