// Between the ranks' stage-2 rows and rows in expert order: what a rank does with its received rows before and
// behind its experts when a token comes to it once (per-rank stage 2), and the adjoints.
//
// Entry k of token i has a row of its rank, row(i,k), which entries on the same rank share, and a place in expert
// order, place(i,k), of its own; both were worked out with the handle.
//   sort:             S[place(i,k)] = X[row(i,k)]
//   unsort:           P[r] = bf16_rne(fma chain in k order from +0 of w[i,k] Y[place(i,k)]) over the entries on r
//   sort, backward:   the same with unit weights
//   the adjoint of adding the ranks' rows up per token: the sort with the token as row, the rank's row as place
//   unsort, backward: dY[place(i,k)] = bf16_rne(w[i,k] dP[row(i,k)]), dw[i,k] = <dP[row(i,k)], Y[place(i,k)]>
//
// All move rows and compute next to nothing, so the memory bounds them (a copy of 2 GiB: 4.87 TB/s of reads and
// writes).  Work is split by token: a token's entries hold all that its rows need, so a sum needs no atomics.  A lane
// owns 16 bytes of a row and starts the loads of all of a token's entries before it uses the first.  Rows and places
// of a token are the same for all lanes (scalar loads), and so are the branches on them.
// 4096 tokens of 8 of 256 experts on 64 ranks, hidden 7168, 30714 rows of ranks (bytes that have to move):
//   sort, FP8 rows     96.5 us, 4.86 TB/s      unsort                      174 us, 5.22 TB/s
//   sort, backward    700 us, 5.20 TB/s (16384 tokens)     unsort, backward   279 us, 4.95 TB/s
// 128 tokens: unsort 7.7 us, 3.7 TB/s; the smallest sort (128 tokens, 512-byte rows) 3.0 us, a launch.
#include "ep_internal.h"
#include "ep_wave_dev.h"

namespace ep {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kBatch = 8;   // entries whose loads are started before the first is used

__device__ __forceinline__ u32x4 load16(const void* p) {
  return __builtin_nontemporal_load(static_cast<const u32x4*>(p));
}
__device__ __forceinline__ void store16(u32x4 v, void* p) { __builtin_nontemporal_store(v, static_cast<u32x4*>(p)); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(lo)) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(hi))) << 16;
}
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = __uint_as_float(v[q] << 16);
    f[2 * q + 1] = __uint_as_float(v[q] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
  return {bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]), bf16x2(f[6], f[7])};
}

// Up to kBatch entries of a token from k0 on: row and place, -1 where there is none or the tensors do not hold it.
// Not MAPPED: a token's one row.
template <bool MAPPED = true>
struct Entries {
  int32_t row[kBatch], place[kBatch];
  bool beyond = false;
  __device__ __forceinline__ Entries(const int32_t* rows, const int32_t* places, int64_t i, int K, int k0, int64_t rows_max,
                                     int64_t places_max) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const bool in = k0 + b < K;
      row[b] = !in ? -1 : MAPPED ? rows[i * K + k0 + b] : static_cast<int32_t>(i);
      place[b] = in ? places[i * K + k0 + b] : -1;
      beyond |= row[b] >= rows_max || place[b] >= places_max;
      if (row[b] >= rows_max) row[b] = -1;
      if (place[b] >= places_max) place[b] = -1;
    }
  }
  __device__ __forceinline__ bool on(int b) const { return row[b] >= 0 && place[b] >= 0; }
  // Bits q > b of the entries that share b's row.
  __device__ __forceinline__ uint32_t behind(int b) const {
    uint32_t m = 0;
#pragma unroll
    for (int q = b + 1; q < kBatch; ++q) m |= row[q] == row[b] ? 1u << q : 0u;
    return m;
  }
};

// Every entry loads its row itself: entries of a token that share one meet in the cache (loading it once for all of
// them took the branches' 51 spilled scalars: the smallest sort 3.45 us, so 3.0).
template <bool MAPPED>
__global__ __launch_bounds__(256) void sort_kernel(SortArgs a) {
  const int at = (blockIdx.x * blockDim.x + threadIdx.x) * 16;
  const int end = a.bytes + a.pad;
  const bool whole = at + 16 <= a.bytes;
  const int words = (end - at) >> 2;      // 4-byte words that this lane writes, four at most
  for (int64_t i = blockIdx.y; i < a.n; i += gridDim.y) {
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
      const Entries<MAPPED> t(a.row, a.place, i, a.K, k0, a.rows_x, a.rows_out);
      if (t.beyond && at == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
      u32x4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!t.on(b) || words <= 0) continue;
        const uint8_t* p = a.x + t.row[b] * a.ld_x + at;
        if (whole) {
          v[b] = load16(p);
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[b][q] = at + 4 * q < a.bytes ? reinterpret_cast<const uint32_t*>(p)[q] : 0;
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (!t.on(b) || words <= 0) continue;
        uint8_t* p = a.out + t.place[b] * a.ld_out + at;
        if (words >= 4) {
          store16(v[b], p);
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (j < words) reinterpret_cast<uint32_t*>(p)[j] = v[b][j];
        }
      }
    }
  }
}

// FEW: K <= kBatch, and all of a token's rows are loaded before the first sum.  Else the entries are taken row by
// row, kBatch loads at a time.
template <bool FEW>
__global__ __launch_bounds__(256) void unsort_kernel(UnsortArgs a) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  const bool active = c < a.H / 8;
  auto add = [&](float (&acc)[8], u32x4 v, float w) {
    float f[8];
    unpack(v, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(w, f[q], acc[q]);
  };
  for (int64_t i = blockIdx.y; i < a.n; i += gridDim.y) {
    if constexpr (FEW) {
      const Entries<> t(a.row, a.place, i, a.K, 0, a.rows_out, a.rows_y);
      if (t.beyond && c == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
      u32x4 v[kBatch];
      float w[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        w[b] = b < a.K ? (a.w ? a.w[i * a.K + b] : 1.0f) : 0.0f;
        if (t.place[b] >= 0 && active) v[b] = load16(a.y + t.place[b] * a.ld_y + 8 * c);
      }
      uint32_t done = 0;   // entries whose row has been written
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (t.row[b] < 0 || (done >> b & 1)) continue;
        const uint32_t more = t.behind(b);
        done |= more;
        float acc[8] = {};
        if (t.place[b] >= 0) add(acc, v[b], w[b]);
        if (more) {
#pragma unroll
          for (int q = b + 1; q < kBatch; ++q)
            if ((more >> q & 1) && t.place[q] >= 0) add(acc, v[q], w[q]);
        }
        if (active) store16(pack(acc), a.out + t.row[b] * a.ld_out + 8 * c);
      }
    } else {
      uint32_t left = 0;   // entries whose row is still to come
      for (int k = 0; k < a.K; ++k) left |= a.row[i * a.K + k] >= 0 ? 1u << k : 0u;
      while (left) {
        const int32_t r = a.row[i * a.K + __builtin_ctz(left)];
        const bool out_in = r < a.rows_out;
        if (!out_in && c == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
        float acc[8] = {};
        uint32_t mine = 0;   // the entries on r
        for (int k = __builtin_ctz(left); k < a.K; ++k) mine |= a.row[i * a.K + k] == r ? 1u << k : 0u;
        left &= ~mine;
        while (mine) {
          u32x4 v[kBatch];
          float w[kBatch];
          bool on[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int k = mine ? __builtin_ctz(mine) : 0;
            const int32_t p = mine ? a.place[i * a.K + k] : -1;
            on[b] = p >= 0 && p < a.rows_y;
            if (p >= a.rows_y && c == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
            w[b] = a.w ? a.w[i * a.K + k] : 1.0f;
            if (on[b] && active) v[b] = load16(a.y + p * a.ld_y + 8 * c);
            mine &= mine - 1;
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
            if (on[b]) add(acc, v[b], w[b]);
        }
        if (active && out_in) store16(pack(acc), a.out + r * a.ld_out + 8 * c);
      }
    }
  }
}

// One workgroup a token, which sums the dot products over its threads' chunks in a fixed order: per-thread fp32
// fma chains, a tree over the lanes, the waves in turn.  An entry loads its gradient row itself; a row read once for
// all entries on it, the entries' branches nested in its own, left the loads waiting for each other: 376 us for the
// 4096 tokens above, 280 so.  Half as many entries at a time take 69 registers instead of 109, and the same time.
// With the lanes' sums by shuffles 1000 tokens of 6 entries on 4 ranks, hidden 2048, take 15.8 us, so 14.8.
__global__ __launch_bounds__(512) void unsort_backward_kernel(UnsortBwdArgs a) {
  __shared__ float part[kBatch][8];
  const int C = a.H / 8;
  const int lane = threadIdx.x & 63, at = threadIdx.x >> 6, waves = blockDim.x >> 6;
  for (int64_t i = blockIdx.x; i < a.n; i += gridDim.x) {
    for (int k0 = 0; k0 < a.K; k0 += kBatch) {
      const Entries<> t(a.row, a.place, i, a.K, k0, a.rows_g, a.rows_y);
      if (t.beyond && threadIdx.x == 0) atomicOr(a.err, EP_DEVERR_ROW_RANGE);
      float w[kBatch], dot[kBatch] = {};
#pragma unroll
      for (int b = 0; b < kBatch; ++b) w[b] = k0 + b < a.K ? a.w[i * a.K + k0 + b] : 0.0f;
      for (int c = threadIdx.x; c < C; c += blockDim.x) {
        u32x4 g[kBatch], y[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          g[b] = t.on(b) ? *reinterpret_cast<const u32x4*>(a.g + t.row[b] * a.ld_g + 8 * c) : u32x4{0, 0, 0, 0};
          y[b] = a.y && t.on(b) ? load16(a.y + t.place[b] * a.ld_y + 8 * c) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (!t.on(b)) continue;
          float f[8], o[8], z[8];
          unpack(g[b], f);
          unpack(y[b], z);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = w[b] * f[j];
          store16(pack(o), a.dy + t.place[b] * a.ld_dy + 8 * c);
#pragma unroll
          for (int j = 0; j < 8; ++j) dot[b] = __builtin_fmaf(f[j], z[j], dot[b]);
        }
      }
      if (a.dw) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (k0 + b >= a.K) continue;
          const float v = wave::add_wave(dot[b]);
          if (lane == 63) part[b][at] = v;
        }
        __syncthreads();
        const int k = k0 + threadIdx.x;
        if (threadIdx.x < kBatch && k < a.K) {
          float sum = 0.0f;   // of an entry without a row or beyond the tensors: nothing was added
          for (int q = 0; q < waves; ++q) sum += part[threadIdx.x][q];
          a.dw[i * a.K + k] = sum;
        }
        __syncthreads();
      }
    }
  }
}

// Threads of a workgroup for rows of C 16-byte chunks, `most` at most: the largest number of waves that the chunks
// fill whole, or as many waves as they need.
int threads_for(int C, int most) {
  for (int t = most; t >= 128; t -= 64)
    if (C % t == 0) return t;
  return C >= most ? most : (C + 63) / 64 * 64;
}

// Column blocks and tokens; with a cap on the blocks, fewer tokens at a time.
dim3 grid_for(int64_t n, int cols, int max_blocks) {
  int64_t rows = n;
  if (max_blocks > 0) rows = rows < max_blocks / cols ? rows : max_blocks / cols > 0 ? max_blocks / cols : 1;
  return dim3(static_cast<unsigned>(cols), static_cast<unsigned>(rows < 65535 ? rows : 65535));
}

}  // namespace

hipError_t launch_sort(const SortArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const int C = (a.bytes + a.pad + 15) / 16, threads = threads_for(C, 256);
  const dim3 grid = grid_for(a.n, (C + threads - 1) / threads, a.max_blocks);
  if (a.row) sort_kernel<true><<<grid, threads, 0, stream>>>(a);
  else sort_kernel<false><<<grid, threads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_unsort(const UnsortArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const int C = a.H / 8, threads = threads_for(C, 256);
  const dim3 grid = grid_for(a.n, (C + threads - 1) / threads, a.max_blocks);
  if (a.K <= kBatch) unsort_kernel<true><<<grid, threads, 0, stream>>>(a);
  else unsort_kernel<false><<<grid, threads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_unsort_backward(const UnsortBwdArgs& a, hipStream_t stream) {
  if (a.n == 0) return hipSuccess;
  const int threads = threads_for(a.H / 8, 512);
  int64_t blocks = a.n;
  if (a.max_blocks > 0 && blocks > a.max_blocks) blocks = a.max_blocks;
  const dim3 grid(grid_blocks(blocks, threads));
  unsort_backward_kernel<<<grid, threads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace ep
