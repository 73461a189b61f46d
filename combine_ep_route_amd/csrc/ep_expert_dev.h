// Device core of the experts' products: LDS-tiled matrix products on the matrix unit, fed by loads
// that go from global memory to LDS without passing registers.
//
// What bounds it: with many rows an expert, the rate at which the matrix unit is fed.  Without a padded row (64
// experts of 7168 x 2048, 512 rows each) the gated bf16 product runs at 1125 TFLOP/s, the linear one at 1040, the
// gradient of the rows at 1145, the FP8 gated product at 1900; plain library products of such sizes at 1440 and
// 2600.  The clock's fall to about 1.6 GHz under the load explains a part: the gated product of zeros, which draws
// less power, runs at 1304.  A wave's 128 x 64 results take 192 operand rows from LDS.
// A workgroup's tile of 256 x 256 takes 32 KiB from the L2 for each 32 contracted bf16 values, half of what tiles of
// 128 x 128 take; the L2 gives a CU 64 bytes a cycle.  With few rows an expert the weights' bytes bound it (6.3 TB/s
// reached of 6.1 to 6.8 for pure reads and writes of large arrays).
// Tried, without gain: five stages of 64 bytes, prefetches three and four steps ahead, 32 x 32 x 16
// instructions, waves of 128 x 128, two workgroups of 256 x 128 a CU, waves' priorities.
//
// A step of the contraction brings one tile of each operand to LDS, whatever its type and direction:
//   "along" operands are contiguous in the contracted index: PIECE bytes of each output row or column
//   (64 bytes: 32 bf16 values; 128: 64 bf16 or 128 FP8 values);
//   "across" operands are contiguous in the output index: PIECE/2 contracted rows of bf16 values.
// Products are formed transposed (weights as the first operand, rows as the second), so that the
// four results a lane holds are four consecutive columns of one output row: 8-byte stores.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ep_internal.h"

namespace ep {
namespace expert {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;


// Loads go through buffer descriptors: 32-bit offsets from a base that all lanes share, and what lies
// outside the descriptor's extent is read as zeros.
constexpr int kOutside = -1;             // an offset outside every extent
constexpr uint32_t kExtent = 0x7fffffffu;   // an extent for offsets that were checked on the host

typedef __amdgpu_buffer_rsrc_t Rsrc;

__device__ __forceinline__ Rsrc rsrc(const uint8_t* base, uint32_t extent) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, static_cast<int>(extent), 0x27000);
}
__device__ __forceinline__ uint32_t extent_of(int64_t bytes) {
  return bytes <= 0 ? 0u : bytes < kExtent ? static_cast<uint32_t>(bytes) : kExtent;
}

// Straight to LDS: lane l's bytes go to l + 16 l (l + 4 l).
__device__ __forceinline__ void load_lds16(Rsrc r, int offset, uint8_t* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, offset, 0, 0, 0);
}
__device__ __forceinline__ void load_lds4(Rsrc r, int offset, uint8_t* l) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 4, offset, 0, 0, 0);
}

// Waits until at most N of this wave's vector loads are in flight and all its LDS reads and writes
// have ended; then all waves meet.  The empty asm statements keep the compiler from moving memory
// accesses over the barrier.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("" ::: "memory");
  // vmcnt: bits 0-3 and 14-15; expcnt (bits 4-6) left at its maximum; lgkmcnt (bits 8-11) 0.
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// ---------------------------------------------------------------------------
// Which rows an expert holds
// ---------------------------------------------------------------------------

// Whether an expert's rows lie in several runs.
__host__ __device__ inline bool scattered(const ExpertRows& r) { return r.list != nullptr || r.sources > 1; }

struct Span {
  int e = -1;             // expert, or -1: none
  int count = 0;          // its rows within the limit
  int all = 0;            // its rows
  int before = 0;         // rows of the experts before it
  int first = 0;          // its first row (without a list)
  int m = 0, n = 0;       // row tile and column tile in it
};

// Inclusive sum over the lanes: shifts by 1, 2, 4 and 8 inside rows of 16, then the rows' last lanes.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int scan64(int v) {
  v = add_dpp<0x111, 0xf>(v);
  v = add_dpp<0x112, 0xf>(v);
  v = add_dpp<0x114, 0xf>(v);
  v = add_dpp<0x118, 0xf>(v);
  v = add_dpp<0x142, 0xa>(v);
  return add_dpp<0x143, 0xc>(v);
}

// Workgroups go to the 8 XCDs in turn: XCD x takes the x-th eighth of the tiles, so that tiles that share
// weights or rows run on one XCD and meet in its L2.
__device__ __forceinline__ int xcd_tile(int block, int total) {
  const int part = (total + 7) >> 3, at = (block & 7) * part + (block >> 3);
  return (block >> 3) < part && at < total ? at : -1;
}

// Every wave scans the counts on its own (E <= 1024: up to 16 consecutive experts a lane).  With BM > 0 the
// workgroup's tile: experts in order, in each the column tiles, in each the row tiles of BM rows.  With
// BM == 0 the span of expert `which`.
template <int BM>
__device__ __forceinline__ Span find_span(const ExpertRows& r, int which, int col_tiles) {
  const int per = (r.E + 63) >> 6, e0 = lane_id() * per;
  int c[16] = {}, rows = 0, tiles = 0;
  auto tiles_of = [](int rows_e) { return BM > 0 ? (rows_e + BM - 1) / (BM > 0 ? BM : 1) : 0; };
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    // all loads at once: what lies outside is read in bounds and counts nothing
    if (i < per) {
      const int32_t* p = r.count + (e0 + i < r.E ? e0 + i : r.E - 1) * r.sources;
      if (r.sources == 1) {
        c[i] = p[0];
      } else {
        int v[kFewSources];
#pragma unroll
        for (int k = 0; k < kFewSources; ++k) v[k] = p[k < r.sources ? k : 0];
#pragma unroll
        for (int k = 0; k < kFewSources; ++k) c[i] += k < r.sources ? v[k] : 0;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    c[i] = i < per && e0 + i < r.E ? c[i] : 0;
    rows += c[i];
    tiles += tiles_of(c[i]);
  }
  const int rows_to = scan64(rows);
  int rows_at = rows_to - rows, tiles_at = 0, tile = 0, q = 0;
  Span s;
  if constexpr (BM > 0) {
    const int tiles_to = scan64(tiles);
    tiles_at = tiles_to - tiles;
    tile = xcd_tile(which, __builtin_amdgcn_readlane(tiles_to, 63) * col_tiles);
    if (tile < 0) return s;
    q = tile / col_tiles;
  }
  int e = -1, count = 0, before = 0, tb = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int t = tiles_of(c[i]);
    if (BM > 0 ? (q >= tiles_at && q < tiles_at + t) : (i < per && e0 + i == which)) {
      e = e0 + i;
      count = c[i];
      before = rows_at;
      tb = tiles_at;
    }
    rows_at += c[i];
    tiles_at += t;
  }
  const uint64_t who = __ballot(e >= 0);
  if (who == 0) return s;
  const int w = __builtin_ctzll(who);
  s.e = __builtin_amdgcn_readlane(e, w);
  s.all = s.count = __builtin_amdgcn_readlane(count, w);
  s.before = __builtin_amdgcn_readlane(before, w);
  s.first = r.stride > 0 ? s.e * r.stride : s.before;
  if constexpr (BM > 0) {
    const int local = tile - __builtin_amdgcn_readlane(tb, w) * col_tiles, t = tiles_of(s.all);
    s.n = local / t;
    s.m = local - s.n * t;
  }
  if (!scattered(r) && s.first + static_cast<int64_t>(s.count) > r.limit)
    s.count = r.limit > s.first ? static_cast<int>(r.limit - s.first) : 0;
  return s;
}

// The row that offsets in a tile from its row m0 on count from.
__device__ __forceinline__ int64_t first_row(const ExpertRows& r, const Span& s, int m0) {
  return scattered(r) ? s.first : s.first + m0;
}
__device__ __forceinline__ int row_of(const ExpertRows& r, const Span& s, int p) {
  if (r.list) return r.list[s.before + p];
  if (r.sources == 1) return s.first + p;
  const int32_t* c = r.count + s.e * r.sources;
  int v[kFewSources], at = s.first;
#pragma unroll
  for (int k = 0; k < kFewSources; ++k) v[k] = c[k < r.sources ? k : 0];
  bool on = true;   // p lies behind the sources so far
#pragma unroll
  for (int k = 0; k + 1 < kFewSources; ++k) {
    on = on && k + 1 < r.sources && p >= v[k];
    p -= on ? v[k] : 0;
    at += on ? r.slots : 0;
  }
  return at + p;
}

// ---------------------------------------------------------------------------
// The product of one tile
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v)));
}
__device__ __forceinline__ uint2 bf16x4(f32x4 v) {
  return {bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
}
__device__ __forceinline__ float from_bf16(uint32_t b) { return __builtin_bit_cast(float, b << 16); }

template <int N>
struct Int {
  static constexpr int value = N;
};

// A plan of one source.
template <class Src>
struct One {
  const Src& src;
  static constexpr int parts() { return 1; }
  __device__ __forceinline__ Src source(int) const { return src; }
};

// BA x BB results from WA x WB waves; ANC / BNC: the operand lies across (else along); F8: E4M3 operands
// with scales (both along); ST: stages of the LDS ring; PIECE: see above.
template <int BA_, int BB_, int WA_, int WB_, bool ANC_, bool BNC_, bool F8_, int ST_, int PIECE_>
struct Core {
  static constexpr int BA = BA_, BB = BB_, WA = WA_, WB = WB_, ST = ST_, PIECE = PIECE_;
  static constexpr bool ANC = ANC_, BNC = BNC_, F8 = F8_;
  static constexpr int NW = WA * WB, NT = NW * 64;
  static constexpr int TA = BA / WA, TB = BB / WB;   // a wave's part
  static constexpr int FA = TA / 16, FB = TB / 16;   // in 16 x 16 fragments
  static constexpr int ROWS = 1024 / PIECE;          // rows of an "along" tile in a 1 KiB load
  static constexpr int KROWS = PIECE / 2;            // contracted rows of a step of an "across" tile
  static constexpr int JA = BA / ROWS / NW, JB = BB / ROWS / NW;   // loads a wave issues per step
  // Scales of a step: the rows' from entry 0, the weights' two at entries WS and WS + 64, each loaded by a
  // wave of its own.
  static constexpr int WS = (BB + 63) / 64 * 64;
  static constexpr int SCALES = F8 ? NT * 4 : 0;
  static constexpr int STAGE = (BA + BB) * PIECE + SCALES;
  static_assert(BA / ROWS % NW == 0 && BB / ROWS % NW == 0, "loads must divide over the waves");
  static_assert(TA % 16 == 0 && TB % 16 == 0, "whole fragments");
  static_assert(PIECE == 64 || PIECE == 128, "32 or 64 contracted bf16 values");
  static_assert(!F8 || (!ANC && !BNC && PIECE == 128 && WS + 128 <= NT), "FP8 operands lie along");
  static_assert(ST >= 2 && ST <= 4 && (JA + JB + 1) * (ST - 1) < 64, "the wait counts at most 63 loads");

  typedef f32x4 Acc[FA][FB];

  static __device__ __forceinline__ uint8_t* stage0() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[STAGE];
    return s;
  }
  static __device__ __forceinline__ uint8_t* stage1() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[STAGE];
    return s;
  }
  static __device__ __forceinline__ uint8_t* stage2() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[ST > 2 ? STAGE : 16];
    return s;
  }
  static __device__ __forceinline__ uint8_t* stage3() {
    __shared__ __attribute__((aligned(1024))) uint8_t s[ST > 3 ? STAGE : 16];
    return s;
  }

  // Where a 16-byte piece of an "along" row lies: rows of 64 or 128 bytes put equal pieces of neighbouring
  // rows on the same banks; the exclusive or spreads the eight rows a read takes at once over all of them.
  static __device__ __forceinline__ int spread(int row) { return PIECE == 128 ? row & 7 : (row >> 1) & 3; }
  // The row, and the piece of it, that this lane loads in a 1 KiB load.
  static __device__ __forceinline__ int along_row() { return lane_id() / (PIECE / 16); }
  static __device__ __forceinline__ int along_piece() { return (lane_id() % (PIECE / 16)) ^ spread(along_row()); }
  // The same for an "across" tile of B columns: contracted row and first column of load g.  32-byte chunks
  // change places by mix(k): the 16 lanes of a transposing read touch four rows k..k+3, its neighbours the
  // rows 8 further on, all at the same chunk.
  static __device__ __forceinline__ int mix(int k) { return (k & 3) | (((k >> 3) & 3) << 2); }
  template <int B>
  static __device__ __forceinline__ int across_row(int g) { return (g * 1024u + lane_id() * 16u) / (B * 2u); }
  template <int B>
  static __device__ __forceinline__ int across_col(int g) {
    const int at = (g * 1024u + lane_id() * 16u) % (B * 2u);
    return ((at >> 5) ^ (mix(across_row<B>(g)) & (B / 16 - 1))) * 16 + ((at >> 4) & 1) * 8;
  }

  // 1 KiB loads of the second operand that NJ fragments of each wave column need, and all loads of a step.
  static constexpr int loads_b(int nj) {
    const int need = (16 * WB * nj + ROWS * NW - 1) / (ROWS * NW);
    return BNC || need > JB ? JB : need;
  }
  static constexpr int loads(int nj) { return JA + loads_b(nj) + (F8 ? 1 : 0); }

  // Load `at` of a step (scales first).  The loads of a step are spread over the products: a burst of them
  // fills the address unit's queue, and a wave that waits there issues no product either.
  template <int NJ, class Src>
  static __device__ __forceinline__ void issue_one(const Src& src, int at, uint8_t* buf) {
    const int w = wave_id();
    if (F8 && at == 0) {
      if constexpr (F8) load_lds4(src.scale_rsrc(), src.scale(), buf + (BA + BB) * PIECE + w * 256);
      return;
    }
    const int j = at - (F8 ? 1 : 0);
    if (j < JA) load_lds16(src.a_rsrc(j), src.a(j), buf + (j * NW + w) * 1024);
    else if (j < JA + loads_b(NJ)) load_lds16(src.b_rsrc(), src.b(j - JA), buf + BA * PIECE + ((j - JA) * NW + w) * 1024);
  }
  template <int NJ, class Src>
  static __device__ __forceinline__ void issue(Src& src, uint8_t* buf) {
    src.step();
#pragma unroll
    for (int i = 0; i < loads(NJ); ++i) issue_one<NJ>(src, i, buf);
  }
  // The part of a step's loads that goes with fragment i of the first operand.
  template <int NJ, class Src>
  static __device__ __forceinline__ void issue_part(const Src& src, int i, uint8_t* buf) {
    constexpr int per = (loads(NJ) + FA - 1) / FA;
#pragma unroll
    for (int k = 0; k < per; ++k)
      if (i * per + k < loads(NJ)) issue_one<NJ>(src, i * per + k, buf);
  }

  // 16 rows or columns from `from` of the step's part s, 8 contracted values a lane: lane group
  // q = l/16 holds k = 32 s + 8 q .. + 7 of row l%16.
  static __device__ __forceinline__ i32x4 along_frag(const uint8_t* t, int from, int s) {
    const int l = lane_id(), r = from + (l & 15);
    return *reinterpret_cast<const i32x4*>(t + r * PIECE + (((s * 4 + (l >> 4)) ^ spread(l & 15)) << 4));
  }
  template <int B>
  static __device__ __forceinline__ i32x4 across_frag(const uint8_t* t, int from, int s) {
    const int l = lane_id(), k = (l >> 4) * 8 + ((l & 15) >> 2);   // mix(k + 32) == mix(k)
    const int at = (k * (B * 2) + ((mix(k) & (B / 16 - 1)) << 5) + (l & 3) * 8) ^ (from << 1);
    const uint8_t* p = t + at + s * 32 * (B * 2);
    typedef __attribute__((address_space(3))) s16x4 lds4;
    union { s16x4 h[2]; i32x4 v; } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * B * 2));
    return u.v;
  }
  static __device__ __forceinline__ i32x4 frag_a(const uint8_t* t, int from, int s) {
    if constexpr (ANC) return across_frag<BA>(t, from, s); else return along_frag(t, from, s);
  }
  static __device__ __forceinline__ i32x4 frag_b(const uint8_t* t, int from, int s) {
    if constexpr (BNC) return across_frag<BB>(t, from, s); else return along_frag(t, from, s);
  }

  // The second operand's 16-row fragments go to the waves in turn, so that a tile with few rows keeps all
  // of them busy: wave column v holds fragments v, v + WB, ...; with NJ of them each, rows from 16 WB NJ on
  // are not multiplied.
  static __device__ __forceinline__ int from_b(int j) { return (j * WB + wave_id() / WA) * 16; }
  // src.frag_a_at(fa, i): first row of the wave's fragment i of the first operand; src.second_scale(fa, i):
  // whether it takes the second of the step's two weight scales (the same for each half of the fragments).

  // One step of E4M3: an instruction contracts the 128 values that share a scale; its result is scaled and
  // added in fp32.  Inside the instruction the matrix unit adds E4M3 products aligned to the largest of them
  // with about 15 bits (2.4e-4 of the largest product at worst in 4096 sums, 1.7e-5 of the result's norm on
  // quantised normal values): far below the bf16 rounding of the output, 2^-8.
  template <int NJ, class Src>
  static __device__ __forceinline__ void compute_fp8(const Src& src, const uint8_t* buf, uint8_t* before, Acc& acc,
                                                     int fa) {
    const uint8_t* ta = buf;
    const uint8_t* tb = buf + BA * PIECE;
    const float* sc = reinterpret_cast<const float*>(buf + (BA + BB) * PIECE);
    const float w0 = sc[WS], w1 = sc[WS + 64];
    i32x8 b[NJ];
    float x[NJ], c[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const i32x4 lo = along_frag(tb, from_b(j), 0), hi = along_frag(tb, from_b(j), 1);
      b[j] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      x[j] = sc[from_b(j) + (lane_id() & 15)];
    }
    i32x4 lo = along_frag(ta, Src::frag_a_at(fa, 0), 0), hi = along_frag(ta, Src::frag_a_at(fa, 0), 1);
    // The sums of a fragment's results follow while the next one's products run.
    f32x4 p[2][NJ];
#pragma unroll
    for (int i = 0; i <= FA; ++i) {
      if (i < FA) {
        const i32x8 a = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        issue_part<NJ>(src, i, before);
        if (i + 1 < FA) {
          lo = along_frag(ta, Src::frag_a_at(fa, i + 1), 0);
          hi = along_frag(ta, Src::frag_a_at(fa, i + 1), 1);
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          p[i & 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b[j], f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
      }
      if (i > 0) {
        if (i - 1 == 0 || i - 1 == FA / 2) {
          const float w = Src::second_scale(fa, i - 1) ? w1 : w0;
#pragma unroll
          for (int j = 0; j < NJ; ++j) c[j] = x[j] * w;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[i - 1][j][k] = __builtin_fmaf(p[(i - 1) & 1][j][k], c[j], acc[i - 1][j][k]);
        // Without these the compiler reads all fragments ahead, puts off all sums and spills them.
#pragma unroll
        for (int j = 0; j < NJ; ++j) asm volatile("" : "+v"(acc[i - 1][j]));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // A step of bf16 that reads all its fragments and then multiplies.
  template <int NJ, class Src>
  static __device__ __forceinline__ void compute(const Src&, const uint8_t* buf, Acc& acc, int fa) {
#pragma unroll
    for (int s = 0; s < PIECE / 64; ++s) {
      i32x4 a[FA], b[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) b[j] = frag_b(buf + BA * PIECE, from_b(j), s);
#pragma unroll
      for (int i = 0; i < FA; ++i) a[i] = frag_a(buf, Src::frag_a_at(fa, i), s);
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[i]),
                                                              __builtin_bit_cast(bf16x8, b[j]), acc[i][j], 0, 0, 0);
    }
  }

  // Ring of ST stages, each an array of its own so that the compiler sees that the loads into one do not
  // touch the others.  At step t: wait for stage t (the loads of ST-2 later steps stay in flight), meet,
  // start the loads of step t+ST-1 into the stage that step t-1 read (every wave has read it: its LDS reads
  // ended before the barrier), multiply.
  template <int NJ, class Src>
  static __device__ __forceinline__ void ring_step(Src& src, uint8_t* cur, uint8_t* before, Acc& acc, int fa) {
    wait_and_meet<loads(NJ) * (ST - 2)>();
    if constexpr (F8) {
      src.step();
      compute_fp8<NJ>(src, cur, before, acc, fa);
    } else {
      issue<NJ>(src, before);
      compute<NJ>(src, cur, acc, fa);
    }
  }

  // The same as a software pipeline over the first operand's fragments (bf16).  While the NJ products of a
  // fragment run, the one after the next is read; with the last two run the reads of the next step's first
  // two and its second operand.  When a stage's last fragment is in registers all waves meet: the next stage
  // is complete, and this one takes the loads of step t+ST, kEarly of them at once and the others with the
  // next step's first fragments.
  static constexpr int kEarly = 4;
  template <int NJ, class Src>
  static __device__ __forceinline__ void piped_step(Src& src, uint8_t* before, uint8_t* cur, uint8_t* next, Acc& acc,
                                                    int fa, i32x4 (&b)[NJ], i32x4 (&a)[2]) {
    constexpr int H = PIECE / 64, N = H * FA;
    i32x4 c[NJ];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = n % FA, s = n / FA, m = n + 2;
      if (kEarly + 2 * n < loads(NJ)) issue_one<NJ>(src, kEarly + 2 * n, before);
      if (kEarly + 2 * n + 1 < loads(NJ)) issue_one<NJ>(src, kEarly + 2 * n + 1, before);
      if (n == N - 2) {
        wait_and_meet<loads(NJ) * (ST - 2)>();
        src.step();
      }
      if (n >= N - 2) {
        const int from = (n - (N - 2)) * 2;
        if (from < loads(NJ) && from < kEarly) issue_one<NJ>(src, from, cur);
        if (from + 1 < loads(NJ) && from + 1 < kEarly) issue_one<NJ>(src, from + 1, cur);
      }
      if (i == FA - 2) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) c[j] = frag_b((s + 1 < H ? cur : next) + BA * PIECE, from_b(j), s + 1 < H ? s + 1 : 0);
      }
      const i32x4 ahead = m < N ? frag_a(cur, Src::frag_a_at(fa, m % FA), m / FA)
                                : frag_a(next, Src::frag_a_at(fa, m - N), 0);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[n & 1]),
                                                            __builtin_bit_cast(bf16x8, b[j]), acc[i][j], 0, 0, 0);
      a[n & 1] = ahead;
      if (i == FA - 1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) b[j] = c[j];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // The main loops hold no condition: with one, the compiler waits for all LDS reads where blocks join.  So
  // loads are started past the last step too, which sources answer with zeros, and waited for at the end.
  template <int NJ, class Src>
  static __device__ __forceinline__ void run_part(Src& src, int steps, Acc& acc, uint8_t* s0, uint8_t* s1, uint8_t* s2,
                                                  uint8_t* s3) {
    const int fa = (wave_id() % WA) * Src::wave_span_a();
    constexpr bool PIPED = !F8 && FA >= 4;
    uint8_t* const last = ST == 2 ? s1 : ST == 3 ? s2 : s3;
    int t = 0;
    issue<NJ>(src, s0);
    if constexpr (ST > 2) issue<NJ>(src, s1);
    if constexpr (ST > 3) issue<NJ>(src, s2);
    if constexpr (PIPED) {
      i32x4 b[NJ], a[2];
      src.step();
#pragma unroll
      for (int i = 0; i < kEarly && i < loads(NJ); ++i) issue_one<NJ>(src, i, last);
      wait_and_meet<loads(NJ) * (ST - 2) + (kEarly < loads(NJ) ? kEarly : loads(NJ))>();
#pragma unroll
      for (int j = 0; j < NJ; ++j) b[j] = frag_b(s0 + BA * PIECE, from_b(j), 0);
      a[0] = frag_a(s0, Src::frag_a_at(fa, 0), 0);
      a[1] = frag_a(s0, Src::frag_a_at(fa, 1), 0);
      for (; t + ST <= steps; t += ST) {
        piped_step<NJ>(src, last, s0, s1, acc, fa, b, a);
        piped_step<NJ>(src, s0, s1, ST == 2 ? s0 : s2, acc, fa, b, a);
        if constexpr (ST > 2) piped_step<NJ>(src, s1, s2, ST == 3 ? s0 : s3, acc, fa, b, a);
        if constexpr (ST > 3) piped_step<NJ>(src, s2, s3, s0, acc, fa, b, a);
      }
      if (t < steps) piped_step<NJ>(src, last, s0, s1, acc, fa, b, a);
      if (ST > 2 && t + 1 < steps) piped_step<NJ>(src, s0, s1, s2, acc, fa, b, a);
      if (ST > 3 && t + 2 < steps) piped_step<NJ>(src, s1, s2, s3, acc, fa, b, a);
    } else {
      for (; t + ST <= steps; t += ST) {
        ring_step<NJ>(src, s0, last, acc, fa);
        ring_step<NJ>(src, s1, s0, acc, fa);
        if constexpr (ST > 2) ring_step<NJ>(src, s2, s1, acc, fa);
        if constexpr (ST > 3) ring_step<NJ>(src, s3, s2, acc, fa);
      }
      if (t < steps) ring_step<NJ>(src, s0, last, acc, fa);
      if (ST > 2 && t + 1 < steps) ring_step<NJ>(src, s1, s0, acc, fa);
      if (ST > 3 && t + 2 < steps) ring_step<NJ>(src, s2, s1, acc, fa);
    }
    // no load into LDS may outlive the workgroup, and the next part starts with all stages free
    wait_and_meet<0>();
  }

  // Sums over the parts of `plan` (plan.parts() sources of `steps` steps each, plan.source(p)).  `rows`:
  // rows of the second operand that count.
  template <class Plan>
  static __device__ __forceinline__ void run(const Plan& plan, int steps, int rows, Acc& acc) {
    uint8_t* const s0 = stage0();
    uint8_t* const s1 = stage1();
    uint8_t* const s2 = stage2();
    uint8_t* const s3 = stage3();
    if (steps <= 0) return;
    auto all = [&](auto nj) {
      for (int p = 0; p < plan.parts(); ++p) {
        auto src = plan.source(p);
        run_part<decltype(nj)::value>(src, steps, acc, s0, s1, s2, s3);
      }
    };
    constexpr int Q = FB >= 4 ? FB / 4 : 1;   // the loop exists for one to four quarters of the fragments
    const int quarters = (rows + 16 * WB * Q - 1) / (16 * WB * Q);
    if (Q < FB && quarters <= 1) all(Int<Q>{});
    else if (2 * Q < FB && quarters == 2) all(Int<(2 * Q < FB ? 2 * Q : FB)>{});
    else if (3 * Q < FB && quarters == 3) all(Int<(3 * Q < FB ? 3 * Q : FB)>{});
    else all(Int<FB>{});
  }

  // -------------------------------------------------------------------------
  // A wave's part of the results between its registers and rows in memory
  // -------------------------------------------------------------------------
  // A lane holds four columns of 16 rows' fragments: stored as they lie, 32 bytes of a row at a time.  Instead
  // they go through LDS (the stages are free behind run()): whole rows of the wave's CF*16 columns, 16 bytes a
  // lane.  64 experts of 2048 x 7168, 512 rows each, gated backward: 7.05 ms with stores as they lie, 6.52 so.
  // Each wave has kRegion bytes of its own; a row's 16-byte pieces are spread over the banks by the row.
  static constexpr int kRegion = 2 * (STAGE - SCALES) / NW / 1024 * 1024;
  static_assert(kRegion >= 8192, "16 rows of 128 fp32 values");
  static __device__ __forceinline__ uint8_t* region() {
    const int w = wave_id();
    return (w < NW / 2 ? stage0() : stage1()) + w % (NW / 2) * kRegion;
  }
  template <int CF, int ES>
  struct Tile {
    static constexpr int ROW = CF * 16 * ES, PIECES = ROW / 16, MASK = (PIECES < 16 ? PIECES : 16) - 1;
    static constexpr int fit(int rows) { return rows * ROW <= kRegion ? rows : fit(rows / 2); }
    static constexpr int ROUND = fit(TB);   // rows that fit the region
    static __device__ __forceinline__ int at(int row, int byte) {
      return row * ROW + ((((byte >> 4) ^ row) & MASK) << 4 | (byte & ~(16 * MASK + 15)) | (byte & 15));
    }
    // 16 bytes a lane, whole rows at a time: f(row of the wave's part, byte in the row, place in the region)
    template <class F>
    static __device__ __forceinline__ void pieces(int round, F f) {
#pragma unroll
      for (int k = 0; k < ROUND * PIECES / 64; ++k) {
        const int n = k * 64 + lane_id(), row = n / PIECES, byte = n % PIECES * 16;
        f(round * ROUND + row, byte, region() + at(row, byte));
      }
    }
  };
  // Between the lanes' writes to the region and their reads of each other's: LDS takes a wave's accesses in
  // order, so only the compiler has to keep them apart.
  static __device__ __forceinline__ void turn() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
  // Row r of the wave's part is row wave_row(r) of the tile.
  static __device__ __forceinline__ int wave_row(int r) { return from_b(0) + r / 16 * (16 * WB) + r % 16; }

  // Stores acc[i0 .. i0+CF-1][..] as bf16 (ES 2) or fp32 (ES 4).  row(r): where the wave's first column of row
  // wave_row(r) goes, or null; bytes: of the wave's columns that are stored, in multiples of 16.  The stores are
  // streaming ones: the results are not read again here, the operands are, and the L2 keeps those (backward of a
  // linear product of 64 experts of 2048 x 1408 and 24 rows each: 217 us with plain stores, 176 with these; of
  // 384 rows: 417 and 408; gated and linear of 96 rows behind each other: 258 and 247).
  template <int CF, int ES, class Row>
  static __device__ __forceinline__ void store_rows(const Acc& acc, int i0, int bytes, Row row) {
    using T = Tile<CF, ES>;
    const int l = lane_id();
#pragma unroll
    for (int round = 0; round < TB / T::ROUND; ++round) {
#pragma unroll
      for (int j = 0; j < T::ROUND / 16; ++j)
#pragma unroll
        for (int i = 0; i < CF; ++i) {
          const f32x4 v = acc[i0 + i][round * (T::ROUND / 16) + j];
          uint8_t* p = region() + T::at(j * 16 + (l & 15), (i * 16 + (l >> 4) * 4) * ES);
          if constexpr (ES == 2) *reinterpret_cast<uint2*>(p) = bf16x4(v);
          else *reinterpret_cast<f32x4*>(p) = v;
        }
      turn();
      T::pieces(round, [&](int r, int byte, const uint8_t* from) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(from);
        uint8_t* to = row(r);
        if (to && byte < bytes) __builtin_nontemporal_store(v, reinterpret_cast<i32x4*>(to + byte));
      });
      turn();
    }
  }
  // The other way: bf16 rows to the lanes' places, v[i][j] four columns as bits.
  template <int CF, class Row>
  static __device__ __forceinline__ void load_rows(uint2 (&v)[CF][FB], int bytes, Row row) {
    using T = Tile<CF, 2>;
    const int l = lane_id();
#pragma unroll
    for (int round = 0; round < TB / T::ROUND; ++round) {
      T::pieces(round, [&](int r, int byte, uint8_t* to) {
        const uint8_t* from = row(r);
        *reinterpret_cast<uint4*>(to) = from && byte < bytes ? *reinterpret_cast<const uint4*>(from + byte) : uint4{0, 0, 0, 0};
      });
      turn();
#pragma unroll
      for (int j = 0; j < T::ROUND / 16; ++j)
#pragma unroll
        for (int i = 0; i < CF; ++i)
          v[i][round * (T::ROUND / 16) + j] =
              *reinterpret_cast<const uint2*>(region() + T::at(j * 16 + (l & 15), (i * 16 + (l >> 4) * 4) * 2));
      turn();
    }
  }
};

// The activation and its derivative.  silu(g) = g s(g) with s the logistic function; the tanh form of
// gelu is g s(2z), z = sqrt(2/pi) (g + 0.044715 g^3), since (1 + tanh z)/2 = s(2z).
enum { kSilu = 0, kGeluTanh = 1 };

__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

template <int ACT>
__device__ __forceinline__ void activate(float g, float* f, float* df) {
  constexpr float c2 = 1.5957691216057308f;   // 2 sqrt(2/pi)
  if constexpr (ACT == kSilu) {
    const float s = logistic(g);
    *f = g * s;
    *df = s * (1.0f + g * (1.0f - s));
  } else {
    const float s = logistic(c2 * g * (1.0f + 0.044715f * g * g));
    const float t = s * (1.0f - s);
    *f = g * s;
    // t is 0 where the polynomial may have left the range
    *df = t == 0.0f ? s : s + t * (c2 * g * (1.0f + 0.134145f * g * g));
  }
}

}  // namespace expert
}  // namespace ep
