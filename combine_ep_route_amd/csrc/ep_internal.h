// Internal declarations of libep: group/handle state and kernel launchers.
// Not installed; the public interface is include/ep.h.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <vector>

#include "ep.h"

#define EP_API extern "C" __attribute__((visibility("default")))

namespace ep {

// Build limits (checked at group creation).
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kMaxNodes = 64;
constexpr int kMaxRanks = 1024;
constexpr int kMaxHidden = 16384;
constexpr int kLayoutTile = 16;    // tokens per layout tile (one workgroup of the count kernel)

// Workgroups of `threads` that one launch takes of `blocks`: a grid dimension counts its threads in 32 bits.  What
// is left is for the kernel's loop, or for another launch.
inline unsigned grid_blocks(int64_t blocks, int threads) {
  const int64_t most = UINT32_MAX / static_cast<uint32_t>(threads);
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

constexpr uint32_t kGroupMagic = 0x45504752u;   // "EPGR"
constexpr uint32_t kHandleMagic = 0x4550484Eu;  // "EPHN"
constexpr uint32_t kDeadMagic = 0xDEADDEADu;

struct CombineArgs {
  const uint16_t* y;      // BF16 rows
  int64_t ld_y;           // elements
  int64_t rows;           // rows available in y
  const float* w;         // [n, K], or null for unit weights (dispatch backward)
  const int32_t* loc;     // [n, K]
  int64_t n;
  int K, H;
  uint16_t* out;
  int64_t ld_out;
  int max_blocks;         // 0 = no cap
  int32_t* err;
};

struct Handle;

// log2(v) if v is a power of two, else -1.
inline int log2_exact(int v) {
  if (v <= 0 || (v & (v - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Routing topology derived from a configuration, checked: shared by group
// creation and the group-free layout.  Checks mode, topology, K, M, T_max,
// S and the stage-2 kind (not the payload, hidden size or buffers).
struct Topology {
  int R, L, P, M, J, E2, s2_rank, sorted;
};
ep_status_t check_topology(const ep_config_t& cfg, Topology* t);

struct Group {
  uint32_t magic = kGroupMagic;
  ep_config_t cfg{};
  int R = 0;          // ranks
  int L = 0;          // experts per rank
  int P = 0;          // experts per node
  int J = 0;          // experts summed per node score (0 = no node limit)
  int M = 0;          // nodes kept (0 = no limit)
  int fp8 = 1;        // payload is FP8 (else BF16)
  int64_t row_bytes = 0;   // FP8: H + H/128*4; BF16: 2H
  int64_t msg_bytes = 0;   // LL: row_bytes + 16
  int64_t row_pitch = 0;   // HT row stride in the buffers: row_bytes up to 128 B
  int64_t msg_pitch = 0;   // LL message stride: msg_bytes up to 128 B
  int64_t n_max = 0;       // S * T_max
  int64_t rows1_max = 0;   // HT stage-1 rows, worst case
  int64_t rows2_max = 0;   // HT stage-2 rows, worst case (n_max * K)
  int s2_rank = 0;         // HT stage 2 per (token, rank)
  int sorted = 0;          // the same, with the places of the ranks' rows in expert order
  int E2 = 0;              // stage-2 keys: E, or R per rank
  int tiles_max = 0;       // layout tiles, worst case

  // Device buffers (owned).
  struct Alloc { void* ptr; size_t bytes; };
  std::vector<Alloc> allocs;
  int64_t bytes = 0;
  // Receive buffers, used in turn: LL fixed-slot buffers, or HT stage-row
  // sets (stage-1 and stage-2 rows with their metadata).
  uint8_t* ll_buf[2] = {nullptr, nullptr};
  struct StageSet {
    uint8_t* st1 = nullptr;
    int32_t* m1_tok = nullptr;
    int32_t* m1_src = nullptr;
    int32_t* m1_topk = nullptr;
    float* m1_w = nullptr;
    uint8_t* st2 = nullptr;
    int32_t* m2_src = nullptr;
    int32_t* m2_tok = nullptr;
    int32_t* m2_k = nullptr;
    int32_t* m2_topk = nullptr;   // per-rank stage 2 only
    float* m2_w = nullptr;
  };
  StageSet ht[2];
  int nbuf = 0;                              // receive buffers (LL) or stage sets (HT)
  int buf_next = 0;                          // the one the next dispatch takes
  uint64_t buf_gen[2] = {0, 0};              // dispatches into each of them
  int32_t* err = nullptr;    // device error word

  std::vector<Handle*> handles;

  // Device facts, read at the first launch.
  bool dev_ready = false;
  int device = -1;
  int num_cu = 0;

  ep_stats_t stats{};   // host-side call counters

  // Pinned host memory for the blocking count queries, allocated at the
  // first query (hipHostMalloc) and freed with the group.
  int32_t* host_counts = nullptr;
  size_t host_counts_len = 0;
};

struct Handle {
  uint32_t magic = kHandleMagic;
  Group* g = nullptr;
  bool in_use = false;
  int64_t n = 0;   // tokens (S*T)
  int T = 0;       // tokens per source
  int tps = 0;     // layout tiles per source
  int n_tiles = 0;
  hipStream_t stream = nullptr;
  bool maps_ready = false;       // slot/row maps written (by dispatch)
  int32_t* topk = nullptr;       // copy of topk_idx [n_max, K]
  int32_t* rank_e = nullptr;     // [n_max, K] rank of (token, k) inside its tile and expert, or -1
  int32_t* rank_n = nullptr;     // [n_max, N] HT: rank inside its tile and destination node, or -1
  int32_t* slot_map = nullptr;   // LL [n_max, K]
  int32_t* ll_count = nullptr;   // LL [E, S]
  int32_t* node_row = nullptr;   // HT [n_max, N]
  int32_t* row2 = nullptr;       // HT [n_max, K]
  int32_t* c1 = nullptr;         // HT [R]
  int32_t* off1 = nullptr;       // HT [R]
  int32_t* c2 = nullptr;         // HT [E]
  int32_t* off2 = nullptr;       // HT [E]
  int32_t* rank_x = nullptr;     // sorted [n_max, K]: ranks of (token, k) inside its tile: by expert | by rank << 8, or -1
  int32_t* place = nullptr;      // sorted [n_max, K]: the entry's row in expert order, or -1
  int32_t* entry_row = nullptr;  // sorted [n_max, K]: the stage-2 row of the entry's rank, or -1
  int32_t* cx = nullptr;         // sorted [E]: rows per expert
  int32_t* hist_x = nullptr;     // sorted [tiles_max, E] tile counts -> prefixes
  int32_t* rows_total = nullptr; // LL, many sources or runs [E]: rows per expert, for the experts' products
  int32_t* rows_list = nullptr;  // the same [n_max * K]: their message indices, expert after expert
  int32_t* hist_e = nullptr;     // [tiles_max, E] tile counts -> prefixes
  int32_t* hist_n = nullptr;     // [tiles_max, N]
  int buf_half = -1;             // receive buffer / stage set of the last dispatch
  bool dispatched = false;       // a dispatch has written this handle's rows
  uint64_t buf_gen = 0;          // the buffer's dispatch count when this handle wrote it

  // Staged (send_only) operation awaiting ep_complete: at most one.
  enum { kPendNone = 0, kPendDispatch = 1, kPendCombine = 2 };
  int pend = kPendNone;
  int32_t* pend_counts = nullptr;   // dispatch: recv_counts destination (or null)
  int pend_per_expert = 0;
  CombineArgs pend_comb{};          // combine: the launch to run
};

// ---------------------------------------------------------------------------
// Kernel launchers (one translation unit each).  All return hipSuccess or the
// launch error; they enqueue on `stream` and never synchronise.
// ---------------------------------------------------------------------------

struct RouteArgs {
  const float* scores;
  int64_t ld;        // row stride of scores, elements
  int64_t n;
  int E, N, K, M, J;
  int32_t* topk;     // [n, K]
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

struct LayoutArgs {
  const int32_t* topk;   // [n, K], or null when the handle is made from scores
  const float* scores;   // [n, E] with row stride ld, or null: route in the same pass
  int64_t ld;
  int M, J;              // routing: nodes kept (0 = no limit), scores summed per node
  int32_t* topk_out;     // routing: the caller's [n, K] output
  int64_t n;
  int S, T, K, E, N, G, P;
  int slots;             // LL slots per (expert, source)
  int ht;                // 1 = HT maps, 0 = LL maps
  int E2;                // stage-2 keys: E, or R with the per-rank stage 2
  int L;                 // experts per rank
  int s2_rank;           // HT stage 2 per (token, rank): key = e / L, first entry only
  int l_shift, p_shift;  // log2 of L and P when powers of two, else -1
  int tps, n_tiles;      // tiles per source, tiles in all
  int32_t* hist_e;       // [tiles, E2] per-tile key counts, rewritten as prefixes over the key's tiles
  int32_t* hist_n;       // [tiles, N] the same per destination node (HT)
  int32_t* topk_copy;    // [n, K]
  int32_t* rank_e;       // [n, K] out: in-tile ranks
  int32_t* rank_n;       // [n, N] out: in-tile node ranks (HT)
  int32_t* ll_count;     // LL out: slots used per (expert, source) [E, S]
  int32_t* c1;           // HT out: stage-1 rows per rank [R]
  int32_t* c2;           // HT out: stage-2 rows per key [E2]
  // With the per-rank stage 2, optionally (hist_x not null) the entries' places in expert order:
  int32_t* rank_x;       // [n, K] out: in-tile ranks by expert | by rank << 8, or -1
  int32_t* hist_x;       // [tiles, E] per-tile expert counts, rewritten as prefixes
  int32_t* cx;           // [E] out: rows per expert
  int32_t* place;        // [n, K] out: rows in expert order
  int32_t* entry_row;    // [n, K] out: the rank's row of every valid entry
  int32_t* err;          // device error word (bad or repeated entries)
};
hipError_t launch_layout(const LayoutArgs& a, hipStream_t stream);

// Receive stage of a dispatch: copy the [E, S] counters to out, or with
// per_expert != 0 write their sums over S ([E]).
hipError_t launch_recv_counts(const int32_t* counts, int E, int S, int per_expert, int32_t* out,
                              hipStream_t stream);

// Set `count` int32 values to `value` with a small kernel (stream-ordered,
// capture-safe).
hipError_t launch_fill_i32(int32_t* p, int64_t count, int32_t value, hipStream_t stream);

struct DispatchArgs {
  const void* x;          // BF16 [n, H] or FP8 [n, H]
  int64_t ld_x;           // elements
  const float* x_scales;  // FP8 input only: [n, H/128]
  int64_t ld_s;
  int in_fp8;             // tokens arrive quantised
  int out_fp8;            // payload is FP8
  int64_t n;
  int T, K, N, G, H, E, S, P, slots, tps;
  int E2, L, s2_rank;     // stage-2 keys (E, or R per rank), experts per rank, per-rank flag
  int64_t row_bytes, msg_bytes;
  int64_t row_pitch, msg_pitch;   // strides of HT rows / LL messages in the buffers
  int ht;
  int payload;            // 0 = compute the maps only
  int num_cu;             // CUs to spread the persistent workgroups over
  int max_blocks;         // 0 = no cap beyond residency
  const int32_t* topk;    // the handle's copy [n, K]
  const int32_t* rank_e;  // in-tile ranks [n, K]
  const int32_t* rank_n;  // in-tile node ranks [n, N]
  const int32_t* hist_e;  // tile prefixes [tiles, E]
  const int32_t* hist_n;  // [tiles, N]
  const int32_t* c1;      // HT: stage-1 rows per rank [R]
  const int32_t* c2;      // HT: stage-2 rows per key [E2]
  int32_t* off1;          // HT out: first stage-1 row of each rank [R] (their exclusive prefix sums)
  int32_t* off2;          // HT out: first stage-2 row of each key [E2]
  int32_t* slot_map;      // LL out [n, K]
  int32_t* row2;          // HT out [n, K]
  int32_t* node_row;      // HT out [n, N]
  // LL
  uint8_t* ll_buf;
  // HT
  const float* w;
  uint8_t* st1;
  int32_t* m1_tok;
  int32_t* m1_src;
  int32_t* m1_topk;
  float* m1_w;
  uint8_t* st2;
  int32_t* m2_src;
  int32_t* m2_tok;
  int32_t* m2_k;
  int32_t* m2_topk;       // per-rank stage 2: the token's entries on the row's rank
  float* m2_w;
};
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream);

// FP8 quantisation alone: BF16 [n, H] -> codes [n, H] + scales [n, H/128],
// the dispatch's own arithmetic (H % 128 == 0).
struct QuantArgs {
  const uint16_t* x;      // BF16 [n, H]
  int64_t ld_x;           // elements
  uint8_t* q;             // codes [n, H]
  int64_t ld_q;           // bytes
  float* scales;          // [n, H/128]
  int64_t ld_s;           // elements
  int64_t n;
  int H;
  // Of the experts' rows those that hold a message, from what a handle's creation has written:
  //   count (HT): the first ones, as many as the E counts' sum, n at most; those beyond `rows` are reported.
  //   topk, rank_e, hist_e (LL): the slots of the n entries, as the dispatch works them out.
  const int32_t* count;
  const int32_t *topk, *rank_e, *hist_e;
  int32_t E, K, S, T, tps, slots;
  int64_t rows;
  int32_t* err;
};
hipError_t launch_quantize(const QuantArgs& a, hipStream_t stream);

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream);

struct CombineBwdArgs {
  const uint16_t* g;      // BF16 [n, H] gradient of the combine's output
  int64_t ld_g;           // elements
  const uint16_t* y;      // BF16 expert-output rows, or null (no dw)
  int64_t ld_y;
  uint16_t* dy;           // BF16 row gradients at the dispatch geometry
  int64_t ld_dy;
  int64_t rows;           // rows valid in dy (and y)
  const float* w;         // [n, K]
  const int32_t* loc;     // [n, K]
  float* dw;              // [n, K] or null
  int64_t n;
  int K, H;
  int max_blocks;         // 0 = no cap
  int32_t* err;
};
hipError_t launch_combine_backward(const CombineBwdArgs& a, hipStream_t stream);

// Between the ranks' stage-2 rows and rows in expert order.  Every entry (i, k) of a token has a place, the row
// in expert order, and a row, the one of its rank; entries of a token on the same rank share it.
struct SortArgs {
  const uint8_t* x;       // the ranks' rows, or without `row` one row a token
  int64_t ld_x;           // bytes
  int64_t rows_x;
  uint8_t* out;           // rows in expert order
  int64_t ld_out;         // bytes
  int64_t rows_out;
  int32_t bytes;          // of a row, a multiple of 4
  int32_t pad;            // bytes behind them that are written as zeros: the row's last line whole, or 0
  const int32_t* row;     // [n, K], or null: entry (i, k) has row i
  const int32_t* place;   // [n, K]
  int64_t n;
  int K;
  int max_blocks;         // 0 = no cap
  int32_t* err;
};
hipError_t launch_sort(const SortArgs& a, hipStream_t stream);

struct UnsortArgs {
  const uint16_t* y;      // BF16 rows in expert order
  int64_t ld_y;           // elements
  int64_t rows_y;
  const float* w;         // [n, K], or null for unit weights (the sort's adjoint)
  uint16_t* out;          // BF16 rows of the ranks
  int64_t ld_out;
  int64_t rows_out;
  const int32_t* row;
  const int32_t* place;
  int64_t n;
  int K, H;
  int max_blocks;
  int32_t* err;
};
hipError_t launch_unsort(const UnsortArgs& a, hipStream_t stream);

struct UnsortBwdArgs {
  const uint16_t* g;      // BF16 gradient of the ranks' rows
  int64_t ld_g;
  int64_t rows_g;
  const uint16_t* y;      // BF16 rows in expert order, or null (no dw)
  int64_t ld_y;
  uint16_t* dy;           // their gradient
  int64_t ld_dy;
  int64_t rows_y;         // rows valid in dy (and y)
  const float* w;         // [n, K]
  float* dw;              // [n, K] or null
  const int32_t* row;
  const int32_t* place;
  int64_t n;
  int K, H;
  int max_blocks;
  int32_t* err;
};
hipError_t launch_unsort_backward(const UnsortBwdArgs& a, hipStream_t stream);

struct DequantArgs {
  const uint8_t* rows;
  int64_t row_stride;     // bytes
  int64_t n;
  int H;
  int fp8;
  uint16_t* y;
  int64_t ld_y;           // elements
};
hipError_t launch_dequant(const DequantArgs& a, hipStream_t stream);

// ---------------------------------------------------------------------------
// The experts' products
// ---------------------------------------------------------------------------

namespace expert {

// Rows of expert e, p = 0 .. n(e)-1, in the receive layout; before(e) is the sum of the n of the experts
// before e.
//   HT:              row before(e) + p;  n(e) = count[e].
//   LL, one source:  row e*stride + p;   n(e) = count[e].
//   LL, few sources: source s fills slots e*stride + s*slots ..; n(e) is the sum of count[e*sources + s].
//   LL, many:        row list[before(e) + p];  n(e) = count[e] (launch_list_rows makes both).
// In a tile, offsets are 32-bit: 256 rows of any operand, and with several sources an expert's slots, span
// less than 2^31 bytes.
constexpr int kFewSources = 8;
struct ExpertRows {
  const int32_t* count;
  const int32_t* list;
  int64_t limit;          // rows that the caller's tensors hold
  int32_t E, stride, sources, slots;
  int32_t* err;           // device error word: rows beyond the limit are left out and reported
};

// The launchers return hipErrorInvalidConfiguration, before any work, for more tiles than one grid holds;
// with `check` they only say whether they would.
// Strides (ld_*, *_expert) and k_bytes are in bytes, those of bf16 outputs (ld_out) and grad in elements.
struct AlongArgs {
  ExpertRows rows;
  int64_t rows_max, per_expert_max;   // bounds that the host knows
  int64_t k_bytes;                    // bytes of a row that are contracted
  int32_t N;
  const uint8_t* x;
  int64_t ld_x;
  const uint8_t* x_scales;            // FP8: one float per 128 values of a row
  int64_t ld_xs;
  const uint8_t* w[2];                // linear: w[0]; gated: gate and up
  int64_t ld_w[2], w_expert[2];
  const uint8_t* w_scales[2];         // FP8: one float per 128 x 128 values
  int64_t ld_ws[2], ws_expert[2];
  uint16_t* out[2];
  int64_t ld_out[2];
  const uint16_t* grad;               // gated gradient: the gradient of the gated product
  int64_t ld_grad;
};
hipError_t launch_linear(const AlongArgs& a, bool fp8, hipStream_t stream, bool check = false);
hipError_t launch_gated(const AlongArgs& a, bool fp8, int act, hipStream_t stream, bool check = false);
// out = the gradients of the gate's and of the up product
hipError_t launch_gated_grad(const AlongArgs& a, int act, hipStream_t stream, bool check = false);

struct RowGradArgs {
  ExpertRows rows;
  int64_t rows_max, per_expert_max;
  int32_t I, N, parts;                // contracted size, columns, 1 or 2 (dy, w)
  const uint8_t* dy[2];
  int64_t ld_dy[2];
  const uint8_t* w[2];
  int64_t ld_w[2], w_expert[2];
  uint16_t* dx;
  int64_t ld_dx;                      // elements
};
hipError_t launch_row_grad(const RowGradArgs& g, hipStream_t stream, bool check = false);

struct WeightGradArgs {
  ExpertRows rows;
  int32_t I, H, parts;
  const uint8_t* dy[2];
  int64_t ld_dy[2];
  const uint8_t* x;
  int64_t ld_x;
  uint8_t* dw[2];
  int64_t ld_dw[2], dw_expert[2];
};
hipError_t launch_weight_grad(const WeightGradArgs& g, bool f32, hipStream_t stream, bool check = false);

// Codes of the experts' rows to bf16: bf16_rne(code * scale), ep_dequantize_rows' values.
// The rows are the first ones, as many as `count` sums up to, or without it the slots of the entries.
struct DecodeArgs {
  const uint8_t* x;                   // codes
  int64_t ld_x;                       // bytes
  const float* scales;                // one per 128 codes of a row
  int64_t ld_s;                       // elements
  int32_t C;                          // codes of a row
  uint16_t* out;
  int64_t ld_out;                     // elements
  int64_t rows;                       // that the tensors hold
  int64_t n;                          // entries: a bound on the rows in use
  const int32_t* count;               // [E]
  const int32_t *topk, *rank_e, *hist_e;   // LL: an entry's expert, its rank among its tile's, the tile's prefix
  int32_t E, K, S, T, tps, slots;
  const int32_t* ll_count;            // LL: launch_list_rows' arguments, if `list` is to be made too
  int32_t *total, *list;
  int32_t* err;
};
hipError_t launch_decode(const DecodeArgs& a, hipStream_t stream);

// LL with several sources: rows per expert and the list of rows, from the slots' counts [E, S].
hipError_t launch_list_rows(const int32_t* counts, int E, int S, int slots, int32_t* total, int32_t* list,
                            hipStream_t stream);

}  // namespace expert

// ---------------------------------------------------------------------------
// Norms around the block
// ---------------------------------------------------------------------------

namespace norm {

constexpr int kNormCus = 256;   // CUs the backward pass plans for

// Strides in elements.
struct NormArgs {
  int64_t n;
  int32_t H;
  const uint16_t* y;
  int64_t ld_y;
  const uint16_t* x;         // the residual stream
  int64_t ld_x;
  const void* w_post;        // or null: no norm on y
  const void* w_pre;
  int32_t post_f32, pre_f32;
  const uint16_t* gate;      // or null
  int64_t ld_gate;
  int32_t gate_rows;         // a gate per token, else per channel
  float a, b, eps;
  uint16_t* out_x;
  int64_t ld_out_x;
  uint16_t* out_n;
  int64_t ld_out_n;
};
hipError_t launch_residual_norm(const NormArgs& a, hipStream_t stream);

struct NormGradArgs {
  int64_t n;
  int32_t H;
  const uint16_t* y;
  int64_t ld_y;
  const uint16_t* x;         // the stream behind the block
  int64_t ld_x;
  const uint16_t* g_res;     // or null: zeros
  int64_t ld_g_res;
  const uint16_t* g_norm;
  int64_t ld_g_norm;
  const void* w_post;
  const void* w_pre;
  int32_t post_f32, pre_f32;
  const uint16_t* gate;
  int64_t ld_gate;
  int32_t gate_rows;
  float a, b, eps;
  uint16_t* dres;
  int64_t ld_dres;
  uint16_t* dy;
  int64_t ld_dy;
  uint16_t* dgate_token;     // optional outputs
  int64_t ld_dgate;
  float* dw_pre;
  float* dw_post;
  float* dgate_channel;
  float* work;               // up to 2 x grad_blocks x H
};
int grad_blocks(int64_t n, int H);   // its workgroups, each with a share of the column sums
hipError_t launch_residual_norm_backward(const NormGradArgs& a, hipStream_t stream);

}  // namespace norm

}  // namespace ep
