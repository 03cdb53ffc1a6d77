// Host-side declarations shared by the ABI layer and the kernel files:
// geometry constants, the workspace layout and the kernel launchers.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dflash.h"

namespace dfk {

// top-K streaming geometry: a wave owns 8 16-byte loads per lane; a block of
// 4 waves owns one segment of a drafter row
constexpr int kTopkThreads = 256;
constexpr int kTopkLoads = 8;
constexpr int kTopkCap = 256;          // candidate buffer per wave
constexpr int kTopkMergeMax = 2048;    // keys the last block of a row merges in LDS

inline int topk_wave_elems(int logit_dtype) { return 64 * kTopkLoads * (logit_dtype == DFLASH_BF16 ? 8 : 4); }
inline int topk_block_elems(int logit_dtype) { return 4 * topk_wave_elems(logit_dtype); }
// blocks per drafter row stay <= 32 so that the partial lists of two rows
// fit the cycle's candidate/score block (kTopkCycleMerge keys of LDS)
constexpr int kTopkCycleMerge = 512;
constexpr int kTopkMaxSeg = kTopkCycleMerge / 16;

constexpr int kChunk = DFLASH_CHUNK;   // target-row chunk (one wave)

// 256-thread blocks of the streaming launch resident at once: eight per CU
// on the 256 CUs of an MI355X
constexpr int kResidentBlocks = 8 * 256;
// statistics blocks dispatched before the edge blocks, in percent of all
// statistics blocks (measured at concurrent-32: 41.3 to 41.9 us per cycle at
// 30 to 40, 42.2 at 0 and at 60, 42.8 at 80; the edges then start while
// the last top-K blocks finish)
constexpr int kEdgePrePct = 40;

// gate: the hidden dimension is cut into slices of kGateSlice; a gate block
// accumulates kGateGroup consecutive slices of one tile on the matrix
// cores, and consumers sum the groups' partial pre-activations W_g h in
// group order before the sigmoid
constexpr int kGateSlice = 256;
constexpr int kGateGroup = 8;
inline int gate_slices(const dflash_dims& d) {
  return d.param_dtype == DFLASH_BF16 ? (d.hidden + kGateSlice - 1) / kGateSlice : 1;
}
inline int gate_groups(const dflash_dims& d) { return (gate_slices(d) + kGateGroup - 1) / kGateGroup; }
// gate blocks of the streaming launch: bf16 tiles of 16 rows x 32 columns
// per slice group, or one fp32 row per block
constexpr int kGateTileRows = 16, kGateTileCols = 32;
inline long long stream_gate_blocks(const dflash_dims& d) {
  const long long R = (long long)d.B * d.L;
  return d.param_dtype == DFLASH_BF16
             ? ((R + kGateTileRows - 1) / kGateTileRows) * ((d.r + kGateTileCols - 1) / kGateTileCols) * gate_groups(d)
             : R;
}

struct ChunkStat {
  float m;      // chunk maximum logit
  float s;      // sum over the chunk of exp((z - m) / T)  (sampling rows)
  int32_t arg;  // first index of the maximum (greedy rows)
  int32_t pad;
};

struct WsLayout {
  int n_sub;    // top-K sub-segments (one wave's registers) per drafter row
  int spb;      // sub-segments per top-K block
  int n_seg;    // top-K blocks per drafter row (a merge kernel runs if > 1)
  int n_chunk;  // target chunks per row
  size_t topk_partial, gate, cand_idx, cand_logit, zc, S, path_rank, draft_tok, q, stats;
  size_t jstar, qtab;  // the fused cycle's trace table: decision and q of every row (t, i)
  // The fused cycle runs its edges inside the streaming launch when its
  // top-K, gate and edge blocks fit the GPU's resident blocks at once
  // (kResidentBlocks); it then hands over through: the cycle epoch (one
  // word, advanced by every cycle's last launch), the top-K lists as
  // (key, check | tag) pairs and the gate partials as (tag | value) words.
  bool edges;
  size_t epoch, tk_tag, gate_tag;
  size_t cycle_total;  // bytes the fused cycles use (the regions above)
  // the split path's gate partials, one per quarter of each tile (bf16
  // parameters) or one per row (fp32), after everything the cycles use
  size_t gate_q;
  size_t total;
};

WsLayout ws_layout(const dflash_dims& d);

// Events the next kernel launch on this thread records at the kernel's own
// start and end (hipExtLaunchKernel: the dispatch's timestamps, not the
// stream's), set by the per-kernel timer and consumed by that launch.
extern thread_local hipEvent_t g_launch_start, g_launch_stop;

template <typename F, typename... Args>
inline void launch(F kernel, dim3 grid, dim3 block, hipStream_t st, Args... args) {
  hipEvent_t a = g_launch_start, b = g_launch_stop;
  g_launch_start = g_launch_stop = nullptr;
  hipExtLaunchKernelGGL(kernel, grid, block, 0, st, a, b, 0, args...);
}

// ---- launchers (each enqueues on `st`; returns the launch status) ----

hipError_t launch_topk(const dflash_dims& d, const WsLayout& w, const void* U, int32_t* cand_idx,
                       float* cand_logit, char* ws, hipStream_t st);
hipError_t launch_gate(const dflash_dims& d, const void* h, const void* W_g, float* gpart, hipStream_t st);
hipError_t launch_scores(const dflash_dims& d, const int32_t* x0, const int32_t* cand_idx,
                         const float* cand_logit, const void* E, const float* gpart, float* S,
                         hipStream_t st);
// first global token index of each vocabulary shard
struct ShardBegins {
  int32_t begin[DFLASH_MAX_SHARDS];
};
// a vocabulary split for the verify: shard s covers tokens
// [begin[s], begin[s + 1]) (begin[n] = V), its residual-draw chunks are
// cbase[s] .. cbase[s + 1] - 1 (the grid restarts at each shard), and its
// target rows Z[s] are [B, L + 1, begin[s + 1] - begin[s]]
struct ShardMap {
  int32_t n;
  int32_t begin[DFLASH_MAX_SHARDS + 1];
  int32_t cbase[DFLASH_MAX_SHARDS + 1];
  const void* Z[DFLASH_MAX_SHARDS];
};
hipError_t launch_topk_merge(const dflash_dims& d, int n_shards, const ShardBegins& sb, const int32_t* idx_parts,
                             const float* val_parts, int32_t* cand_idx, float* cand_logit, hipStream_t st);
hipError_t launch_shard_stats(const dflash_dims& d, const ShardMap& m, int shard, const void* Zs, const float* T,
                              ChunkStat* stats, hipStream_t st);
hipError_t launch_finalize_shards(const dflash_dims& d, const ShardMap& m, const int32_t* cand_idx,
                                  const int32_t* path_rank, const float* q, const float* T, const uint64_t* seed,
                                  uint64_t cycle, const ChunkStat* stats, int32_t* accept_len, int32_t* out_tok,
                                  hipStream_t st);
hipError_t launch_trace_viterbi(const dflash_dims& d, const float* S, const int32_t* cand_idx, int32_t* path_rank,
                                int32_t* draft_tok, float* q, hipStream_t st);
hipError_t launch_trace(const dflash_dims& d, const float* S, const int32_t* cand_idx, const float* T,
                        const uint64_t* seed, uint64_t cycle, int32_t* path_rank, int32_t* draft_tok,
                        float* q, hipStream_t st);
hipError_t launch_stats(const dflash_dims& d, const WsLayout& w, const void* Z, const float* T, ChunkStat* stats,
                        hipStream_t st);
hipError_t launch_finalize(const dflash_dims& d, const WsLayout& w, const void* Z,
                           const int32_t* cand_idx, const int32_t* path_rank, const float* q,
                           const float* T, const uint64_t* seed, uint64_t cycle,
                           const ChunkStat* stats, int32_t* accept_len, int32_t* out_tok,
                           hipStream_t st);
// dflash_cycle: (1) top-K lists + chunk statistics + gate slices,
// (2) candidates + pair scores, (3) trace + verify
hipError_t launch_topk_lists(const dflash_dims& d, const WsLayout& w, const void* U, char* ws, hipStream_t st);
// the edge work folded into the streaming launch (its candidates, scores
// and trace-table rows; zc, jstar and qtab go to the workspace)
struct CycleEdges {
  int n_pre;  // statistics blocks dispatched before the edge blocks
  const int32_t* x0;
  const void* E;
  const uint64_t* seed;
  uint64_t cycle;
  int32_t* cand_idx;
  float* cand_logit;
  float* S;
};
hipError_t launch_cycle_stream(const dflash_dims& d, const WsLayout& w, const void* U, const void* Z, const void* h,
                               const void* W_g, const float* T, char* ws, hipStream_t st,
                               const CycleEdges* edges = nullptr);
hipError_t launch_cycle_scores(const dflash_dims& d, const WsLayout& w, const int32_t* x0, const void* E,
                               const void* Z, const float* T, const uint64_t* seed, uint64_t cycle, char* ws,
                               int32_t* cand_idx, float* cand_logit, float* S, hipStream_t st);
hipError_t launch_cycle_finalize(const dflash_dims& d, const WsLayout& w, const void* Z, const int32_t* cand_idx,
                                 const float* T, const uint64_t* seed, uint64_t cycle, char* ws, const float* S_maxsum,
                                 int32_t* path_rank, int32_t* draft_tok, float* q, int32_t* accept_len,
                                 int32_t* out_tok, hipStream_t st, bool advance_epoch = false);
hipError_t launch_conv2tap(const dflash_dims& d, const void* x, const void* x0, const void* Wt, float* y,
                           hipStream_t st);
// ---- rows of vocabulary logits (dflash_rows) ----

// dflash_sample / dflash_filter
constexpr int kSampleThreads = 512;
constexpr int kSampleBins = 512;
constexpr int kSampleMaxSeg = 512;   // blocks per row
constexpr int kSampleMaxLoads = 8;
// tokens that a segment of `loads` slots a thread lists
constexpr int sample_cap(int loads, bool all) { return all ? kSampleThreads * 4 * loads : loads == 2 ? 256 : 64; }
constexpr int kSampleOne = 8192;     // longest fp32 row that one block does by itself
constexpr int kSampleAsk = 8192;     // tokens outside the lists that a row can ask for: these or an eighth
// a segment of an fp32 row: kSampleThreads * loads slots
struct SamplePart {
  double J;      // the segment's maximum in eighths of an octave, rounded; -inf: nothing unmasked
  float max;     // the maximum
  uint32_t n;    // unmasked tokens
  int32_t nb;    // bins in use
  int32_t listed;  // the tokens of bins 0 .. listed - 1 are in the segment's list
  double mass[kSampleBins];    // bin b: weights over 2^((J - b) / 8)
  uint32_t upto[kSampleBins];  // tokens of bins 0 .. b
};
// a segment of a bf16 row: seg_slots slots, at most 65528 elements (a count fits 16 bits)
constexpr int kSampleItems = 6144;
constexpr int kSampleOdd = 64;
constexpr int kSampleMaxSegSlots = 8191;
constexpr int kSampleMostParts = 8192;  // segments a pass over the workspace counts (12.5 KB each)
struct SampleValues {
  uint16_t counts[kSampleItems];
  uint32_t odd[kSampleOdd];      // tokens near zero: value << 16 | place in the segment
};
// bins whose tokens a row needs beyond the lists: up to two ranges
enum { kSampleAskNone = 0, kSampleAskBins = 1, kSampleAskRow = 2 /* more tokens than a row can ask for: it is read again */ };
struct SampleAsk {
  int32_t kind;
  uint32_t n;  // tokens collected
  int32_t b0[2], b1[2];
  uint32_t klo[2], khi[2];
};
struct SampleArgs {
  const void* Z;
  int64_t R, stride;
  int32_t V, group;
  const float* T;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
};
struct SampleOut {
  const double* u;
  int32_t* token;
  float* prob;
  int32_t* kept;
  void* out;  // the filtered rows (dflash_filter)
  int64_t out_stride;
  uint32_t fill;  // fill value in the element type
};
struct SamplePlan {
  bool one;       // one launch, a block a row
  int n_seg;      // blocks per row
  int seg_slots;  // bf16: slots of a block
  int loads;      // fp32: slots of a thread
  bool all;       // fp32: every token is listed
  int cap;        // fp32: tokens a block lists
  uint32_t ask;   // fp32: tokens outside the lists that a row can ask for
  int64_t batch;  // rows per pass over the workspace
  size_t parts, lists, cuts, asks, asked, total;
};
SamplePlan sample_plan(const dflash_rows& r);
size_t rows_workspace(const dflash_rows& r);
hipError_t launch_sample(int32_t dtype, const SampleArgs& a, const SampleOut& o, char* ws, const SamplePlan& pl,
                         hipStream_t st);

// dflash_distill: a block sums `units` times kDistillUnit slots of a row;
// dflash_distill_grad: a block writes kDistillThreads * grad_loads slots
constexpr int kDistillThreads = 256;
constexpr int kDistillUnit = 1024;
constexpr int kDistillMaxUnits = 8;
struct DistillPart {
  double m, s;  // log2 of the largest term (rounded) and sum of 2^(x - m) over the segment's tokens
};
struct DistillArgs {
  const void* S;
  int64_t R, stride;
  int32_t V, K;
  double tau;
  const int32_t* t_idx;
  const float* t_logit;
  const double* t_lse;   // or null: the list alone is the teacher
  const float* weight;   // or null
};
struct DistillPlan {
  int units, n_seg;
  int grad_loads, grad_seg;
  size_t total;
};
DistillPlan distill_plan(const dflash_rows& r);
hipError_t launch_distill(int32_t dtype, const DistillArgs& a, float* loss, double* lse, double* lse_rest, char* ws,
                          const DistillPlan& pl, hipStream_t st);
hipError_t launch_distill_grad(int32_t dtype, const DistillArgs& a, const float* grad_loss, const double* lse,
                               const double* lse_rest, void* dS, int64_t d_stride, const DistillPlan& pl, hipStream_t st);
// dflash_logprobs: a block streams seg_slots slots of a row; the gradient as dflash_distill's
constexpr int kLogprobsThreads = 256;
constexpr int kLogprobsMaxSeg = 256;   // segments of a row: one a thread of the join
constexpr int kLogprobsBlocks = 2048;  // eight a CU
struct LogprobsPart {
  double M, s, h;  // reference (a whole exponent of two), sums of 2^t and 2^t t over the segment
  float m;         // its largest logit
};
struct LogprobsArgs {
  const void* Z;
  int64_t R, stride;
  int32_t V, group;
  const float* T;  // or null
  int32_t M, N;
  const int32_t* tok;
};
struct LogprobsOut {
  float* logp;
  float* norm;
  float* entropy;  // or null
  int32_t* top_idx;
  float* top_logp;
};
struct LogprobsPlan {
  int threads, n_seg, seg_slots;
  int unit;  // slots a thread loads at a time
  int grad_loads, grad_seg;
  size_t lists, total;
};
LogprobsPlan logprobs_plan(const dflash_rows& r, int N);
hipError_t launch_logprobs(int32_t dtype, const LogprobsArgs& a, const LogprobsOut& o, char* ws, const LogprobsPlan& pl,
                           hipStream_t st);
hipError_t launch_logprobs_grad(int32_t dtype, const LogprobsArgs& a, const float* g_logp, const float* g_ent,
                                const float* norm, const float* entropy, void* dZ, int64_t d_stride,
                                const LogprobsPlan& pl, hipStream_t st);

// ---- rows in 8 bits ----
struct QuantArgs {
  const void* X;
  int64_t R, stride;
  int32_t H;
  int8_t* q;
  int64_t q_stride;
  float* scale;
};
hipError_t launch_quant_i8(int32_t dtype, const QuantArgs& a, hipStream_t st);
struct LinearArgs {
  int64_t R, xq_stride, wq_stride, y_stride;
  int32_t N, H;
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  void* y;
};
// blocks of the launch (a block has at most 512 threads)
int64_t linear_blocks(int64_t R, int32_t N, int32_t H);
hipError_t launch_linear_i8(int32_t dtype, const LinearArgs& a, hipStream_t st);

hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t st);
// device address and size of the library's static scratch on the current
// device (looked up once per device)
hipError_t static_scratch(void** out, size_t* bytes);
hipError_t launch_read_probe(const void* buf, size_t bytes, uint32_t* sink, hipStream_t st);
hipError_t launch_copy_probe(void* dst, const void* src, size_t bytes, hipStream_t st);

}  // namespace dfk
