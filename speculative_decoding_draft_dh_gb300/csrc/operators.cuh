// Internal declarations of the training, search and state operators (row_stats.cu, distill.cu,
// distill_ring.cu, beam.cu, states.cu).
//
// Programmatic dependent launch: the passes over the logits let the next kernel of their call start
// once they have waited themselves, and a call's last kernel lets the next call's start where it writes
// losses or a selection.  One that writes states or a gradient lets nothing start before it has ended:
// the rescoring kernels load their hidden rows before their own wait, and those may be rows that a
// reordering or a gradient has just written.
#pragma once

#include "dh_internal.cuh"

namespace dh {

// Distillation from a teacher's top logits (row_stats.cu, distill.cu).
struct DistillArgs {
  const void* logits;  // [N] rows of `vocab`, stride ld elements
  long long ld;
  void* grad;  // rows of stride gld; may be the logits
  long long gld;
  const int32_t* idx;      // [N x K]
  const float* teacher;    // [N x K]
  const int32_t* n_valid;  // [N] or null
  const float* weight;     // [N]
  const float2* stats;     // [N] (max, sum)
  const float2* seg;       // [N x n_seg] (max, sum) of the segments
  float2* stats_out;
  float* loss_out;
  float* gathered;         // [N x K] the entries' logits, where the gradient overwrites them; or null
  int* status;             // device status word, or null
  int N, vocab, K, n_seg, splits;
  float temperature, inv_t, c;  // c = log2(e) / T
};
int row_segments(int vocab, int dtype);
bool rows_aligned(const void* logits, long long rs, long long ws, int R, int W, int elem);
// Statistics of every segment of the rows [r][w] at logits + r rs + w ws, into seg [R W x n_seg].
// With `score` given, the rows whose score is not finite or whose `finished` (may be null) is not 0
// are left out.
cudaError_t launch_row_stats(const Ctx& c, const void* logits, long long rs, long long ws, int R, int W, int vocab,
                             int dtype, float temperature, const float* score, const int32_t* finished, float2* seg);
// The kernels of distill.cu and distill_ring.cu; which of them a call takes is api.cu's choice.
// launch_distill_ring: statistics (stats_out) and dense gradient; *done is false, and nothing was
// launched, where the rows are too long.  `test` (fp32 only): what the self-test of its waits holds back
// in the last CTA of every cluster, from row `row` on, and the waits' limit.
struct RingTest {
  enum Hold { NOTHING = 0, COPIES, PAIRS, SLOTS };
  int hold, row, limit_us;
};
cudaError_t launch_distill_ring(const Ctx& c, const DistillArgs& a, int dtype, bool* done,
                                const RingTest* test = nullptr);
// Rows for launch_distill_short: distill_short on a device of num_sms SMs; whatever the device (and so
// without a workspace) if distill_short_always.
bool distill_short_always(int N, int n_seg, bool step);
bool distill_short(const DistillArgs& a, int num_sms, bool step);
cudaError_t launch_distill_short(const Ctx& c, const DistillArgs& a, int dtype, bool loss, bool grad);
cudaError_t launch_distill_gather(const Ctx& c, const DistillArgs& a, int dtype);
cudaError_t launch_distill_dense(const Ctx& c, const DistillArgs& a, int dtype);
cudaError_t launch_distill_finish(const Ctx& c, const DistillArgs& a, int dtype, bool loss, bool grad);
cudaError_t launch_distill_grad(const Ctx& c, const DistillArgs& a, int dtype);

// Beam selection (beam.cu).
cudaError_t launch_beam_select(const Ctx& c, const void* logits, long long rs, long long ws, const float* score,
                               const int32_t* finished, const float2* seg, int R, int W, int vocab, int M, int dtype,
                               float temperature, int pad_token, int32_t* parent, int32_t* token, float* score_out);

// Reordering of states (states.cu).  Sizes and byte strides of (A, R, slot, H, T) and a contiguous
// unit of bytes.
struct ReorderArgs {
  const char* src;
  char* dst;
  long long ss[5], ds[5];
  const int32_t* idx;                            // [R x M]
  const int32_t *lengths, *src_base, *dst_base;  // [R] or null
  int A, R, src_slots, dst_slots, M, H, T;
  long long unit;
  bool in_place;
};
long long reorder_columns(const ReorderArgs& a);
long long reorder_blocks(const ReorderArgs& a);
cudaError_t launch_reorder(const Ctx& c, const ReorderArgs& a);

}  // namespace dh
