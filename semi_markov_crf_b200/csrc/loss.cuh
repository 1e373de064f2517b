// loss.cuh -- sizes, workspace and launchers of the training losses over rows
// of label scores (loss_row.cuh, loss_seq.cu, loss_api.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "device.cuh"

namespace semicrf {

constexpr int LOSS_V_MAX = 1 << 24;            // labels per row
constexpr long long LOSS_ROWS_MAX = 1 << 27;   // B * T
constexpr int LOSS_K_MAX = 1024;               // teacher entries per position

// LM_SCALED: the gradient pass of the preference loss, g = wseq_b / temperature ([v = y] - q_v)
// from the statistics that its first pass left.
enum LossMode : int { LM_LOGPROB = 0, LM_POLICY = 1, LM_PREFERENCE = 2, LM_DISTILL = 3, LM_SCALED = 4 };
// Sites of the bounds-checking build, after the recursions' (ring.cuh).
enum LossSite : int {
  SITE_LOSS_SCORE = 14,   // a row's element at a label or a teacher's entry
  SITE_LOSS_EDGE = 15,    // a single element beside a row's 16-byte vectors
  SITE_LOSS_VECTOR = 16,  // a vector of a row, read or written
  SITE_LOSS_ENTRY = 17,   // a teacher's entry in shared memory, its word of the table
  SITE_LOSS_CHUNK = 18,   // a chunk's source inside its row, its place inside the ring
  SITE_LOSS_SLOT = 19,    // a slot of a ring's state, of this CTA or of a peer
  SITE_LOSS_SUM = 20      // a position of a sequence, a CTA's place among the sums
};
enum LossType : int { LT_F32 = 0, LT_BF16 = 1, LT_F16 = 2 };

// Everything a row kernel reads or writes.  Row r = b * T + t; z = x / temperature.
struct RowArgs {
  const void* x;        // [B * T] rows of V scores, ldx elements apart
  void* g;              // gradient rows (nullptr: none), ldg elements apart
  long long ldx, ldg;
  int B, T, V;
  int add;              // 1: g += gradient (float32 only)
  const int32_t* lengths;
  const int32_t* labels;  // [B, T], negative: does not count (not for LM_DISTILL)
  float sl;             // log2(e) / temperature
  double s;             // 1 / temperature
  double tau;           // temperature
  double inv_sl;        // 1 / sl
  const float* grad_logp;  // LM_LOGPROB: d loss / d logp [B, T] (nullptr: ones)
  const float* old_logp;   // LM_POLICY
  const float* ref_logp;   // LM_POLICY, LM_PREFERENCE; nullptr: no reference
  const float* adv;        // [B] or, with adv_tok, [B, T]
  int adv_tok;
  double clip_lo, clip_hi, kl_coef;  // the clip's corners, the KL term's weight
  const double* w;         // [B] upstream weights (nullptr: ones)
  const int32_t* ids;      // LM_DISTILL: [B, T, k] labels, negative: unused entry
  const float* tl;         // their teacher logits
  const float* tlse;       // [B, T] teacher log-sum-exp (nullptr: normalise over the entries)
  int k;
  float* logp;             // [B, T] output (not LM_DISTILL)
  float* tok;              // [B, T] per-position term that the sequence pass sums
  float* kl;               // [B, T] LM_POLICY
  uint8_t* clip;           // [B, T] LM_POLICY
  float2* stat;            // [B, T] LM_PREFERENCE: a row's base and sum of exponentials
  float* wseq;             // [B] LM_SCALED: d loss / d logp of the sequence's positions
  int* status;             // cleared by the pass, unless
  int keep_status;         // it follows another one of the same call
  // One position a sequence (T = 1): the pass writes the sequences' sums itself.
  int single;
  float* seq_sum;          // [B] each nullable
  float* seq_kl;
  int32_t* seq_clipped;
};

// Workspace of the loss entry points: the status word first, as in the
// recursions' workspace.
struct LossWs {
  int* status;
  float* tok;
  float* kl;
  uint8_t* clip;
  float2* stat;
  float* wseq;
};
size_t loss_layout(int B, int T, void* base, LossWs* p);

// Sums of a sequence's positions and what follows from them (loss_seq.cu).
struct SeqArgs {
  int B, T;
  const int32_t* lengths;
  const int32_t* labels;   // LM_PREFERENCE: which positions count, which are malformed
  int V;
  int* status;
  const float* tok;
  const float* kl;
  const uint8_t* clip;
  float* sum;              // [B] sums of tok (nullptr: none)
  float* kl_sum;           // [B] LM_POLICY (nullptr: none)
  int32_t* clipped;        // [B] LM_POLICY (nullptr: none)
  // LM_PREFERENCE: sequences [0, B/2) chosen, [B/2, B) rejected
  double beta, margin, smoothing;
  int average;
  const double* w;         // [B/2]
  float* loss;             // [B/2]
  float* reward;           // [B] (nullptr: none)
  float* wseq;             // [B]
};

// One pass over the rows (loss_row.cuh, compiled once for each type).
cudaError_t launch_rows_f32(int mode, const RowArgs& a, cudaStream_t st);
cudaError_t launch_rows_bf16(int mode, const RowArgs& a, cudaStream_t st);
cudaError_t launch_rows_f16(int mode, const RowArgs& a, cudaStream_t st);

inline cudaError_t launch_loss_rows(int mode, int type, const RowArgs& a, cudaStream_t st) {
  return type == LT_F32 ? launch_rows_f32(mode, a, st)
                        : type == LT_BF16 ? launch_rows_bf16(mode, a, st) : launch_rows_f16(mode, a, st);
}
int loss_sm_count();  // of the current device
int loss_ring_stall();  // semicrf_selftest_ring_stall's polls (bounds-checking build)

// A launch that may be set up while the kernel before it in the stream ends:
// the kernel calls after_previous() before it touches anything.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
inline cudaLaunchAttribute follows() {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  return at;
}
cudaError_t launch_loss_sums(const SeqArgs& a, cudaStream_t st);
cudaError_t launch_loss_pairs(const SeqArgs& a, cudaStream_t st);

cudaError_t launch_policy_scores(const double* logp, const double* old_logp, const double* ref,
                                 const double* adv, long long n, double clip_lo, double clip_hi,
                                 double kl_coef, const double* w, double* loss, double* kl,
                                 double* grad, cudaStream_t st);
cudaError_t launch_preference_scores(const double* chosen, const double* rejected,
                                     const double* ref_chosen, const double* ref_rejected,
                                     long long n, double beta, double margin, double smoothing,
                                     const double* w, double* loss, double* grad_chosen,
                                     double* grad_rejected, cudaStream_t st);

// Per-kernel timing of semicrf_profile_enable (api.cu).
class LaunchTimer {
 public:
  LaunchTimer(const char* name, cudaStream_t st);
  ~LaunchTimer();
  LaunchTimer(const LaunchTimer&) = delete;
  LaunchTimer& operator=(const LaunchTimer&) = delete;

 private:
  const char* name_;
  cudaStream_t st_;
  cudaEvent_t a_ = nullptr, b_ = nullptr;
};

// ---------------------------------------------------------------- shared arithmetic
// The clipped policy term of one ratio: r = exp(delta), delta = logp - old.
//   loss = -min(r A, clip(r, 1 - lo, 1 + hi) A) + c (e^d - d - 1),  d = ref - logp
// and its slope in logp.  On the corners of the clip the unclipped side counts.
// An advantage of 0 counts for nothing however large the ratio.
template <typename F>
struct PolicyTerm {
  F loss, kl, slope;
  bool clipped;
};

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// e^d - d - 1 without its cancellation: near zero the Taylor series from d^2/2
// (|d| < 1/2: the first omitted term, d^14/14!, is below 2^-47 of d^2/2).
template <typename F>
__device__ __forceinline__ F exp_less_linear(F d) {
  if (fabs(d) < F(0.5)) {
    F p = F(1.0 / 6227020800.0);
    p = p * d + F(1.0 / 479001600.0);
    p = p * d + F(1.0 / 39916800.0);
    p = p * d + F(1.0 / 3628800.0);
    p = p * d + F(1.0 / 362880.0);
    p = p * d + F(1.0 / 40320.0);
    p = p * d + F(1.0 / 5040.0);
    p = p * d + F(1.0 / 720.0);
    p = p * d + F(1.0 / 120.0);
    p = p * d + F(1.0 / 24.0);
    p = p * d + F(1.0 / 6.0);
    p = p * d + F(0.5);
    return p * d * d;
  }
  const F e = exp_of(d);
  return e > F(1e30) ? e : e - d - F(1);  // d may be infinite: a label of probability zero
}

// The clip is given by its corners lo = 1 - clip_low and hi = 1 + clip_high.
template <typename F>
__device__ __forceinline__ PolicyTerm<F> policy_term(F delta, F adv, F lo, F hi, F c, bool has_ref,
                                                     F d) {
  PolicyTerm<F> o;
  const F r = exp_of(delta);
  const F rc = r < lo ? lo : (r > hi ? hi : r);  // NaN stays NaN
  const bool none = adv == F(0) && r == r;       // r may be infinite
  const F free_ = none ? F(0) : r * adv, cut = none ? F(0) : rc * adv;
  o.clipped = (adv > F(0) && r > hi) || (adv < F(0) && r < lo);
  o.loss = -(cut < free_ ? cut : free_);
  o.slope = o.clipped ? F(0) : -free_;
  o.kl = F(0);
  if (has_ref) {
    o.kl = exp_less_linear(d);
    if (c != F(0)) {
      o.loss += c * o.kl;
      o.slope -= c * (fabs(d) < F(0.5) ? d + o.kl : exp_of(d) - F(1));
    }
  }
  return o;
}

// A position's term from float64 log-ratios.  Ratios and what follows are float32
// (their rounding is that of the outputs) while their exponentials stay well within
// it, and float64 beyond: the ratio leaves float32 at 88.7, its product with a small
// advantage much later.  (float64 throughout costs 4% where rows are short: 262144
// rows of 1000 bfloat16, loss and gradient, 214 against 206 us.)
constexpr double POLICY_F32 = 64.0;

// (apart, for its registers: inlined it made some 60 row kernels spill)
static __device__ __noinline__ PolicyTerm<double> policy_term_far(double delta, double adv, double lo,
                                                                  double hi, double c, bool has_ref,
                                                                  double d) {
  return policy_term<double>(delta, adv, lo, hi, c, has_ref, d);
}

__device__ __forceinline__ PolicyTerm<double> policy_term_of(double delta, double adv, double lo,
                                                             double hi, double c, bool has_ref,
                                                             double d) {
  if (fabs(delta) <= POLICY_F32 && fabs(d) <= POLICY_F32) {
    const PolicyTerm<float> o = policy_term<float>((float)delta, (float)adv, (float)lo, (float)hi,
                                                   (float)c, has_ref, (float)d);
    return PolicyTerm<double>{o.loss, o.kl, o.slope, o.clipped};
  }
  return policy_term_far(delta, adv, lo, hi, c, has_ref, d);
}

}  // namespace semicrf
