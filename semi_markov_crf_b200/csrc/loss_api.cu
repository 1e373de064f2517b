// loss_api.cu -- the C ABI of the training losses over label scores
// (semicrf.h): argument checks, workspace layout and launches.  Host code only.
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "loss.cuh"
#include "semicrf.h"

namespace semicrf {

size_t loss_layout(int B, int T, void* base, LossWs* p) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = (off + bytes + 255) & ~size_t(255);
    return o;
  };
  const size_t n = (size_t)B * T;
  const size_t o_status = take(256);
  const size_t o_tok = take(n * 4);
  const size_t o_kl = take(n * 4);
  const size_t o_clip = take(n);
  const size_t o_stat = take(n * 8);
  const size_t o_wseq = take((size_t)B * 4);
  if (base && p) {
    char* c = static_cast<char*>(base);
    p->status = reinterpret_cast<int*>(c + o_status);
    p->tok = reinterpret_cast<float*>(c + o_tok);
    p->kl = reinterpret_cast<float*>(c + o_kl);
    p->clip = reinterpret_cast<uint8_t*>(c + o_clip);
    p->stat = reinterpret_cast<float2*>(c + o_stat);
    p->wseq = reinterpret_cast<float*>(c + o_wseq);
  }
  return off;
}

namespace {

int check_sizes(int B, int T) {
  if (B < 0 || T < 0) return SEMICRF_ERR_INVALID_ARG;
  if (B > (1 << 20) || T > (1 << 26) || (long long)B * T > LOSS_ROWS_MAX)
    return SEMICRF_ERR_UNSUPPORTED;
  return SEMICRF_OK;
}

bool is_finite(double v) { return std::isfinite(v); }

// An array of a call; a null or empty one overlaps nothing.
struct Span {
  const void* p;
  size_t bytes;
};

// A row's inputs are read by several warps and CTAs, one of which writes its
// outputs: an output in an input's place would change what the others read.
bool overlap(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span& o : outputs)
    for (const Span& i : inputs) {
      const uintptr_t po = (uintptr_t)o.p, pi = (uintptr_t)i.p;
      if (po && pi && o.bytes && i.bytes && po < pi + i.bytes && pi < po + o.bytes) return true;
    }
  return false;
}

size_t row_bytes(const RowArgs& a, int dtype, int64_t ld) {
  const size_t rows = (size_t)a.B * a.T, es = dtype == SEMICRF_F32 ? 4 : 2;
  return rows ? ((rows - 1) * (size_t)ld + a.V) * es : 0;
}

// The checks every logits form shares, and the arguments they fill.
int prepare_rows(const void* logits, int dtype, int64_t ld, const int32_t* lengths, int B, int T,
                 int V, double temperature, unsigned flags, unsigned known, void* ws,
                 size_t ws_bytes, void* grad_logits, int64_t grad_ld, RowArgs& a, LossWs& p) {
  if (flags & ~known) return SEMICRF_ERR_INVALID_ARG;
  if (dtype < SEMICRF_F32 || dtype > SEMICRF_F16) return SEMICRF_ERR_INVALID_ARG;
  int rc = check_sizes(B, T);
  if (rc) return rc;
  if (V < 1) return SEMICRF_ERR_INVALID_ARG;
  if (V > LOSS_V_MAX) return SEMICRF_ERR_UNSUPPORTED;
  if (!(temperature >= 1e-3 && temperature <= 1e3)) return SEMICRF_ERR_INVALID_ARG;
  const long long rows = (long long)B * T;
  if (!ws || (uintptr_t)ws % 256 || (B > 0 && !lengths)) return SEMICRF_ERR_INVALID_ARG;
  if (rows > 0 && (!logits || ld < V || (grad_logits && grad_ld < V))) return SEMICRF_ERR_INVALID_ARG;
  if (rows > 0 && (ld > INT64_MAX / 4 / rows || (grad_logits && grad_ld > INT64_MAX / 4 / rows)))
    return SEMICRF_ERR_INVALID_ARG;
  const unsigned es = dtype == SEMICRF_F32 ? 4 : 2;
  if ((uintptr_t)logits % es || (uintptr_t)grad_logits % es) return SEMICRF_ERR_INVALID_ARG;
  if ((flags & SEMICRF_FLAG_ACCUMULATE) && dtype != SEMICRF_F32) return SEMICRF_ERR_INVALID_ARG;
  if (ws_bytes < loss_layout(B, T, nullptr, nullptr)) return SEMICRF_ERR_WORKSPACE_TOO_SMALL;
  loss_layout(B, T, ws, &p);
  a = RowArgs{};
  a.x = logits;
  a.g = grad_logits;
  a.ldx = ld;
  a.ldg = grad_ld;
  a.B = B;
  a.T = T;
  a.V = V;
  a.add = (flags & SEMICRF_FLAG_ACCUMULATE) ? 1 : 0;
  a.lengths = lengths;
  a.s = 1.0 / temperature;
  a.tau = temperature;
  a.sl = (float)(LOG2E_D / temperature);
  a.inv_sl = 1.0 / (double)a.sl;
  a.status = p.status;
  return SEMICRF_OK;
}

int run_rows(int mode, int dtype, const RowArgs& a, cudaStream_t st) {
  if (a.T == 0)  // no rows: the pass that clears the status word does not run
    return a.keep_status || cudaMemsetAsync(a.status, 0, sizeof(int), st) == cudaSuccess
               ? SEMICRF_OK
               : SEMICRF_ERR_CUDA;
  LaunchTimer lt("loss_rows_kernel", st);
  return launch_loss_rows(mode, dtype, a, st) == cudaSuccess ? SEMICRF_OK : SEMICRF_ERR_CUDA;
}

// The rows, then the sums over each sequence (which the row pass writes itself
// where a sequence has one position).
int run_rows_and_sums(int mode, int dtype, RowArgs& a, const LossWs& p, float* sum, float* kl_sum,
                      int32_t* clipped, cudaStream_t st) {
  if (a.T == 1) {
    a.single = 1;
    a.seq_sum = sum;
    a.seq_kl = kl_sum;
    a.seq_clipped = clipped;
  }
  const int rc = run_rows(mode, dtype, a, st);
  if (rc || a.single) return rc;
  SeqArgs q{};
  q.B = a.B;
  q.T = a.T;
  q.lengths = a.lengths;
  q.status = p.status;
  q.tok = a.tok;
  q.kl = p.kl;
  q.clip = p.clip;
  q.sum = sum;
  q.kl_sum = kl_sum;
  q.clipped = clipped;
  LaunchTimer lt("loss_sums_kernel", st);
  return launch_loss_sums(q, st) == cudaSuccess ? SEMICRF_OK : SEMICRF_ERR_CUDA;
}

// An empty batch: only the status word is written.
int empty_batch(const LossWs& p, cudaStream_t st) {
  return cudaMemsetAsync(p.status, 0, sizeof(int), st) == cudaSuccess ? SEMICRF_OK
                                                                      : SEMICRF_ERR_CUDA;
}

bool clip_ok(double lo, double hi, double kl) {
  return lo >= 0.0 && lo <= 1.0 && hi >= 0.0 && is_finite(kl);
}

}  // namespace

int loss_sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) {
    cudaGetLastError();
    return 148;  // B200
  }
  return v;
}

namespace {
std::atomic<int> ring_stall{0};
}
int loss_ring_stall() { return ring_stall.load(std::memory_order_relaxed); }

}  // namespace semicrf

using namespace semicrf;

extern "C" int semicrf_loss_workspace_bytes(int B, int T, size_t* bytes) {
  if (!bytes) return SEMICRF_ERR_INVALID_ARG;
  const int rc = check_sizes(B, T);
  if (rc) return rc;
  *bytes = loss_layout(B, T, nullptr, nullptr);
  return SEMICRF_OK;
}

extern "C" int semicrf_selftest_ring_stall(int spins) {
  if (spins < 0) return SEMICRF_ERR_INVALID_ARG;
#ifdef SEMICRF_BOUNDS_CHECK
  ring_stall.store(spins, std::memory_order_relaxed);
  return SEMICRF_OK;
#else
  return SEMICRF_ERR_UNSUPPORTED;  // the release build's rings do not stall on request
#endif
}

extern "C" int semicrf_label_logprob(const void* logits, int dtype, int64_t ld,
                                     const int32_t* lengths, const int32_t* labels, int B, int T,
                                     int V, double temperature, unsigned flags, void* ws,
                                     size_t ws_bytes, const float* grad_logp, float* logp,
                                     float* score, void* grad_logits, int64_t grad_ld,
                                     semicrf_stream_t stream) {
  RowArgs a;
  LossWs p;
  const int rc = prepare_rows(logits, dtype, ld, lengths, B, T, V, temperature, flags,
                              SEMICRF_FLAG_ACCUMULATE, ws, ws_bytes, grad_logits, grad_ld, a, p);
  if (rc) return rc;
  if ((long long)B * T > 0 && !labels) return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return empty_batch(p, st);
  const size_t n = (size_t)B * T * 4;
  if (overlap({{logp, n}, {score, (size_t)B * 4}, {grad_logits, row_bytes(a, dtype, grad_ld)}},
              {{logits, row_bytes(a, dtype, ld)}, {lengths, (size_t)B * 4}, {labels, n}, {grad_logp, n}}))
    return SEMICRF_ERR_INVALID_ARG;
  a.labels = labels;
  a.grad_logp = grad_logp;
  a.logp = logp;
  a.tok = p.tok;
  return run_rows_and_sums(LM_LOGPROB, dtype, a, p, score, nullptr, nullptr, st);
}

extern "C" int semicrf_policy_loss(const void* logits, int dtype, int64_t ld,
                                   const int32_t* lengths, const int32_t* labels, int B, int T,
                                   int V, double temperature, const float* old_logp,
                                   const float* ref_logp, const float* adv, int adv_per_token,
                                   double clip_low, double clip_high, double kl_coef,
                                   unsigned flags, void* ws, size_t ws_bytes,
                                   const double* grad_loss, float* loss, float* kl,
                                   int32_t* clipped, float* logp, void* grad_logits,
                                   int64_t grad_ld, semicrf_stream_t stream) {
  RowArgs a;
  LossWs p;
  const int rc = prepare_rows(logits, dtype, ld, lengths, B, T, V, temperature, flags,
                              SEMICRF_FLAG_ACCUMULATE, ws, ws_bytes, grad_logits, grad_ld, a, p);
  if (rc) return rc;
  if (!clip_ok(clip_low, clip_high, kl_coef)) return SEMICRF_ERR_INVALID_ARG;
  if ((long long)B * T > 0 && (!labels || !old_logp || !adv)) return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return empty_batch(p, st);
  const size_t n = (size_t)B * T * 4, nb = (size_t)B * 4;
  if (overlap({{logp, n}, {loss, nb}, {kl, nb}, {clipped, nb}, {grad_logits, row_bytes(a, dtype, grad_ld)}},
              {{logits, row_bytes(a, dtype, ld)}, {lengths, nb}, {labels, n}, {old_logp, n}, {ref_logp, n},
               {adv, adv_per_token ? n : nb}, {grad_loss, 2 * nb}}))
    return SEMICRF_ERR_INVALID_ARG;
  a.labels = labels;
  a.old_logp = old_logp;
  a.ref_logp = ref_logp;
  a.adv = adv;
  a.adv_tok = adv_per_token ? 1 : 0;
  a.clip_lo = 1.0 - clip_low;
  a.clip_hi = 1.0 + clip_high;
  a.kl_coef = kl_coef;
  a.w = grad_loss;
  a.logp = logp;
  a.tok = p.tok;
  a.kl = kl ? p.kl : nullptr;
  a.clip = clipped ? p.clip : nullptr;
  return run_rows_and_sums(LM_POLICY, dtype, a, p, loss, kl, clipped, st);
}

extern "C" int semicrf_preference_loss(const void* logits, int dtype, int64_t ld,
                                       const int32_t* lengths, const int32_t* labels, int B, int T,
                                       int V, double temperature, const float* ref_logp,
                                       double beta, double margin, double smoothing,
                                       unsigned flags, void* ws, size_t ws_bytes,
                                       const double* grad_loss, float* loss, float* reward,
                                       float* logp, void* grad_logits, int64_t grad_ld,
                                       semicrf_stream_t stream) {
  RowArgs a;
  LossWs p;
  const int rc =
      prepare_rows(logits, dtype, ld, lengths, B, T, V, temperature, flags,
                   SEMICRF_FLAG_ACCUMULATE | SEMICRF_FLAG_AVERAGE, ws, ws_bytes, grad_logits,
                   grad_ld, a, p);
  if (rc) return rc;
  if (B % 2 || !is_finite(beta) || !is_finite(margin) || !(smoothing >= 0.0 && smoothing <= 1.0))
    return SEMICRF_ERR_INVALID_ARG;
  if ((long long)B * T > 0 && !labels) return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return empty_batch(p, st);
  const size_t n = (size_t)B * T * 4, nb = (size_t)B * 4;
  if (overlap({{logp, n}, {loss, nb / 2}, {reward, nb}, {grad_logits, row_bytes(a, dtype, grad_ld)}},
              {{logits, row_bytes(a, dtype, ld)}, {lengths, nb}, {labels, n}, {ref_logp, n}, {grad_loss, nb}}))
    return SEMICRF_ERR_INVALID_ARG;
  a.labels = labels;
  a.ref_logp = ref_logp;
  a.logp = logp;
  a.tok = p.tok;
  a.stat = p.stat;
  a.wseq = p.wseq;
  const int rr = run_rows(LM_PREFERENCE, dtype, a, st);
  if (rr) return rr;
  SeqArgs q{};
  q.B = B;
  q.T = T;
  q.lengths = lengths;
  q.labels = labels;
  q.V = V;
  q.status = p.status;
  q.tok = p.tok;
  q.beta = beta;
  q.margin = margin;
  q.smoothing = smoothing;
  q.average = (flags & SEMICRF_FLAG_AVERAGE) ? 1 : 0;
  q.w = grad_loss;
  q.loss = loss;
  q.reward = reward;
  q.wseq = p.wseq;
  {
    LaunchTimer lt("loss_pairs_kernel", st);
    if (launch_loss_pairs(q, st) != cudaSuccess) return SEMICRF_ERR_CUDA;
  }
  if (!grad_logits) return SEMICRF_OK;
  a.keep_status = 1;
  return run_rows(LM_SCALED, dtype, a, st);
}

extern "C" int semicrf_distill_loss(const void* logits, int dtype, int64_t ld,
                                    const int32_t* lengths, const int32_t* teacher_ids,
                                    const float* teacher_logits, const float* teacher_lse, int k,
                                    int B, int T, int V, double temperature, unsigned flags,
                                    void* ws, size_t ws_bytes, const double* grad_loss,
                                    float* loss, float* token_loss, void* grad_logits,
                                    int64_t grad_ld, semicrf_stream_t stream) {
  RowArgs a;
  LossWs p;
  const int rc = prepare_rows(logits, dtype, ld, lengths, B, T, V, temperature, flags,
                              SEMICRF_FLAG_ACCUMULATE, ws, ws_bytes, grad_logits, grad_ld, a, p);
  if (rc) return rc;
  if (k < 1) return SEMICRF_ERR_INVALID_ARG;
  if (k > LOSS_K_MAX) return SEMICRF_ERR_UNSUPPORTED;
  if ((long long)B * T > 0 && (!teacher_ids || !teacher_logits)) return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return empty_batch(p, st);
  const size_t n = (size_t)B * T * 4, nb = (size_t)B * 4;
  if (overlap({{token_loss, n}, {loss, nb}, {grad_logits, row_bytes(a, dtype, grad_ld)}},
              {{logits, row_bytes(a, dtype, ld)}, {lengths, nb}, {teacher_ids, n * k},
               {teacher_logits, n * k}, {teacher_lse, n}, {grad_loss, 2 * nb}}))
    return SEMICRF_ERR_INVALID_ARG;
  a.ids = teacher_ids;
  a.tl = teacher_logits;
  a.tlse = teacher_lse;
  a.k = k;
  a.w = grad_loss;
  a.tok = token_loss ? token_loss : p.tok;
  return run_rows_and_sums(LM_DISTILL, dtype, a, p, loss, nullptr, nullptr, st);
}

extern "C" int semicrf_policy_scores(const double* logp, const double* old_logp,
                                     const double* ref_logp, const double* adv, int N,
                                     double clip_low, double clip_high, double kl_coef,
                                     const double* grad_loss, double* loss, double* kl,
                                     double* grad_logp, semicrf_stream_t stream) {
  if (N < 0 || !clip_ok(clip_low, clip_high, kl_coef)) return SEMICRF_ERR_INVALID_ARG;
  if (N == 0) return SEMICRF_OK;
  if (!logp || !old_logp || !adv) return SEMICRF_ERR_INVALID_ARG;
  const size_t n = (size_t)N * 8;
  if (overlap({{loss, n}, {kl, n}, {grad_logp, n}},
              {{logp, n}, {old_logp, n}, {ref_logp, n}, {adv, n}, {grad_loss, n}}))
    return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchTimer lt("policy_scores_kernel", st);
  return launch_policy_scores(logp, old_logp, ref_logp, adv, N, 1.0 - clip_low, 1.0 + clip_high,
                              kl_coef, grad_loss, loss, kl, grad_logp, st) == cudaSuccess
             ? SEMICRF_OK
             : SEMICRF_ERR_CUDA;
}

extern "C" int semicrf_preference_scores(const double* chosen, const double* rejected,
                                         const double* ref_chosen, const double* ref_rejected,
                                         int N, double beta, double margin, double smoothing,
                                         const double* grad_loss, double* loss,
                                         double* grad_chosen, double* grad_rejected,
                                         semicrf_stream_t stream) {
  if (N < 0 || !is_finite(beta) || !is_finite(margin) || !(smoothing >= 0.0 && smoothing <= 1.0))
    return SEMICRF_ERR_INVALID_ARG;
  if ((ref_chosen == nullptr) != (ref_rejected == nullptr)) return SEMICRF_ERR_INVALID_ARG;
  if (N == 0) return SEMICRF_OK;
  if (!chosen || !rejected) return SEMICRF_ERR_INVALID_ARG;
  const size_t n = (size_t)N * 8;
  if (overlap({{loss, n}, {grad_chosen, n}, {grad_rejected, n}},
              {{chosen, n}, {rejected, n}, {ref_chosen, n}, {ref_rejected, n}, {grad_loss, n}}))
    return SEMICRF_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  LaunchTimer lt("preference_scores_kernel", st);
  return launch_preference_scores(chosen, rejected, ref_chosen, ref_rejected, N, beta, margin,
                                  smoothing, grad_loss, loss, grad_chosen, grad_rejected,
                                  st) == cudaSuccess
             ? SEMICRF_OK
             : SEMICRF_ERR_CUDA;
}
