// loss_seq.cu -- what the training losses compute once the rows are done:
// sums over a sequence's positions, the paired loss, and the path forms of
// both (one score per segmentation).
//
//   loss_sums_kernel    a CTA, or a cluster, per sequence: the float64 sums of
//                       the per-position terms in a fixed order; a bad length
//                       goes to the status word, which the row pass cleared.
//   loss_pairs_kernel   a CTA, or a cluster, per pair: S = sum of logp - ref of both
//                       sequences (or its mean), the logistic loss on
//                       u = beta (S_c - S_r) - margin, and the weight of each
//                       sequence's positions for the gradient pass.
//   policy_scores_kernel, preference_scores_kernel   one thread per path or
//                       pair, float64 throughout, like the path scores and
//                       log Z that feed them and take their gradients.
// The arrays are B * T floats against the rows' B * T * V: a few microseconds
// of latency, not bandwidth, is what these cost.
#include <algorithm>

#include "loss.cuh"

namespace semicrf {

namespace {

constexpr int SUM_THREADS = 1024;  // at most
constexpr int SUM_CTAS = 8;        // of a cluster, at most
constexpr int SUM_UNROLL = 8;      // independent loads a thread has in flight

// Threads and CTAs for sequences of T positions: one sweep of the loads covers
// most sequences, and a long one is spread over a cluster (T = 10^6 with one
// CTA of 256 threads, a load at a time, took 0.5 ms).
struct SumShape {
  int threads, ctas;
};
inline SumShape sum_shape(int T) {
  SumShape s{T <= 2048 ? 256 : SUM_THREADS, 1};
  const long long per = (long long)s.threads * SUM_UNROLL;
  s.ctas = (int)std::min<long long>(SUM_CTAS, std::max<long long>(1, (T + per - 1) / per));
  return s;
}

struct SumState {
  double warp[3][SUM_THREADS / 32];
  double cta[SUM_CTAS][3];
};

// Sums of up to three per-position arrays over t < n, split over the CTAs of
// the cluster, in a fixed order; complete in every thread of CTA 0.  `value`:
// (array, position) -> double.  Every thread of every CTA calls it.
template <int N, typename F>
__device__ __forceinline__ void sequence_sums(int n, int T, int* status, int rank, int ctas, SumState& st,
                                              F value, double (&out)[N]) {
  const int threads = blockDim.x, tid = threadIdx.x;
  double s[N] = {};
  for (long long t0 = (long long)rank * threads * SUM_UNROLL + tid; t0 < n;
       t0 += (long long)ctas * threads * SUM_UNROLL) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      double v[SUM_UNROLL];
#pragma unroll
      for (int u = 0; u < SUM_UNROLL; ++u) {
        const long long t = t0 + (long long)u * threads;
        v[u] = t < n && SEMICRF_INB(status, t >= 0 && t < T, SITE_LOSS_SUM) ? value(k, (int)t) : 0.0;
      }
#pragma unroll
      for (int u = 0; u < SUM_UNROLL; ++u) s[k] += v[u];
    }
  }
  __syncthreads();  // the state may still be read from the sums before
#pragma unroll
  for (int k = 0; k < N; ++k) {
    double v = s[k];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    if ((tid & 31) == 0) st.warp[k][tid >> 5] = v;
  }
  __syncthreads();
  if (tid < N && SEMICRF_INB(status, rank >= 0 && rank < ctas && ctas <= SUM_CTAS, SITE_LOSS_SUM)) {
    double v = 0.0;
    for (int i = 0; i < threads / 32; ++i) v += st.warp[tid][i];
    // to CTA 0 of the cluster
    uint32_t to = smem_addr(&st.cta[rank][tid]);
    if (ctas > 1) to = cluster_addr(&st.cta[rank][tid], 0);
    if (ctas > 1) asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(v) : "memory");
    else st.cta[0][tid] = v;
  }
  __syncthreads();
  if (ctas > 1) cluster_sync();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    out[k] = 0.0;
    if (rank == 0)
      for (int i = 0; i < ctas; ++i) out[k] += st.cta[i][k];
  }
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// loss, d loss / d u of the smoothed logistic loss.
__device__ __forceinline__ void logistic(double u, double smoothing, double& loss, double& slope) {
  const double t = exp(-fabs(u)), l = log1p(t);
  const double below = fmax(-u, 0.0) + l, above = fmax(u, 0.0) + l;  // -log sigma(u), -log sigma(-u)
  const double lesser = t / (1.0 + t), greater = 1.0 / (1.0 + t);
  const double sig = u >= 0.0 ? greater : lesser, gis = u >= 0.0 ? lesser : greater;
  // either may be infinite, and a weight of 0 leaves it out
  loss = (smoothing < 1.0 ? (1.0 - smoothing) * below : 0.0) + (smoothing > 0.0 ? smoothing * above : 0.0);
  slope = -(1.0 - smoothing) * gis + smoothing * sig;
  if (u != u) loss = slope = u;
}

}  // namespace

__global__ void __launch_bounds__(SUM_THREADS) loss_sums_kernel(SeqArgs a, int ctas) {
  __shared__ SumState st;
  const int b = blockIdx.x / ctas, rank = blockIdx.x - b * ctas;
  if (ctas > 1) cluster_sync();  // the peers are running
  after_previous();
  const int L = a.lengths[b];
  const bool bad = L < 0 || L > a.T;
  const long long row = (long long)b * a.T;
  double out[3];
  sequence_sums<3>(bad ? 0 : L, a.T, a.status, rank, ctas, st, [&](int k, int t) -> double {
    if (k == 0) return a.sum ? (double)a.tok[row + t] : 0.0;
    if (k == 1) return a.kl_sum ? (double)a.kl[row + t] : 0.0;
    return a.clipped ? (double)a.clip[row + t] : 0.0;
  }, out);
  if (rank != 0 || threadIdx.x != 0) return;
  if (bad) set_status(a.status, ST_BAD_LENGTH);
  if (a.sum) a.sum[b] = bad ? quiet_nan() : (float)out[0];
  if (a.kl_sum) a.kl_sum[b] = bad ? quiet_nan() : (float)out[1];
  if (a.clipped) a.clipped[b] = (int32_t)out[2];
}

__global__ void __launch_bounds__(SUM_THREADS) loss_pairs_kernel(SeqArgs a, int ctas) {
  __shared__ SumState st;
  const int i = blockIdx.x / ctas, rank = blockIdx.x - i * ctas, P = a.B / 2;
  if (ctas > 1) cluster_sync();  // the peers are running
  after_previous();
  double reward[2], inv[2];
  bool off[2];
  for (int side = 0; side < 2; ++side) {
    const int b = i + side * P;
    const int L = a.lengths[b];
    off[side] = L < 0 || L > a.T;
    const long long row = (long long)b * a.T;
    double out[2];
    sequence_sums<2>(off[side] ? 0 : L, a.T, a.status, rank, ctas, st, [&](int k, int t) -> double {
      if (k == 0) return (double)a.tok[row + t];
      return a.average && a.labels[row + t] >= 0 ? 1.0 : 0.0;
    }, out);
    if (ctas > 1) cluster_sync();  // CTA 0 has read the other side's sums
    inv[side] = 1.0 / fmax(out[1], 1.0);
    reward[side] = a.beta * out[0] * inv[side];
  }
  if (rank != 0) return;
  const double u = reward[0] - reward[1] - a.margin;
  // A pair with a malformed sequence has loss NaN and no gradient; one whose loss is
  // NaN for its numbers has a NaN gradient, for whoever looks for that.  A malformed
  // label shows in the sum, so that few pairs have theirs searched.
  bool none = off[0] || off[1];
  if (!none && u != u) {
    int wrong = 0;
    for (int side = 0; side < 2; ++side) {
      const int b = i + side * P, L = a.lengths[b];
      for (int t = threadIdx.x; t < L; t += blockDim.x) wrong |= a.labels[(long long)b * a.T + t] >= a.V;
    }
    none = __syncthreads_or(wrong);
  }
  if (threadIdx.x != 0) return;
  double loss, slope;
  logistic(u, a.smoothing, loss, slope);
  const double w = (a.w ? a.w[i] : 1.0) * a.beta * slope;
  if (off[0] || off[1]) set_status(a.status, ST_BAD_LENGTH);
  if (a.loss) a.loss[i] = none ? quiet_nan() : (float)loss;
  for (int side = 0; side < 2; ++side) {
    const int b = i + side * P;
    if (a.reward) a.reward[b] = off[side] ? quiet_nan() : (float)reward[side];
    a.wseq[b] = none ? 0.0f : (float)(side ? -w * inv[1] : w * inv[0]);
  }
}

__global__ void policy_scores_kernel(const double* __restrict__ logp,
                                     const double* __restrict__ old_logp,
                                     const double* __restrict__ ref, const double* __restrict__ adv,
                                     long long n, double lo, double hi, double c,
                                     const double* __restrict__ w, double* __restrict__ loss,
                                     double* __restrict__ kl, double* __restrict__ grad) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const double lp = logp[i];
  const PolicyTerm<double> o = policy_term<double>(lp - old_logp[i], adv[i], lo, hi, c,
                                                   ref != nullptr, ref ? ref[i] - lp : 0.0);
  if (loss) loss[i] = o.loss;
  if (kl) kl[i] = o.kl;
  if (grad) grad[i] = (w ? w[i] : 1.0) * o.slope;
}

__global__ void preference_scores_kernel(const double* __restrict__ chosen,
                                         const double* __restrict__ rejected,
                                         const double* __restrict__ ref_chosen,
                                         const double* __restrict__ ref_rejected, long long n,
                                         double beta, double margin, double smoothing,
                                         const double* __restrict__ w, double* __restrict__ loss,
                                         double* __restrict__ grad_chosen,
                                         double* __restrict__ grad_rejected) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  double d = chosen[i] - rejected[i];
  if (ref_chosen) d -= ref_chosen[i] - ref_rejected[i];
  double l, slope;
  logistic(beta * d - margin, smoothing, l, slope);
  if (loss) loss[i] = l;
  const double g = (w ? w[i] : 1.0) * beta * slope;
  if (grad_chosen) grad_chosen[i] = g;
  if (grad_rejected) grad_rejected[i] = -g;
}

namespace {

cudaError_t launch_after(void (*kern)(SeqArgs, int), int sequences, const SeqArgs& a,
                         cudaStream_t st) {
  const SumShape shape = sum_shape(a.T);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sequences * shape.ctas);
  cfg.blockDim = dim3(shape.threads);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  cfg.attrs = at;
  if (a.T > 0) at[cfg.numAttrs++] = follows();  // without rows no kernel came before
  if (shape.ctas > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = shape.ctas;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kern, a, shape.ctas);
}

}  // namespace

cudaError_t launch_loss_sums(const SeqArgs& a, cudaStream_t st) {
  return launch_after(loss_sums_kernel, a.B, a, st);
}

cudaError_t launch_loss_pairs(const SeqArgs& a, cudaStream_t st) {
  return launch_after(loss_pairs_kernel, a.B / 2, a, st);
}

cudaError_t launch_policy_scores(const double* logp, const double* old_logp, const double* ref,
                                 const double* adv, long long n, double clip_lo, double clip_hi,
                                 double kl_coef, const double* w, double* loss, double* kl,
                                 double* grad, cudaStream_t st) {
  policy_scores_kernel<<<(unsigned)((n + 127) / 128), 128, 0, st>>>(
      logp, old_logp, ref, adv, n, clip_lo, clip_hi, kl_coef, w, loss, kl, grad);
  return cudaGetLastError();
}

cudaError_t launch_preference_scores(const double* chosen, const double* rejected,
                                     const double* ref_chosen, const double* ref_rejected,
                                     long long n, double beta, double margin, double smoothing,
                                     const double* w, double* loss, double* grad_chosen,
                                     double* grad_rejected, cudaStream_t st) {
  preference_scores_kernel<<<(unsigned)((n + 127) / 128), 128, 0, st>>>(
      chosen, rejected, ref_chosen, ref_rejected, n, beta, margin, smoothing, w, loss, grad_chosen,
      grad_rejected);
  return cudaGetLastError();
}

}  // namespace semicrf
