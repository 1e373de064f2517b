// loss_seq.cu -- what the training losses compute once the rows are done:
// sums over a sequence's positions, the paired loss, and the path forms of
// both (one score per segmentation).
//
//   loss_sums_kernel    one CTA per sequence: the float64 sums of the
//                       per-position terms in a fixed order; a bad length goes
//                       to the status word, which the row pass cleared.
//   loss_pairs_kernel   one CTA per pair: S = sum of logp - ref of both
//                       sequences (or its mean), the logistic loss on
//                       u = beta (S_c - S_r) - margin, and the weight of each
//                       sequence's positions for the gradient pass.
//   policy_scores_kernel, preference_scores_kernel   one thread per path or
//                       pair, float64 throughout, like the path scores and
//                       log Z that feed them and take their gradients.
// The arrays are B * T floats against the rows' B * T * V: a few microseconds
// of latency, not bandwidth, is what these cost.
#include "loss.cuh"

namespace semicrf {

namespace {

constexpr int SUM_THREADS = 256;

__device__ __forceinline__ double warp_sum(double v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
  return v;
}

// Sum over the CTA in a fixed order, in every thread.
__device__ __forceinline__ double cta_sum(double v, double* red) {
  v = warp_sum(v);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < SUM_THREADS / 32; ++i) s += red[i];
  return s;
}

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// loss, d loss / d u of the smoothed logistic loss.
__device__ __forceinline__ void logistic(double u, double smoothing, double& loss, double& slope) {
  const double t = exp(-fabs(u)), l = log1p(t);
  const double below = fmax(-u, 0.0) + l, above = fmax(u, 0.0) + l;  // -log sigma(u), -log sigma(-u)
  const double lesser = t / (1.0 + t), greater = 1.0 / (1.0 + t);
  const double sig = u >= 0.0 ? greater : lesser, gis = u >= 0.0 ? lesser : greater;
  loss = (1.0 - smoothing) * below + (smoothing > 0.0 ? smoothing * above : 0.0);
  slope = -(1.0 - smoothing) * gis + smoothing * sig;
  if (u != u) loss = slope = u;
}

}  // namespace

__global__ void __launch_bounds__(SUM_THREADS) loss_sums_kernel(SeqArgs a) {
  __shared__ double red[SUM_THREADS / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  after_previous();
  const int L = a.lengths[b];
  const bool bad = L < 0 || L > a.T;
  if (bad && tid == 0) set_status(a.status, ST_BAD_LENGTH);
  const int n = bad ? 0 : L;
  const long long row = (long long)b * a.T;
  double s = 0.0, k = 0.0, c = 0.0;
  for (int t = tid; t < n; t += SUM_THREADS) {
    s += (double)a.tok[row + t];
    if (a.kl_sum) k += (double)a.kl[row + t];
    if (a.clipped) c += (double)a.clip[row + t];
  }
  if (a.sum) {
    s = cta_sum(s, red);
    if (tid == 0) a.sum[b] = bad ? quiet_nan() : (float)s;
  }
  if (a.kl_sum) {
    k = cta_sum(k, red);
    if (tid == 0) a.kl_sum[b] = bad ? quiet_nan() : (float)k;
  }
  if (a.clipped) {
    c = cta_sum(c, red);
    if (tid == 0) a.clipped[b] = (int32_t)c;
  }
}

__global__ void __launch_bounds__(SUM_THREADS) loss_pairs_kernel(SeqArgs a) {
  __shared__ double red[SUM_THREADS / 32];
  const int i = blockIdx.x, P = a.B / 2, tid = threadIdx.x;
  after_previous();
  double reward[2], inv[2];
  bool bad = false;
  for (int side = 0; side < 2; ++side) {
    const int b = i + side * P;
    const int L = a.lengths[b];
    const bool off = L < 0 || L > a.T;
    bad |= off;
    if (off && tid == 0) set_status(a.status, ST_BAD_LENGTH);
    const int n = off ? 0 : L;
    const long long row = (long long)b * a.T;
    double s = 0.0, c = 0.0;
    for (int t = tid; t < n; t += SUM_THREADS) {
      s += (double)a.tok[row + t];
      if (a.average) c += a.labels[row + t] >= 0 ? 1.0 : 0.0;
    }
    s = cta_sum(s, red);
    c = a.average ? cta_sum(c, red) : 1.0;
    inv[side] = 1.0 / fmax(c, 1.0);
    reward[side] = a.beta * s * inv[side];
  }
  if (tid != 0) return;
  double loss, slope;
  logistic(reward[0] - reward[1] - a.margin, a.smoothing, loss, slope);
  const double w = (a.w ? a.w[i] : 1.0) * a.beta * slope;
  // a pair with a malformed sequence has loss NaN and no gradient
  const bool none = bad || loss != loss;
  if (a.loss) a.loss[i] = none ? quiet_nan() : (float)loss;
  for (int side = 0; side < 2; ++side) {
    const int b = i + side * P;
    const bool off = a.lengths[b] < 0 || a.lengths[b] > a.T;
    if (a.reward) a.reward[b] = off ? quiet_nan() : (float)reward[side];
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

cudaError_t launch_after(void (*kern)(SeqArgs), int grid, const SeqArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(SUM_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at = follows();
  cfg.attrs = &at;
  cfg.numAttrs = a.T > 0 ? 1 : 0;  // without rows no kernel came before
  return cudaLaunchKernelEx(&cfg, kern, a);
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
