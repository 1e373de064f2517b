// loss_rows.cu -- one pass over rows of label scores: the log-sum-exp of a
// row, the loss term of its position and the gradient row.
//
// With z = x / temperature, q = softmax(z) and lse = log sum exp z:
//   label losses   logp = z_y - lse;  d logp / d x_v = ([v = y] - q_v) / temperature
//                  so a position with d loss / d logp = a gets the row
//                  a / temperature * ([v = y] - q_v)
//   distillation   p_j over the teacher's entries j (labels id_j):
//                  loss = temperature^2 * sum_j p_j (log p_j - log q_{id_j});
//                  row  = temperature * (P q_v - sum_{j: id_j = v} p_j),  P = sum_j p_j
//
// A position costs one read of its V scores, and one write of V gradient
// entries: bytes bound it (about five float32 operations and one exponential
// an element).  Sums of exponentials are float32 relative to the running
// maximum, which is kept in the scores' own units so that rows masked with
// the type's lowest value still have a softmax; what follows from them for a
// position (logp, the ratio, the loss) is float64 or exact differences.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "loss.cuh"

namespace semicrf {

namespace {

// ------------------------------------------------------------------ elements
template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

// ------------------------------------------------------- exponentials of a row
// 2^((x - m) sl): the product m sl is taken once and its rounding error put
// back as a factor (unshift), so that an element costs one fused multiply-add
// and one ex2.  Where m sl leaves float32's range (a row whose scores all sit
// at the type's lowest value) the difference is taken first.
struct Shift {
  float m, mb, unshift;
  bool direct;  // m sl is finite
};

__device__ __forceinline__ Shift make_shift(float m, float sl) {
  Shift h;
  h.m = m == NEG_INF ? 0.0f : m;  // no element above -inf: every exponential is 0
  h.mb = h.m * sl;
  h.direct = fabsf(h.mb) <= 3.402823466e38f;
  h.unshift = h.direct ? ex2(-fmaf(h.m, sl, -h.mb)) : 1.0f;
  return h;
}

__device__ __forceinline__ float shifted_exp(float x, float sl, const Shift& h) {
  return ex2(h.direct ? fmaf(x, sl, -h.mb) : (x - h.m) * sl);
}

// log S for S = 1 .. V: exponent and mantissa apart, so that the error is that
// of log2 on [1, 2) whatever V is.
__device__ __forceinline__ double log_of_sum(float S) {
  if (!(S > 0.0f && S <= 3.402823466e38f)) return (double)logf(S);
  const int bits = __float_as_int(S);
  const float mant = __int_as_float((bits & 0x007fffff) | 0x3f800000);
  return LN2_D * ((double)((bits >> 23) - 127) + (double)log2f(mant));
}

// ------------------------------------------------------------ rows in memory
template <typename T>
__device__ __forceinline__ T* row_at(const void* base, long long r, long long ld) {
  return static_cast<T*>(const_cast<void*>(base)) + r * ld;
}

// A row's head: whether its position counts, its label.
struct Head {
  int b;
  bool live;       // counts: the row is read and the loss term computed
  bool malformed;  // counts, but a label lies outside [0, V)
  int y;
};

template <int MODE>
__device__ __forceinline__ Head row_head(const RowArgs& a, long long r) {
  Head h;
  h.b = (int)(r / a.T);
  const int t = (int)(r - (long long)h.b * a.T);
  const int L = a.lengths[h.b];
  h.live = L <= a.T && t < L;
  h.malformed = false;
  h.y = -1;
  if (MODE != LM_DISTILL && h.live) {
    h.y = a.labels[r];
    h.live = h.y >= 0;
    h.malformed = h.y >= a.V;
  }
  return h;
}

// The outputs of a position that does not count, or whose labels are malformed.
template <int MODE>
__device__ __forceinline__ void blank_outputs(const RowArgs& a, long long r, bool malformed) {
  const float v = malformed ? quiet_nan() : 0.0f;
  if (a.tok) a.tok[r] = v;
  if (MODE != LM_DISTILL && a.logp) a.logp[r] = v;
  if (MODE == LM_POLICY) {
    if (a.kl) a.kl[r] = v;
    if (a.clip) a.clip[r] = 0;
  }
}

// What follows from a row's maximum M and sum S for a label loss: the
// position's outputs (written by one thread) and a = d loss / d logp / temperature.
template <int MODE>
__device__ __forceinline__ float label_outputs(const RowArgs& a, long long r, int b, float xy,
                                               float M, float S, bool writer) {
  const double logp = ((double)xy - (double)M) * a.s - log_of_sum(S);
  float slope = 0.0f;
  float term = (float)logp;
  if (MODE == LM_LOGPROB) slope = a.grad_logp ? a.grad_logp[r] : 1.0f;
  if (MODE == LM_PREFERENCE) term = (float)(a.ref_logp ? logp - (double)a.ref_logp[r] : logp);
  if (MODE == LM_POLICY) {
    const float adv = a.adv[a.adv_tok ? r : (long long)b];
    const PolicyTerm<float> o = policy_term<float>(
        (float)(logp - (double)a.old_logp[r]), adv, (float)a.clip_lo, (float)a.clip_hi,
        (float)a.kl_coef, a.ref_logp != nullptr,
        a.ref_logp ? (float)((double)a.ref_logp[r] - logp) : 0.0f);
    term = o.loss;
    slope = o.slope;
    if (writer) {
      if (a.kl) a.kl[r] = o.kl;
      if (a.clip) a.clip[r] = o.clipped;
    }
  }
  if (writer) {
    if (a.tok) a.tok[r] = term;
    if (a.logp) a.logp[r] = (float)logp;
    if (MODE == LM_PREFERENCE) a.stat[r] = make_float2(M, S);
  }
  return (float)((a.w ? a.w[b] : 1.0) * (double)slope * a.s);
}

// --------------------------------------------------------- reductions in a CTA
constexpr int LT = 256;  // threads of the looping kernel

// (m, s) of the CTA's threads -> the row's maximum and sum, in every thread.
// `red`: one float2 per warp.
__device__ __forceinline__ void cta_softmax(float& m, float& s, float sl, float2* red) {
  const float wm = group_max(m, 32);
  s = group_sum(m == NEG_INF && s == 0.0f ? 0.0f : s * ex2((m - wm) * sl), 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(wm, s);
  __syncthreads();
  float M = NEG_INF;
  for (int i = 0; i < LT / 32; ++i) M = fmaxf(M, red[i].x);
  float S = 0.0f;
  for (int i = 0; i < LT / 32; ++i) {
    const float2 v = red[i];
    S += v.x == NEG_INF && v.y == 0.0f ? 0.0f : v.y * ex2((v.x - M) * sl);
  }
  m = M;
  s = M == NEG_INF ? quiet_nan() : S;  // nothing but -inf: no distribution
}

__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = group_sum(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < LT / 32; ++i) s += red[i];
  return s;
}

__device__ __forceinline__ float cta_max(float v, float* red) {
  v = group_max(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = NEG_INF;
  for (int i = 0; i < LT / 32; ++i) s = fmaxf(s, red[i]);
  return s;
}

// ------------------------------------------------------- any V, any alignment
// One CTA per row, elements strided over its threads; the row is read twice
// (the second time mostly from L2).
template <typename T, int MODE>
__global__ void __launch_bounds__(LT) loss_loop_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float2 red2[LT / 32];
  __shared__ float red[LT / 32];
  __shared__ float pj[MODE == LM_DISTILL ? LOSS_K_MAX : 1];
  __shared__ int idj[MODE == LM_DISTILL ? LOSS_K_MAX : 1];
  __shared__ float oldg[MODE == LM_DISTILL ? LOSS_K_MAX : 1];
  const long long r = blockIdx.x;
  const int tid = threadIdx.x, V = a.V;
  Head h = row_head<MODE>(a, r);
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = a.g ? row_at<T>(a.g, r, a.ldg) : nullptr;

  float P = 0.0f, tm = 0.0f, tlog = 0.0f;
  if (MODE == LM_DISTILL && h.live) {
    // the teacher's probabilities over the entries in use
    const float st = (float)a.s;
    bool out = false;
    float m = NEG_INF;
    for (int j = tid; j < a.k; j += LT) {
      const int id = a.ids[r * a.k + j];
      const float t = id >= 0 ? a.tl[r * a.k + j] : NEG_INF;
      out |= id >= V;
      idj[j] = id;
      pj[j] = t;
      m = fmaxf(m, t);
    }
    h.malformed = __syncthreads_or(out);
    m = cta_max(m, red);
    const float m0 = m == NEG_INF ? 0.0f : m;
    float s = 0.0f;
    for (int j = tid; j < a.k; j += LT)
      if (idj[j] >= 0) s += expf((pj[j] - m0) * st);
    s = cta_sum(s, red);
    tm = m0;
    if (a.tlse) {
      tlog = (float)((double)a.tlse[r] - (double)m0 * a.s);
      P = s * expf(-tlog);
    } else {
      tlog = logf(s);
      P = s > 0.0f ? 1.0f : s;  // no entry with a probability: no loss, no gradient
    }
  }

  if (!h.live || h.malformed) {
    if (tid == 0) blank_outputs<MODE>(a, r, h.live);
    if (g && !a.add)
      for (int v = tid; v < V; v += LT) g[v] = from_f32<T>(0.0f);
    return;
  }

  // the row's maximum and sum of exponentials, in one pass
  float m = NEG_INF, s = 0.0f;
  for (int v = tid; v < V; v += LT) {
    const float xv = to_f32<T>(x[v]);
    if (xv > m) {
      s *= ex2((m - xv) * a.sl);
      m = xv;
    }
    s += ex2((xv - (m == NEG_INF ? 0.0f : m)) * a.sl);
  }
  cta_softmax(m, s, a.sl, red2);

  float cq, cy = 0.0f;  // gradient of the row: cq q_v, and cy more at the label
  if (MODE == LM_DISTILL) {
    const double logS = log_of_sum(s);
    float part = 0.0f;
    for (int j = tid; j < a.k; j += LT) {
      const int id = idj[j];
      float p = 0.0f;
      if (id >= 0 && pj[j] != NEG_INF) {
        const float lt = (float)((double)(pj[j] - tm) * a.s - (double)tlog);
        p = expf(lt);
        const float lq = (float)(((double)to_f32<T>(x[id]) - (double)m) * a.s - logS);
        if (p != 0.0f) part += p * (lt - lq);
      }
      if (id >= 0 && a.add && g) oldg[j] = to_f32<T>(g[id]);
      pj[j] = p;
    }
    part = cta_sum(part, red);  // pj is complete behind its barriers
    const double tau = 1.0 / a.s;
    if (tid == 0) a.tok[r] = (float)(tau * tau * (double)part);
    cq = (float)((a.w ? a.w[h.b] : 1.0) * tau);
  } else {
    const float c = label_outputs<MODE>(a, r, h.b, to_f32<T>(x[h.y]), m, s, tid == 0);
    cq = -c;
    cy = c;
  }
  if (!g || MODE == LM_PREFERENCE) return;

  const Shift hs = make_shift(m, a.sl);
  const float scale = hs.unshift / s * cq * (MODE == LM_DISTILL ? P : 1.0f);
  for (int v = tid; v < V; v += LT) {
    float gv = shifted_exp(to_f32<T>(x[v]), a.sl, hs) * scale;
    if (MODE != LM_DISTILL && v == h.y) gv += cy;
    if (a.add) gv += to_f32<T>(g[v]);
    g[v] = from_f32<T>(gv);
  }
  if (MODE == LM_DISTILL) {
    __syncthreads();  // the row is written; its teacher entries follow
    for (int j = tid; j < a.k; j += LT) {
      const int id = idj[j];
      if (id < 0) continue;
      // the first of equal labels takes the sum over them, in order
      bool first = true;
      float p = 0.0f;
      for (int i = 0; i < a.k; ++i) {
        if (idj[i] != id) continue;
        if (i < j) first = false;
        p += pj[i];
      }
      if (!first) continue;
      float gv = shifted_exp(to_f32<T>(x[id]), a.sl, hs) * scale - cq * p;
      if (a.add) gv += oldg[j];
      g[id] = from_f32<T>(gv);
    }
  }
}

// The gradient pass of the preference loss, from the statistics of its first
// pass: one read of the row, one write.
template <typename T>
__global__ void __launch_bounds__(LT) loss_scaled_kernel(const __grid_constant__ RowArgs a) {
  const long long r = blockIdx.x;
  const int tid = threadIdx.x, V = a.V;
  const Head h = row_head<LM_PREFERENCE>(a, r);
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = row_at<T>(a.g, r, a.ldg);
  const float w = a.wseq[h.b];
  // a weight of zero writes zeros: a malformed pair has no gradient
  if (!h.live || h.malformed || w == 0.0f) {
    if (!a.add)
      for (int v = tid; v < V; v += LT) g[v] = from_f32<T>(0.0f);
    return;
  }
  const float2 st = a.stat[r];
  const float c = (float)((double)w * a.s);
  const Shift hs = make_shift(st.x, a.sl);
  const float scale = -hs.unshift / st.y * c;
  for (int v = tid; v < V; v += LT) {
    float gv = shifted_exp(to_f32<T>(x[v]), a.sl, hs) * scale;
    if (v == h.y) gv += c;
    if (a.add) gv += to_f32<T>(g[v]);
    g[v] = from_f32<T>(gv);
  }
}

template <typename T>
cudaError_t rows_of(int mode, const RowArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((long long)a.B * a.T);
  switch (mode) {
    case LM_LOGPROB: loss_loop_kernel<T, LM_LOGPROB><<<grid, LT, 0, st>>>(a); break;
    case LM_POLICY: loss_loop_kernel<T, LM_POLICY><<<grid, LT, 0, st>>>(a); break;
    case LM_PREFERENCE: loss_loop_kernel<T, LM_PREFERENCE><<<grid, LT, 0, st>>>(a); break;
    default: loss_loop_kernel<T, LM_DISTILL><<<grid, LT, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_loss_rows(int mode, int type, const RowArgs& a, cudaStream_t st) {
  switch (type) {
    case LT_BF16: return rows_of<__nv_bfloat16>(mode, a, st);
    case LT_F16: return rows_of<__half>(mode, a, st);
    default: return rows_of<float>(mode, a, st);
  }
}

cudaError_t launch_loss_scaled(int type, const RowArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((long long)a.B * a.T);
  switch (type) {
    case LT_BF16: loss_scaled_kernel<__nv_bfloat16><<<grid, LT, 0, st>>>(a); break;
    case LT_F16: loss_scaled_kernel<__half><<<grid, LT, 0, st>>>(a); break;
    default: loss_scaled_kernel<float><<<grid, LT, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace semicrf
