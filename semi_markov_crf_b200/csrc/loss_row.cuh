// loss_row.cuh -- one pass over rows of label scores: the log-sum-exp of a
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
// an element).  Sums of exponentials are float32 around the row's maximum;
// what follows from them for a position (logp, the ratio, the loss) is float64
// or small differences, rounded once.
//
// By length of the row: loss_lanes.cuh (to 2048 scores, lane groups),
// loss_cta.cuh (to 8192, a CTA a row), loss_ring.cuh (persistent CTAs and
// clusters), loss_wide.cuh (what a cluster does not hold).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

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
// Exponentials are taken in base 2 around the row's scaled maximum mb = m sl
// (sl = log2(e) / temperature): 2^(x sl - mb), one fused multiply-add and one
// ex2 an element.  mb is rounded, and the product in the fused operation is
// not: the greatest exponent is mb's rounding error, at most 1 up to BASE_MAX,
// but beyond 2^31 enough to overflow (a row of nothing but a mask's -1e30).
// There, and where m sl leaves float32, they are 2^((x - m) sl) instead.
struct Base {
  float at;     // mb, or m where not direct
  bool direct;
};

constexpr float F32_MAX = 3.402823466e38f;
constexpr float BASE_MAX = 16777216.0f;  // 2^24: half a step there is 1

__device__ __forceinline__ Base make_base(float m, float sl) {
  const float mb = m * sl;
  Base h;
  h.direct = fabsf(mb) <= BASE_MAX;
  h.at = h.direct ? mb : m;
  return h;
}

__device__ __forceinline__ float based_exp(float x, float sl, const Base& h) {
  return ex2(h.direct ? fmaf(x, sl, -h.at) : (x - h.at) * sl);
}

// The base in the scores' units.  sl is rounded to float32; taking the base
// over that same factor keeps its error out of the dominant terms of the sum.
__device__ __forceinline__ double base_score(const Base& h, double inv_sl) {
  return h.direct ? (double)h.at * inv_sl : (double)h.at;
}

// (base, sum) of a row in one float2: a sum is positive, so its sign tells which base it is.
__device__ __forceinline__ float2 pack_stat(const Base& h, float S) {
  return make_float2(h.at, h.direct ? S : -S);
}
__device__ __forceinline__ Base unpack_stat(float2 v, float& S) {
  Base h;
  h.at = v.x;
  h.direct = !signbit(v.y);
  S = h.direct ? v.y : -v.y;
  return h;
}

// log S for S = 1 .. V: exponent and mantissa apart, so that the error is that
// of log2 on [1, 2) whatever V is.
__device__ __forceinline__ double log_of_sum(float S) {
  if (!(S > 0.0f && S <= F32_MAX)) return (double)logf(S);
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
  bool malformed;  // counts, but the label lies outside [0, V)
  int y;
};

// The two loads behind a head, so that they can be issued a row ahead.
struct HeadLoad {
  int b, t, L, y;
};

constexpr bool has_label(int mode) { return mode != LM_DISTILL; }

template <int MODE>
__device__ __forceinline__ HeadLoad load_head(const RowArgs& a, long long r) {
  HeadLoad l;
  l.b = (int)((unsigned)r / (unsigned)a.T);  // r < 2^27
  l.t = (int)r - l.b * a.T;
  l.L = a.lengths[l.b];
  l.y = has_label(MODE) ? a.labels[r] : 0;
  return l;
}

template <int MODE>
__device__ __forceinline__ Head make_head(const RowArgs& a, const HeadLoad& l) {
  Head h;
  h.b = l.b;
  h.live = l.L <= a.T && l.t < l.L && l.y >= 0;
  h.y = l.y;
  h.malformed = has_label(MODE) && h.live && l.y >= a.V;
  return h;
}

// The per-position inputs of a label loss, loaded when its row starts.
template <typename T>
struct LabelIn {
  T score;  // of the label, as loaded: converting it would wait for it
  float slope, old_logp, ref_logp, adv;
  float lse;    // LM_DISTILL: the teacher's
  float2 stat;  // LM_SCALED
  double w;
  __device__ float xy() const { return to_f32<T>(score); }
};

template <typename T, int MODE>
__device__ __forceinline__ LabelIn<T> load_label(const RowArgs& a, long long r, const Head& h,
                                              const T* x) {
  LabelIn<T> in{};
  in.w = 1.0;
  if (a.w) in.w = a.w[h.b];
  if (MODE == LM_DISTILL && a.tlse) in.lse = a.tlse[r];
  if (MODE == LM_SCALED) in.stat = a.stat[r];
  if (!has_label(MODE)) return in;
  if (SEMICRF_INB(a.status, h.y >= 0 && h.y < a.V, SITE_LOSS_SCORE)) in.score = x[h.y];
  if (MODE == LM_LOGPROB) in.slope = a.grad_logp ? a.grad_logp[r] : 1.0f;
  if (MODE == LM_PREFERENCE || MODE == LM_POLICY) in.ref_logp = a.ref_logp ? a.ref_logp[r] : 0.0f;
  if (MODE == LM_POLICY) {
    in.old_logp = a.old_logp[r];
    in.adv = a.adv[a.adv_tok ? r : (long long)h.b];
  }
  return in;
}

// The pass starts with a clear status word.  With one position a sequence there
// is no pass over the sequences that would look at the lengths, so the first
// CTA does.  Called by all threads of every CTA.
__device__ __forceinline__ void start_status(const RowArgs& a) {
  if (blockIdx.x != 0 || !a.status || a.keep_status) return;
  int bad = 0;
  if (a.single)
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) bad |= a.lengths[b] < 0 || a.lengths[b] > a.T;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = bad ? ST_BAD_LENGTH : 0;
}

// A position's term, and its sequence's sum where that is all of it.
__device__ __forceinline__ void put_term(const RowArgs& a, long long r, float v) {
  if (a.tok) a.tok[r] = v;
  if (a.single && a.seq_sum) a.seq_sum[r] = v;
}
__device__ __forceinline__ void put_policy(const RowArgs& a, long long r, float kl, bool clipped) {
  if (a.kl) a.kl[r] = kl;
  if (a.clip) a.clip[r] = clipped;
  if (a.single && a.seq_kl) a.seq_kl[r] = kl;
  if (a.single && a.seq_clipped) a.seq_clipped[r] = clipped;
}

// The outputs of a position that does not count, or whose labels are malformed.
template <int MODE>
__device__ __forceinline__ void blank_outputs(const RowArgs& a, long long r, bool malformed) {
  float v = malformed ? quiet_nan() : 0.0f;
  if (has_label(MODE) && a.logp) a.logp[r] = v;
  if (MODE == LM_DISTILL && a.tok) a.tok[r] = v;
  if (a.single && (a.lengths[r] < 0 || a.lengths[r] > a.T)) v = quiet_nan();
  if (MODE == LM_DISTILL) {
    if (a.single && a.seq_sum) a.seq_sum[r] = v;
  } else {
    put_term(a, r, v);
  }
  if (MODE == LM_POLICY) put_policy(a, r, v, false);
}

// What follows from a row's base and sum for a label loss: the position's
// outputs (written by one thread) and d loss / d logp / temperature.
template <int MODE, typename T>
__device__ __forceinline__ float label_outputs(const RowArgs& a, long long r, const LabelIn<T>& in,
                                               const Base& h, float S, bool writer) {
  const double logp = ((double)in.xy() - base_score(h, a.inv_sl)) * a.s - log_of_sum(S);
  double slope = (double)in.slope;
  float term = (float)logp;
  if (MODE == LM_PREFERENCE) term = (float)(logp - (double)in.ref_logp);
  if (MODE == LM_POLICY) {
    const bool has_ref = a.ref_logp != nullptr;
    const PolicyTerm<double> o =
        policy_term_of(logp - (double)in.old_logp, (double)in.adv, a.clip_lo, a.clip_hi, a.kl_coef,
                       has_ref, has_ref ? (double)in.ref_logp - logp : 0.0);
    term = (float)o.loss;
    slope = o.slope;
    if (writer) put_policy(a, r, (float)o.kl, o.clipped);
  }
  if (writer) {
    put_term(a, r, term);
    if (a.logp) a.logp[r] = (float)logp;
    if (MODE == LM_PREFERENCE) a.stat[r] = pack_stat(h, S);
  }
  return (float)(in.w * slope * a.s);
}

// ------------------------------------------------------ the teacher's entries
// Kept in shared memory by the lanes that look after them.
struct Teacher {
  float* p;    // [k] logits, then probabilities
  int* id;     // [k]
  float* x;    // [k] the row's scores at those labels
  float* old;  // [k] the gradient's value before this call (accumulation)
  int* table;  // [teacher_table(k, V)] scratch
};

constexpr int TEACHER_WORDS = 4;

// Words of scratch that tell whether a label comes twice: a bit a label of the
// row or, where that is shorter, a hash table.  None for short lists, whose
// entries are compared with one another.  (75480 rows of 627 bfloat16: 16 entries
// 81 us compared, 66 with bits; 133 entries 128 us in a table, 110 with bits.)
constexpr int TEACHER_SHORT = 16, TEACHER_FEW = 4;
constexpr int TEACHER_FEW_BITS = 64;  // words of bits that are cheaper than comparing
__host__ __device__ inline int teacher_bits(int V) { return (V + 31) / 32; }
__host__ __device__ inline int teacher_table(int k, int V) {
  const int bits = teacher_bits(V);
  if (k <= (bits <= TEACHER_FEW_BITS ? TEACHER_FEW : TEACHER_SHORT)) return 0;
  int n = 64;
  while (n < 2 * k) n *= 2;
  return bits < n ? bits : n;
}

// A label's first slot in the table: the high bits of a multiplicative hash, so
// that labels with equal low bits spread too.
__device__ __forceinline__ unsigned teacher_slot(int id, int size) {
  return (unsigned)id * 2654435769u >> (__clz(size) + 1);
}

__device__ __forceinline__ void teacher_clear(int* table, int size, int V, int lane, int n) {
  const int none = size == teacher_bits(V) ? 0 : -1;
  for (int i = lane; i < size; i += n) table[i] = none;
}

// Whether the label was there; it is from now on.  (A hash table is at least half
// empty, so that every probe ends.)
__device__ __forceinline__ bool teacher_again(const RowArgs& a, int* table, int size, int V, int id) {
  if (size == teacher_bits(V)) {
    if (!SEMICRF_INB(a.status, id >= 0 && id >> 5 < size, SITE_LOSS_ENTRY)) return false;
    const unsigned bit = 1u << (id & 31);
    return atomicOr(reinterpret_cast<unsigned*>(&table[id >> 5]), bit) & bit;
  }
  if (!SEMICRF_INB(a.status, size >= 2 && (size & (size - 1)) == 0, SITE_LOSS_ENTRY)) return false;
  for (unsigned at = teacher_slot(id, size);; ++at) {
    const int was = atomicCAS(&table[at & (size - 1)], -1, id);
    if (was == -1 || was == id) return was == id;
  }
}

struct TeacherHead {
  float tm, pT, P;
  double tlog;
  bool malformed;
  bool none;     // no entry has a probability: no loss and no gradient
  bool repeats;  // two entries may have the same label
};

// The elements of a row that a CTA writes: [lo, hi) and those from `tail` on.
struct Range {
  int lo, hi, tail;
  __device__ bool has(int i) const { return i >= lo && (i < hi || i >= tail); }
};

// Max and sum over aligned groups of n lanes, of which `mm` is this one's.
__device__ __forceinline__ float lanes_max(float v, int n, unsigned mm) {
  for (int o = n >> 1; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mm, v, o));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int n, unsigned mm) {
  for (int o = n >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(mm, v, o);
  return v;
}

// The first TEACHER_AHEAD entries of each lane, loaded before they are needed.
constexpr int TEACHER_AHEAD = 4;
template <int U>
struct TeacherLoad {
  int id[U];
  float t[U];
  __device__ __forceinline__ void load(const RowArgs& a, long long r, int from, int lane, int n) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = from + u * n + lane;
      id[u] = j < a.k ? a.ids[r * a.k + j] : -1;
      t[u] = j < a.k ? a.tl[r * a.k + j] : NEG_INF;
    }
  }
};
using TeacherAhead = TeacherLoad<TEACHER_AHEAD>;

// Total probability of a teacher whose greatest logit is tm and whose
// exponentials around it sum to s: an entry's probability is its exponential
// times pT.  Without an entry in use s is 0, and the log-sum-exp is not looked at.
__device__ __forceinline__ void teacher_total(const RowArgs& a, float lse, float s, TeacherHead& th) {
  th.none = s == 0.0f;
  if (th.none) {
    th.tlog = 0.0;
    th.pT = th.P = 0.0f;
  } else if (a.tlse) {
    th.tlog = (double)lse - (double)th.tm * a.s;
    const float hi = (float)th.tlog;
    th.pT = expf(-hi) * (1.0f - (float)(th.tlog - (double)hi));
    th.P = s * th.pT;
  } else {
    th.tlog = log_of_sum(s);
    th.pT = 1.0f / s;
    th.P = s > 0.0f ? 1.0f : s;  // NaN stays
  }
}

// log p - log q of an entry with logit t and score x is ((t - tm) - (x - xm))
// / temperature + c: the two maxima and logarithms of sums are taken apart in
// float64 once a row, and what is left to float32 are small differences.
struct TeacherGap {
  float xm, c;
};
__device__ __forceinline__ TeacherGap teacher_gap(const RowArgs& a, const TeacherHead& th, const Base& h,
                                                  float S) {
  const double m = base_score(h, a.inv_sl);
  TeacherGap g;
  g.xm = (float)m;
  g.c = (float)(log_of_sum(S) - th.tlog - ((double)g.xm - m) * a.s);
  return g;
}

// An entry's probability; its term of the loss goes to `part`.
__device__ __forceinline__ float teacher_p(const RowArgs& a, const TeacherHead& th, const TeacherGap& g,
                                           float t, float x, float& part) {
  if (t == NEG_INF) return 0.0f;
  const float dt = t - th.tm, p = expf(dt * (float)a.s) * th.pT;
  if (p != 0.0f) part += p * fmaf(dt - (x - g.xm), (float)a.s, g.c);
  return p;
}

// Takes the entries in (the first ones are in `ahead`); the maximum and
// log-sum-exp of the teacher's logits over those in use.
template <typename T>
__device__ __forceinline__ TeacherHead teacher_head(const RowArgs& a, long long r, float lse,
                                                    const Teacher& tc, TeacherAhead& ahead, const T* x, const T* g,
                                                    const Range& rg, int lane, int n, unsigned mm) {
  TeacherHead th;
  const float st = (float)a.s;
  float out = 0.0f, m = NEG_INF;
  for (int from = 0; from < a.k; from += TEACHER_AHEAD * n) {
    if (from) ahead.load(a, r, from, lane, n);
    T xs[TEACHER_AHEAD];
#pragma unroll
    for (int u = 0; u < TEACHER_AHEAD; ++u) {
      const bool inside = ahead.id[u] >= 0 && ahead.id[u] < a.V;
      xs[u] = from_f32<T>(0.0f);
      if (inside && SEMICRF_INB(a.status, ahead.id[u] < a.V, SITE_LOSS_SCORE)) xs[u] = x[ahead.id[u]];
      if (ahead.id[u] >= a.V) out = 1.0f;
      if (!inside) ahead.id[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < TEACHER_AHEAD; ++u) {
      const int j = from + u * n + lane, id = ahead.id[u];
      if (j >= a.k) break;
      const float t = id >= 0 ? ahead.t[u] : NEG_INF;
      tc.id[j] = id;
      tc.p[j] = t;
      tc.x[j] = to_f32<T>(xs[u]);
      if (a.add && g && id >= 0 && rg.has(id)) tc.old[j] = to_f32<T>(g[id]);
      m = fmaxf(m, t);
    }
  }
  th.malformed = lanes_max(out, n, mm) > 0.0f;
  m = lanes_max(m, n, mm);
  th.tm = m == NEG_INF ? 0.0f : m;
  float s = 0.0f;
#pragma unroll 4
  for (int j = lane; j < a.k; j += n)
    if (tc.id[j] >= 0) s += expf((tc.p[j] - th.tm) * st);
  s = lanes_sum(s, n, mm);
  teacher_total(a, lse, s, th);
  th.repeats = true;
  const int size = teacher_table(a.k, a.V);
  if (size) {
    teacher_clear(tc.table, size, a.V, lane, n);
    __syncwarp(mm);
    float twice = 0.0f;
    for (int j = lane; j < a.k; j += n)
      if (tc.id[j] >= 0 && teacher_again(a, tc.table, size, a.V, tc.id[j])) twice = 1.0f;
    th.repeats = lanes_max(twice, n, mm) > 0.0f;
  }
  return th;
}

// The entries' probabilities and, where `loss`, the position's loss.
__device__ __forceinline__ void teacher_terms(const RowArgs& a, long long r, const Teacher& tc,
                                              const TeacherHead& th, const Base& h, float S,
                                              bool loss, int lane, int n, unsigned mm) {
  const TeacherGap gap = teacher_gap(a, th, h, S);
  float part = 0.0f;
#pragma unroll 4
  for (int j = lane; j < a.k; j += n)
    tc.p[j] = tc.id[j] >= 0 ? teacher_p(a, th, gap, tc.p[j], tc.x[j], part) : 0.0f;
  __syncwarp(mm);
  if (loss) {
    part = lanes_sum(part, n, mm);
    if (lane == 0) put_term(a, r, (float)(a.tau * a.tau) * part);
  }
}

// The gradient at the teacher's labels within `rg`: the row's value there
// less the entries' probabilities (the first of equal labels takes the sum
// over them, in order).
template <typename T>
__device__ __forceinline__ void teacher_fix(const RowArgs& a, const Teacher& tc, T* g,
                                            const Base& h, float scale, float cq, bool repeats,
                                            int lane, int n, const Range& rg) {
#pragma unroll 4
  for (int j = lane; j < a.k; j += n) {
    const int id = tc.id[j];
    if (id < 0 || !rg.has(id) || !SEMICRF_INB(a.status, id < a.V, SITE_LOSS_SCORE)) continue;
    float p = tc.p[j];
    if (repeats) {
      bool first = true;
      p = 0.0f;
      for (int i = 0; i < a.k; ++i) {
        if (tc.id[i] != id) continue;
        if (i < j) first = false;
        p += tc.p[i];
      }
      if (!first) continue;
    }
    float gv = based_exp(tc.x[j], a.sl, h) * scale - cq * p;
    if (a.add) gv += tc.old[j];
    g[id] = from_f32<T>(gv);
  }
}

// ------------------------------------------------------------ vectors of a row
template <typename T>
constexpr int vec_of = 16 / (int)sizeof(T);  // elements of a 16-byte vector

// Two float32 in one 64-bit register pair: a fused multiply-add, an addition
// or a multiplication of both is one instruction on sm_100.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void halves(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
  float lo, hi;
  halves(v, lo, hi);
  return pair(ex2(lo), ex2(hi));
}

// A 16-byte vector of T as pairs of float32, its greatest element, -inf, and back.
template <typename T>
struct Vec;

template <>
struct Vec<float> {
  static constexpr int PAIRS = 2;
  static constexpr uint32_t LOWEST = 0xff800000u;  // -inf
  static __device__ __forceinline__ void unpack(const uint4& u, f32x2 (&v)[2]) {
    v[0] = pair(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = pair(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2 (&v)[2]) {
    float a, b, c, d;
    halves(v[0], a, b);
    halves(v[1], c, d);
    return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
  }
  template <int N>
  static __device__ __forceinline__ float greatest(const uint4 (&u)[N]) {
    float m[2] = {NEG_INF, NEG_INF};
#pragma unroll
    for (int i = 0; i < N; ++i) {
      m[0] = fmaxf(m[0], fmaxf(__uint_as_float(u[i].x), __uint_as_float(u[i].y)));
      m[1] = fmaxf(m[1], fmaxf(__uint_as_float(u[i].z), __uint_as_float(u[i].w)));
    }
    return fmaxf(m[0], m[1]);
  }
};

// Both 16-bit types: elements 2i and 2i + 1 share a word.
template <typename H, typename H2>
struct Vec16 {
  static constexpr int PAIRS = 4;
  template <int N>
  static __device__ __forceinline__ float greatest(const uint4 (&u)[N]) {
    H2 m[4];
    const uint4 first = u[0];
    m[0] = *reinterpret_cast<const H2*>(&first.x);
    m[1] = *reinterpret_cast<const H2*>(&first.y);
    m[2] = *reinterpret_cast<const H2*>(&first.z);
    m[3] = *reinterpret_cast<const H2*>(&first.w);
#pragma unroll
    for (int i = 1; i < N; ++i) {
      const uint4 q = u[i];
      m[0] = __hmax2(m[0], *reinterpret_cast<const H2*>(&q.x));
      m[1] = __hmax2(m[1], *reinterpret_cast<const H2*>(&q.y));
      m[2] = __hmax2(m[2], *reinterpret_cast<const H2*>(&q.z));
      m[3] = __hmax2(m[3], *reinterpret_cast<const H2*>(&q.w));
    }
    const H2 t = __hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3]));
    return fmaxf(to_f32<H>(t.x), to_f32<H>(t.y));
  }
};

template <>
struct Vec<__nv_bfloat16> : Vec16<__nv_bfloat16, __nv_bfloat162> {
  static constexpr uint32_t LOWEST = 0xff80ff80u;  // -inf twice
  static __device__ __forceinline__ void unpack(const uint4& u, f32x2 (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const f32x2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      halves(v[i], lo, hi);
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <>
struct Vec<__half> : Vec16<__half, __half2> {
  static constexpr uint32_t LOWEST = 0xfc00fc00u;
  static __device__ __forceinline__ void unpack(const uint4& u, f32x2 (&v)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[i] = pair(f.x, f.y);
    }
  }
  static __device__ __forceinline__ uint4 pack(const f32x2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      halves(v[i], lo, hi);
      const __half2 h = __floats2half2_rn(lo, hi);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// How a row divides: `head` elements up to the first 16-byte boundary, nb
// vectors, and the rest.  head + tail <= 2 VE - 2 elements are taken one by a
// thread.
struct Split {
  int head, nb, edge;  // edge: head + tail
};

template <typename T>
__device__ __forceinline__ Split split_row(const T* x, int V) {
  constexpr int VE = vec_of<T>;
  Split s;
  const int off = (int)(reinterpret_cast<uintptr_t>(x) & 15) / (int)sizeof(T);
  s.head = min(V, off ? VE - off : 0);
  s.nb = (V - s.head) / VE;
  s.edge = V - s.nb * VE;
  return s;
}

// Element index of edge element i (0 <= i < edge).
template <typename T>
__device__ __forceinline__ int edge_index(const Split& s, int i) {
  return i < s.head ? i : s.nb * vec_of<T> + i;
}

// Whether vector i of a row (from its first 16-byte boundary) lies inside it.
template <typename T>
__device__ __forceinline__ bool vector_inside(const RowArgs& a, const Split& s, int i) {
  return SEMICRF_INB(a.status, i >= 0 && i < s.nb && s.head + (i + 1) * vec_of<T> <= a.V, SITE_LOSS_VECTOR);
}
__device__ __forceinline__ bool edge_inside(const RowArgs& a, int at) {
  return SEMICRF_INB(a.status, at >= 0 && at < a.V, SITE_LOSS_EDGE);
}

#include "loss_lanes.cuh"
#include "loss_cta.cuh"
#include "loss_ring.cuh"
#include "loss_wide.cuh"

// ----------------------------------------------------------------- launches
template <typename T, int MODE>
cudaError_t rows_in_mode(const RowArgs& a, cudaStream_t st) {
  cudaError_t e;
  if (launch_lanes<T, MODE>(a, st, e)) return e;
  if constexpr (MODE != LM_PREFERENCE) {  // (that pass writes no gradient)
    if (launch_cta<T, MODE>(a, st, e)) return e;
  }
  if (launch_ring<T, MODE>(a, st, e)) return e;
  // the rings decline only rows that they would have to hold between two passes
  if constexpr (MODE != LM_PREFERENCE && MODE != LM_SCALED) return launch_wide<T, MODE>(a, st);
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t rows_of(int mode, const RowArgs& a, cudaStream_t st) {
  switch (mode) {
    case LM_LOGPROB: return rows_in_mode<T, LM_LOGPROB>(a, st);
    case LM_POLICY: return rows_in_mode<T, LM_POLICY>(a, st);
    case LM_PREFERENCE: return rows_in_mode<T, LM_PREFERENCE>(a, st);
    case LM_SCALED: return rows_in_mode<T, LM_SCALED>(a, st);
    default: return rows_in_mode<T, LM_DISTILL>(a, st);
  }
}

}  // namespace
}  // namespace semicrf
