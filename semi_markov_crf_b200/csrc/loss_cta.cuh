// loss_cta.cuh -- rows of a few thousand scores: one CTA of 2 or 4 warps a row,
// the row in registers, 64 elements a thread (included by loss_row.cuh).
//
// As the lane groups of short rows: nothing is kept between rows, and many
// small CTAs an SM hide one another's loads and reductions.  The rings hand
// every row over between warps three times, 1 to 2 microseconds a row: 32768
// rows of 4096 bfloat16, policy loss and gradient, 113 us there and 95 us here;
// with 64 teacher's entries a row 210 and 146 us.

constexpr int CTA_NE = 64;
constexpr int CTA_V_MAX = 128 * CTA_NE;

template <int L>
__device__ __forceinline__ float cta_max(float v, float* red) {
  v = group_max(v, 32);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = red[0];
#pragma unroll
  for (int i = 1; i < L / 32; ++i) m = fmaxf(m, red[i]);
  return m;
}
template <int L>
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = group_sum(v, 32);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < L / 32; ++i) s += red[i];
  return s;
}

template <typename T, int MODE, int L>
__global__ void __launch_bounds__(L, 640 / L)
    loss_cta_kernel(const __grid_constant__ RowArgs a) {
  constexpr int VE = vec_of<T>, NV = CTA_NE / VE;
  __shared__ float red[2][L / 32];
  __shared__ float tshare[2];
  extern __shared__ float dyn[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
  const int r = blockIdx.x;
  start_status(a);
  const Head h = make_head<MODE>(a, load_head<MODE>(a, r));
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = a.g ? row_at<T>(a.g, r, a.ldg) : nullptr;
  const Split sp = split_row(x, V);
  const int ei = tid < sp.edge && edge_inside(a, edge_index<T>(sp, tid)) ? edge_index<T>(sp, tid) : -1;
  auto fill_zero = [&]() {
    if (!g || a.add) return;
    uint4* out = reinterpret_cast<uint4*>(g + sp.head);
    for (int i = tid; i < sp.nb; i += L) out[i] = make_uint4(0, 0, 0, 0);
    if (ei >= 0) g[ei] = from_f32<T>(0.0f);
  };
  const float w = MODE == LM_SCALED && h.live ? a.wseq[h.b] : 0.0f;
  if (!h.live || h.malformed || (MODE == LM_SCALED && w == 0.0f)) {
    if (MODE != LM_SCALED && tid == 0) blank_outputs<MODE>(a, r, h.live);
    fill_zero();
    return;
  }
  uint4 q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    constexpr uint32_t none = Vec<T>::LOWEST;
    q[i] = make_uint4(none, none, none, none);
    if (i * L + tid < sp.nb && vector_inside<T>(a, sp, i * L + tid)) q[i] = __ldg(reinterpret_cast<const uint4*>(x + sp.head) + (i * L + tid));
  }
  float xe = NEG_INF;
  if (ei >= 0) xe = to_f32<T>(x[ei]);
  const LabelIn<T> in = load_label<T, MODE>(a, r, h, x);
  const Range all{0, V, V};
  const Teacher tc{dyn, reinterpret_cast<int*>(dyn + a.k), dyn + 2 * a.k, dyn + 3 * a.k,
                   reinterpret_cast<int*>(dyn + TEACHER_WORDS * a.k)};
  TeacherHead th{};
  if (MODE == LM_DISTILL && warp == 0) {
    TeacherAhead ahead;
    ahead.load(a, r, 0, lane, 32);
    th = teacher_head<T>(a, r, in.lse, tc, ahead, x, g, all, lane, 32, FULL_MASK);
    if (lane == 0) {
      tshare[0] = th.P;
      tshare[1] = th.malformed ? 1.0f : th.none ? 2.0f : 0.0f;
    }
  }

  Base base;
  float S = 0.0f;
  if (MODE == LM_SCALED) base = unpack_stat(in.stat, S);
  else base = make_base(cta_max<L>(fmaxf(Vec<T>::greatest(q), xe), red[0]), a.sl);
  if (MODE == LM_DISTILL && tshare[1] != 0.0f) {
    if (tid == 0) blank_outputs<MODE>(a, r, tshare[1] == 1.0f);
    fill_zero();
    return;
  }
  f32x2 v[CTA_NE / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    f32x2 two[VE / 2];
    Vec<T>::unpack(q[i], two);
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) v[i * (VE / 2) + e] = two[e];
  }
  if (base.direct) {
    const f32x2 sl2 = pair(a.sl, a.sl), at2 = pair(-base.at, -base.at);
#pragma unroll
    for (int i = 0; i < CTA_NE / 2; ++i) v[i] = ex2_2(fma2(v[i], sl2, at2));
  } else {
#pragma unroll
    for (int i = 0; i < CTA_NE / 2; ++i) {
      float lo, hi;
      halves(v[i], lo, hi);
      v[i] = pair(ex2((lo - base.at) * a.sl), ex2((hi - base.at) * a.sl));
    }
  }
  xe = based_exp(xe, a.sl, base);
  if (MODE != LM_SCALED) {
    f32x2 part[2] = {v[0], v[1]};
#pragma unroll
    for (int i = 2; i < CTA_NE / 2; ++i) part[i & 1] = add2(part[i & 1], v[i]);
    float lo, hi;
    halves(add2(part[0], part[1]), lo, hi);
    S = cta_sum<L>(lo + hi + xe, red[1]);
  }

  float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
  if (MODE == LM_SCALED) {
    cy = (float)((double)w * a.s);
    cq = -cy;
  } else if (MODE == LM_DISTILL) {
    P = tshare[0];
    if (warp == 0) teacher_terms(a, r, tc, th, base, S, true, lane, 32, FULL_MASK);
    cq = (float)(in.w * a.tau);
  } else {
    cy = label_outputs<MODE>(a, r, in, base, S, tid == 0);
    cq = -cy;
  }
  if (!g) return;
  const float scale = __fdividef(cq * P, S);
  const f32x2 scale2 = pair(scale, scale);
  uint4* out = reinterpret_cast<uint4*>(g + sp.head);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * L + tid >= sp.nb || !vector_inside<T>(a, sp, i * L + tid)) continue;
    f32x2 two[VE / 2];
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) two[e] = mul2(v[i * (VE / 2) + e], scale2);
    if (sizeof(T) == 4 && a.add) {
      f32x2 old[VE / 2];
      Vec<T>::unpack(out[i * L + tid], old);
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) two[e] = add2(two[e], old[e]);
    }
    out[i * L + tid] = Vec<T>::pack(two);
  }
  if (ei >= 0) g[ei] = from_f32<T>(xe * scale + (a.add ? to_f32<T>(g[ei]) : 0.0f));
  __syncthreads();  // the row is written; its label or teacher's entries follow
  if (has_label(MODE)) {
    if (tid == 0) {
      const float gv = based_exp(in.xy(), a.sl, base) * scale + cy;
      g[h.y] = from_f32<T>(a.add ? to_f32<T>(g[h.y]) + cy : gv);
    }
  } else if (warp == 0) {
    teacher_fix<T>(a, tc, g, base, scale, cq, th.repeats, lane, 32, all);
  }
}

// False where the row is longer, or its gradient lies otherwise in its 16-byte vectors.
template <typename T, int MODE>
bool launch_cta(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  const uintptr_t px = reinterpret_cast<uintptr_t>(a.x), pg = reinterpret_cast<uintptr_t>(a.g);
  const bool grad = a.g != nullptr;
  if (a.V > CTA_V_MAX) return false;
  // without a gradient a ring's warps all reduce: 62 against 68 us at 4096 scores
  if (!grad && MODE != LM_DISTILL) return false;
  if (grad && ((px ^ pg) % 16 != 0 || (a.ldx - a.ldg) % vec_of<T> != 0)) return false;
  const size_t smem =
      MODE == LM_DISTILL ? (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k, a.V)) * sizeof(float) : 0;
  const unsigned rows = (unsigned)((long long)a.B * a.T);
  if (a.V <= 64 * CTA_NE) loss_cta_kernel<T, MODE, 64><<<rows, 64, smem, st>>>(a);
  else loss_cta_kernel<T, MODE, 128><<<rows, 128, smem, st>>>(a);
  e = cudaGetLastError();
  return true;
}
