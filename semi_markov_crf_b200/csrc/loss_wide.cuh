// loss_wide.cuh -- rows too wide for the rings of a cluster (with a gradient,
// from about 1.5 MB): one CTA per row, elements strided over its threads, the
// row read twice, the second time mostly from L2 (included by loss_row.cuh).
// This was the first form of all rows: 8192 of 131072 bfloat16, policy loss and
// gradient, in 2.5 ms.

constexpr int WIDE_THREADS = 512;

__device__ __forceinline__ float wide_max(float v, float* red) {
  v = group_max(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = NEG_INF;
  for (int i = 0; i < WIDE_THREADS / 32; ++i) s = fmaxf(s, red[i]);
  return s;
}

__device__ __forceinline__ float wide_sum(float v, float* red) {
  v = group_sum(v, 32);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < WIDE_THREADS / 32; ++i) s += red[i];
  return s;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(WIDE_THREADS) loss_wide_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float red[WIDE_THREADS / 32];
  __shared__ float tshare[2];
  extern __shared__ float dyn[];
  const long long r = blockIdx.x;
  const int tid = threadIdx.x, V = a.V, warp = tid >> 5, lane = tid & 31;
  start_status(a);
  const Head h = make_head<MODE>(a, load_head<MODE>(a, r));
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = a.g ? row_at<T>(a.g, r, a.ldg) : nullptr;
  bool blank = !h.live || h.malformed;
  bool malformed = h.live;
  const Range all{0, V, V};
  Teacher tc{dyn, reinterpret_cast<int*>(dyn + a.k), dyn + 2 * a.k, dyn + 3 * a.k,
             reinterpret_cast<int*>(dyn + TEACHER_WORDS * a.k)};
  TeacherHead th{};
  if (MODE == LM_DISTILL && h.live) {
    if (warp == 0) {
      TeacherAhead ahead;
      ahead.load(a, r, 0, lane, 32);
      th = teacher_head<T>(a, r, a.tlse ? a.tlse[r] : 0.0f, tc, ahead, x, g, all, lane, 32, FULL_MASK);
      if (lane == 0) {
        tshare[0] = th.P;
        tshare[1] = th.malformed ? 1.0f : th.none ? 2.0f : 0.0f;
      }
    }
    __syncthreads();
    blank = tshare[1] != 0.0f;
    malformed = tshare[1] == 1.0f;
  }
  if (blank) {
    if (tid == 0) blank_outputs<MODE>(a, r, malformed);
    if (g && !a.add)
      for (int v = tid; v < V; v += WIDE_THREADS) g[v] = from_f32<T>(0.0f);
    return;
  }

  // maximum and sum of exponentials in one pass
  float m = NEG_INF, s = 0.0f;
  for (int v = tid; v < V; v += WIDE_THREADS) {
    const float xv = to_f32<T>(x[v]);
    if (xv > m) {
      s *= ex2((m - xv) * a.sl);
      m = xv;
    }
    s += ex2((xv - (m == NEG_INF ? 0.0f : m)) * a.sl);
  }
  const float M = wide_max(m, red);
  float S = wide_sum(m == NEG_INF && s == 0.0f ? 0.0f : s * ex2((m - M) * a.sl), red);
  if (M == NEG_INF) S = quiet_nan();  // nothing but -inf: no distribution
  const Base base{M, false};
  float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
  if (MODE == LM_DISTILL) {
    P = tshare[0];
    if (warp == 0) teacher_terms(a, r, tc, th, base, S, true, lane, 32, FULL_MASK);
    cq = (float)((a.w ? a.w[h.b] : 1.0) * a.tau);
    if (a.add) __syncthreads();  // the gradient's old values at the entries are read
  } else {
    cy = label_outputs<MODE>(a, r, load_label<T, MODE>(a, r, h, x), base, S, tid == 0);
    cq = -cy;
  }
  if (!g) return;
  const float scale = __fdividef(cq * P, S);
  for (int v = tid; v < V; v += WIDE_THREADS) {
    float gv = based_exp(to_f32<T>(x[v]), a.sl, base) * scale;
    if (has_label(MODE) && v == h.y) gv += cy;
    if (a.add) gv += to_f32<T>(g[v]);
    g[v] = from_f32<T>(gv);
  }
  if (MODE == LM_DISTILL) {
    __syncthreads();  // the row is written; its teacher entries follow
    if (warp == 0) teacher_fix<T>(a, tc, g, base, scale, cq, th.repeats, lane, 32, all);
  }
}

template <typename T, int MODE>
cudaError_t launch_wide(const RowArgs& a, cudaStream_t st) {
  const size_t smem = MODE == LM_DISTILL ? (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k, a.V)) * sizeof(float) : 0;
  loss_wide_kernel<T, MODE><<<(unsigned)((long long)a.B * a.T), WIDE_THREADS, smem, st>>>(a);
  return cudaGetLastError();
}
