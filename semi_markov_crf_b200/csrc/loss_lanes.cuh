// loss_lanes.cuh -- short rows: L lanes of a warp keep a row in registers,
// NE elements each (included by loss_row.cuh).
//
// Rows of a few hundred bytes come by the hundred thousand (the emissions of
// a batch of sequences), so what counts is instructions a row: the groups of a
// warp work on neighbouring rows, the loads of a warp are one contiguous
// stretch of memory, and reductions are log2 L shuffles.

constexpr int LANES_THREADS = 128;

template <typename T, int MODE, int L, int NE>
__global__ void __launch_bounds__(LANES_THREADS) loss_lanes_kernel(
    const __grid_constant__ RowArgs a) {
  extern __shared__ float dyn[];
  const int tid = threadIdx.x, V = a.V;
  const long long r = (long long)blockIdx.x * (blockDim.x / L) + tid / L;
  if (blockIdx.x == 0 && tid == 0 && a.status) *a.status = 0;
  if (r >= (long long)a.B * a.T) return;
  const int lane = tid % L;
  const unsigned mm = L == 32 ? FULL_MASK : ((1u << (L & 31)) - 1u) << ((tid & 31) / L * L);
  const Head h = make_head<MODE>(a, load_head<MODE>(a, r));
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = a.g ? row_at<T>(a.g, r, a.ldg) : nullptr;
  const float w = MODE == LM_SCALED && h.live ? a.wseq[h.b] : 0.0f;
  if (!h.live || h.malformed || (MODE == LM_SCALED && w == 0.0f)) {
    if (MODE != LM_SCALED && lane == 0) blank_outputs<MODE>(a, r, h.live);
    if (g && !a.add)
      for (int v = lane; v < V; v += L) g[v] = from_f32<T>(0.0f);
    return;
  }

  TeacherAhead ahead;
  if (MODE == LM_DISTILL) ahead.load(a, r, 0, lane, L);
  float v[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) v[i] = i * L + lane < V ? to_f32<T>(x[i * L + lane]) : NEG_INF;
  const LabelIn<T> in = load_label<T, MODE>(a, r, h, x);
  const Range all{0, V, V};
  float* mine =
      dyn + (size_t)(tid / L) * (MODE == LM_DISTILL ? TEACHER_WORDS * a.k + teacher_table(a.k) : 0);
  Teacher tc{mine, reinterpret_cast<int*>(mine + a.k), mine + 2 * a.k, mine + 3 * a.k,
             reinterpret_cast<int*>(mine + TEACHER_WORDS * a.k)};
  TeacherHead th{};
  if (MODE == LM_DISTILL) {
    th = teacher_head<T>(a, r, tc, ahead, x, g, all, lane, L, mm);
    if (th.malformed) {
      if (lane == 0) blank_outputs<MODE>(a, r, true);
      if (g && !a.add)
        for (int i = lane; i < V; i += L) g[i] = from_f32<T>(0.0f);
      return;
    }
  }

  Base base;
  float S;
  if (MODE == LM_SCALED) {
    base = unpack_stat(a.stat[r], S);
  } else {
    float m = NEG_INF;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = fmaxf(m, v[i]);
    m = lanes_max(m, L, mm);
    base = make_base(m, a.sl);
    S = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    // past the row: no score, whatever the base is (-inf - -inf is not a number)
    v[i] = i * L + lane < V ? based_exp(v[i], a.sl, base) : 0.0f;
    if (MODE != LM_SCALED) S += v[i];
  }
  if (MODE != LM_SCALED) S = lanes_sum(S, L, mm);

  float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
  if (MODE == LM_SCALED) {
    cy = (float)((double)w * a.s);
    cq = -cy;
  } else if (MODE == LM_DISTILL) {
    P = th.P;
    teacher_terms(a, r, tc, th, base, S, true, lane, L, mm);
    cq = (float)((a.w ? a.w[h.b] : 1.0) / a.s);
  } else {
    cy = label_outputs<MODE>(a, r, in, base, S, lane == 0);
    cq = -cy;
  }
  if (!g || MODE == LM_PREFERENCE) return;
  const float scale = cq * P / S;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * L + lane;
    if (e >= V) continue;
    float gv = v[i] * scale;
    if (has_label(MODE) && e == h.y) gv += cy;
    if (a.add) gv += to_f32<T>(g[e]);
    g[e] = from_f32<T>(gv);
  }
  if (MODE == LM_DISTILL) {
    __syncwarp(mm);  // the row is written; its teacher entries follow
    teacher_fix<T>(a, tc, g, base, scale, cq, th.repeats, lane, L, all);
  }
}

template <typename T, int MODE, int L, int NE>
cudaError_t launch_lanes_shape(const RowArgs& a, cudaStream_t st) {
  // 48 KB of shared memory for the teacher's entries: fewer rows a CTA where k is large
  int threads = LANES_THREADS;
  size_t smem = 0;
  if (MODE == LM_DISTILL) {
    const size_t row = (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k)) * sizeof(float);
    while (threads > 32 && threads / L * row > 48 * 1024) threads /= 2;
    smem = threads / L * row;
  }
  const long long rows = (long long)a.B * a.T, per = threads / L;
  loss_lanes_kernel<T, MODE, L, NE>
      <<<(unsigned)((rows + per - 1) / per), threads, smem, st>>>(a);
  return cudaGetLastError();
}

// False where the row is too long for these kernels (or the teacher's lists
// do not fit 48 KB for one warp's rows).
template <typename T, int MODE>
bool launch_lanes(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  const int V = a.V;
  int L = V <= 8 ? 1 : V <= 16 ? 2 : V <= 32 ? 4 : V <= 64 ? 8 : V <= 128 ? 16 : 32;
  if (V > 256) return false;
  if (MODE == LM_DISTILL)
    while (L < 32 && 32 / L * (TEACHER_WORDS * a.k + teacher_table(a.k)) * sizeof(float) > 48 * 1024)
      L *= 2;
  switch (L) {
    case 1: e = launch_lanes_shape<T, MODE, 1, 8>(a, st); break;
    case 2: e = launch_lanes_shape<T, MODE, 2, 8>(a, st); break;
    case 4: e = launch_lanes_shape<T, MODE, 4, 8>(a, st); break;
    case 8: e = launch_lanes_shape<T, MODE, 8, 8>(a, st); break;
    case 16: e = launch_lanes_shape<T, MODE, 16, 8>(a, st); break;
    default: e = launch_lanes_shape<T, MODE, 32, 8>(a, st); break;
  }
  return true;
}
