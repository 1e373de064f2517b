// loss_lanes.cuh -- short rows: L lanes of a warp keep a row in registers,
// NE elements each (included by loss_row.cuh).
//
// Rows of a few hundred bytes come by the hundred thousand (the emissions of
// a batch of sequences).  What counts is instructions a row (the scalar work
// of a position costs as much as its elements) and rows in flight: few lanes a
// row, so that a warp works on several at once and a reduction is log2 L
// shuffles, one row a group, and no more registers than 16, 32 or 40 warps an
// SM leave (64, 32 or up to 16 elements a lane).  (Loading a row ahead costs the
// registers of a third of the warps and was slower: 31 against 21 us for 80000
// rows of 128 float32; tiles in shared memory behind TMA copies, 16 warps an SM,
// took 33.)
//
// Layouts: VECTORS, rows on 16-byte boundaries; SPLIT, the 16-byte vectors
// within a row and up to 14 single elements, one a lane; ELEMENTS, neighbouring
// lanes neighbouring elements.

enum LaneLayout : int { ELEMENTS = 0, VECTORS = 1, SPLIT = 2 };
constexpr int LANES_THREADS = 128;
constexpr int LANES_V_MAX = 2048;
constexpr int LANES_ELEMENTS = 256;  // longer rows that are not on 16-byte boundaries are split
constexpr int lanes_ctas(int NE) { return NE > 32 ? 4 : NE > 16 ? 8 : 10; }  // an SM, by registers

// A row as loaded: 16-byte vectors, or elements (one beside the vectors where they split).
template <typename T, int NE, int LAY>
struct LaneRow {
  uint4 q[LAY ? NE / vec_of<T> : 1];
  T e[LAY ? 1 : NE];
};

template <typename T, int L, int LAY>
struct LaneMap {
  static constexpr int VE = LAY ? vec_of<T> : 1;
  // element of this lane's i-th
  static __device__ __forceinline__ int at(int i, int lane) {
    return (i / VE) * (L * VE) + lane * VE + i % VE;
  }
};

// The row at hand and what is on its way for it.
template <typename T, int NE, int LAY, int AHEAD>
struct LaneLoad {
  Head h;
  bool blank;
  float w;
  float2 stat;
  LabelIn<T> in;
  LaneRow<T, NE, LAY> x;
  TeacherLoad<AHEAD> ahead;
};

template <typename T, int MODE, int L, int NE, int LAY, int AHEAD>
__device__ __forceinline__ void lane_load(const RowArgs& a, LaneLoad<T, NE, LAY, AHEAD>& l,
                                          const HeadLoad& head, int row, int lane) {
  using Map = LaneMap<T, L, LAY>;
  constexpr int VE = vec_of<T>;
  l.h = make_head<MODE>(a, head);
  l.w = MODE == LM_SCALED && l.h.live ? a.wseq[l.h.b] : 0.0f;
  l.blank = !l.h.live || l.h.malformed;
  if (l.blank) return;
  const T* x = row_at<T>(a.x, row, a.ldx);
  // past the row: -inf, whose exponential is 0 around any base of a row that has one
  if (LAY) {
    Split sp{0, a.V / VE, 0};
    if (LAY == SPLIT) sp = split_row(x, a.V);
#pragma unroll
    for (int i = 0; i < NE / VE; ++i) {
      constexpr uint32_t none = Vec<T>::LOWEST;
      l.x.q[i] = make_uint4(none, none, none, none);
      if (i * L + lane < sp.nb && vector_inside<T>(a, sp, i * L + lane))
        l.x.q[i] = __ldg(reinterpret_cast<const uint4*>(x + sp.head) + (i * L + lane));
    }
    if (LAY == SPLIT) {
      l.x.e[0] = from_f32<T>(NEG_INF);
      if (lane < sp.edge && edge_inside(a, edge_index<T>(sp, lane))) l.x.e[0] = x[edge_index<T>(sp, lane)];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      l.x.e[i] = from_f32<T>(NEG_INF);
      if (Map::at(i, lane) < a.V) l.x.e[i] = x[Map::at(i, lane)];
    }
  }
  if (MODE == LM_SCALED) l.stat = a.stat[row];
  if (MODE != LM_SCALED) l.in = load_label<T, MODE>(a, row, l.h, x);
  if (MODE == LM_DISTILL) {
    l.ahead.load(a, row, 0, lane, L);
  }
}

// One row.  KEEP: teacher's entries that a lane keeps in registers; 0: they go
// through shared memory (lists of more than 128).
template <typename T, int MODE, int L, int NE, int LAY, int KEEP, int AHEAD>
__device__ __forceinline__ void lane_row(const RowArgs& a, LaneLoad<T, NE, LAY, AHEAD>& now, int r,
                                         const Teacher& tc, int lane, unsigned mm) {
  using Map = LaneMap<T, L, LAY>;
  constexpr int VE = vec_of<T>;
  constexpr bool SHORT = KEEP > 0;
  const int V = a.V;
  const T* x = row_at<T>(a.x, r, a.ldx);
  T* g = a.g && MODE != LM_PREFERENCE ? row_at<T>(a.g, r, a.ldg) : nullptr;
  const Range all{0, V, V};
  bool blank = now.blank || (MODE == LM_SCALED && now.w == 0.0f);
  bool malformed = now.blank && now.h.live;
  TeacherHead th{};
  float tx[AHEAD], tp[AHEAD];  // SHORT: the row's scores at the entries, their probabilities
  if (MODE == LM_DISTILL && !blank) {
    if constexpr (SHORT) {
      float m = NEG_INF, out = 0.0f, s = 0.0f;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int id = now.ahead.id[u];
        if (id >= V) out = 1.0f;
        if (id < 0 || id >= V) now.ahead.t[u] = NEG_INF;
        tx[u] = 0.0f;
        if (id >= 0 && id < V && SEMICRF_INB(a.status, id < a.V, SITE_LOSS_SCORE)) tx[u] = to_f32<T>(x[id]);
        m = fmaxf(m, now.ahead.t[u]);
      }
      th.malformed = lanes_max(out, L, mm) > 0.0f;
      m = lanes_max(m, L, mm);
      th.tm = m == NEG_INF ? 0.0f : m;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (now.ahead.id[u] >= 0) s += expf((now.ahead.t[u] - th.tm) * (float)a.s);
      teacher_total(a, now.in.lse, lanes_sum(s, L, mm), th);
    } else {
      th = teacher_head<T>(a, r, now.in.lse, tc, now.ahead, x, g, all, lane, L, mm);
    }
    malformed = th.malformed;
    blank = malformed || th.none;
  }
  if (blank) {
    if (MODE != LM_SCALED && lane == 0) blank_outputs<MODE>(a, r, malformed);
    if (g && !a.add)
      for (int v = lane; v < V; v += L) g[v] = from_f32<T>(0.0f);
    return;
  }

  f32x2 v[NE / 2];
  float top = NEG_INF;
  float xe = NEG_INF;
  if constexpr (LAY != ELEMENTS) {
    top = Vec<T>::greatest(now.x.q);
    if (LAY == SPLIT) {
      xe = to_f32<T>(now.x.e[0]);
      top = fmaxf(top, xe);
    }
#pragma unroll
    for (int i = 0; i < NE / VE; ++i) {
      f32x2 two[VE / 2];
      Vec<T>::unpack(now.x.q[i], two);
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) v[i * (VE / 2) + e] = two[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
      const float lo = to_f32<T>(now.x.e[2 * i]), hi = to_f32<T>(now.x.e[2 * i + 1]);
      top = fmaxf(top, fmaxf(lo, hi));
      v[i] = pair(lo, hi);
    }
  }
  Base base;
  float S = 0.0f;
  if (MODE == LM_SCALED) {
    base = unpack_stat(now.stat, S);
  } else {
    base = make_base(lanes_max(top, L, mm), a.sl);
  }
  if (base.direct) {
    const f32x2 sl2 = pair(a.sl, a.sl), at2 = pair(-base.at, -base.at);
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) v[i] = ex2_2(fma2(v[i], sl2, at2));
  } else {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
      float lo, hi;
      halves(v[i], lo, hi);
      v[i] = pair(ex2((lo - base.at) * a.sl), ex2((hi - base.at) * a.sl));
    }
  }
  if (LAY == SPLIT) xe = based_exp(xe, a.sl, base);
  if (MODE != LM_SCALED) {
    f32x2 part[2] = {v[0], v[1]};
#pragma unroll
    for (int i = 2; i < NE / 2; ++i) part[i & 1] = add2(part[i & 1], v[i]);
    float lo, hi;
    halves(add2(part[0], part[1]), lo, hi);
    if (LAY == SPLIT) lo += xe;
    S = lanes_sum(lo + hi, L, mm);
  }

  float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
  if (MODE == LM_SCALED) {
    cy = (float)((double)now.w * a.s);
    cq = -cy;
  } else if (MODE == LM_DISTILL) {
    P = th.P;
    if constexpr (SHORT) {
      const TeacherGap gap = teacher_gap(a, th, base, S);
      float part = 0.0f;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        tp[u] = now.ahead.id[u] >= 0 ? teacher_p(a, th, gap, now.ahead.t[u], tx[u], part) : 0.0f;
      part = lanes_sum(part, L, mm);
      if (lane == 0) put_term(a, r, (float)(a.tau * a.tau) * part);
    } else {
      teacher_terms(a, r, tc, th, base, S, true, lane, L, mm);
    }
    cq = (float)(now.in.w * a.tau);
  } else {
    cy = label_outputs<MODE>(a, r, now.in, base, S, lane == 0);
    cq = -cy;
  }
  if (!g) return;
  const float scale = __fdividef(cq * P, S);
  const f32x2 scale2 = pair(scale, scale);
#pragma unroll
  for (int i = 0; i < NE / 2; ++i) v[i] = mul2(v[i], scale2);
  if constexpr (LAY != ELEMENTS) {
    Split sp{0, V / VE, 0};
    if (LAY == SPLIT) sp = split_row(x, V);
    uint4* out = reinterpret_cast<uint4*>(g + sp.head);
#pragma unroll
    for (int i = 0; i < NE / VE; ++i) {
      if (i * L + lane >= sp.nb || !vector_inside<T>(a, sp, i * L + lane)) continue;
      f32x2 two[VE / 2];
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) two[e] = v[i * (VE / 2) + e];
      if (sizeof(T) == 4 && a.add) {
        f32x2 old[VE / 2];
        Vec<T>::unpack(out[i * L + lane], old);
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) two[e] = add2(two[e], old[e]);
      }
      out[i * L + lane] = Vec<T>::pack(two);
    }
    if (LAY == SPLIT && lane < sp.edge) {
      const int at = edge_index<T>(sp, lane);
      if (edge_inside(a, at)) g[at] = from_f32<T>(xe * scale + (a.add ? to_f32<T>(g[at]) : 0.0f));
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE / 2; ++i) {
      float gv[2];
      halves(v[i], gv[0], gv[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = Map::at(2 * i + e, lane);
        if (at >= V) continue;
        if (a.add) gv[e] += to_f32<T>(g[at]);
        g[at] = from_f32<T>(gv[e]);
      }
    }
  }
  __syncwarp(mm);  // the row is written; its label or teacher's entries follow
  if (has_label(MODE)) {
    if (lane == 0) {
      const T score = MODE == LM_SCALED ? x[now.h.y] : now.in.score;
      const float gv = based_exp(to_f32<T>(score), a.sl, base) * scale + cy;
      g[now.h.y] = from_f32<T>(a.add ? to_f32<T>(g[now.h.y]) + cy : gv);
    }
  } else if constexpr (SHORT) {
    // entries of one label add up, in order, into the first of them
    float sum[AHEAD];
    bool first[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      sum[u] = 0.0f;
      first[u] = now.ahead.id[u] >= 0;
    }
    bool repeats = true;
    const int size = teacher_table(a.k, V);
    if (size) {
      teacher_clear(tc.table, size, V, lane, L);
      __syncwarp(mm);
      float twice = 0.0f;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (now.ahead.id[u] >= 0 && teacher_again(a, tc.table, size, V, now.ahead.id[u])) twice = 1.0f;
      repeats = lanes_max(twice, L, mm) > 0.0f;
      if (!repeats)
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) sum[u] = tp[u];
    }
    for (int s = 0; repeats && s < a.k; ++s) {
      const int from = s % L, slot = s / L;
      int id = now.ahead.id[0];
      float p = tp[0];
#pragma unroll
      for (int u = 1; u < AHEAD; ++u)
        if (slot == u) {
          id = now.ahead.id[u];
          p = tp[u];
        }
      id = __shfl_sync(mm, id, from, L);
      p = __shfl_sync(mm, p, from, L);
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (id == now.ahead.id[u]) {
          if (s < u * L + lane) first[u] = false;
          sum[u] += p;
        }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u)
      if (first[u] && SEMICRF_INB(a.status, now.ahead.id[u] >= 0 && now.ahead.id[u] < V, SITE_LOSS_SCORE)) {
        const int id = now.ahead.id[u];
        // where the call accumulates, the row's own term is in already
        const float own = a.add ? to_f32<T>(g[id]) : based_exp(tx[u], a.sl, base) * scale;
        g[id] = from_f32<T>(own - cq * sum[u]);
      }
  } else {
    teacher_fix<T>(a, tc, g, base, scale, cq, th.repeats, lane, L, all);
    __syncwarp(mm);  // the entries' shared memory is the next row's
  }
}

template <typename T, int MODE, int L, int NE, int LAY, int KEEP>
__global__ void __launch_bounds__(LANES_THREADS, lanes_ctas(NE))
    loss_lanes_kernel(const __grid_constant__ RowArgs a) {
  constexpr int AHEAD = KEEP ? KEEP : TEACHER_AHEAD;
  extern __shared__ float dyn[];
  const int tid = threadIdx.x, lane = tid % L;
  const int rows = a.B * a.T;  // <= 2^27
  const int r = (int)(blockIdx.x * (blockDim.x / L) + tid / L);
  start_status(a);
  if (r >= rows) return;
  const unsigned mm = L == 32 ? FULL_MASK : ((1u << (L & 31)) - 1u) << ((tid & 31) / L * L);
  const int words = KEEP ? 0 : TEACHER_WORDS * a.k;
  float* mine = dyn + (size_t)(tid / L) * (MODE == LM_DISTILL ? words + teacher_table(a.k, a.V) : 0);
  const Teacher tc{mine, reinterpret_cast<int*>(mine + a.k), mine + 2 * a.k, mine + 3 * a.k,
                   reinterpret_cast<int*>(mine + words)};
  LaneLoad<T, NE, LAY, AHEAD> row;
  lane_load<T, MODE, L>(a, row, load_head<MODE>(a, r), r, lane);
  lane_row<T, MODE, L, NE, LAY, KEEP>(a, row, r, tc, lane, mm);
}

template <typename T, int MODE, int L, int NE, int LAY, int KEEP>
cudaError_t launch_lanes_shape(const RowArgs& a, cudaStream_t st) {
  // 48 KB of shared memory for the teacher's entries: fewer rows a CTA where k is large
  int threads = LANES_THREADS;
  size_t smem = 0;
  if (MODE == LM_DISTILL) {
    const size_t row =
        (size_t)((KEEP ? 0 : TEACHER_WORDS * a.k) + teacher_table(a.k, a.V)) * sizeof(float);
    while (threads > 32 && threads / L * row > 48 * 1024) threads /= 2;
    smem = threads / L * row;
  }
  const long long rows = (long long)a.B * a.T, per = threads / L;
  loss_lanes_kernel<T, MODE, L, NE, LAY, KEEP>
      <<<(unsigned)((rows + per - 1) / per), threads, smem, st>>>(a);
  return cudaGetLastError();
}

// Whether launch_lanes() below ever takes a shape: only those are compiled (308 of
// the 562 that the ranges of lanes, elements, layouts and kept entries span, for
// float32 and one 16-bit type).  Rows take the fewest lanes that hold them, more
// only for a teacher's entries, so that most have half of NE in use at least.
template <typename T, int MODE>
constexpr bool lanes_reached(int L, int NE, int LAY, int KEEP) {
  constexpr bool half = sizeof(T) == 2, read_only = MODE == LM_PREFERENCE;
  if (L < 32 && NE == 32 && LAY == ELEMENTS) return false;
  if (L < 32 && NE == 64 && (LAY == ELEMENTS || L == 1 || !half || MODE == LM_SCALED)) return false;
  if (LAY == SPLIT && L < 16) return false;
  if (MODE == LM_DISTILL && KEEP == 0) return L == 32 && !(LAY == SPLIT && NE == 8);
  if (KEEP == 4) {
    if (LAY == SPLIT) return NE >= (L == 16 ? 32 : 16);
    return L >= (LAY == ELEMENTS ? 4 : 8);
  }
  if (LAY == ELEMENTS)
    return L == 1 || (L == 32 ? NE >= 16 && !read_only : NE == 16 || (MODE == LM_DISTILL && L <= 4));
  if (read_only && half && NE == 32 && L > (LAY == SPLIT ? 16 : 2)) return false;
  return NE >= 32 || (LAY == VECTORS && (L == 1 || (MODE == LM_DISTILL && L <= 8)));
}

template <typename T, int MODE, int LAY, int KEEP>
cudaError_t launch_lanes_with(const RowArgs& a, int L, cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;  // stays where the two rules disagree
  auto shape = [&](auto lanes, auto elements) {
    constexpr int N = decltype(lanes)::value, NE = decltype(elements)::value;
    if constexpr (lanes_reached<T, MODE>(N, NE, LAY, KEEP))
      if (L == N && a.V <= NE * N && (NE == 8 || a.V > NE / 2 * N))
        e = launch_lanes_shape<T, MODE, N, NE, LAY, KEEP>(a, st);
  };
  auto of = [&](auto lanes) {
    shape(lanes, std::integral_constant<int, 8>{});
    shape(lanes, std::integral_constant<int, 16>{});
    shape(lanes, std::integral_constant<int, 32>{});
    shape(lanes, std::integral_constant<int, 64>{});
  };
  of(std::integral_constant<int, 1>{});
  of(std::integral_constant<int, 2>{});
  of(std::integral_constant<int, 4>{});
  of(std::integral_constant<int, 8>{});
  of(std::integral_constant<int, 16>{});
  of(std::integral_constant<int, 32>{});
  return e;
}

// False where the row is too long for these kernels.
template <typename T, int MODE>
bool launch_lanes(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  if (a.V > LANES_V_MAX) return false;
  constexpr int VE = vec_of<T>;
  constexpr int ES = sizeof(T);
  const bool grad = a.g != nullptr && MODE != LM_PREFERENCE;
  const uintptr_t px = reinterpret_cast<uintptr_t>(a.x), pg = reinterpret_cast<uintptr_t>(a.g);
  const bool vec = a.V % VE == 0 && a.ldx % VE == 0 && px % 16 == 0 &&
                   (!grad || (a.ldg % VE == 0 && pg % 16 == 0));
  // gradient rows must share their scores' offset from a 16-byte boundary
  const bool split = !vec && a.V > LANES_ELEMENTS &&
                     (!grad || ((px ^ pg) % 16 == 0 && (a.ldx - a.ldg) % VE == 0));
  int L = 1;
  // elements a lane; 16-bit rows that are only read leave registers for more
  // (262144 rows of 1000: 116 against 130 us)
  const int most = !vec ? 16 : grad || ES == 4 ? 32 : 64;
  while (L < 32 && a.V > (L == 1 ? std::min(32, most) : most) * L) L *= 2;
  if (split) L = a.V <= (grad || ES == 4 ? 512 : 1024) ? 16 : 32;  // a lane for each of up to 14 single elements
  auto with = [&](auto keep, int lanes) {
    constexpr int KEEP = decltype(keep)::value;
    return vec ? launch_lanes_with<T, MODE, VECTORS, KEEP>(a, lanes, st)
               : split ? launch_lanes_with<T, MODE, SPLIT, KEEP>(a, lanes, st)
                       : launch_lanes_with<T, MODE, ELEMENTS, KEEP>(a, lanes, st);
  };
  if constexpr (MODE == LM_DISTILL) {
    // Two or four entries a lane in registers rather than more lanes: 200000 rows of 38
    // float32 with 17 entries take 52 us on 8 lanes, 78 on 16; with 16 entries 39 us on
    // 4 lanes, 46 on 8.  Four lanes with 32 elements each have no registers for it
    // (100000 rows of 128 float32, 16 entries: 33 us, 31 on 8 lanes).
    if (a.k <= 128) {
      while (L < (vec ? 8 : 4) && a.k > 2 * L) L *= 2;
      while (a.k > 4 * L) L *= 2;
      e = a.k <= 2 * L ? with(std::integral_constant<int, 2>{}, L)
                       : with(std::integral_constant<int, 4>{}, L);
      return true;
    }
    // a lane holds its first entries in registers, and 48 KB hold a warp's rows
    const size_t row = (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k, a.V)) * sizeof(float);
    while (L < 32 && (a.k > TEACHER_AHEAD * L || 32 / L * row > 48 * 1024)) L *= 2;
  }
  e = with(std::integral_constant<int, 0>{}, L);
  return true;
}
