// loss_lanes.cuh -- short rows: L lanes of a warp keep a row in registers,
// NE elements each (included by loss_row.cuh).
//
// Rows of a few hundred bytes come by the hundred thousand (the emissions of
// a batch of sequences).  What counts is instructions a row (the scalar work
// of a position costs as much as its elements) and latency: few lanes a row,
// so that a warp works on several, reductions of log2 L shuffles, and
// persistent groups that load the next row and the head after that while they
// work on this one.  VEC: 16-byte loads and stores (rows on 16-byte
// boundaries); otherwise element by element, neighbouring lanes neighbouring
// elements.

constexpr int LANES_THREADS = 128;
constexpr int LANES_CTAS = 7;  // an SM, by registers
constexpr int LANES_V_MAX = 512;

// A row as loaded.
template <typename T, int NE, bool VEC>
struct LaneRow {
  uint4 q[VEC ? NE / vec_of<T> : 1];
  T e[VEC ? 1 : NE];
};

template <typename T, int L, int NE, bool VEC>
struct LaneMap {
  static constexpr int VE = VEC ? vec_of<T> : 1;
  // element of this lane's i-th
  static __device__ __forceinline__ int at(int i, int lane) {
    return (i / VE) * (L * VE) + lane * VE + i % VE;
  }
};

// SHORT: the teacher's entries are at most one a lane and stay in its registers.
template <typename T, int MODE, int L, int NE, bool VEC, bool SHORT>
__global__ void __launch_bounds__(LANES_THREADS, LANES_CTAS)
    loss_lanes_kernel(const __grid_constant__ RowArgs a) {
  using Map = LaneMap<T, L, NE, VEC>;
  constexpr int VE = vec_of<T>;
  extern __shared__ float dyn[];
  const int tid = threadIdx.x, V = a.V, lane = tid % L;
  const int rows = a.B * a.T;  // <= 2^27
  const int units = (int)(gridDim.x * (blockDim.x / L));
  int r = (int)(blockIdx.x * (blockDim.x / L) + tid / L);
  start_status(a);
  if (r >= rows) return;
  const unsigned mm = L == 32 ? FULL_MASK : ((1u << (L & 31)) - 1u) << ((tid & 31) / L * L);
  const Range all{0, V, V};
  float* mine =
      dyn + (size_t)(tid / L) * (MODE == LM_DISTILL ? TEACHER_WORDS * a.k + teacher_table(a.k) : 0);
  const Teacher tc{mine, reinterpret_cast<int*>(mine + a.k), mine + 2 * a.k, mine + 3 * a.k,
                   reinterpret_cast<int*>(mine + TEACHER_WORDS * a.k)};

  // the row at hand and what is on its way for it
  struct Load {
    Head h;
    bool blank;
    float w;
    float2 stat;
    LabelIn<T> in;
    LaneRow<T, NE, VEC> x;
    TeacherLoad<SHORT ? 1 : TEACHER_AHEAD> ahead;
  };
  auto start = [&](Load& l, const HeadLoad& head, int row) {
    l.h = make_head<MODE>(a, head);
    l.w = MODE == LM_SCALED && l.h.live ? a.wseq[l.h.b] : 0.0f;
    l.blank = !l.h.live || l.h.malformed;
    if (l.blank) return;
    const T* x = row_at<T>(a.x, row, a.ldx);
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NE / VE; ++i)
        if (Map::at(i * VE, lane) < V)
          l.x.q[i] = __ldg(reinterpret_cast<const uint4*>(x) + (i * L + lane));
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (Map::at(i, lane) < V) l.x.e[i] = x[Map::at(i, lane)];
    }
    if (MODE == LM_SCALED) l.stat = a.stat[row];
    if (has_label(MODE) && MODE != LM_SCALED) l.in = load_label<T, MODE>(a, row, l.h, x);
    if (MODE == LM_DISTILL) {
      l.ahead.load(a, row, 0, lane, L);
      if (a.w) l.in.w = a.w[l.h.b];
      else l.in.w = 1.0;
    }
  };

  Load now;
  start(now, load_head<MODE>(a, r), r);
  HeadLoad soon{};
  if (r + units < rows) soon = load_head<MODE>(a, r + units);
  for (; r < rows; r += units) {
    Load next;
    next.blank = true;
    if (r + units < rows) {
      start(next, soon, r + units);
      if (r + 2 * (long long)units < rows) soon = load_head<MODE>(a, r + 2 * units);
    }
    const T* x = row_at<T>(a.x, r, a.ldx);
    T* g = a.g && MODE != LM_PREFERENCE ? row_at<T>(a.g, r, a.ldg) : nullptr;
    bool blank = now.blank || (MODE == LM_SCALED && now.w == 0.0f);
    bool malformed = now.blank && now.h.live;
    TeacherHead th{};
    float tx = 0.0f;
    if (MODE == LM_DISTILL && !blank) {
      if constexpr (SHORT) {
        const int id = now.ahead.id[0];
        if (id >= 0 && id < V) {
          tx = to_f32<T>(x[id]);
        } else {
          now.ahead.t[0] = NEG_INF;
        }
        th.malformed = lanes_max(id >= V ? 1.0f : 0.0f, L, mm) > 0.0f;
        const float m = lanes_max(now.ahead.t[0], L, mm);
        th.tm = m == NEG_INF ? 0.0f : m;
        const bool used = id >= 0 && id < V;
        teacher_total(a, r, lanes_sum(used ? expf((now.ahead.t[0] - th.tm) * (float)a.s) : 0.0f, L, mm),
                      th);
      } else {
        th = teacher_head<T>(a, r, tc, now.ahead, x, g, all, lane, L, mm);
      }
      blank = malformed = th.malformed;
    }
    if (blank) {
      if (MODE != LM_SCALED && lane == 0) blank_outputs<MODE>(a, r, malformed);
      if (g && !a.add)
        for (int v = lane; v < V; v += L) g[v] = from_f32<T>(0.0f);
      now = next;
      continue;
    }

    float v[NE];
    if (VEC) {
#pragma unroll
      for (int i = 0; i < NE / VE; ++i) {
        f32x2 two[Vec<T>::PAIRS];
        Vec<T>::unpack(now.x.q[i], two);
#pragma unroll
        for (int e = 0; e < Vec<T>::PAIRS; ++e) halves(two[e], v[i * VE + 2 * e], v[i * VE + 2 * e + 1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = to_f32<T>(now.x.e[i]);
    }

    Base base;
    float S = 0.0f;
    if (MODE == LM_SCALED) {
      base = unpack_stat(now.stat, S);
    } else {
      float m = NEG_INF;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (Map::at(i, lane) < V) m = fmaxf(m, v[i]);
      base = make_base(lanes_max(m, L, mm), a.sl);
    }
    // past the row: no score, whatever the base is (-inf - -inf is not a number)
    if (base.direct) {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = Map::at(i, lane) < V ? ex2(fmaf(v[i], a.sl, -base.at)) : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) v[i] = Map::at(i, lane) < V ? ex2((v[i] - base.at) * a.sl) : 0.0f;
    }
    if (MODE != LM_SCALED) {
      float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < NE; ++i) part[i & 3] += v[i];
      S = lanes_sum((part[0] + part[1]) + (part[2] + part[3]), L, mm);
    }

    float tp = 0.0f;  // SHORT: the entry's probability
    float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
    if (MODE == LM_SCALED) {
      cy = (float)((double)now.w * a.s);
      cq = -cy;
    } else if (MODE == LM_DISTILL) {
      P = th.P;
      if constexpr (SHORT) {
        float part = 0.0f;
        tp = now.ahead.id[0] >= 0
                 ? teacher_p(a, th, base, log2f(S), now.ahead.t[0], tx, part) : 0.0f;
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
    if (g) {
      const float scale = __fdividef(cq * P, S);
#pragma unroll
      for (int i = 0; i < NE; ++i) {
        v[i] *= scale;
        if (has_label(MODE) && Map::at(i, lane) == now.h.y) v[i] += cy;
      }
      if (VEC) {
        uint4* out = reinterpret_cast<uint4*>(g);
#pragma unroll
        for (int i = 0; i < NE / VE; ++i) {
          if (Map::at(i * VE, lane) >= V) continue;
          f32x2 two[Vec<T>::PAIRS];
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e) two[e] = pair(v[i * VE + 2 * e], v[i * VE + 2 * e + 1]);
          if (sizeof(T) == 4 && a.add) {
            f32x2 old[Vec<T>::PAIRS];
            Vec<T>::unpack(out[i * L + lane], old);
#pragma unroll
            for (int e = 0; e < Vec<T>::PAIRS; ++e) two[e] = add2(two[e], old[e]);
          }
          out[i * L + lane] = Vec<T>::pack(two);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          const int e = Map::at(i, lane);
          if (e >= V) continue;
          if (a.add) v[i] += to_f32<T>(g[e]);
          g[e] = from_f32<T>(v[i]);
        }
      }
      if (MODE == LM_DISTILL) {
        float old = 0.0f;
        const int id = SHORT ? now.ahead.id[0] : -1;
        __syncwarp(mm);  // the row is written; its teacher entries follow
        if constexpr (SHORT) {
          // the first of the lanes with one label takes the sum over them, in order
          const unsigned same = __match_any_sync(mm, id);
          const int first = __ffs(same) - 1;
          float p = 0.0f;
          for (unsigned left = same; __any_sync(mm, left != 0); left &= left - 1) {
            const int from = left ? __ffs(left) - 1 : (tid & 31);
            const float other = __shfl_sync(mm, tp, from);
            if (left) p += other;
          }
          if (id >= 0 && first == (tid & 31)) {
            // where the call accumulates, the row's own term is in already
            if (a.add) old = to_f32<T>(g[id]);
            g[id] = from_f32<T>(a.add ? old - cq * p : based_exp(tx, a.sl, base) * scale - cq * p);
          }
          __syncwarp(mm);
        } else {
          teacher_fix<T>(a, tc, g, base, scale, cq, th.repeats, lane, L, all);
        }
      }
    }
    if (MODE == LM_DISTILL && !SHORT) __syncwarp(mm);
    now = next;
  }
}

template <typename T, int MODE, int L, int NE, bool VEC, bool SHORT>
cudaError_t launch_lanes_shape(const RowArgs& a, cudaStream_t st) {
  // 48 KB of shared memory for the teacher's entries: fewer rows a CTA where k is large
  int threads = LANES_THREADS;
  size_t smem = 0;
  if (MODE == LM_DISTILL && !SHORT) {
    const size_t row = (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k)) * sizeof(float);
    while (threads > 32 && threads / L * row > 48 * 1024) threads /= 2;
    smem = threads / L * row;
  }
  const long long rows = (long long)a.B * a.T, per = threads / L;
  const long long fit = (long long)loss_sm_count() * LANES_CTAS * (LANES_THREADS / threads);
  loss_lanes_kernel<T, MODE, L, NE, VEC, SHORT>
      <<<(unsigned)std::min(fit, (rows + per - 1) / per), threads, smem, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int MODE, int L>
cudaError_t launch_lanes_of(const RowArgs& a, cudaStream_t st) {
  constexpr int VE = vec_of<T>;
  const bool grad = a.g != nullptr;
  const bool vec = a.V % VE == 0 && a.ldx % VE == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0 &&
                   (!grad || (a.ldg % VE == 0 && reinterpret_cast<uintptr_t>(a.g) % 16 == 0));
  const bool half = a.V <= 8 * L;
  auto shape = [&](auto one_a_lane) {
    constexpr bool SHORT = decltype(one_a_lane)::value;
    if (vec) return half ? launch_lanes_shape<T, MODE, L, 8, true, SHORT>(a, st)
                         : launch_lanes_shape<T, MODE, L, 16, true, SHORT>(a, st);
    return half ? launch_lanes_shape<T, MODE, L, 8, false, SHORT>(a, st)
                : launch_lanes_shape<T, MODE, L, 16, false, SHORT>(a, st);
  };
  if constexpr (MODE == LM_DISTILL) {
    if (a.k <= L) return shape(std::true_type{});
  }
  return shape(std::false_type{});
}

// False where the row is too long for these kernels.
template <typename T, int MODE>
bool launch_lanes(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  if (a.V > LANES_V_MAX) return false;
  int L = 1;
  while (a.V > 16 * L) L *= 2;
  if (MODE == LM_DISTILL) {
    // a lane holds its first entries in registers, and 48 KB hold a warp's rows
    const size_t row = (size_t)(TEACHER_WORDS * a.k + teacher_table(a.k)) * sizeof(float);
    while (L < 32 && (a.k > L || 32 / L * row > 48 * 1024)) L *= 2;
  }
  switch (L) {
    case 1: e = launch_lanes_of<T, MODE, 1>(a, st); break;
    case 2: e = launch_lanes_of<T, MODE, 2>(a, st); break;
    case 4: e = launch_lanes_of<T, MODE, 4>(a, st); break;
    case 8: e = launch_lanes_of<T, MODE, 8>(a, st); break;
    case 16: e = launch_lanes_of<T, MODE, 16>(a, st); break;
    default: e = launch_lanes_of<T, MODE, 32>(a, st); break;
  }
  return true;
}
