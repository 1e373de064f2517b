// loss_ring.cuh -- long rows: persistent CTAs that stream rows through a ring
// of shared-memory chunks (included by loss_row.cuh).
//
// A CTA has 16 consumer warps, divided into groups of W warps, and one warp
// that only issues copies.  Each group has a ring of its own and works on a
// row at a time:
//   pass 1  as its chunks arrive (TMA bulk copies, one mbarrier a chunk), the
//           running maximum and sum of exponentials;
//   join    the group's warps (and, for rows wider than one ring, the CTAs of
//           a cluster, through distributed shared memory) exchange (maximum,
//           sum); the position's terms follow;
//   pass 2  the gradient from the same chunks, still in shared memory, which
//           gives each back to the ring.
// A row is read from memory once, and the next row's chunks arrive while this
// one is joined and written.  Without a gradient a chunk goes back after pass
// 1, and the second pass of the preference loss (LM_SCALED) runs pass 2 alone.
//
// Every wait is bounded: a wait that gives up records ST_DEVICE_TIMEOUT in the
// status word and the kernel runs on without waiting (every access stays
// within the rows and the ring), so that it ends.

constexpr int RING_WARPS = 16;                        // consumer warps of a CTA
constexpr int RING_THREADS = (RING_WARPS + 1) * 32;   // and the copying warp
constexpr int RING_NV = 4;                            // vectors of a chunk a thread takes
constexpr int RING_WARP_BYTES = RING_NV * 32 * 16;    // a warp's part of a chunk
constexpr int RING_SLOTS_MAX = 16;                    // chunks of a group's ring
constexpr int RING_CLUSTER_MAX = 8;
constexpr int RING_SMEM = 220 * 1024;

struct RingShape {
  int W;      // warps of a group
  int slots;  // chunks of a group's ring
  int cl;     // CTAs that share a row
};

struct RingBars {
  uint64_t full[RING_WARPS * RING_SLOTS_MAX];
  uint64_t empty[RING_WARPS * RING_SLOTS_MAX];
  uint64_t peer[2];
  float2 red[2][RING_WARPS];
  float2 part[2][RING_CLUSTER_MAX];
  float tshare[2][RING_WARPS][2];
};

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// A position in a group's ring.
struct Cursor {
  int slot;
  uint32_t phase;
  __device__ void next(int slots) {
    if (++slot == slots) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// The vectors of row x that CTA `rank` of `cl` takes.
struct Part {
  Split sp;
  int lo, n;
};
template <typename T>
__device__ __forceinline__ Part part_of(const T* x, int V, int rank, int cl) {
  Part p;
  p.sp = split_row(x, V);
  const int per = (p.sp.nb + cl - 1) / cl;
  p.lo = min(rank * per, p.sp.nb);
  p.n = min(per, p.sp.nb - p.lo);
  return p;
}

// Rows whose weight is 0 get a zero gradient without being read.
template <int MODE>
__device__ __forceinline__ bool row_blank(const Head& h, float w) {
  return !h.live || h.malformed || (MODE == LM_SCALED && w == 0.0f);
}

// Maximum and sum of a warp's (base, sum) pairs; -inf beside 0 is nothing.
__device__ __forceinline__ void join_lanes(float& mb, float& s, int n) {
  const float M = lanes_max(mb, n, FULL_MASK);
  s = lanes_sum(mb == NEG_INF && s == 0.0f ? 0.0f : s * ex2(mb - M), n, FULL_MASK);
  mb = M;
}

// This thread's vectors of a chunk, -inf where the chunk ends before them.
template <typename T>
__device__ __forceinline__ void take_chunk(uint4 (&raw)[RING_NV], const uint4* chunk, int gt, int GT,
                                           int have) {
  if (have >= RING_NV * GT) {
#pragma unroll
    for (int i = 0; i < RING_NV; ++i) raw[i] = chunk[i * GT + gt];
  } else {
#pragma unroll
    for (int i = 0; i < RING_NV; ++i) {
      constexpr uint32_t none = Vec<T>::LOWEST;
      raw[i] = make_uint4(none, none, none, none);
      if (i * GT + gt < have) raw[i] = chunk[i * GT + gt];
    }
  }
}

template <typename T, int MODE, bool GRAD>
__global__ void __launch_bounds__(RING_THREADS, 1)
    loss_ring_kernel(const __grid_constant__ RowArgs a, const RingShape shape) {
  constexpr int VE = vec_of<T>;
  constexpr bool PASS1 = MODE != LM_SCALED;
  extern __shared__ __align__(128) unsigned char ring_smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int W = shape.W, slots = shape.slots, cl = shape.cl, groups = RING_WARPS / W;
  const int chunk_vecs = W * 32 * RING_NV;
  const size_t ring_bytes = (size_t)slots * W * RING_WARP_BYTES;
  RingBars& bars = *reinterpret_cast<RingBars*>(ring_smem + groups * ring_bytes);
  float* teachers = reinterpret_cast<float*>(&bars + 1);
  const int rank = cl > 1 ? (int)cluster_ctarank() : 0;
  const int rows = a.B * a.T, V = a.V;  // rows <= 2^27
  const int units = (int)(gridDim.x / cl) * groups;

  if (blockIdx.x == 0 && tid == 0 && a.status) *a.status = 0;
  if (tid == 0) {
    for (int i = 0; i < groups * slots; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], W);
    }
    mbar_init(&bars.peer[0], 1);
    mbar_init(&bars.peer[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (cl > 1) cluster_sync();

  if (warp == RING_WARPS) {
    // ---- the copying warp: lane g feeds group g
    const bool mine = lane < groups;
    const int gi = mine ? lane : 0;
    unsigned char* ring = ring_smem + gi * ring_bytes;
    uint64_t* full = bars.full + gi * slots;
    uint64_t* empty = bars.empty + gi * slots;
    int r = (int)(blockIdx.x / cl) * groups + gi;
    bool done = !mine || r >= rows, open = false;
    HeadLoad next{};
    float next_w = 0.0f;
    if (!done) {
      next = load_head<MODE>(a, r);
      if (MODE == LM_SCALED) next_w = a.wseq[next.b];
    }
    Cursor cur{0, 0};
    const unsigned char* src = nullptr;
    int left = 0;
    int idle = 0;
    while (!__all_sync(FULL_MASK, done)) {
      bool moved = false;
      if (!done && !open) {
        // the head loaded a row ahead; skip rows that are not read
        if (r >= rows) {
          done = true;
        } else {
          const Head h = make_head<MODE>(a, next);
          if (!row_blank<MODE>(h, next_w)) {
            const T* x = row_at<T>(a.x, r, a.ldx);
            const Part p = part_of(x, V, rank, cl);
            src = reinterpret_cast<const unsigned char*>(x + p.sp.head) + (size_t)p.lo * 16;
            left = p.n;
            open = left > 0;
          }
          r += units;
          if (r < rows) {
            next = load_head<MODE>(a, r);
            if (MODE == LM_SCALED) next_w = a.wseq[next.b];
          }
        }
        moved = true;
      } else if (open && mbar_test(&empty[cur.slot], cur.phase ^ 1)) {
        const int n = min(left, chunk_vecs);
        mbar_expect_tx(&full[cur.slot], n * 16);
        bulk_g2s(ring + (size_t)cur.slot * W * RING_WARP_BYTES, src, n * 16, &full[cur.slot]);
        src += (size_t)n * 16;
        left -= n;
        open = left > 0;
        cur.next(slots);
        moved = true;
      }
      if (__any_sync(FULL_MASK, moved)) {
        idle = 0;
      } else {
        __nanosleep(64);
        if (++idle >= WAIT_SPIN_LIMIT) {
          if (lane == 0 && a.status) set_status(a.status, ST_DEVICE_TIMEOUT);
          break;
        }
      }
    }
    // the CTA's shared memory outlives its copies: wait for those still in flight
    if (mine)
      for (int i = 0; i < slots; ++i) {
        // a slot's last copy: of this pass over the ring, or of the one before (a
        // barrier that was never used counts as past that one)
        mbar_wait(&full[i], i < cur.slot ? cur.phase : cur.phase ^ 1, WAIT_SPIN_LIMIT);
      }
    return;
  }

  // ---- consumers
  const int gi = warp / W, gw = warp - gi * W, gt = gw * 32 + lane, GT = W * 32;
  const unsigned char* ring = ring_smem + gi * ring_bytes;
  uint64_t* full = bars.full + gi * slots;
  uint64_t* empty = bars.empty + gi * slots;
  float* tm = teachers + (size_t)gi * (MODE == LM_DISTILL ? TEACHER_WORDS * a.k : 0);
  const Teacher tc{tm, reinterpret_cast<int*>(tm + a.k), tm + 2 * a.k, tm + 3 * a.k};
  auto group_sync = [&]() {
    if (W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + gi), "r"(GT) : "memory");
  };
  bool dead = false;  // a wait gave up: wait no more
  auto gave_up = [&]() {
    dead = true;
    if (a.status) set_status(a.status, ST_DEVICE_TIMEOUT);
  };

  Cursor cur{0, 0};
  int turn = 0;  // rows joined so far, modulo 2
  uint32_t peer_phase = 0;
  int r = (int)(blockIdx.x / cl) * groups + gi;
  HeadLoad next{};
  float next_w = 0.0f;
  if (r < rows) {
    next = load_head<MODE>(a, r);
    if (MODE == LM_SCALED) next_w = a.wseq[next.b];
  }
  for (; r < rows; r += units) {
    const Head h = make_head<MODE>(a, next);
    const float w = next_w;
    if (r + units < rows) {
      next = load_head<MODE>(a, r + units);
      if (MODE == LM_SCALED) next_w = a.wseq[next.b];
    }
    const T* x = row_at<T>(a.x, r, a.ldx);
    T* g = GRAD ? row_at<T>(a.g, r, a.ldg) : nullptr;
    const Part p = part_of(x, V, rank, cl);
    const int head = p.sp.head, n = p.n;
    // gradient rows of another alignment are stored element by element
    const bool same =
        GRAD && ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15) == 0;
    T* gb = GRAD ? g + head + (size_t)p.lo * VE : nullptr;
    const int ei = rank == 0 && gt < p.sp.edge ? edge_index<T>(p.sp, gt) : -1;

    auto fill_zero = [&]() {
      if (!GRAD || a.add) return;
      for (int i = gt; i < n; i += GT) {
        if (same) {
          reinterpret_cast<uint4*>(gb)[i] = make_uint4(0, 0, 0, 0);
        } else {
          for (int e = 0; e < VE; ++e) gb[(size_t)i * VE + e] = from_f32<T>(0.0f);
        }
      }
      if (ei >= 0) g[ei] = from_f32<T>(0.0f);
    };
    if (row_blank<MODE>(h, w)) {
      if (PASS1 && gt == 0 && rank == 0) blank_outputs<MODE>(a, r, h.live);
      fill_zero();
      continue;
    }

    const int chunks = (n + chunk_vecs - 1) / chunk_vecs;
    float xe = ei >= 0 ? to_f32<T>(x[ei]) : NEG_INF;
    const LabelIn in = load_label<T, MODE>(a, r, h, x);
    const Range rg = rank == 0 ? Range{0, head + n * VE, head + p.sp.nb * VE}
                               : Range{head + p.lo * VE, head + (p.lo + n) * VE, V};
    TeacherHead th{};
    if (MODE == LM_DISTILL && gw == 0) {
      th = teacher_head<T>(a, r, tc, x, g, rg, lane, 32, FULL_MASK);
      if (lane == 0) {
        bars.tshare[turn][gi][0] = th.P;
        bars.tshare[turn][gi][1] = th.malformed ? 1.0f : 0.0f;
      }
    }

    Base base;
    float S = 0.0f;
    const Cursor start = cur;
    if (PASS1) {
      float mb = xe == NEG_INF ? NEG_INF : xe * a.sl;
      float s = ei >= 0 ? ex2(mb == NEG_INF ? NEG_INF : fmaf(xe, a.sl, -mb)) : 0.0f;
      for (int c = 0; c < chunks; ++c) {
        if (!dead && !mbar_wait(&full[cur.slot], cur.phase, WAIT_SPIN_LIMIT)) gave_up();
        const uint4* chunk =
            reinterpret_cast<const uint4*>(ring + (size_t)cur.slot * W * RING_WARP_BYTES);
        uint4 raw[RING_NV];
        take_chunk<T>(raw, chunk, gt, GT, n - c * chunk_vecs);
        if (!GRAD) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[cur.slot]);
        }
        const float nb = fmaxf(mb, Vec<T>::greatest(raw) * a.sl);
        const float at = nb == NEG_INF ? 0.0f : nb;  // nothing above -inf yet: exponentials of 0
        const f32x2 sl2 = pair(a.sl, a.sl), at2 = pair(-at, -at);
        f32x2 sum2[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
#pragma unroll
        for (int i = 0; i < RING_NV; ++i) {
          f32x2 v[Vec<T>::PAIRS];
          Vec<T>::unpack(raw[i], v);
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e)
            sum2[e & 1] = add2(sum2[e & 1], ex2_2(fma2(v[e], sl2, at2)));
        }
        float sum, odd;
        halves(add2(sum2[0], sum2[1]), sum, odd);
        sum += odd;
        s = (mb == NEG_INF && s == 0.0f ? 0.0f : s * ex2(mb - nb)) + sum;
        mb = nb;
        cur.next(slots);
      }
      // ---- the row's base and sum
      join_lanes(mb, s, 32);
      if (W > 1) {
        if (lane == 0) bars.red[turn][warp] = make_float2(mb, s);
        group_sync();
        const float2 mine = lane < W ? bars.red[turn][gi * W + lane] : make_float2(NEG_INF, 0.0f);
        mb = mine.x;
        s = mine.y;
        join_lanes(mb, s, 32);
      } else if (MODE == LM_DISTILL) {
        __syncwarp();
      }
      if (cl > 1) {
        // one group a CTA here (W == RING_WARPS); two barriers and two sets of
        // slots, so that a peer's next row cannot meet this one's
        if (gt == 0) mbar_expect_tx(&bars.peer[turn], 8 * cl);
        if (gt < cl) {
          st_async_cluster(&bars.part[turn][rank].x, &bars.peer[turn], gt, mb);
          st_async_cluster(&bars.part[turn][rank].y, &bars.peer[turn], gt, s);
        }
        __syncwarp();
        if (!dead && !mbar_wait_cluster(&bars.peer[turn], peer_phase, WAIT_SPIN_LIMIT)) gave_up();
        if (turn) peer_phase ^= 1;
        const float2 mine = lane < cl ? bars.part[turn][lane] : make_float2(NEG_INF, 0.0f);
        mb = mine.x;
        s = mine.y;
        join_lanes(mb, s, 32);
      }
      base.at = mb;
      base.direct = true;
      S = s;
      if (!(fabsf(mb) <= F32_MAX)) {
        // the scaled scores leave float32 (or the row holds nothing but -inf,
        // or an infinity): once more over the row, differences first
        float m = NEG_INF;
        for (int i = gt; i < V; i += GT) m = fmaxf(m, to_f32<T>(x[i]));
        m = group_max(m, 32);
        if (W > 1) {
          group_sync();
          if (lane == 0) bars.red[turn][warp].x = m;
          group_sync();
          m = group_max(lane < W ? bars.red[turn][gi * W + lane].x : NEG_INF, 32);
        }
        float t = 0.0f;
        for (int i = gt; i < V; i += GT) t += ex2((to_f32<T>(x[i]) - m) * a.sl);
        t = group_sum(t, 32);
        if (W > 1) {
          group_sync();
          if (lane == 0) bars.red[turn][warp].y = t;
          group_sync();
          t = group_sum(lane < W ? bars.red[turn][gi * W + lane].y : 0.0f, 32);
        }
        base.at = m;
        base.direct = false;
        S = t;
      }
    }

    float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
    bool blank = false;
    if (MODE == LM_SCALED) {
      base = unpack_stat(a.stat[r], S);
      cy = (float)((double)w * a.s);
      cq = -cy;
    } else if (MODE == LM_DISTILL) {
      P = bars.tshare[turn][gi][0];
      blank = bars.tshare[turn][gi][1] != 0.0f;
      if (blank) {
        if (gt == 0 && rank == 0) blank_outputs<MODE>(a, r, true);
      } else if (gw == 0) {
        teacher_terms(a, r, tc, th, base, S, rank == 0, lane, 32, FULL_MASK);
      }
      cq = (float)((a.w ? a.w[h.b] : 1.0) / a.s);
      if (GRAD && a.add) group_sync();  // the gradient's old values at the entries are read
    } else {
      cy = label_outputs<MODE>(a, r, in, base, S, gt == 0 && rank == 0);
      cq = -cy;
    }
    turn ^= 1;
    if (!GRAD) continue;

    const float scale = cq * P / S;
    cur = start;
    for (int c = 0; c < chunks; ++c) {
      if (!PASS1 && !dead && !mbar_wait(&full[cur.slot], cur.phase, WAIT_SPIN_LIMIT)) gave_up();
      const uint4* chunk =
          reinterpret_cast<const uint4*>(ring + (size_t)cur.slot * W * RING_WARP_BYTES);
      const int have = n - c * chunk_vecs;
      uint4 raw[RING_NV];
      take_chunk<T>(raw, chunk, gt, GT, have);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[cur.slot]);
#pragma unroll
      for (int i = 0; i < RING_NV; ++i) {
        if (i * GT + gt >= have) break;
        const size_t slot = (size_t)c * chunk_vecs + i * GT + gt;
        f32x2 v[Vec<T>::PAIRS];
        Vec<T>::unpack(raw[i], v);
        if (base.direct) {
          const f32x2 sl2 = pair(a.sl, a.sl), at2 = pair(-base.at, -base.at),
                      scale2 = pair(scale, scale);
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e) v[e] = mul2(ex2_2(fma2(v[e], sl2, at2)), scale2);
        } else {
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e) {
            float lo, hi;
            halves(v[e], lo, hi);
            v[e] = pair(based_exp(lo, a.sl, base) * scale, based_exp(hi, a.sl, base) * scale);
          }
        }
        if (MODE == LM_DISTILL && blank) {
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e) v[e] = pair(0.0f, 0.0f);
        }
        if (sizeof(T) == 4 && a.add) {
#pragma unroll
          for (int e = 0; e < Vec<T>::PAIRS; ++e)
            v[e] = add2(v[e], pair(to_f32<T>(gb[slot * VE + 2 * e]), to_f32<T>(gb[slot * VE + 2 * e + 1])));
        }
        const uint4 q = Vec<T>::pack(v);
        if (same) {
          reinterpret_cast<uint4*>(gb)[slot] = q;
        } else {
          const T* each = reinterpret_cast<const T*>(&q);
#pragma unroll
          for (int e = 0; e < VE; ++e) gb[slot * VE + e] = each[e];
        }
      }
      cur.next(slots);
    }
    if (ei >= 0) {
      float gv = blank ? 0.0f : based_exp(xe, a.sl, base) * scale;
      if (a.add) gv += to_f32<T>(g[ei]);
      g[ei] = from_f32<T>(gv);
    }
    if (has_label(MODE)) {
      // the thread that wrote the label's element puts it right
      const int at = h.y - head - p.lo * VE;
      const bool owner = at >= 0 && at < n * VE ? at / VE % GT == gt : ei == h.y;
      if (owner) {
        float gv = based_exp(in.xy, a.sl, base) * scale + cy;
        if (a.add) gv = to_f32<T>(g[h.y]) + cy;
        g[h.y] = from_f32<T>(gv);
      }
    } else {
      group_sync();  // this CTA's part of the row is written; its teacher entries follow
      if (gw == 0 && !blank) teacher_fix<T>(a, tc, g, base, scale, cq, lane, 32, rg);
      __syncwarp();
    }
  }
}

// Warps a group: enough rows in flight to hide one row's join behind the
// others', without cutting the rings below a row and a half.
inline int ring_warps(size_t row_bytes) {
  int W = 1;
  while (W < RING_WARPS && row_bytes > (size_t)W * 8 * 1024) W *= 2;
  return W;
}

// False where a row with a gradient does not fit the rings of a cluster.
template <typename T, int MODE>
bool launch_ring(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  const bool grad = a.g != nullptr;
  const bool hold = grad && MODE != LM_SCALED && MODE != LM_PREFERENCE;  // the row stays in the ring between the passes
  const size_t row = (size_t)a.V * sizeof(T);
  const size_t entry = MODE == LM_DISTILL ? (size_t)TEACHER_WORDS * a.k * sizeof(float) : 0;
  RingShape s;
  s.W = ring_warps(row);
  while (s.W < RING_WARPS && RING_WARPS / s.W * entry > 24 * 1024) s.W *= 2;
  size_t room, chunk;
  for (;; s.W *= 2) {
    const int groups = RING_WARPS / s.W;
    chunk = (size_t)s.W * RING_WARP_BYTES;
    room = (RING_SMEM - sizeof(RingBars) - groups * entry) / groups;
    s.slots = (int)std::min<size_t>(RING_SLOTS_MAX, room / chunk);
    if (!hold || row <= (size_t)(s.slots - 1) * chunk || s.W == RING_WARPS) break;
  }
  s.cl = 1;
  if (hold && row > (size_t)(s.slots - 1) * chunk)
    while (s.cl <= RING_CLUSTER_MAX && row > (size_t)s.cl * (s.slots - 1) * chunk) s.cl *= 2;
  if (s.cl > RING_CLUSTER_MAX) return false;
  const int groups = RING_WARPS / s.W;
  const size_t smem = groups * (s.slots * chunk + entry) + sizeof(RingBars);
  void (*kern)(const RowArgs, const RingShape) =
      grad ? (void (*)(const RowArgs, const RingShape))loss_ring_kernel<T, MODE, MODE != LM_PREFERENCE>
           : (void (*)(const RowArgs, const RingShape))loss_ring_kernel<T, MODE, MODE == LM_SCALED>;
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return true;
  const long long rows = (long long)a.B * a.T;
  const long long want = (rows + groups - 1) / groups * s.cl;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(RING_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = s.cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = s.cl > 1 ? 1 : 0;
  const int sms = loss_sm_count();
  cfg.gridDim = dim3((unsigned)std::min<long long>(want, sms / s.cl * s.cl));
  e = cudaLaunchKernelEx(&cfg, kern, a, s);
  return true;
}
