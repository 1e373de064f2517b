// loss_ring.cuh -- long rows: persistent CTAs that stream rows through rings of
// shared-memory chunks (included by loss_row.cuh).
//
// The warps of a CTA have roles, and pass rows on to one another through
// mbarriers, so that copies, both passes and a position's scalar work overlap:
//   copier    (one warp)  issues the TMA bulk copies of every group's ring;
//   reducers  take each chunk as it arrives: running maximum and sum of
//             exponentials;
//   scalar    (one warp a group) joins the reducers' pairs (and, for a row wider
//             than a ring, those of the CTAs of a cluster, through distributed
//             shared memory), computes the position's terms, looks after the
//             row's unaligned ends, and publishes what the writers need;
//   teachers  (distillation; two or three warps a group, which take its rows in
//             turn) take the teacher's entries in ahead of the row, compute the
//             position's loss and put the entries into the gradient behind the
//             writers;
//   writers   compute the gradient from the same chunks, still in shared
//             memory, and give them back to the ring.
// A row is read from memory once.  While its gradient is written the next row
// arrives and is reduced.  Without a gradient all warps reduce; in the second
// pass of the preference loss (LM_SCALED) all of them write.
//
// The 16 reducing and writing warps form groups of W, each with a ring of its
// own and a row at a time: short rows need several rows in flight.
//
// What bounds it.  8192 rows of 131072 bfloat16, policy loss and gradient: 4.3
// GB in 700 us (6.1 TB/s, 94% of the copy rate), 785 us once the clocks have
// dropped under load; two exponentials an element keep the special-function
// units at 68%.  With all 16 warps first reducing, then writing, memory stood
// still during the first half and the join: 974 us.  Taking every fourth pair
// of exponentials with a polynomial on the FMA pipe instead changed nothing
// there (979), nor did 24 warps (1049) or chunks of half the size (1026).
// Forward only, 2.1 GB: 300 us.  A row goes through three hand-overs, 1 to 2 us,
// which is what rows below 16 KB see (12000 bfloat16: 0.85 of the copy rate).
//
// Every wait is bounded: one that gives up records ST_DEVICE_TIMEOUT in the
// status word, and its thread runs on without waiting (every access stays
// within the rows and the rings), so that the kernel ends.  It passes nothing on
// any more, neither to the barriers of its CTA (a chunk given back twice would be
// filled twice at once) nor to the other CTAs of its cluster, so that their waits
// give up in turn; and a CTA to which others may still send ends last.

constexpr int RING_WARPS = 16;                      // reducers and writers of a CTA
constexpr int RING_GROUPS = 8;                      // at most
constexpr int RING_GROUPS_DISTILL = 4;              // at most, with its teacher warps:
constexpr int TEACHERS_MAX = 3;
__host__ __device__ constexpr int teacher_warps(int groups) { return groups == 4 ? 2 : TEACHERS_MAX; }
// A teacher warp that skips a row's `written` phase knows it closed before it looks at
// the next: its next row's note means that the note two rows before is free again.
static_assert(teacher_warps(1) >= 2 && teacher_warps(2) >= 2 && teacher_warps(4) >= 2,
              "a teacher warp takes at most every second row");
template <int MODE>
constexpr int ring_threads =  // at most
    (RING_WARPS + 1 +
     (MODE == LM_DISTILL ? RING_GROUPS_DISTILL * (1 + teacher_warps(RING_GROUPS_DISTILL))
                         : RING_GROUPS)) * 32;
constexpr int RING_NV = 4;                          // vectors of a chunk a thread takes
constexpr int RING_WARP_BYTES = RING_NV * 32 * 16;  // a warp's part of a chunk
constexpr int RING_SLOTS_MAX = 16;                  // chunks of a group's ring
constexpr int RING_CLUSTER_MAX = 8;
constexpr int RING_SMEM = 224 * 1024;

struct RingShape {
  int W;      // warps of a group
  int slots;  // chunks of a group's ring
  int cl;     // CTAs that share a row
#ifdef SEMICRF_BOUNDS_CHECK
  int stall;  // semicrf_selftest_ring_stall; 0: none
#endif
};

// What the scalar warp tells the writers about a row.
struct RowNote {
  float at, scale, cy, gy;  // base, factor of the exponentials, addend and value at the label
  int y;                    // the label (-1: none)
  int kind;                 // NOTE_*
  float sum;                // of the exponentials (for the teacher warps)
};
constexpr int NOTE_DIRECT = 0, NOTE_DIFFERENCE = 1, NOTE_ZERO = 2;

// What a teacher warp tells the scalar warp about a row.
struct TeacherNote {
  float P;    // the entries' total probability
  int blank;  // why the row has no gradient: ENTRY_OUTSIDE the labels, ENTRY_NONE in use
};
constexpr int ENTRY_OUTSIDE = 1, ENTRY_NONE = 2;

// float32 words of a teacher warp's entries.
__host__ __device__ inline size_t teacher_entry(int k, int V) {
  return (size_t)TEACHER_WORDS * k + teacher_table(k, V);
}

struct GroupState {
  uint64_t full[RING_SLOTS_MAX], empty[RING_SLOTS_MAX];
  uint64_t red_full[2], red_free[2], note_full[2], note_free[2], peer[2];
  // a teacher warp's own, a phase for each of its rows: barriers that alternate with
  // all rows may be two phases on when it looks
  uint64_t teacher_full[TEACHERS_MAX], told[TEACHERS_MAX], written[TEACHERS_MAX];
  float2 red[2][RING_WARPS];
  float2 part[2][RING_CLUSTER_MAX];
  RowNote note[2];
  TeacherNote teacher[TEACHERS_MAX];
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

// Rows alternate between two sets of barriers and slots: which, and its parity.
struct Turn {
  int i;
  uint32_t phase;
  __device__ void next() {
    phase ^= (uint32_t)i;
    i ^= 1;
  }
};

// A thread's waits and arrivals, which end once and for all when one wait gives up.
struct Waiter {
  int* status;
  int spins;
  bool dead;
  __device__ void operator()(uint64_t* bar, uint32_t parity) {
    if (!dead && !mbar_wait(bar, parity, spins)) give_up();
  }
  __device__ void give_up() {
    dead = true;
    if (status) set_status(status, ST_DEVICE_TIMEOUT);
  }
  __device__ void arrive(uint64_t* bar) const {
    if (!dead) mbar_arrive(bar);
  }
};

// This warp is done with a chunk.  Its reads are ordinary accesses and the copy
// that follows is an asynchronous one: without the fence between the two the
// copy may overtake reads that are still under way.
__device__ __forceinline__ void give_back(const Waiter& wait, uint64_t* empty, int lane) {
  fence_proxy_async();
  __syncwarp();
  if (lane == 0) wait.arrive(empty);
}

// The vectors of row x that CTA `rank` of `cl` takes.
struct Part {
  Split sp;
  int lo, n;
};
template <typename T>
__device__ __forceinline__ Part part_of(const T* x, int V, int rank, int cl) {
  Part p;
  p.sp = split_row(x, V);
  if (cl == 1) {
    p.lo = 0;
    p.n = p.sp.nb;
  } else {
    const int per = (p.sp.nb + cl - 1) / cl;
    p.lo = min(rank * per, p.sp.nb);
    p.n = min(per, p.sp.nb - p.lo);
  }
  return p;
}

// Row i of a pass.  The second pass of the preference loss runs backwards: what
// the first read last is still in L2.
template <int MODE>
__device__ __forceinline__ int pass_row(int i, int rows) {
  return MODE == LM_SCALED ? rows - 1 - i : i;
}

// Heads of a unit's rows, loaded a row ahead.
template <int MODE>
struct HeadStream {
  HeadLoad next;
  float next_w;
  __device__ void load(const RowArgs& a, int r, int rows) {
    if (r >= rows) return;
    next = load_head<MODE>(a, pass_row<MODE>(r, rows));
    if (MODE == LM_SCALED) next_w = a.wseq[next.b];
  }
  // Rows that do not count, and rows of weight 0, are not read.
  __device__ Head take(const RowArgs& a, float& w, bool& blank) const {
    const Head h = make_head<MODE>(a, next);
    w = next_w;
    blank = !h.live || h.malformed || (MODE == LM_SCALED && w == 0.0f);
    return h;
  }
};

// Maximum over a warp (a NaN is ignored, as fmaxf does).
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Maximum and sum of a warp's (base, sum) pairs; -inf beside 0 is nothing.
__device__ __forceinline__ void join_lanes(float& mb, float& s) {
  const float M = warp_max(mb);
  s = group_sum(mb == NEG_INF && s == 0.0f ? 0.0f : s * ex2(mb - M), 32);
  mb = M;
}

// One more (base, sum) pair.
__device__ __forceinline__ void join_pair(float& mb, float& s, float mb2, float s2) {
  const float M = fmaxf(mb, mb2);
  s = (mb == NEG_INF && s == 0.0f ? 0.0f : s * ex2(mb - M)) +
      (mb2 == NEG_INF && s2 == 0.0f ? 0.0f : s2 * ex2(mb2 - M));
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

// What a role's loop over rows needs.
struct RingPlace {
  unsigned char* ring;
  GroupState* st;
  int first, units, rows;  // this group's rows: first, first + units, ...
  int rank, cl, slots, chunk_bytes;
  int teachers;  // warps
  int spins;     // polls before a wait gives up
};

// ---------------------------------------------------------------------- copier
template <typename T, int MODE>
__device__ __forceinline__ void ring_copier(const RowArgs& a, unsigned char* rings, GroupState* states,
                                            int groups, size_t ring_bytes, const RingPlace& pl,
                                            int lane) {
  const bool mine = lane < groups;
  unsigned char* ring = rings + (mine ? lane : 0) * ring_bytes;
  GroupState& st = states[mine ? lane : 0];
  int r = pl.first + lane;
  bool done = !mine || r >= pl.rows, open = false;
  HeadStream<MODE> heads{};
  if (!done) heads.load(a, r, pl.rows);
  Cursor cur{0, 0};
  const unsigned char *src = nullptr, *row = nullptr;
  int left = 0, idle = 0;
  while (!__all_sync(FULL_MASK, done)) {
    bool moved = false;
    if (!done && !open) {
      if (r >= pl.rows) {
        done = true;
      } else {
        float w;
        bool blank;
        heads.take(a, w, blank);
        if (!blank) {
          const T* x = row_at<T>(a.x, pass_row<MODE>(r, pl.rows), a.ldx);
          const Part p = part_of(x, a.V, pl.rank, pl.cl);
          row = reinterpret_cast<const unsigned char*>(x);
          src = row + (size_t)p.sp.head * sizeof(T) + (size_t)p.lo * 16;
          left = p.n * 16;
          open = left > 0;
        }
        r += pl.units;
        heads.load(a, r, pl.rows);
      }
      moved = true;
    } else if (open && mbar_test(&st.empty[cur.slot], cur.phase ^ 1)) {
      const int n = min(left, pl.chunk_bytes);
      if (SEMICRF_INB(a.status, cur.slot >= 0 && cur.slot < pl.slots && n > 0 && n % 16 == 0 &&
                                    reinterpret_cast<uintptr_t>(src) % 16 == 0 && src >= row &&
                                    src + n <= row + (size_t)a.V * sizeof(T),
                      SITE_LOSS_CHUNK)) {
        mbar_expect_tx(&st.full[cur.slot], n);
        bulk_g2s(ring + (size_t)cur.slot * pl.chunk_bytes, src, n, &st.full[cur.slot]);
        src += n;
        left -= n;
        open = left > 0;
        cur.next(pl.slots);
      } else {
        open = false;  // whoever waits for the chunk gives up
        done = true;
      }
      moved = true;
    }
    if (__any_sync(FULL_MASK, moved)) {
      idle = 0;
    } else {
      __nanosleep(100);
      if (++idle >= pl.spins) {
        if (lane == 0 && a.status) set_status(a.status, ST_DEVICE_TIMEOUT);
        break;
      }
    }
  }
  // The CTA's shared memory outlives its copies: wait for those still in flight.
  // A slot's last copy is of this pass over the ring or of the one before (a
  // barrier that was never used counts as past that one).
  if (mine)
    for (int i = 0; i < pl.slots; ++i)
      mbar_wait(&st.full[i], i < cur.slot ? cur.phase : cur.phase ^ 1, WAIT_SPIN_LIMIT);
}

// -------------------------------------------------------------------- reducers
// GT threads, this one gt.  RELEASE: nobody else needs the chunks.
template <typename T, int MODE, bool RELEASE>
__device__ __forceinline__ void ring_reduce(const RowArgs& a, const RingPlace& pl, int gt, int GT) {
  GroupState& st = *pl.st;
  const int lane = gt & 31, gw = gt >> 5, chunk_vecs = pl.chunk_bytes / 16;
  Waiter wait{a.status, pl.spins, false};
  Cursor cur{0, 0};
  Turn turn{0, 0};
  HeadStream<MODE> heads{};
  heads.load(a, pl.first, pl.rows);
  const f32x2 sl2 = pair(a.sl, a.sl);
  for (int r = pl.first; r < pl.rows; r += pl.units) {
    float w;
    bool blank;
    heads.take(a, w, blank);
    heads.load(a, r + pl.units, pl.rows);
    if (blank) continue;
    const int n = part_of(row_at<T>(a.x, r, a.ldx), a.V, pl.rank, pl.cl).n;
    float mb = NEG_INF, s = 0.0f;
    for (int c = 0; c < n; c += chunk_vecs) {
      wait(&st.full[cur.slot], cur.phase);
      uint4 raw[RING_NV];
      take_chunk<T>(raw, reinterpret_cast<const uint4*>(pl.ring + (size_t)cur.slot * pl.chunk_bytes),
                    gt, GT, n - c);
      const float nb = fmaxf(mb, Vec<T>::greatest(raw) * a.sl);
      // nothing but masked scores yet: their exponentials around 0 are 0, as beside any
      // score of a row whose base is direct (if there is none, the row is done again)
      const float at = nb < -BASE_MAX ? 0.0f : nb;
      const f32x2 at2 = pair(-at, -at);
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
      if (RELEASE) give_back(wait, &st.empty[cur.slot], lane);
      cur.next(pl.slots);
      s = (mb == NEG_INF && s == 0.0f ? 0.0f : s * ex2(mb - nb)) + (sum + odd);
      mb = nb;
    }
    join_lanes(mb, s);
    wait(&st.red_free[turn.i], turn.phase ^ 1);
    if (lane == 0 && SEMICRF_INB(a.status, gw >= 0 && gw < RING_WARPS, SITE_LOSS_SLOT)) {
      st.red[turn.i][gw] = make_float2(mb, s);
      wait.arrive(&st.red_full[turn.i]);
    }
    turn.next();
  }
}

// ---------------------------------------------------------------------- writers
template <typename T, int MODE>
__device__ __forceinline__ void ring_write(const RowArgs& a, const RingPlace& pl, int gt, int GT) {
  constexpr int VE = vec_of<T>;
  GroupState& st = *pl.st;
  const int lane = gt & 31, chunk_vecs = pl.chunk_bytes / 16;
  Waiter wait{a.status, pl.spins, false};
  Cursor cur{0, 0};
  Turn turn{0, 0};
  Cursor teacher{0, 0};
  const f32x2 sl2 = pair(a.sl, a.sl);
  for (int i = pl.first; i < pl.rows; i += pl.units) {
    const int r = pass_row<MODE>(i, pl.rows);
    const T* x = row_at<T>(a.x, r, a.ldx);
    T* g = row_at<T>(a.g, r, a.ldg);
    const Part p = part_of(x, a.V, pl.rank, pl.cl);
    // gradient rows of another alignment are stored element by element
    const bool same = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(g)) & 15) == 0;
    T* gb = g + p.sp.head + (size_t)p.lo * VE;
    wait(&st.note_full[turn.i], turn.phase);
    const RowNote note = st.note[turn.i];
    if (note.kind == NOTE_ZERO && note.y < 0) {  // not read: zeros, unless added to
      if (!a.add) {
        for (int i = gt; i < p.n; i += GT) {
          if (!vector_inside<T>(a, p.sp, p.lo + i)) continue;
          if (same) {
            reinterpret_cast<uint4*>(gb)[i] = make_uint4(0, 0, 0, 0);
          } else {
            for (int e = 0; e < VE; ++e) gb[(size_t)i * VE + e] = from_f32<T>(0.0f);
          }
        }
      }
    } else {
      const f32x2 at2 = pair(-note.at, -note.at), scale2 = pair(note.scale, note.scale);
      const bool plain = note.kind == NOTE_DIRECT && same && !a.add;
      for (int c = 0; c < p.n; c += chunk_vecs) {
        wait(&st.full[cur.slot], cur.phase);
        const uint4* chunk =
            reinterpret_cast<const uint4*>(pl.ring + (size_t)cur.slot * pl.chunk_bytes);
        const int have = p.n - c;
        if (plain) {
          uint4 raw[RING_NV];
          take_chunk<T>(raw, chunk, gt, GT, have);
#pragma unroll
          for (int i = 0; i < RING_NV; ++i) {
            f32x2 v[Vec<T>::PAIRS];
            Vec<T>::unpack(raw[i], v);
#pragma unroll
            for (int e = 0; e < Vec<T>::PAIRS; ++e)
              v[e] = mul2(ex2_2(fma2(v[e], sl2, at2)), scale2);
            raw[i] = Vec<T>::pack(v);
          }
          give_back(wait, &st.empty[cur.slot], lane);
          uint4* out = reinterpret_cast<uint4*>(gb) + c + gt;
          if (have >= chunk_vecs) {
#pragma unroll
            for (int i = 0; i < RING_NV; ++i)
              if (vector_inside<T>(a, p.sp, p.lo + c + gt + i * GT)) out[i * GT] = raw[i];
          } else {
#pragma unroll
            for (int i = 0; i < RING_NV; ++i)
              if (i * GT + gt < have && vector_inside<T>(a, p.sp, p.lo + c + gt + i * GT)) out[i * GT] = raw[i];
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < RING_NV; ++i) {
            const int at = i * GT + gt;
            if (at >= have || !vector_inside<T>(a, p.sp, p.lo + c + at)) break;
            const T* each = reinterpret_cast<const T*>(chunk + at);
            T* to = gb + (size_t)(c + at) * VE;
#pragma unroll 1
            for (int e = 0; e < VE; ++e) {
              float gv = 0.0f;
              if (note.kind == NOTE_DIRECT) gv = ex2(fmaf(to_f32<T>(each[e]), a.sl, -note.at)) * note.scale;
              if (note.kind == NOTE_DIFFERENCE) gv = ex2((to_f32<T>(each[e]) - note.at) * a.sl) * note.scale;
              if (a.add) gv += to_f32<T>(to[e]);
              to[e] = from_f32<T>(gv);
            }
          }
          give_back(wait, &st.empty[cur.slot], lane);
        }
        cur.next(pl.slots);
      }
      if (has_label(MODE)) {
        // the thread that wrote the label's element puts it right
        const int at = note.y - p.sp.head - p.lo * VE;
        if (at >= 0 && at < p.n * VE && at / VE % GT == gt &&
            SEMICRF_INB(a.status, note.y < a.V, SITE_LOSS_SCORE))
          g[note.y] = from_f32<T>(a.add ? to_f32<T>(g[note.y]) + note.cy : note.gy);
      }
    }
    __syncwarp();
    if (lane == 0) {
      if (MODE == LM_DISTILL) wait.arrive(&st.written[teacher.slot]);
      wait.arrive(&st.note_free[turn.i]);
    }
    if (MODE == LM_DISTILL) teacher.next(pl.teachers);
    turn.next();
  }
}

// ----------------------------------------------------------------- scalar warp
// Returns whether a wait gave up; `stall`: as if one had from the start.
template <typename T, int MODE, bool GRAD>
__device__ __forceinline__ bool ring_scalar(const RowArgs& a, const RingPlace& pl, int warps, int lane,
                                            bool stall) {
  constexpr bool PASS1 = MODE != LM_SCALED;
  constexpr bool NOTES = GRAD || MODE == LM_DISTILL;
  GroupState& st = *pl.st;
  Waiter wait{a.status, pl.spins, false};
  if (stall) wait.give_up();
  Turn turn{0, 0}, rows_read{0, 0};
  Cursor teacher{0, 0};
  HeadStream<MODE> heads{};
  heads.load(a, pl.first, pl.rows);
  auto publish = [&](const RowNote& note) {
    wait(&st.note_free[turn.i], turn.phase ^ 1);
    __syncwarp();
    if (lane == 0) {
      st.note[turn.i] = note;
      wait.arrive(&st.note_full[turn.i]);
      if (MODE == LM_DISTILL) wait.arrive(&st.told[teacher.slot]);
    }
  };
  for (int i = pl.first; i < pl.rows; i += pl.units) {
    const int r = pass_row<MODE>(i, pl.rows);
    float w;
    bool blank;
    const Head h = heads.take(a, w, blank);
    heads.load(a, i + pl.units, pl.rows);
    const T* x = row_at<T>(a.x, r, a.ldx);
    T* g = GRAD ? row_at<T>(a.g, r, a.ldg) : nullptr;
    const Part p = part_of(x, a.V, pl.rank, pl.cl);
    int ei = pl.rank == 0 && lane < p.sp.edge ? edge_index<T>(p.sp, lane) : -1;
    if (ei >= 0 && !edge_inside(a, ei)) ei = -1;
    RowNote note{};
    note.kind = NOTE_ZERO;
    note.y = -1;
    const Turn now = turn;
    if (blank) {
      if (PASS1 && pl.rank == 0 && lane == 0) blank_outputs<MODE>(a, r, h.live);
      if (GRAD && !a.add && ei >= 0) g[ei] = from_f32<T>(0.0f);
      // (this row's phase is taken note of)
      if (MODE == LM_DISTILL) wait(&st.teacher_full[teacher.slot], teacher.phase);
    } else {
      const LabelIn<T> in = load_label<T, MODE>(a, r, h, x);
      T xe = from_f32<T>(0.0f);
      if (ei >= 0) xe = x[ei];
      Base base;
      float S;
      if (PASS1) {
        wait(&st.red_full[rows_read.i], rows_read.phase);
        float mb = NEG_INF, s = 0.0f;
        if (lane < warps) {
          const float2 v = st.red[rows_read.i][lane];
          mb = v.x;
          s = v.y;
        }
        __syncwarp();
        if (lane == 0) wait.arrive(&st.red_free[rows_read.i]);
        if (ei >= 0) {
          const float xv = to_f32<T>(xe), eb = xv * a.sl;
          join_pair(mb, s, eb, eb < -BASE_MAX ? 0.0f : ex2(fmaf(xv, a.sl, -eb)));
        }
        join_lanes(mb, s);
        if (pl.cl > 1) {
          // two barriers and two sets of slots, so that a peer's next row cannot
          // meet this one's
          uint64_t* bar = &st.peer[rows_read.i];
          if (lane == 0 && !wait.dead) mbar_expect_tx(bar, 8 * pl.cl);
          __syncwarp();
          if (lane < pl.cl && !wait.dead &&
              SEMICRF_INB(a.status, pl.cl <= RING_CLUSTER_MAX && pl.rank < pl.cl, SITE_LOSS_SLOT)) {
            st_async_cluster(&st.part[rows_read.i][pl.rank].x, bar, lane, mb);
            st_async_cluster(&st.part[rows_read.i][pl.rank].y, bar, lane, s);
          }
          if (!wait.dead && !mbar_wait_cluster(bar, rows_read.phase, pl.spins)) wait.give_up();
          mb = NEG_INF;
          s = 0.0f;
          if (lane < pl.cl) {
            const float2 v = st.part[rows_read.i][lane];
            mb = v.x;
            s = v.y;
          }
          join_lanes(mb, s);
        }
        rows_read.next();
        base.at = mb;
        base.direct = fabsf(mb) <= BASE_MAX;
        S = s;
        if (!base.direct) {
          // the scaled maximum is too far from 0 (or the row holds nothing but -inf,
          // or an infinity): once more over the row, differences first
          float m = NEG_INF;
          for (int i = lane; i < a.V; i += 32) m = fmaxf(m, to_f32<T>(x[i]));
          m = warp_max(m);
          double part = 0.0;  // a lane's terms are V / 32: too many for a float32 sum
          for (int i = lane; i < a.V; i += 32) part += (double)ex2((to_f32<T>(x[i]) - m) * a.sl);
          S = group_sum((float)part, 32);
          base.at = m;
        }
      } else {
        base = unpack_stat(in.stat, S);
      }

      float cq, cy = 0.0f, P = 1.0f;  // gradient of the row: cq q_v, and cy more at the label
      bool zero = false;
      if (MODE == LM_SCALED) {
        cy = (float)((double)w * a.s);
        cq = -cy;
      } else if (MODE == LM_DISTILL) {
        wait(&st.teacher_full[teacher.slot], teacher.phase);
        P = st.teacher[teacher.slot].P;
        // without an entry P is 0, and so is the row's factor: its writers need not be
        // told, unless the row has no sum
        const int blank_entries = st.teacher[teacher.slot].blank;
        zero = blank_entries == ENTRY_OUTSIDE || (blank_entries == ENTRY_NONE && !(S <= F32_MAX));
        cq = (float)(in.w * a.tau);
      } else {
        cy = label_outputs<MODE>(a, r, in, base, S, lane == 0 && pl.rank == 0);
        cq = -cy;
      }
      const float scale = __fdividef(cq * P, S);
      if (NOTES) {
        note.at = base.at;
        note.scale = scale;
        note.cy = cy;
        note.sum = S;
        note.kind = zero ? NOTE_ZERO : base.direct ? NOTE_DIRECT : NOTE_DIFFERENCE;
        note.y = has_label(MODE) ? h.y : 0;  // >= 0: the row's chunks are in the ring
        if (has_label(MODE)) note.gy = based_exp(in.xy(), a.sl, base) * scale + cy;
        publish(note);
      }
      if (GRAD && ei >= 0 && !(zero && a.add)) {
        float gv = zero ? 0.0f : based_exp(to_f32<T>(xe), a.sl, base) * scale;
        if (has_label(MODE) && ei == h.y) gv += cy;
        if (a.add) gv += to_f32<T>(g[ei]);
        g[ei] = from_f32<T>(gv);
      }
    }
    if (NOTES) {
      if (blank) publish(note);
      if (MODE == LM_DISTILL) {
        __syncwarp();  // the edges are written: the teacher warp may change them
        if (GRAD && lane == 0) wait.arrive(&st.written[teacher.slot]);
        teacher.next(pl.teachers);
      }
      turn.next();
    }
  }
  return wait.dead;
}

// --------------------------------------------------------------- teacher warps
// Number `me` of pl.teachers, which take the group's rows in turn.  With the
// entries in the scalar warp's hands the writers waited for the next row's
// gathers: 2 x 1024 x 100003 float32 with 128 entries took 384 us, 333 with one
// warp for the entries, 293 with three.
template <typename T, bool GRAD>
__device__ __forceinline__ void ring_teacher(const RowArgs& a, const RingPlace& pl, float* entries,
                                             int me, int lane) {
  constexpr int VE = vec_of<T>;
  GroupState& st = *pl.st;
  Waiter wait{a.status, pl.spins, false};
  const int step = pl.units * pl.teachers;
  const Teacher tc{entries, reinterpret_cast<int*>(entries + a.k), entries + 2 * a.k,
                   entries + 3 * a.k, reinterpret_cast<int*>(entries + TEACHER_WORDS * a.k)};
  HeadStream<LM_DISTILL> heads{};
  TeacherAhead ahead{};
  int n = me, ahead_row = -1;  // the row's number in the group; the row that `ahead` is of
  uint32_t own = 1;            // parity of this warp's rows
  heads.load(a, pl.first + me * pl.units, pl.rows);
  for (int r = pl.first + me * pl.units; r < pl.rows; r += step, n += pl.teachers) {
    float w;
    bool blank;
    const Head h = heads.take(a, w, blank);
    heads.load(a, r + step, pl.rows);
    const T* x = row_at<T>(a.x, r, a.ldx);
    T* g = GRAD ? row_at<T>(a.g, r, a.ldg) : nullptr;
    TeacherHead th{};
    Range rg{};
    float cq = 0.0f;
    if (!blank) {
      const LabelIn<T> in = load_label<T, LM_DISTILL>(a, r, h, x);
      const Part p = part_of(x, a.V, pl.rank, pl.cl);
      rg = pl.rank == 0 ? Range{0, p.sp.head + p.n * VE, p.sp.head + p.sp.nb * VE}
                        : Range{p.sp.head + p.lo * VE, p.sp.head + (p.lo + p.n) * VE, a.V};
      cq = (float)(in.w * a.tau);
      if (ahead_row != r) ahead.load(a, r, 0, lane, 32);
      th = teacher_head<T>(a, r, in.lse, tc, ahead, x, g, rg, lane, 32, FULL_MASK);
      ahead_row = r + step;
      if (ahead_row < pl.rows) ahead.load(a, ahead_row, 0, lane, 32);
    }
    __syncwarp();  // (accumulation: all have read the values that the writers will change)
    if (lane == 0) {
      st.teacher[me] = TeacherNote{th.P, th.malformed ? ENTRY_OUTSIDE : th.none ? ENTRY_NONE : 0};
      wait.arrive(&st.teacher_full[me]);
    }
    own ^= 1;
    const int i = n & 1;
    wait(&st.told[me], own);
    const RowNote note = st.note[i];
    __syncwarp();
    if (lane == 0) wait.arrive(&st.note_free[i]);
    if (blank) continue;
    if (th.malformed || th.none) {
      if (lane == 0 && pl.rank == 0) blank_outputs<LM_DISTILL>(a, r, th.malformed);
      continue;
    }
    const Base base{note.at, note.kind == NOTE_DIRECT};
    teacher_terms(a, r, tc, th, base, note.sum, pl.rank == 0, lane, 32, FULL_MASK);
    if (GRAD) {
      wait(&st.written[me], own);  // the row and its edges
      teacher_fix<T>(a, tc, g, base, note.scale, cq, th.repeats, lane, 32, rg);
    }
    __syncwarp();
  }
}

template <typename T, int MODE, bool GRAD>
__global__ void __launch_bounds__(ring_threads<MODE>, 1)
    loss_ring_kernel(const __grid_constant__ RowArgs a, const RingShape shape) {
  extern __shared__ __align__(128) unsigned char ring_smem[];
  constexpr bool PASS1 = MODE != LM_SCALED;
  constexpr bool BOTH = PASS1 && GRAD;  // half of a group's warps reduce, the others write
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = shape.W, groups = RING_WARPS / W;
  const int role_warps = BOTH ? W / 2 : W;
  RingPlace pl;
  pl.cl = shape.cl;
  pl.slots = shape.slots;
  pl.chunk_bytes = role_warps * RING_WARP_BYTES;
  pl.rank = pl.cl > 1 ? (int)cluster_ctarank() : 0;
  pl.rows = a.B * a.T;  // <= 2^27
  pl.units = (int)(gridDim.x / pl.cl) * groups;
#ifdef SEMICRF_BOUNDS_CHECK
  pl.spins = shape.stall ? shape.stall : WAIT_SPIN_LIMIT;
  const bool stall = shape.stall && pl.rank == pl.cl - 1;
#else
  pl.spins = WAIT_SPIN_LIMIT;
  constexpr bool stall = false;
#endif
  const size_t ring_bytes = (size_t)pl.slots * pl.chunk_bytes;
  GroupState* states = reinterpret_cast<GroupState*>(ring_smem + groups * ring_bytes);
  float* entries = reinterpret_cast<float*>(states + groups);
  pl.teachers = teacher_warps(groups);
  const int first = (int)(blockIdx.x / pl.cl) * groups;

  start_status(a);
  if (threadIdx.x < groups) {
    GroupState& st = states[threadIdx.x];
    for (int i = 0; i < pl.slots; ++i) {
      mbar_init(&st.full[i], 1);
      mbar_init(&st.empty[i], role_warps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&st.red_full[i], role_warps);
      mbar_init(&st.red_free[i], 1);
      mbar_init(&st.note_full[i], 1);
      // the writers and the row's teacher warp
      mbar_init(&st.note_free[i], (GRAD ? role_warps : 0) + (MODE == LM_DISTILL ? 1 : !GRAD));
      mbar_init(&st.peer[i], 1);
    }
    for (int i = 0; i < TEACHERS_MAX; ++i) {
      mbar_init(&st.teacher_full[i], 1);
      mbar_init(&st.told[i], 1);
      mbar_init(&st.written[i], role_warps + 1);  // the writers and, for the edges, the scalar warp
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (pl.cl > 1) cluster_sync();
  if (MODE == LM_SCALED) after_previous();

  const int teacher = warp - (RING_WARPS + groups + 1);
  const int gi = warp < RING_WARPS ? warp / W : teacher < 0 ? warp - RING_WARPS : teacher / pl.teachers;
  pl.first = first + gi;
  pl.ring = ring_smem + gi * ring_bytes;
  pl.st = states + gi;
  bool gave_up = false;
  if (warp == RING_WARPS + groups) {
    pl.first = first;
    ring_copier<T, MODE>(a, ring_smem, states, groups, ring_bytes, pl, lane);
  } else if (MODE == LM_DISTILL && teacher >= 0) {
    ring_teacher<T, GRAD>(a, pl, entries + teacher * teacher_entry(a.k, a.V), teacher % pl.teachers, lane);
  } else if (warp >= RING_WARPS) {
    gave_up = ring_scalar<T, MODE, GRAD>(a, pl, role_warps, lane, stall);
  } else {
    const int gw = warp - gi * W;
    if (BOTH) {
      if (gw < role_warps) ring_reduce<T, MODE, false>(a, pl, gw * 32 + lane, role_warps * 32);
      else ring_write<T, MODE>(a, pl, (gw - role_warps) * 32 + lane, role_warps * 32);
    } else if (PASS1) {
      ring_reduce<T, MODE, true>(a, pl, gw * 32 + lane, role_warps * 32);
    } else {
      ring_write<T, MODE>(a, pl, gw * 32 + lane, role_warps * 32);
    }
  }
  if (PASS1 && pl.cl > 1) {
    // A CTA that has had its peers' pairs of all rows may end, for they send no
    // more.  One that has not keeps its shared memory until every thread of the
    // cluster is through, and then until what they sent last has come.
    __syncwarp();
    cluster_arrive();
    if (__any_sync(FULL_MASK, gave_up)) {
      cluster_wait();
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
  }
}

// A kernel's limits on a device, asked for once.
struct RingLimits {
  std::atomic<uint64_t> raised{0};                       // devices whose shared-memory limit is raised
  std::atomic<int> clusters[RING_CLUSTER_MAX + 1][8]{};  // resident clusters of each size, device < 8
};

// Clusters of `cl` CTAs that run at once (a GPC need not hold a multiple of cl
// SMs: of 148 SMs clusters of 4 reach 132, clusters of 8 reach 120).
template <typename K>
cudaError_t resident_clusters(K kern, RingLimits& lim, int dev, int cl, int& n) {
  n = loss_sm_count();
  if (cl == 1) return cudaSuccess;
  if (dev < 8 && (n = lim.clusters[cl][dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(loss_sm_count() / cl * cl);
  cfg.blockDim = dim3((RING_WARPS + 2 + TEACHERS_MAX) * 32);  // one group's, at most
  cfg.dynamicSmemBytes = RING_SMEM;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
  n = std::max(n, 1);
  if (e == cudaSuccess && dev < 8) lim.clusters[cl][dev].store(n, std::memory_order_relaxed);
  return e;
}

// False where a row with a gradient does not fit the rings of a cluster.
template <typename T, int MODE>
bool launch_ring(const RowArgs& a, cudaStream_t st, cudaError_t& e) {
  const bool grad = a.g != nullptr && MODE != LM_PREFERENCE;
  const bool hold = grad && MODE != LM_SCALED;  // the row stays in the ring between the passes
  const size_t row = (size_t)a.V * sizeof(T);
  auto entries = [&](int groups) {
    return MODE == LM_DISTILL ? groups * teacher_warps(groups) * teacher_entry(a.k, a.V) * sizeof(float) : 0;
  };
  const long long rows = (long long)a.B * a.T;
  static RingLimits limits[2];
  RingLimits& lim = limits[grad];
  void (*kern)(const RowArgs, const RingShape) =
      grad ? (void (*)(const RowArgs, const RingShape))loss_ring_kernel<T, MODE, MODE != LM_PREFERENCE>
           : (void (*)(const RowArgs, const RingShape))loss_ring_kernel<T, MODE, MODE == LM_SCALED>;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return true;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(lim.raised.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kern),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, RING_SMEM);
    if (e != cudaSuccess) return true;
    lim.raised.fetch_or(bit, std::memory_order_relaxed);
  }
  const int sms = loss_sm_count();

  // Warps a group: 8 KB of a row for each (rows in flight hide one another's
  // latency), all 16 where there are too few rows for more groups.
  RingShape s;
#ifdef SEMICRF_BOUNDS_CHECK
  s.stall = loss_ring_stall();
#endif
  s.W = MODE == LM_DISTILL ? RING_WARPS / RING_GROUPS_DISTILL : 2;
  while (s.W < RING_WARPS &&
         (row > (size_t)s.W * 8 * 1024 || rows <= (long long)sms * (RING_WARPS / s.W) / 2 ||
          entries(RING_WARPS / s.W) > 64 * 1024))
    s.W *= 2;
  size_t chunk, fixed;
  for (;; s.W *= 2) {
    const int groups = RING_WARPS / s.W;
    chunk = (size_t)(hold ? s.W / 2 : s.W) * RING_WARP_BYTES;
    fixed = groups * sizeof(GroupState) + entries(groups);
    s.slots = (int)std::min<size_t>(RING_SLOTS_MAX, (RING_SMEM - fixed) / groups / chunk);
    if (!hold || row <= (size_t)(s.slots - 1) * chunk || s.W == RING_WARPS) break;
  }
  s.cl = 1;
  if (hold && s.W == RING_WARPS) {
    // a row takes at most 0.7 of the rings, so that the next one can follow it (90000
    // bfloat16: 368 us on two CTAs, 401 on one whose ring it fills to 0.9) ...
    const size_t ring = (s.slots - 1) * chunk;
    while (s.cl < RING_CLUSTER_MAX && row * 10 > s.cl * ring * 7) ++s.cl;
    if (row > s.cl * ring) return false;  // ... or all of the largest cluster's
  }
  int resident;
  e = resident_clusters(kern, lim, dev, s.cl, resident);
  if (e != cudaSuccess) return true;
  if (s.W == RING_WARPS && rows * s.cl * 2 <= sms) {
    // a handful of rows: each is spread over as many CTAs as they leave, 4 KB at least
    for (int cl = RING_CLUSTER_MAX; cl > s.cl; --cl) {
      int n;
      if (row < (size_t)cl * 4096) continue;
      e = resident_clusters(kern, lim, dev, cl, n);
      if (e != cudaSuccess) return true;
      if (rows <= n) {
        s.cl = cl;
        resident = n;
        break;
      }
    }
  }
  const int groups = RING_WARPS / s.W;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((RING_WARPS + groups + 1 + (MODE == LM_DISTILL ? groups * teacher_warps(groups) : 0)) * 32);
  cfg.dynamicSmemBytes = groups * s.slots * chunk + fixed;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  cfg.attrs = at;
  if (s.cl > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = s.cl;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
  }
  if (MODE == LM_SCALED) at[cfg.numAttrs++] = follows();
  const long long want = (rows + groups - 1) / groups;
  cfg.gridDim = dim3((unsigned)(std::min<long long>(want, resident) * s.cl));
  e = cudaLaunchKernelEx(&cfg, kern, a, s);
  return true;
}
