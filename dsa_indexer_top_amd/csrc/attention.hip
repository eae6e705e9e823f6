// Attention of query heads over rows of a latent cache (echo_sparse_attention,
// echo_prefix_attention).  One row of 576 values per token serves all heads:
//   s_t = scale * q . row_t,   out = sum_t softmax(s)_t row_t[0 .. 512),   lse = log sum_t exp s_t.
//
// A workgroup takes 32 QT queries that share their tokens (heads of one row, or of the rows behind one
// prefix) and a chunk of those tokens, in tiles of 32.  Four of its eight waves score, four add up, one of each on a SIMD:
//   scores   wave w multiplies 16 of the tile's tokens (w % 2) with 16 QT of the queries (w / 2), whose 576 values
//            stay in registers; the rows come from LDS.
//   softmax  base 2, relative to a maximum per query that all waves know.  It is raised only when a score exceeds
//            it by 2^8: weights up to 2^8 are as exact as those up to 1, and neither the waves' maxima have to be
//            exchanged nor the sums multiplied but then.  The weights go to LDS.
//   sum      wave 4 + w adds up columns 128 w .. 128 w + 127 of all queries over all 32 tokens: the weights from
//            LDS, the rows' columns from LDS through transposing reads.
// Tile t + 1 is scored while tile t is added up, so one barrier a tile is enough, and where one wave of a SIMD computes
// exponentials or waits for LDS the other has products.  Rows go from the cache straight to LDS, two to
// three tiles (74 to 110 KB) ahead, loaded by the adding waves, which have less to do.
//
// Weights are rounded to the cache's type for the product, as the matrix core takes them (off by half a
// step of the type each, which in a sum of many is what the result's own rounding is); scores, sums,
// maxima and the results are fp32.
//
// What bounds it: the matrix core.  With 64 queries a tile's products take 1092 cycles of a SIMD (580 for the scores, 512
// for the sums) of about 1830 that pass; the adding waves' reads, loads and products one after the other are the
// longest chain (1630).  Measured on MI355X: 2048 rows x 128 heads x 2048 tokens 1.20 ms = 975 TFLOP/s (a library
// product of 8192^3 1570), 64 x 16 in two groups behind 32768 107 us, 8 x 128 x 2048 22.8 us, 1 x 16 x 2048 13.3 us.
//
// A chunk's result goes straight to the outputs where it is the only one, otherwise unnormalised to
// the workspace with its maximum and sum, and join_kernel adds the chunks up.
#include <algorithm>

#include "latent.cuh"

namespace echo {

constexpr int WAVES = 8, ADD = 4, TILE = 32, STAGES = 4;   // waves, those that add up; tokens of a tile, tiles in LDS
constexpr int KSTEPS = LATENT / 32, COLS = VALUES / ADD;   // products of a score, columns of a wave
constexpr int OWN = TILE / ADD, LOADS = OWN + 1;           // rows of a tile that an adding wave loads, its loads
constexpr int BATCH = 1536;                                // tokens whose rows are looked up at once
constexpr float SLACK = 8.f;

// A tile in LDS: the rows' first 512 values, 1024 bytes a row and then 64 of weights, every four rows 16 bytes
// more apart; then the rows' last 64 values, 128 bytes a row.  So the reads of 16 rows at one place (scores,
// weights) and of four rows at 64 bytes (sums) touch every bank once, and every read of a lane is one address and
// a constant.  In the last 64 values the pieces of 16 bytes are exchanged within a row instead.
constexpr int ROW_STEP = 1024 + 64, ROPE_AT = TILE * ROW_STEP + TILE / 4 * 16, STAGE = ROPE_AT + TILE * 128;
ECHO_DEV constexpr int row_at(int row) { return row * ROW_STEP + (row >> 2) * 16; }
ECHO_DEV constexpr int swap_r(int row) { return (row >> 1) & 7; }
// Weights of query `at` for tile t (by t % 2): behind row at % 32 of stage 2 (t % 2) + at / 32, 32 tokens.
ECHO_DEV constexpr int weights_at(int t, int at) { return (2 * (t & 1) + (at >> 5)) * STAGE + row_at(at & 31) + 1024; }

struct AttArgs {
  LatentArgs a;
  // where chunks' results go
  void *out;
  int64_t o_row, o_head;
  float *lse;
  float *part, *part_ml;         // [query, parts, 512], [query, parts, 2]
  int32_t chunk, n_chunks, parts, first_part;
  // groups of rows that share a prefix (echo_prefix_attention): the first workgroups
  const int32_t *group_begin, *prefix_len, *prefix_table;
  int32_t n_groups, prefix_pages, max_prefix, prefix_chunk, prefix_chunks;
  uint32_t prefix_blocks;
};

// Queries [q0, q1) (row * n_heads + head) over tokens [t0, t1) of `src`; part < 0: the only chunk.
struct Work {
  int64_t q0, q1;
  Tokens src;
  int32_t t0, t1, part;
};

struct Lds {
  uint8_t stage[STAGES * STAGE];
  float m[64], top[2][64];       // maxima; a tile's, or at the end the sums
  int32_t raise[2];              // t + 1: tile t (by t % 2) has a score far above its maximum
  uint32_t real[STAGES];         // which tokens of a tile there are
  int32_t rows[BATCH];           // cache rows of a batch of tokens, -1: none
};
static_assert(sizeof(Lds) <= 160 * 1024, "a workgroup's LDS");

// Cache rows of the chunk's tokens from `first` on, up to a batch of them, by the adding waves.  Entries and pages are loaded
// for a batch at once: loaded tile by tile, their waits held up the rows on their way (the same counter).
ECHO_DEV void look_up(const Work &w, int32_t first, int32_t *__restrict__ rows) {
  const int32_t t0 = w.t0 + first, count = min(w.t1 - t0, BATCH);
  constexpr int N = ADD * 64, PER = BATCH / N;
  const int tid = threadIdx.x & (N - 1);
  int32_t e[PER], page[PER];
  int64_t pos[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) e[i] = 0;
  if (w.src.list) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * N < count) e[i] = w.src.list[(t0 + min(i * N + tid, count - 1)) >> w.src.shift];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) pos[i] = i * N + tid < count ? w.src.position(t0 + i * N + tid, e[i]) : -1;
  if (w.src.table && w.src.max_pages > 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t p = pos[i] >> w.src.pshift;            // -1: none
      page[i] = w.src.table[p < 0 || p >= w.src.max_pages ? 0 : p];
      if (p >= w.src.max_pages) page[i] = -1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) page[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * N < count) rows[i * N + tid] = w.src.row(pos[i], page[i]);
}

// 8 rows on their way to LDS, 1024 bytes and then the last 128 bytes of each; lane i (and every 8th after it) has the
// address of row i.  For queries.
ECHO_DEV void load_rows(uint64_t at, uint8_t *__restrict__ stage, int r0) {
  const int l = lane_id(), lo = static_cast<int>(at), hi = static_cast<int>(at >> 32);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, i)), b = static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, i));
    const uint8_t *src = reinterpret_cast<const uint8_t *>(static_cast<uint64_t>(b) << 32 | a);
    __builtin_amdgcn_global_load_lds((glb_void *)(src + l * 16), (lds_void *)(stage + row_at(r0) + row_at(i)), 16, 0, 0);
  }
  const uint64_t rope = static_cast<uint64_t>(static_cast<uint32_t>(__shfl(hi, l >> 3, 64))) << 32 | static_cast<uint32_t>(__shfl(lo, l >> 3, 64));
  __builtin_amdgcn_global_load_lds((glb_void *)(reinterpret_cast<const uint8_t *>(rope) + 1024 + (((l & 7) ^ swap_r(r0 + (l >> 3))) << 4)),
                                   (lds_void *)(stage + ROPE_AT + r0 * 128), 16, 0, 0);
}

// An adding wave's 8 rows of a tile on their way to LDS, a part at a time; the tile's cache rows are at `rows`.  Through a
// buffer descriptor: one lane's offset and the place in LDS are all that a row takes, and unlike a global
// load it does not make the compiler wait for every LDS read under way.  A cache of 4 GB and more (WIDE) adds
// the upper half of an offset to the descriptor's base.  Where there is no row it is the cache's first; zero() takes it out.
template <bool WIDE>
struct Fetch {
  int32_t row, rope_row;
  int lo, hi, r0;
  uint64_t rope;
  const void *kv;
  ECHO_DEV void look(const int32_t *__restrict__ rows, int wa) {
    r0 = wa * OWN;
    row = rows[lane_id() & 31];
    rope_row = rows[r0 + (lane_id() >> 3)];
  }
  // Returns which of the tile's 32 tokens there are.
  ECHO_DEV uint32_t prepare(const AttArgs &x) {
    const int l = lane_id();
    const uint32_t stride = static_cast<uint32_t>(x.a.kv_stride * 2);
    kv = x.a.kv;
    const uint64_t at = static_cast<uint64_t>(static_cast<uint32_t>(max(row, 0))) * stride;
    lo = static_cast<int>(at);
    hi = static_cast<int>(at >> 32);
    rope = static_cast<uint64_t>(static_cast<uint32_t>(max(rope_row, 0))) * stride + 1024 + (((l & 7) ^ swap_r(r0 + (l >> 3))) << 4);
    return static_cast<uint32_t>(__ballot(row >= 0));
  }
  ECHO_DEV void load(uint8_t *__restrict__ stage, int i) const {
    if (i < OWN) {                                         // r0 is a multiple of 4
      const uint32_t at = static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, r0 + i));
      // A descriptor's offsets are added up in 32 bits, so rows of a wide cache get a descriptor each.
      const uint64_t from = WIDE ? static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, r0 + i))) << 32 | at : 0;
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(reinterpret_cast<uint64_t>(kv) + from), 0, -1, 0x00027000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void *)(stage + row_at(r0) + row_at(i)), 16, lane_id() * 16, WIDE ? 0 : at, 0, 0);
    } else if (WIDE) {                                     // eight rows in one load: addresses by lane
      __builtin_amdgcn_global_load_lds((glb_void *)(static_cast<const uint8_t *>(kv) + rope), (lds_void *)(stage + ROPE_AT + r0 * 128), 16, 0, 0);
    } else {
      const auto buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(kv), 0, -1, 0x00027000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_void *)(stage + ROPE_AT + r0 * 128), 16, static_cast<uint32_t>(rope), 0, 0, 0);
    }
  }
};
// Rows that this wave has loaded and that are no token's, once they are there: zeros, so that nothing of the cache gets
// into a sum through a weight of 0.
ECHO_DEV void zero(uint8_t *__restrict__ stage, uint32_t real, int wa) {
  if (real == ~0u) return;                                 // the same for the whole wave
  const int l = lane_id(), r0 = wa * OWN;
#pragma unroll
  for (int i = 0; i < OWN; ++i)
    if (!(real >> (r0 + i) & 1)) *reinterpret_cast<u32x4 *>(stage + row_at(r0) + row_at(i) + 16 * l) = u32x4{0, 0, 0, 0};
  if (!(real >> (r0 + (l >> 3)) & 1)) *reinterpret_cast<u32x4 *>(stage + ROPE_AT + r0 * 128 + 16 * l) = u32x4{0, 0, 0, 0};
}

// An empty statement that takes and gives accumulation registers: between two of them the compiler copies one
// group of sums to where it can be multiplied, and holds them all where the matrix core adds them up otherwise.
// It also keeps its place among the reads of LDS, so that an operand is read as far ahead of its product as is written
// here; left to itself the compiler reads it right before, and the matrix core waits for LDS.
ECHO_DEV void pin(v16f &v) { asm volatile("" : "+a"(v)); }
ECHO_DEV void pin(v4f &v) { asm volatile("" : "+a"(v)); }
template <typename X8> ECHO_DEV void pin_operand(X8 &v) { asm volatile("" : "+a"(v)); }

template <typename T, int QT>
struct Scorer {
  typedef typename Mma<T>::x8 x8;
  x8 q[QT][KSTEPS];              // 16 QT queries: lane (j, g) values of query qb + 16 i + j
  v4f acc[QT], s[QT];            // products; those of the tile whose weights were given last: tokens 4 g .. 4 g + 3 of the wave's 16
  float m[QT], far[QT], sum[QT], tile_sum[QT];             // maxima (base 2), the product from which on they are raised; sums of weights
  float scale2;
  int qb, th;

  struct Rows {                  // product k of the wave's 16 rows
    const uint8_t *v, *r;
    int g, swap;
    ECHO_DEV x8 read(int k) const { return k < 16 ? read16<x8>(v + 16 * k) : read16<x8>(r + (((4 * (k - 16) + g) ^ swap) << 4)); }
  };
  ECHO_DEV static Rows rows_of(const uint8_t *__restrict__ stage, int half) {
    const int l = lane_id(), j = l & 15, g = l >> 4;
    return Rows{stage + row_at(half * 16 + j) + 256 * g, stage + ROPE_AT + (half * 16 + j) * 128, g, swap_r(j)};
  }
  ECHO_DEV void set(int i, float to) {
    m[i] = to;
    far[i] = (to + SLACK) / scale2;
  }
  ECHO_DEV void init(const Lds &lds, int q_stage, int wv, float scale) {
    qb = (wv >> 1) * 16 * QT;
    th = wv & 1;
    // A negative scale goes into the queries' signs, no scale makes them 0: a masked product then stays at -infinity.
    const uint32_t flip = scale < 0.f ? 0x80008000u : 0u, keep = scale == 0.f ? 0u : ~0u;
    scale2 = scale == 0.f ? 1.f : fabsf(scale);
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int at = qb + 16 * i;
      const Rows r = rows_of(lds.stage + (q_stage + (at >> 5)) * STAGE, (at >> 4) & 1);
#pragma unroll
      for (int k = 0; k < KSTEPS; ++k) {
        q[i][k] = __builtin_bit_cast(x8, (__builtin_bit_cast(u32x4, r.read(k)) & keep) ^ flip);
        pin_operand(q[i][k]);                              // in accumulation registers, from where products take them as well
      }
      set(i, NO_SCORE);
      sum[i] = tile_sum[i] = 0.f;
    }
  }
  ECHO_DEV void products(const uint8_t *__restrict__ stage) {
    constexpr int AHEAD = 6;
    const Rows r = rows_of(stage, th);
    x8 row[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) row[k] = r.read(k);
#pragma unroll
    for (int i = 0; i < QT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KSTEPS; ++k) {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        pin(acc[i]);
        acc[i] = Mma<T>::mul(row[k % AHEAD], q[i][k], acc[i]);
      }
      pin(acc[0]);
      if (k + AHEAD < KSTEPS) row[k % AHEAD] = r.read(k + AHEAD);
    }
  }
  // Weights of tile t from its products; `real`: its tokens.
  ECHO_DEV void weigh(Lds &lds, int t) {
    const int l = lane_id(), j = l & 15, g = l >> 4;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      v4f w;
#pragma unroll
      for (int v = 0; v < 4; ++v) w[v] = exp2_(fmaf(s[i][v], scale2, -m[i]));
      tile_sum[i] = (w[0] + w[1]) + (w[2] + w[3]);
      *reinterpret_cast<u32x2 *>(lds.stage + weights_at(t, qb + 16 * i + j) + 32 * th + 8 * g) = pack4<T>(w);
    }
  }
  ECHO_DEV float top(int i) const { return fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3])); }
  ECHO_DEV void weights(Lds &lds, int t, uint32_t real) {
#pragma unroll
    for (int i = 0; i < QT; ++i) s[i] = acc[i];
    if (real != ~0u) {                                     // the same for the whole wave
      const uint32_t mine = real >> (16 * th + 4 * (lane_id() >> 4));
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int i = 0; i < QT; ++i) s[i][v] = mine >> v & 1 ? s[i][v] : -INFINITY;
    }
    weigh(lds, t);
    bool above = false;
#pragma unroll
    for (int i = 0; i < QT; ++i) above |= top(i) > far[i];
    if (__ballot(above) && lane_id() == 0) atomicMax(&lds.raise[t & 1], t + 1);     // by any of the waves
  }
  // Maxima up to those of tile t, whose weights are given anew; with Adder::raise.
  ECHO_DEV void raise(Lds &lds, int t) {
    const int l = lane_id(), j = l & 15, g = l >> 4;
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      float a = top(i) * scale2;
      a = fmaxf(a, __shfl_xor(a, 16, 64));
      a = fmaxf(a, __shfl_xor(a, 32, 64));
      if (g == 0) lds.top[th][qb + 16 * i + j] = a;
    }
    meet();
    float to[QT];
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int at = qb + 16 * i + j;
      to[i] = fmaxf(m[i], fmaxf(lds.top[0][at], lds.top[1][at]));
      sum[i] *= exp2_(m[i] - to[i]);
      set(i, to[i]);
    }
    meet();
    if (th == 0 && g == 0)
#pragma unroll
      for (int i = 0; i < QT; ++i) lds.m[qb + 16 * i + j] = to[i];
    weigh(lds, t);
    meet();
  }
  ECHO_DEV void count() {
#pragma unroll
    for (int i = 0; i < QT; ++i) sum[i] += tile_sum[i];
  }
};

template <typename T, int QT>
struct Adder {
  typedef typename Mma<T>::x8 x8;
  v16f o[QT][COLS / 32];         // lane (j, h): columns 32 c + 8 (v / 4) + 4 h + v % 4 of query 32 i + j
  int wa;

  // The operands: weights of query 32 i + j and columns 32 c .. of the wave's, tokens 16 k + 8 h .. + 7.
  const uint8_t *p, *v;
  ECHO_DEV x8 weights(int i, int k) const { return read16<x8>(p + i * STAGE + 32 * k); }
  ECHO_DEV x8 cols(int c, int k) const {
    struct { v4s lo, hi; } e;
    e.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(v + row_at(16 * k) + 64 * c));
    e.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(v + row_at(16 * k + 4) + 64 * c));
    return __builtin_bit_cast(x8, e);
  }
  ECHO_DEV void raise(const Lds &lds) {
    const int l = lane_id();
    meet();
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int at = 32 * i + (l & 31);
      const float was = lds.m[at], less = exp2_(was - fmaxf(was, fmaxf(lds.top[0][at], lds.top[1][at])));
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) {
        pin(o[i][c]);
#pragma unroll
        for (int u = 0; u < 16; ++u) o[i][c][u] *= less;
        pin(o[i][c]);
      }
    }
    meet();
    meet();
  }
  // Adds up the tile in `cur`.  With a fetch the loads of a later tile, to `next`, stand between the products.  (Three
  // pointers that the compiler may take for different memory: it waits for loads to LDS before reads of the same.)
  template <bool FETCH, typename F>
  ECHO_DEV void add(const uint8_t *__restrict__ cur, const uint8_t *__restrict__ weights_of_tile, uint8_t *__restrict__ next, const Lds &lds, int t, const F &f) {
    constexpr int STEPS = COLS / 16, AHEAD = 4;
    const int l = lane_id(), h = l >> 5;
    p = weights_of_tile + 16 * h;
    v = cur + row_at(8 * h) + ((l & 15) >> 2) * ROW_STEP + wa * (2 * COLS) + 32 * ((l >> 4) & 1) + 8 * (l & 3);
    const int32_t far = lds.raise[t & 1];
    x8 col[AHEAD], w[QT][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) col[u] = cols(u >> 1, u & 1);
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) w[i][k] = weights(i, k);
    if (__builtin_amdgcn_readfirstlane(far) == t + 1) {
      raise(lds);
#pragma unroll
      for (int i = 0; i < QT; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) w[i][k] = weights(i, k);
    }
    if (FETCH) f.load(next, 0);
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        pin(o[i][u >> 1]);
        o[i][u >> 1] = Mma<T>::mul(col[u % AHEAD], w[i][u & 1], o[i][u >> 1]);
      }
      pin(o[0][u >> 1]);
      if (u + AHEAD < STEPS) col[u % AHEAD] = cols((u + AHEAD) >> 1, (u + AHEAD) & 1);
      if (FETCH) f.load(next, 1 + u);
    }
  }
};
static_assert(COLS / 16 == LOADS - 1, "a load for each product of the sum, one before");

template <typename T, int QT, bool WIDE>
ECHO_DEV void attend(const AttArgs &x, const Work &w, Lds &lds) {
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l = lane_id();
  // The queries' rows go to registers by way of LDS, to the stages that the first two tiles of tokens do not
  // need: read by the waves themselves they were four pieces of a row a load, a line each.
  constexpr int Q_STAGE = STAGES - QT;
  if (wv < 4 * QT) {
    const int64_t qi = min(w.q0 + 8 * wv + (l & 7), w.q1 - 1), r = qi / x.a.n_heads;
    load_rows(reinterpret_cast<uint64_t>(x.a.q + r * x.a.q_row + (qi - r * x.a.n_heads) * x.a.q_head), lds.stage + (Q_STAGE + (wv >> 2)) * STAGE, 8 * (wv & 3));
  }
  if (threadIdx.x < 64) lds.m[threadIdx.x] = NO_SCORE;
  if (threadIdx.x < 2) lds.raise[threadIdx.x] = 0;
  const int n = (w.t1 - w.t0 + TILE - 1) / TILE;
  constexpr int TILES = BATCH / TILE;
  const bool adding = wv >= ADD;
  if (adding && n > 0) look_up(w, 0, lds.rows);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt(0));
  meet();
  // Both sides go through the same barriers: [queries taken] [tile 0] and, for every tile t, [tile t + 1 and the weights of
  // tile t are there, and tile t - 1 is done with], where a score is far above its maximum three more, and one more where a
  // batch of rows is looked up.
  v16f o[QT][COLS / 32];
  if (!adding) {
    Scorer<T, QT> a;
    a.init(lds, Q_STAGE, wv, x.a.scale2);
    meet();
    if (n > 0) {
      meet();
      a.products(lds.stage);
      a.weights(lds, 0, lds.real[0]);
      for (int t = 0; t < n; ++t) {
        meet();
        if (t + 3 < n && (t + 3) % TILES == 0) meet();
        const int32_t far = lds.raise[t & 1];
        const uint32_t have = lds.real[(t + 1) % STAGES];
        if (t + 1 < n) a.products(lds.stage + (t + 1) % STAGES * STAGE);
        if (__builtin_amdgcn_readfirstlane(far) == t + 1) a.raise(lds, t);
        a.count();
        if (t + 1 < n) a.weights(lds, t + 1, static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(have))));
      }
    }
    meet();
    // The sums of a query: four lane groups, two waves.
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      float s = a.sum[i];
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if (l < 16) lds.top[a.th][a.qb + 16 * i + l] = s;
    }
  } else {
    Adder<T, QT> a;
    a.wa = wv - ADD;
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) a.o[i][c] = v16f{};
    uint32_t real[3] = {};                                 // of tiles t + 1, t + 2, t + 3
    Fetch<WIDE> f;
    const auto tell = [&](int t, uint32_t have) { if (a.wa == 0) lds.real[t % STAGES] = have; };
    const auto first = [&](int t) {
      if (t >= n) return;
      f.look(lds.rows + t * TILE, a.wa);
      real[t] = f.prepare(x);
      tell(t, real[t]);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) f.load(lds.stage + t * STAGE, i);
    };
    first(0);
    first(1);
    meet();
    first(2);
    // The tiles but the `later` youngest of this wave's loads are in LDS, of tile t rows that are no token's made zeros.
    const auto arrived = [&](int later, int t, uint32_t have) {
      asm volatile("" ::: "memory");
      if (later > 1) __builtin_amdgcn_s_waitcnt(vmcnt(2 * LOADS));
      else if (later == 1) __builtin_amdgcn_s_waitcnt(vmcnt(LOADS));
      else __builtin_amdgcn_s_waitcnt(vmcnt(0));
      asm volatile("" ::: "memory");
      zero(lds.stage + t % STAGES * STAGE, have, a.wa);
      meet();
    };
    if (n > 0) {
      arrived(min(n - 1, 2), 0, real[0]);
      int t = 0;
      for (; t + 3 < n; ++t) {
        arrived(1, t + 1, real[1]);
        const int in = (t + 3) % TILES;
        if (in == 0) {                                     // every wave has taken the last batch's rows
          look_up(w, (t + 3) * TILE, lds.rows);
          meet();
        }
        f.look(lds.rows + in * TILE, a.wa);
        real[1] = real[2];
        real[2] = f.prepare(x);
        tell(t + 3, real[2]);
        a.template add<true>(lds.stage + t % STAGES * STAGE, lds.stage + weights_at(t, l & 31), lds.stage + (t + 3) % STAGES * STAGE, lds, t, f);
      }
      for (; t < n; ++t) {
        arrived(t + 2 < n ? 1 : 0, t + 1, t + 1 < n ? real[1] : ~0u);
        real[1] = real[2];
        a.template add<false>(lds.stage + t % STAGES * STAGE, lds.stage + weights_at(t, l & 31), nullptr, lds, t, f);
      }
    }
    meet();
#pragma unroll
    for (int i = 0; i < QT; ++i)
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) o[i][c] = a.o[i][c];
  }
  meet();
  // Results by way of LDS, a query's row after the other, so that a store writes whole lines.
  const bool whole = w.part < 0;
  const int h = l >> 5;
  constexpr int OUT_ROW = VALUES * static_cast<int>(sizeof(T)) + 16, PART_ROW = VALUES * 4 + 16;
  static_assert(64 * PART_ROW <= STAGES * STAGE, "results fit the stages");
  if (adding) {
#pragma unroll
    for (int i = 0; i < QT; ++i) {
      const int at = 32 * i + (l & 31);
      const float sum = lds.top[0][at] + lds.top[1][at];
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int c = 0; c < COLS / 32; ++c) {
        pin(o[i][c]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const v4f v = {o[i][c][4 * b], o[i][c][4 * b + 1], o[i][c][4 * b + 2], o[i][c][4 * b + 3]};
          const int col = (wv - ADD) * COLS + 32 * c + 8 * b + 4 * h;
          if (whole) *reinterpret_cast<u32x2 *>(lds.stage + at * OUT_ROW + col * sizeof(T)) = pack4<T>(v * inv);
          else *reinterpret_cast<v4f *>(lds.stage + at * PART_ROW + col * 4) = v;
        }
      }
    }
  }
  meet();
  constexpr int PER = 32 * QT / WAVES;                     // queries that a wave stores
  const int64_t mine = min(w.q0 + wv * PER + (l % PER), w.q1 - 1), r = mine / x.a.n_heads;
  const uint64_t to = whole ? reinterpret_cast<uint64_t>(static_cast<T *>(x.out) + r * x.o_row + (mine - r * x.a.n_heads) * x.o_head)
                            : reinterpret_cast<uint64_t>(x.part + (mine * x.parts + w.part) * VALUES);
  const int lo = static_cast<int>(to), hi = static_cast<int>(to >> 32);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int at = wv * PER + i;
    const uint32_t u = static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, i)), v = static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, i));
    uint8_t *p = reinterpret_cast<uint8_t *>(static_cast<uint64_t>(v) << 32 | u) + 16 * l;
    if (w.q0 + at >= w.q1) break;
    if (whole) {                                           // past the caches, which hold the rows (202 x 128 heads x 73 tokens 36.0 -> 34.6 us)
      __builtin_nontemporal_store(*reinterpret_cast<const u32x4 *>(lds.stage + at * OUT_ROW + 16 * l), reinterpret_cast<u32x4 *>(p));
    } else {
      *reinterpret_cast<u32x4 *>(p) = *reinterpret_cast<const u32x4 *>(lds.stage + at * PART_ROW + 16 * l);
      *reinterpret_cast<u32x4 *>(p + 1024) = *reinterpret_cast<const u32x4 *>(lds.stage + at * PART_ROW + 1024 + 16 * l);
    }
  }
  const int at = threadIdx.x;
  if (at < 32 * QT && w.q0 + at < w.q1) {
    const float sum = lds.top[0][at] + lds.top[1][at], m = lds.m[at];
    if (!whole) {
      const int64_t p = (w.q0 + at) * x.parts + w.part;
      x.part_ml[2 * p] = m;
      x.part_ml[2 * p + 1] = sum;
    } else if (x.lse) {
      x.lse[w.q0 + at] = sum == 0.f ? -INFINITY : (m + log2_(sum)) * LN2;
    }
  }
}

ECHO_DEV int32_t clamp_row(int32_t r, int32_t n) { return r < 0 ? 0 : r > n ? n : r; }

// The tokens that a query row lists (or, without a list, its own).  Workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: the head tiles of a chunk follow each other by 8, so that they share the one that the
// chunk's rows are in.
template <int QT>
ECHO_DEV bool rows_work(const AttArgs &x, Work &w) {
  const uint32_t head_tiles = (x.a.n_heads + 32 * QT - 1) / (32 * QT), units = static_cast<uint32_t>(x.a.n_rows) * static_cast<uint32_t>(x.n_chunks);
  const uint32_t id = blockIdx.x - x.prefix_blocks, eight = id / (8 * head_tiles), in = id - eight * 8 * head_tiles;
  const uint32_t u = eight * 8 + (in & 7), ht = in >> 3;
  if (u >= units) return false;
  const int32_t r = static_cast<int32_t>(u / x.n_chunks), c = static_cast<int32_t>(u - static_cast<uint32_t>(r) * x.n_chunks);
  w.src = x.a.tokens(r);
  w.t0 = c * x.chunk;
  w.t1 = min(w.t0 + x.chunk, x.a.n_tok);
  if (!x.a.idx) {
    w.src.list = nullptr;
    w.t1 = static_cast<int32_t>(min<int64_t>(w.t1, max<int64_t>(w.src.limit, 0)));
    if (w.t0 >= w.t1 && x.parts > 0) return false;         // join_kernel goes by the length too
  }
  if (x.a.n_kv < 1) w.t1 = w.t0;                           // no rows: no tokens
  w.q0 = static_cast<int64_t>(r) * x.a.n_heads + ht * (32 * QT);
  w.q1 = static_cast<int64_t>(r + 1) * x.a.n_heads;
  w.part = x.parts > 0 ? x.first_part + c : -1;
  return true;
}

// The prefixes: a tile of the groups' queries in order, a chunk.  With eight chunks and more a chunk's workgroups are
// a multiple of 8 apart, on one XCD, so that its L2 has the chunk's rows for all of them.
__host__ __device__ constexpr int32_t chunk_step(int32_t chunks) { return chunks < 8 ? chunks : (chunks + 7) & ~7; }
template <int QT>
ECHO_DEV bool prefix_work(const AttArgs &x, Work &w) {
  const int32_t step = chunk_step(x.prefix_chunks), c = blockIdx.x % step;
  if (c >= x.prefix_chunks) return false;
  uint32_t tile = blockIdx.x / step;
  int32_t gi = -1, r0 = 0, r1 = 0;
  for (int32_t g0 = 0; g0 < x.n_groups; g0 += 64) {        // 64 groups at a time
    const int32_t g = min(g0 + lane_id(), x.n_groups - 1);
    const int32_t a = clamp_row(x.group_begin[g], x.a.n_rows), b = max(a, clamp_row(x.group_begin[g + 1], x.a.n_rows));
    const uint32_t has = g0 + lane_id() < x.n_groups ? static_cast<uint32_t>((static_cast<int64_t>(b - a) * x.a.n_heads + 32 * QT - 1) / (32 * QT)) : 0u;
    const uint32_t upto = wave_incl_scan(has);
    const uint64_t in = __ballot(tile < upto);
    if (in) {
      const int at = __ffsll(static_cast<unsigned long long>(in)) - 1;
      gi = g0 + at;
      r0 = __builtin_amdgcn_readlane(a, at);
      r1 = __builtin_amdgcn_readlane(b, at);
      tile -= static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto - has), at));
      break;
    }
    tile -= static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(upto), 63));
  }
  if (gi < 0) return false;
  w.src = Tokens{nullptr, x.prefix_table + static_cast<int64_t>(gi) * x.prefix_pages, x.prefix_len[gi], 0, x.a.pshift, x.prefix_pages, x.a.n_kv};
  w.t0 = c * x.prefix_chunk;
  w.t1 = static_cast<int32_t>(min<int64_t>(min<int64_t>(w.t0 + x.prefix_chunk, x.max_prefix), w.src.limit));
  if (w.t0 >= w.t1) return false;
  if (x.a.n_kv < 1) w.t1 = w.t0;                           // no rows: no tokens
  w.q0 = static_cast<int64_t>(r0) * x.a.n_heads + static_cast<int64_t>(tile) * (32 * QT);
  w.q1 = static_cast<int64_t>(r1) * x.a.n_heads;
  w.part = c;
  return true;
}

// QP: of a prefix's workgroups, QR of the rows'.
template <typename T, int QP, int QR, bool WIDE>
__global__ __launch_bounds__(WAVES * 64) void attention_kernel(AttArgs x) {
  __shared__ __attribute__((aligned(16))) Lds lds;
  Work w;
  if (QP == QR) {
    const bool any = blockIdx.x < x.prefix_blocks ? prefix_work<QP>(x, w) : rows_work<QR>(x, w);
    if (any) attend<T, QR, WIDE>(x, w, lds);
  } else if (blockIdx.x < x.prefix_blocks) {
    if (prefix_work<QP>(x, w)) attend<T, QP, WIDE>(x, w, lds);
  } else {
    if (rows_work<QR>(x, w)) attend<T, QR, WIDE>(x, w, lds);
  }
}

// ---------------------------------------------------------------- joining chunks
struct JoinArgs {
  const float *part, *ml;
  void *out;
  int64_t o_row, o_head;
  float *lse;
  int32_t n_rows, n_heads, parts;
  // numbers of parts: all, or by length
  const int32_t *len, *group_begin, *prefix_len;
  int32_t n_groups, prefix_chunk, max_prefix, prefix_parts, own_chunk, max_own;
};

// Group of row r: the first g with group_begin[g] <= r < group_begin[g + 1], 64 groups at a time; -1: none.
ECHO_DEV int32_t group_of(const int32_t *__restrict__ begin, int32_t n_groups, int32_t r) {
  for (int32_t g0 = 0; g0 < n_groups; g0 += 64) {
    const int32_t g = min(g0 + lane_id(), n_groups - 1);
    const uint64_t in = __ballot(begin[g] <= r && r < begin[g + 1]);
    if (in) return min(g0 + __ffsll(static_cast<unsigned long long>(in)) - 1, n_groups - 1);
  }
  return -1;
}

// out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p, M the largest m_p.  W waves take a query's parts in turn, 8
// columns a lane: as many as a workgroup has where there are few queries.  Eight parts are on their way at
// once, the first ones while the parts' maxima are.
template <typename T, int W>
__global__ __launch_bounds__(256) void join_kernel(JoinArgs x) {
  __shared__ float lds[W > 1 ? W : 1][W > 1 ? VALUES + 4 : 1];
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)), l = lane_id();
  const int64_t qi = W > 1 ? static_cast<int64_t>(blockIdx.x) : blockIdx.x * 4ll + wv;
  if (qi >= static_cast<int64_t>(x.n_rows) * x.n_heads) return;
  const int32_t r = static_cast<int32_t>(qi / x.n_heads);
  int32_t n0 = x.parts, skip = 0, n1 = 0;                  // parts [0, n0) and [skip, skip + n1)
  if (x.own_chunk) {
    const int32_t gi = group_of(x.group_begin, x.n_groups, r);
    n0 = gi < 0 ? 0 : (max(0, min(x.prefix_len[gi], x.max_prefix)) + x.prefix_chunk - 1) / x.prefix_chunk;
    skip = x.prefix_parts;
    n1 = (max(0, min(x.len[r], x.max_own)) + x.own_chunk - 1) / x.own_chunk;
  }
  const int64_t p0 = qi * x.parts;
  const int32_t first = W > 1 ? wv : 0, n = (n0 + n1 - first + W - 1) / W;       // this wave's parts: first, first + W, ..
  const auto part = [&](int32_t i) { const int32_t at = first + i * W; return p0 + (at < n0 ? at : skip + at - n0); };
  float m = NO_SCORE, sum = 0.f, o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int32_t i0 = 0; i0 < n; i0 += 64) {
    const int32_t some = min(n - i0, 64);
    const int64_t mine = part(i0 + min(l, some - 1));
    const float pm = x.ml[2 * mine], ps = x.ml[2 * mine + 1];
    v4f v[8][2];
    const auto load = [&](int32_t i) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float *at = x.part + part(i0 + min(i + u, some - 1)) * VALUES + 8 * l;
        v[u][0] = *reinterpret_cast<const v4f *>(at);
        v[u][1] = *reinterpret_cast<const v4f *>(at + 4);
      }
    };
    load(0);
    float top = fmaxf(m, pm);
#pragma unroll
    for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d, 64));
    const float was = exp2_(m - top), scale = l < some ? exp2_(pm - top) : 0.f;
    float add = scale == 0.f ? 0.f : ps * scale;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) add += __shfl_xor(add, d, 64);
    sum = sum * was + add;
    m = top;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] *= was;
    for (int32_t i = 0; i < some; i += 8) {
      if (i) load(i);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (i + u >= some) break;                          // the same for the whole wave
        const float f = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale), i + u));
#pragma unroll
        for (int c = 0; c < 8; ++c) o[c] = fmaf(v[u][c >> 2][c & 3], f, o[c]);
      }
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int c = 0; c < 8; c += 4) *reinterpret_cast<v4f *>(&lds[wv][8 * l + c]) = v4f{o[c], o[c + 1], o[c + 2], o[c + 3]};
    if (l == 0) {
      lds[wv][VALUES] = m;
      lds[wv][VALUES + 1] = sum;
    }
    __syncthreads();
    if (wv) return;
    float top = m;
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, lds[w][VALUES]);
    const float mine = exp2_(m - top);
    sum *= mine;
    m = top;
#pragma unroll
    for (int c = 0; c < 8; ++c) o[c] *= mine;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float f = exp2_(lds[w][VALUES] - top);
      sum = fmaf(lds[w][VALUES + 1], f, sum);
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = fmaf(lds[w][8 * l + c], f, o[c]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int v = 0; v < 8; ++v) o[v] *= inv;
  T *out = static_cast<T *>(x.out) + r * x.o_row + (qi - static_cast<int64_t>(r) * x.n_heads) * x.o_head + 8 * l;
  store8(out, o);
  if (x.lse && l == 0) x.lse[qi] = sum == 0.f ? -INFINITY : (m + log2_(sum)) * LN2;
}

// ---------------------------------------------------------------- host
// Groups of 32 queries in a workgroup (QT), chunks of the tokens and their size.  Measured on MI355X over lists of
// 2048 tokens (us; one group and two, chunks for 256 workgroups):
//   128 heads of 1 row 15.3 and 18.5, 8 rows 22.8 and 26.0, 32 rows 43.2 and 40.6, 64 rows 62.8 and 61.8, 128 rows 122 and 92
// so with one group the CUs have less to write and to join as long as each of them gets one workgroup, and beyond that
// two groups have half the rows to load; so they have where a workgroup has many tiles to go through (prefixes, 64
// tiles with two groups: 16 heads of 64 requests behind 32768 tokens 127 and 112; 32 tiles, 32 requests: 62 and 66).  More chunks than CUs, or less than two tiles in one, cost more than
// they give (8 rows: 16 chunks instead of 8 30.7; 1 row: 64 instead of 32 18.3).
constexpr int CUS = 256;
struct Plan { int qt; int64_t tiles; int32_t chunk, n_chunks; };
Plan plan_of(int64_t rows, int64_t queries, int64_t n_tok) {           // `rows` times `queries` that share n_tok tokens
  Plan p;
  const int64_t one = rows * ((queries + 31) / 32), two = rows * ((queries + 63) / 64);
  const int64_t n = (n_tok + TILE - 1) / TILE;
  p.qt = queries <= 32 || (one <= CUS && n * two <= 32 * CUS) ? 1 : 2;
  p.tiles = p.qt == 1 ? one : two;
  const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((n + 1) / 2, CUS / std::max<int64_t>(p.tiles, 1)));
  p.chunk = std::max<int32_t>(1, static_cast<int32_t>((n + chunks - 1) / chunks)) * TILE;
  p.n_chunks = std::max<int32_t>(1, static_cast<int32_t>((n_tok + p.chunk - 1) / p.chunk));
  return p;
}
constexpr int64_t PART_BYTES = (VALUES + 2) * 4;
constexpr int64_t MAX_GROUPS = 1 << 23;                    // workgroups of 512 threads in a launch
constexpr int32_t MAX_HEADS = 1024, MAX_TOKENS = 1 << 28;

int64_t sparse_ws(int32_t n_rows, int32_t n_heads, int64_t n_tok) {
  const int32_t c = plan_of(n_rows, n_heads, n_tok).n_chunks;
  return c > 1 ? static_cast<int64_t>(n_rows) * n_heads * c * PART_BYTES : 0;
}

struct PrefixPlan { Plan own, prefix; int64_t tiles; int32_t prefix_parts, own_parts; };
PrefixPlan prefix_plan(int32_t n_rows, int32_t n_heads, int32_t n_groups, int32_t max_prefix, int32_t max_own) {
  PrefixPlan p;
  p.own = plan_of(n_rows, n_heads, max_own);
  p.own_parts = max_own > 0 ? p.own.n_chunks : 0;
  const int64_t queries = static_cast<int64_t>(n_rows) * n_heads, groups = std::min(n_groups, n_rows);
  p.prefix = plan_of(std::max<int64_t>(groups, 1), groups ? (queries + groups - 1) / groups : queries, max_prefix);
  if (p.own.qt == 2) p.prefix.qt = 2;                      // kernels are built for 1 and 1, 2 and 1, 2 and 2
  p.tiles = groups ? queries / (32 * p.prefix.qt) + groups : 0;        // at least what the groups' last, partly filled tiles take
  p.prefix_parts = groups && max_prefix > 0 ? p.prefix.n_chunks : 0;
  return p;
}

template <typename T, bool WIDE>
int launch_attention(const AttArgs &x, int qp, int qr, uint32_t grid, hipStream_t st) {
  if (qr == 2) attention_kernel<T, 2, 2, WIDE><<<grid, WAVES * 64, 0, st>>>(x);
  else if (qp == 2) attention_kernel<T, 2, 1, WIDE><<<grid, WAVES * 64, 0, st>>>(x);
  else attention_kernel<T, 1, 1, WIDE><<<grid, WAVES * 64, 0, st>>>(x);
  return check_launch("attention");
}
int launch_attention(const AttArgs &x, int type, int qp, int qr, int64_t row_blocks, hipStream_t st) {
  const bool wide = static_cast<int64_t>(x.a.n_kv) * x.a.kv_stride * 2 >= (1ll << 32) - 4096;
  const uint32_t grid = x.prefix_blocks + static_cast<uint32_t>(row_blocks);
  if (type == ECHO_BF16) return wide ? launch_attention<bf16_t, true>(x, qp, qr, grid, st) : launch_attention<bf16_t, false>(x, qp, qr, grid, st);
  return wide ? launch_attention<fp16_t, true>(x, qp, qr, grid, st) : launch_attention<fp16_t, false>(x, qp, qr, grid, st);
}
// Workgroups of the rows: rows_work's numbering goes by eights of (row, chunk).
int64_t row_blocks(int32_t n_rows, int32_t n_heads, const Plan &p) {
  return (static_cast<int64_t>(n_rows) * p.n_chunks + 7) / 8 * 8 * ((n_heads + 32 * p.qt - 1) / (32 * p.qt));
}
template <typename T>
int launch_join(const JoinArgs &j, hipStream_t st) {
  const int64_t q = static_cast<int64_t>(j.n_rows) * j.n_heads;
  if (q <= 1024 && j.parts > 8) join_kernel<T, 4><<<static_cast<uint32_t>(q), 256, 0, st>>>(j);
  else join_kernel<T, 1><<<static_cast<uint32_t>((q + 3) / 4), 256, 0, st>>>(j);
  return check_launch("attention join");
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Queries and cache of either call.
int check_cache(const char *fn, int32_t n_rows, int32_t n_heads, int32_t type, float scale, const void *q, int64_t q_row,
                int64_t q_head, const void *kv, int64_t kv_stride, int32_t n_kv) {
  if (n_rows < 0 || n_heads < 0 || n_kv < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (type != ECHO_BF16 && type != ECHO_FP16) return fail(ECHO_EINVAL, "%s: type %d", fn, type);
  if (!(scale >= -1.0e38f && scale <= 1.0e38f)) return fail(ECHO_EINVAL, "%s: scale outside [-1e38, 1e38]", fn);
  if (n_heads > MAX_HEADS || n_rows > 1 << 22) return fail(ECHO_EUNSUPPORTED, "%s: more than %d heads or 2^22 rows", fn, MAX_HEADS);
  if (n_rows == 0 || n_heads == 0) return ECHO_OK;
  if (!q || (n_kv && !kv)) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if (q_row < 0 || q_head < 0 || kv_stride < 0 || (n_kv > 1 && kv_stride < LATENT)) return fail(ECHO_EINVAL, "%s: a stride below 0 or below the row", fn);
  if (kv_stride > 1 << 30) return fail(ECHO_EUNSUPPORTED, "%s: rows of kv more than 2^30 elements apart", fn);
  if (!aligned(q, 16) || !aligned(kv, 16) || q_row % 8 || q_head % 8 || (n_kv > 1 && kv_stride % 8))
    return fail(ECHO_EUNSUPPORTED, "%s: q, kv or their strides are not multiples of 16 bytes", fn);
  return ECHO_OK;
}
int check_out(const char *fn, int32_t n_rows, int32_t n_heads, const void *out, int64_t o_row, int64_t o_head, const float *lse) {
  if (!out) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if (o_row < 0 || o_head < 0 || rows_overlap(n_rows, o_row, n_heads, o_head, VALUES)) return fail(ECHO_EINVAL, "%s: heads of out overlap", fn);
  if (!aligned(out, 16) || (n_rows > 1 && o_row % 8) || (n_heads > 1 && o_head % 8))
    return fail(ECHO_EUNSUPPORTED, "%s: out or its strides are not multiples of 16 bytes", fn);
  if (!aligned(lse, 4)) return fail(ECHO_EINVAL, "%s: lse is not aligned to its type", fn);
  return ECHO_OK;
}
int check_pages(const char *fn, const int32_t *table, int32_t page_size, int32_t max_pages) {
  if (max_pages < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)))
    return fail(ECHO_EUNSUPPORTED, "%s: page size %d is not a power of two in [16, 65536]", fn, page_size);
  if (max_pages && !table) return fail(ECHO_EINVAL, "%s: NULL page table", fn);
  if (!aligned(table, 4)) return fail(ECHO_EINVAL, "%s: a page table is not aligned to its type", fn);
  return ECHO_OK;
}
int check_ws(const char *fn, const void *ws, size_t bytes, int64_t need) {
  if (need <= 0) return ECHO_OK;
  if (!ws || bytes < static_cast<size_t>(need)) return fail(ECHO_EWORKSPACE, "%s: a workspace of %lld bytes is needed", fn, static_cast<long long>(need));
  if (!aligned(ws, 16)) return fail(ECHO_EINVAL, "%s: the workspace is not aligned to 16 bytes", fn);
  return ECHO_OK;
}

// echo_latent_args, checked, as the kernels take them.
int latent_args(const char *fn, const echo_latent_args *a, LatentArgs *x) {
  if (!a) return fail(ECHO_EINVAL, "%s: NULL arguments", fn);
  int rc = check_cache(fn, a->n_rows, a->n_heads, a->type, a->scale, a->q, a->q_row_stride, a->q_head_stride, a->kv, a->kv_stride, a->n_kv);
  if (rc != ECHO_OK) return rc;
  if (a->k < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (a->block < 1 || a->block > 65536 || (a->block & (a->block - 1)))
    return fail(ECHO_EUNSUPPORTED, "%s: block %d is not a power of two in [1, 65536]", fn, a->block);
  if (static_cast<int64_t>(a->k) * a->block > MAX_TOKENS) return fail(ECHO_EUNSUPPORTED, "%s: more than 2^28 tokens a row", fn);
  if (a->page_size) {
    if (a->n_tables < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
    rc = check_pages(fn, a->page_table, a->page_size, a->n_tables ? a->max_pages : 0);
    if (rc != ECHO_OK) return rc;
    if (a->max_pages < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  }
  if (a->n_rows && a->n_heads && a->k && !a->idx) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if (a->idx_stride < 0) return fail(ECHO_EINVAL, "%s: a stride below 0", fn);
  if (!aligned(a->idx, 4) || !aligned(a->len, 4) || !aligned(a->req, 4)) return fail(ECHO_EINVAL, "%s: an array is not aligned to its type", fn);
  const auto log2 = [](int32_t v) { int s = 0; while ((1 << s) < v) ++s; return s; };
  *x = LatentArgs{static_cast<const uint16_t *>(a->q), a->q_row_stride, a->q_head_stride, static_cast<const uint16_t *>(a->kv), a->kv_stride,
                  a->idx, a->idx_stride, a->len, a->page_size ? a->page_table : nullptr, a->req, a->n_rows, a->n_heads, a->n_kv,
                  a->k * a->block, log2(a->block), a->page_size ? log2(a->page_size) : 0, a->page_size && a->n_tables ? a->max_pages : 0,
                  a->n_tables, a->scale * LOG2E};
  if (a->page_size && !x->table) x->n_kv = 0;              // pages, but none of them: no tokens
  return ECHO_OK;
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_sparse_attention_workspace_bytes(int32_t n_rows, int32_t n_heads, int32_t n_tok) {
  if (n_rows < 1 || n_heads < 1 || n_tok < 0 || n_heads > MAX_HEADS) return 0;
  return static_cast<size_t>(sparse_ws(n_rows, n_heads, n_tok));
}

extern "C" int echo_sparse_attention(const echo_latent_args *a, void *out, int64_t out_row_stride, int64_t out_head_stride, float *lse,
                                     void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "echo_sparse_attention";
  AttArgs x = {};
  int rc = latent_args(fn, a, &x.a);
  if (rc != ECHO_OK || a->n_rows == 0 || a->n_heads == 0) return rc;
  rc = check_out(fn, a->n_rows, a->n_heads, out, out_row_stride, out_head_stride, lse);
  if (rc != ECHO_OK) return rc;
  const Plan p = plan_of(a->n_rows, a->n_heads, x.a.n_tok);
  const int64_t blocks = row_blocks(a->n_rows, a->n_heads, p);
  if (blocks >= MAX_GROUPS)
    return fail(ECHO_EUNSUPPORTED, "%s: more rows, heads and tokens than a launch holds", fn);
  const int64_t need = sparse_ws(a->n_rows, a->n_heads, x.a.n_tok);
  rc = check_ws(fn, ws, ws_bytes, need);
  if (rc != ECHO_OK) return rc;
  const int64_t queries = static_cast<int64_t>(a->n_rows) * a->n_heads;
  x.out = out; x.o_row = out_row_stride; x.o_head = out_head_stride; x.lse = lse;
  x.chunk = p.chunk; x.n_chunks = p.n_chunks;
  if (p.n_chunks > 1) {
    x.parts = p.n_chunks;
    x.part = static_cast<float *>(ws);
    x.part_ml = x.part + queries * p.n_chunks * VALUES;
  }
  rc = launch_attention(x, a->type, 1, p.qt, blocks, S(stream));
  if (rc != ECHO_OK || p.n_chunks == 1) return rc;
  JoinArgs j = {};
  j.part = x.part; j.ml = x.part_ml; j.out = out; j.o_row = out_row_stride; j.o_head = out_head_stride; j.lse = lse;
  j.n_rows = a->n_rows; j.n_heads = a->n_heads; j.parts = p.n_chunks;
  return a->type == ECHO_BF16 ? launch_join<bf16_t>(j, S(stream)) : launch_join<fp16_t>(j, S(stream));
}

extern "C" size_t echo_prefix_attention_workspace_bytes(int32_t n_rows, int32_t n_heads, int32_t n_groups, int32_t max_prefix, int32_t max_own) {
  if (n_rows < 1 || n_heads < 1 || n_groups < 0 || max_prefix < 0 || max_own < 0 || n_heads > MAX_HEADS) return 0;
  const PrefixPlan p = prefix_plan(n_rows, n_heads, n_groups, max_prefix, max_own);
  return static_cast<size_t>(static_cast<int64_t>(n_rows) * n_heads * (p.prefix_parts + p.own_parts) * PART_BYTES);
}

extern "C" int echo_prefix_attention(const echo_prefix_args *a, void *out, int64_t out_row_stride, int64_t out_head_stride, float *lse,
                                     void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "echo_prefix_attention";
  if (!a) return fail(ECHO_EINVAL, "%s: NULL arguments", fn);
  int rc = check_cache(fn, a->n_rows, a->n_heads, a->type, a->scale, a->q, a->q_row_stride, a->q_head_stride, a->kv, a->kv_stride, a->n_kv);
  if (rc != ECHO_OK) return rc;
  if (a->n_groups < 0 || a->max_prefix < 0 || a->max_own < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (a->n_groups > 65536 || a->max_prefix > MAX_TOKENS || a->max_own > MAX_TOKENS)
    return fail(ECHO_EUNSUPPORTED, "%s: more than 65536 groups or 2^28 tokens", fn);
  rc = check_pages(fn, a->prefix_table, a->page_size, a->n_groups ? a->prefix_pages : 0);
  if (rc == ECHO_OK) rc = check_pages(fn, a->own_table, a->page_size, a->n_rows ? a->own_pages : 0);
  if (rc != ECHO_OK) return rc;
  if (a->n_rows == 0 || a->n_heads == 0) return ECHO_OK;
  if ((a->n_groups && (!a->group_begin || !a->prefix_len)) || !a->own_len) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if (!aligned(a->group_begin, 4) || !aligned(a->prefix_len, 4) || !aligned(a->own_len, 4)) return fail(ECHO_EINVAL, "%s: an array is not aligned to its type", fn);
  rc = check_out(fn, a->n_rows, a->n_heads, out, out_row_stride, out_head_stride, lse);
  if (rc != ECHO_OK) return rc;
  const PrefixPlan p = prefix_plan(a->n_rows, a->n_heads, a->n_groups, a->max_prefix, a->max_own);
  const int64_t queries = static_cast<int64_t>(a->n_rows) * a->n_heads;
  const int64_t blocks = p.own_parts ? row_blocks(a->n_rows, a->n_heads, p.own) : 0;
  const int64_t prefix_blocks = p.prefix_parts ? p.tiles * chunk_step(p.prefix_parts) : 0;
  if (blocks + prefix_blocks >= MAX_GROUPS || queries / 4 >= MAX_GROUPS)
    return fail(ECHO_EUNSUPPORTED, "%s: more rows, heads and tokens than a launch holds", fn);
  const int32_t parts = p.prefix_parts + p.own_parts;
  rc = check_ws(fn, ws, ws_bytes, queries * parts * PART_BYTES);
  if (rc != ECHO_OK) return rc;
  int shift = 0;
  while ((1 << shift) < a->page_size) ++shift;
  AttArgs x = {};
  x.a = LatentArgs{static_cast<const uint16_t *>(a->q), a->q_row_stride, a->q_head_stride, static_cast<const uint16_t *>(a->kv), a->kv_stride,
                   nullptr, 0, a->own_len, a->own_table, nullptr, a->n_rows, a->n_heads, a->n_kv, a->max_own, 0, shift, a->own_pages, a->n_rows,
                   a->scale * LOG2E};
  x.out = out; x.o_row = out_row_stride; x.o_head = out_head_stride; x.lse = lse;
  x.parts = parts;
  x.part = static_cast<float *>(ws);
  x.part_ml = x.part + queries * parts * VALUES;
  x.chunk = p.own.chunk; x.n_chunks = p.own.n_chunks; x.first_part = p.prefix_parts;
  if (p.prefix_parts) {
    x.group_begin = a->group_begin; x.prefix_len = a->prefix_len; x.prefix_table = a->prefix_table;
    x.n_groups = a->n_groups; x.prefix_pages = a->prefix_pages;
    x.max_prefix = a->max_prefix; x.prefix_chunk = p.prefix.chunk; x.prefix_chunks = p.prefix_parts;
    x.prefix_blocks = static_cast<uint32_t>(prefix_blocks);
  }
  if (blocks + prefix_blocks > 0) {
    rc = launch_attention(x, a->type, p.prefix.qt, p.own.qt, blocks, S(stream));
    if (rc != ECHO_OK) return rc;
  }
  const JoinArgs j = {x.part, x.part_ml, out, out_row_stride, out_head_stride, lse, a->n_rows, a->n_heads, parts, a->own_len, a->group_begin,
                      a->prefix_len, p.prefix_parts ? a->n_groups : 0, p.prefix.chunk, a->max_prefix, p.prefix_parts, p.own.chunk, a->max_own};
  return a->type == ECHO_BF16 ? launch_join<bf16_t>(j, S(stream)) : launch_join<fp16_t>(j, S(stream));
}
