// Block-scaled FP8 product on gfx950 (echo_matmul_fp8):
//   c[i][j] = sum_t sa(i, t) * sb(j / 128, t) * sum_{p in block t} a[i][p] * b[j][p]
//
// v_mfma_f32_16x16x128_f8f6f4 multiplies 16 x 16 x 128, exactly one scale block, so its result is
// one term of the sum over t.  The weights are its first operand (result rows), the activations
// its second (result columns): lane l then holds c[i = l%16][j = 4 (l/16) .. + 3], four
// consecutive outputs of one row, and one activation scale for all of them, while the weight
// scale is the same for the whole tile.  Folding a term in is one FMA per element with
// s = sa * sb; those FMAs run on the VALU while the matrix core multiplies the next tile.
#include "float_types.cuh"
#include "score_tile.cuh"

namespace echo {

struct MatArgs {
  const uint8_t *a, *b;
  const float *sa, *sb;
  int64_t lda, ldb, as_row, as_blk, bs_row, bs_blk, ldc;
  int32_t m, n, k;
  void *c;
  bool odd;                       // a row of c may start between two dwords
};

ECHO_DEV v8i operand(const u32x4 &x, const u32x4 &y) {
  return v8i{static_cast<int>(x[0]), static_cast<int>(x[1]), static_cast<int>(x[2]), static_cast<int>(x[3]),
             static_cast<int>(y[0]), static_cast<int>(y[1]), static_cast<int>(y[2]), static_cast<int>(y[3])};
}

// Bytes [32 g, 32 g + 32) of a row's 128-byte block that holds `left` bytes, zeros behind them.
// Pieces that start behind the end are read from the block's first piece, which every row has.
ECHO_DEV v8i load_operand(const uint8_t *__restrict__ blk, int g, int left) {
  const int o0 = 32 * g, o1 = o0 + 16;
  u32x4 p[2] = {*reinterpret_cast<const u32x4 *>(blk + (o0 < left ? o0 : 0)),
                *reinterpret_cast<const u32x4 *>(blk + (o1 < left ? o1 : 0))};
  if (left < 128) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int keep = left - (o0 + 16 * h + 4 * i);       // valid bytes of this word
        const uint32_t mask = keep >= 4 ? ~0u : keep <= 0 ? 0u : (1u << (8 * keep)) - 1u;
        p[h][i] &= mask;
      }
  }
  return operand(p[0], p[1]);
}

// One 16 x 16 x 128 term on the FP8 matrix core, or exactly (EXACT) on the bf16 one.
//
// The FP8 core adds products in groups of eight neighbours: within a group it cuts every product
// at 2^-13 of the largest one's power of two (measured: a product survives next to one 2^13 times
// larger and is gone at 2^14, the groups are then summed in fp32).  For normally distributed
// operands a sum is off by 1.6e-5 of its size, far below the half step of a bf16 (2^-9) or fp16
// (2^-12) result, so those use it where there are many outputs.  Results in fp32 convert the codes to bf16, which holds every
// E4M3FN number and multiplies exactly into fp32, and take four bf16 MFMAs at half the rate.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <bool EXACT> struct Operand;
template <> struct Operand<false> {
  v8i v;
  ECHO_DEV void set(const v8i &x) { v = x; }
};
template <> struct Operand<true> {
  bf16x8 v[4];
  ECHO_DEV void set(const v8i &x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned word = static_cast<unsigned>(x[2 * i + h]);
        const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.f, false);
        const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.f, true);
        v[i][4 * h] = lo[0]; v[i][4 * h + 1] = lo[1]; v[i][4 * h + 2] = hi[0]; v[i][4 * h + 3] = hi[1];
      }
  }
};
ECHO_DEV v4f mfma128(const Operand<false> &x, const Operand<false> &y) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
ECHO_DEV v4f mfma128(const Operand<true> &x, const Operand<true> &y) {
  v4f c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v[i], y.v[i], c, 0, 0, 0);
  return c;
}

// Outputs at any address their type allows: gfx950 writes 8 or 16 bytes there.  Written one by one,
// rows of odd length cost more (16384 x 8191 x 2048 in bf16 on MI355X: 431 us, 352 in wide stores
// between dwords, 313 in wide stores a dword on).
typedef v4f v4f_any __attribute__((aligned(4)));
typedef uint32_t u32_any __attribute__((aligned(2)));

template <typename T>
ECHO_DEV u32x2 pack4(const v4f &v) {
  T e[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) e[u] = from_f32<T>(v[u]);
  u32x2 w;
  __builtin_memcpy(&w, e, 8);
  return w;
}
// Stores the lane's four consecutive outputs of row i, columns j .. j + 3.
template <typename T>
ECHO_DEV void store_c(const MatArgs &a, int64_t i, int32_t j, const v4f &v) {
  if (i >= a.m || j >= a.n) return;
  T *p = static_cast<T *>(a.c) + i * a.ldc + j;
  if (j + 4 <= a.n) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<v4f_any *>(p) = v;
    else *reinterpret_cast<u32x2_any *>(p) = pack4<T>(v);
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (j + u < a.n) p[u] = from_f32<T>(v[u]);
  }
}

// The first `count` of eight 16-bit outputs.
template <typename T>
ECHO_DEV void store_some(T *p, const u32x4 &v, int count) {
  if (count >= 8) {
    *reinterpret_cast<u32x4_any *>(p) = v;
  } else if (count > 0) {
    const bool half = count & 4;
    if (half) *reinterpret_cast<u32x2_any *>(p) = u32x2{v[0], v[1]};
    if (count & 2) *reinterpret_cast<u32_any *>(p + (count & 4)) = half ? v[2] : v[0];
    const uint32_t last = count & 2 ? (half ? v[3] : v[1]) : (half ? v[2] : v[0]);
    if (count & 1) reinterpret_cast<uint16_t *>(p)[count - 1] = static_cast<uint16_t>(last);
  }
}

// ---------------------------------------------------------------- few outputs
// One workgroup per 16 * NT weight rows and 16 * MT activation rows; its 8 waves take the scale blocks
// in turn and their sums are joined in LDS in wave order (four waves are 3% faster up to K = 1000, 20 to
// 40% slower at 6000; sixteen up to 30% slower).  Reading the weights is what costs here (1 x 8192 x
// 8192 on MI355X: 13.5 us = 5.0 TB/s), so every output type gets the exact products.  A wave fetches a
// block once the one before has arrived: 1 x 8192 x 2048, two blocks a wave, is the launch, two trips to
// memory in a row and the join (5.2 us).
constexpr int SW = 8;
template <typename T, int MT, int NT>
__global__ __launch_bounds__(SW * 64) void matmul_few_kernel(MatArgs a) {
  __shared__ float part[SW][MT * NT][64 * 4];
  const int wv = threadIdx.x >> 6, l = lane_id(), j = l & 15, g = l >> 4;
  const int32_t n0 = blockIdx.x * (16 * NT), m0 = blockIdx.y * (16 * MT);
  const int nb = (a.k + 127) >> 7;
  const uint8_t *bp[NT], *ap[MT];
#pragma unroll
  for (int i = 0; i < NT; ++i) bp[i] = a.b + static_cast<int64_t>(min(n0 + 16 * i + j, a.n - 1)) * a.ldb;
#pragma unroll
  for (int i = 0; i < MT; ++i) ap[i] = a.a + static_cast<int64_t>(min(m0 + 16 * i + j, a.m - 1)) * a.lda;
  v4f acc[MT][NT];
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y) acc[x][y] = v4f{0.f, 0.f, 0.f, 0.f};
  // The next block's loads are under way while a block is converted and multiplied.
  v8i nbv[NT], nav[MT];
  float nsa[MT], nsb = 0.f;
  auto fetch = [&](int t) {
    const int left = min(a.k - t * 128, 128);
    const int64_t o = static_cast<int64_t>(t) * 128;
#pragma unroll
    for (int y = 0; y < NT; ++y) nbv[y] = load_operand(bp[y] + o, g, left);
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      nav[x] = load_operand(ap[x] + o, g, left);
      nsa[x] = a.sa[min(m0 + 16 * x + j, a.m - 1) * a.as_row + t * a.as_blk];
    }
    nsb = a.sb[(n0 >> 7) * a.bs_row + t * a.bs_blk];
  };
  if (wv < nb) fetch(wv);
  for (int t = wv; t < nb; t += SW) {
    Operand<true> bv[NT], av[MT];
    float s[MT];
#pragma unroll
    for (int y = 0; y < NT; ++y) bv[y].set(nbv[y]);
#pragma unroll
    for (int x = 0; x < MT; ++x) {
      av[x].set(nav[x]);
      s[x] = nsa[x] * nsb;
    }
    if (t + SW < nb) fetch(t + SW);
#pragma unroll
    for (int x = 0; x < MT; ++x)
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        const v4f c = mfma128(bv[y], av[x]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[x][y][v] = fmaf(c[v], s[x], acc[x][y][v]);
      }
  }
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y) *reinterpret_cast<v4f *>(&part[wv][x * NT + y][l * 4]) = acc[x][y];
  __syncthreads();
  for (int i = wv; i < MT * NT; i += SW) {
    v4f sum = *reinterpret_cast<const v4f *>(&part[0][i][l * 4]);
#pragma unroll
    for (int w = 1; w < SW; ++w) sum += *reinterpret_cast<const v4f *>(&part[w][i][l * 4]);
    store_c<T>(a, m0 + 16 * (i / NT) + j, n0 + 16 * (i % NT) + 4 * g, sum);
  }
}

// ---------------------------------------------------------------- tiles
// s_waitcnt's operand for "at most n vector memory operations outstanding" and nothing else.
constexpr int vmcnt(int n) { return (n & 15) | 0x0F70 | (n >> 4) << 14; }

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

// A row of a stage is 128 bytes in eight 16-byte pieces; piece s of row r sits at place
// s ^ ((r >> 1) & 7), so the 16 rows of an operand read hit different banks.
ECHO_DEV int place(int row, int seg) { return row * 128 + ((seg ^ ((row >> 1) & 7)) << 4); }

// ROWS rows of one stage from global memory straight to LDS by NW waves: a wave's load puts 64
// consecutive 16-byte pieces (8 rows), so the exchange of pieces is made on the global side.  A
// thread's piece is the same byte of every row it loads (NW is even), and rows are 32-bit
// offsets from the tile's first one.
template <int ROWS, int NW>
struct StageLoad {
  static_assert(NW % 2 == 0, "the exchange repeats every 16 rows");
  static constexpr int N = ROWS * 8 / (NW * 64);       // loads per thread
  const uint8_t *tile;                                 // uniform
  uint32_t off[N];
  ECHO_DEV void init(const uint8_t *base, int64_t ld, int32_t r0, int32_t n_rows, int wv, int seg) {
    tile = base + static_cast<int64_t>(r0) * ld;
#pragma unroll
    for (int i = 0; i < N; ++i)
      off[i] = static_cast<uint32_t>(min((i * NW + wv) * 8 + (lane_id() >> 3), n_rows - 1 - r0)) * static_cast<uint32_t>(ld) + seg;
  }
  // Load i of block t; back: 0, or, behind a short block's end, the distance to the row's first
  // piece.
  ECHO_DEV void load(uint8_t *__restrict__ stage, int t, int i, int wv, uint32_t back) const {
    __builtin_amdgcn_global_load_lds((glb_void *)(tile + static_cast<int64_t>(t) * 128 + (off[i] - back)),
                                     (lds_void *)(stage + (i * NW + wv) * 1024), 16, 0, 0);
  }
};

// The lane's 32 bytes of row `row` of a stage, pieces g and g + 4; their places repeat every 16 rows
// (2048 bytes).  Which bytes of a row a lane group multiplies does not matter as long as both
// operands agree; with these two no read has a bank conflict, while pieces 2g and 2g + 1 had one
// in every read (the sixteen lanes served together come from rows of two neighbouring lane groups:
// SQ_LDS_BANK_CONFLICT half of the LDS cycles, 8192^3 2078 against 2105 TFLOP/s).
struct Pieces {
  int32_t p0, p1;
  ECHO_DEV void init(int row, int g) { p0 = place(row, g); p1 = place(row, g + 4); }
  ECHO_DEV v8i read(const uint8_t *__restrict__ stage, int rows16) const {
    return operand(*reinterpret_cast<const u32x4 *>(stage + p0 + rows16 * 2048),
                   *reinterpret_cast<const u32x4 *>(stage + p1 + rows16 * 2048));
  }
};
ECHO_DEV v8i keep_bytes(v8i v, int g, int left) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int keep = left - ((i < 4 ? 16 * g : 16 * g + 48) + 4 * i);
    v[i] &= keep >= 4 ? -1 : keep <= 0 ? 0 : static_cast<int>((1u << (8 * keep)) - 1u);
  }
  return v;
}

// BM activation rows x BN weight rows per workgroup, WM x WN per wave; STAGES blocks in LDS.  While
// one is multiplied the loads of a later one are issued one by one between the products: issued
// together at the start of the block they held up its first operand reads (8192^3 on MI355X: 2105
// against 2188 TFLOP/s).
//
// What bounds the 256 x 256 tile: an MFMA takes 32 cycles of its SIMD's matrix core and its result
// four FMAs of 4 cycles, so the products could hide everything else.  At 8192^3 (478 us, 2300
// TFLOP/s) counters give 59% of cycles multiplying at the 1.84 GHz the chip then ran; with 50% it
// ran at 1.98 GHz: the clock falls as the cores fill.  Measured on an earlier form of the loop at
// 2110 TFLOP/s: without its loads 2650, without three of the four FMAs 2200, without barriers 2%
// more.  A wave's accumulators are 128 registers, the most that two waves per SIMD allow beside the
// operands: 64 x 128 outputs per wave.  At 16384 x 8192 x 2048 (264 to 317 us, by box and clock)
// writing the result adds 50 to 60 us: tiles of a size end together and the next ones wait for HBM.
//
// Workgroups go to the 8 XCDs in turn, each with an L2 of its own, so consecutive tiles of one XCD
// are neighbours: it gets one eighth of the tiles, taken in bands of BAND tile rows.  Its 32 CUs then
// hold about 5 x 6 tiles, which read the fewest different rows of a and b (16384 x 8192 x 2048 on
// MI355X: 308 us with bands of 8, 291 with 4, 287 with 5, 289 with 6).
constexpr int BAND = 5;
ECHO_DEV void tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t &tm, uint32_t &tn) {
  const uint32_t total = mt * nt, xcd = id & 7u, i = id >> 3;
  const uint32_t each = total >> 3, more = total & 7u;         // the first `more` XCDs take one more
  uint32_t t = xcd * each + (xcd < more ? xcd : more) + i;
  const uint32_t band = t / (BAND * nt), in = t - band * BAND * nt;
  const uint32_t rows = min(static_cast<uint32_t>(BAND), mt - band * BAND);
  tn = in / rows;
  tm = band * BAND + in - tn * rows;
}

// Empty asm statements stay in program order and emit nothing: each product takes its operand from
// one and hands its result to the next, so the compiler keeps AHEAD products in flight and no more.
ECHO_DEV void pin(Operand<false> &o, v4f &c) { asm volatile("" : "+v"(o.v), "+v"(c)); }
ECHO_DEV void pin(Operand<true> &, v4f &c) { asm volatile("" : "+v"(c)); }
ECHO_DEV void pin(v4f &n, v4f &c) { asm volatile("" : "+v"(n), "+v"(c)); }
ECHO_DEV void pin(Pieces &p) { asm volatile("" : "+v"(p.p0), "+v"(p.p1)); }

template <typename T, int BM, int BN, int WM, int WN, int STAGES>
struct Tile {
  static constexpr int NW = (BM / WM) * (BN / WN), MT = WM / 16, NT = WN / 16;
  static constexpr int AHEAD = 2;                        // products in flight ahead of their FMAs
  static constexpr int LOADS = StageLoad<BM, NW>::N + StageLoad<BN, NW>::N + 1;   // a thread's loads of a block
  static constexpr int EVERY = MT * NT / LOADS / 2 > 0 ? MT * NT / LOADS / 2 + 1 : 1;   // products between two of them
  static constexpr int ROWS = (BM + BN) * 128, STAGE = ROWS + NW * 256;           // bytes: codes, each wave's scales
  static constexpr bool EXACT = sizeof(T) == 4;
  static_assert(WN <= 128 && WM <= 64, "one weight scale per wave, one activation scale per lane");
  static_assert(MT >= AHEAD && NT % 2 == 0, "the products ahead are of this or the next operand");
  static_assert(LOADS * EVERY <= MT * NT + AHEAD, "every load has its place");
  static_assert((STAGES - 2) * LOADS < 64, "the wait counts them");
  static_assert(STAGES * STAGE <= 160 * 1024, "a workgroup's LDS");
  StageLoad<BM, NW> la;
  StageLoad<BN, NW> lb;
  const float *sa, *sb;                                  // uniform
  uint32_t sa_off;                                       // the lane's row of the wave's tile
  int64_t as_blk, bs_blk;
  int nb, k, wv, wm, wn, j, g, seg;
  Pieces pa, pb;
  v4f acc[MT][NT];
  float sbv;                                             // weight scales of 64 blocks, one per lane

  ECHO_DEV void load_one(int t, int i, uint8_t *__restrict__ stage) const {
    constexpr int NA = StageLoad<BM, NW>::N, NB = StageLoad<BN, NW>::N;
    const uint32_t back = seg < k - t * 128 ? 0u : static_cast<uint32_t>(seg);
    if (i < NA) la.load(stage, t, i, wv, back);
    else if (i < NA + NB) lb.load(stage + BM * 128, t, i - NA, wv, back);
    else
      __builtin_amdgcn_global_load_lds((glb_void *)(sa + t * as_blk + sa_off), (lds_void *)(stage + ROWS + wv * 256), 4, 0, 0);
  }
  ECHO_DEV void load(int t, uint8_t *__restrict__ stage) const {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load_one(t, i, stage);
  }
  ECHO_DEV void load_weight_scales(int t) { sbv = sb[min(t + lane_id(), nb - 1) * bs_blk]; }
  template <bool TAIL>
  ECHO_DEV void operand_of(Operand<EXACT> &o, const uint8_t *__restrict__ stage, const Pieces &p, int rows16, int left) const {
    v8i v = p.read(stage, rows16);
    if (TAIL) v = keep_bytes(v, g, left);
    o.set(v);
  }
  // Waits until the loads of all blocks but the `later` youngest have arrived, at most STAGES - 2.
  template <int R = STAGES - 2>
  ECHO_DEV static void wait(int later) {
    if constexpr (R == 0) {
      __builtin_amdgcn_s_waitcnt(vmcnt(0));
    } else {
      if (later >= R) __builtin_amdgcn_s_waitcnt(vmcnt(R * LOADS));
      else wait<R - 1>(later);
    }
  }
  // Block t from `cur`; with NEXT block t + STAGES - 1's loads go to `nxt`.  Product i is issued before the
  // FMAs of product i - AHEAD; a weight operand is read once the one before the last has been used.
  template <bool TAIL, bool NEXT>
  ECHO_DEV void block(int t, uint8_t *__restrict__ cur, uint8_t *__restrict__ nxt) {
    if (t > 0 && (t & 63) == 0) {
      load_weight_scales(t);
      __builtin_amdgcn_s_waitcnt(vmcnt(0));              // here, not on every block's way
    }
    const float sbt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sbv), t & 63));
    float s[MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) s[x] = reinterpret_cast<const float *>(cur + ROWS + wv * 256)[16 * x + j] * sbt;
    const int left = k - t * 128;
    Operand<EXACT> av[MT], bv[2];
    operand_of<TAIL>(bv[0], cur + BM * 128, pb, 0, left);
#pragma unroll
    for (int x = 0; x < MT; ++x) operand_of<TAIL>(av[x], cur, pa, x, left);
    v4f c[AHEAD];
#pragma unroll
    for (int i = 0; i < MT * NT + AHEAD; ++i) {
      const int x = i % MT, y = i / MT, e = i - AHEAD;
      if (x == 0 && y + 1 < NT) {
        pin(pb);
        operand_of<TAIL>(bv[(y + 1) & 1], cur + BM * 128, pb, y + 1, left);
      }
      if (NEXT && i % EVERY == EVERY - 1 && i / EVERY < LOADS) load_one(t + STAGES - 1, i / EVERY, nxt);
      v4f co = {0.f, 0.f, 0.f, 0.f};
      if (e >= 0) co = c[e % AHEAD];
      if (i < MT * NT) {
        pin(bv[y & 1], co);
        v4f cn = mfma128(bv[y & 1], av[x]);
        pin(cn, co);
        c[i % AHEAD] = cn;
      }
      if (e >= 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[e % MT][e / MT][v] = fmaf(co[v], s[e % MT], acc[e % MT][e / MT][v]);
      }
    }
  }
};

template <typename T, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void matmul_tile_kernel(MatArgs a) {
  typedef Tile<T, BM, BN, WM, WN, STAGES> K;
  __shared__ __attribute__((aligned(16))) uint8_t lds[STAGES][K::STAGE];
  K w;
  w.wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l = lane_id();
  w.j = l & 15;
  w.g = l >> 4;
  w.seg = ((l & 7) ^ ((w.wv * 4 + (l >> 4)) & 7)) << 4;
  uint32_t tm, tn;
  tile_of(blockIdx.x, (a.m + BM - 1) / BM, (a.n + BN - 1) / BN, tm, tn);
  const int32_t m0 = tm * BM, n0 = tn * BN;
  w.wm = (w.wv % (BM / WM)) * WM;
  w.wn = (w.wv / (BM / WM)) * WN;
  w.pa.init(w.wm + w.j, w.g);
  w.pb.init(w.wn + w.j, w.g);
  w.k = a.k;
  w.nb = (a.k + 127) >> 7;
  w.la.init(a.a, a.lda, m0, a.m, w.wv, w.seg);
  w.lb.init(a.b, a.ldb, n0, a.n, w.wv, w.seg);
  w.as_blk = a.as_blk;
  w.bs_blk = a.bs_blk;
  w.sa = a.sa + m0 * a.as_row;
  w.sa_off = static_cast<uint32_t>(min(w.wm + min(l, WM - 1), a.m - 1 - m0)) * static_cast<uint32_t>(a.as_row);
  w.sb = a.sb + (min(n0 + w.wn, a.n - 1) >> 7) * a.bs_row;
#pragma unroll
  for (int x = 0; x < K::MT; ++x)
#pragma unroll
    for (int y = 0; y < K::NT; ++y) w.acc[x][y] = v4f{0.f, 0.f, 0.f, 0.f};
  if (w.nb > 0) {
    w.load_weight_scales(0);
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) w.load(min(t, w.nb - 1), lds[t]);   // no branch: the loads stay countable
  }
  // Block t is in LDS for every wave, and every wave has read block t - 1 (its products have taken
  // the operands).  A plain barrier: __syncthreads() would wait for the younger blocks' loads too.
  auto arrive = [&](int t) {
    K::wait(w.nb - 1 - t);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  int t = 0, cur = 0, nxt = STAGES - 1;
  for (; t + STAGES - 1 < w.nb; ++t) {
    arrive(t);
    w.template block<false, true>(t, lds[cur], lds[nxt]);
    nxt = cur;
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  }
  for (; t < w.nb; ++t) {                                // nothing more to load; the last block may be short
    arrive(t);
    w.template block<true, false>(t, lds[cur], lds[nxt]);
    nxt = cur;
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int y = 0; y < K::NT; ++y)
#pragma unroll
      for (int x = 0; x < K::MT; ++x)
        store_c<T>(a, m0 + w.wm + 16 * x + w.j, n0 + w.wn + 16 * y + 4 * w.g, w.acc[x][y]);
  } else {
    // Two neighbouring tiles: lane rows of 16 exchange halves, so that a lane holds eight
    // consecutive outputs, lane groups 0 and 2 those of the first tile.
    constexpr int PAIRS = K::NT / 2;
    const auto eight = [&](int x, int y) {
      const u32x2 p = pack4<T>(w.acc[x][2 * y]), q = pack4<T>(w.acc[x][2 * y + 1]);
      const v2u lo = __builtin_amdgcn_permlane16_swap(p[0], q[0], false, false);
      const v2u hi = __builtin_amdgcn_permlane16_swap(p[1], q[1], false, false);
      return u32x4{lo[0], hi[0], lo[1], hi[1]};
    };
    const int32_t col = n0 + w.wn + 16 * (w.g & 1) + 8 * (w.g >> 1);
    if (m0 + BM <= a.m && n0 + BN <= a.n && !a.odd) {    // a whole tile of even rows: no bounds
#pragma unroll
      for (int x = 0; x < K::MT; ++x) {
        T *row = static_cast<T *>(a.c) + static_cast<int64_t>(m0 + w.wm + 16 * x + w.j) * a.ldc + col;
#pragma unroll
        for (int y = 0; y < PAIRS; ++y) *reinterpret_cast<u32x4_any *>(row + 32 * y) = eight(x, y);
      }
      return;
    }
    // Stores that start between two dwords take twice as long (8192 x 6273 x 128: 70 us, 6272 columns
    // 30).  Such rows are written one output further on: a lane gives up its first output to the lane in
    // front and takes the next lane's (35 us).
    const int next = w.j + 16 * (0x0132 >> (4 * w.g) & 3);
#pragma unroll
    for (int x = 0; x < K::MT; ++x) {
      const int32_t i = m0 + w.wm + 16 * x + w.j;
      T *row = static_cast<T *>(a.c) + static_cast<int64_t>(i) * a.ldc;
      const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(row + n0) >> 1) & 1;
      u32x4 d = eight(x, 0);
#pragma unroll
      for (int y = 0; y < PAIRS; ++y) {
        const u32x4 after = y + 1 < PAIRS ? eight(x, y + 1) : d;
        const uint32_t end = __shfl(w.g == 0 ? after[0] : d[0], next);
        const int32_t to = col + 32 * y + odd;
        const int count = i >= a.m ? 0 : min(a.n - to, y + 1 == PAIRS && w.g == 3 ? 8 - odd : 8);
        if (odd && y == 0 && w.g == 0 && i < a.m && col < a.n) reinterpret_cast<uint16_t *>(row)[col] = static_cast<uint16_t>(d[0]);
        const u32x4 v = odd ? u32x4{d[0] >> 16 | d[1] << 16, d[1] >> 16 | d[2] << 16, d[2] >> 16 | d[3] << 16, d[3] >> 16 | end << 16} : d;
        store_some(row + to, v, count);
        d = after;
      }
    }
  }
}

// ---------------------------------------------------------------- few tiles
template <bool V> struct Const { static constexpr bool value = V; };
template <int V> struct Int { static constexpr int value = V; };

// 64 x 64 outputs per workgroup, its waves taking the scale blocks in turn: each multiplies whole
// blocks through LDS stages of its own, so no wave waits for another until the sums are joined at the
// end, in wave order.  Where no more than one tile falls to a CU this keeps a block in flight for
// every wave.
template <typename T, int SW, int STAGES>
__global__ __launch_bounds__(SW * 64) void matmul_split_kernel(MatArgs a) {
  constexpr int MT = 4, NT = 4, SIDE = 64, LOADS = 2 * SIDE / 8 + 1;
  constexpr int STAGE = 2 * SIDE * 128 + 256;
  constexpr bool EXACT = sizeof(T) == 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[SW][STAGES][STAGE];
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l = lane_id(), j = l & 15, g = l >> 4;
  uint32_t tm, tn;
  tile_of(blockIdx.x, (a.m + SIDE - 1) / SIDE, (a.n + SIDE - 1) / SIDE, tm, tn);
  const int32_t m0 = tm * SIDE, n0 = tn * SIDE;
  const int nb = (a.k + 127) >> 7, own = nb > wv ? (nb - wv + SW - 1) / SW : 0;    // this wave's blocks

  // a load is 8 rows of 8 pieces; the pieces' exchange alternates between loads
  uint32_t row[2][SIDE / 8];
#pragma unroll
  for (int i = 0; i < SIDE / 8; ++i) {
    const int r = i * 8 + (l >> 3);
    row[0][i] = static_cast<uint32_t>(min(r, a.m - 1 - m0)) * static_cast<uint32_t>(a.lda);
    row[1][i] = static_cast<uint32_t>(min(r, a.n - 1 - n0)) * static_cast<uint32_t>(a.ldb);
  }
  const uint32_t sa_off = static_cast<uint32_t>(min(l, a.m - 1 - m0)) * static_cast<uint32_t>(a.as_row);
  const uint8_t *pa0 = a.a + m0 * a.lda, *pb0 = a.b + n0 * a.ldb;
  const float *sa = a.sa + m0 * a.as_row, *sb = a.sb + (n0 >> 7) * a.bs_row;
  const int seg0 = ((l & 7) ^ (l >> 4)) << 4;
  auto load_one = [&](int t, int i, uint8_t *__restrict__ stage) {
    if (i < 2 * SIDE / 8) {
      const int side = i / (SIDE / 8), r = i % (SIDE / 8);
      const int seg = seg0 ^ ((r & 1) << 6);
      const uint8_t *p = (side ? pb0 : pa0) + static_cast<int64_t>(t) * 128;
      __builtin_amdgcn_global_load_lds((glb_void *)(p + (row[side][r] + (seg < a.k - t * 128 ? seg : 0))),
                                       (lds_void *)(stage + (side * SIDE + r * 8) * 128), 16, 0, 0);
    } else {
      __builtin_amdgcn_global_load_lds((glb_void *)(sa + t * a.as_blk + sa_off), (lds_void *)(stage + 2 * SIDE * 128), 4, 0, 0);
    }
  };
  Pieces pa, pb;
  pa.init(j, g);
  pb = pa;
  v4f acc[MT][NT];
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y) acc[x][y] = v4f{0.f, 0.f, 0.f, 0.f};
  float sbv = 0.f;                                       // weight scales of 64 own blocks, one per lane

  // Own block i (block t) from cur, with MORE own block i + STAGES - 1's loads going to nxt; without, it
  // may be short.
  auto block = [&](int i, uint8_t *__restrict__ cur, uint8_t *__restrict__ nxt, auto more) {
    constexpr bool MORE = decltype(more)::value;
    const int t = wv + i * SW, left = a.k - t * 128;
    const float sbt = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sbv), i & 63));
    float s[MT];
#pragma unroll
    for (int x = 0; x < MT; ++x) s[x] = reinterpret_cast<const float *>(cur + 2 * SIDE * 128)[16 * x + j] * sbt;
    Operand<EXACT> av[MT], bv[2];
    auto get = [&](Operand<EXACT> &o, const uint8_t *__restrict__ stage, const Pieces &p, int rows16) {
      v8i v = p.read(stage, rows16);
      if (!MORE) v = keep_bytes(v, g, left);
      o.set(v);
    };
    get(bv[0], cur + SIDE * 128, pb, 0);
#pragma unroll
    for (int x = 0; x < MT; ++x) get(av[x], cur, pa, x);
    constexpr int AHEAD = 2;
    v4f c[AHEAD];
#pragma unroll
    for (int u = 0; u < MT * NT + AHEAD; ++u) {
      const int x = u % MT, y = u / MT, e = u - AHEAD;
      if (x == 0 && y + 1 < NT) {
        pin(pb);
        get(bv[(y + 1) & 1], cur + SIDE * 128, pb, y + 1);
      }
      if (MORE && u < LOADS) load_one(t + (STAGES - 1) * SW, u, nxt);
      v4f co = {0.f, 0.f, 0.f, 0.f};
      if (e >= 0) co = c[e % AHEAD];
      if (u < MT * NT) {
        pin(bv[y & 1], co);
        v4f cn = mfma128(bv[y & 1], av[x]);
        pin(cn, co);
        c[u % AHEAD] = cn;
      }
      if (e >= 0) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[e % MT][e / MT][v] = fmaf(co[v], s[e % MT], acc[e % MT][e / MT][v]);
      }
    }
  };
  static_assert(LOADS <= MT * NT + 2 && STAGES >= 2, "every load has its place");
  if (own > 0) {
    sbv = sb[min(wv + l * SW, nb - 1) * a.bs_blk];
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
#pragma unroll
      for (int q = 0; q < LOADS; ++q) load_one(wv + min(i, own - 1) * SW, q, lds[wv][i]);
  }
  int i = 0, cur = 0, nxt = STAGES - 1;
  auto arrive = [&](auto full) {                         // full: STAGES - 2 younger blocks are on their way
    if (i > 0 && (i & 63) == 0) {
      sbv = sb[min(wv + (i + l) * SW, nb - 1) * a.bs_blk];
      __builtin_amdgcn_s_waitcnt(vmcnt(0));
    }
    __builtin_amdgcn_s_waitcnt(vmcnt(decltype(full)::value ? (STAGES - 2) * LOADS : 0));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  auto step = [&] {
    __builtin_amdgcn_wave_barrier();
    nxt = cur;
    cur = cur + 1 == STAGES ? 0 : cur + 1;
  };
  for (; i + STAGES - 1 < own; ++i) {
    arrive(Const<true>{});
    block(i, lds[wv][cur], lds[wv][nxt], Const<true>{});
    step();
  }
  for (; i < own; ++i) {
    arrive(Const<false>{});
    block(i, lds[wv][cur], lds[wv][nxt], Const<false>{});
    step();
  }
  // join, 16 KB per wave in the stages it no longer reads
  float *part = reinterpret_cast<float *>(lds[wv][0]);
  asm volatile("" ::: "memory");
#pragma unroll
  for (int x = 0; x < MT; ++x)
#pragma unroll
    for (int y = 0; y < NT; ++y) *reinterpret_cast<v4f *>(part + ((x * NT + y) * 64 + l) * 4) = acc[x][y];
  __syncthreads();
  for (int i = wv; i < MT * NT; i += SW) {
    v4f sum = *reinterpret_cast<const v4f *>(reinterpret_cast<const float *>(lds[0][0]) + (i * 64 + l) * 4);
#pragma unroll
    for (int q = 1; q < SW; ++q) sum += *reinterpret_cast<const v4f *>(reinterpret_cast<const float *>(lds[q][0]) + (i * 64 + l) * 4);
    store_c<T>(a, m0 + 16 * (i / NT) + j, n0 + 16 * (i % NT) + 4 * g, sum);
  }
}

template <typename T, int BM, int BN, int WM, int WN, int STAGES>
static void launch_tiles(const MatArgs &a, hipStream_t st) {
  const uint32_t tiles = static_cast<uint32_t>((static_cast<int64_t>(a.m) + BM - 1) / BM * ((static_cast<int64_t>(a.n) + BN - 1) / BN));
  matmul_tile_kernel<T, BM, BN, WM, WN, STAGES><<<tiles, (BM / WM) * (BN / WN) * 64, 0, st>>>(a);
}

// The kernels a product can take.
enum Form { FEW_16_16, FEW_32_16, FEW_32_32, SPLIT_64, TILE_64, TILE_64_128, TILE_128_ONE, TILE_128, TILE_256 };
static const char *const FORM_NAMES[] = {"few 16x16", "few 32x16", "few 32x32", "split 64x64", "tile 64x64",
                                         "tile 64x128", "tile 128x128, 3 stages", "tile 128x128", "tile 256x256"};

static uint32_t cdiv(int32_t x, int32_t y) { return static_cast<uint32_t>((static_cast<int64_t>(x) + y - 1) / y); }

// The smallest tile that gives each of the 256 CUs at most one: below that, what a CU can load is what
// takes the time.  All times are us on MI355X, in bf16 unless said.
static Form form_of(int32_t m, int32_t n, int32_t k, bool fp32) {
  const auto tiles = [&](int bm, int bn) { return static_cast<int64_t>(cdiv(m, bm)) * cdiv(n, bn); };
  if (m <= 16 || tiles(16, 16) <= 256) return FEW_16_16;       // 116 x 100 x 6000: 6.4, split 64 x 64 tiles 10.5
  if ((m <= 32 && n < 256 * 32) || tiles(32, 16) <= 256) return FEW_32_16;   // 64 x 2048 x 6000: 9.3, 10.6 and
                                                               // 14.0 in 16 x 16 and 64 x 64
  if (m <= 32 || tiles(32, 32) <= 256) return FEW_32_32;       // 512 x 512 x 6000: 12.5 and 16.5 in 64 x 64,
                                                               // 600 x 530 x 2048, more than 256: 10.8 and 6.3
  // The split form's waves share out the scale blocks (700 x 700 x 4000: 12.3, with shared stages 13.0; fp32
  // 14.6 and 19.4) unless there are hardly more than waves (1000 x 1000 x 300: 4.5 and 4.2).
  if (tiles(64, 64) <= 256) return k > 5 * 128 ? SPLIT_64 : TILE_64;
  if (tiles(64, 128) <= 256) return TILE_64_128;               // 1728 x 640 x 5000: 21.3, 26.2 in 64 x 64
  // fp32 results hold their operands as bf16: too many registers for the largest tile, and always
  // two stages (2112 x 1024 x 2048: 20.6, 22.1 with three)
  if (fp32) return TILE_128;
  // One 128 x 128 tile a CU wants a third stage (2000 x 2000 x 5000: 31.7, 41.9 with two), more a
  // second workgroup (2500 x 3000 x 5000: 50.5 with two stages, 59.7 with three).  From two a CU
  // 256 x 256 tiles are faster (5117 x 2046 x 5000: 67.9 and 89.5) unless their last round leaves
  // more than a quarter of the CUs without one (280 tiles, 5117 x 3582 x 2048: 58.7 and 50.7; 448
  // tiles, 7165 x 4094 x 2048: 64.7 and 75.1).
  if (tiles(128, 128) <= 256) return TILE_128_ONE;
  const int64_t big = tiles(256, 256), rounds = (big + 255) / 256;
  return tiles(128, 128) > 512 && (rounds == 1 || big >= rounds * 192) ? TILE_256 : TILE_128;
}

template <typename T>
static int launch_matmul(const MatArgs &a, hipStream_t st) {
  const auto few = [&](auto mt, auto nt) {
    constexpr int MT = decltype(mt)::value, NT = decltype(nt)::value;
    matmul_few_kernel<T, MT, NT><<<dim3(cdiv(a.n, 16 * NT), cdiv(a.m, 16 * MT)), SW * 64, 0, st>>>(a);
  };
  constexpr bool FP32 = sizeof(T) == 4;
  switch (form_of(a.m, a.n, a.k, FP32)) {
    case FEW_16_16: few(Int<1>{}, Int<1>{}); break;
    case FEW_32_16: few(Int<2>{}, Int<1>{}); break;
    case FEW_32_32: few(Int<2>{}, Int<2>{}); break;
    case SPLIT_64: matmul_split_kernel<T, 4, 2><<<cdiv(a.m, 64) * cdiv(a.n, 64), 256, 0, st>>>(a); break;
    case TILE_64: launch_tiles<T, 64, 64, 32, 32, 4>(a, st); break;
    case TILE_64_128: launch_tiles<T, 64, 128, 32, 64, 3>(a, st); break;
    case TILE_128: launch_tiles<T, 128, 128, 64, 64, 2>(a, st); break;
    case TILE_128_ONE:
      if constexpr (!FP32) launch_tiles<T, 128, 128, 64, 64, 3>(a, st);
      break;
    case TILE_256:
      if constexpr (!FP32) launch_tiles<T, 256, 256, 64, 128, 2>(a, st);
      break;
  }
  return check_launch("matmul_fp8");
}

}  // namespace echo

using namespace echo;

extern "C" const char *echo_matmul_fp8_form(int32_t m, int32_t n, int32_t k, int32_t c_type) {
  return m <= 0 || n <= 0 || k < 0 ? "" : FORM_NAMES[form_of(m, n, k, c_type == ECHO_FP32)];
}

extern "C" int echo_matmul_fp8(const uint8_t *a, int64_t lda, const float *a_scale, int64_t as_row, int64_t as_blk,
                               const uint8_t *b, int64_t ldb, const float *b_scale, int64_t bs_row, int64_t bs_blk,
                               int32_t m, int32_t n, int32_t k, void *c, int64_t ldc, int32_t c_type, void *stream) {
  if (m < 0 || n < 0 || k < 0) return fail(ECHO_EINVAL, "echo_matmul_fp8: negative size");
  if (c_type != ECHO_BF16 && c_type != ECHO_FP16 && c_type != ECHO_FP32)
    return fail(ECHO_EINVAL, "echo_matmul_fp8: type %d", c_type);
  if (m == 0 || n == 0) return ECHO_OK;
  if (!c || (k && (!a || !b || !a_scale || !b_scale))) return fail(ECHO_EINVAL, "echo_matmul_fp8: NULL pointer");
  if (lda < k || ldb < k || ldc < n) return fail(ECHO_EINVAL, "echo_matmul_fp8: row stride below the row");
  if (k == 0) a = b = nullptr, lda = ldb = 0;             // no byte of them is read
  if (reinterpret_cast<uintptr_t>(a) % 16 || reinterpret_cast<uintptr_t>(b) % 16 || lda % 16 || ldb % 16)
    return fail(ECHO_EUNSUPPORTED, "echo_matmul_fp8: a, b, lda or ldb is not a multiple of 16");
  const int64_t tiles = ((static_cast<int64_t>(m) + 127) / 128) * ((static_cast<int64_t>(n) + 127) / 128);
  if (k > 0x7FFFFFFF - 256 || n > (1 << 26) || m > (1 << 26) || tiles >= (1 << 24))
    return fail(ECHO_EUNSUPPORTED, "echo_matmul_fp8: size beyond the grid");
  if (as_row < 0 || as_row > (1 << 22) || as_blk < 0 || bs_row < 0 || bs_blk < 0)
    return fail(ECHO_EUNSUPPORTED, "echo_matmul_fp8: a scale stride below 0, or activation scales more than 2^22 apart");
  if (lda > (1 << 22) || ldb > (1 << 22)) return fail(ECHO_EUNSUPPORTED, "echo_matmul_fp8: rows of more than 2^22 bytes");
  if (reinterpret_cast<uintptr_t>(a_scale) % 4 || reinterpret_cast<uintptr_t>(b_scale) % 4)
    return fail(ECHO_EINVAL, "echo_matmul_fp8: a scale is not aligned to its type");
  const size_t size = c_type == ECHO_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(c) % size) return fail(ECHO_EINVAL, "echo_matmul_fp8: c is not aligned to its type");
  const MatArgs x = {a, b, a_scale, b_scale, lda, ldb, as_row, as_blk, bs_row, bs_blk, ldc, m, n, k, c,
                     reinterpret_cast<uintptr_t>(c) % 4 != 0 || ldc * size % 4 != 0};
  switch (c_type) {
    case ECHO_BF16: return launch_matmul<bf16_t>(x, S(stream));
    case ECHO_FP16: return launch_matmul<fp16_t>(x, S(stream));
    default: return launch_matmul<float>(x, S(stream));
  }
}
