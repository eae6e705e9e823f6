// Norms of query and key heads with the position rotation in the same pass, written back in the
// inputs' type (echo_qk_norm_rope) or as FP8 queries, folded score weights and rows of the
// indexer's key cache (echo_indexer_qk).
//
// One head of one token is a row of D values.  With the row's 32-bit values x_i:
//   RMS norm     n_i = x_i / sqrt(mean(x^2) + eps) * w_i
//   layer norm   n_i = (x_i - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * w_i + b_i
//   rotation     the pair (u, v) at angle index p becomes (u c_p - v s_p, v c_p + u s_p),
//                c and s from row pos of the table; pairs are (i, i + R/2) or (2i, 2i + 1) of
//                the R rotated values, which start at rot_begin
//   FP8          scale = max(amax(n) / 448, 2^-126), codes n / scale
//
// A row is held by G lanes of 8 values (G the power of two that covers D), so a wave reads 64/G
// rows with 16-byte loads, the sums are butterflies over those lanes, and the partner of a
// rotated half comes from another lane of the row.  Everything is read once and written once.
//
// A wave takes HU loads' worth of rows.  Where a side has at least as many heads as a load has
// rows, they are heads of ONE token: its position, its angles and every address but the lane's
// part are the same for the whole wave, so they are scalar work and the angles are read once for
// all its heads.  With fewer heads (the indexer's single key) a load takes several tokens instead,
// lest most lanes idle.
#include "float_types.cuh"

namespace echo {

constexpr int HT = 256;          // threads per workgroup

struct HeadSide {                // the query or the key side
  const void *x;
  void *y;
  int64_t xt, xh, yt, yh;        // strides of tokens and heads, in elements
  const float *weight, *bias;
  int32_t heads, norm;
  uint32_t chunks;               // waves per token; 0: a load takes several tokens
  int32_t across;                // heads of a token in one load, a power of two, where chunks is 0
};
struct Fp8Side {                 // what the FP8 form writes
  const float *w;
  int64_t wt;
  float w_mul;
  uint8_t *q8;
  float *w_out;
  uint8_t *k_cache;
  float *k_scale;
  const int64_t *slot;
  int64_t n_slots;
};
struct HeadArgs {
  HeadSide side[2];
  Fp8Side f;
  const int32_t *pos;
  const float *cos_sin;
  int32_t n_tok, dim, rot_begin, rot, n_pos;
  uint32_t waves[2];             // of each side
  float eps;
};

// Eight floats; the table's and the weights' rows are 16-byte aligned (checked by the host).
ECHO_DEV void load_f8(const float *__restrict__ p, float (&v)[VEC]) {
  const f32x4 a = reinterpret_cast<const f32x4 *>(p)[0], b = reinterpret_cast<const f32x4 *>(p)[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
}

// One wave's rows of side s.  ONE: heads of one token, HU loads of 64 / G; otherwise HU loads of
// several tokens' heads.
template <typename T, int G, bool FP8, bool NEXT, int HU, bool ONE>
ECHO_DEV void heads_wave(const HeadArgs &a, const HeadSide &s, bool is_k, uint32_t wave) {
  constexpr int ROWS = 64 / G;                       // rows of one load
  const int l = lane_id(), sub = l / G, j = l % G;
  const bool in_row = j * VEC < a.dim;

  // this lane's place in the rotation
  const int e = j * VEC - a.rot_begin, half = a.rot >> 1;
  const bool turns = in_row && e >= 0 && e < a.rot;
  const bool second = !NEXT && e >= half;
  const int angle = NEXT ? e >> 1 : (second ? e - half : e);
  const int mate = turns && !NEXT ? l + (second ? -(half / VEC) : half / VEC) : l;

  // its tokens and heads: token tok + u * tok_step, head head + u * head_step
  int32_t tok, head, tok_step, head_step;
  if (ONE) {
    tok = static_cast<int32_t>(wave / s.chunks);
    head = static_cast<int32_t>(wave - tok * s.chunks) * (HU * ROWS) + sub;
    tok_step = 0;
    head_step = ROWS;
  } else {
    tok_step = ROWS / s.across;
    tok = static_cast<int32_t>(wave) * HU * tok_step + sub / s.across;
    head = sub % s.across;
    head_step = 0;
  }
  Raw8<T> raw[HU];
  int32_t pos[HU];
  bool live[HU];
  float w[HU];                                       // FP8: the head's weight, or the key's row
  int64_t slot[HU];
#pragma unroll
  for (int u = 0; u < HU; ++u) {
    const int32_t t = tok + u * tok_step, h = head + u * head_step;
    const bool in = t < a.n_tok && h < s.heads;
    pos[u] = ONE ? a.pos[t] : in ? a.pos[t] : -1;
    raw[u] = in && in_row ? load8(static_cast<const T *>(s.x) + t * s.xt + (h * s.xh + j * VEC)) : zero8<T>();
    live[u] = in && pos[u] >= 0 && pos[u] < a.n_pos;
    if (FP8) {                                       // here, or each would be one more round trip at the end
      w[u] = in && !is_k ? a.f.w[t * a.f.wt + h] : 0.f;
      slot[u] = in && is_k ? a.f.slot[t] : -1;
    }
  }
  float wt[VEC], bi[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) { wt[i] = 1.f; bi[i] = 0.f; }
  if (s.norm != ECHO_NORM_NONE && in_row) {
    if (s.weight) load_f8(s.weight + j * VEC, wt);
    if (s.bias) load_f8(s.bias + j * VEC, bi);
  }
  float c[VEC], d[VEC];                              // cosines and sines of the lane's angles
#pragma unroll
  for (int u = 0; u < HU; ++u) {
    if (u == 0 || !ONE) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) { c[i] = 1.f; d[i] = 0.f; }
      if (turns && (ONE ? pos[u] >= 0 && pos[u] < a.n_pos : live[u])) {
        const float *cs = a.cos_sin + static_cast<int64_t>(pos[u]) * a.rot + angle;
        if (NEXT) {
          const f32x4 cv = *reinterpret_cast<const f32x4 *>(cs), sv = *reinterpret_cast<const f32x4 *>(cs + half);
#pragma unroll
          for (int i = 0; i < 4; ++i) { c[i] = cv[i]; d[i] = sv[i]; }
        } else {
          load_f8(cs, c);
          load_f8(cs + half, d);
#pragma unroll
          for (int i = 0; i < VEC; ++i) d[i] = second ? d[i] : -d[i];
        }
      }
    }
    float x[VEC];
    unpack8(raw[u], x);
    if (s.norm != ECHO_NORM_NONE) {                  // uniform over the workgroup
      float mean = 0.f;
      if (s.norm == ECHO_NORM_LAYER) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) t += x[i];
        mean = group_sum<G>(t) / static_cast<float>(a.dim);
      }
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        x[i] = in_row ? x[i] - mean : 0.f;
        t = fmaf(x[i], x[i], t);
      }
      const float r = 1.f / sqrtf(group_sum<G>(t) / static_cast<float>(a.dim) + a.eps);
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = fmaf(x[i] * r, wt[i], bi[i]);
    }
    if (NEXT) {
      if (turns) {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const float p = x[i], q = x[i + 1];
          x[i] = p * c[i / 2] - q * d[i / 2];
          x[i + 1] = q * c[i / 2] + p * d[i / 2];
        }
      }
    } else if (a.rot) {                              // uniform: the lanes exchange
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float p = __shfl(x[i], mate, 64);
        if (turns) x[i] = x[i] * c[i] + p * d[i];
      }
    }
    Fp8Scale sc = {};
    u32x2 code = {0, 0};
    if (FP8) {                                       // by all lanes, live or not
      sc = fp8_scale<sizeof(T) == 4>(group_amax<G>(x));
      code = quantise8<sizeof(T) == 4>(x, sc);
    }
    if (!live[u]) continue;
    const int32_t t = tok + u * tok_step, h = head + u * head_step;
    if (!FP8) {
      if (in_row) store8(static_cast<T *>(s.y) + t * s.yt + (h * s.yh + j * VEC), x);
      continue;
    }
    if (!is_k) {
      const int64_t row = static_cast<int64_t>(t) * s.heads + h;
      // 8 bytes a lane: past the caches a prefill chunk's codes leave faster (32768 tokens: 163 us with
      // plain stores where these took 157; 1400 tokens 13.2 and 11.6)
      __builtin_nontemporal_store(code, reinterpret_cast<u32x2 *>(a.f.q8 + row * D + j * VEC));
      if (j == 0) a.f.w_out[row] = w[u] * sc.scale * a.f.w_mul;
    } else {
      if (slot[u] < 0 || slot[u] >= a.f.n_slots) continue;
      *reinterpret_cast<u32x2 *>(a.f.k_cache + slot[u] * D + j * VEC) = code;
      if (j == 0) a.f.k_scale[slot[u]] = sc.scale;
    }
  }
}

// Waves of the query side first, then those of the key side.
template <typename T, int G, bool FP8, bool NEXT, int HU>
__global__ __launch_bounds__(HT) void heads_kernel(HeadArgs a) {
  const uint32_t id = blockIdx.x * (HT / 64) + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const bool is_k = id >= a.waves[0];
  const uint32_t wave = is_k ? id - a.waves[0] : id;
  if (is_k && wave >= a.waves[1]) return;
  const HeadSide &s = a.side[is_k ? 1 : 0];
  if (s.chunks) heads_wave<T, G, FP8, NEXT, HU, true>(a, s, is_k, wave);
  else heads_wave<T, G, FP8, NEXT, HU, false>(a, s, is_k, wave);
}

template <typename T, int G, bool FP8, int HU>
static void launch_heads_u(const HeadArgs &a, bool next, uint32_t grid, hipStream_t st) {
  if (next)
    heads_kernel<T, G, FP8, true, HU><<<grid, HT, 0, st>>>(a);
  else
    heads_kernel<T, G, FP8, false, HU><<<grid, HT, 0, st>>>(a);
}
template <typename T, int G, bool FP8>
static void launch_heads_g(const HeadArgs &a, int loads, bool next, uint32_t grid, hipStream_t st) {
  if (loads == 1) launch_heads_u<T, G, FP8, 1>(a, next, grid, st);
  else if (loads == 2) launch_heads_u<T, G, FP8, 2>(a, next, grid, st);
  else launch_heads_u<T, G, FP8, 4>(a, next, grid, st);
}

// Shares a side's rows out to waves; returns their number.
static uint32_t side_waves(HeadSide &s, int64_t n_tok, int g, int loads) {
  const int rows = 64 / g;
  if (s.heads == 0) return 0;
  if (s.heads >= rows) {
    s.chunks = static_cast<uint32_t>((s.heads + loads * rows - 1) / (loads * rows));
    return static_cast<uint32_t>(n_tok * s.chunks);
  }
  s.chunks = 0;
  s.across = 1;
  while (s.across < s.heads) s.across *= 2;
  const int64_t per = static_cast<int64_t>(loads) * (rows / s.across);
  return static_cast<uint32_t>((n_tok + per - 1) / per);
}

template <typename T, bool FP8>
static int launch_heads(HeadArgs &a, bool next, hipStream_t st) {
  int g = 2;
  while (g * VEC < a.dim) g *= 2;
  // Several loads a wave, for their common angles and weights, where there are waves enough and few
  // of their loads are of nothing; fewer rows are over sooner spread thin.  On MI355X in us with one,
  // two and four: indexer inputs of 64 tokens 4.9, 4.9, 6.6 a call, of 1400 12.5, 11.6, 13.0, of 8192 54,
  // 47, 45, of 32768 201, 170, 157 (before scales without divisions, which take 5 off the last); 8191
  // tokens of 40 + 5 heads 41.3, 35.2, 38.7 (a quarter of four are of nothing); 5384 tokens of 4 + 2 heads
  // of 256 10.1, 10.8, 14.6 (a quarter of two, five eighths of four).
  const auto share = [&](int loads) {
    for (int i = 0; i < 2; ++i) a.waves[i] = side_waves(a.side[i], a.n_tok, g, loads);
    return static_cast<uint64_t>(a.waves[0]) + a.waves[1];
  };
  const uint64_t single = share(1);
  const auto full = [&](int loads) { return 8 * single >= 7 * loads * share(loads); };
  int loads = 1;
  if (single >= 1u << 16 && (full(4) || single >= 1u << 25)) loads = 4;
  else if (single >= 1u << 13 && full(2)) loads = 2;
  else share(1);
  if (static_cast<uint64_t>(a.waves[0]) + a.waves[1] >= (1u << 26))
    return fail(ECHO_EUNSUPPORTED, "qk heads: more waves than a launch holds (2^26)");
  const uint32_t grid = static_cast<uint32_t>((static_cast<uint64_t>(a.waves[0]) + a.waves[1] + HT / 64 - 1) / (HT / 64));
  if (FP8) {
    launch_heads_g<T, 16, FP8>(a, loads, next, grid, st);
  } else {
    switch (g) {
      case 2: launch_heads_g<T, 2, false>(a, loads, next, grid, st); break;
      case 4: launch_heads_g<T, 4, false>(a, loads, next, grid, st); break;
      case 8: launch_heads_g<T, 8, false>(a, loads, next, grid, st); break;
      case 16: launch_heads_g<T, 16, false>(a, loads, next, grid, st); break;
      default: launch_heads_g<T, 32, false>(a, loads, next, grid, st); break;
    }
  }
  return check_launch("qk heads");
}

template <bool FP8>
static int launch_typed(const echo_qk_args *q, HeadArgs &a, hipStream_t st) {
  const bool next = q->interleaved != 0;
  switch (q->type) {
    case ECHO_BF16: return launch_heads<bf16_t, FP8>(a, next, st);
    case ECHO_FP16: return launch_heads<fp16_t, FP8>(a, next, st);
    default: return launch_heads<float, FP8>(a, next, st);
  }
}

static bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// The checks both entry points share; *empty is set for a call with nothing to do.
static int check_heads(const char *fn, const echo_qk_args *q, bool *empty) {
  *empty = false;
  if (!q) return fail(ECHO_EINVAL, "%s: NULL args", fn);
  if (q->n_tok < 0 || q->n_q_heads < 0 || q->n_k_heads < 0 || q->n_pos < 0 || q->rot_begin < 0 || q->rot_dim < 0)
    return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (q->type != ECHO_BF16 && q->type != ECHO_FP16 && q->type != ECHO_FP32)
    return fail(ECHO_EINVAL, "%s: type %d", fn, q->type);
  for (int32_t n : {q->q_norm, q->k_norm})
    if (n != ECHO_NORM_NONE && n != ECHO_NORM_RMS && n != ECHO_NORM_LAYER)
      return fail(ECHO_EINVAL, "%s: norm %d", fn, n);
  if (q->head_dim < 8 || q->head_dim > 256 || q->head_dim % 8)
    return fail(ECHO_EUNSUPPORTED, "%s: head_dim %d is not a multiple of 8 in [8, 256]", fn, q->head_dim);
  if (q->rot_dim % 16 || q->rot_begin % 8)
    return fail(ECHO_EUNSUPPORTED, "%s: rot_dim %d / rot_begin %d are not multiples of 16 / 8", fn, q->rot_dim, q->rot_begin);
  if (q->rot_dim > q->head_dim || q->rot_begin > q->head_dim - q->rot_dim)
    return fail(ECHO_EINVAL, "%s: the rotated part ends behind the head", fn);
  if (!(q->eps >= 0.f)) return fail(ECHO_EINVAL, "%s: eps below 0", fn);
  if (q->n_tok == 0 || (q->n_q_heads == 0 && q->n_k_heads == 0)) { *empty = true; return ECHO_OK; }
  if (!q->pos || (q->n_q_heads && !q->q) || (q->n_k_heads && !q->k) || (q->rot_dim && q->n_pos && !q->cos_sin))
    return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  const int64_t most = 0x7FFFFFFF - 65536;
  if (static_cast<int64_t>(q->n_tok) * q->n_q_heads > most || static_cast<int64_t>(q->n_tok) * q->n_k_heads > most)
    return fail(ECHO_EUNSUPPORTED, "%s: more than 2^31 - 2^16 heads in all", fn);
  if (misaligned(q->pos, 4)) return fail(ECHO_EINVAL, "%s: pos is not aligned to its type", fn);
  const int64_t vec = q->type == ECHO_FP32 ? 4 : 8;                 // elements in 16 bytes
  if (misaligned(q->q_weight, 16) || misaligned(q->q_bias, 16) || misaligned(q->k_weight, 16) ||
      misaligned(q->k_bias, 16) || misaligned(q->cos_sin, 16) ||
      (q->n_q_heads && (misaligned(q->q, 16) || q->q_tok_stride % vec || q->q_head_stride % vec)) ||
      (q->n_k_heads && (misaligned(q->k, 16) || q->k_tok_stride % vec || q->k_head_stride % vec)))
    return fail(ECHO_EUNSUPPORTED, "%s: a pointer or stride is not a multiple of 16 bytes", fn);
  return ECHO_OK;
}

static HeadArgs head_args(const echo_qk_args *q) {
  HeadArgs a = {};
  a.side[0] = HeadSide{q->q, nullptr, q->q_tok_stride, q->q_head_stride, 0, 0, q->q_weight, q->q_bias, q->n_q_heads, q->q_norm, 0, 1};
  a.side[1] = HeadSide{q->k, nullptr, q->k_tok_stride, q->k_head_stride, 0, 0, q->k_weight, q->k_bias, q->n_k_heads, q->k_norm, 0, 1};
  a.pos = q->pos;
  a.cos_sin = q->cos_sin;
  a.n_tok = q->n_tok;
  a.dim = q->head_dim;
  a.rot_begin = q->rot_begin;
  a.rot = q->rot_dim;
  a.n_pos = q->n_pos;
  a.eps = q->eps;
  return a;
}

}  // namespace echo

using namespace echo;

extern "C" int echo_qk_norm_rope(const echo_qk_args *q, void *q_out, int64_t qo_tok_stride, int64_t qo_head_stride,
                                 void *k_out, int64_t ko_tok_stride, int64_t ko_head_stride, void *stream) {
  bool empty;
  const int rc = check_heads("echo_qk_norm_rope", q, &empty);
  if (rc != ECHO_OK || empty) return rc;
  if ((q->n_q_heads && !q_out) || (q->n_k_heads && !k_out)) return fail(ECHO_EINVAL, "echo_qk_norm_rope: NULL output");
  const int64_t vec = q->type == ECHO_FP32 ? 4 : 8;
  if ((q->n_q_heads && (misaligned(q_out, 16) || qo_tok_stride % vec || qo_head_stride % vec)) ||
      (q->n_k_heads && (misaligned(k_out, 16) || ko_tok_stride % vec || ko_head_stride % vec)))
    return fail(ECHO_EUNSUPPORTED, "echo_qk_norm_rope: an output or its stride is not a multiple of 16 bytes");
  const auto overlaps = [&](int32_t heads, int64_t tok, int64_t head) {
    return heads > 0 && rows_overlap(q->n_tok, tok, heads, head, q->head_dim);
  };
  if (overlaps(q->n_q_heads, qo_tok_stride, qo_head_stride))
    return fail(ECHO_EINVAL, "echo_qk_norm_rope: the heads of q_out overlap");
  if (overlaps(q->n_k_heads, ko_tok_stride, ko_head_stride))
    return fail(ECHO_EINVAL, "echo_qk_norm_rope: the heads of k_out overlap");
  HeadArgs a = head_args(q);
  a.side[0].y = q_out; a.side[0].yt = qo_tok_stride; a.side[0].yh = qo_head_stride;
  a.side[1].y = k_out; a.side[1].yt = ko_tok_stride; a.side[1].yh = ko_head_stride;
  return launch_typed<false>(q, a, S(stream));
}

extern "C" int echo_indexer_qk(const echo_qk_args *q, const float *w, int64_t w_tok_stride, float w_mul, uint8_t *q8,
                               float *w_out, uint8_t *k_cache, float *k_scale, const int64_t *slot, int64_t n_slots,
                               void *stream) {
  bool empty;
  const int rc = check_heads("echo_indexer_qk", q, &empty);
  if (rc != ECHO_OK) return rc;
  if (q->head_dim != D) return fail(ECHO_EUNSUPPORTED, "echo_indexer_qk: head_dim %d is not %d", q->head_dim, D);
  if (q->n_k_heads > 1) return fail(ECHO_EUNSUPPORTED, "echo_indexer_qk: %d key heads; a token has one key", q->n_k_heads);
  if (n_slots < 0) return fail(ECHO_EINVAL, "echo_indexer_qk: negative size");
  if (empty) return ECHO_OK;
  if ((q->n_q_heads && (!w || !q8 || !w_out)) || (q->n_k_heads && ((n_slots && (!k_cache || !k_scale)) || !slot)))
    return fail(ECHO_EINVAL, "echo_indexer_qk: NULL pointer");
  if (misaligned(q8, 8) || misaligned(k_cache, 8))
    return fail(ECHO_EUNSUPPORTED, "echo_indexer_qk: q8 or k_cache is not 8-byte aligned");
  if (misaligned(w, 4) || misaligned(w_out, 4) || misaligned(k_scale, 4) || misaligned(slot, 8))
    return fail(ECHO_EINVAL, "echo_indexer_qk: a pointer is not aligned to its type");
  HeadArgs a = head_args(q);
  a.f = Fp8Side{w, w_tok_stride, w_mul, q8, w_out, k_cache, k_scale, slot, n_slots};
  return launch_typed<true>(q, a, S(stream));
}
