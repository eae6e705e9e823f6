// Blocks of a row's tokens that its scores select (echo_block_topk): a block's score is the largest of
// its tokens' scores; the row's first and last blocks may be kept whatever they score.
//
// Reading the scores is all there is to it: a wave takes 1024 of them at a time in four loads, and the
// lanes of a block are joined with moves between lanes.  The blocks' scores, a 16th of the row or less, are selected
// from by one wave, in the same launch where a workgroup takes a row, or, above 512, by the exact top-k of
// topk.hip.  On MI355X 4096 rows of 65536 scores (0.8 GB by their lengths) with blocks of 128 take 139 us = 5.8 TB/s, 4 rows of
// 8192 4.6 us, a launch.  One load a wave, as at first, took 242 us for the maxima alone.
#include <algorithm>

#include "float_types.cuh"
#include "internal.hpp"

namespace echo {

typedef f32x4 f32x4_any __attribute__((aligned(4)));
struct OpMaxF {
  ECHO_DEV uint32_t operator()(uint32_t a, uint32_t b) const {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
};

// The blocks of 1024 tokens from u * 1024 on, or, where blocks are larger, block u, by one wave; four loads on their way.
constexpr int SPAN = 1024;
template <int G, typename S>                               // lanes of a block, 64 for blocks of 256 and more
ECHO_DEV void span_max(const float *row, int32_t n, int32_t block, int32_t u, const S &store) {
  const int32_t span = max(block, SPAN), l = lane_id();
  const int64_t t0 = static_cast<int64_t>(u) * span;
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};             // of the four 256ths
  for (int64_t t = t0 + 4 * l; t < t0 + span; t += SPAN) {
    if (t - 4 * l + SPAN <= n) {
      f32x4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const f32x4_any *>(row + t + 256 * i);
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], fmaxf(fmaxf(v[i][0], v[i][1]), fmaxf(v[i][2], v[i][3])));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        for (int64_t e = t + 256 * i; e < min<int64_t>(n, t + 256 * i + 4); ++e) m[i] = fmaxf(m[i], row[e]);
    }
  }
  if (G < 64) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = __uint_as_float(group_reduce<G < 32 ? G : 32>(__float_as_uint(m[i]), OpMaxF{}));
      if (l % G == 0) store((4 * u + i) * (64 / G) + l / G, v);
    }
  } else {                                                 // 4, 2 or 1 blocks
    if (block > 256) { m[0] = fmaxf(m[0], m[1]); m[2] = fmaxf(m[2], m[3]); }
    if (block > 512) m[0] = fmaxf(m[0], m[2]);
    const int32_t step = min(block, SPAN) / 256;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = __uint_as_float(group_reduce<32>(__float_as_uint(m[i]), OpMaxF{}));
      v = fmaxf(v, __shfl_xor(v, 32, 64));
      if (l == 0 && i % step == 0) store((4 * u + i) / step, v);
    }
  }
}

// The k highest of n <= 64 V blocks' scores by one wave: the k-th highest key bit by bit, each bit a count of the
// keys that are not below (a ballot for 64 of them, no waits), then the blocks above it and the first of those that
// equal it, in order.
template <int V>
ECHO_DEV void select(const float *pooled, int32_t n, int32_t k, int32_t *out) {
  const int32_t l = lane_id();
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = 64 * v + l < n ? f32_key(pooled[64 * v + l]) : 0u;    // a score's key is above 0
  const auto number = [](uint64_t m) { return static_cast<int32_t>(__popcll(m)); };
  const auto at_least = [&](uint32_t x) {
    int32_t c = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) c += number(__ballot(key[v] >= x));
    return c;
  };
  uint32_t least = 1;                                      // of the keys taken
  int32_t ties = n;                                        // how many that equal it are
  if (n > k) {
    least = 0;
    int32_t have = n;
    for (uint32_t bit = 1u << 31; bit && have != k; bit >>= 1) {
      const int32_t c = at_least(least | bit);
      if (c >= k) { least |= bit; have = c; }
    }
    if (have != k) ties = k - (least == ~0u ? 0 : at_least(least + 1));
  }
  const uint64_t below = (1ull << l) - 1;
  int32_t pos = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint64_t eq = __ballot(key[v] == least);
    const bool take = key[v] > least || (key[v] == least && number(eq & below) < ties);
    const uint64_t all = __ballot(take);
    if (take) out[pos + number(all & below)] = 64 * v + l;
    ties -= number(eq);
    pos += number(all);
  }
  for (int32_t j = pos + l; j < k; j += 64) out[j] = -1;
}

struct BlockArgs {
  const float *scores;
  int64_t ld;
  const int32_t *len;
  int32_t n_rows, max_len, block, n_blocks, n_first, n_last, k;
  ECHO_DEV int32_t length(int32_t r) const { return max(0, min(len[r], max_len)); }
  ECHO_DEV int32_t blocks(int32_t n) const { return static_cast<int32_t>((static_cast<int64_t>(n) + block - 1) / block); }
  ECHO_DEV bool kept(int32_t b, int32_t nb) const { return b < n_first || b >= nb - n_last; }
};

// One launch: a workgroup a row, its blocks' scores in LDS, selected from by the first wave.
constexpr int ROW_WAVES = 8, ROW_BLOCKS = 512;
template <int G>
__global__ __launch_bounds__(ROW_WAVES * 64) void block_row_kernel(BlockArgs x, int32_t *__restrict__ idx) {
  __shared__ float pooled[ROW_BLOCKS];
  const int32_t r = blockIdx.x, n = x.length(r), nb = x.blocks(n), span = max(x.block, SPAN);
  const int32_t wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int32_t spans = static_cast<int32_t>((static_cast<int64_t>(n) + span - 1) / span);
  for (int32_t u = wv; u < spans; u += ROW_WAVES)
    span_max<G>(x.scores + r * x.ld, n, x.block, u, [&](int32_t b, float v) { if (b < nb) pooled[b] = x.kept(b, nb) ? INFINITY : v; });
  __syncthreads();
  if (wv) return;
  int32_t *out = idx + static_cast<int64_t>(r) * x.k;
  if (nb <= 128) select<2>(pooled, nb, x.k, out);
  else select<ROW_BLOCKS / 64>(pooled, nb, x.k, out);
}

// Two launches: the blocks' scores to memory, a wave a span, then the selection, a wave a row or topk.hip's.
template <int G>
__global__ __launch_bounds__(256) void block_max_kernel(BlockArgs x, int64_t waves, int32_t per_row, float *__restrict__ pooled, int32_t *__restrict__ count) {
  const int64_t wave = blockIdx.x * 4ll + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  if (wave >= waves) return;
  const int32_t r = static_cast<int32_t>(wave / per_row), u = static_cast<int32_t>(wave - static_cast<int64_t>(r) * per_row);
  const int32_t n = x.length(r), nb = x.blocks(n);
  if (u == 0 && lane_id() == 0) count[r] = nb;
  if (static_cast<int64_t>(u) * max(x.block, SPAN) >= n) return;
  float *out = pooled + static_cast<int64_t>(r) * x.n_blocks;
  span_max<G>(x.scores + r * x.ld, n, x.block, u, [&](int32_t b, float v) { if (b < nb) out[b] = x.kept(b, nb) ? INFINITY : v; });
}
__global__ __launch_bounds__(256) void block_select_kernel(const float *__restrict__ pooled, int32_t n_blocks, const int32_t *__restrict__ count,
                                                           int32_t n_rows, int32_t k, int32_t *__restrict__ idx) {
  const int32_t r = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  if (r < n_rows) select<ROW_BLOCKS / 64>(pooled + static_cast<int64_t>(r) * n_blocks, count[r], k, idx + static_cast<int64_t>(r) * k);
}

template <int G>
int launch(const BlockArgs &x, bool one, int64_t waves, int32_t per_row, float *pooled, int32_t *count, int32_t *idx, hipStream_t st) {
  if (one) block_row_kernel<G><<<x.n_rows, ROW_WAVES * 64, 0, st>>>(x, idx);
  else block_max_kernel<G><<<static_cast<uint32_t>((waves + 3) / 4), 256, 0, st>>>(x, waves, per_row, pooled, count);
  return check_launch("block maxima");
}

}  // namespace echo

using namespace echo;

static int64_t blocks_in(int32_t max_len, int32_t block) { return (static_cast<int64_t>(max_len) + block - 1) / block; }

extern "C" size_t echo_block_topk_workspace_bytes(int32_t n_rows, int32_t max_len, int32_t block) {
  if (n_rows < 1 || max_len < 0 || block < 1) return 0;
  return static_cast<size_t>(n_rows) * 4 * static_cast<size_t>(blocks_in(max_len, block) + 1);
}

extern "C" int echo_block_topk(const float *scores, int64_t ld, const int32_t *len, int32_t n_rows, int32_t max_len, int32_t block, int32_t n_first,
                               int32_t n_last, int32_t k, int32_t *idx, void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "echo_block_topk";
  if (n_rows < 0 || max_len < 0 || n_first < 0 || n_last < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (block < 16 || block > 65536 || (block & (block - 1)))
    return fail(ECHO_EUNSUPPORTED, "%s: block %d is not a power of two in [16, 65536]", fn, block);
  if (k < 1 || k > ECHO_MAX_TOPK) return fail(ECHO_EUNSUPPORTED, "%s: k %d outside [1, %d]", fn, k, ECHO_MAX_TOPK);
  if (ld < max_len) return fail(ECHO_EINVAL, "%s: ld < max_len", fn);
  if (n_rows == 0) return ECHO_OK;
  if ((max_len && !scores) || !len || !idx) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if ((reinterpret_cast<uintptr_t>(scores) | reinterpret_cast<uintptr_t>(len) | reinterpret_cast<uintptr_t>(idx)) % 4)
    return fail(ECHO_EINVAL, "%s: an array is not aligned to its type", fn);
  const int32_t n_blocks = static_cast<int32_t>(blocks_in(max_len, block)), span = std::max(block, SPAN);
  const int32_t per_row = std::max<int32_t>(1, static_cast<int32_t>(blocks_in(max_len, span)));
  const int64_t waves = static_cast<int64_t>(n_rows) * per_row;
  if (waves >= 1 << 26 || n_rows >= 1 << 22) return fail(ECHO_EUNSUPPORTED, "%s: more rows and tokens than a launch holds", fn);
  const size_t need = echo_block_topk_workspace_bytes(n_rows, max_len, block);
  if (!ws || ws_bytes < need) return fail(ECHO_EWORKSPACE, "%s: a workspace of %zu bytes is needed", fn, need);
  if (reinterpret_cast<uintptr_t>(ws) % 4) return fail(ECHO_EINVAL, "%s: the workspace is not aligned to its type", fn);
  float *pooled = static_cast<float *>(ws);
  int32_t *count = reinterpret_cast<int32_t *>(pooled + static_cast<int64_t>(n_rows) * n_blocks);
  const hipStream_t st = S(stream);
  const BlockArgs x = {scores, ld, len, n_rows, max_len, block, n_blocks, n_first, n_last, k};
  // One launch for rows that a workgroup reads fast enough, or as many rows as fill the card.  Measured on MI355X (us, in
  // one launch and in two): 4 rows of 8192 4.6 and 7.1, 1 of 32768 7.7 and 9.2, 256 of 65536 15.7 and 19.0, 4096 of 65536 139 and
  // 148; 64 of 65536 13.8 and 13.1, 4096 of 8192 27.4 and 26.2.
  const bool one = n_blocks <= ROW_BLOCKS && (max_len <= 65536 || n_rows >= 512);
  const auto go = block == 16 ? launch<4> : block == 32 ? launch<8> : block == 64 ? launch<16> : block == 128 ? launch<32> : launch<64>;
  const int rc = go(x, one, waves, per_row, pooled, count, idx, st);
  if (rc != ECHO_OK || one) return rc;
  // 512 blocks of 1 row 9.0 us, 14.4 with topk.hip's; 1024 16.4 and 15.0, 2048 of 64 rows 29 and 22.5.
  if (n_blocks > ROW_BLOCKS) return launch_topk_rows(pooled, n_blocks, count, n_rows, n_blocks, k, nullptr, idx, st);
  block_select_kernel<<<(n_rows + 3) / 4, 256, 0, st>>>(pooled, n_blocks, count, n_rows, k, idx);
  return check_launch("block selection");
}
