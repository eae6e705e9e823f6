// Blocks of a row's tokens that its scores select (echo_block_topk): a block's score is the largest of
// its tokens' scores; the row's first and last blocks may be kept whatever they score.
//
// Reading the scores is all there is to it: a wave takes 256 of them at a time, 4 a lane, and the
// lanes of a block are joined with moves between lanes.  The blocks' scores, a 16th of the row or less, go through
// the exact top-k of topk.hip.
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

// One wave per 256 tokens of a row, or per block where blocks are larger.
template <int G>                                           // lanes of a block, 64 for blocks of 256 and more
__global__ __launch_bounds__(256) void block_max_kernel(const float *__restrict__ scores, int64_t ld, const int32_t *__restrict__ len,
                                                        int64_t waves, int32_t per_row, int32_t max_len, int32_t block, int32_t n_blocks,
                                                        int32_t n_first, int32_t n_last, float *__restrict__ pooled, int32_t *__restrict__ count) {
  const int64_t wave = blockIdx.x * 4ll + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  if (wave >= waves) return;
  const int32_t r = static_cast<int32_t>(wave / per_row), u = static_cast<int32_t>(wave - static_cast<int64_t>(r) * per_row);
  const int32_t n = max(0, min(len[r], max_len)), l = lane_id();
  const int32_t nb = static_cast<int32_t>((static_cast<int64_t>(n) + block - 1) / block);
  if (u == 0 && l == 0) count[r] = nb;
  const int32_t span = max(block, 256);
  const int64_t t0 = static_cast<int64_t>(u) * span;
  if (t0 >= n) return;
  const float *row = scores + r * ld;
  float m = -INFINITY;
  for (int32_t i = 4 * l; i < span; i += 256) {
    const int64_t t = t0 + i;
    if (t + 4 <= n) {
      const f32x4 v = *reinterpret_cast<const f32x4_any *>(row + t);
      m = fmaxf(m, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
    } else {
      for (int64_t e = t; e < n; ++e) m = fmaxf(m, row[e]);
    }
  }
  m = __uint_as_float(group_reduce<G < 32 ? G : 32>(__float_as_uint(m), OpMaxF{}));
  if (G == 64) m = fmaxf(m, __shfl_xor(m, 32, 64));
  const int32_t b = G == 64 ? u : u * (64 / G) + l / G;
  if (l % G == 0 && b < nb) pooled[static_cast<int64_t>(r) * n_blocks + b] = b < n_first || b >= nb - n_last ? INFINITY : m;
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
  const int32_t n_blocks = static_cast<int32_t>(blocks_in(max_len, block)), span = std::max(block, 256);
  const int32_t per_row = std::max<int32_t>(1, static_cast<int32_t>(blocks_in(max_len, span)));
  const int64_t waves = static_cast<int64_t>(n_rows) * per_row;
  if (waves >= 1 << 26 || n_rows >= 1 << 22) return fail(ECHO_EUNSUPPORTED, "%s: more rows and tokens than a launch holds", fn);
  const size_t need = echo_block_topk_workspace_bytes(n_rows, max_len, block);
  if (!ws || ws_bytes < need) return fail(ECHO_EWORKSPACE, "%s: a workspace of %zu bytes is needed", fn, need);
  if (reinterpret_cast<uintptr_t>(ws) % 4) return fail(ECHO_EINVAL, "%s: the workspace is not aligned to its type", fn);
  float *pooled = static_cast<float *>(ws);
  int32_t *count = reinterpret_cast<int32_t *>(pooled + static_cast<int64_t>(n_rows) * n_blocks);
  const uint32_t grid = static_cast<uint32_t>((waves + 3) / 4);
  const hipStream_t st = S(stream);
#define RUN(G) block_max_kernel<G><<<grid, 256, 0, st>>>(scores, ld, len, waves, per_row, max_len, block, n_blocks, n_first, n_last, pooled, count)
  switch (block) {
    case 16: RUN(4); break;
    case 32: RUN(8); break;
    case 64: RUN(16); break;
    case 128: RUN(32); break;
    default: RUN(64); break;
  }
#undef RUN
  const int rc = check_launch("block maxima");
  if (rc != ECHO_OK) return rc;
  return launch_topk_rows(pooled, n_blocks, count, n_rows, n_blocks, k, nullptr, idx, st);
}
