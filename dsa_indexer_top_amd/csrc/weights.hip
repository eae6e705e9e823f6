// What each listed token got in an attention that has run (echo_attention_weights), and its way into
// the pool's eviction order (echo_pool_weigh).
//
//   w[r][t] = sum_h exp(scale * q[r][h] . row_t - lse[r][h])
//
// A workgroup takes 64 or 128 tokens of one query row, a quarter a wave, whose 576 values stay in registers, and goes through
// the heads in tiles of 16 that it stages in LDS: each cache row is read once for all heads, and the sum
// over the heads ends in the workgroup.  The product runs on the matrix core as in attention.hip; its
// result's columns are heads, so a lane adds up its own head's weights and the 16 lanes are joined at the end.
// Measured on MI355X: 64 rows x 16 heads x 2048 tokens 27 us = 5.6 TB/s of rows, what reading them takes; 64 x 128 x 2048 44
// us, where the heads' reads from LDS (1 KB for two products) bound it; 1 x 16 x 2048 5.0 us.
#include <algorithm>

#include "latent.cuh"

namespace echo {

constexpr int KSTEPS = LATENT / 32, WAVES = 4;

struct WeightArgs {
  LatentArgs a;
  const float *lse;
  float *w;
  int64_t w_ld;
  int32_t chunks;
};

constexpr int QROPE = 16 * 1024, QSTAGE = 16 * LATENT * 2;
ECHO_DEV constexpr int swap_v(int row) { return ((row & 7) << 1) | ((row >> 3) & 1); }
ECHO_DEV constexpr int swap_r(int row) { return (row >> 1) & 7; }

// Heads 16 ht .. 16 ht + 15 of a row to LDS, the last one again behind the end: every wave 4 heads' first 512
// values, waves 0 and 1 the last 64 of 8 heads.
ECHO_DEV void stage_heads(const uint8_t *q, int64_t head_bytes, int32_t ht, int32_t n_heads, uint8_t *__restrict__ stage, int wv) {
  const int l = lane_id();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = wv * 4 + i;
    const uint8_t *src = q + min(ht * 16 + at, n_heads - 1) * head_bytes;
    __builtin_amdgcn_global_load_lds((glb_void *)(src + ((l ^ swap_v(at)) << 4)), (lds_void *)(stage + at * 1024), 16, 0, 0);
  }
  if (wv < 2) {
    const int at = wv * 8 + (l >> 3);
    const uint8_t *src = q + min(ht * 16 + at, n_heads - 1) * head_bytes;
    __builtin_amdgcn_global_load_lds((glb_void *)(src + 1024 + (((l & 7) ^ swap_r(at)) << 4)), (lds_void *)(stage + QROPE + wv * 1024), 16, 0, 0);
  }
}

typedef v4f v4f_any __attribute__((aligned(4)));

template <typename T, int TT>                              // 16 TT tokens a wave
__global__ __launch_bounds__(WAVES * 64, TT == 1 ? 4 : 2) void weights_kernel(WeightArgs x) {
  typedef typename Mma<T>::x8 x8;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][QSTAGE];
  const int wv = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int l = lane_id(), j = l & 15, g = l >> 4;
  const int32_t r = static_cast<int32_t>(blockIdx.x / x.chunks), c = static_cast<int32_t>(blockIdx.x % x.chunks);
  const Tokens src = x.a.tokens(r);
  const uint8_t *q = reinterpret_cast<const uint8_t *>(x.a.q + r * x.a.q_row);
  const int32_t tiles = (x.a.n_heads + 15) >> 4, t0 = (c * WAVES + wv) * TT * 16;
  stage_heads(q, x.a.q_head * 2, 0, x.a.n_heads, lds[0], wv);
  x8 k[TT][KSTEPS];
  uint32_t real[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    const int32_t t = t0 + i * 16 + j;
    const int64_t pos = t < x.a.n_tok ? src.position(t, src.entry(t)) : -1;
    const int32_t row = src.row(pos, src.page(pos));
    real[i] = (static_cast<uint32_t>(__ballot(row >= 0)) & 0xFFFFu) >> (4 * g);
    const uint16_t *p = x.a.kv + (row < 0 ? 0 : row) * x.a.kv_stride + 8 * g;
#pragma unroll
    for (int s = 0; s < KSTEPS; ++s) {
      u32x4 v = {0, 0, 0, 0};
      if (row >= 0) v = *reinterpret_cast<const u32x4 *>(p + 32 * s);
      k[i][s] = __builtin_bit_cast(x8, v);
    }
  }
  v4f sum[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) sum[i] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int32_t ht = 0; ht < tiles; ++ht) {
    uint8_t *cur = lds[ht & 1];
    const int32_t h = ht * 16 + j;
    const float less = h < x.a.n_heads ? x.lse[static_cast<int64_t>(r) * x.a.n_heads + h] * LOG2E : INFINITY;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(WAIT_VM0);
    meet();
    if (ht + 1 < tiles) stage_heads(q, x.a.q_head * 2, ht + 1, x.a.n_heads, lds[(ht + 1) & 1], wv);
    v4f s[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) s[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < KSTEPS; ++n) {
      const x8 head = n < 16 ? read16<x8>(cur + j * 1024 + (((4 * n + g) ^ swap_v(j)) << 4))
                             : read16<x8>(cur + QROPE + j * 128 + (((4 * (n - 16) + g) ^ swap_r(j)) << 4));
#pragma unroll
      for (int i = 0; i < TT; ++i) s[i] = Mma<T>::mul(k[i][n], head, s[i]);
    }
#pragma unroll
    for (int i = 0; i < TT; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) sum[i][v] += h < x.a.n_heads ? exp2_(fmaf(s[i][v], x.a.scale2, -less)) : 0.f;
  }
  // Lane (j, g): tokens 4 g .. 4 g + 3 of a tile, its own heads; all 16 lanes j get the sum.
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    v4f w;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      w[v] = group_sum<16>(sum[i][v]);
      if (!(real[i] >> v & 1)) w[v] = 0.f;
    }
    const int32_t t = t0 + i * 16 + 4 * g;
    float *out = x.w + r * x.w_ld + t;
    if (j == 0) {
      if (t + 4 <= x.a.n_tok) *reinterpret_cast<v4f_any *>(out) = w;
      else
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (t + v < x.a.n_tok) out[v] = w[v];
    }
  }
}

// ---------------------------------------------------------------- eviction order
// Weights of a slot are added up as whole numbers of 2^-32, so that the order in which they come does
// not matter; bit 63 marks a slot that the step has filled anew.
constexpr uint64_t FRESH = 1ull << 63;
constexpr float WEIGHT_MAX = 1024.f;
constexpr int64_t MAX_ENTRIES = 1 << 21;                   // 2^21 * 1024 * 2^32 = 2^63

ECHO_DEV unsigned long long units(float w) {               // a NaN counts as 0
  return static_cast<unsigned long long>(rintf(fminf(fmaxf(w, 0.f), WEIGHT_MAX) * 0x1p32f));
}
ECHO_DEV float weighed(uint64_t a, float mass, float decay) {
#pragma clang fp contract(off)
  const float old = a & FRESH ? 0.f : fmaxf(mass, 0.f) * decay;
  return old + static_cast<float>(a & ~FRESH) * 0x1p-32f;
}
ECHO_DEV void weigh(uint64_t a, int32_t i, const uint8_t *__restrict__ gpu_free, int32_t *__restrict__ priority, float *__restrict__ mass, float decay) {
  const bool is_free = gpu_free[i] != 0;
  const float m = is_free ? 0.f : weighed(a, mass[i], decay);
  mass[i] = m;
  priority[i] = is_free ? -1 : __float_as_int(m);
}

// One launch: a workgroup has `per` slots' sums in LDS and looks through every entry for theirs.
// Every workgroup reads every entry, so this is the faster way for few of either.  Measured on MI355X (us, and in three
// launches): 2048 entries on 16384 slots (32 workgroups) 3.9 and 9.0, on 2^20 slots (256) 6.2 and 11.0; 16384 on 32768 (64) 6.4 and
// 8.3; 131072 on 16384 (32) 6.5 and 8.9; 32768 on 65536 (128) 9.8 and 8.8; 65536 on 2^20 (256) 28 and 13.5.
constexpr int64_t SEARCHED = 1 << 21;                      // entries times workgroups
static_assert(256 * 16384 >= 1 << 22, "256 workgroups hold every slot");
constexpr int HELD = 16384, SEARCH = 1024, AT_ONCE = 4;
typedef int32_t i32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
__global__ __launch_bounds__(SEARCH) void weigh_search_kernel(const int32_t *__restrict__ slot, const float *__restrict__ w, int32_t n,
                                                              const int32_t *__restrict__ fresh, int32_t n_fresh, const uint8_t *__restrict__ gpu_free,
                                                              int32_t *__restrict__ priority, float *__restrict__ mass, float decay, int32_t n_gpu, int32_t per) {
  __shared__ unsigned long long acc[HELD];
  const int32_t tid = threadIdx.x, s0 = blockIdx.x * per, held = min(per, n_gpu - s0);
  for (int32_t i = tid; i < held; i += SEARCH) acc[i] = 0;
  __syncthreads();
  const auto mine = [&](int32_t s) { return static_cast<uint32_t>(s) - static_cast<uint32_t>(s0) < static_cast<uint32_t>(held); };
  for (int32_t i0 = 0; i0 < n; i0 += 4 * SEARCH * AT_ONCE) {
    i32x4_any s[AT_ONCE];
    f32x4_any v[AT_ONCE];                                  // of every entry: read one by one where needed, each is a wait
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u) {
      const int32_t i = i0 + 4 * (u * SEARCH + tid);
      if (i + 4 <= n) {
        s[u] = *reinterpret_cast<const i32x4_any *>(slot + i);
        v[u] = *reinterpret_cast<const f32x4_any *>(w + i);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[u][e] = i + e < n ? slot[i + e] : -1;
          v[u][e] = i + e < n ? w[i + e] : 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < AT_ONCE; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (mine(s[u][e])) atomicAdd(&acc[s[u][e] - s0], units(v[u][e]));
  }
  for (int32_t i = tid; i < n_fresh; i += SEARCH) {
    const int32_t s = fresh[i];
    if (mine(s)) atomicOr(&acc[s - s0], static_cast<unsigned long long>(FRESH));
  }
  __syncthreads();
  for (int32_t i = tid; i < held; i += SEARCH) weigh(acc[i], s0 + i, gpu_free, priority, mass, decay);
}

// Three launches, the sums in global memory.
typedef uint64_t u64x4_any __attribute__((ext_vector_type(4), aligned(8)));
__global__ __launch_bounds__(256) void weigh_clear_kernel(uint64_t *acc, int32_t n) {
  const int32_t i = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (i + 4 <= n) *reinterpret_cast<u64x4_any *>(acc + i) = u64x4_any{0, 0, 0, 0};
  else
    for (int32_t e = i; e < n; ++e) acc[e] = 0;
}

__global__ __launch_bounds__(256) void weigh_add_kernel(const int32_t *__restrict__ slot, const float *__restrict__ w, int32_t n,
                                                        const int32_t *__restrict__ fresh, int32_t n_fresh, unsigned long long *acc, int32_t n_gpu) {
  const int32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) {
    const int32_t s = slot[i];
    if (s >= 0 && s < n_gpu) atomicAdd(&acc[s], units(w[i]));
  } else if (i - n < n_fresh) {
    const int32_t s = fresh[i - n];
    if (s >= 0 && s < n_gpu) atomicOr(&acc[s], static_cast<unsigned long long>(FRESH));
  }
}

// Four slots a thread.
typedef uint8_t u8x4_any __attribute__((ext_vector_type(4), aligned(1)));
__global__ __launch_bounds__(256) void weigh_kernel(const uint64_t *__restrict__ acc, const uint8_t *__restrict__ gpu_free,
                                                    int32_t *__restrict__ priority, float *__restrict__ mass, float decay, int32_t n) {
  const int32_t i = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (i + 4 <= n) {
    const u64x4_any a = *reinterpret_cast<const u64x4_any *>(acc + i);
    const u8x4_any f = *reinterpret_cast<const u8x4_any *>(gpu_free + i);
    const f32x4_any m = *reinterpret_cast<const f32x4_any *>(mass + i);
    f32x4_any to;
    i32x4_any prio;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      to[e] = f[e] ? 0.f : weighed(a[e], m[e], decay);
      prio[e] = f[e] ? -1 : __float_as_int(to[e]);
    }
    *reinterpret_cast<f32x4_any *>(mass + i) = to;
    *reinterpret_cast<i32x4_any *>(priority + i) = prio;
  } else {
    for (int32_t e = i; e < n; ++e) weigh(acc[e], e, gpu_free, priority, mass, decay);
  }
}

// 16 tokens a wave have more waves on a SIMD and more workgroups, 32 read the heads from LDS half as often, which is what
// many heads of many rows wait for.  Measured on MI355X, 2048 tokens a row (us, 16 and 32): 16 heads of 1 row 5.0 and 7.1, of 256
// rows 95.8 and 97.7; 128 heads of 8 rows 12.2 and 14.1, of 64 rows 47.7 and 44.6.
template <typename T>
int launch_weights(WeightArgs x, hipStream_t st) {
  const auto chunks = [&](int tt) { return (x.a.n_tok + WAVES * tt * 16 - 1) / (WAVES * tt * 16); };
  const bool few = x.a.n_heads <= 32 || static_cast<int64_t>(x.a.n_rows) * chunks(2) <= 512;
  x.chunks = chunks(few ? 1 : 2);
  const uint32_t grid = static_cast<uint32_t>(x.a.n_rows) * static_cast<uint32_t>(x.chunks);
  if (few) weights_kernel<T, 1><<<grid, WAVES * 64, 0, st>>>(x);
  else weights_kernel<T, 2><<<grid, WAVES * 64, 0, st>>>(x);
  return check_launch("attention weights");
}

}  // namespace echo

using namespace echo;

extern "C" int echo_attention_weights(const echo_latent_args *a, const float *lse, float *w, int64_t w_stride, void *stream) {
  const char *fn = "echo_attention_weights";
  WeightArgs x = {};
  const int rc = latent_args(fn, a, &x.a);
  if (rc != ECHO_OK) return rc;
  if (w_stride < 0 || (a->n_rows > 1 && w_stride < x.a.n_tok)) return fail(ECHO_EINVAL, "%s: rows of w overlap", fn);
  if (a->n_rows == 0 || x.a.n_tok == 0) return ECHO_OK;
  if (a->n_heads == 0) return fail(ECHO_EINVAL, "%s: no heads", fn);
  if (!lse || !w) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  if (reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(w) % 4) return fail(ECHO_EINVAL, "%s: an array is not aligned to its type", fn);
  x.lse = lse; x.w = w; x.w_ld = w_stride;
  if (static_cast<int64_t>(a->n_rows) * ((x.a.n_tok + 63ll) / 64) >= 1 << 24) return fail(ECHO_EUNSUPPORTED, "%s: more rows and tokens than a launch holds", fn);
  return a->type == ECHO_BF16 ? launch_weights<bf16_t>(x, S(stream)) : launch_weights<fp16_t>(x, S(stream));
}

extern "C" size_t echo_pool_weigh_workspace_bytes(int32_t n_gpu) { return n_gpu < 1 ? 0 : static_cast<size_t>(n_gpu) * 8; }

extern "C" int echo_pool_weigh(const uint8_t *gpu_free, int32_t *gpu_priority, float *mass, int32_t n_gpu, const int32_t *slot, const float *w,
                               int64_t n_entries, const int32_t *fresh, int64_t n_fresh, float decay, void *ws, size_t ws_bytes, void *stream) {
  const char *fn = "echo_pool_weigh";
  if (n_gpu < 0 || n_entries < 0 || n_fresh < 0) return fail(ECHO_EINVAL, "%s: negative size", fn);
  if (!(decay >= 0.f && decay <= 1.f)) return fail(ECHO_EINVAL, "%s: decay outside [0, 1]", fn);
  if (n_gpu > 1 << 22 || n_entries > MAX_ENTRIES || n_fresh > MAX_ENTRIES)
    return fail(ECHO_EUNSUPPORTED, "%s: more than 2^22 slots or 2^21 entries", fn);
  if (n_gpu == 0) return ECHO_OK;
  if (!gpu_free || !gpu_priority || !mass || (n_entries && (!slot || !w)) || (n_fresh && !fresh)) return fail(ECHO_EINVAL, "%s: NULL pointer", fn);
  const uintptr_t words = reinterpret_cast<uintptr_t>(gpu_priority) | reinterpret_cast<uintptr_t>(mass) | reinterpret_cast<uintptr_t>(slot) |
                          reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(fresh);
  if (words % 4) return fail(ECHO_EINVAL, "%s: an array is not aligned to its type", fn);
  const size_t need = echo_pool_weigh_workspace_bytes(n_gpu);
  if (!ws || ws_bytes < need) return fail(ECHO_EWORKSPACE, "%s: a workspace of %zu bytes is needed", fn, need);
  if (reinterpret_cast<uintptr_t>(ws) % 8) return fail(ECHO_EINVAL, "%s: the workspace is not aligned to 8 bytes", fn);
  const hipStream_t st = S(stream);
  const int32_t per = std::max(512, (n_gpu + 255) / 256), groups = (n_gpu + per - 1) / per;
  if ((n_entries + n_fresh) * groups <= SEARCHED) {
    weigh_search_kernel<<<groups, SEARCH, 0, st>>>(slot, w, static_cast<int32_t>(n_entries), fresh, static_cast<int32_t>(n_fresh),
                                                                   gpu_free, gpu_priority, mass, decay, n_gpu, per);
    return check_launch("pool weigh");
  }
  weigh_clear_kernel<<<(n_gpu + 1023) / 1024, 256, 0, st>>>(static_cast<uint64_t *>(ws), n_gpu);
  const uint32_t n = static_cast<uint32_t>(n_entries + n_fresh);
  weigh_add_kernel<<<(n + 255) / 256, 256, 0, st>>>(slot, w, static_cast<int32_t>(n_entries), fresh, static_cast<int32_t>(n_fresh),
                                                      static_cast<unsigned long long *>(ws), n_gpu);
  weigh_kernel<<<(n_gpu + 1023) / 1024, 256, 0, st>>>(static_cast<const uint64_t *>(ws), gpu_free, gpu_priority, mass, decay, n_gpu);
  return check_launch("pool weigh");
}
