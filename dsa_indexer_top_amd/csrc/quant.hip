// Quantisation to FP8 E4M3FN with one fp32 scale per row and block of 128 columns.
//
//   scale[r][b] = max(amax_{c in block b} |x[r][c]| / 448, 2^-126)
//   y[r][c]     = fl(x[r][c] / scale[r][c / 128]), rounded to the nearest E4M3FN number
//
// One pass: a block is 16 lanes of 8 elements, its largest magnitude a four-step DPP butterfly,
// so a value is read once and its code written once.  Bound by HBM (32768 x 4096 bf16 on MI355X: 73 us,
// 5.6 TB/s) or, with few rows, by the launch.
#include "float_types.cuh"

namespace echo {

constexpr int QT = 256;          // threads per workgroup

// QU groups of four blocks per wave.  WIDE: rows start 16-byte aligned in x and 8-byte aligned in y;
// otherwise whole 8-element pieces are read and written at any address.  The end of a row that is
// no whole piece goes element by element.
template <typename T, bool WIDE, int QU>
__global__ __launch_bounds__(QT) void quant_kernel(const T *__restrict__ x, int64_t ldx, int32_t n_cols,
                                                   uint32_t n_blk, uint32_t total, uint8_t *__restrict__ y,
                                                   int64_t ldy, float *__restrict__ scale, int64_t s_row,
                                                   int64_t s_blk) {
  const int l = lane_id(), sub = l >> 4, j = l & 15;
  const uint32_t wave = blockIdx.x * (QT / 64) + (threadIdx.x >> 6);
  Raw8<T> raw[QU];
  int left[QU];
  uint32_t row[QU], blk[QU];
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    const uint64_t i = (static_cast<uint64_t>(wave) * QU + u) * 4 + sub;
    const bool in = i < total;
    row[u] = in ? static_cast<uint32_t>(i) / n_blk : 0u;
    blk[u] = in ? static_cast<uint32_t>(i) - row[u] * n_blk : 0u;
    const int c = static_cast<int>(blk[u]) * 128 + j * VEC;
    left[u] = in ? min(max(n_cols - c, 0), VEC) : -1;        // -1: no such block
    const T *p = x + row[u] * ldx + c;
    if (left[u] <= 0) raw[u] = zero8<T>();
    else if (left[u] == VEC) raw[u] = WIDE ? load8(p) : load8_any(p);
    else raw[u] = load8_part(p, left[u]);
  }
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    float v[VEC];
    unpack8(raw[u], v);
    const Fp8Scale s = fp8_scale<sizeof(T) == 4>(group_amax<16>(v));
    const u32x2 code = quantise8<sizeof(T) == 4>(v, s);
    if (left[u] < 0) continue;
    if (j == 0) scale[row[u] * s_row + blk[u] * s_blk] = s.scale;
    uint8_t *p = y + row[u] * ldy + static_cast<int>(blk[u]) * 128 + j * VEC;
    if (left[u] == VEC) {
      if (WIDE) *reinterpret_cast<u32x2 *>(p) = code;
      else *reinterpret_cast<u32x2_any *>(p) = code;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < left[u]) p[i] = static_cast<uint8_t>(code[i >> 2] >> (8 * (i & 3)));
    }
  }
}

template <typename T, int QU>
static void launch_quant_u(const void *x, int64_t ldx, int32_t n_cols, uint32_t n_blk, uint32_t total, uint8_t *y,
                           int64_t ldy, float *scale, int64_t s_row, int64_t s_blk, hipStream_t st) {
  constexpr uint32_t PER = QU * 4 * (QT / 64);                   // blocks of a workgroup
  const uint32_t grid = (total + PER - 1) / PER;
  const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * sizeof(T) % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(y) % 8 == 0 && ldy % 8 == 0;
  if (wide)
    quant_kernel<T, true, QU><<<grid, QT, 0, st>>>(static_cast<const T *>(x), ldx, n_cols, n_blk, total, y, ldy, scale, s_row, s_blk);
  else
    quant_kernel<T, false, QU><<<grid, QT, 0, st>>>(static_cast<const T *>(x), ldx, n_cols, n_blk, total, y, ldy, scale, s_row, s_blk);
}

template <typename T>
static int launch_quant(const void *x, int64_t n_rows, int32_t n_cols, int64_t ldx, uint8_t *y, int64_t ldy,
                        float *scale, int64_t s_row, int64_t s_blk, hipStream_t st) {
  const uint32_t n_blk = (static_cast<uint32_t>(n_cols) + 127u) / 128u;
  const uint32_t total = static_cast<uint32_t>(n_rows * n_blk);
  // One group a wave up to 2^16 blocks, four beyond (MI355X, rows of 2048 bf16 values: 33 rows 2.3 us
  // with one, 3.5 with four; 2048 rows 3.9 and 4.3; 4096 rows 7.0 and 7.0).
  if (total >= 1u << 16) launch_quant_u<T, 4>(x, ldx, n_cols, n_blk, total, y, ldy, scale, s_row, s_blk, st);
  else launch_quant_u<T, 1>(x, ldx, n_cols, n_blk, total, y, ldy, scale, s_row, s_blk, st);
  return check_launch("quant_fp8");
}

}  // namespace echo

using namespace echo;

extern "C" int echo_quant_fp8(const void *x, int32_t x_type, int64_t n_rows, int32_t n_cols, int64_t ldx,
                              uint8_t *y, int64_t ldy, float *scale, int64_t scale_row, int64_t scale_blk,
                              void *stream) {
  if (n_rows < 0 || n_cols < 0) return fail(ECHO_EINVAL, "echo_quant_fp8: negative size");
  if (x_type != ECHO_BF16 && x_type != ECHO_FP16 && x_type != ECHO_FP32)
    return fail(ECHO_EINVAL, "echo_quant_fp8: type %d", x_type);
  if (n_rows == 0 || n_cols == 0) return ECHO_OK;
  if (!x || !y || !scale) return fail(ECHO_EINVAL, "echo_quant_fp8: NULL pointer");
  if (n_rows > 1 && (ldx < n_cols || ldy < n_cols)) return fail(ECHO_EINVAL, "echo_quant_fp8: row stride below n_cols");
  if (n_cols > (1 << 30)) return fail(ECHO_EUNSUPPORTED, "echo_quant_fp8: more than 2^30 columns");
  const int64_t n_blk = (static_cast<int64_t>(n_cols) + 127) / 128;
  if (n_rows >= (1 << 30) / n_blk) return fail(ECHO_EUNSUPPORTED, "echo_quant_fp8: 2^30 blocks or more");
  if (rows_overlap(n_rows, scale_row, n_blk, scale_blk, 1))
    return fail(ECHO_EINVAL, "echo_quant_fp8: scales overlap (strides %lld and %lld)", static_cast<long long>(scale_row),
                static_cast<long long>(scale_blk));
  const size_t size = x_type == ECHO_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size || reinterpret_cast<uintptr_t>(scale) % 4)
    return fail(ECHO_EINVAL, "echo_quant_fp8: x or scale not aligned to its type");
  switch (x_type) {
    case ECHO_BF16: return launch_quant<bf16_t>(x, n_rows, n_cols, ldx, y, ldy, scale, scale_row, scale_blk, S(stream));
    case ECHO_FP16: return launch_quant<fp16_t>(x, n_rows, n_cols, ldx, y, ldy, scale, scale_row, scale_blk, S(stream));
    default: return launch_quant<float>(x, n_rows, n_cols, ldx, y, ldy, scale, scale_row, scale_blk, S(stream));
  }
}
