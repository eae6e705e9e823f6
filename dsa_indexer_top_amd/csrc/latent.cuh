// What the kernels that read a latent cache share: the matrix core's operands for the cache's type,
// and where the tokens of a list, a block list or a paged request are.
//
// v_mfma_f32_16x16x32: lane l = 16 g + j supplies row j of the first operand and column j of the
// second for eight products, and receives rows 4 g .. 4 g + 3 of column j of the result.
// v_mfma_f32_32x32x16: lane l = 32 h + j likewise, and rows 8 b + 4 h + e of column j as element 4 b + e.
// Which eight products a lane group takes does not matter as long as both operands agree.
#pragma once

#include "float_types.cuh"

namespace echo {

constexpr int LATENT = ECHO_ROW_ELEMS;           // values of a row: what a head is multiplied with
constexpr int VALUES = ECHO_VALUE_ELEMS;         // its first values: what is summed
constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;
constexpr float NO_SCORE = -3.0e38f;             // a running maximum before the first token: finite, so that
                                                 // differences of two of them are 0

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void glb_void;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8 __attribute__((ext_vector_type(8)));

template <typename T> struct Mma;
template <> struct Mma<bf16_t> {
  typedef bf16x8 x8;
  ECHO_DEV static v4f mul(x8 a, x8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  ECHO_DEV static v16f mul(x8 a, x8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Mma<fp16_t> {
  typedef fp16x8 x8;
  ECHO_DEV static v4f mul(x8 a, x8 b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  ECHO_DEV static v16f mul(x8 a, x8 b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};

template <typename X8, typename P>
ECHO_DEV X8 read16(const P *p) { return __builtin_bit_cast(X8, *reinterpret_cast<const u32x4 *>(p)); }

template <typename T>
ECHO_DEV u32x2 pack4(const v4f &v) {
  T e[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) e[u] = from_f32<T>(v[u]);
  u32x2 w;
  __builtin_memcpy(&w, e, 8);
  return w;
}

// 2^x and log2 x as the hardware gives them, off by a unit in the last place; 2^x below 2^-126 is 0.
ECHO_DEV float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
ECHO_DEV float log2_(float x) { return __builtin_amdgcn_logf(x); }

// s_waitcnt: at most n vector memory operations under way; every LDS operation done.
constexpr int vmcnt(int n) { return (n & 15) | 0x0F70 | (n >> 4) << 14; }
constexpr int WAIT_VM0 = vmcnt(0), WAIT_LDS0 = 0xC07F;

// The workgroup's waves meet, their LDS operations done.  Loads under way stay under way, which
// __syncthreads() would wait for.
ECHO_DEV void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(WAIT_LDS0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- tokens
// Tokens t = 0, 1, .. of one query row.  With a list, token t is token t % 2^shift of block
// list[t >> shift], without one position t.  A position in [0, limit) is row
// table[pos >> pshift] * 2^pshift + pos % 2^pshift of the cache, or, without a table, row pos.
struct Tokens {
  const int32_t *list;
  const int32_t *table;
  int64_t limit;
  int32_t shift, pshift, max_pages, n_kv;
  // The list's entry of token t (t in range), and its position; negative: none.
  ECHO_DEV int32_t entry(int32_t t) const { return list ? list[t >> shift] : 0; }
  ECHO_DEV int64_t position(int32_t t, int32_t e) const {
    const int64_t p = list ? (e < 0 ? -1 : (static_cast<int64_t>(e) << shift) + (t & ((1 << shift) - 1))) : t;
    return p < limit ? p : -1;
  }
  ECHO_DEV int32_t page(int64_t pos) const {
    return table && pos >= 0 && (pos >> pshift) < max_pages ? table[pos >> pshift] : -1;
  }
  // The cache's row, -1 where there is none.
  ECHO_DEV int32_t row(int64_t pos, int32_t page) const {
    const int64_t r = table ? (page < 0 || pos < 0 ? -1 : (static_cast<int64_t>(page) << pshift) + (pos & ((1 << pshift) - 1))) : pos;
    return r >= 0 && r < n_kv ? static_cast<int32_t>(r) : -1;
  }
};

// Arguments of echo_sparse_attention and echo_attention_weights.
struct LatentArgs {
  const uint16_t *q;
  int64_t q_row, q_head;
  const uint16_t *kv;
  int64_t kv_stride;
  const int32_t *idx;
  int64_t idx_ld;
  const int32_t *len, *table, *req;
  int32_t n_rows, n_heads, n_kv, n_tok, shift, pshift, max_pages, n_tables;
  float scale2;                  // scale * log2 e
  ECHO_DEV Tokens tokens(int32_t r) const {
    Tokens s = {idx + static_cast<int64_t>(r) * idx_ld, nullptr, len ? len[r] : INT64_MAX, shift, pshift, max_pages, n_kv};
    if (table) {
      const int32_t t = req ? req[r] : r;
      if (t < 0 || t >= n_tables) s.limit = 0;             // no request: no tokens
      s.table = table + static_cast<int64_t>(t < 0 || t >= n_tables ? 0 : t) * max_pages;
    }
    return s;
  }
};

// ---------------------------------------------------------------- host
// echo_latent_args, checked, as the kernels take them; fn names the entry point.
int latent_args(const char *fn, const echo_latent_args *a, LatentArgs *x);

}  // namespace echo
