// Page tables and slot maps of a paged key cache, advanced by one step on the GPU from the
// requests' lengths (echo_page_step).
//
// Per request r with old length L_r (0 for a finished one), n_r new tokens and pages of P:
//   back_r = ceil(len_r / P) for a finished request, else 0      pages that return to the stack
//   old_r  = ceil(L_r / P),  need_r = ceil((L_r + n_r) / P) - old_r
// Exclusive prefix sums over the requests place everything: the pages of finished requests go on
// the stack in (request, page) order, the i-th new page is the i-th from its top, and token t of
// the step belongs to the last request whose first token is <= t.  A new page's first token is
// always a token of the step, so the lane that maps that token also writes the page's table entry
// and no second pass over pages is needed.
//
// All of it is latency: the bytes of a decode step fit in a few cache lines per request.  A step of
// few tokens therefore runs as ONE workgroup and one launch, its prefix sums in LDS (256 requests
// on MI355X: 4.5 us a step, 2048 of which 128 are finished: 10.2).  A step of many tokens (chunked prefill: 16 bytes written
// per token) takes two launches: the plan (prefix sums, made by every workgroup for itself, and the
// return of the finished requests' pages, shared out among them) and the fill of the maps from the
// whole chip (61 requests with up to 8192 new tokens each: 4.0 + 5.5 us; with a launch of its own
// for the return and the searches in global memory it took 14.8 us).
#include "float_types.cuh"

namespace echo {

constexpr int PT = 512;                        // threads of the one-workgroup kernels
constexpr int PG_ONE_ROWS = 2048;              // requests whose prefix sums fit in LDS
constexpr int PG_ONE_TOKENS = 7 * PT;          // new tokens one workgroup maps: 64 requests' 1024 tokens
                                               // 4.1 us against 6.2 in two launches, 4096 6.8 against 6.4
constexpr int PF_T = 256;                      // threads of the fill and the return of pages
constexpr uint32_t FEW = 4;                    // new tokens that a request's own thread maps
constexpr uint32_t SAT = 0x7FFFFFFFu;

// A sum that stops at 2^31 - 1, still associative: the prefix sums of a step whose totals are
// refused stay defined.
struct OpSat {
  ECHO_DEV uint32_t operator()(uint32_t a, uint32_t b) const {
    const uint32_t s = a + b;                  // both at most 2^31 - 1: no wrap
    return s > SAT ? SAT : s;
  }
};

struct PageArgs {
  int32_t n_rows, shift, max_pages, n_pages, max_new;
  const int32_t *len_in, *new_len;
  const uint8_t *done;
  int32_t *page_table, *free_list;
  const int32_t *count_in;
  int32_t *len_out, *count_out, *row_begin;
  int64_t *slot;
  int32_t *row, *pos, *status;
};

// Lengths of one request: what it had, what it returns, what it needs.
struct PageRow { uint32_t back, need, fresh; int32_t len, old; bool bad; };

ECHO_DEV PageRow page_row(const PageArgs &a, int r) {
  PageRow p = {0, 0, 0, 0, 0, false};
  const int32_t len = a.len_in[r], n = a.new_len[r];
  const bool done = a.done && a.done[r];
  const int64_t room = static_cast<int64_t>(a.max_pages) << a.shift, up = (1 << a.shift) - 1;
  p.bad = len < 0 || n < 0 || len > room || (done ? 0 : static_cast<int64_t>(len)) + n > room ||
          (done ? 0 : static_cast<int64_t>(len)) + n > 0x7FFFFFFF;
  if (p.bad) return p;
  p.len = done ? 0 : len;
  p.back = done ? static_cast<uint32_t>((len + up) >> a.shift) : 0u;
  p.old = static_cast<int32_t>((p.len + up) >> a.shift);
  p.need = static_cast<uint32_t>((static_cast<int64_t>(p.len) + n + up) >> a.shift) - p.old;
  p.fresh = static_cast<uint32_t>(n);
  return p;
}

// The plan of a step, in LDS or the workspace: prefix sums, the lengths that are kept, and totals.
struct PagePlan {
  int32_t *back, *need, *begin;  // [n_rows + 1]: returned pages, new pages, new tokens before a request
  int32_t *kept;                 // [n_rows + 1]: its length without the new tokens (the last is not used)
  int32_t *head;                 // [0] free pages after the return, [1] after the step, [2] a request has
                                 // more than FEW new tokens
};
constexpr int PLAN_HEAD = 4;
ECHO_DEV PagePlan plan_at(int32_t *p, int rows) {
  return PagePlan{p, p + (rows + 1), p + 2 * (rows + 1), p + 3 * (rows + 1), p + 4 * (rows + 1)};
}

// Plan of a step by one workgroup of PT threads, each of which owns a run of consecutive requests
// (PER > 0: at most PER of them, kept in registers between the sums and the writing).  A step that
// is refused gets zero sums, the old lengths and count, and its status bits (set by `tell` alone).
template <int PER>
ECHO_DEV void make_plan(const PageArgs &a, const PagePlan &s, uint32_t *tmp, bool tell) {
  constexpr int NW = PT / 64;
  const int t = threadIdx.x, w = t >> 6, l = lane_id();
  const int per = (a.n_rows + PT - 1) / PT;
  const int r0 = min(t * per, a.n_rows), r1 = min(r0 + per, a.n_rows);
  uint32_t sum[3] = {0, 0, 0};
  bool bad = false, many = false;
  auto add = [&](const PageRow &p) {
    sum[0] = OpSat{}(sum[0], p.back);
    sum[1] = OpSat{}(sum[1], p.need);
    sum[2] = OpSat{}(sum[2], p.fresh);
    bad |= p.bad;
    many |= p.fresh > FEW;
  };
  const int32_t count = a.count_in[0];
  PageRow own[PER > 0 ? PER : 1];
  if constexpr (PER > 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (r0 + i < r1) { own[i] = page_row(a, r0 + i); add(own[i]); }
  } else {
    for (int r = r0; r < r1; ++r) add(page_row(a, r));
  }
  uint32_t incl[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    incl[i] = wave_incl_scan_op(sum[i], 0u, OpSat{});
    if (l == 63) tmp[i * NW + w] = incl[i];
  }
  const uint32_t flags = (__ballot(bad) != 0 ? 1u : 0u) | (__ballot(many) != 0 ? 2u : 0u);
  if (l == 63) tmp[3 * NW + w] = flags;
  __syncthreads();
  uint32_t base[3] = {0, 0, 0}, total[3] = {0, 0, 0}, seen = 0;
  for (int v = 0; v < NW; ++v) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t x = tmp[i * NW + v];
      if (v < w) base[i] = OpSat{}(base[i], x);
      total[i] = OpSat{}(total[i], x);
    }
    seen |= tmp[3 * NW + v];
  }
  const int64_t have = static_cast<int64_t>(count) + total[0];
  int32_t why = 0;
  if ((seen & 1u) || total[2] == SAT || total[2] > static_cast<uint32_t>(a.max_new)) why |= ECHO_ST_BAD_LEN;
  if (count < 0 || total[0] == SAT || total[1] == SAT || have > a.n_pages || static_cast<int64_t>(total[1]) > have)
    why |= ECHO_ST_NO_PAGES;
  // exclusive prefix of the thread's first request; exact whenever the step is not refused
  uint32_t at[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) at[i] = why ? 0u : base[i] + incl[i] - sum[i];
  auto put = [&](int r, const PageRow &p) {
    s.back[r] = at[0];
    s.need[r] = at[1];
    s.begin[r] = at[2];
    s.kept[r] = why ? a.len_in[r] : p.len;
    if (!why) { at[0] += p.back; at[1] += p.need; at[2] += p.fresh; }
  };
  if constexpr (PER > 0) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (r0 + i < r1) put(r0 + i, own[i]);
  } else {
    for (int r = r0; r < r1; ++r) put(r, page_row(a, r));
  }
  if (t == 0) {
    const int n = a.n_rows;
    s.back[n] = why ? 0 : total[0];
    s.need[n] = why ? 0 : total[1];
    s.begin[n] = why ? 0 : total[2];
    s.kept[n] = 0;
    s.head[0] = why ? count : static_cast<int32_t>(have);
    s.head[1] = s.head[0] - s.need[n];
    s.head[2] = seen >> 1;
    if (why && tell) atomicOr(a.status, why);
  }
  __syncthreads();
}

// The step's lengths, count and row_begin, by n threads; nothing reads the old ones any more.
ECHO_DEV void publish(const PageArgs &a, const PagePlan &s, int t, int n) {
  for (int r = t; r < a.n_rows; r += n) {
    const int32_t b = s.begin[r];
    a.row_begin[r] = b;
    a.len_out[r] = s.kept[r] + (s.begin[r + 1] - b);
  }
  if (t == 0) {
    a.row_begin[a.n_rows] = s.begin[a.n_rows];
    a.count_out[0] = s.head[1];
  }
}

// The last request of [lo, hi) whose first token is <= t; begin[lo] <= t < begin[hi].
ECHO_DEV int find_row(const int32_t *begin, int lo, int hi, int32_t t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (begin[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Returned pages of the step onto the stack by one workgroup.  A wave looks at 64 requests together
// and takes four finished ones with 16 lanes each, four pages a lane on their way (481 requests of which
// 109 return up to 445 pages on MI355X: 11.2 us a step, 16.7 with a wave per request and one page a
// lane; 256 with one finished 4.0 and 3.8.  With one or four requests a wave, whichever there are,
// 11.8 and 4.1; every page found by a search in the prefix sums took longer than any).
ECHO_DEV void return_rows(const PageArgs &a, const PagePlan &s) {
  constexpr int NW = PT / 64, U = 4, G = 16;
  const int l = lane_id();
  int32_t *top = a.free_list + (s.head[0] - s.back[a.n_rows]);
  for (int r0 = threadIdx.x >> 6; r0 < a.n_rows; r0 += 64 * NW) {
    const int r = r0 + l * NW;
    uint64_t some = __ballot(r < a.n_rows && s.back[r + 1] > s.back[r]);
    while (some) {
      uint64_t mine = some;
#pragma unroll
      for (int u = 0; u < 64 / G; ++u) {
        if (u < l / G) mine &= mine - 1;
        some &= some - 1;
      }
      const int q = mine ? r0 + (__ffsll(static_cast<unsigned long long>(mine)) - 1) * NW : 0;
      const int32_t cnt = mine ? s.back[q + 1] - s.back[q] : 0;
      const int32_t *__restrict__ src = a.page_table + static_cast<int64_t>(q) * a.max_pages;
      int32_t *__restrict__ dst = top + s.back[q];
      int i = l % G;
      for (; i + (U - 1) * G < cnt; i += U * G) {
        int32_t id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = src[i + u * G];
#pragma unroll
        for (int u = 0; u < U; ++u) dst[i + u * G] = id[u];
      }
#pragma unroll 1
      for (; i < cnt; i += G) dst[i] = src[i];
    }
  }
}

// Maps token t of the step (request r), and writes the table entry of a page that starts with it.
ECHO_DEV void map_token(const PageArgs &a, const PagePlan &s, int r, int32_t t) {
  const int32_t kept = s.kept[r], pos = kept + (t - s.begin[r]);
  const int32_t up = (1 << a.shift) - 1, page = pos >> a.shift, in_page = pos & up;
  const int32_t old = static_cast<int32_t>((static_cast<int64_t>(kept) + up) >> a.shift);
  int32_t *entry = a.page_table + static_cast<int64_t>(r) * a.max_pages + page;
  const int32_t id = page < old ? *entry : a.free_list[s.head[0] - 1 - (s.need[r] + page - old)];
  if (page >= old && in_page == 0) *entry = id;
  a.slot[t] = (static_cast<int64_t>(id) << a.shift) + in_page;
  if (a.row) a.row[t] = r;
  a.pos[t] = pos;
}

ECHO_DEV void map_none(const PageArgs &a, int32_t t) {
  a.slot[t] = -1;
  if (a.row) a.row[t] = -1;
  a.pos[t] = -1;
}

constexpr int PG_PER = PG_ONE_ROWS / PT;

__global__ __launch_bounds__(PT) void page_step_kernel(PageArgs a) {
  __shared__ int32_t plan[4 * (PG_ONE_ROWS + 1) + PLAN_HEAD];
  __shared__ uint32_t tmp[4 * (PT / 64)];
  const PagePlan s = plan_at(plan, a.n_rows);
  const int tid = threadIdx.x;
  make_plan<PG_PER>(a, s, tmp, true);
  publish(a, s, tid, PT);
  if (s.back[a.n_rows] > 0) return_rows(a, s);
  __syncthreads();                             // returned pages may be handed out again
  const int32_t total = s.begin[a.n_rows];
  if (!s.head[2]) {                            // a decode step: a thread per request, nothing to search
    for (int r = tid; r < a.n_rows; r += PT)
      for (int32_t t = s.begin[r]; t < s.begin[r + 1]; ++t) map_token(a, s, r, t);
  } else {
    for (int32_t t = tid; t < total; t += PT) map_token(a, s, find_row(s.begin, 0, a.n_rows, t), t);
  }
  for (int32_t t = total + tid; t < a.max_new; t += PT) map_none(a, t);
}

// Up to PG_ONE_ROWS requests: every workgroup makes the plan in its LDS and returns its share of the
// pages; the first one writes the plan out.  Nothing that another workgroup reads is written.
__global__ __launch_bounds__(PT) void page_plan_kernel(PageArgs a, int32_t *ws) {
  __shared__ int32_t plan[4 * (PG_ONE_ROWS + 1) + PLAN_HEAD];
  __shared__ uint32_t tmp[4 * (PT / 64)];
  const PagePlan s = plan_at(plan, a.n_rows);
  make_plan<PG_PER>(a, s, tmp, blockIdx.x == 0);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < 4 * (a.n_rows + 1) + 2; i += PT) ws[i] = plan[i];
  // the finished requests' pages, a workgroup per request
  int32_t *top = a.free_list + (s.head[0] - s.back[a.n_rows]);
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x)
    for (int i = s.back[r] + threadIdx.x; i < s.back[r + 1]; i += PT)
      top[i] = a.page_table[static_cast<int64_t>(r) * a.max_pages + (i - s.back[r])];
}

// More requests: one workgroup, the plan in the workspace.
__global__ __launch_bounds__(PT) void page_plan_many_kernel(PageArgs a, int32_t *ws) {
  __shared__ uint32_t tmp[4 * (PT / 64)];
  const PagePlan s = plan_at(ws, a.n_rows);
  make_plan<0>(a, s, tmp, true);
  if (s.back[a.n_rows] > 0) return_rows(a, s);
}

// One token per lane (four of them, their loads together, took 8.1 us where one takes 5.5).  The
// requests of a wave's 64 tokens lie between those of its first and last token, found first (all
// lanes alike); a wave inside one request, the usual case of a prefill, searches no further.  LDS:
// with a copy of the plan in LDS.  The last workgroup publishes the lengths.
template <bool LDS>
__global__ __launch_bounds__(PF_T) void page_fill_kernel(PageArgs a, int32_t *ws) {
  __shared__ int32_t copy[LDS ? 4 * (PG_ONE_ROWS + 1) + PLAN_HEAD : 1];
  if (LDS) {
    for (int i = threadIdx.x; i < 4 * (a.n_rows + 1) + 2; i += PF_T) copy[i] = ws[i];
    __syncthreads();
  }
  const PagePlan s = plan_at(LDS ? copy : ws, a.n_rows);
  if (blockIdx.x == gridDim.x - 1) { publish(a, s, threadIdx.x, PF_T); return; }
  const int32_t total = s.begin[a.n_rows];
  const int64_t t = static_cast<int64_t>(blockIdx.x) * PF_T + threadIdx.x, w0 = t - lane_id();
  if (t < total) {
    const int32_t last = static_cast<int32_t>(min(w0 + 63, static_cast<int64_t>(total) - 1));
    const int lo = find_row(s.begin, 0, a.n_rows, static_cast<int32_t>(w0));
    const int hi = find_row(s.begin, lo, a.n_rows, last);
    map_token(a, s, find_row(s.begin, lo, hi + 1, static_cast<int32_t>(t)), static_cast<int32_t>(t));
  } else if (t < a.max_new) {
    map_none(a, static_cast<int32_t>(t));
  }
}

// A workgroup per request copies its newest token's query and weights (8 KB of 64 heads: launch bound).
__global__ __launch_bounds__(PF_T) void newest_kernel(const uint8_t *__restrict__ q8, const float *__restrict__ w,
                                                      const int32_t *__restrict__ row_begin,
                                                      const int32_t *__restrict__ len, int32_t n_tok, int32_t heads,
                                                      uint8_t *__restrict__ q_out, float *__restrict__ w_out,
                                                      int32_t *__restrict__ len_out) {
  const int32_t r = blockIdx.x, begin = row_begin[r], end = row_begin[r + 1];
  const bool got = begin >= 0 && begin < end && end <= n_tok;
  if (threadIdx.x == 0) len_out[r] = got ? len[r] : 0;
  if (!got) return;
  const int64_t from = static_cast<int64_t>(end - 1) * heads, to = static_cast<int64_t>(r) * heads;
  const u32x2 *src = reinterpret_cast<const u32x2 *>(q8 + from * D);
  u32x2 *dst = reinterpret_cast<u32x2 *>(q_out + to * D);
  for (int64_t i = threadIdx.x; i < static_cast<int64_t>(heads) * (D / 8); i += PF_T) dst[i] = src[i];
  for (int64_t h = threadIdx.x; h < heads; h += PF_T) w_out[to + h] = w[from + h];
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_page_workspace_bytes(int32_t n_rows, int32_t max_new) {
  (void)max_new;
  if (n_rows < 0) return 0;
  return sizeof(int32_t) * (4 * (static_cast<size_t>(n_rows) + 1) + PLAN_HEAD);
}

extern "C" int echo_page_step(const echo_page_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p) return fail(ECHO_EINVAL, "echo_page_step: NULL args");
  if (p->n_rows < 0 || p->max_new < 0 || p->max_pages < 0 || p->n_pages < 0)
    return fail(ECHO_EINVAL, "echo_page_step: negative size");
  if (p->page_size < 16 || p->page_size > 65536 || (p->page_size & (p->page_size - 1)))
    return fail(ECHO_EUNSUPPORTED, "echo_page_step: page size %d is not a power of two in [16, 65536]", p->page_size);
  if (p->n_rows > 65535) return fail(ECHO_EUNSUPPORTED, "echo_page_step: %d requests, more than 65535", p->n_rows);
  // Without requests and room for tokens a step still has its count and row_begin[0] to write, unless
  // the call keeps no place for the second apart from the first (arrays may not overlap).
  if (p->n_rows == 0 && p->max_new == 0 && p->count_out == p->count_in && p->row_begin == p->count_out) return ECHO_OK;
  if ((p->n_pages && !p->free_list) || !p->count_in || !p->count_out || !p->row_begin || !p->status ||
      (p->n_rows && (!p->len_in || !p->new_len || (p->max_pages && !p->page_table) || !p->len_out)) ||
      (p->max_new && (!p->slot || !p->pos)))
    return fail(ECHO_EINVAL, "echo_page_step: NULL pointer");
  uintptr_t bits = reinterpret_cast<uintptr_t>(p->slot) % 8 ? 1 : 0;
  const int32_t *const words[] = {p->len_in, p->new_len, p->page_table, p->free_list, p->count_in, p->len_out,
                                  p->count_out, p->row_begin, p->row, p->pos, p->status};
  for (const int32_t *q : words) bits |= reinterpret_cast<uintptr_t>(q) % 4;
  if (bits) return fail(ECHO_EINVAL, "echo_page_step: an array is not aligned to its type");
  PageArgs a = {p->n_rows, __builtin_ctz(p->page_size), p->max_pages, p->n_pages, p->max_new, p->len_in, p->new_len,
                p->done, p->page_table, p->free_list, p->count_in, p->len_out, p->count_out, p->row_begin, p->slot,
                p->row, p->pos, p->status};
  const hipStream_t st = S(stream);
  if (p->n_rows <= PG_ONE_ROWS && p->max_new <= PG_ONE_TOKENS) {
    page_step_kernel<<<1, PT, 0, st>>>(a);
    return check_launch("page_step");
  }
  if (!ws || ws_bytes < echo_page_workspace_bytes(p->n_rows, p->max_new))
    return fail(ECHO_EWORKSPACE, "echo_page_step: workspace of %zu bytes, %zu needed", ws ? ws_bytes : 0,
                echo_page_workspace_bytes(p->n_rows, p->max_new));
  if (reinterpret_cast<uintptr_t>(ws) % 4) return fail(ECHO_EINVAL, "echo_page_step: workspace is not 4-byte aligned");
  int32_t *w = static_cast<int32_t *>(ws);
  const bool lds = p->n_rows <= PG_ONE_ROWS;
  if (lds)
    page_plan_kernel<<<p->done ? max(1, min(p->n_rows, 64)) : 1, PT, 0, st>>>(a, w);
  else
    page_plan_many_kernel<<<1, PT, 0, st>>>(a, w);
  // one workgroup more than the tokens take publishes the lengths
  const uint32_t fill = static_cast<uint32_t>((static_cast<int64_t>(p->max_new) + PF_T - 1) / PF_T) + 1;
  if (lds) page_fill_kernel<true><<<fill, PF_T, 0, st>>>(a, w);
  else page_fill_kernel<false><<<fill, PF_T, 0, st>>>(a, w);
  return check_launch("page_step");
}

extern "C" int echo_newest_queries(const uint8_t *q8, const float *w, const int32_t *row_begin, const int32_t *len,
                                   int32_t n_rows, int32_t n_tok, int32_t n_q_heads, uint8_t *q_out, float *w_out,
                                   int32_t *len_out, void *stream) {
  if (n_rows < 0 || n_tok < 0 || n_q_heads < 0) return fail(ECHO_EINVAL, "echo_newest_queries: negative size");
  if (n_rows > 65535) return fail(ECHO_EUNSUPPORTED, "echo_newest_queries: %d requests, more than 65535", n_rows);
  if (n_rows == 0) return ECHO_OK;
  const bool rows = n_tok && n_q_heads;
  if (!row_begin || !len || !len_out || (rows && (!q8 || !w)) || (n_q_heads && (!q_out || !w_out)))
    return fail(ECHO_EINVAL, "echo_newest_queries: NULL pointer");
  const auto off = [](const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(q8, 8) || off(q_out, 8))
    return fail(ECHO_EUNSUPPORTED, "echo_newest_queries: q8 or q_out is not 8-byte aligned");
  if (off(w, 4) || off(w_out, 4) || off(row_begin, 4) || off(len, 4) || off(len_out, 4))
    return fail(ECHO_EINVAL, "echo_newest_queries: a pointer is not aligned to its type");
  newest_kernel<<<static_cast<uint32_t>(n_rows), PF_T, 0, S(stream)>>>(q8, w, row_begin, len, n_tok, n_q_heads, q_out,
                                                                      w_out, len_out);
  return check_launch("newest_queries");
}
