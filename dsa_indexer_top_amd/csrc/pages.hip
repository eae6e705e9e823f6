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
// All of it is latency: the bytes of a decode step fit in a few cache lines per request.  A step
// of few tokens therefore runs as ONE workgroup and one launch, its prefix sums in LDS.  A step of
// many tokens (chunked prefill: 16 bytes written per token) takes the prefix sums in one
// workgroup and then fills the maps from the whole chip, with a launch in between for the pages
// that come back.
#include "float_types.cuh"

namespace echo {

constexpr int PT = 512;                        // threads of the one-workgroup kernels
constexpr int PG_ONE_ROWS = 2048;              // requests whose prefix sums fit in LDS
constexpr int PG_ONE_TOKENS = 8192;            // new tokens one workgroup maps
constexpr int PF_T = 256;                      // threads of the fill and the return of pages
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

// Workspace (or LDS): prefix sums of the returned and the needed pages, and the step's totals.
struct PageSums {
  int32_t *back, *need;          // [n_rows + 1]
  int32_t *head;                 // [0] free pages after the return, [1] new tokens
};

// Prefix sums of a step by one workgroup of PT threads; each thread owns a run of consecutive
// requests.  Writes the sums, row_begin, the new lengths and the new count, or, for a step that is
// refused, zero sums, the old lengths, the old count and a status bit.  begin: where the kernel
// itself reads row_begin from (LDS or the output).
ECHO_DEV void page_sums(const PageArgs &a, const PageSums &s, int32_t *begin, uint32_t *tmp) {
  constexpr int NW = PT / 64;
  const int t = threadIdx.x, w = t >> 6, l = lane_id();
  const int per = (a.n_rows + PT - 1) / PT;
  const int r0 = min(t * per, a.n_rows), r1 = min(r0 + per, a.n_rows);
  uint32_t sum[3] = {0, 0, 0};
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const PageRow p = page_row(a, r);
    sum[0] = OpSat{}(sum[0], p.back);
    sum[1] = OpSat{}(sum[1], p.need);
    sum[2] = OpSat{}(sum[2], p.fresh);
    bad |= p.bad;
  }
  const int32_t count = a.count_in[0];
  uint32_t incl[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    incl[i] = wave_incl_scan_op(sum[i], 0u, OpSat{});
    if (l == 63) tmp[i * NW + w] = incl[i];
  }
  const bool any_bad = __ballot(bad) != 0;
  if (l == 63) tmp[3 * NW + w] = any_bad;
  __syncthreads();
  uint32_t base[3] = {0, 0, 0}, total[3] = {0, 0, 0}, refuse = 0;
  for (int v = 0; v < NW; ++v) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t x = tmp[i * NW + v];
      if (v < w) base[i] = OpSat{}(base[i], x);
      total[i] = OpSat{}(total[i], x);
    }
    refuse |= tmp[3 * NW + v];
  }
  const int64_t have = static_cast<int64_t>(count) + total[0];
  int32_t why = 0;
  if (refuse || total[2] == SAT || total[2] > static_cast<uint32_t>(a.max_new)) why |= ECHO_ST_BAD_LEN;
  if (count < 0 || total[0] == SAT || total[1] == SAT || have > a.n_pages || static_cast<int64_t>(total[1]) > have)
    why |= ECHO_ST_NO_PAGES;
  // exclusive prefix of the thread's first request; exact whenever the step is not refused
  uint32_t at[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) at[i] = why ? 0u : base[i] + incl[i] - sum[i];
  for (int r = r0; r < r1; ++r) {
    const PageRow p = page_row(a, r);
    s.back[r] = at[0];
    s.need[r] = at[1];
    begin[r] = at[2];
    if (begin != a.row_begin) a.row_begin[r] = at[2];
    const int32_t len = a.len_in[r];
    a.len_out[r] = why ? len : p.len + static_cast<int32_t>(p.fresh);
    if (!why) { at[0] += p.back; at[1] += p.need; at[2] += p.fresh; }
  }
  if (t == 0) {
    const int n = a.n_rows;
    s.back[n] = why ? 0 : total[0];
    s.need[n] = why ? 0 : total[1];
    begin[n] = why ? 0 : total[2];
    if (begin != a.row_begin) a.row_begin[n] = begin[n];
    s.head[0] = why ? count : static_cast<int32_t>(have);
    s.head[1] = begin[n];
    if (why) atomicOr(a.status, why);
  }
  __syncthreads();                             // count_in is read before count_out is written
  if (t == 0) a.count_out[0] = s.head[0] - s.need[a.n_rows];
}

// Request r's returned pages onto the stack, by `n` threads.
ECHO_DEV void return_pages(const PageArgs &a, const PageSums &s, int32_t first_free, int r, int t, int n) {
  const int32_t b = s.back[r], cnt = s.back[r + 1] - b;
  const int32_t *src = a.page_table + static_cast<int64_t>(r) * a.max_pages;
  for (int i = t; i < cnt; i += n) a.free_list[first_free + b + i] = src[i];
}

// The last request of [lo, hi) whose first token is <= t; begin[lo] <= t < begin[hi].
ECHO_DEV int find_row(const int32_t *begin, int lo, int hi, int32_t t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (begin[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Maps token t of the step (request r), and writes the table entry of a page that starts here.
ECHO_DEV void map_token(const PageArgs &a, const PageSums &s, const int32_t *begin, int32_t top, int r, int32_t t) {
  const int32_t b = begin[r], fresh = begin[r + 1] - b;
  const int32_t end = a.len_out[r], pos = end - fresh + (t - b);
  const int32_t page = pos >> a.shift, in_page = pos & ((1 << a.shift) - 1);
  const int32_t up = (1 << a.shift) - 1;
  const int32_t old = static_cast<int32_t>((static_cast<int64_t>(end - fresh) + up) >> a.shift);
  int32_t *entry = a.page_table + static_cast<int64_t>(r) * a.max_pages + page;
  int32_t id;
  if (page < old) {
    id = *entry;
  } else {
    id = a.free_list[top - 1 - (s.need[r] + page - old)];
    if (in_page == 0) *entry = id;
  }
  a.slot[t] = (static_cast<int64_t>(id) << a.shift) + in_page;
  if (a.row) a.row[t] = r;
  a.pos[t] = pos;
}

ECHO_DEV void map_none(const PageArgs &a, int32_t t) {
  a.slot[t] = -1;
  if (a.row) a.row[t] = -1;
  a.pos[t] = -1;
}

__global__ __launch_bounds__(PT) void page_step_kernel(PageArgs a) {
  __shared__ int32_t back[PG_ONE_ROWS + 1];
  __shared__ int32_t need[PG_ONE_ROWS + 1];
  __shared__ int32_t begin[PG_ONE_ROWS + 1];
  __shared__ int32_t head[2];
  __shared__ uint32_t tmp[4 * (PT / 64)];
  const PageSums s = {back, need, head};
  const int tid = threadIdx.x;
  page_sums(a, s, begin, tmp);
  const int32_t top = head[0], total = head[1];
  if (back[a.n_rows] > 0) {                    // a wave per request with pages to return
    const int32_t first_free = top - back[a.n_rows];
    for (int r = tid >> 6; r < a.n_rows; r += PT / 64) return_pages(a, s, first_free, r, tid & 63, 64);
  }
  __syncthreads();                             // returned pages may be handed out again
  for (int32_t t = tid; t < a.max_new; t += PT) {
    if (t < total) map_token(a, s, begin, top, find_row(begin, 0, a.n_rows, t), t);
    else map_none(a, t);
  }
}

__global__ __launch_bounds__(PT) void page_sums_kernel(PageArgs a, PageSums s) {
  __shared__ uint32_t tmp[4 * (PT / 64)];
  page_sums(a, s, a.row_begin, tmp);
}

__global__ __launch_bounds__(PF_T) void page_return_kernel(PageArgs a, PageSums s) {
  const int32_t first_free = s.head[0] - s.back[a.n_rows];
  for (int r = blockIdx.x; r < a.n_rows; r += gridDim.x)
    return_pages(a, s, first_free, r, threadIdx.x, PF_T);
}

// One token per lane.  The requests of a wave's 64 tokens lie between those of its first and last
// token, found first (all lanes alike); a wave inside one request, the usual case of a prefill,
// searches no further.
__global__ __launch_bounds__(PF_T) void page_fill_kernel(PageArgs a, PageSums s) {
  const int32_t top = s.head[0], total = s.head[1];
  const int64_t t64 = static_cast<int64_t>(blockIdx.x) * PF_T + threadIdx.x;
  const int64_t w0 = t64 - lane_id();
  if (t64 >= a.max_new) return;
  const int32_t t = static_cast<int32_t>(t64);
  if (t >= total) { map_none(a, t); return; }
  const int32_t last = static_cast<int32_t>(min(w0 + 63, static_cast<int64_t>(total) - 1));
  const int lo = find_row(a.row_begin, 0, a.n_rows, static_cast<int32_t>(w0));
  const int hi = find_row(a.row_begin, lo, a.n_rows, last);
  map_token(a, s, a.row_begin, top, find_row(a.row_begin, lo, hi + 1, t), t);
}

}  // namespace echo

using namespace echo;

extern "C" size_t echo_page_workspace_bytes(int32_t n_rows, int32_t max_new) {
  (void)max_new;
  if (n_rows < 0) return 0;
  return sizeof(int32_t) * (2 * (static_cast<size_t>(n_rows) + 1) + 2);
}

extern "C" int echo_page_step(const echo_page_args *p, void *ws, size_t ws_bytes, void *stream) {
  if (!p) return fail(ECHO_EINVAL, "echo_page_step: NULL args");
  if (p->n_rows < 0 || p->max_new < 0 || p->max_pages < 0 || p->n_pages < 0)
    return fail(ECHO_EINVAL, "echo_page_step: negative size");
  if (p->page_size < 16 || p->page_size > 65536 || (p->page_size & (p->page_size - 1)))
    return fail(ECHO_EUNSUPPORTED, "echo_page_step: page size %d is not a power of two in [16, 65536]", p->page_size);
  if (p->n_rows > 65535) return fail(ECHO_EUNSUPPORTED, "echo_page_step: %d requests, more than 65535", p->n_rows);
  if (p->n_rows == 0 && p->max_new == 0) return ECHO_OK;
  if (!p->free_list || !p->count_in || !p->count_out || !p->row_begin || !p->status ||
      (p->n_rows && (!p->len_in || !p->new_len || !p->page_table || !p->len_out)) ||
      (p->max_new && (!p->slot || !p->pos)))
    return fail(ECHO_EINVAL, "echo_page_step: NULL pointer");
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
  int32_t *w = static_cast<int32_t *>(ws);
  const PageSums s = {w, w + p->n_rows + 1, w + 2 * (p->n_rows + 1)};
  page_sums_kernel<<<1, PT, 0, st>>>(a, s);
  if (p->done && p->n_rows) page_return_kernel<<<min(p->n_rows, 1024), PF_T, 0, st>>>(a, s);
  if (p->max_new) page_fill_kernel<<<(static_cast<uint32_t>(p->max_new) + PF_T - 1) / PF_T, PF_T, 0, st>>>(a, s);
  return check_launch("page_step");
}
