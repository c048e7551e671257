// Page tables and slot maps of a paged KV cache, built on the GPU from request
// lengths.  A call takes every request of a pool from its present length to a
// new one: a request that grows is granted pages from the free stack, one that
// shrinks (a finished request, rejected drafted tokens) gives pages back, and
// each new token gets its position and its slot in the cache.
//
// With p(x) = ceil(x / page_size), released pages r = 0 .. R-1 and granted
// pages g = 0 .. G-1 counted in (request, page) order, and a stack of `count`
// free pages:
//   page g  = released[g] if g < R, else stack[count - 1 - (g - R)];
//   pages r >= G go to stack[count + R - 1 - r];  count' = count + R - G.
// Growing and then shrinking by the same amounts restores the stack exactly.
//
// What bounds it: latency.  A decode step of 64 requests moves about 2 KB (4.3 to
// 5.1 us), the prefill of 64 prompts with pages of 16 moves 2.8 MB (6.1 us), a step
// of 1021 requests' trees 0.6 MB (8.4 us).  So one launch does everything: every CTA
// scans all requests on its own (a few KB out of L2, cheaper than a second launch
// that waits for the first) and fills its share of the tables.  No entry that one
// CTA reads is written by another (grants go to table entries at or above a
// request's old page count, pushes to stack entries at or above `count`), except the
// lengths and the count themselves: the CTA that finishes last, by a ticket, writes
// those.
#include "internal.h"

namespace msa {

msa_status check_page_geometry(int32_t num_pages, int32_t page_size);

namespace {

constexpr int kThreads = 512;
constexpr int kMaxRequests = 8192;  // five int32 per request in shared memory
constexpr int kMaxCtas = 152;
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - (1 << 19);  // an index may step one round past the last token
static_assert(4 * kMaxCtas * kThreads < 1 << 19, "indexes within int32");
constexpr int scan_bytes(int requests) { return 5 * (requests + 1) * (int)sizeof(int32_t); }
constexpr int kStaticBytes = 1024;  // at least the kernel's static shared memory
static_assert(scan_bytes(kMaxRequests) + kStaticBytes <= 227 * 1024, "shared memory budget");

struct PageArgs {
  int32_t S, N, shift, max_pages, T, cap;
  const int32_t* new_len;
  const int32_t* depth;
  int32_t *table, *seq_len, *stack, *state, *cu, *slots, *pos;
  int* err;
};

struct Sum3 {
  int64_t tok, grow, rel;
};

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Exclusive prefix of this thread's sums over the CTA, and the CTA's totals.
__device__ Sum3 block_exclusive(Sum3 v, Sum3* part, Sum3& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Sum3 inc = {warp_inclusive(v.tok, lane), warp_inclusive(v.grow, lane), warp_inclusive(v.rel, lane)};
  __syncthreads();
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  Sum3 base = {0, 0, 0};
  total = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const Sum3 p = part[w];
    if (w < warp) { base.tok += p.tok; base.grow += p.grow; base.rel += p.rel; }
    total.tok += p.tok;
    total.grow += p.grow;
    total.rel += p.rel;
  }
  return {base.tok + inc.tok - v.tok, base.grow + inc.grow - v.grow, base.rel + inc.rel - v.rel};
}

// The request that holds flat index x: the last s with pre[s] <= x.
__device__ __forceinline__ int find(const int32_t* pre, int S, int x) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) page_table_kernel(const PageArgs A) {
  extern __shared__ int32_t sm[];
  __shared__ Sum3 part[kThreads / 32];
  __shared__ int s_last, s_refused;
  static_assert(sizeof(part) + sizeof(s_last) + sizeof(s_refused) <= kStaticBytes, "static shared memory");
  int32_t* s_tok = sm;               // tokens of the requests before
  int32_t* s_gr = sm + (A.S + 1);    // pages granted before
  int32_t* s_rel = s_gr + (A.S + 1); // pages released before
  int32_t* s_len = s_rel + (A.S + 1);  // length after the call
  int32_t* s_old = s_len + (A.S + 1);  // and before

  const int tid = threadIdx.x, up = (1 << A.shift) - 1;
  const int most = A.max_pages << A.shift;
  auto pages = [&](int x) { return (x + up) >> A.shift; };
  int count = A.state[0];
  const bool sane = count >= 0 && count <= A.N;
  if (!sane) count = 0;
  if (tid == 0) s_refused = 0;

  // ---- what every request asks for, and who is served
  const int per = (A.S + kThreads - 1) / kThreads, s0 = min(A.S, tid * per), s1 = min(A.S, s0 + per);
  const bool tokens = A.slots != nullptr;
  auto ask = [&](int old, int& len) -> Sum3 {
    Sum3 v = {0, 0, 0};
    if (!sane || len < 0 || len > most || old < 0 || old > most || (tokens && A.T && len - old > A.T)) {
      len = -1;
      return v;
    }
    if (len > old) { v.tok = len - old; v.grow = pages(len) - pages(old); }
    else v.rel = pages(old) - pages(len);
    return v;
  };
  Sum3 mine = {0, 0, 0}, all;
  for (int s = s0; s < s1; ++s) {
    const int old = A.seq_len[s];
    int len = A.new_len[s];
    const Sum3 v = ask(old, len);
    if (len < 0) atomicCAS(A.err, 0, (int)kErrIndex);
    s_old[s] = old;
    s_len[s] = len;
    mine.tok += v.tok; mine.grow += v.grow; mine.rel += v.rel;
  }
  Sum3 run = block_exclusive(mine, part, all);
  const Sum3 start = run;
  // a pool whose tables and stack hold more pages than it has is left as it is
  const int64_t avail = count + all.rel;
  const bool fits = sane && avail <= A.N;
  if (!fits && tid == 0) atomicCAS(A.err, 0, (int)kErrIndex);
  const int R = fits ? (int)all.rel : 0;
  mine = {0, 0, 0};
  int refused = 0;
  for (int s = s0; s < s1; ++s) {
    const int old = s_old[s];
    int len = s_len[s];
    const Sum3 v = ask(old, len);
    run.tok += v.tok; run.grow += v.grow;
    const bool ok = fits && len >= 0 && (v.grow == 0 || run.grow <= avail) &&
                    (!tokens || A.T || v.tok == 0 || run.tok <= A.cap);
    s_len[s] = ok ? len : old;
    s_rel[s] = fits ? (int)run.rel : 0;
    run.rel += v.rel;
    if (ok) { mine.tok += v.tok; mine.grow += v.grow; }
    else ++refused;
  }
  if (refused) atomicAdd(&s_refused, refused);
  Sum3 fin = all;
  if (__syncthreads_or(refused)) run = block_exclusive(mine, part, fin);  // without the refused ones
  else run = start;
  const int G = (int)fin.grow;
  for (int s = s0; s < s1; ++s) {
    const int old = s_old[s], len = s_len[s];
    s_tok[s] = (int)run.tok;
    s_gr[s] = (int)run.grow;
    if (len > old) { run.tok += len - old; run.grow += pages(len) - pages(old); }
  }
  if (tid == 0) { s_tok[A.S] = (int)fin.tok; s_gr[A.S] = G; s_rel[A.S] = R; }
  __syncthreads();

  const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  auto checked = [&](int page) {
    if ((unsigned)page < (unsigned)A.N) return page;
    atomicCAS(A.err, 0, (int)kErrIndex);
    return -1;
  };
  auto released = [&](int r) {
    const int s = find(s_rel, A.S, r);
    return A.table[(int64_t)s * A.max_pages + pages(s_len[s]) + (r - s_rel[s])];
  };
  auto granted = [&](int g) { return checked(g < R ? released(g) : A.stack[count - 1 - (g - R)]); };

  // ---- granted pages into the table, released ones that stay free onto the stack: four a thread, loads first
  for (int g0 = 4 * gtid; g0 < G; g0 += 4 * gsize) {
    int page[4], s = find(s_gr, A.S, g0);
#pragma unroll
    for (int x = 0; x < 4; ++x) page[x] = g0 + x < G ? granted(g0 + x) : 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (g0 + x >= G) break;
      while (s + 1 < A.S && s_gr[s + 1] <= g0 + x) ++s;
      A.table[(int64_t)s * A.max_pages + pages(s_old[s]) + (g0 + x - s_gr[s])] = page[x];
    }
  }
  for (int r0 = G + 4 * gtid; r0 < R; r0 += 4 * gsize) {
    int page[4], s = find(s_rel, A.S, r0);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      page[x] = 0;
      if (r0 + x >= R) continue;
      while (s + 1 < A.S && s_rel[s + 1] <= r0 + x) ++s;
      page[x] = A.table[(int64_t)s * A.max_pages + pages(s_len[s]) + (r0 + x - s_rel[s])];
    }
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (r0 + x < R) A.stack[count + R - 1 - (r0 + x)] = checked(page[x]);  // below N: count + R <= N
  }
  // ---- slots and positions of the new tokens
  if (A.cu)
    for (int s = gtid; s <= A.S; s += gsize) A.cu[s] = s_tok[s];
  if (tokens) {
    // four tokens a thread: one search, a page entry for each page they touch, 16-byte stores
    const int total = A.T ? A.S * A.T : A.cap;
    for (int t0 = 4 * gtid; t0 < total; t0 += 4 * gsize) {
      int slot[4], pos[4];
      int s = A.T ? t0 / A.T : t0 < s_tok[A.S] ? find(s_tok, A.S, t0) : A.S;
      int i = s < A.S ? t0 - (A.T ? s * A.T : s_tok[s]) : 0;
      int held = -1, page = -1;  // page index and page of the token before, if it was of the same request
#pragma unroll
      for (int x = 0; x < 4; ++x, ++i) {
        slot[x] = pos[x] = -1;
        // (requests without tokens are passed over in the packed form)
        while (s < A.S && i >= (A.T ? A.T : s_tok[s + 1] - s_tok[s])) {
          i = 0;
          ++s;
          held = -1;
        }
        if (s >= A.S || t0 + x >= total || (A.T && i >= s_tok[s + 1] - s_tok[s])) continue;
        const int old = s_old[s], at = old + i, p = at >> A.shift, po = pages(old);
        if (p != held) {
          page = p < po ? checked(A.table[(int64_t)s * A.max_pages + p]) : granted(s_gr[s] + p - po);
          held = p;
        }
        if (page >= 0) slot[x] = (page << A.shift) + (at & up);
        pos[x] = old + (A.depth ? A.depth[t0 + x] : i);
      }
      auto store = [&](int32_t* to, const int (&v)[4]) {
        if (t0 + 4 <= total && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
          *reinterpret_cast<int4*>(to + t0) = make_int4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (t0 + x < total) to[t0 + x] = v[x];
        }
      };
      store(A.slots, slot);
      if (A.pos) store(A.pos, pos);
    }
  }

  // ---- the last CTA to get here (every read above is done) writes the new lengths and count
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = gridDim.x == 1 || atomicAdd(&A.state[2], 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (s_last) {
    for (int s = tid; s < A.S; s += kThreads) A.seq_len[s] = s_len[s];
    if (tid == 0) {
      if (fits) A.state[0] = count + R - G;
      A.state[1] = s_refused;
      A.state[2] = 0;
    }
  }
}

bool aligned4(const void* p, bool required) {
  if (!p) return !required;
  return reinterpret_cast<uintptr_t>(p) % 4 == 0;
}

}  // namespace

// Page sizes and pools the paged entry points take: 16 to 128 tokens a page
// (powers of two; a 128-key tile holds whole pages), slots within int32.
msa_status check_page_geometry(int32_t num_pages, int32_t page_size) {
  if (num_pages < 1 || page_size < 1) return MSA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)num_pages * page_size >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_build_page_tables(const msa_page_pool* pool, const int32_t* new_len, const int32_t* depth,
                                            int32_t seq_tokens, int32_t tok_cap, int32_t* cu_new, int32_t* slots,
                                            int32_t* positions, void* stream) {
  if (!pool || pool->n_seqs < 1 || pool->max_pages < 1 || seq_tokens < 0 || tok_cap < 0) return MSA_ERR_INVALID_ARG;
  const msa_status geo = check_page_geometry(pool->num_pages, pool->page_size);
  if (geo != MSA_OK) return geo;
  if (pool->n_seqs > kMaxRequests || (int64_t)pool->max_pages * pool->page_size >= ((int64_t)1 << 31) ||
      (int64_t)pool->n_seqs * seq_tokens >= kMaxTokens || tok_cap >= kMaxTokens)
    return MSA_ERR_UNSUPPORTED;
  if (!aligned4(pool->page_table, true) || !aligned4(pool->seq_len, true) || !aligned4(pool->free_pages, true) ||
      !aligned4(pool->state, true) || !aligned4(new_len, true) || !aligned4(depth, false) ||
      !aligned4(cu_new, false) || !aligned4(slots, false) || !aligned4(positions, false))
    return MSA_ERR_INVALID_ARG;
  if ((positions || depth) && !slots) return MSA_ERR_INVALID_ARG;
  if (new_len == pool->seq_len) return MSA_ERR_INVALID_ARG;  // the lengths change in place while new_len is read
  PageArgs a;
  a.S = pool->n_seqs;
  a.N = pool->num_pages;
  a.shift = __builtin_ctz((unsigned)pool->page_size);
  a.max_pages = pool->max_pages;
  a.T = seq_tokens;
  a.cap = tok_cap;
  a.new_len = new_len;
  a.depth = depth;
  a.table = pool->page_table;
  a.seq_len = pool->seq_len;
  a.stack = pool->free_pages;
  a.state = pool->state;
  a.cu = cu_new;
  a.slots = slots;
  a.pos = positions;
  a.err = device_error_word();
  if (!a.err) return MSA_ERR_CUDA;
  // How many pages move is not known here.  A call with tokens takes about what those need; one without mostly gives
  // back: at most what the tables hold, or the pool.  Four a thread and round: 64 requests of a million tokens are
  // freed in 9.4 us (28.7 us with at most 24 CTAs, 8192 of 1000 tokens in 32 against 45 us); and one CTA (and no
  // ticket) where it can do: a decode step of 64 requests takes 4.3 us, 4.4 us with eight CTAs.
  const int64_t tok = !slots ? 0 : seq_tokens ? (int64_t)a.S * seq_tokens : tok_cap;
  const int64_t held = (int64_t)a.S * a.max_pages < a.N ? (int64_t)a.S * a.max_pages : a.N;
  const int64_t moved = slots ? tok / pool->page_size + a.S : held;
  const int64_t want = (tok / 4 + moved / 4 + kThreads - 1) / kThreads;
  const int grid = (int)(want < 1 ? 1 : want > kMaxCtas ? kMaxCtas : want);
  const int smem = scan_bytes(a.S);
  // The default limit of 48 KB counts the kernel's static bytes too.  It is raised to the same size whatever the call,
  // so that it holds for calls of other sizes from other host threads.
  if (smem + kStaticBytes > 48 * 1024 &&
      cudaFuncSetAttribute(page_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, scan_bytes(kMaxRequests)) !=
          cudaSuccess)
    return MSA_ERR_CUDA;
  page_table_kernel<<<grid, kThreads, smem, (cudaStream_t)stream>>>(a);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
