// What the attentions of drafted tokens over a paged cache share: the line of
// key tiles of all (request, KV head, row block) items, its cut into equal
// parts, what a window leaves of a request, and the kernel that joins the parts
// of the items that were cut.
#pragma once
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "internal.h"
#include "ptx.cuh"
#include "warps.cuh"

namespace msa {

msa_status check_shape(const msa_shape* s);
msa_status check_tree_shape(const msa_shape* s);
msa_status check_page_geometry(int32_t num_pages, int32_t page_size);
float effective_scale(const msa_shape& s);

namespace {

constexpr int kCtas = 152;

struct Cut;

struct TreeArgs {
  int32_t B, Hq, Hkv, n, R, RB, page_shift, max_pages, num_pages, words, q_box, max_parts;
  const int32_t *table, *seq_len, *tree_len;
  const uint32_t* mask;
  int64_t mask_stride;  // words between the masks of two requests (0: one mask for all)
  __nv_bfloat16* o;
  float* lse;
  int32_t* count;   // parts of the line
  Cut* cuts;        // [max_parts] what they cut
  float4* part;     // [2 max_parts][d/4][rows] unnormalised O of the cut items
  float2* part_ml;  // [2 max_parts][rows] their maximum (log2) and row sum
  float scale_log2;
  int* err;
  int32_t sink, window;  // kWin: see msa_tree_window
  const int32_t* depth;  // kWin: [B][n] or null
  int32_t step;  // kWin: drafted tokens of an item if those are consecutive and a chain, else 0
};

// The piece of one item that lies in a part: tiles t0 .. t1 of its `tiles`.
struct Seg {
  int32_t b, kvh, rb, t0, t1, tiles;  // b < 0: no more
  int32_t L, T;
  int32_t r0, r1;  // tiles that its result covers: t0, t1, or more where both groups' segments are joined
};

// The item that a part's beginning cuts, if this is the first cut through it: n parts, the first in slot `first` of
// the workspace, k = 1 .. inner in slots base + step k, another one in `tail`.
struct __align__(16) Cut {
  int32_t n;  // 1 or less: nothing to join
  int32_t b, item, inner, first, base, step, tail;
};

// Keys and drafted tokens of request b; false (nothing to compute) when it has
// none or its numbers break the contract (flagged once by the loader).
__device__ __forceinline__ bool request(const TreeArgs& A, int b, int& L, int& T, bool& bad) {
  L = A.seq_len[b];
  T = A.tree_len ? A.tree_len[b] : A.n;
  bad = T < 0 || T > A.n || L < T || L > ((int64_t)A.max_pages << A.page_shift);
  return !bad && T > 0;
}
__device__ __forceinline__ int key_tiles(int L) { return (L + 127) >> 7; }

// The keys and tiles of a request that some row sees.  Keys hole .. lo - 1 are seen by none (lo <= hole: there are no
// such); tile t of the item's line holds the keys from key0(t) on.  Items of one request have the same number of tiles.
// Where an item is `step` tokens of a chain they are those of its own windows (a chunk of 1024 tokens in items of 256,
// window 1024: 11 tiles an item where the chunk has 17), with what is missing to the number from the keys around them.
struct Span {
  int tiles, head, skip;  // tiles of the line; those of the first tokens, tiles left out behind them
  int hole, lo;
  int all0, all1;  // every row sees the keys from all0 (kWin) up to all1 - 1
  __device__ __forceinline__ int tile(int t) const { return t < head ? t : t + skip; }
  __device__ __forceinline__ int key0(int t) const { return 128 * tile(t); }
  // some row may not see every key of the tile that begins at key0
  template <bool kWin>
  __device__ __forceinline__ bool masked(int key0, int sink) const {
    return key0 + 128 > all1 || (kWin && key0 + 128 > sink && key0 < all0);
  }
  // page p of the request, of 2^shift tokens, holds no key that is seen
  __device__ __forceinline__ bool gone(int p, int shift) const {
    return (int64_t)p << shift >= hole && (int64_t)(p + 1) << shift <= lo;
  }
};
template <bool kWin>
__device__ __forceinline__ Span span_of(const TreeArgs& A, int L, int T, int rb = 0) {
  Span s = {key_tiles(L), 0x7FFFFFFF, 0, 0, 0, 0, L - T};
  if constexpr (kWin) {
    s.hole = min(A.sink, L);
    s.lo = max(0, L - T + 1 - A.window);  // the first row stands at L - T
    s.head = key_tiles(s.hole);
    s.skip = max(0, (s.lo >> 7) - s.head);
    s.tiles -= s.skip;
    int end = A.n;  // the rows lie in front of it
    if (A.step) {
      // window - 1 + step keys, which begin anywhere in a tile, and the first tokens'
      const int most = s.head + (int)((uint32_t)(min(A.window, L) + A.step + 253) >> 7);
      const int i0 = min(A.step * (rb % (A.n / A.step)), T), lo = max(0, L - T + i0 + 1 - A.window);
      s.tiles = min(s.tiles, most);
      s.skip = max(s.skip, min((lo >> 7) - s.head, key_tiles(L) - s.tiles));
      end = i0 + A.step;
      s.all1 = L - T + i0 + 1;  // a chain
    }
    s.all0 = L - T + min(end - A.window, T);
  }
  return s;
}
// Keys sink .. behind(i) - 1 are outside the window of row i of request b.
__device__ __forceinline__ int behind(const TreeArgs& A, int b, int i, int C) {
  const int e = A.depth ? min(max(A.depth[(int64_t)b * A.n + min(i, A.n - 1)], 0), A.n - 1) : i;
  const int end = max(0, C + e + 1 - A.window);
  return A.mask ? min(end, C) : end;
}
// The line of W tiles in G = min(W, max_parts) parts.  CTA c's groups take parts 2 c and 2 c + 1 if there are
// max_parts of them (of two per CTA), else parts c and kCtas + c.
__device__ __forceinline__ int parts(int64_t W, int most) { return W < most ? (int)W : most; }
__device__ __forceinline__ int part_of(int64_t W, int most, int cta, int X) {
  return most > kCtas && W >= most ? 2 * cta + X : cta + kCtas * X;
}
__device__ __forceinline__ int64_t part_begin(int64_t W, int most, int p) { return W < most ? p : W * p / most; }

// kPairs (two parts a CTA), all of them present: the odd part of a CTA that lies within one item [s0, s1) which its even part reaches too
// is joined with it in the CTA.
__device__ __forceinline__ bool joined_in_cta(bool many, int64_t W, int most, int p, int64_t s0, int64_t s1) {
  return many && W >= most && (p & 1) && part_begin(W, most, p) > s0 && part_begin(W, most, p + 1) <= s1;
}

// a / b for a >= 0, b > 0, in 32 bits where they suffice (64-bit division takes some hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// What the beginning of part p cuts, which lies in request b, whose tiles begin at `at`.
template <bool kPairs, int kMost, bool kWin>
__device__ void note_cut(const TreeArgs& A, int64_t W, int p, int b, int64_t at) {
  const int64_t lo = part_begin(W, kMost, p);
  const int tiles = span_of<kWin>(A, A.seq_len[b], A.tree_len ? A.tree_len[b] : A.n).tiles;
  const int64_t item = quotient(lo - at, tiles), s0 = at + item * tiles, s1 = s0 + tiles;
  Cut c = {0, b, (int32_t)item, 0, 0, 0, 0, 0};
  if (lo > s0 && part_begin(W, kMost, p - 1) <= s0) {
    // kPairs, all parts present: an odd part that was joined in its CTA stands in the slot of the even one; only the
    // first and the last part of an item can be odd and not
    const bool pairs = kPairs && W >= kMost;
    const int c0 = p - 1, c1 = (int)quotient(s1 * parts(W, kMost) - 1, W);  // the largest part that begins below s1
    const int lead = pairs && !(c0 & 1) ? 2 : 1;
    const bool tail = pairs && (c1 & 1) && c1 != c0 && !joined_in_cta(true, W, kMost, c1, s0, s1);
    c.step = pairs ? 2 : 1;
    c.inner = c0 + lead <= c1 ? (c1 - c0 - lead) / c.step + 1 : 0;
    c.n = 1 + c.inner + (tail ? 1 : 0);
    c.first = 2 * c0 + 1;
    c.base = 2 * (c0 + lead - c.step);
    c.step *= 2;
    c.tail = 2 * c1;
  }
  A.cuts[p] = c;
}

// Joins the parts of the items that the line's cuts went through, in a fixed
// order.  Latency bounds it where there is little to join, and else what the parts
// hold (up to 40 MB, in the L2).  There are fewer cuts than parts, so each CTA looks
// through all of them (those that are the first through their item stand for it)
// and takes its share of the cut items' chunks, however many items there are; with
// a grid over the items most CTAs find nothing to do: 152 requests of 1072 tokens
// with 192 rows 167 us so, 211 us with it.
//   kShare = 1: a thread takes 16 columns of a row, two parts in flight, a chunk is
//     a warp's width of those;
//   kShare = 8, where items have four parts or more each and about every chunk has an
//     idle CTA: 8 columns, the eight warps of a CTA divide a chunk's parts, four in
//     flight each (one request of 5000 tokens in 38 parts a head: 18 us, 26 us with
//     kShare = 1; with more chunks than four an SM, 4 requests with 64 rows over 8000
//     tokens, 36 us, 33 us with kShare = 1).
constexpr int kJoinThreads = 256, kJoinPerSm = 3;
constexpr int join_cols(int share) { return share > 1 ? 8 : 16; }

template <int D, int kMost, int kBlock, int kShare>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) tree_join_kernel(const TreeArgs A) {
  constexpr int kWarps = kJoinThreads / 32, kWords = (kMost + 31) / 32;
  constexpr int kCols = join_cols(kShare), kAhead = kShare > 1 ? 4 : 2;
  static_assert(kShare == 1 || kShare == kWarps, "a chunk per warp or CTA");
  __shared__ unsigned found[kWords];
  __shared__ float joined[kShare][kCols + 2][32];  // (kShare = 1: unused)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int full = min(kBlock, A.R), chunks = (full * (D / kCols) + 31) / 32;
  const int G = *A.count;
  for (int x = warp; x < kWords; x += kWarps) {
    const int p = 32 * x + lane, n = A.cuts[min(p, kMost - 1)].n;
    const unsigned f = __ballot_sync(0xFFFFFFFFu, p < G && n > 1);  // (behind G: of another call)
    if (lane == 0) found[x] = f;
  }
  __syncthreads();
  const int first = blockIdx.x + (kShare > 1 ? 0 : warp * gridDim.x), step = gridDim.x * (kWarps / kShare);
  for (int u = first;; u += step) {
    // the cut that stands for this chunk's item
    int left = u / chunks, p = -1;
    const int e = 32 * (u - left * chunks) + lane;
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      const unsigned f = found[x];
      const int here = __popc(f);
      if (left >= 0 && left < here) {
        const bool mine = (f >> lane & 1u) && __popc(f & ((1u << lane) - 1u)) == left;
        p = 32 * x + __ffs(__ballot_sync(0xFFFFFFFFu, mine)) - 1;
      }
      left -= here;
    }
    if (p < 0) return;  // no more
    const Cut it = A.cuts[p];
    const int rb = it.item % A.RB, kvh = it.item / A.RB;
    const int width = min(kBlock, A.R - kBlock * rb);
    const int c = e / width, rw = e - c * width, rr = kBlock * rb + rw;  // group of columns, row of the block
    const bool there = e < width * (D / kCols);
    const int T = A.tree_len ? A.tree_len[it.b] : A.n;
    const float2* ml = A.part_ml + rw;
    const float4* part = A.part + (int64_t)(kCols / 4 * c) * width + rw;
    float m = -INFINITY, l = 0.f, o[kCols];
#pragma unroll
    for (int x = 0; x < kCols; ++x) o[x] = 0.f;
    if (there)
      for (int y0 = kShare > 1 ? warp : 0; y0 < it.n; y0 += kAhead * kShare) {
        float2 state[kAhead];
        float4 v[kAhead][kCols / 4];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int y = y0 + k * kShare;
          state[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int x = 0; x < kCols / 4; ++x) v[k][x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (y < it.n) {
            const int64_t slot = y == 0 ? it.first : y <= it.inner ? it.base + it.step * y : it.tail;
            state[k] = ml[slot * full];
#pragma unroll
            for (int x = 0; x < kCols / 4; ++x) v[k][x] = part[slot * (D / 4) * full + x * width];
          }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) top = fmaxf(top, state[k].x);
        const float ref = top == -INFINITY ? 0.f : top, keep = ex2(m - ref);
        m = top;
        l *= keep;
#pragma unroll
        for (int x = 0; x < kCols; ++x) o[x] *= keep;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const float w = ex2(state[k].x - ref);
          l += w * state[k].y;
#pragma unroll
          for (int x = 0; x < kCols / 4; ++x) {
            o[4 * x] += w * v[k][x].x;
            o[4 * x + 1] += w * v[k][x].y;
            o[4 * x + 2] += w * v[k][x].z;
            o[4 * x + 3] += w * v[k][x].w;
          }
        }
      }
    if (kShare > 1) {
      joined[warp][0][lane] = m;
      joined[warp][1][lane] = l;
#pragma unroll
      for (int x = 0; x < kCols; ++x) joined[warp][2 + x][lane] = o[x];
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int k = 1; k < kShare; ++k) m = fmaxf(m, joined[k][0][lane]);
        const float ref = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int x = 0; x < kCols; ++x) o[x] = 0.f;
#pragma unroll
        for (int k = 0; k < kShare; ++k) {
          const float w = ex2(joined[k][0][lane] - ref);
          l += w * joined[k][1][lane];
#pragma unroll
          for (int x = 0; x < kCols; ++x) o[x] += w * joined[k][2 + x][lane];
        }
      }
      __syncthreads();
    }
    if ((kShare > 1 && warp > 0) || !there || rr % A.n >= T) continue;  // (rows not drafted: parts hold anything)
    const bool some = !(l == 0.f);
    const float inv = some ? 1.f / l : 0.f;
    const int64_t grow = (int64_t)(it.b * A.Hq + kvh * (A.Hq / A.Hkv)) * A.n + rr;
    uint32_t w[kCols / 2];
#pragma unroll
    for (int x = 0; x < kCols / 2; ++x) w[x] = pack_bf16x2(o[2 * x] * inv, o[2 * x + 1] * inv);
    __nv_bfloat16* dst = A.o + grow * D + kCols * c;
#pragma unroll
    for (int x = 0; x < kCols / 2; x += 4)
      *reinterpret_cast<uint4*>(dst + 2 * x) = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
    if (c == 0 && A.lse) A.lse[grow] = some ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

bool aligned(const void* p, size_t a, bool required) {
  if (!p) return !required;
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// TreeArgs::step for items of `rows` rows.
int32_t chain_step(const TreeArgs& a, int rows) { return !a.mask && a.n % rows == 0 ? rows : 0; }

bool window_ok(const msa_tree_window* w, const uint32_t* mask) {
  return w->sink >= 0 && w->window >= 1 && aligned(w->depth, 4, false) && (!w->depth || mask);
}

// Behind the attention kernel on its stream; starts while that still runs.
template <int D, int kMost, int kBlock>
msa_status launch_join(const TreeArgs& a, cudaStream_t stream) {
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  const int full = a.R < kBlock ? a.R : kBlock;
  const int64_t items = (int64_t)a.B * a.Hkv * a.RB, most = items < a.max_parts ? items : a.max_parts - 1;  // cut ones
  const int64_t split = items * ceil_div((int64_t)full * (D / join_cols(8)), 32);  // chunks, if their parts are divided
  const bool share = 4 * items <= a.max_parts && split <= 4 * kCtas;
  // (kShare = 1 has a chunk per warp, but few chunks go to all SMs first)
  const int64_t ctas = share ? split : most * ceil_div((int64_t)full * (D / join_cols(1)), 32);
  cfg.gridDim = dim3((unsigned)(ctas < kJoinPerSm * kCtas ? ctas : kJoinPerSm * kCtas));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((share ? cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kMost, kBlock, 8>, a)
             : cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kMost, kBlock, 1>, a)) != cudaSuccess)
    return MSA_ERR_CUDA;
  note_launch();
  return MSA_OK;
}

}  // namespace

}  // namespace msa
