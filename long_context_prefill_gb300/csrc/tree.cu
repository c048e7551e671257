// Attention of drafted tokens over a paged KV cache (decode, speculative
// trees), sm_103a.
//
// What it computes: request b holds L = seq_len[b] keys in its pages, the last
// T of them drafted tokens.  Row i < T of every query head attends the L - T
// context keys and the drafted keys that its mask names (none given: j <= i):
//   o_i = Σ_j e^{s_ij} v_j / Σ_j e^{s_ij},  s_ij = scale q_i . k_j.
//
// What bounds it: HBM.  A KV head's keys serve the g = Hq / Hkv query heads of
// its group for all n drafted tokens, R = g n rows, so each byte of K and V
// meets R multiply-adds: below about 280 rows (1925 TFLOP/s over 6.8 TB/s)
// the cache cannot be read as fast as the tensor core would multiply.  So the
// rows of a group sit together in one or two 128-row MMA tiles (row r = head r / n,
// token r % n: contiguous in Q's layout) and every K/V tile is loaded once for
// all of them, rows that do not exist costing nothing but idle lanes.
//
// Split.  The tiles of 128 keys of all (request, KV head, 256-row block) items
// form one line, cut into equal parts, one per softmax group (below): no group
// has more than one tile above another's, whatever the lengths.  An item that
// lies in one part is finished there; of one that is cut, each part leaves its
// unnormalised sum, maximum and row sum in the workspace, and a second kernel
// (launched early, waiting for the first) joins them in key order, so results
// do not depend on timing.
//
// A CTA (12 warps, kMany 16 of which three have no task; one CTA per SM):
//   warp 10    loader of group 0's part (kTwo: of the CTA's) and one more warp for
//              group 1's: walk its segments, publish their descriptors, load Q
//              rows and the K and V pages of every tile by TMA into one ring (K
//              and V tiles alternate; the two parts' tiles take turns);
//   warp 8     waits for the ring's tiles one after another and declares each
//              ready; in a request's last V tile it first zeroes the rows past
//              the end: pages may hold anything there, and a weight of zero
//              does not hide an infinity or NaN in an MMA.  (The order matters:
//              loads land in any order, and an issuer that skips a tile must
//              not take the phase of a slot's earlier use for the one it waits
//              for.  With declarations in order, the tile it saw last proves
//              every earlier use of the slot over);
//   warps 9/11 MMA issuers;
//   warps 0-7  softmax groups X = 0, 1 (4 warps each, thread = row = TMEM lane).
// Three row layouts (Rows):
//   kFew   up to 64 rows: the groups work on parts of their own; group 1 has its
//          rows in TMEM lanes 64 .., so that the groups' warps sit on different
//          schedulers, and Q is double-buffered.  A group's chain (scores,
//          softmax, values) takes longer than a tile takes out of HBM; two
//          chains side by side do not;
//   kMany  up to 128 rows: the same with all lanes and one Q buffer a group;
//   kTwo   above: one part per CTA, group X owns rows 128 X .. of the 256-row
//          block, and both use every tile.  One warp issues the scores of both,
//          one the products with V; the scores of a group go to one shared TMEM
//          tile that is free again once they are in its registers, so a group's
//          next scores do not wait for its product with V.
//
// Measured (captured, 32 / 8 heads of 128): decode of 64 requests of 1K to 16K
// tokens 188 to 191 us (6.7 TB/s, 0.98 of the measured copy rate), of 256 requests
// of 100 to 1000 tokens 76.5 us (floor 58), a million-token context with 5 drafted
// tokens 585 us (7.3 TB/s), 128K with a tree of 32 (128 rows) 88 to 90 us (0.89 of
// the floor), 16 trees of up to 48 (192 rows) over 4K to 32K 164 us (0.73); one
// request of 2047 tokens with 2 / 1 heads of 64 10 us (two kernels' latency).  kTwo
// takes 1.70 us a tile (1.47 at HBM speed): the groups' scores go through one TMEM
// tile in turn, 560 to 1000 cycles from the reading of one's to the issue of the
// other's and 950 to compute them (1400 where a product with V runs beside).  Tried
// and slower there (against 162 to 174 us): a score tile per group with P over it
// 194 us, turns of the groups on a scheduler 192 to 253 us, scores by halves of 64
// keys 208 us, products held back while scores are computed 175 us.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace msa {

msa_status check_shape(const msa_shape* s);
msa_status check_page_geometry(int32_t num_pages, int32_t page_size);
float effective_scale(const msa_shape& s);

namespace {

constexpr int kCtas = 152;
constexpr int kCleanWarp = 8, kMmaWarp0 = 9, kLoaderWarp = 10, kMmaWarp1 = 11;
constexpr int kSegSlots = 3;
enum Rows { kFew = 0, kMany = 1, kTwo = 2 };
constexpr int threads_of(Rows r) { return r == kMany ? 512 : 384; }
constexpr uint32_t kTmemCols = 512;
// TMEM columns.  kFew, kMany: S of group X at 128 X, P over its first 64.
// kTwo: one S that the groups use in turn, P of group X at 128 + 64 X.  O of
// group X at 256 + 128 X.
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kPChunk = 4;
constexpr uint32_t kIdleNs = 64;
constexpr uint64_t kDrainNs = MSA_WAIT_LIMIT_NS / 16;  // a CTA that gave up: for each copy and product in flight
constexpr int kMaxDrafts = 1024;

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
};

struct TreeMaps {
  CUtensorMap q, k, v;  // [rows, d] views, boxes of 64 columns x q_box rows (q), x page_size rows (k, v)
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

// Barriers; [X]: per group (kTwo: segments and Q once, at X = 0)
enum {
  kBarQFull = 0,                         // [X][2 buffers]
  kBarQEmpty = 4,                        // [X][2]
  kBarSFull = 8,                         // [X] scores are in TMEM
  kBarPFull = 10,                        // [X] weights are in TMEM
  kBarODone = 12,                        // [X] every product of the segment is done (kTwo: of a group without rows)
  kBarOFree = 14,                        // [X] O of the segment has been read
  kBarPV = 16,                           // [X] kTwo: the group's last P has been used
  kBarSFree = 18,                        // kTwo: the scores are in registers
  kBarML = 19,                           // kMany: both groups' maxima and sums are written
  kBarDrain = 20,                        // [issuer] after giving up: its products are done
  kBarSegFull = 22,                      // [X][kSegSlots]
  kBarSegEmpty = kBarSegFull + 2 * kSegSlots,
  kBarRing = kBarSegEmpty + 2 * kSegSlots  // full[kSlots], empty[kSlots], ready[kSlots]
};

template <int D>
struct Lay {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kSlots = 5 * (128 / D);
  static constexpr int kQ = 0;  // two Q tiles, one per group (kFew: of two 64-row buffers)
  static constexpr int kRing = 2 * kTile;
  static constexpr int kSeg = kRing + kSlots * kTile;
  static constexpr int kML = kSeg + 2 * kSegSlots * (int)sizeof(Seg);  // kMany: [2][128] maximum and row sum
  static constexpr int kBars = kML + 2 * 128 * 8;
  static constexpr int kNumBars = kBarRing + 3 * kSlots;
  static constexpr int kMisc = kBars + kNumBars * 8;  // [0] TMEM base, [2] abort, [4 + X] tiles loaded, [6 + X] Q's asked for
  static constexpr int kStart = kMisc + 32;           // [X][2] int64: request in which a part begins, its first tile
  static constexpr int kLast = kStart + 32;           // [X][kSlots] the last ring load of loader X into a slot, -1: none
  static constexpr int kAlloc = kLast + 2 * kSlots * 4;
  static_assert(kStart % 8 == 0 && kML % 8 == 0, "int64 in shared memory");
  static_assert(kAlloc <= 227 * 1024 && kAlloc > 120 * 1024, "shared memory: one CTA per SM");
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
// The line of W tiles in G = min(W, max_parts) parts.  CTA c's groups take parts 2 c and 2 c + 1 if there are
// max_parts of them (of two per CTA), else parts c and kCtas + c.
__device__ __forceinline__ int parts(int64_t W, int most) { return W < most ? (int)W : most; }
__device__ __forceinline__ int part_of(int64_t W, int most, int cta, int X) {
  return most > kCtas && W >= most ? 2 * cta + X : cta + kCtas * X;
}
__device__ __forceinline__ int64_t part_begin(int64_t W, int most, int p) { return W < most ? p : W * p / most; }

// kMany, all parts present: the odd part of a CTA that lies within one item [s0, s1) which its even part reaches too
// is joined with it in the CTA.
__device__ __forceinline__ bool joined_in_cta(bool many, int64_t W, int most, int p, int64_t s0, int64_t s1) {
  return many && W >= most && (p & 1) && part_begin(W, most, p) > s0 && part_begin(W, most, p + 1) <= s1;
}

// a / b for a >= 0, b > 0, in 32 bits where they suffice (64-bit division takes some hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// What the beginning of part p cuts, which lies in request b, whose tiles begin at `at`.
template <Rows kRows, int kMost>
__device__ void note_cut(const TreeArgs& A, int64_t W, int p, int b, int64_t at) {
  const int64_t lo = part_begin(W, kMost, p);
  const int tiles = key_tiles(A.seq_len[b]);
  const int64_t item = quotient(lo - at, tiles), s0 = at + item * tiles, s1 = s0 + tiles;
  Cut c = {0, b, (int32_t)item, 0, 0, 0, 0, 0};
  if (lo > s0 && part_begin(W, kMost, p - 1) <= s0) {
    // kMany, all parts present: an odd part that was joined in its CTA stands in the slot of the even one; only the
    // first and the last part of an item can be odd and not
    const bool pairs = kRows == kMany && W >= kMost;
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

template <int D, Rows kRows>
__global__ void __launch_bounds__(threads_of(kRows), 1)
    tree_attn_kernel(const __grid_constant__ TreeMaps M, const TreeArgs A) {
  using Ly = Lay<D>;
  constexpr bool kPair = kRows == kTwo;
  constexpr int kThreads = threads_of(kRows);
  // Each group's part has a loader of its own (kFew: the second one is a softmax warp without rows): opening a segment
  // (lengths, division, page entries, Q) takes one about 3000 cycles, a tile's boxes up to 1700, and short requests
  // need both every other tile.  With one loader for both parts 256 requests of 100 to 1000 tokens take 81 us instead
  // of 77 (16-token pages 83 instead of 77), 512 of 20 to 400 tokens 93 instead of 86, long ones the same.
  constexpr int kLoaderWarp1 = kRows == kFew ? 2 : 12;
  constexpr int kSlots = Ly::kSlots;
  constexpr int kMost = kPair ? kCtas : 2 * kCtas;  // parts (A.max_parts)
  constexpr int kGroupWarps = kRows == kFew ? 2 : 4;
  constexpr int kSegReaders = kPair ? 11 : kGroupWarps + 2;  // softmax warps, issuer(s), the cleaner
  constexpr int kQBufs = kRows == kFew ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t sm[];  // swizzled tiles start on 1 KB
  if (smem_u32(sm) & 1023) {
    if (threadIdx.x == 0) atomicCAS(A.err, 0, (int)kErrTimeout);
    if (blockIdx.x == 0 && threadIdx.x == 0) *A.count = 0;  // nothing to join
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::kBars);
  uint64_t* bFull = bars + kBarRing;
  uint64_t* bEmpty = bFull + kSlots;
  uint64_t* bReady = bEmpty + kSlots;
  Seg* segs = reinterpret_cast<Seg*>(sm + Ly::kSeg);  // [2][kSegSlots]
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + Ly::kMisc);
  volatile int* lasts = reinterpret_cast<volatile int*>(sm + Ly::kLast);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    tmem_alloc(const_cast<uint32_t*>(&misc[0]), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * kLoaderWarp) {
    tma_prefetch_desc(&M.q);
    tma_prefetch_desc(&M.k);
    tma_prefetch_desc(&M.v);
  }
  if (threadIdx.x == 32 * kMmaWarp0) {
    for (int x = 0; x < 4; ++x) {
      mbar_init(&bars[kBarQFull + x], 1);
      mbar_init(&bars[kBarQEmpty + x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[kBarSFull + x], 1);
      mbar_init(&bars[kBarPFull + x], kGroupWarps);
      mbar_init(&bars[kBarODone + x], 1);
      mbar_init(&bars[kBarOFree + x], kGroupWarps);
      mbar_init(&bars[kBarPV + x], 1);
      mbar_init(&bars[kBarDrain + x], 1);
    }
    mbar_init(&bars[kBarSFree], 4);
    mbar_init(&bars[kBarML], 8);
    for (int s = 0; s < 2 * kSegSlots; ++s) {
      mbar_init(&bars[kBarSegFull + s], 1);
      mbar_init(&bars[kBarSegEmpty + s], kSegReaders);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bFull[s], 1);
      mbar_init(&bEmpty[s], 1);
      mbar_init(&bReady[s], 1);
    }
    misc[2] = misc[4] = misc[5] = 0;
    fence_mbar_init();
  }
  // ---- this CTA's parts of the line of tiles, and the requests they start in
  const int items = A.Hkv * A.RB;  // items of a request
  // The warps' sums lie where kMany's maxima and sums come at the end: they are read before the __syncthreads below, and
  // those are written by the roles behind it.  `start` is read by the loaders and the cleaner as they begin, and group 0
  // may have its maxima while the loader of group 1 has not begun yet: it has bytes of its own.
  int64_t* wsum = reinterpret_cast<int64_t*>(sm + Ly::kML);
  int64_t* start = reinterpret_cast<int64_t*>(sm + Ly::kStart);
  int64_t W = 0;                                               // all tiles
  {
    const int per = (A.B + kThreads - 1) / kThreads;
    const int b0 = min(A.B, (int)threadIdx.x * per), b1 = min(A.B, b0 + per);
    auto tiles = [&](int b) -> int64_t {
      int L, T;
      bool bad;
      const bool live = request(A, b, L, T, bad);
      if (bad && blockIdx.x == 0) atomicCAS(A.err, 0, (int)kErrIndex);
      return live ? (int64_t)items * key_tiles(L) : 0;
    };
    int64_t own = 0, mine = 0;  // of the last request, of all of this thread's
    for (int b = b0; b < b1; ++b) mine += own = tiles(b);
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int64_t base = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += wsum[w];
      W += wsum[w];
    }
    int64_t at = base + inc - mine;
    for (int b = b0; b < b1; ++b) {
      const int64_t t = per == 1 ? own : tiles(b);
#pragma unroll
      for (int X = 0; X < (kPair ? 1 : 2); ++X) {
        const int64_t lo = part_begin(W, kMost, part_of(W, kMost, blockIdx.x, X));  // at or above W: no part
        if (at <= lo && lo < at + t) { start[2 * X] = b; start[2 * X + 1] = at; }
      }
      at += t;
    }
  }
  const int G = parts(W, kMost);
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.count = G;
  // tiles of this CTA's parts; tile k of group X is tile turn(X, k) of the ring (the parts' tiles take turns)
  int64_t begin[2] = {0, 0};
  int cnt[2] = {0, 0};
#pragma unroll
  for (int X = 0; X < (kPair ? 1 : 2); ++X) {
    const int p = part_of(W, kMost, blockIdx.x, X);
    if (p < G) {
      begin[X] = part_begin(W, kMost, p);
      cnt[X] = (int)(part_begin(W, kMost, p + 1) - begin[X]);
    }
  }
  const int both = min(cnt[0], cnt[1]);
  auto turn = [&](int X, int k) { return kPair ? k : k < both ? 2 * k + X : both + k; };
  auto owner = [&](int j) { return kPair ? 0 : j < 2 * both ? j & 1 : cnt[0] > cnt[1] ? 0 : 1; };
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if ((int)blockIdx.x >= G) {  // no part
    if (warp == 0) tmem_dealloc(misc[0], kTmemCols);
    return;
  }
  const uint32_t tmem = misc[0];

  // Segment s of group X's part as its readers see it; false: no more, or gave up.
  bool ok = true;
  auto next_seg = [&](int X, int s, Seg& g) -> bool {
    const int slot = (kPair ? 0 : X * kSegSlots) + s % kSegSlots;
    if (misc[2] || !mbar_wait(&bars[kBarSegFull + slot], (s / kSegSlots) & 1)) { ok = false; return false; }
    g = segs[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBarSegEmpty + slot]);
    return g.b >= 0;
  };
  auto ready = [&](int idx) { return mbar_wait(&bReady[idx % kSlots], (idx / kSlots) & 1); };
  // Q of group X, buffer buf.  The MMA reads 128 rows from 64 X above it in kFew (group 1's rows come to lanes 64 ..);
  // rows that are not the group's hold anything and only reach their own lanes.
  auto q_at = [&](int X, int buf) { return Ly::kQ + X * Ly::kTile + buf * 8192; };
  constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
  constexpr uint64_t kTileDesc = Ly::kTile >> 4;
  auto q_desc = [&](int X, int buf) {
    return sdesc_sw128(smem_u32(sm + q_at(X, buf)) - (kRows == kFew ? 8192u * X : 0u), 16, 1024);
  };
  const uint64_t dk = sdesc_sw128(smem_u32(sm + Ly::kRing), 16, 1024);     // + slot * kTileDesc
  const uint64_t dv = sdesc_sw128(smem_u32(sm + Ly::kRing), 16384, 1024);
  auto issue_qk = [&](uint32_t d, uint64_t q0, uint64_t k0) {  // S = Q K^T of one tile, by one thread
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);
      mma_bf16_ss(d, q0 + off, k0 + off, id_qk, kk > 0 ? 1u : 0u);
    }
  };
  auto issue_pv_mma = [&](uint32_t d, uint32_t p, uint64_t v0, bool first) {  // O (+)= P V
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      mma_bf16_ts(d, p + 8 * kk, v0 + (uint64_t)(kk * 128), id_pv, (!first || kk > 0) ? 1u : 0u);
  };
  // rows of softmax group X in the 256-row block rb
  auto group_rows = [&](int rb, int X) { return min(128, A.R - 256 * rb - (kPair ? 128 * X : 0)); };

  // kTwo: the block starts with 3 x 128 threads x 168 registers; the softmax threads (a row's 128 scores each) take
  // 192 and the others 120: 2 x 192 + 120 = 3 x 168
  if (warp >= 8 || (kRows == kFew && warp == kLoaderWarp1)) {
    if (kPair) asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
    if (warp == kLoaderWarp || (!kPair && warp == kLoaderWarp1)) {
      // ---------------------------------------------------------- loader of group X's part (kTwo: of the CTA's)
      const int X = warp == kLoaderWarp ? 0 : 1;
      const uint64_t policy = A.RB == 1 ? policy_evict_first() : policy_evict_last();
      const int pshift = 7 - A.page_shift, pp = 1 << pshift;  // pages of a tile
      const int P = 1 << A.page_shift;
      const int count = X ? cnt[1] : cnt[0];
      int64_t at = start[2 * X + 1], pos = X ? begin[1] : begin[0];  // first tile of request b, of the next segment
      const int64_t hi = pos + count;                                // the part's end
      int b = (int)start[2 * X], s = 0, t = 0;        // request, segments so far, next tile of the segment
      int last = -1, asked = 0;  // the last ring load into slot `lane`; segments whose Q was asked for
      Seg g;
      int base, ids, ahead;  // lane x holds the page of entry base + x, and of base + 32 + x
      auto publish = [&](const Seg& g) -> bool {
        const int slot = X * kSegSlots + s % kSegSlots;
        if (misc[2] || !mbar_wait_idle(&bars[kBarSegEmpty + slot], ((s / kSegSlots) & 1) ^ 1, kIdleNs)) return false;
        if (lane == 0) {
          segs[slot] = g;
          mbar_arrive(&bars[kBarSegFull + slot]);
        }
        return true;
      };
      auto entry = [&](const Seg& g, int p) {
        return p < (g.L + P - 1) >> A.page_shift ? A.table[(int64_t)g.b * A.max_pages + p] : 0;
      };
      auto checked = [&](int page) {
        if ((unsigned)page < (unsigned)A.num_pages) return page;
        atomicCAS(A.err, 0, (int)kErrIndex);  // skipped: an existing page stands in, the call has failed
        return 0;
      };
      // The next segment: its descriptor, its Q rows, its first page entries.
      auto open = [&]() -> bool {
        bool bad;
        int64_t tiles = 0;
        for (; b < A.B; ++b) {  // pos < hi <= W: a request holding it exists
          tiles = request(A, b, g.L, g.T, bad) ? (int64_t)items * key_tiles(g.L) : 0;
          if (pos < at + tiles) break;
          at += tiles;
        }
        if (b >= A.B) return false;
        g.b = b;
        g.tiles = key_tiles(g.L);
        const int item = (int)quotient(pos - at, g.tiles);
        g.kvh = item / A.RB;
        g.rb = item - g.kvh * A.RB;
        g.t0 = (int)(pos - at - (int64_t)item * g.tiles);
        const int64_t left = hi - pos;
        g.t1 = left < g.tiles - g.t0 ? g.t0 + (int)left : g.tiles;
        g.r0 = g.t0;
        g.r1 = g.t1;
        if (kRows == kMany) {
          const int64_t i0 = at + (int64_t)item * g.tiles;
          const int p = part_of(W, kMost, blockIdx.x, 1);
          // (of the even part only its last segment reaches the item)
          if (joined_in_cta(true, W, kMost, p, i0, i0 + g.tiles)) {
            g.r0 = (int)max((int64_t)0, begin[0] - i0);
            g.r1 = (int)(begin[1] + cnt[1] - i0);
          }
        }
        pos += g.t1 - g.t0;
        t = g.t0;
        base = g.t0 << pshift;
        ids = entry(g, base + lane);  // on their way until the Q rows are
        ahead = entry(g, base + 32 + lane);
        if (!publish(g)) return false;
        const int buf = s % kQBufs;
        if (!mbar_wait_idle(&bars[kBarQEmpty + 2 * X + buf], ((s / kQBufs) & 1) ^ 1, kIdleNs)) return false;
        const int rows = min(kPair ? 256 : 128, A.R - 256 * g.rb), boxes = (rows + A.q_box - 1) / A.q_box;
        uint64_t* full = &bars[kBarQFull + 2 * X + buf];
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(boxes * A.q_box * D * 2));
        ++asked;
        __syncwarp();
        const int qrow = (g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + 256 * g.rb;
        if (lane < boxes * (D / 64)) {  // at most 8
          const int c = lane & (D / 64 - 1), r = lane / (D / 64) * A.q_box;
          uint8_t* to = sm + q_at(kPair ? r >> 7 : X, buf) + c * 16384 + (r & 127) * 128;
          tma_load_3d(to, &M.q, full, 64 * c, qrow + r, 0);
        }
        ++s;
        ids = checked(ids);
        ahead = checked(ahead);
        return true;
      };
      // Before a slot's wait: the use of the slot before is loaded, if that is the other loader's task, so that the
      // phase waited for is of that use and not of the one before it.
      auto loaded = [&](int idx) -> bool {
        const int j = idx >> 1;
        if (kPair || idx < 0 || owner(j) == X) return true;
        const int k = j < 2 * both ? j >> 1 : j - both;  // the other's tile
        if ((int)misc[4 + (X ^ 1)] > k) return true;
        const uint64_t since = global_timer_ns();
        while ((int)misc[4 + (X ^ 1)] <= k)
          if (misc[2] || global_timer_ns() - since > MSA_WAIT_LIMIT_NS) return false;
        return true;
      };
      // the part's tile k
      auto step = [&](int k) -> bool {
        if ((s == 0 || t == g.t1) && !open()) return false;
        int off = (t << pshift) - base;
        if (off >= 32) {
          base += 32;
          off -= 32;
          ids = ahead;
          ahead = checked(entry(g, base + 32 + lane));
        }
        const int np = (g.L + P - 1) >> A.page_shift;
        const int boxes = min(pp, np - (t << pshift)) * (D / 64);  // pages of this tile that hold keys, by 64 columns
        const int c = lane & (D / 64 - 1), x = lane / (D / 64);
        const int krow = (__shfl_sync(0xFFFFFFFFu, ids, (off + x) & 31) * A.Hkv + g.kvh) << A.page_shift;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v) {
          const int idx = 2 * turn(X, k) + is_v, st = idx % kSlots;
          if (misc[2] || !loaded(idx - kSlots)) return false;
          if (!mbar_wait_idle(&bEmpty[st], ((idx / kSlots) & 1) ^ 1, kIdleNs)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&bFull[st], (uint32_t)(boxes * P * 128));
          __syncwarp();
          last = lane == st ? idx : last;
          if (lane < boxes)
            tma_load_3d_hint(sm + Ly::kRing + st * Ly::kTile + c * 16384 + x * P * 128, is_v ? &M.v : &M.k, &bFull[st],
                             64 * c, krow, 0, policy);
        }
        __syncwarp();
        if (!kPair && lane == 0) misc[4 + X] = k + 1;
        ++t;
        return true;
      };
      for (int k = 0; k < count && ok; ++k) ok = step(k);
      Seg end;
      end.b = -1;
      if (ok) ok = publish(end);
      if (lane < kSlots) lasts[X * kSlots + lane] = last;
      if (lane == 0) misc[6 + X] = asked;
    } else if (warp == kCleanWarp) {
      // ---------------------------------------------------------- tiles in order, rows past a request's end
      struct Walk {
        int b_end, L, t, s;  // end of the segment, keys of its request, next tile, segments so far
      };
      Walk w = {0, 0, 0, 0}, other = {0, 0, 0, 0};
      int X = 0;
      if (lane < 2 && (lane ? cnt[1] : cnt[0]) > 0)  // what the parts cut, for the second kernel
        note_cut<kRows, kMost>(A, W, part_of(W, kMost, blockIdx.x, lane), (int)start[2 * lane], start[2 * lane + 1]);
      for (int j = 0; j < cnt[0] + cnt[1] && ok; ++j) {
        if (owner(j) != X) {
          const Walk t = w;
          w = other;
          other = t;
          X ^= 1;
        }
        if (w.t == w.b_end) {
          Seg g;
          if (!next_seg(X, w.s++, g)) { ok = false; break; }
          w.t = g.t0;
          w.b_end = g.t1;
          w.L = g.L;
        }
        const int keys = w.L - 128 * w.t++;
#pragma unroll 1
        for (int idx = 2 * j; idx < 2 * j + 2; ++idx) {
          const int st = idx % kSlots;
          if (misc[2] || !mbar_wait(&bFull[st], (idx / kSlots) & 1)) { ok = false; break; }
          if ((idx & 1) && keys < 128) {
            uint8_t* v = sm + Ly::kRing + st * Ly::kTile;
#pragma unroll 1
            for (int x = keys * 8 + lane; x < 1024; x += 32)
#pragma unroll
              for (int c = 0; c < D / 64; ++c)
                *reinterpret_cast<uint4*>(v + c * 16384 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&bReady[st]);
        }
      }
    } else if (kPair && warp == kMmaWarp0) {
      // ------------------------------------------------------------ scores of both groups
      int tile = 0, use = 0;  // tiles so far, uses of S so far
      Seg g;
      for (int s = 0; next_seg(0, s, g); ++s) {
        if (!mbar_wait(&bars[kBarQFull], s & 1)) { ok = false; break; }
        for (int t = g.t0; t < g.t1 && ok; ++t, ++tile) {
          const int kst = 2 * tile % kSlots;
          if (misc[2] || !ready(2 * tile)) { ok = false; break; }
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (group_rows(g.rb, X) <= 0) continue;
            if (use > 0 && !mbar_wait(&bars[kBarSFree], (use - 1) & 1)) { ok = false; break; }
            ++use;
            tc_fence_after();
            if (lane == 0) {
              issue_qk(tmem + kColS, q_desc(X, 0), dk + (uint64_t)kst * kTileDesc);
              mma_commit(&bars[kBarSFull + X]);
            }
            __syncwarp();
          }
          if (ok && lane == 0) mma_commit(&bEmpty[kst]);
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) mma_commit(&bars[kBarQEmpty]);
        __syncwarp();
      }
    } else if (kPair) {
      // ------------------------------------------------------------ O += P V of both groups
      int tile = 0, seen[2] = {0, 0};  // tiles so far, P's of each group
      Seg g;
      for (int s = 0; next_seg(0, s, g); ++s) {
        // O_X of the segment before has been read: its first PV here, or (no rows) its end, waits for that
        auto o_free = [&](int X) { return s == 0 || mbar_wait(&bars[kBarOFree + X], (s - 1) & 1); };
        for (int t = g.t0; t < g.t1 && ok; ++t, ++tile) {
          const int vst = (2 * tile + 1) % kSlots;
          if (misc[2] || !ready(2 * tile + 1)) { ok = false; break; }
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (group_rows(g.rb, X) <= 0) continue;
            if (t == g.t0 && !o_free(X)) { ok = false; break; }
            if (!mbar_wait(&bars[kBarPFull + X], seen[X] & 1)) { ok = false; break; }
            ++seen[X];
            tc_fence_after();
            if (lane == 0) {
              issue_pv_mma(tmem + kColO + 128 * X, tmem + kColP + 64 * X, dv + (uint64_t)vst * kTileDesc, t == g.t0);
              mma_commit(&bars[kBarPV + X]);
            }
            __syncwarp();
          }
          if (ok && lane == 0) mma_commit(&bEmpty[vst]);
          __syncwarp();
        }
        for (int X = 0; X < 2 && ok; ++X)
          if (group_rows(g.rb, X) <= 0) {
            ok = o_free(X);
            if (ok && lane == 0) mbar_arrive(&bars[kBarODone + X]);
            __syncwarp();
          }
        if (!ok) break;
      }
    } else if (!kPair && (warp == kMmaWarp0 || warp == kMmaWarp1)) {
      // ---------------------------------------------------------- MMA issuer of group X
      const int X = warp == kMmaWarp0 ? 0 : 1;
      const uint32_t tS = tmem + kColS + 128 * X, tO = tmem + kColO + 128 * X;
      int k = 0;  // tiles of this group so far
      Seg g;
      for (int s = 0; next_seg(X, s, g); ++s) {
        const int buf = s % kQBufs;
        const uint64_t q0 = q_desc(X, buf);
        if (!mbar_wait(&bars[kBarQFull + 2 * X + buf], (s / kQBufs) & 1)) { ok = false; break; }
        // O += P V of the group's tile k - 1 (the segment's first product waits until O of the one before is read)
        auto issue_pv = [&](bool first) -> bool {
          if (first && s > 0 && !mbar_wait(&bars[kBarOFree + X], (s - 1) & 1)) return false;
          if (!mbar_wait(&bars[kBarPFull + X], (k - 1) & 1)) return false;
          const int vidx = 2 * turn(X, k - 1) + 1, vst = vidx % kSlots;
          if (!ready(vidx)) return false;
          tc_fence_after();
          if (lane == 0) {
            issue_pv_mma(tO, tS, dv + (uint64_t)vst * kTileDesc, first);
            mma_commit(&bEmpty[vst]);
          }
          __syncwarp();
          return true;
        };
        for (int t = g.t0; t < g.t1; ++t, ++k) {
          if (misc[2] || (t > g.t0 && !issue_pv(t == g.t0 + 1))) { ok = false; break; }
          const int kidx = 2 * turn(X, k), kst = kidx % kSlots;
          if (!ready(kidx)) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            issue_qk(tS, q0, dk + (uint64_t)kst * kTileDesc);
            mma_commit(&bars[kBarSFull + X]);
            mma_commit(&bEmpty[kst]);
            if (t + 1 == g.t1) mma_commit(&bars[kBarQEmpty + 2 * X + buf]);
          }
          __syncwarp();
        }
        if (!ok || !issue_pv(g.t1 == g.t0 + 1)) { ok = false; break; }
        if (lane == 0) mma_commit(&bars[kBarODone + X]);
        __syncwarp();
      }
    }
  } else {
    if (kPair) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    // ------------------------------------------------------------ softmax group X
    const int X = warp >> 2, quarter = warp & 3;
    const bool used = kRows != kFew || X == quarter >> 1;  // kFew: warps 0, 1 and 6, 7
    const int lane0 = 32 * quarter - (kRows == kFew ? 64 * X : 0), r = lane0 + lane;  // row of lane 0, of this thread
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + kColS + (kPair ? 0 : 128 * X), tO = tmem + lane_base + kColO + 128 * X;
    const uint32_t tP = kPair ? tmem + lane_base + kColP + 64 * X : tS;
    int seen = 0;  // tiles of this group so far (phase of S)
    int idle = 0;  // segments without rows for this group
    // kTwo: P and O of this group are its own once the product with its last P is done
    auto pv_done = [&]() -> bool {
      if (!kPair || seen == 0) return true;
      if (!mbar_wait(&bars[kBarPV + X], (seen - 1) & 1)) return false;
      tc_fence_after();
      return true;
    };
    const int i_first = r % A.n;  // (a block of rows other than the first is kTwo's)
    Seg g;
    for (int s = 0; used && next_seg(X, s, g); ++s) {
      const int rb = kPair ? g.rb : 0;
      const int rows = group_rows(rb, X);
      const int rr = 256 * rb + (kPair ? 128 * X : 0) + r;  // row within the KV group
      const bool row_in = r < rows;
      const bool warp_in = lane0 < rows;
      const int i = kPair ? rr % A.n : i_first;  // drafted token of this row
      const bool row_ok = row_in && i < g.T;
      const int C = g.L - g.T;
      const uint32_t* mrow = A.mask ? A.mask + g.b * A.mask_stride + (int64_t)i * A.words : nullptr;
      // bit k: this row attends key key0 + k (keys from the end of the context on; lanes without a row see all)
      auto mask32 = [&](int key0) -> uint32_t {
        const int rel = key0 - C;  // drafted index of bit 0 (negative: context)
        if (rel <= -32 || !row_ok) return ~0u;
        if (!mrow) return low_mask32(min(i + 1, g.T) - rel);
        const int w0 = rel >> 5, sh = rel & 31;  // floor for negative rel
        const uint32_t a = (w0 >= 0 && w0 < A.words) ? __ldg(mrow + w0) : 0u;
        const uint32_t c = (w0 + 1 < A.words) ? __ldg(mrow + w0 + 1) : 0u;
        const uint32_t bits = __funnelshift_r(a, c, sh) & low_mask32(g.T - rel);
        return rel < 0 ? bits | low_mask32(-rel) : bits;
      };
      float m_used = -INFINITY, l = 0.f;
      bool first = true;      // no product into O yet
      bool alpha_any = false;  // a row of the warp raises its reference
      const float c2 = A.scale_log2;
      auto load64 = [&](uint32_t t, float* sv) {
        uint32_t* u = reinterpret_cast<uint32_t*>(sv);
        tmem_ld32(t, *reinterpret_cast<uint32_t(*)[32]>(u));
        tmem_ld32(t + 32, *reinterpret_cast<uint32_t(*)[32]>(u + 32));
        tmem_ld_wait();
      };
      auto max64 = [&](const float* sv, float m) -> float {
        float mx[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) mx[x] = max3f(sv[x], sv[8 + x], sv[16 + x]);
#pragma unroll
        for (int k = 24; k < 56; k += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x) mx[x] = max3f(mx[x], sv[k + x], sv[k + 8 + x]);
#pragma unroll
        for (int x = 0; x < 8; ++x) mx[x] = fmaxf(mx[x], sv[56 + x]);
        return fmaxf(max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])), m);
      };
      // A tile's maximum: the reference rises when it has to by more than 2^8; returns the factor for what was summed.
      auto raise = [&](float mt) -> float {
        const float m_new = fmaxf(m_used, mt * c2);
        // lanes without a row hold whatever shared memory held: they have no vote, or runs would differ
        alpha_any = __any_sync(0xFFFFFFFFu, row_ok && m_new > m_used + kRescaleThreshold);
        if (!alpha_any || m_new == -INFINITY) return 1.f;
        const float alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_new);
        m_used = m_new;
        return alpha;
      };
      // 64 weights e^{s - reference}, their sum in fp32.  The second product takes them as bf16, since its operands have
      // V's type: an output's error is 1.25 to 1.4 times that of its one rounding.  With a second bf16 term for what the
      // first one leaves it is 1.0 times, and 256 short requests take 99 us instead of 82 (64 long ones 198 instead of
      // 192): not kept, the prefill kernels round theirs the same way.
      auto weights = [&](const float* sv, uint32_t t, uint64_t (&acc)[2]) {
        const float mref = (m_used == -INFINITY) ? 0.f : m_used;
        const uint64_t c2x2 = pk2(c2, c2), negm = pk2(-mref, -mref);
#pragma unroll
        for (int h = 0; h < 32 / kPChunk; ++h) {
          uint32_t pk[kPChunk];
#pragma unroll
          for (int k = 0; k < kPChunk; ++k) {
            const int e = 2 * kPChunk * h + 2 * k;
            float x0, x1, p0, p1;
            up2(fma2(pk2(sv[e], sv[e + 1]), c2x2, negm), x0, x1);
            const uint64_t p = pk2(ex2(x0), ex2(x1));
            acc[k & 1] = add2(acc[k & 1], p);
            up2(p, p0, p1);
            pk[k] = pack_bf16x2(p0, p1);
          }
          tmem_st4(t + kPChunk * h, pk);
        }
      };
      auto add_row = [&](const uint64_t (&acc)[2], float alpha) {
        float a0, a1, a2, a3;
        up2(acc[0], a0, a1);
        up2(acc[1], a2, a3);
        l = l * alpha + ((a0 + a1) + (a2 + a3));
      };
      auto rescale = [&](float alpha) {  // O: its previous product is done (before S was ready, or waited for)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
          tmem_st32(tO + 32 * c, o);
        }
      };
      if (rows > 0)
        for (int t = g.t0; t < g.t1; ++t) {
          if (misc[2]) { ok = false; break; }
          const int key0 = 128 * t;
          const bool masked = key0 + 128 > C;
          if (!mbar_wait(&bars[kBarSFull + X], seen & 1)) { ok = false; break; }
          tc_fence_after();
          if constexpr (kPair) {
            float sv[128];
            if (warp_in) {
              uint32_t* u = reinterpret_cast<uint32_t*>(sv);
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(u + 32 * c));
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int k = 0; k < 128; ++k) sv[k] = 0.f;
            }
            tc_fence_before();  // the scores are in registers: S is free for the other group's
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kBarSFree]);
            if (warp_in) {
              if (masked) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const uint32_t vw = mask32(key0 + 32 * c);
#pragma unroll
                  for (int k = 0; k < 32; ++k) sv[32 * c + k] = ((vw >> k) & 1u) ? sv[32 * c + k] : -INFINITY;
                }
              }
              const float alpha = raise(max64(sv, max64(sv + 64, -INFINITY)));
              ok = pv_done();  // P and O may be written
              uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
              weights(sv, tP, acc);
              weights(sv + 64, tP + 32, acc);
              add_row(acc, alpha);
              if (alpha_any && !first) rescale(alpha);
              tmem_st_wait();
              first = false;
            } else {
              ok = pv_done();
            }
          } else if (warp_in) {
            // Two passes over the scores in TMEM, half a tile at a time: the rolled loops keep the code of all roles
            // within the instruction cache, which 128 scores in registers at once do not (a third of the fetches
            // missed, and one warp a scheduler has nothing to hide that with).
            float mt = -INFINITY;
            if (masked) {  // masked scores are put back as -inf
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                uint32_t u[32];
                const uint32_t vw = mask32(key0 + 32 * c);
                tmem_ld32(tS + 32 * c, u);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                  u[k] = ((vw >> k) & 1u) ? u[k] : 0xFF800000u;
                  mt = fmaxf(mt, __uint_as_float(u[k]));
                }
                tmem_st32(tS + 32 * c, u);
              }
              tmem_st_wait();
            } else {
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                float sv[64];
                load64(tS + 64 * h, sv);
                mt = max64(sv, mt);
              }
            }
            const float alpha = raise(mt);
            uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {  // P of half 0 lies over its scores, that of half 1 as well
              float sv[64];
              load64(tS + 64 * h, sv);
              weights(sv, tP + 32 * h, acc);
            }
            add_row(acc, alpha);
            if (alpha_any && !first) rescale(alpha);
            tmem_st_wait();
            first = false;
          }
          if (!ok) break;
          ++seen;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPFull + X]);
        }
      if (!ok) break;

      // ---- the segment's end: O / l and LSE, or the part's unnormalised state.
      // O goes to registers first, so that the next segment's products may start
      // while it is written.
      const bool joins = kRows == kMany && (g.r0 != g.t0 || g.r1 != g.t1);
      const bool whole = g.r0 == 0 && g.r1 == g.tiles;
      const int64_t grow = (int64_t)(g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + rr;
      const int width = min(256, A.R - 256 * rb), full = min(256, A.R), rw = rr - 256 * rb;
      const int64_t slot = 2 * part_of(W, kMost, blockIdx.x, kPair || joins ? 0 : X) + (g.r0 > 0 ? 0 : 1);
      bool some = !(l == 0.f);  // an attended key (a NaN among them shows in l)
      float inv = some ? 1.f / l : 0.f;
      if (kPair && rows > 0 ? !pv_done()
                            : !mbar_wait(&bars[kBarODone + X], (kPair ? idle++ : s) & 1)) { ok = false; break; }
      tc_fence_after();
      float w0 = 1.f, w1 = 0.f;
      if (joins) {  // both groups' last segments, once per CTA: each takes half of the columns of both O's
        float2* ml = reinterpret_cast<float2*>(sm + Ly::kML);
        ml[128 * X + r] = make_float2(m_used, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarML]);  // and every product into this group's O is done
        if (!mbar_wait(&bars[kBarML], 0)) { ok = false; break; }
        tc_fence_after();
        const float2 a = ml[r], b = ml[128 + r];
        const float m = fmaxf(a.x, b.x), ref = m == -INFINITY ? 0.f : m;
        w0 = ex2(a.x - ref);
        w1 = ex2(b.x - ref);
        m_used = m;
        l = a.y * w0 + b.y * w1;
        some = !(l == 0.f);
        inv = some ? 1.f / l : 0.f;
      }
      // N columns from c0 on
      auto write = [&](const float* ov, int c0, auto N) {
        if (kRows == kMany && N == 64 && whole) {
          // Four lanes turn their rows' pieces round, so that a store covers 64 bytes each of 8 rows and not 16 of 32:
          // 256 requests of 100 to 1000 tokens with 128 rows 118 -> 113 us.  (kFew has too few rows a request for it;
          // in kTwo 192 rows gain 2 % by it and 256 lose 1 %.)
          const unsigned live = __ballot_sync(0xFFFFFFFFu, row_ok);
          const int q = lane & 3;
          uint4* dst = reinterpret_cast<uint4*>(A.o + (grow - q) * D + c0) + q;
#pragma unroll
          for (int h = 0; h < N / 32; ++h) {
            uint32_t v[4][4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const int e = 32 * h + 8 * x + 2 * y;
                v[x][y] = pack_bf16x2(ov[e] * inv, ov[e + 1] * inv);
              }
#pragma unroll
            for (int step = 1; step < 4; step <<= 1)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (!(x & step))
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, q & step ? v[x][y] : v[x | step][y], step);
                    (q & step ? v[x][y] : v[x | step][y]) = got;
                  }
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (live >> ((lane & 28) + x) & 1u)
                dst[x * (D / 8) + 4 * h] = make_uint4(v[x][0], v[x][1], v[x][2], v[x][3]);
          }
          return;
        }
        if (!row_ok) return;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(A.o + grow * D + c0);
#pragma unroll
          for (int x = 0; x < N / 8; ++x) {
            uint32_t pk[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) pk[y] = pack_bf16x2(ov[8 * x + 2 * y] * inv, ov[8 * x + 2 * y + 1] * inv);
            dst[x] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else {
          float4* part = A.part + slot * (D / 4) * full + (int64_t)(c0 / 4) * width + rw;
#pragma unroll
          for (int x = 0; x < N / 4; ++x, part += width)
            *part = make_float4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
        }
      };
      if (joins) {
#pragma unroll 1
        for (int c = X * (D / 2); c < (X + 1) * (D / 2); c += 32) {
          float ov[32], q[32];
          __syncwarp();
          tmem_ld32(tmem + lane_base + kColO + c, *reinterpret_cast<uint32_t(*)[32]>(ov));
          tmem_ld32(tmem + lane_base + kColO + 128 + c, *reinterpret_cast<uint32_t(*)[32]>(q));
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) ov[x] = ov[x] * w0 + q[x] * w1;
          write(ov, c, std::integral_constant<int, 32>());
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          float ov[64];
          __syncwarp();
          load64(tO + c, ov);
          if (c + 64 == D) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kBarOFree + X]);
          }
          write(ov, c, std::integral_constant<int, 64>());
        }
      }
      if (row_ok && (!joins || X == 0)) {
        if (!whole) A.part_ml[slot * full + rw] = make_float2(m_used, l);
        else if (A.lse) A.lse[grow] = some ? (m_used + __log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
    }
  }
  if (!ok) {
    misc[2] = 1;
    atomicCAS(A.err, 0, (int)kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (misc[2]) {
    // A role gave up, so others may have left copies and products in flight that nobody waited for, whether or not they
    // gave up themselves: those end before the CTA's shared memory and TMEM go.
    if (warp == kMmaWarp0 || warp == kMmaWarp1) {
      uint64_t* drained = &bars[kBarDrain + (warp == kMmaWarp0 ? 0 : 1)];
      if (lane == 0) mma_commit(drained);
      mbar_wait(drained, 0, kDrainNs);
    } else if (warp == kLoaderWarp || (!kPair && warp == kLoaderWarp1)) {
      const int X = warp == kLoaderWarp ? 0 : 1, asked = misc[6 + X];
      for (int x = max(0, asked - kQBufs); x < asked; ++x)
        mbar_wait(&bars[kBarQFull + 2 * X + x % kQBufs], (x / kQBufs) & 1, kDrainNs);
      // A slot's last load only: the one before had landed and been used.
      const int x = lane < kSlots ? lasts[X * kSlots + lane] : -1;
      if (x >= 0 && (kPair || x > lasts[(X ^ 1) * kSlots + lane])) mbar_wait(&bFull[lane], (x / kSlots) & 1, kDrainNs);
      __syncwarp();
    }
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
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

template <int D, Rows kRows, int kShare>
__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) tree_join_kernel(const TreeArgs A) {
  constexpr int kMost = kRows == kTwo ? kCtas : 2 * kCtas, kWarps = kJoinThreads / 32, kWords = (kMost + 31) / 32;
  constexpr int kCols = join_cols(kShare), kAhead = kShare > 1 ? 4 : 2;
  static_assert(kShare == 1 || kShare == kWarps, "a chunk per warp or CTA");
  __shared__ unsigned found[kWords];
  __shared__ float joined[kShare][kCols + 2][32];  // (kShare = 1: unused)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int full = min(256, A.R), chunks = (full * (D / kCols) + 31) / 32;
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
    const int width = min(256, A.R - 256 * rb);
    const int c = e / width, rw = e - c * width, rr = 256 * rb + rw;  // group of columns, row of the block
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

struct TreeWs {
  size_t cuts, ml, part, total;
};
int max_parts(int64_t R) { return R > 128 ? kCtas : 2 * kCtas; }
TreeWs tree_ws(const msa_shape& s) {
  const int64_t R = (int64_t)(s.Hq / s.Hkv) * s.n, rows = 2 * max_parts(R) * (R < 256 ? R : 256);
  TreeWs w;
  w.cuts = 16;  // behind their count
  w.ml = align256(w.cuts + max_parts(R) * sizeof(Cut));
  w.part = align256(w.ml + (size_t)rows * 8);
  w.total = align256(w.part + (size_t)rows * s.d_h * 4);
  return w;
}

msa_status check_tree_shape(const msa_shape* s) {
  const msa_status st = check_shape(s);
  if (st != MSA_OK) return st;
  const int64_t rows = (int64_t)s->B * s->Hq * s->n;
  const int64_t R = (int64_t)(s->Hq / s->Hkv) * s->n, RB = (R + 255) / 256;
  if (s->n > kMaxDrafts || rows + 256 >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)s->B * s->Hkv * RB >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

bool aligned(const void* p, size_t a, bool required) {
  if (!p) return !required;
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

template <int D, Rows kRows>
msa_status launch_tree(const TreeMaps& maps, const TreeArgs& a, bool join, cudaStream_t stream) {
  auto kern = tree_attn_kernel<D, kRows>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kAlloc) != cudaSuccess)
    return MSA_ERR_CUDA;
  kern<<<kCtas, threads_of(kRows), Lay<D>::kAlloc, stream>>>(maps, a);
  note_launch();
  if (cudaGetLastError() != cudaSuccess) return MSA_ERR_CUDA;
  if (!join) return MSA_OK;
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  const int full = a.R < 256 ? a.R : 256;
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
  if ((share ? cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kRows, 8>, a)
             : cudaLaunchKernelEx(&cfg, tree_join_kernel<D, kRows, 1>, a)) != cudaSuccess)
    return MSA_ERR_CUDA;
  note_launch();
  return MSA_OK;
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attn_tree_workspace(const msa_shape* shape) {
  return check_tree_shape(shape) == MSA_OK ? tree_ws(*shape).total : 0;
}

extern "C" msa_status msa_attn_tree(const msa_shape* shape, const void* q, const msa_kv_pages* pages,
                                    const int32_t* page_table, int32_t max_pages, const int32_t* seq_len,
                                    const int32_t* tree_len, const uint32_t* tree_mask, int64_t mask_stride, void* o,
                                    float* lse, void* ws, size_t ws_bytes, void* stream) {
  msa_status st = check_tree_shape(shape);
  if (st != MSA_OK) return st;
  if (!pages || max_pages < 1) return MSA_ERR_INVALID_ARG;
  st = check_page_geometry(pages->num_pages, pages->page_size);
  if (st != MSA_OK) return st;
  if (!aligned(q, 16, true) || !aligned(o, 16, true) || !aligned(pages->k, 16, true) || !aligned(pages->v, 16, true) ||
      !aligned(page_table, 4, true) || !aligned(seq_len, 4, true) || !aligned(tree_len, 4, false) ||
      !aligned(tree_mask, 4, false) || !aligned(lse, 4, false) || !aligned(ws, 16, true))
    return MSA_ERR_INVALID_ARG;
  if (q == o) return MSA_ERR_INVALID_ARG;
  const int32_t words = (shape->n + 31) / 32;
  if (tree_mask && mask_stride != 0 && mask_stride < (int64_t)shape->n * words) return MSA_ERR_INVALID_ARG;
  if ((int64_t)pages->num_pages * pages->page_size * shape->Hkv + 256 >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * pages->page_size >= ((int64_t)1 << 31) - 256) return MSA_ERR_UNSUPPORTED;
  const TreeWs w = tree_ws(*shape);
  if (ws_bytes < w.total) return MSA_ERR_WORKSPACE_TOO_SMALL;
  TreeArgs a;
  memset(&a, 0, sizeof(a));
  a.B = shape->B;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.n = shape->n;
  a.R = shape->Hq / shape->Hkv * shape->n;
  a.RB = (a.R + 255) / 256;
  a.max_parts = max_parts(a.R);
  // a load costs about 100 cycles whatever its size: few of them, and few rows that are not the group's
  a.q_box = a.R <= 16 ? 16 : a.R <= 32 ? 32 : 64;
  a.page_shift = __builtin_ctz((unsigned)pages->page_size);
  a.max_pages = max_pages;
  a.num_pages = pages->num_pages;
  a.words = words;
  a.table = page_table;
  a.seq_len = seq_len;
  a.tree_len = tree_len;
  a.mask = tree_mask;
  a.mask_stride = mask_stride;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.count = reinterpret_cast<int32_t*>(base);
  a.cuts = reinterpret_cast<Cut*>(base + w.cuts);
  a.part_ml = reinterpret_cast<float2*>(base + w.ml);
  a.part = reinterpret_cast<float4*>(base + w.part);
  a.scale_log2 = effective_scale(*shape) * 1.4426950408889634f;
  a.err = device_error_word();
  if (!a.err) return MSA_ERR_CUDA;
  TreeMaps maps;
  const int64_t krows = (int64_t)pages->num_pages * shape->Hkv * pages->page_size;
  if (!make_bf16_map(&maps.q, q, 1, (int64_t)shape->B * shape->Hq * shape->n, shape->d_h, a.q_box) ||
      !make_bf16_map(&maps.k, pages->k, 1, krows, shape->d_h, pages->page_size) ||
      !make_bf16_map(&maps.v, pages->v, 1, krows, shape->d_h, pages->page_size))
    return MSA_ERR_CUDA;
  // a table of at most 128 keys holds no item of two tiles: none is cut
  const bool join = (int64_t)max_pages * pages->page_size > 128;
  cudaStream_t stm = (cudaStream_t)stream;
  const bool d128 = shape->d_h == 128;
  if (a.R <= 64) return d128 ? launch_tree<128, kFew>(maps, a, join, stm) : launch_tree<64, kFew>(maps, a, join, stm);
  if (a.R <= 128)
    return d128 ? launch_tree<128, kMany>(maps, a, join, stm) : launch_tree<64, kMany>(maps, a, join, stm);
  return d128 ? launch_tree<128, kTwo>(maps, a, join, stm) : launch_tree<64, kTwo>(maps, a, join, stm);
}
