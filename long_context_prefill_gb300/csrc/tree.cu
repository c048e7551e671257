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
// form one line, cut into equal parts, one per CTA and SM: no CTA has more
// than one tile above another's, whatever the lengths.  An item that lies in
// one part is finished there; of one that is cut, each part leaves its
// unnormalised sum, maximum and row sum in the workspace, and a second kernel
// (launched early, waiting for the first) joins them in key order, so results
// do not depend on timing.
//
// A CTA (12 warps):
//   warp 10    loader: walks the parts' segments, publishes their descriptors,
//              loads Q rows and the K and V pages of every tile by TMA into a
//              ring (K and V tiles alternate);
//   warp 8     waits for the ring's tiles one after another and declares each
//              ready; in a request's last V tile it first zeroes the rows past
//              the end: pages may hold anything there, and a weight of zero
//              does not hide an infinity or NaN in an MMA.  (The order matters:
//              loads land in any order, and an issuer that skips a tile must
//              not take the phase of a slot's earlier use for the one it waits
//              for.  With declarations in order, the tile it saw last proves
//              every earlier use of the slot over);
//   warps 9/11 MMA issuers of the two softmax groups;
//   warps 0-7  softmax groups X = 0, 1 (4 warps each, thread = row = TMEM lane).
// Up to 128 rows (kTwo false): the groups take turns on the key tiles, each
// with its own running maximum, sum and O, joined at the segment's end.  Above (kTwo):
// group X owns rows 128 X .. of the 256-row block, and both see every tile.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "internal.h"
#include "ptx.cuh"

namespace msa {

msa_status check_shape(const msa_shape* s);
msa_status check_page_geometry(int32_t num_pages, int32_t page_size);
float effective_scale(const msa_shape& s);

namespace {

constexpr int kCtas = 152;  // parts of the line of tiles, if it has as many tiles
constexpr int kThreads = 384;
constexpr int kCleanWarp = 8, kMmaWarp0 = 9, kLoaderWarp = 10;  // 11: the other issuer
constexpr int kSegSlots = 4;
constexpr int kSegReaders = 11;  // 8 softmax warps, 2 issuers, the cleaner
constexpr uint32_t kTmemCols = 512;
// TMEM columns.  Up to 128 rows: S of group X at 128 X, P over its first 64.
// Above: one S that the groups use in turn, P of group X at 128 + 64 X.  O of
// group X at 256 + 128 X.
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr int kPChunk = 4;
constexpr uint32_t kIdleNs = 64;
constexpr int kMaxDrafts = 1024;

struct TreeArgs {
  int32_t B, Hq, Hkv, n, R, RB, page_shift, max_pages, num_pages, words, q_box;
  const int32_t *table, *seq_len, *tree_len;
  const uint32_t* mask;
  int64_t mask_stride;  // words between the masks of two requests (0: one mask for all)
  __nv_bfloat16* o;
  float* lse;
  int64_t* prefix;  // [B + 1] tiles of the requests before
  float4* part;     // [2 kCtas][d/4][rows] unnormalised O of the cut items
  float2* part_ml;  // [2 kCtas][rows] their maximum (log2) and row sum
  float scale_log2;
  int* err;
};

struct TreeMaps {
  CUtensorMap q, k, v;  // [rows, d] views, boxes of 64 columns x q_box rows (q), x page_size rows (k, v)
};

// The part of one item that a CTA processes: tiles t0 .. t1 of its `tiles`.
struct Seg {
  int32_t b, kvh, rb, t0, t1, tiles;  // b < 0: no more
  int32_t L, T;
};

enum {
  kBarQFull = 0,                    // [2]
  kBarQEmpty = 2,                   // [2]
  kBarSFull = 4,                    // [2]
  kBarPFull = 6,                    // [2]
  kBarODone = 8,                    // [2] every product of the group's segment is done (kTwo: of a group without rows)
  kBarOFree = 10,                   // [2] O of the segment has been read
  kBarML = 12,                      // maxima and sums of both groups are written
  kBarSFree = 13,                   // kTwo: the scores are in registers
  kBarPV = 14,                      // [2] kTwo: the group's last P has been used
  kBarSegFull = 16,                 // [kSegSlots]
  kBarSegEmpty = kBarSegFull + kSegSlots,
  kBarRing = kBarSegEmpty + kSegSlots  // full[kSlots], empty[kSlots], ready[kSlots]
};

template <int D>
struct Lay {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kSlots = 5 * (128 / D);
  static constexpr int kQ = 0;  // two Q tiles: two segments' (one row tile each) or one segment's two
  static constexpr int kRing = 2 * kTile;
  static constexpr int kSeg = kRing + kSlots * kTile;
  static constexpr int kML = kSeg + kSegSlots * (int)sizeof(Seg);
  static constexpr int kBars = kML + 2 * 128 * 8;
  static constexpr int kNumBars = kBarRing + 3 * kSlots;
  static constexpr int kMisc = kBars + kNumBars * 8;  // [0] TMEM base, [2] abort
  static constexpr int kAlloc = kMisc + 16;
  static_assert(kAlloc <= 227 * 1024 && kAlloc > 120 * 1024, "shared memory: one CTA per SM");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pk2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void up2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t low_mask32(int c) {
  c = c < 0 ? 0 : (c > 32 ? 32 : c);
  return c >= 32 ? 0xFFFFFFFFu : ((1u << c) - 1u);
}

// Keys and drafted tokens of request b; false (nothing to compute) when it has
// none or its numbers break the contract (flagged once by the loader).
__device__ __forceinline__ bool request(const TreeArgs& A, int b, int& L, int& T, bool& bad) {
  L = A.seq_len[b];
  T = A.tree_len ? A.tree_len[b] : A.n;
  bad = T < 0 || T > A.n || L < T || L > ((int64_t)A.max_pages << A.page_shift);
  return !bad && T > 0;
}
__device__ __forceinline__ int key_tiles(int L) { return (L + 127) >> 7; }
__device__ __forceinline__ int parts(int64_t W) { return W < kCtas ? (int)W : kCtas; }
__device__ __forceinline__ int64_t part_begin(int64_t W, int c) { return W < kCtas ? c : W * c / kCtas; }

template <int D, bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeMaps M, const TreeArgs A) {
  using Ly = Lay<D>;
  constexpr int kSlots = Ly::kSlots;
  extern __shared__ __align__(1024) uint8_t sm[];  // swizzled tiles start on 1 KB
  if (smem_u32(sm) & 1023) {
    if (threadIdx.x == 0) atomicCAS(A.err, 0, (int)kErrTimeout);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::kBars);
  uint64_t* bFull = bars + kBarRing;
  uint64_t* bEmpty = bFull + kSlots;
  uint64_t* bReady = bEmpty + kSlots;
  Seg* segs = reinterpret_cast<Seg*>(sm + Ly::kSeg);
  float2* ml = reinterpret_cast<float2*>(sm + Ly::kML);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + Ly::kMisc);
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[kBarQFull + x], 1);
      mbar_init(&bars[kBarQEmpty + x], kTwo ? 1 : 2);
      mbar_init(&bars[kBarSFull + x], 1);
      mbar_init(&bars[kBarPFull + x], 4);
      mbar_init(&bars[kBarODone + x], 1);
      mbar_init(&bars[kBarOFree + x], kTwo ? 4 : 8);
      mbar_init(&bars[kBarPV + x], 1);
    }
    mbar_init(&bars[kBarML], 8);
    mbar_init(&bars[kBarSFree], 4);
    for (int s = 0; s < kSegSlots; ++s) {
      mbar_init(&bars[kBarSegFull + s], 1);
      mbar_init(&bars[kBarSegEmpty + s], kSegReaders);
    }
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bFull[s], 1);
      mbar_init(&bEmpty[s], 1);
      mbar_init(&bReady[s], 1);
    }
    misc[2] = 0;
    fence_mbar_init();
  }
  // ---- this CTA's part [lo, hi) of the line of tiles, and the request it starts in
  const int items = A.Hkv * A.RB;  // items of a request
  int64_t* wsum = reinterpret_cast<int64_t*>(sm + Ly::kRing);  // scratch until the pipeline starts
  int64_t* start = wsum + 16;                                  // [0] request, [1] its first tile
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
    const int64_t lo = part_begin(W, blockIdx.x);  // at or above W in a CTA without a part
    int64_t at = base + inc - mine;
    for (int b = b0; b < b1; ++b) {
      const int64_t t = per == 1 ? own : tiles(b);
      if (at <= lo && lo < at + t) { start[0] = b; start[1] = at; }
      if (blockIdx.x == 0) A.prefix[b] = at;
      at += t;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) A.prefix[A.B] = W;
  }
  const int64_t lo = part_begin(W, blockIdx.x), hi = part_begin(W, blockIdx.x + 1);
  fence_proxy_async_smem();  // the scratch above lies in the ring that TMA fills
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if ((int)blockIdx.x >= parts(W)) {  // no part
    if (warp == 0) tmem_dealloc(misc[0], kTmemCols);
    return;
  }
  const int first_b = (int)start[0];
  const int64_t first_tile = start[1];
  const uint32_t tmem = misc[0];

  // Segment s of this CTA as the readers see it; false: no more, or gave up.
  bool ok = true;
  auto next_seg = [&](int s, Seg& g) -> bool {
    if (misc[2] || !mbar_wait(&bars[kBarSegFull + s % kSegSlots], (s / kSegSlots) & 1)) { ok = false; return false; }
    g = segs[s % kSegSlots];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBarSegEmpty + s % kSegSlots]);
    return g.b >= 0;
  };
  auto ready = [&](int idx) { return mbar_wait(&bReady[idx % kSlots], (idx / kSlots) & 1); };
  constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
  constexpr uint64_t kTileDesc = Ly::kTile >> 4;
  const uint64_t dq = sdesc_sw128(smem_u32(sm + Ly::kQ), 16, 1024);
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
  // rows of softmax group X in the 256-row block rb (one group's rows serve both groups unless kTwo)
  auto group_rows = [&](int rb, int X) { return min(128, A.R - 256 * rb - (kTwo ? 128 * X : 0)); };

  // the block starts with 3 x 128 threads x 168 registers; the softmax threads (a row's 128 scores each) take
  // 208 and the others' 72: 2 x 208 + 72 <= 3 x 168
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if (warp == kLoaderWarp) {
    // ------------------------------------------------------------ loader
    const uint64_t policy = A.RB == 1 ? policy_evict_first() : policy_evict_last();
    const int pshift = 7 - A.page_shift, pp = 1 << pshift;  // pages of a tile
    const int P = 1 << A.page_shift;
    int64_t at = first_tile;  // first tile of item 0 of request b
    int64_t pos = lo;
    int idx = 0, s = 0;  // ring index (2 per tile), segment
    int b = first_b;
    for (; ok; ++s) {
      // ---- next segment
      Seg g;
      g.b = -1;
      if (pos < hi) {
        int L = 0, T = 0;
        bool bad;
        int64_t t = 0;
        for (; b < A.B; ++b) {  // pos < hi <= W: a request holding it exists
          t = request(A, b, L, T, bad) ? (int64_t)items * key_tiles(L) : 0;
          if (pos < at + t) break;
          at += t;
        }
        if (b >= A.B) { ok = false; break; }
        g.b = b;
        g.L = L;
        g.T = T;
        g.tiles = key_tiles(L);
        const int item = (int)((pos - at) / g.tiles);
        g.kvh = item / A.RB;
        g.rb = item - g.kvh * A.RB;
        g.t0 = (int)(pos - at - (int64_t)item * g.tiles);
        const int64_t left = hi - pos;
        g.t1 = left < g.tiles - g.t0 ? g.t0 + (int)left : g.tiles;
        pos += g.t1 - g.t0;
      }
      if (misc[2] || !mbar_wait_idle(&bars[kBarSegEmpty + s % kSegSlots], ((s / kSegSlots) & 1) ^ 1, kIdleNs)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        segs[s % kSegSlots] = g;
        mbar_arrive(&bars[kBarSegFull + s % kSegSlots]);
      }
      if (g.b < 0) break;
      // ---- Q rows (their load overlaps the page entries')
      {
        const int nq = kTwo ? 1 : 2, buf = s % nq;
        if (!mbar_wait_idle(&bars[kBarQEmpty + buf], ((s / nq) & 1) ^ 1, kIdleNs)) { ok = false; break; }
        const int rows = min(kTwo ? 256 : 128, A.R - 256 * g.rb), boxes = (rows + A.q_box - 1) / A.q_box;
        uint64_t* full = &bars[kBarQFull + buf];
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(boxes * A.q_box * D * 2));
        __syncwarp();
        const int qrow = (g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + 256 * g.rb;
        if (lane < boxes * (D / 64)) {  // at most 8
          const int c = lane & (D / 64 - 1), r = lane / (D / 64) * A.q_box;
          tma_load_3d(sm + Ly::kQ + (kTwo ? r >> 7 : buf) * Ly::kTile + c * 16384 + (r & 127) * 128, &M.q, full, 64 * c,
                      qrow + r, 0);
        }
      }
      // ---- pages of the first tiles: lane x holds entry base + x, and base + 32 + x ahead
      const int32_t* row = A.table + (int64_t)g.b * A.max_pages;
      const int np = (g.L + P - 1) >> A.page_shift;
      auto entry = [&](int p) {
        int page = p < np ? row[p] : 0;
        if ((unsigned)page >= (unsigned)A.num_pages) {  // skipped: an existing page stands in, the call has failed
          atomicCAS(A.err, 0, (int)kErrIndex);
          page = 0;
        }
        return page;
      };
      int base = g.t0 << pshift;
      int ids = entry(base + lane), ahead = entry(base + 32 + lane);
      // ---- K and V tiles
      for (int t = g.t0; t < g.t1 && ok; ++t) {
        int off = (t << pshift) - base;
        if (off >= 32) {
          base += 32;
          off -= 32;
          ids = ahead;
          ahead = entry(base + 32 + lane);
        }
        const int have = min(pp, np - (t << pshift));  // pages of this tile that hold keys
        const int c = lane >> 3, x = lane & 7;
        const int page = __shfl_sync(0xFFFFFFFFu, ids, (off + x) & 31);
        const int krow = (page * A.Hkv + g.kvh) << A.page_shift;
#pragma unroll
        for (int is_v = 0; is_v < 2; ++is_v, ++idx) {
          const int st = idx % kSlots;
          if (misc[2] || !mbar_wait_idle(&bEmpty[st], ((idx / kSlots) & 1) ^ 1, kIdleNs)) {
            ok = false;
            break;  // before ++idx: nothing was loaded into this slot
          }
          if (lane == 0) mbar_arrive_expect_tx(&bFull[st], (uint32_t)(have * P * D * 2));
          __syncwarp();
          if (c < D / 64 && x < have)
            tma_load_3d_hint(sm + Ly::kRing + st * Ly::kTile + c * 16384 + x * P * 128, is_v ? &M.v : &M.k,
                             &bFull[st], 64 * c, krow, 0, policy);
        }
      }
    }
    if (!ok)  // gave up: the copies in flight land before the shared memory goes
      for (int x = max(0, idx - kSlots); x < idx; ++x) mbar_wait(&bFull[x % kSlots], (x / kSlots) & 1);
  } else if (warp == kCleanWarp) {
    // ------------------------------------------------------------ tiles in order, rows past a request's end
    int idx = 0;
    Seg g;
    for (int s = 0; next_seg(s, g); ++s)
      for (int t = 2 * g.t0; t < 2 * g.t1; ++t, ++idx) {  // K and V of every tile
        const int st = idx % kSlots;
        if (misc[2] || !mbar_wait(&bFull[st], (idx / kSlots) & 1)) { ok = false; break; }
        const int keys = g.L - 64 * (t & ~1);
        if ((t & 1) && keys < 128) {
          uint8_t* v = sm + Ly::kRing + st * Ly::kTile;
          for (int x = keys * 8 + lane; x < 1024; x += 32)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * 16384 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&bReady[st]);
      }
  } else if (kTwo && warp == kMmaWarp0) {
    // ------------------------------------------------------------ scores of both groups
    int tile = 0, use = 0;  // tiles so far, uses of S so far
    Seg g;
    for (int s = 0; next_seg(s, g); ++s) {
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
            issue_qk(tmem + kColS, dq + (uint64_t)X * kTileDesc, dk + (uint64_t)kst * kTileDesc);
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
  } else if (kTwo) {
    // ------------------------------------------------------------ O += P V of both groups
    int tile = 0, seen[2] = {0, 0};  // tiles so far, P's of each group
    Seg g;
    for (int s = 0; next_seg(s, g); ++s) {
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
  } else if (!kTwo) {
    // ------------------------------------------------------------ MMA issuer of group X
    const int X = warp == kMmaWarp0 ? 0 : 1;
    const uint32_t tS = tmem + kColS + 128 * X, tO = tmem + kColO + 128 * X;
    int tile0 = 0;   // CTA tile index of the segment's first tile
    int pphase = 0;  // tiles whose P this issuer has waited for
    Seg g;
    for (int s = 0; next_seg(s, g); ++s) {
      const int buf = s & 1, nt = g.t1 - g.t0;
      const uint64_t q0 = dq + (uint64_t)buf * kTileDesc;
      if (!mbar_wait(&bars[kBarQFull + buf], (s >> 1) & 1)) { ok = false; break; }
      int pending = -1;
      bool first = true;
      // O_X of the segment before has been read: its first PV here, or its end, waits for that
      auto o_free = [&]() -> bool { return s == 0 || mbar_wait(&bars[kBarOFree + X], (s - 1) & 1); };
      auto issue_pv = [&]() -> bool {
        if (first && !o_free()) return false;
        const int vidx = 2 * pending + 1, vst = vidx % kSlots;
        if (!mbar_wait(&bars[kBarPFull + X], pphase & 1)) return false;
        ++pphase;
        if (!ready(vidx)) return false;
        tc_fence_after();
        if (lane == 0) {
          issue_pv_mma(tO, tS, dv + (uint64_t)vst * kTileDesc, first);
          mma_commit(&bEmpty[vst]);
        }
        __syncwarp();
        first = false;
        pending = -1;
        return true;
      };
      for (int t = X; t < nt; t += 2) {
        if (misc[2]) { ok = false; break; }
        const int kidx = 2 * (tile0 + t), kst = kidx % kSlots;
        if (pending >= 0 && !issue_pv()) { ok = false; break; }
        if (!ready(kidx)) { ok = false; break; }
        tc_fence_after();
        if (lane == 0) {
          issue_qk(tS, q0, dk + (uint64_t)kst * kTileDesc);
          mma_commit(&bars[kBarSFull + X]);
          mma_commit(&bEmpty[kst]);
        }
        __syncwarp();
        pending = tile0 + t;
      }
      if (!ok) break;
      if (lane == 0) mma_commit(&bars[kBarQEmpty + buf]);  // every S of this segment
      __syncwarp();
      if (pending >= 0 ? !issue_pv() : first && !o_free()) { ok = false; break; }
      if (lane == 0) mma_commit(&bars[kBarODone + X]);
      __syncwarp();
      tile0 += nt;
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ softmax group X
    const int X = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_base + kColS + (kTwo ? 0 : 128 * X), tO = tmem + lane_base + kColO + 128 * X;
    const uint32_t tP = kTwo ? tmem + lane_base + kColP + 64 * X : tS;
    const float c2 = A.scale_log2;
    int seen = 0;  // tiles of this group so far (phase of S)
    int idle = 0;  // segments without rows for this group
    // kTwo: P and O of this group are its own once the product with its last P is done
    auto pv_done = [&]() -> bool {
      if (!kTwo || seen == 0) return true;
      if (!mbar_wait(&bars[kBarPV + X], (seen - 1) & 1)) return false;
      tc_fence_after();
      return true;
    };
    Seg g;
    for (int s = 0; next_seg(s, g); ++s) {
      const int rows = group_rows(g.rb, X);
      const int rr = 256 * g.rb + (kTwo ? 128 * X : 0) + r;  // row within the KV group
      const bool row_in = r < rows;
      const bool warp_in = 32 * quarter < rows;
      const int i = rr % A.n;  // drafted token of this row
      const bool row_ok = row_in && i < g.T;
      const int C = g.L - g.T;
      const uint32_t* mrow = A.mask ? A.mask + g.b * A.mask_stride + (int64_t)i * A.words : nullptr;
      const int nt = g.t1 - g.t0;
      float m_used = -INFINITY, l = 0.f;
      bool first = true;
      if (rows > 0)
        for (int t = kTwo ? 0 : X; t < nt; t += kTwo ? 1 : 2) {
          if (misc[2]) { ok = false; break; }
          const int key0 = 128 * (g.t0 + t);
          const bool masked = key0 + 128 > C;
          uint32_t vw[4] = {~0u, ~0u, ~0u, ~0u};
          if (masked && row_ok) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int rel = key0 + 32 * w - C;  // drafted index of bit 0 (negative: context)
              if (rel <= -32) continue;
              uint32_t bits;
              if (!mrow) {
                bits = low_mask32(min(i + 1, g.T) - rel);
              } else {
                const int w0 = rel >> 5, sh = rel & 31;  // floor for negative rel
                const uint32_t a = (w0 >= 0 && w0 < A.words) ? __ldg(mrow + w0) : 0u;
                const uint32_t c = (w0 + 1 < A.words) ? __ldg(mrow + w0 + 1) : 0u;
                bits = __funnelshift_r(a, c, sh) & low_mask32(g.T - rel);
                if (rel < 0) bits |= low_mask32(-rel);
              }
              vw[w] = bits;
            }
          }
          if (!mbar_wait(&bars[kBarSFull + X], seen & 1)) { ok = false; break; }
          tc_fence_after();
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
          if (kTwo) {  // the scores are in registers: S is free for the other group's
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[kBarSFree]);
          }
          if (warp_in) {
            if (masked) {
#pragma unroll
              for (int k = 0; k < 128; ++k) sv[k] = ((vw[k >> 5] >> (k & 31)) & 1u) ? sv[k] : -INFINITY;
            }
            float mx[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) mx[x] = max3f(sv[x], sv[8 + x], sv[16 + x]);
#pragma unroll
            for (int k = 24; k < 120; k += 16)
#pragma unroll
              for (int x = 0; x < 8; ++x) mx[x] = max3f(mx[x], sv[k + x], sv[k + 8 + x]);
#pragma unroll
            for (int x = 0; x < 8; ++x) mx[x] = fmaxf(mx[x], sv[120 + x]);
            const float mt = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
            const float m_new = fmaxf(m_used, mt * c2);
            // lanes without a row hold whatever shared memory held: they have no vote, or runs would differ
            const bool need = row_ok && m_new > m_used + kRescaleThreshold;
            const bool any = __any_sync(0xFFFFFFFFu, need);
            float alpha = 1.f;
            if (any && m_new != -INFINITY) {
              alpha = (m_used == -INFINITY) ? 0.f : ex2(m_used - m_new);
              m_used = m_new;
            }
            const float mref = (m_used == -INFINITY) ? 0.f : m_used;
            const uint64_t c2x2 = pk2(c2, c2), negm = pk2(-mref, -mref);
            uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
            if (!pv_done()) { ok = false; break; }
            // P rounded to bf16 for the second MMA (its operand type is V's); the row sum keeps fp32
#pragma unroll
            for (int h = 0; h < 64 / kPChunk; ++h) {
              uint32_t pk[kPChunk];
#pragma unroll
              for (int k = 0; k < kPChunk; ++k) {
                const int e = 2 * kPChunk * h + 2 * k;
                const uint64_t x = fma2(pk2(sv[e], sv[e + 1]), c2x2, negm);
                float x0, x1;
                up2(x, x0, x1);
                const uint64_t p = pk2(ex2(x0), ex2(x1));
                acc[k & 1] = add2(acc[k & 1], p);
                float p0, p1;
                up2(p, p0, p1);
                pk[k] = pack_bf16x2(p0, p1);
              }
              tmem_st4(tP + kPChunk * h, pk);
            }
            float a0, a1, a2, a3;
            up2(acc[0], a0, a1);
            up2(acc[1], a2, a3);
            l = l * alpha + ((a0 + a1) + (a2 + a3));
            if (any && !first) {  // O_X: its previous PV has completed (before S was ready, or waited for)
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                tmem_st32(tO + 32 * c, o);
              }
            }
            tmem_st_wait();
            first = false;
          } else if (!pv_done()) {
            ok = false;
            break;
          }
          ++seen;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarPFull + X]);
        }
      if (!ok) break;

      // ---- the segment's end: O / l and LSE, or the part's unnormalised state.
      // O goes to registers first, so that the next segment's products may start
      // while it is written.  Up to 128 rows, each group takes half of the
      // columns of both groups' O.
      constexpr int kCols = kTwo ? D : D / 2;  // columns that a thread writes
      const int col0 = kTwo ? 0 : X * kCols;
      float ov[kCols];
      if (kTwo) {
        if (rows > 0 ? !pv_done() : !mbar_wait(&bars[kBarODone + X], idle++ & 1)) { ok = false; break; }
        // every warp loads, with rows or not: values defined on one path only would stay live around the loop
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) tmem_ld32(tO + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(ov + 32 * c));
        tmem_ld_wait();
      } else {
        if (s > 0 && !mbar_wait(&bars[kBarOFree], (s - 1) & 1)) { ok = false; break; }  // ml has been read
        ml[128 * X + r] = make_float2(m_used, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarML]);
        if (!mbar_wait(&bars[kBarML], s & 1) || !mbar_wait(&bars[kBarODone], s & 1) ||
            !mbar_wait(&bars[kBarODone + 1], s & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const float2 s0 = ml[r], s1 = ml[128 + r];
        const float m = fmaxf(s0.x, s1.x), ref = m == -INFINITY ? 0.f : m;
        const float w0 = ex2(s0.x - ref), w1 = ex2(s1.x - ref);
        m_used = m;
        l = s0.y * w0 + s1.y * w1;
        const uint32_t t0 = tmem + lane_base + kColO + col0;
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t q[32];
          tmem_ld32(t0 + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(ov + 32 * c));
          tmem_ld32(t0 + 128 + 32 * c, q);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x)  // a group without a tile has no O
            ov[32 * c + x] = ov[32 * c + x] * w0 + (nt > 1 ? __uint_as_float(q[x]) * w1 : 0.f);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars[kBarOFree + (kTwo ? X : 0)]);
        if (!kTwo) mbar_arrive(&bars[kBarOFree + 1]);
      }
      if (!row_ok) continue;
      const bool some = !(l == 0.f);  // an attended key (a NaN among them shows in l)
      if (g.t0 == 0 && g.t1 == g.tiles) {
        const int64_t grow = (int64_t)(g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + rr;
        const float inv = some ? 1.f / l : 0.f;
        uint4* dst = reinterpret_cast<uint4*>(A.o + grow * D + col0);
#pragma unroll
        for (int x = 0; x < kCols / 8; ++x) {
          uint32_t pk[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) pk[y] = pack_bf16x2(ov[8 * x + 2 * y] * inv, ov[8 * x + 2 * y + 1] * inv);
          dst[x] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
        if (A.lse && col0 == 0) A.lse[grow] = some ? (m_used + __log2f(l)) * 0.69314718055994531f : -INFINITY;
      } else {
        const int width = min(256, A.R - 256 * g.rb), full = min(256, A.R), rw = rr - 256 * g.rb;
        const int64_t slot = 2 * blockIdx.x + (g.t0 > 0 ? 0 : 1);
        float4* part = A.part + slot * (D / 4) * full + (int64_t)(col0 / 4) * width + rw;
#pragma unroll
        for (int x = 0; x < kCols / 4; ++x, part += width)
          *part = make_float4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
        if (col0 == 0) A.part_ml[slot * full + rw] = make_float2(m_used, l);
      }
    }
  }
  if (!ok) {
    misc[2] = 1;
    atomicCAS(A.err, 0, (int)kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of the items that the line's cuts went through, in key
// order.  Grid: (items, chunks of a block's rows x d/4 values).
constexpr int kJoinThreads = 128;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int items = A.Hkv * A.RB;
  const int b = (int)(blockIdx.x / items), item = (int)(blockIdx.x % items);
  const int64_t W = A.prefix[A.B], p0 = A.prefix[b], p1 = A.prefix[b + 1];
  if (p1 == p0) return;
  const int64_t tiles = (p1 - p0) / items, s0 = p0 + item * tiles, s1 = s0 + tiles;
  const int G = parts(W);  // part c holds tile x: the largest c with W c / G <= x
  const int c0 = (int)(((s0 + 1) * G - 1) / W), c1 = (int)((s1 * G - 1) / W);
  if (c0 == c1) return;  // one CTA finished it
  const int rb = item % A.RB, kvh = item / A.RB;
  const int width = min(256, A.R - 256 * rb), full = min(256, A.R);
  const int e = blockIdx.y * kJoinThreads + threadIdx.x;
  if (e >= width * (D / 4)) return;
  const int c4 = e / width, rw = e - c4 * width, rr = 256 * rb + rw;
  const int T = A.tree_len ? A.tree_len[b] : A.n;
  if (rr % A.n >= T) return;
  auto slot = [&](int c) { return (int64_t)(2 * c + (c == c0 ? 1 : 0)); };  // the first part starts the item
  // one pass, kAhead parts at a time: their loads are all in flight before the first is used
  constexpr int kAhead = 8;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float2* ml = A.part_ml + rw;
  const float4* part = A.part + (int64_t)c4 * width + rw;
  for (int c = c0; c <= c1; c += kAhead) {
    float2 x[kAhead];
    float4 y[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int64_t sl = slot(min(c + k, c1));
      x[k] = ml[sl * full];
      y[k] = part[sl * (D / 4) * full];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k > c1) x[k] = make_float2(-INFINITY, 0.f);
      top = fmaxf(top, x[k].x);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    const float keep = ex2(m - ref);
    m = top;
    l *= keep;
    o.x *= keep;
    o.y *= keep;
    o.z *= keep;
    o.w *= keep;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (c + k > c1) continue;  // a repeated last part carries nothing (its values may be NaN)
      const float w = ex2(x[k].x - ref);
      l += w * x[k].y;
      o.x += w * y[k].x;
      o.y += w * y[k].y;
      o.z += w * y[k].z;
      o.w += w * y[k].w;
    }
  }
  const bool some = !(l == 0.f);
  const float inv = some ? 1.f / l : 0.f;
  const int64_t grow = (int64_t)(b * A.Hq + kvh * (A.Hq / A.Hkv)) * A.n + rr;
  *reinterpret_cast<uint2*>(A.o + grow * D + 4 * c4) =
      make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (c4 == 0 && A.lse) A.lse[grow] = some ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct TreeWs {
  size_t prefix, ml, part, total;
};
TreeWs tree_ws(const msa_shape& s) {
  const int64_t R = (int64_t)(s.Hq / s.Hkv) * s.n, full = R < 256 ? R : 256;
  TreeWs w;
  w.prefix = 0;
  w.ml = align256((size_t)(s.B + 1) * 8);
  w.part = align256(w.ml + (size_t)(2 * kCtas * full) * 8);
  w.total = align256(w.part + (size_t)(2 * kCtas * full) * s.d_h * 4);
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

template <int D, bool kTwo>
msa_status launch_tree(const TreeMaps& maps, const TreeArgs& a, bool join, cudaStream_t stream) {
  auto kern = tree_attn_kernel<D, kTwo>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kAlloc) != cudaSuccess)
    return MSA_ERR_CUDA;
  kern<<<kCtas, kThreads, Lay<D>::kAlloc, stream>>>(maps, a);
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
  cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * a.RB), (unsigned)ceil_div((int64_t)full * (D / 4), kJoinThreads));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_join_kernel<D>, a) != cudaSuccess) return MSA_ERR_CUDA;
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
  a.prefix = reinterpret_cast<int64_t*>(base + w.prefix);
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
  if (a.R > 128)
    return shape->d_h == 128 ? launch_tree<128, true>(maps, a, join, stm) : launch_tree<64, true>(maps, a, join, stm);
  return shape->d_h == 128 ? launch_tree<128, false>(maps, a, join, stm) : launch_tree<64, false>(maps, a, join, stm);
}
