// Attention of drafted tokens over a paged cache held in 4 bits (decode,
// speculative trees, windows), sm_103a.
//
// What it computes: msa_attn_tree's o_i = Σ_j e^{s_ij} v_j / Σ_j e^{s_ij} over
// keys and values that are e2m1 codes times e4m3 scales of 16 channels.
//
// What bounds it: HBM, 144 bytes a key and KV head (d = 128) where the bf16 cache
// has 512; at that rate an SM has about 790 cycles for a tile of 128 keys, so
// nothing else may cost more.  Codes become fp16 (exact: 6 bits) for the tensor
// core; the products are turned round so that the few query rows are the
// narrow side:
//   S^T [128 keys x N rows] = K Q^T   A = K in TMEM, where the threads that
//                                     decode it put it: it passes shared memory
//                                     once, as codes
//   O^T [d x N] += V^T P^T            A = V in shared memory, [key][channel]
// N = 16, 32 or 64 rows; a group of more rows is cut into blocks of 64 (with
// bf16's layout, rows as the wide side, a tile of one row costs as much softmax
// as one of 32: a warp's lanes are rows).  Softmax threads are keys: all lanes
// work whatever the number of rows, and a weight goes to shared memory as it is
// made.  q is fp16 too: a power of two per row (undone in the scores) brings its
// largest value to 2^14, so that every bf16 down to 2^-30 of it is exact.  Weights are
// rounded to fp16 at 2^7 times their share of the reference, a maximum that
// rises when a score passes it by 2^8.
//
// Split: as tree.cu's (tree.cuh), one part of the line of tiles per CTA.
//
// A CTA (32 warps, 24 for 64 rows; one CTA per SM):
//   softmax (8)  thread = key = TMEM lane, in two groups that take the tiles
//                in turn, each with its own references, sums and O: a tile's
//                chain (scores, exponentials, weights) is latency, two of them
//                side by side are not
//   K (4 or 8)   decode: global memory -> shared memory (cp.async into slots of
//                the thread's own) -> registers -> TMEM (four buffers, two for
//                64 rows)
//   V (4 or 8)   the same into shared memory (three buffers, two for 64 rows).  A
//                row that no query sees becomes zeros (its page may hold anything)
//   plan (1)     the part's segments
//   scores (1), products with V (1): the issuers, an elected thread each
//   output (4)   thread = channel: both groups' O joined, beside the softmax of
//                the next segment; Q of the one behind that to fp16
//
// Measured (one launch and its join, captured, inputs larger than the L2; floor =
// bytes at 6.8 TB/s): 64 requests of 1K to 16K tokens, one row group of 4
// (32/8 heads of 128) 110 us (floor 53; the bf16 cache's 188); one request of a
// million tokens, 20 rows, 374 (178); 16 requests of 4K to 32K tokens with trees of
// 48 (192 rows: three passes over the codes) 431 (66); of 16 (64 rows) 154 (34),
// of 8 (32 rows) 100 (33); 256 requests of 100 to 1000 tokens 121 (17); heads of 64 94 (26); through 128 + 1024
// keys 53 (13); one of 2047 tokens, 2 / 1 heads of 64, 13.4.  The next 1024 tokens behind 128K
// (4096 rows: 64 passes) 4149 (1154, of operations; the bf16 cache 1559), behind 16K 614 (152; 245).
//
// What bounds it now: 16 warps that decode issue about 300 instructions for 32 keys of
// K or V (16 conversions and 16 products a 32 channels, at half rate each), 600 of a
// scheduler's 1350 cycles a tile with 8 rows; the schedulers issue 0.72 a cycle, the
// rest is instruction fetch (eight roles) and waits for each other.  With 64 rows a
// softmax group's chain, 3300 cycles a tile (taken when 192 rows were at 451 us): scores 300,
// first pass 600, vote 250, weights 900, raises 600 where references are passed often.
//
// Tried and slower (the two cases were at 114 and 451 us then): codes through a ring of bulk
// copies with a loading warp (121 us for 114 in the decode case: one more hand-over a tile,
// and its warp's waits), or loaded into
// registers a tile ahead (spills); one softmax group for all tiles (139 us; 64 rows and
// 24 warps were even: 450); the chunk loop of the decode unrolled twice (118 us: fetch);
// raising only the rows whose reference was passed (557 us for 451 with 192 rows: the
// others follow soon after, a raise each).
#include "kv4.cuh"
#include "tree.cuh"

namespace msa {

namespace {

constexpr int kBlock = 64;  // rows of an item
constexpr int kSegSlots = 16;

// Warps of a CTA for blocks of up to kR rows.  With 64 rows the softmax threads' scores and sums leave the others few
// registers, and the softmax is the longer part: K and V are decoded by one group of warps each.
template <int kR>
struct Roles {
  static constexpr int kGroups = kR >= 64 ? 1 : 2;  // of four warps that decode K, and V
  static constexpr int kK = 8, kV = kK + 4 * kGroups, kPlan = kV + 4 * kGroups, kIssueQK = kPlan + 1,
                       kIssuePV = kPlan + 2, kOut = kPlan + 4, kThreads = 32 * (kOut + 4);
};
constexpr uint32_t kTmemCols = 512;
// TMEM columns of products of N rows: K (four buffers of 64 columns, with N = 64 two), S [2], O [segment parity][group]
constexpr int k_bufs(int N) { return N == 64 ? 2 : 4; }
constexpr uint32_t col_s(int N) { return 64 * k_bufs(N); }
constexpr uint32_t col_o(int N) { return col_s(N) + 2 * N; }
constexpr float kTop = 7.f, kRaise = 8.f;                // log2: weight of the reference, how far a score may pass it

// of tiles j: [2] in use j & 1, [4] j & 3, [3] j % 3 (fewer with 64 rows)
enum {
  kBarKFull = 0,     // [4] K is in TMEM
  kBarKFree = 4,     // [4] its product is done
  kBarVFull = 8,     // [3] V is in shared memory
  kBarVFree = 12,    // [3]
  kBarQK = 16,       // [2] scores are in TMEM
  kBarSEmpty = 18,   // [2] scores are in registers
  kBarPFull = 20,    // [2] weights are in shared memory
  kBarPV = 22,       // [2] the product with V is done: weights are free
  kBarQFull = 24,    // [2] Q of the segment
  kBarQEmpty = 26,   // [2] its products are done, its factors have been read
  kBarGroup = 28,    // [2] the warps of a softmax group among themselves
  kBarSums = 30,     // [2] a segment's references and sums are written
  kBarODone = 32,    // [2] its products are done
  kBarOFree = 34,    // [2] its O and sums have been read
  kBarOut = 36,      // the output warps among themselves
  kBarDrain = 37,    // [2] after giving up: an issuer's products are done
  kBarSegFull = 39,  // [kSegSlots]
  kBarSegEmpty = kBarSegFull + kSegSlots,
  kNumBars = kBarSegEmpty + kSegSlots
};

// N: rows of a product.  Up to 32, both buffers of weights lie side by side in one tile of 64, and V has three buffers.
template <int D, int N>
struct Lay4 {
  static constexpr int kUnit = D / 2 + D / 16;   // bytes of a token, K or V
  static constexpr int kTile = 128 * D * 2;      // a tile of V in fp16
  static constexpr int kQTile = N * D * 2, kVBufs = N == 64 ? 2 : 3;
  static constexpr int kPTile = N == 64 ? 128 * kBlock * 2 : 64, kPTiles = N == 64 ? 2 : 1;  // (64: half of a row of 128 bytes)
  static constexpr int kV = 0, kP = kV + kVBufs * kTile, kQ = kP + kPTiles * 128 * kBlock * 2, kRaw = kQ + 2 * kQTile;
  static constexpr int kSlot = 128 * kUnit, kDepth = 4 * (128 / D);  // codes of a tile's K or V; tiles ahead, of all groups
  static constexpr int kSeg = kRaw + 2 * kDepth * kSlot;
  static constexpr int kRows = (kSeg + kSegSlots * (int)sizeof(Seg) + 15) / 16 * 16;
  // per row, [segment parity]: factors, rows, window ends; [group]: references, factors of a raise, maxima [warp];
  // [segment parity][group]: factors of O, last references, sums [warp]; [group]: the keys of a tile that it sees
  static constexpr int kWsum = kRows + (6 + 4 + 8 + 4 + 4 + 16 + 8) * kBlock * 4;
  static constexpr int kBars = kWsum + 32 * 8;
  static constexpr int kMisc = kBars + kNumBars * 8;  // [0] TMEM base, [2] abort, [3] tiles issued, [4] flags [group][2]
  static constexpr int kStart = kMisc + 32;
  static constexpr int kNeed = kStart + 16;
  static constexpr int kAlloc = kNeed > 120 * 1024 ? kNeed : 120 * 1024;  // one CTA per SM: its TMEM is all there is
  static_assert(kRows % 16 == 0 && kWsum % 8 == 0 && kStart % 8 == 0, "alignment");
  static_assert(kAlloc <= 227 * 1024, "shared memory");
};

struct Kv4Args {
  TreeArgs t;
  const __nv_bfloat16* q;
  const uint8_t* data;
  float v_scale;
};

// Instruction descriptor, kind::f16 with fp16 inputs and an fp32 accumulator (fields as in idesc_bf16_f32).
constexpr uint32_t idesc_f16_f32(int M, int N, bool a_mn_major, bool b_mn_major) {
  return idesc_bf16_f32(M, N, a_mn_major, b_mn_major) & ~((1u << 7) | (1u << 10));
}

// `bytes` (16, or 8 or 4 for scales) of a thread's own to shared memory; none of them: zeros.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint8_t* dst, const uint8_t* src, bool there) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? kBytes : 0), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ float warp_max(float x) {  // a NaN among others is left out
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 32 channels of a token: 16 bytes of codes and two scales, as 16 fp16 pairs.
__device__ __forceinline__ void decode32(uint4 codes, uint32_t scales, uint32_t (&r)[16]) {
  const uint32_t two = f16x2_of_e4m3x2(scales & 0xFFFFu);
  const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
  f16_of_codes(codes.x, s0, *reinterpret_cast<uint32_t(*)[4]>(r));
  f16_of_codes(codes.y, s0, *reinterpret_cast<uint32_t(*)[4]>(r + 4));
  f16_of_codes(codes.z, s1, *reinterpret_cast<uint32_t(*)[4]>(r + 8));
  f16_of_codes(codes.w, s1, *reinterpret_cast<uint32_t(*)[4]>(r + 12));
}
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&s)[D / 64]) {
  if constexpr (D == 128) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    s[0] = x.x;
    s[1] = x.y;
  } else {
    s[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
// The scales of the next 32 channels to the front.
template <int D>
__device__ __forceinline__ void next_scales(uint32_t (&s)[D / 64]) {
  if constexpr (D == 128) {
    s[0] = __funnelshift_r(s[0], s[1], 16);
    s[1] >>= 16;
  } else {
    s[0] >>= 16;
  }
}

// Sums l[0 .. n) over the warp; each step halves what a lane keeps: 64 rows end as rows 2 lane and 2 lane + 1 in l[0] and
// l[1], 32 as row `lane`, 16 as row lane / 2 in l[0].
template <int n, int o>
__device__ __forceinline__ void lane_sums(float* l, int lane) {
  if constexpr (n > 1) {
    const bool up = lane & o;
#pragma unroll
    for (int x = 0; x < n / 2; ++x) {
      const float give = up ? l[x] : l[x + n / 2], keep = up ? l[x + n / 2] : l[x];
      l[x] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  } else {
    l[0] += __shfl_xor_sync(0xFFFFFFFFu, l[0], o);
  }
  if constexpr (o > 1) lane_sums<(n > 1 ? n / 2 : 1), o / 2>(l, lane);
}

template <int D, int kR, bool kWin>
__global__ void __launch_bounds__(Roles<kR>::kThreads, 1) kv4_attn_kernel(const __grid_constant__ Kv4Args X) {
  constexpr int kN = kR < 16 ? 16 : kR;  // rows of a product (columns behind kR hold anything)
  using Ly = Lay4<D, kN>;
  using Ro = Roles<kR>;
  constexpr int kVBufs = Ly::kVBufs;
  constexpr int kThreads = Ro::kThreads, kGroups = Ro::kGroups;
  const TreeArgs& A = X.t;
  extern __shared__ __align__(1024) uint8_t sm[];  // swizzled tiles start on 1 KB
  if (smem_u32(sm) & 1023) {
    if (threadIdx.x == 0) atomicCAS(A.err, 0, (int)kErrTimeout);
    if (blockIdx.x == 0 && threadIdx.x == 0) *A.count = 0;  // nothing to join
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Ly::kBars);
  Seg* segs = reinterpret_cast<Seg*>(sm + Ly::kSeg);
  float* rowf = reinterpret_cast<float*>(sm + Ly::kRows);  // [2][kBlock]
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + Ly::kMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    tmem_alloc(const_cast<uint32_t*>(&misc[0]), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 32 * Ro::kIssueQK) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars[kBarQK + x], 1);
      mbar_init(&bars[kBarSEmpty + x], 4);
      mbar_init(&bars[kBarPFull + x], 4);
      mbar_init(&bars[kBarPV + x], 1);
      mbar_init(&bars[kBarQFull + x], 4);
      mbar_init(&bars[kBarQEmpty + x], 9);
      mbar_init(&bars[kBarGroup + x], 4);
      mbar_init(&bars[kBarSums + x], 8);
      mbar_init(&bars[kBarODone + x], 1);
      mbar_init(&bars[kBarOFree + x], 4);
      mbar_init(&bars[kBarDrain + x], 1);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(&bars[kBarKFull + x], 4);
      mbar_init(&bars[kBarKFree + x], 1);
      mbar_init(&bars[kBarVFull + x], 4);
      mbar_init(&bars[kBarVFree + x], 1);
    }
    mbar_init(&bars[kBarOut], 4);
    for (int s = 0; s < kSegSlots; ++s) {
      mbar_init(&bars[kBarSegFull + s], 1);
      mbar_init(&bars[kBarSegEmpty + s], 8 + 8 * kGroups + 2 + 4);  // softmax, K and V, issuers, output
    }
    misc[2] = misc[3] = 0;
    for (int x = 4; x < 8; ++x) misc[x] = 0xFFFFFFFFu;
    fence_mbar_init();
  }
  // ---- this CTA's part of the line of tiles, and the request it starts in
  const int items = A.Hkv * A.RB;  // items of a request
  int64_t* wsum = reinterpret_cast<int64_t*>(sm + Ly::kWsum);
  int64_t* start = reinterpret_cast<int64_t*>(sm + Ly::kStart);
  int64_t W = 0;  // all tiles
  {
    const int per = (A.B + kThreads - 1) / kThreads;
    const int b0 = min(A.B, (int)threadIdx.x * per), b1 = min(A.B, b0 + per);
    auto tiles = [&](int b) -> int64_t {
      int L, T;
      bool bad;
      const bool live = request(A, b, L, T, bad);
      if (bad && blockIdx.x == 0) atomicCAS(A.err, 0, (int)kErrIndex);
      return live ? (int64_t)items * span_of<kWin>(A, L, T).tiles : 0;
    };
    int64_t own = 0, mine = 0;
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
    const int64_t lo = part_begin(W, kCtas, blockIdx.x);  // at or above W: no part
    for (int b = b0; b < b1; ++b) {
      const int64_t t = per == 1 ? own : tiles(b);
      if (at <= lo && lo < at + t) { start[0] = b; start[1] = at; }
      at += t;
    }
  }
  const int G = parts(W, kCtas);
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.count = G;
  const int64_t begin = part_begin(W, kCtas, blockIdx.x);
  const int cnt = (int)blockIdx.x < G ? (int)(part_begin(W, kCtas, blockIdx.x + 1) - begin) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (cnt == 0) {  // no part
    if (warp == 0) tmem_dealloc(misc[0], kTmemCols);
    return;
  }
  const uint32_t tmem = misc[0];

  auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_long(bar, parity, &misc[2]); };
  // A wait for the end of a segment, of any number of tiles: again as long as tiles are issued meanwhile.
  auto wait_segment = [&](uint64_t* bar, uint32_t parity) -> bool {
    for (uint32_t issued = misc[3];;) {
      if (wait(bar, parity)) return true;
      if (misc[2] || misc[3] == issued) return false;
      issued = misc[3];
    }
  };
  // Segment s of the part as its readers see it; false: no more, or gave up.  (The planner may be waiting for a slot.)
  bool ok = true;
  auto next_seg = [&](int s, Seg& g) -> bool {
    const int slot = s % kSegSlots;
    if (misc[2] || !wait_segment(&bars[kBarSegFull + slot], (s / kSegSlots) & 1)) { ok = false; return false; }
    g = segs[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[kBarSegEmpty + slot]);
    return g.b >= 0;
  };
  // Tile j of the part is in buffer j & 1, use number j >> 1 of it (K and V: of kKBufs and kVBufs); segment s likewise.
  auto done = [&](int bar, int j) { return wait(&bars[bar + (j & 1)], (j >> 1) & 1); };
  constexpr int kKBufs = k_bufs(kN);
  constexpr uint32_t kColS = col_s(kN), kColO = col_o(kN);
  static_assert(kColO + 4 * kN <= kTmemCols, "TMEM columns");
  auto used_before = [&](int bar, int j) { return wait(&bars[bar + (j & 1)], ((j >> 1) & 1) ^ 1); };  // (first use: at once)
  // numbers of the rows (see Lay4)
  float* rows = rowf;
  int* rowi = reinterpret_cast<int*>(rows + 2 * kBlock);    // [parity] drafted token of the row, -1: no row
  int* rowend = reinterpret_cast<int*>(rows + 4 * kBlock);  // [parity] kWin: end of the keys behind its window
  constexpr int kRowRef = 6 * kBlock, kRowAlpha = 8 * kBlock, kRowMax = 10 * kBlock, kRowFo = 18 * kBlock,
                kRowLast = 22 * kBlock, kRowSums = 26 * kBlock, kRowMask = 42 * kBlock;
  const int P = 1 << A.page_shift;

  // The softmax threads hold kR scores and sums, so they take registers of the others: the block starts with 8 x 128
  // threads x 64 (kR = 64: 6 x 128 x 80); 2 x 88 + 6 x 56 = 8 x 64, 2 x 128 + 4 x 56 = 6 x 80
  if (warp >= Ro::kK) {
    if (kR >= 16) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < Ro::kPlan) {
      // ------------------------------------------------------------ K to TMEM, V to shared memory: group H the tiles
      // j = H mod kGroups, thread = key.  A thread copies its key's codes into slots of its own, kDepth tiles ahead, and
      // looks up their page one tile earlier still; nobody waits for anybody until they are decoded.  One loop for K and V.
      constexpr int kDepth = Ly::kDepth / kGroups;
      const bool is_v = warp >= Ro::kV;
      const int H = ((warp - Ro::kK) >> 2) & (kGroups - 1), q = warp & 3, r = 32 * q + lane;
      const uint32_t to = tmem + ((uint32_t)(32 * q) << 16);
      const uint32_t turn = (r & 7) << 4;  // the 128-byte swizzle of row r
      const int free_bar = is_v ? kBarVFree : kBarKFree, full_bar = is_v ? kBarVFull : kBarKFull;
      const int bufs = is_v ? kVBufs : kKBufs;
      int buf = H, use = 0;  // of tile j: its buffer, and whose use it is
      const uint8_t* const codes0 = X.data + (is_v ? P * Ly::kUnit : 0) + (r & (P - 1)) * 16;
      const int scales_at = P * (D / 2) + (r & (P - 1)) * (D / 16 - 16);  // behind the token's codes
      uint8_t* const slots = sm + Ly::kRaw + ((is_v ? kGroups : 0) + H) * kDepth * Ly::kSlot + r * 16;
      const int slot_scales = 128 * (D / 2) + r * (D / 16 - 16);
      Seg g;
      Span span = {};
      int s = 0, x = 0;       // of the tile that is looked up: its segment, its place there
      int page = 0, kvh = -1;  // its page, not used before fetch (a load is on its way); its head, -1: not read
      bool more = next_seg(s++, g);
      if (more) span = span_of<kWin>(A, g.L, g.T, g.rb);
      // the next tile of this group, `by` on, and the unit that holds its row
      auto look = [&](int by) {
        x += by;
        while (more && x >= g.t1 - g.t0) {
          x -= g.t1 - g.t0;
          more = next_seg(s++, g);
          if (more) span = span_of<kWin>(A, g.L, g.T, g.rb);
        }
        // (no branch round the load: its value would be waited for where the paths meet)
        const int key = span.key0(g.t0 + x) + r;
        const bool seen = more && key < g.L && !(kWin && key >= span.hole && key < span.lo);  // else zeros, whatever is there
        page = __ldg(A.table + (seen ? (int64_t)g.b * A.max_pages + (key >> A.page_shift) : 0));
        kvh = seen ? g.kvh : -1;
      };
      auto fetch = [&](uint8_t* slot) {  // what was looked up
        bool there = kvh >= 0;
        if (there && (unsigned)page >= (unsigned)A.num_pages) {
          atomicCAS(A.err, 0, (int)kErrIndex);  // not followed, the call has failed
          there = false;
        }
        const uint8_t* src = codes0 + (there ? (int64_t)page * A.Hkv + kvh : 0) * (2 * P * Ly::kUnit);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) copy_async<16>(slot + c * 2048, src + c * 16 * P, there);
        copy_async<D / 16>(slot + slot_scales, src + scales_at, there);
        copy_commit();
      };
      look(H);
#pragma unroll 1
      for (int d = 0; d < kDepth; ++d) {
        fetch(slots + d * Ly::kSlot);
        look(kGroups);
      }
      int at = 0;  // slot of tile j
      for (int j = H; j < cnt && ok; j += kGroups) {
        uint8_t* const slot = slots + at * Ly::kSlot;
        at = at + 1 == kDepth ? 0 : at + 1;
        copy_wait<kDepth - 1>();
        uint32_t scales[D / 64];
        load_scales<D>(slot + slot_scales, scales);
        if (!wait(&bars[free_bar + buf], (use & 1) ^ 1)) { ok = false; break; }
        tc_fence_after();
        uint8_t* v = sm + Ly::kV + buf * Ly::kTile + r * 128;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[16];
          decode32(*reinterpret_cast<const uint4*>(slot + c * 2048), scales[0], w);
          next_scales<D>(scales);
          if (is_v) {
            uint8_t* dst = v + (c >> 1) * 16384;
            const uint32_t at = turn ^ (uint32_t)((c & 1) << 6);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<uint4*>(dst + (at ^ (uint32_t)(y << 4))) = make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
          } else {
            tmem_st16(to + 64 * buf + 16 * c, w);
          }
        }
        if (is_v) {
          fence_proxy_async_smem();
        } else {
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[full_bar + buf]);
        buf += kGroups;
        if (buf >= bufs) buf -= bufs, ++use;
        fetch(slot);
        look(kGroups);
      }
      copy_wait<0>();  // (a CTA does not leave with copies under way)
    } else if (warp == Ro::kPlan) {
      // ------------------------------------------------------------ planner: the part's segments, as far ahead as the slots go
      int64_t at = start[1], pos = begin;  // first tile of request b, of the next segment
      const int64_t hi = begin + cnt;
      int b = (int)start[0], s = 0;
      if (lane == 0) note_cut<false, kCtas, kWin>(A, W, blockIdx.x, (int)start[0], start[1]);
      __syncwarp();
      while (ok) {
        Seg g;
        g.b = -1;  // the end's mark
        if (pos < hi) {
          bool bad;
          int64_t tiles = 0;
          for (; b < A.B; ++b) {  // pos < hi <= W: a request holding it exists
            const bool live = request(A, b, g.L, g.T, bad);
            g.tiles = span_of<kWin>(A, g.L, g.T).tiles;
            tiles = live ? (int64_t)items * g.tiles : 0;
            if (pos < at + tiles) break;
            at += tiles;
          }
          if (b >= A.B) { ok = false; break; }
          g.b = b;
          const int item = (int)quotient(pos - at, g.tiles);
          g.kvh = item / A.RB;
          g.rb = item - g.kvh * A.RB;
          g.t0 = (int)(pos - at - (int64_t)item * g.tiles);
          const int64_t left = hi - pos;
          g.t1 = left < g.tiles - g.t0 ? g.t0 + (int)left : g.tiles;
          g.r0 = g.t0;
          g.r1 = g.t1;
          pos += g.t1 - g.t0;
        }
        const int slot = s % kSegSlots;
        if (misc[2] || !wait_segment(&bars[kBarSegEmpty + slot], ((s / kSegSlots) & 1) ^ 1)) { ok = false; break; }
        if (lane == 0) {
          segs[slot] = g;
          mbar_arrive(&bars[kBarSegFull + slot]);
        }
        ++s;
        if (g.b < 0) break;
      }
    } else if (warp == Ro::kIssueQK) {
      // ------------------------------------------------------------ scores.  (A warp of their own: behind a product
      // with V that waits for its weights, a group's next scores would come a whole chain later.)
      constexpr uint32_t id = idesc_f16_f32(128, kN, false, false);
      const uint64_t dq = sdesc_sw128(smem_u32(sm + Ly::kQ), 16, 1024);
      const bool leader = elect_one();
      int j = 0;
      Seg g;
      for (int s = 0; j < cnt && next_seg(s, g); ++s) {
        if (!wait(&bars[kBarQFull + (s & 1)], (s >> 1) & 1)) { ok = false; break; }
        const uint64_t q = dq + (uint64_t)((s & 1) * (Ly::kQTile >> 4));
        for (int t = g.t0; t < g.t1; ++t, ++j) {
          const int buf = j & (kKBufs - 1), use = kKBufs == 4 ? j >> 2 : j >> 1;
          if (!wait(&bars[kBarKFull + buf], use & 1) || !used_before(kBarSEmpty, j)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
#pragma unroll 2
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ts(tmem + kColS + kN * (j & 1), tmem + 64 * buf + 8 * kk,
                          q + (uint64_t)((kk >> 2) * (kN * 8) + (kk & 3) * 2), id, kk > 0 ? 1u : 0u);
            mma_commit(&bars[kBarQK + (j & 1)]);
            mma_commit(&bars[kBarKFree + buf]);
            if (t + 1 == g.t1) mma_commit(&bars[kBarQEmpty + (s & 1)]);
          }
          __syncwarp();
        }
        if (!ok) break;
      }
    } else if (warp == Ro::kIssuePV) {
      // ------------------------------------------------------------ products with V
      constexpr uint32_t id = idesc_f16_f32(128, kN, true, true);  // (d = 64: rows 64 .. of O^T hold anything)
      const uint64_t dv = sdesc_sw128(smem_u32(sm + Ly::kV), 16384, 1024);
      const uint64_t dp = sdesc_sw128(smem_u32(sm + Ly::kP), 16384, 1024);
      const bool leader = elect_one();
      int j = 0, buf = 0, use = 0;  // V's buffer, and whose use it is
      Seg g;
      for (int s = 0; j < cnt && next_seg(s, g); ++s) {
        if (!used_before(kBarOFree, s)) { ok = false; break; }
        const uint32_t o = tmem + kColO + 2 * kN * (s & 1);
        for (int t = g.t0; t < g.t1; ++t, ++j) {
          if (!wait(&bars[kBarVFull + buf], use & 1) || !done(kBarPFull, j)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
            const bool more = t - g.t0 >= 2;  // not the first of its group in the segment
            const uint64_t v = dv + (uint64_t)(buf * (Ly::kTile >> 4)), p = dp + (uint64_t)((j & 1) * (Ly::kPTile >> 4));
#pragma unroll 2
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(o + kN * (j & 1), v + (uint64_t)(kk * 128), p + (uint64_t)(kk * 128), id, (more || kk > 0) ? 1u : 0u);
            mma_commit(&bars[kBarPV + (j & 1)]);
            mma_commit(&bars[kBarVFree + buf]);
            if (t + 1 == g.t1) mma_commit(&bars[kBarODone + (s & 1)]);
            misc[3] = j + 1;
          }
          __syncwarp();
          if (++buf == kVBufs) buf = 0, ++use;
        }
        if (!ok) break;
      }
    } else if (warp >= Ro::kOut) {
      // ------------------------------------------------------------ Q to fp16; output: both groups' O joined, thread = channel
      const int w4 = warp & 3, tid = 32 * w4 + lane;
      const uint32_t lane_base = (uint32_t)(32 * w4) << 16;
      // Q of segment s: eight rows a warp at a time, all on their way before the first is used
      auto convert = [&](int s, const Seg& g) {
        constexpr int kPer = D / 32;
        uint8_t* to = sm + Ly::kQ + (s & 1) * Ly::kQTile;
        float* f = rowf + (s & 1) * kBlock;
        const int64_t q0 = (int64_t)(g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + kBlock * g.rb;
        const int ch = kPer * lane;
#pragma unroll 1
        for (int r0 = w4; r0 < kR; r0 += 32) {
          constexpr int kRows8 = kR < 32 ? kR / 4 : 8;  // rows r0, r0 + 4 ..
          uint32_t u[kRows8][kPer / 2];
          uint32_t live = 0;
#pragma unroll
          for (int y = 0; y < kRows8; ++y) {
            const int r = r0 + 4 * y, rr = kBlock * g.rb + r;
            const bool in = rr < A.R && rr % A.n < g.T;
            live |= (in ? 1u : 0u) << y;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(X.q + (q0 + r) * D + ch);
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x) u[y][x] = in ? __ldg(src + x) : 0u;
          }
#pragma unroll
          for (int y = 0; y < kRows8; ++y) {
            const int r = r0 + 4 * y;
            if (!(live >> y & 1u)) {  // no row: whatever its column holds stays there
              if (lane == 0) f[r] = 0x1p-126f;
              continue;
            }
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x) top = max(top, max(u[y][x] & 0x7FFFu, u[y][x] >> 16 & 0x7FFFu));
            top = max(1u, __reduce_max_sync(0xFFFFFFFFu, top) >> 7);  // exponent of the largest value
            const int up = 141 - (int)top, a = up / 2, c = up - a;      // to 2^14; two factors, since 2^141 is no fp32 number
            const float fa = __uint_as_float((uint32_t)(127 + a) << 23), fc = __uint_as_float((uint32_t)(127 + c) << 23);
            uint32_t h[kPer / 2];
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x)
              h[x] = pack_f16x2(__uint_as_float(u[y][x] << 16) * fa * fc, __uint_as_float(u[y][x] & 0xFFFF0000u) * fa * fc);
            uint8_t* dst = to + (ch >> 6) * (kN * 128) + sw128_offset(r, (ch & 63) >> 3) + (ch & 7) * 2;
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x) reinterpret_cast<uint32_t*>(dst)[x] = h[x];
            if (lane == 0)  // (not zero: -inf times it stays -inf)
              f[r] = fmaxf(0x1p-126f, A.scale_log2 * __uint_as_float((uint32_t)(127 - a) << 23) * __uint_as_float((uint32_t)(127 - c) << 23));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarQFull + (s & 1)]);
      };
      int outs = 0, j0 = 0;
      Seg g, next;
      bool more = next_seg(0, g);
      if (more) convert(0, g);
      if (more) more = next_seg(1, next);
      if (more) convert(1, next);
      for (int s = 0; j0 < cnt && ok; ++s) {
        const int par = s & 1, set = par * kBlock, tiles = g.t1 - g.t0;
        float* fo = rows + kRowFo + 2 * set;
        const bool whole = g.r0 == 0 && g.r1 == g.tiles;
        const int full = min(kBlock, A.R), width = min(kBlock, A.R - kBlock * g.rb);
        const int64_t slot = 2 * (int64_t)blockIdx.x + (g.r0 > 0 ? 0 : 1);
        const int64_t grow = (int64_t)(g.b * A.Hq + g.kvh * (A.Hq / A.Hkv)) * A.n + kBlock * g.rb;
        if (!wait_segment(&bars[kBarSums + par], (s >> 1) & 1)) { ok = false; break; }
        if (tid < kR) {
          // both groups' sums and products at the larger reference
          const float* last = rows + kRowLast + 2 * set + tid;
          const float m0 = last[0], m1 = last[kBlock], m = fmaxf(m0, m1), ref = m == -INFINITY ? 0.f : m;
          const float f0 = ex2(m0 - ref), f1 = ex2(m1 - ref);
          const float* x = rows + kRowSums + 8 * set + tid;
          const float s0 = (x[0] + x[kBlock]) + (x[2 * kBlock] + x[3 * kBlock]);
          const float s1 = (x[4 * kBlock] + x[5 * kBlock]) + (x[6 * kBlock] + x[7 * kBlock]);
          const float sum = f0 * s0 + f1 * s1;
          const bool some = !(sum == 0.f);
          const float inv = whole ? (some ? X.v_scale / sum : 0.f) : X.v_scale;
          fo[tid] = f0 * inv;
          fo[kBlock + tid] = f1 * inv;
          if (rowi[set + tid] >= 0) {
            // (sums are 2^kTop times those of the reference)
            if (!whole) A.part_ml[slot * full + tid] = make_float2(m - kTop, sum);
            else if (A.lse) A.lse[grow + tid] = some ? (m - kTop + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarOut]);
        if (!wait(&bars[kBarOut], outs++ & 1) || !done(kBarODone, s)) { ok = false; break; }
        tc_fence_after();
        // (a segment of one tile has one group's products)
        const int end = (j0 + tiles - 1) & 1;
        const bool two = tiles > 1;
        const uint32_t o0 = tmem + lane_base + kColO + 2 * kN * par;
        if (D == 128 || w4 < 2) {
#pragma unroll 1
          for (int c = 0; c < kR && c < width; c += 8) {
            uint32_t o[8], q[8];
            tmem_ld8(o0 + kN * end + c, o);
            tmem_ld8(o0 + kN * (end ^ 1) + c, q);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int r = c + x;
              if (rowi[set + r] < 0) continue;
              float y = __uint_as_float(o[x]) * fo[end * kBlock + r];
              if (two) y = fmaf(__uint_as_float(q[x]), fo[(end ^ 1) * kBlock + r], y);
              if (whole) A.o[(grow + r) * D + tid] = __float2bfloat16(y);
              else reinterpret_cast<float*>(A.part + slot * (D / 4) * full + (int64_t)(tid >> 2) * width + r)[tid & 3] = y;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarOFree + par]);
        j0 += tiles;
        g = next;
        if (more && (more = next_seg(s + 2, next))) {  // into the buffer of the segment that is done
          if (!used_before(kBarQEmpty, s + 2)) { ok = false; break; }
          convert(s + 2, next);
        }
      }
    }
  } else {
    if (kR == 16 || kR == 32) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    if (kR == 64) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // ------------------------------------------------------------ softmax group H: the part's tiles j = H mod 2; thread = key
    const int H = warp >> 2, w4 = warp & 3, tid = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * w4) << 16, tS = tmem + lane_base + kColS + kN * H;
    float* nref = rows + kRowRef + H * kBlock;
    float* alpha = rows + kRowAlpha + H * kBlock;
    float* wmax = rows + kRowMax + 4 * H * kBlock;
    uint4* maskbits = reinterpret_cast<uint4*>(rows + kRowMask) + H * kBlock;
    int syncs = 0;
    auto group_arrive = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarGroup + H]);
    };
    auto group_wait = [&]() { return wait(&bars[kBarGroup + H], syncs++ & 1); };
    auto group_sync = [&]() {
      group_arrive();
      return group_wait();
    };
    int j0 = 0;  // the segment's first tile
    Seg g;
    for (int s = 0; j0 < cnt && next_seg(s, g); ++s) {
      const Span span = span_of<kWin>(A, g.L, g.T, g.rb);
      const int C = g.L - g.T, set = (s & 1) * kBlock;
      float m_used = -INFINITY;  // of row `tid`
      if (!used_before(kBarOFree, s)) { ok = false; break; }  // the rows' numbers of segment s - 2 have been read
      if (tid < kR) {
        const int rr = kBlock * g.rb + tid, i = rr % A.n;
        rowi[set + tid] = rr < A.R && i < g.T ? i : -1;
        if (kWin) rowend[set + tid] = behind(A, g.b, i, C);
      }
      uint64_t l[kR / 2];  // sums of this key's lane, rows in pairs
#pragma unroll
      for (int r = 0; r < kR / 2; ++r) l[r] = pk2(0.f, 0.f);
      if (!wait(&bars[kBarQFull + (s & 1)], (s >> 1) & 1) || !group_sync()) { ok = false; break; }
      const float* f = rowf + set;
      const uint32_t tO = tmem + lane_base + kColO + 2 * kN * (s & 1) + kN * H;
      const int tiles = g.t1 - g.t0, first = (j0 ^ H) & 1;  // the group's first tile of them
      for (int x = first; x < tiles; x += 2) {
        const int t = g.t0 + x, j = j0 + x;
        const int key0 = span.key0(t);
        const bool masked = kWin ? span.masked<kWin>(key0, A.sink) : key0 + 128 > C;
        if (!done(kBarQK, j)) { ok = false; break; }
        tc_fence_after();
        uint32_t see[(kR + 31) / 32];  // masked: rows that see this key
        if (masked) {
          // thread = row: the 128 keys that it sees, as bits; then thread = key: the rows that see it
          if (tid < kR) {
            const int i = rowi[set + tid], end = kWin ? rowend[set + tid] : 0;
            const uint32_t* mrow = A.mask && i >= 0 ? A.mask + g.b * A.mask_stride + (int64_t)i * A.words : nullptr;
            uint32_t bits[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int rel = key0 + 32 * c - C;  // drafted index of bit 0 (negative: context)
              uint32_t w = ~0u;
              if (rel > -32) {
                if (A.mask) {
                  const int w0 = rel >> 5;  // floor for negative rel
                  const uint32_t a = mrow && w0 >= 0 && w0 < A.words ? __ldg(mrow + w0) : 0u;
                  const uint32_t b = mrow && w0 + 1 < A.words ? __ldg(mrow + w0 + 1) : 0u;
                  w = __funnelshift_r(a, b, rel & 31) & low_mask32(g.T - rel);
                  if (rel < 0) w |= low_mask32(-rel);
                } else {
                  w = low_mask32(min(i + 1, g.T) - rel);
                }
              }
              if (kWin) w &= ~(low_mask32(end - (key0 + 32 * c)) & ~low_mask32(A.sink - (key0 + 32 * c)));
              bits[c] = w;
            }
            maskbits[tid] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
          }
          if (!group_sync()) { ok = false; break; }
          const uint32_t* word = reinterpret_cast<const uint32_t*>(maskbits) + w4;
#pragma unroll
          for (int x = 0; x < (kR + 31) / 32; ++x) {
            uint32_t bits = 0;
#pragma unroll 8
            for (int r = 0; r < (kR < 32 ? kR : 32); ++r) bits |= (word[4 * (32 * x + r)] >> lane & 1u) << r;
            see[x] = bits;
          }
        }
        // kR = 32 and 64: scores by halves (all of them and the sums in registers spill: 32 rows 116 us for 108 then).  The
        // second is read from TMEM again for its weights; of 64 rows the first is too (451 us, 475 where it is kept)
        constexpr int kC = kR >= 32 ? kR / 2 : kR;
        constexpr bool kKeep = kR < 64;
        float y[kC];
        auto load_scores = [&](int c0) {  // of rows c0 .., -inf where a row does not see the key
#pragma unroll
          for (int c = 0; c < kC; c += 16) {
            uint32_t* u = reinterpret_cast<uint32_t*>(y) + c;
            if constexpr (kC == 8) tmem_ld8(tS + c0 + c, *reinterpret_cast<uint32_t(*)[8]>(u));
            else tmem_ld16(tS + c0 + c, u);
          }
          tmem_ld_wait();
          if (masked)
#pragma unroll
            for (int r = 0; r < kC; ++r) y[r] = (see[c0 >> 5] >> ((c0 + r) & 31) & 1u) ? y[r] : -INFINITY;
        };
        // log2 of the weights; returns the largest
        auto scale_scores = [&](int c0) -> float {
          float top = -INFINITY;
#pragma unroll
          for (int r = 0; r < kC; r += 4) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(f + c0 + r);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(nref + c0 + r);
            up2(fma2(pk2(y[r], y[r + 1]), a.x, b.x), y[r], y[r + 1]);
            up2(fma2(pk2(y[r + 2], y[r + 3]), a.y, b.y), y[r + 2], y[r + 3]);
            top = max3f(max3f(y[r], y[r + 1], y[r + 2]), y[r + 3], top);
          }
          return top;
        };
        auto exponentials = [&]() {
#pragma unroll
          for (int r = 0; r < kC; ++r) y[r] = ex2(y[r]);
        };
        bool far = x == first;
        if (!far) {
          // Does one of the four warps' scores pass its reference too far?  The exponentials are under way meanwhile.
          float top = -INFINITY;
#pragma unroll
          for (int c = kR - kC; c >= 0; c -= kC) {
            load_scores(c);
            top = fmaxf(top, scale_scores(c));
          }
          const int at = syncs;
          if (__any_sync(0xFFFFFFFFu, top > kTop + kRaise) && lane == 0) misc[4 + 2 * H + (at & 1)] = at;
          group_arrive();
          if (kKeep) exponentials();  // (of rows 0 ..)
          if (!group_wait()) { ok = false; break; }
          far = misc[4 + 2 * H + (at & 1)] == (uint32_t)at;
        }
        if (far) {
          // the rows' maxima over the tile, new references, and what was summed comes to them
#pragma unroll
          for (int c = 0; c < kR; c += kC) {
            load_scores(c);
            float mine = 0.f;
#pragma unroll
            for (int r = 0; r < kC; ++r) {
              const float m = warp_max(y[r] * f[c + r]);
              if (lane == r) mine = m;
            }
            if (lane < kC) wmax[w4 * kBlock + c + lane] = mine;
          }
          if (!group_sync()) { ok = false; break; }
          if (tid < kR) {
            float m = m_used;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, wmax[w * kBlock + tid]);
            // A column without a row holds whatever shared memory held: with a reference of -inf for its scores it never
            // asks for a raise, or the others' weights would round to what ran before
            const bool row = rowi[set + tid] >= 0;
            alpha[tid] = m == m_used ? 1.f : ex2(m_used - m);
            nref[tid] = row ? fminf(kTop - m, 3e38f) : -INFINITY;  // (no key met yet: the first one is too far above)
            if (row) m_used = m;
          }
          if (!group_sync()) { ok = false; break; }
          if (x > first) {
#pragma unroll
            for (int r = 0; r < kR; r += 2) l[r / 2] = mul2(l[r / 2], pk2(alpha[r], alpha[r + 1]));
            if (!done(kBarPV, j - 2)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kR; c += 8) {
              uint32_t o[8];
              tmem_ld8(tO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha[c + k]);
              tmem_st8(tO + c, o);
            }
            tmem_st_wait();
          }
          if (kKeep) {
            if (kC < kR) load_scores(0);
            scale_scores(0);
            exponentials();
          }
        }
        auto release = [&]() {  // the scores are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[kBarSEmpty + H]);
        };
        if (kC == kR) release();
        if (!used_before(kBarPV, j)) { ok = false; break; }
        uint8_t* p = sm + Ly::kP + (kN == 64 ? H * Ly::kPTile : 0);
        constexpr int kSide = kN == 64 ? 0 : 4;  // chunks of 16 bytes to the second buffer in the same rows
#pragma unroll
        for (int c = 0; c < kR; c += kC) {
          if (!kKeep || c > 0) {
            load_scores(c);
            if (c + kC == kR) release();
            scale_scores(c);
            exponentials();
          }
#pragma unroll
          for (int r = 0; r < kC; r += 8) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              w[k] = pack_f16x2(y[r + 2 * k], y[r + 2 * k + 1]);
              uint64_t& sum = l[(c + r) / 2 + k];
              sum = add2(sum, pk2(y[r + 2 * k], y[r + 2 * k + 1]));
            }
            *reinterpret_cast<uint4*>(p + sw128_offset(tid, ((c + r) >> 3) + kSide * H)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[kBarPFull + H]);
      }
      if (!ok) break;

      // ---- the segment's end: row sums over lanes and warps, then O^T (thread = channel)
      if (lane == 0) mbar_arrive(&bars[kBarQEmpty + (s & 1)]);  // (behind the last barrier of the group: all have read f)
      float sums[kR];
#pragma unroll
      for (int r = 0; r < kR; r += 2) up2(l[r / 2], sums[r], sums[r + 1]);
      lane_sums<kR, 16>(sums, lane);
      float* own = rows + kRowSums + 8 * set + (4 * H + w4) * kBlock;
      if constexpr (kR == 64) *reinterpret_cast<float2*>(own + 2 * lane) = make_float2(sums[0], sums[1]);
      else if (lane % (32 / kR) == 0) own[lane / (32 / kR)] = sums[0];
      if (tid < kR) rows[kRowLast + 2 * set + H * kBlock + tid] = m_used;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[kBarSums + (s & 1)]);
      j0 += tiles;
    }
  }
  if (!ok) {
    misc[2] = 1;
    atomicCAS(A.err, 0, (int)kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (misc[2]) {
    // A role gave up: copies and products that nobody waited for end before the CTA's shared memory and TMEM go.
    if (warp == Ro::kIssueQK || warp == Ro::kIssuePV) {
      uint64_t* drained = &bars[kBarDrain + (warp == Ro::kIssueQK ? 0 : 1)];
      if (elect_one()) mma_commit(drained);
      mbar_wait_long(drained, 0, nullptr, MSA_WAIT_LIMIT_NS / 16);
    }
    __syncthreads();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

struct Ws4 {
  size_t cuts, ml, part, total;
};
Ws4 kv4_ws(const msa_shape& s) {
  const int64_t R = (int64_t)(s.Hq / s.Hkv) * s.n, rows = 2 * kCtas * (R < kBlock ? R : kBlock);
  Ws4 w;
  w.cuts = 16;  // behind their count
  w.ml = align256(w.cuts + kCtas * sizeof(Cut));
  w.part = align256(w.ml + (size_t)rows * 8);
  w.total = align256(w.part + (size_t)rows * s.d_h * 4);
  return w;
}

template <int D, int kR, bool kWin>
msa_status launch(const Kv4Args& a, bool join, cudaStream_t stream) {
  constexpr int kN = kR < 16 ? 16 : kR;
  auto kern = kv4_attn_kernel<D, kR, kWin>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay4<D, kN>::kAlloc) != cudaSuccess)
    return MSA_ERR_CUDA;
  kern<<<kCtas, Roles<kR>::kThreads, Lay4<D, kN>::kAlloc, stream>>>(a);
  note_launch();
  if (cudaGetLastError() != cudaSuccess) return MSA_ERR_CUDA;
  return join ? launch_join<D, kCtas, kBlock>(a.t, stream) : MSA_OK;
}

template <int D, bool kWin>
msa_status launch_rows(const Kv4Args& a, bool join, cudaStream_t stream) {
  if (a.t.R <= 8) return launch<D, 8, kWin>(a, join, stream);
  if (a.t.R <= 16) return launch<D, 16, kWin>(a, join, stream);
  if (a.t.R <= 32) return launch<D, 32, kWin>(a, join, stream);
  return launch<D, 64, kWin>(a, join, stream);
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attn_tree_kv4_workspace(const msa_shape* shape) {
  return check_tree_shape(shape) == MSA_OK ? kv4_ws(*shape).total : 0;
}

extern "C" msa_status msa_attn_tree_kv4(const msa_shape* shape, const void* q, const msa_kv4_pages* pages,
                                        const int32_t* page_table, int32_t max_pages, const int32_t* seq_len,
                                        const int32_t* tree_len, const uint32_t* tree_mask, int64_t mask_stride,
                                        const msa_tree_window* window, void* o, float* lse, void* ws, size_t ws_bytes,
                                        void* stream) {
  msa_status st = check_tree_shape(shape);
  if (st != MSA_OK) return st;
  st = check_kv4_pages(pages);
  if (st != MSA_OK) return st;
  if (max_pages < 1) return MSA_ERR_INVALID_ARG;
  if (!aligned(q, 16, true) || !aligned(o, 16, true) || !aligned(page_table, 4, true) || !aligned(seq_len, 4, true) ||
      !aligned(tree_len, 4, false) || !aligned(tree_mask, 4, false) || !aligned(lse, 4, false) || !aligned(ws, 16, true))
    return MSA_ERR_INVALID_ARG;
  if (q == o) return MSA_ERR_INVALID_ARG;
  const int32_t words = (shape->n + 31) / 32;
  if (tree_mask && mask_stride != 0 && mask_stride < (int64_t)shape->n * words) return MSA_ERR_INVALID_ARG;
  if (window && !window_ok(window, tree_mask)) return MSA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * pages->page_size >= ((int64_t)1 << 31) - 256) return MSA_ERR_UNSUPPORTED;
  const Ws4 w = kv4_ws(*shape);
  if (ws_bytes < w.total) return MSA_ERR_WORKSPACE_TOO_SMALL;
  Kv4Args a;
  memset(&a, 0, sizeof(a));
  TreeArgs& t = a.t;
  t.B = shape->B;
  t.Hq = shape->Hq;
  t.Hkv = shape->Hkv;
  t.n = shape->n;
  t.R = shape->Hq / shape->Hkv * shape->n;
  t.RB = (t.R + kBlock - 1) / kBlock;
  if ((int64_t)t.B * t.Hkv * t.RB >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  t.max_parts = kCtas;
  t.page_shift = __builtin_ctz((unsigned)pages->page_size);
  t.max_pages = max_pages;
  t.num_pages = pages->num_pages;
  t.words = words;
  t.table = page_table;
  t.seq_len = seq_len;
  t.tree_len = tree_len;
  t.mask = tree_mask;
  t.mask_stride = mask_stride;
  t.o = static_cast<__nv_bfloat16*>(o);
  t.lse = lse;
  uint8_t* base = static_cast<uint8_t*>(ws);
  t.count = reinterpret_cast<int32_t*>(base);
  t.cuts = reinterpret_cast<Cut*>(base + w.cuts);
  t.part_ml = reinterpret_cast<float2*>(base + w.ml);
  t.part = reinterpret_cast<float4*>(base + w.part);
  t.scale_log2 = effective_scale(*shape) * 1.4426950408889634f * kv4_scale(pages->k_scale);
  if (window) {
    t.sink = window->sink;
    t.window = window->window;
    t.depth = window->depth;
    t.step = chain_step(t, kBlock);
  }
  t.err = device_error_word();
  if (!t.err) return MSA_ERR_CUDA;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.data = static_cast<const uint8_t*>(pages->data);
  a.v_scale = kv4_scale(pages->v_scale);
  // a table of at most 128 keys holds no item of two tiles: none is cut
  const bool join = (int64_t)max_pages * pages->page_size > 128;
  cudaStream_t stm = (cudaStream_t)stream;
  if (shape->d_h == 128) return window ? launch_rows<128, true>(a, join, stm) : launch_rows<128, false>(a, join, stm);
  return window ? launch_rows<64, true>(a, join, stm) : launch_rows<64, false>(a, join, stm);
}
