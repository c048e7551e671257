// Norms of queries and keys for each head with the position rotation, from the
// projection's token-major rows into the layouts the library reads: the
// head-major layer tensors and, in the same pass, the pages of a KV cache.
//
// Per head row x of d_h values: y = x / sqrt(mean(x^2) + eps) * w (when the
// norm is on), then the first rot_dim columns turn by position: the pair
// (a, b) = (i, i + rot/2), or (2i, 2i+1) when interleaved, becomes
// (a cos - b sin, b cos + a sin) with the angle position * f_i.  V is moved
// unchanged.  Everything is fp32 and rounded to bf16 once, at the store: the
// normed value is not rounded before the rotation.
//
// Angles.  An fp32 product position * f_i has an error of 0.06 rad at a
// position of a million.  The host turns f_i into F = f_i / (2 pi) in units of
// 2^-64 turns; position * F in 64-bit integers wraps exactly at whole turns,
// and its top 32 bits are the angle to 2^-31 turns, whatever the position.  It
// is rounded to fp32 half turns in [-1, 1) for the sine and cosine: to 2^-26
// turns at worst, and relative to the angle where that is near a whole turn.
//
// Into a 4-bit cache (kKv4) keys and values leave as the codes and scales of
// "4-bit pages" below, the layer's layout as without it.
//
// What bounds it: HBM, every value read once and written once per
// destination.  4-bit pages: issue, 188 us for the 32K tokens that take 151 into bf16
// pages (of which the second computation of the heads in question is 22; it
// is out of line: inlined, its registers spilled and cost 70 us), 135 for 23K packed ones; 64 tokens of a decode
// step 8.3 us one after another and 12.8 behind other kernels with the caches cold, most of it the sines' and the exact
// path's chains (without a head in question 4.7 and 10.7, with a block's scale in question, three steps of ten, 9.2 and
// 14.8).  A lane holds both members of its pairs (two 16-byte chunks, a
// head in 8 lanes for d_h = 128), so the rotation needs no exchange and the
// norm three shuffles; the cosines of a token are computed once per CTA and
// serve all its heads.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace msa {

msa_status check_shape(const msa_shape* s);
msa_status check_page_geometry(int32_t num_pages, int32_t page_size);

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;    // tokens of a CTA: 5 and 16 measured 1 % and 6 % slower on 32K tokens
constexpr int kPerSm = 8;        // CTAs per SM below which they take fewer tokens
constexpr int kMaxBatch = 1024;  // sequences of a launch

struct RopeArgs {
  const __nv_bfloat16 *q, *k, *v;     // token-major inputs
  int64_t q_stride, k_stride, v_stride;  // elements from one token to the next
  int32_t Hq, Hkv, has_v;
  int32_t tok0, tok1;  // tokens of this launch
  int32_t n;           // tokens of a sequence (uniform batch)
  int32_t per_cta;
  const int32_t* positions;
  const __nv_bfloat16 *q_w, *k_w;
  int32_t norm, rot, interleaved;
  float eps, rot_scale;
  __nv_bfloat16 *qo, *ko, *vo;  // layer layout (ko, vo may be null)
  __nv_bfloat16 *kp, *vp;       // pages (may be null)
  uint8_t* kv4;                 // or 4-bit pages
  float k_inv, v_inv;           // 1 / their scales (powers of two)
  const int32_t* slots;
  int32_t page_shift, num_pages;
  int* err;
  uint64_t turn[64];  // f_i in 2^-64 turns
};

// Varlen: the sequences of a launch and their first tokens.  (4 KB of parameters, which a uniform batch does not pay
// for: they cost its call 0.5 us on the host.)
template <bool kVarlen>
struct Seqs {
  int32_t count;
  int32_t cu[kMaxBatch + 1];
};
template <>
struct Seqs<false> {};

struct Token {
  int32_t seq0, n, i;  // first token and length of its sequence, index in it
  int32_t slot;        // cache slot, < 0: not stored
};
static_assert(sizeof(Token) == 16, "one load of shared memory");

// 8 bf16 values (16 bytes) as four pairs
__device__ __forceinline__ void unpack8(uint4 u, uint64_t (&f)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int x = 0; x < 4; ++x) f[x] = pk2(__uint_as_float(w[x] << 16), __uint_as_float(w[x] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    float a, b;
    up2(f[x], a, b);
    w[x] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 floats of shared memory as four pairs: floats 0 .. 3 at p, 4 .. 7 at q
__device__ __forceinline__ void load8(const float* p, const float* q, uint64_t (&f)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(q);
  f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

// ---------------------------------------------------------------- 4-bit pages
// A block of 16 channels is held as e2m1 codes and an e4m3 scale: scale = RN(max |x| / 6), code = RN(x / scale), both
// ties to even and of the exact x.  V is exact: a quotient x / scale of 8 by 4 significant bits is a border of two codes
// or at least 2^-8 of it away (a border times a scale has 7 bits), so rounding it to 2^-12 gives the borders back that
// the reciprocal's error moved.  K is rounded here in fp32 first, to kOff of its pair's size, so it is
// rounded from both ends of that range; where the two differ (in 0.6 % of the heads) it is computed again to 42
// bits.  What the cache holds is then what the definition gives in 64 bits, whatever order a kernel sums in.

// Numbers as unevaluated sums of two floats (Dekker 1971; the exact sum is Knuth's): products and sums are good to about
// 2^-45.  fp64 would do as well, but its instructions take 16 cycles of a whole SM each.
struct Two {
  float h, l;
};
__host__ __device__ constexpr Two two(double x) { return {(float)x, (float)(x - (double)(float)x)}; }
__device__ __forceinline__ Two fast_sum(float a, float b) {  // |a| >= |b| or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two operator+(Two x, Two y) {
  const Two s = sum(x.h, y.h);
  return fast_sum(s.h, __fadd_rn(s.l, __fadd_rn(x.l, y.l)));
}
__device__ __forceinline__ Two operator*(Two x, Two y) {
  const Two p = product(x.h, y.h);
  return fast_sum(p.h, __fmaf_rn(x.h, y.l, __fmaf_rn(x.l, y.h, p.l)));
}
__device__ __forceinline__ Two operator*(Two x, float y) {
  const Two p = product(x.h, y);
  return fast_sum(p.h, __fmaf_rn(x.l, y, p.l));
}
__device__ __forceinline__ Two operator-(Two x) { return {-x.h, -x.l}; }

// 1 / sqrt(x): a step of Newton's method from rsqrtf.
__device__ __forceinline__ Two inverse_root(Two x) {
  const float r = rsqrtf(x.h);
  const Two t = x * product(r, r);
  return fast_sum(r, 0.5f * r * __fsub_rn(__fsub_rn(1.f, t.h), t.l));
}

// Sine and cosine of `turns` 2^-64 turns: whole quarters, then Taylor's series up to pi / 4.
__device__ __forceinline__ void sine_cosine(int64_t turns, Two& s, Two& c) {
  const int64_t quarters = (int64_t)((uint64_t)turns + ((uint64_t)1 << 61)) >> 62;
  const int64_t rest = (int64_t)((uint64_t)turns - ((uint64_t)quarters << 62));
  const float h = (float)rest;
  const Two x = fast_sum(h * 0x1p-63f, (float)(rest - (int64_t)h) * 0x1p-63f) * two(3.141592653589793);
  const Two y = x * x;
  Two t = {__fmaf_rn(y.h, __fmaf_rn(y.h, 1.f / 6227020800.f, -1.f / 39916800.f), 1.f / 362880.f), 0.f};
  t = y * t + two(-1.0 / 5040);
  t = y * t + two(1.0 / 120);
  t = y * t + two(-1.0 / 6);
  const Two sn = x + x * (y * t);
  t = {__fmaf_rn(y.h, __fmaf_rn(y.h, 1.f / 479001600.f, -1.f / 3628800.f), 1.f / 40320.f), 0.f};
  t = y * t + two(-1.0 / 720);
  t = y * t + two(1.0 / 24);
  t = y * t + two(-0.5);
  const Two cs = y * t + two(1.0);
  const bool odd = quarters & 1;
  s = odd ? cs : sn;
  c = odd ? sn : cs;
  if (quarters & 2) s = -s;
  if ((quarters + 1) & 2) c = -c;
}

// Value `c` of the key head at `x` to about 2^-40; r: the norm's factor.
__device__ __noinline__ Two exact_key(const RopeArgs& A, const __nv_bfloat16* x, int c, int pos, Two r) {
  auto normed = [&](int i) {
    const float v = __bfloat162float(x[i]);
    return A.norm ? r * (A.k_w ? v * __bfloat162float(A.k_w[i]) : v) : Two{v, 0.f};  // (v w has 16 bits)
  };
  if (c >= A.rot) return normed(c);
  const int half = A.rot >> 1, p = A.interleaved ? c >> 1 : c % half;
  const bool second = A.interleaved ? c & 1 : c >= half;
  const Two own = normed(c), other = normed(A.interleaved ? c ^ 1 : second ? c - half : c + half);
  Two s, co;
  sine_cosine((int64_t)((uint64_t)(int64_t)pos * A.turn[p]), s, co);
  return (own * co + (second ? other : -other) * s) * A.rot_scale;
}

// |x| inv / d (inv a power of two), cut to fp32 with its last bit set where something was cut: rounds to fewer bits as
// the quotient itself does.
__device__ __forceinline__ float sticky(Two x, float inv, float d) {
  if (x.h < 0.f) x = -x;
  const float a = x.h * inv, q = __fdiv_rn(a, d), left = __fadd_rn(__fmaf_rn(-q, d, a), x.l * inv);
  if (left == 0.f || q == INFINITY) return q;
  return __uint_as_float((__float_as_uint(q) - (left < 0.f ? 1u : 0u)) | 1u);
}

// What fp32 may be off in a turned value, in sizes of its pair (half steps of 2^-24): 13 in the sum of squares, half of
// that in its root, 4 for rsqrtf, 2 for two products; sine and cosine 2.6 (one step, and the angle's rounding), two
// products and their sum 2, a factor 1: below 20.
constexpr float kOff = 1.1920928955078125e-06f;  // 20 x 2^-24
constexpr float kQuot = 4.76837158203125e-07f;  // 2^-21: how far a quotient by a reciprocal is off, relatively

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The scale of a block whose largest value is a, off by up to `off` (both in units of the tensor's scale).  A NaN among
// its values makes a one, and the scale: whoever reads the block finds it, as in the bf16 cache.
__device__ __forceinline__ uint32_t block_scale(float a, float off, bool& unsure) {
  unsure = false;
  if (!(a < INFINITY)) return a != a ? 0x7Fu : 0x7Eu;
  const float q = a * (1.f / 6.f);
  if (off > 0.f) {
    const float e = off * 0.25f + q * 0.5f * kQuot;
    unsure = e4m3_of(fmaxf(q - e, 0.f)) != e4m3_of(q + e);
    return e4m3_of(q);
  }
  // to 16 bits: exact where it is halfway between two scales (5 bits; a has 8, so else it is 2^-8 of it away at least)
  return e4m3_of(__uint_as_float((__float_as_uint(q) + 0x80u) & 0xFFFFFF00u));
}

// Codes of the 8 values v r; e > 0: they are off by up to e, and a code that may be another one has bits set in `unsure`;
// e = 0: they are exact.
__device__ __forceinline__ uint32_t round8(const uint64_t (&v)[4], float r, float e, uint32_t& unsure) {
  const uint64_t rr = pk2(r, r);
  float f[8];
  unsure = 0;
  if (e > 0.f) {
    const uint64_t ee = pk2(e, e), minus = pk2(-e, -e);
#pragma unroll
    for (int x = 0; x < 4; ++x) up2(fma2(v[x], rr, ee), f[2 * x], f[2 * x + 1]);
    const uint32_t c = e2m1x8_of(f);
#pragma unroll
    for (int x = 0; x < 4; ++x) up2(fma2(v[x], rr, minus), f[2 * x], f[2 * x + 1]);
    unsure = c ^ e2m1x8_of(f);
    return c;
  }
  const uint64_t big = pk2(0x1.8p11f, 0x1.8p11f), back = pk2(-0x1.8p11f, -0x1.8p11f);  // to 2^-12
#pragma unroll
  for (int x = 0; x < 4; ++x) up2(add2(fma2(v[x], rr, big), back), f[2 * x], f[2 * x + 1]);
  return e2m1x8_of(f);
}

// A key head of which a scale or a code may not be that of the exact values: computed again.  One lane's share, in local
// memory: a call, so that the registers it needs are not taken from the other heads' path (with the code in its place 32K
// tokens take 276 us, reloading what was spilled for it).
template <int D>
struct Again {
  const RopeArgs& A;
  float2* top;
  const __nv_bfloat16* src;  // the head
  unsigned group;
  int pos, c[2];
  float inv, off[2];
  uint64_t v[2][4];  // chunks, fp32
  uint32_t scale[2], codes[2], unsure[2];
  bool far[2];

  __device__ __noinline__ void round() {
    Two ss = {0.f, 0.f};
#pragma unroll 1
    for (int x = 0; x < 16; ++x) {
      const float y = __bfloat162float(src[c[x >> 3] + (x & 7)]);
      ss = ss + Two{y * y, 0.f};  // (squares of 8 bits are exact)
    }
#pragma unroll 1
    for (int o = D / 32; o; o >>= 1)
      ss = ss + Two{__shfl_xor_sync(group, ss.h, o), __shfl_xor_sync(group, ss.l, o)};
    const Two r = A.norm ? inverse_root(Two{ss.h * (1.f / D), ss.l * (1.f / D)} + Two{A.eps, 0.f}) : Two{1.f, 0.f};
    if (__any_sync(group, far[0] || far[1])) {
      // The largest value of each block in question, of those that may be it (quotients cut with a mark keep their order
      // and round as the exact ones), and the codes by the scale that it gives.
      float m[2];
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        m[k] = 0.f;
        if (!far[k]) continue;
        const float2 t0 = top[c[k] >> 3], t1 = top[(c[k] >> 3) ^ 1];
        const float least = fmaxf(t0.x, t1.x) - 2.f * fmaxf(t0.y, t1.y);
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
          float y, z;
          up2(v[k][x >> 1], y, z);
          if (fabsf(x & 1 ? z : y) * inv >= least) m[k] = fmaxf(m[k], sticky(exact_key(A, src, c[k] + x, pos, r), inv, 6.f));
        }
      }
      __syncwarp(group);
      top[c[0] >> 3].x = m[0];
      top[c[1] >> 3].x = m[1];
      __syncwarp(group);
#pragma unroll 1
      for (int k = 0; k < 2; ++k)
        if (far[k]) {
          scale[k] = e4m3_of(fmaxf(top[c[k] >> 3].x, top[(c[k] >> 3) ^ 1].x));
          const float s = e4m3_value(scale[k]), q = s > 0.f ? __fdividef(inv, s) : 0.f;
          codes[k] = round8(v[k], q, off[k] * q > 0.f ? fmaf(off[k], q, 7.f * kQuot) : 0.f, unsure[k]);
        }
    }
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const float s = e4m3_value(scale[k]);
#pragma unroll 1
      for (int x = 0; x < 8; ++x) {
        if (!(unsure[k] >> (4 * x) & 0xFu)) continue;
        float z0, z1;
        up2(v[k][x >> 1], z0, z1);
        if (!(fabsf(x & 1 ? z1 : z0) < INFINITY)) {  // (its neighbours' error passes fp32's range)
          codes[k] = (codes[k] & ~(0xFu << (4 * x))) | (((x & 1 ? z1 : z0) < 0.f ? 0xFu : 7u) << (4 * x));
          continue;
        }
        const Two y = exact_key(A, src, c[k] + x, pos, r);
        const uint32_t code = (e2m1x2_of(s > 0.f ? sticky(y, inv, s) : 0.f, 0.f) & 7u) | (y.h < 0.f ? 8u : 0u);
        codes[k] = (codes[k] & ~(0xFu << (4 * x))) | code << (4 * x);
      }
    }
    __syncwarp(group);
  }
};

// A lane's 16 values of a head: chunks c0 and c1 of 8.  In the rotated columns
// chunk 0 holds the first and chunk 1 the second members of 8 pairs
// (half-split), or both hold whole pairs (interleaved).
//
// With scalar arithmetic the issue slots were 65 % taken at 5.2 TB/s, so it is in
// packed pairs; and a lane keeps the loads of its next two heads in flight (with one
// the 4 CTAs an SM's registers hold had too little on the way: 162 us).  32K tokens
// of 32 + 8 + 8 heads of 128 into layer and cache take 151 us, 6.2 TB/s (0.92 of the
// measured copy rate), 105K tokens 458 us (0.97), 64 tokens of a decode step 3.5 us.
template <int D, bool kVarlen, bool kKv4>
__global__ void __launch_bounds__(kThreads, 4)
    norm_rope_kernel(const __grid_constant__ RopeArgs A, const __grid_constant__ Seqs<kVarlen> T) {
  constexpr int kLanes = D / 16;               // lanes of a head
  constexpr int kHeads = kThreads / kLanes;    // heads in flight per CTA
  // Shared tables hold what a lane reads as two float4, and those of the lanes of a head side by side (no two lanes
  // on one bank): value x of lane l at 4 (l + (x / 4) lanes) + x % 4.
  __shared__ __align__(16) float cosines[kMaxTokens][D / 2], sines[kMaxTokens][D / 2];
  __shared__ __align__(16) float weights[2][2][D / 2];  // [q or k][chunk]
  __shared__ __align__(16) Token toks[kMaxTokens];
  __shared__ int32_t places[kKv4 ? kMaxTokens : 1];  // kKv4: their positions
  // kKv4: the largest values of a head's chunks of 8, and how far they may be off
  __shared__ float2 tops[kKv4 ? kHeads : 1][kKv4 ? D / 8 : 1];
  const int tid = threadIdx.x;
  const int H = A.Hq + A.Hkv * (1 + A.has_v);
  const int first = A.tok0 + blockIdx.x * A.per_cta;
  const int cnt = min(A.per_cta, A.tok1 - first);
  const int half = A.rot >> 1;
  const int l = tid % kLanes;
  // this lane's two chunks
  const bool rotated = 16 * l < A.rot;
  const int c0 = rotated ? 8 * l : 16 * l, c1 = rotated ? half + 8 * l : 16 * l + 8;
  const int rl = A.rot >> 4;  // lanes of a head that rotate, 8 pairs each
  auto at = [&](int lane, int x, int lanes) { return 4 * (lane + (x >> 2) * lanes) + (x & 3); };
  // position of pair p: value x of the lane whose chunks hold it (interleaved: 4 pairs in each chunk)
  auto pair_at = [&](int p) {
    if (!A.interleaved) return at(p >> 3, p & 7, rl);
    const int second = p >= (half >> 1), q = second ? p - (half >> 1) : p;
    return at(q >> 2, (q & 3) + 4 * second, rl);
  };

  auto load = [&](int t, int h, uint4& x0, uint4& x1) {
    const __nv_bfloat16* src;
    if (h < A.Hq) src = A.q + (first + t) * A.q_stride + h * D;
    else if (h < A.Hq + A.Hkv) src = A.k + (first + t) * A.k_stride + (h - A.Hq) * D;
    else src = A.v + (first + t) * A.v_stride + (h - A.Hq - A.Hkv) * D;
    x0 = __ldcs(reinterpret_cast<const uint4*>(src + c0));
    x1 = __ldcs(reinterpret_cast<const uint4*>(src + c1));
  };
  int t = 0, h = tid / kLanes;  // token and head of this lane
  auto next = [&](int& t, int& h) {
    h += kHeads;
    while (h >= H) {
      h -= H;
      ++t;
    }
  };
  while (h >= H) {
    h -= H;
    ++t;
  }
  uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
  if (t < cnt) load(t, h, x0, x1);  // in flight while the angles are computed
  uint4 y0 = make_uint4(0, 0, 0, 0), y1 = y0;  // and its next one
  int nt = t, nh = h;
  next(nt, nh);
  if (nt < cnt) load(nt, nh, y0, y1);

  if (tid < cnt) {
    const int tk = first + tid;
    Token k;
    if constexpr (kVarlen) {
      const int s = seq_search(T.count, [&](int x) { return T.cu[x]; }, tk);
      k.seq0 = T.cu[s];
      k.n = T.cu[s + 1] - T.cu[s];
    } else {
      k.seq0 = tk / A.n * A.n;
      k.n = A.n;
    }
    k.i = tk - k.seq0;
    if constexpr (kKv4) places[tid] = A.positions ? A.positions[tk] : k.i;
    k.slot = -1;
    if (A.slots) {
      k.slot = A.slots[tk];
      if (k.slot >= 0 && (k.slot >> A.page_shift) >= A.num_pages) {
        atomicCAS(A.err, 0, (int)kErrIndex);
        k.slot = -1;
      }
    }
    toks[tid] = k;
  }
  if (A.norm && tid < 2 * kLanes) {  // this lane's weights of a query (tid < kLanes) or key head
    const __nv_bfloat16* w = tid < kLanes ? A.q_w : A.k_w;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      weights[tid / kLanes][0][at(l, x, kLanes)] = w ? __bfloat162float(w[c0 + x]) : 1.f;
      weights[tid / kLanes][1][at(l, x, kLanes)] = w ? __bfloat162float(w[c1 + x]) : 1.f;
    }
  }
  if (half)
    for (int x = tid; x < cnt * half; x += kThreads) {
      const int t = x / half, p = x - t * half, tk = first + t;
      int pos;
      if (A.positions) pos = A.positions[tk];
      else if constexpr (kVarlen) pos = tk - T.cu[seq_search(T.count, [&](int y) { return T.cu[y]; }, tk)];
      else pos = tk % A.n;
      const uint64_t turns = (uint64_t)(int64_t)pos * A.turn[p];
      float s, c;
      sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
      cosines[t][pair_at(p)] = c * A.rot_scale;
      sines[t][pair_at(p)] = s * A.rot_scale;
    }
  __syncthreads();

  while (t < cnt) {
    int mt = nt, mh = nh;
    next(mt, mh);
    uint4 z0 = make_uint4(0, 0, 0, 0), z1 = z0;
    if (mt < cnt) load(mt, mh, z0, z1);
    const Token tk = toks[t];
    const bool is_v = h >= A.Hq + A.Hkv, is_q = h < A.Hq;
    const unsigned group = (kLanes == 8 ? 0xFFu : 0xFu) << ((tid & 31) / kLanes * kLanes);  // lanes of this head
    uint64_t a[4], b[4];  // this lane's chunks
    float size[2] = {0.f, 0.f};  // kKv4, K: the largest finite |first| + |second| of a pair that has a value in the chunk
    if (kKv4 || !is_v) {
      unpack8(x0, a);
      unpack8(x1, b);
    }
    if (!is_v) {
      if (A.norm) {
        uint64_t sum = pk2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 4; ++x) sum = fma2(b[x], b[x], fma2(a[x], a[x], sum));
        float s0, s1;
        up2(sum, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
        const float r = rsqrtf(ss * (1.f / D) + A.eps);
        const uint64_t rr = pk2(r, r);
        uint64_t w[4];
        const float* wa = &weights[is_q ? 0 : 1][0][4 * l];
        load8(wa, wa + 4 * kLanes, w);
#pragma unroll
        for (int x = 0; x < 4; ++x) a[x] = mul2(mul2(a[x], rr), w[x]);
        load8(wa + D / 2, wa + D / 2 + 4 * kLanes, w);
#pragma unroll
        for (int x = 0; x < 4; ++x) b[x] = mul2(mul2(b[x], rr), w[x]);
      }
      if (kKv4 && !is_q) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float a0, a1, b0, b1;
          up2(a[x], a0, a1);
          up2(b[x], b0, b1);
          auto pair = [](float p, float q) {  // an infinite one: NaN, which the maximum leaves out
            const float t = fabsf(p) + fabsf(q);
            return fmaf(t, 0.f, t);
          };
          if (A.interleaved) {
            size[0] = fmaxf(size[0], pair(a0, a1));
            size[1] = fmaxf(size[1], pair(b0, b1));
          } else {
            size[0] = size[1] = max3f(size[0], pair(a0, b0), pair(a1, b1));
          }
        }
      }
      if (rotated) {
        uint64_t c[4], s[4];
        load8(&cosines[t][4 * l], &cosines[t][4 * (l + rl)], c);
        load8(&sines[t][4 * l], &sines[t][4 * (l + rl)], s);
        if (A.interleaved) {
          auto turn = [&](uint64_t v, float c, float s) {  // (p, q) -> (p c - q s, q c + p s)
            float p, q;
            up2(v, p, q);
            return fma2(v, pk2(c, c), mul2(pk2(-q, p), pk2(s, s)));
          };
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float c0, c1, s0, s1;
            up2(c[x], c0, c1);
            up2(s[x], s0, s1);
            a[2 * x] = turn(a[2 * x], c0, s0);
            a[2 * x + 1] = turn(a[2 * x + 1], c1, s1);
            up2(c[2 + x], c0, c1);
            up2(s[2 + x], s0, s1);
            b[2 * x] = turn(b[2 * x], c0, s0);
            b[2 * x + 1] = turn(b[2 * x + 1], c1, s1);
          }
        } else {
          const uint64_t minus = pk2(-1.f, -1.f);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint64_t p = a[x];
            a[x] = fma2(p, c[x], mul2(mul2(b[x], s[x]), minus));
            b[x] = fma2(b[x], c[x], mul2(p, s[x]));
          }
        }
      }
      x0 = pack8(a);
      x1 = pack8(b);
    }
    const int kh = is_q ? h : is_v ? h - A.Hq - A.Hkv : h - A.Hq;
    const int64_t heads = is_q ? A.Hq : A.Hkv;
    __nv_bfloat16* out = is_q ? A.qo : is_v ? A.vo : A.ko;
    if (out) {
      __nv_bfloat16* dst = out + (heads * tk.seq0 + (int64_t)kh * tk.n + tk.i) * D;
      __stcs(reinterpret_cast<uint4*>(dst + c0), x0);
      __stcs(reinterpret_cast<uint4*>(dst + c1), x1);
    }
    if (kKv4 && !is_q && tk.slot >= 0) {
      const float inv = is_v ? A.v_inv : A.k_inv, rs = fmaxf(1.f, fabsf(A.rot_scale));
      const bool exact = is_v || (!A.norm && !rotated);  // neither normed nor turned
      float2* top = tops[tid / kLanes];
      // (kOff of the largest pair; a value that is not turned: of more than its own size)
      const float off0 = exact ? 0.f : size[0] * rs * kOff, off1 = exact ? 0.f : size[1] * rs * kOff;
      auto largest = [&](const uint64_t (&v)[4]) {
        float m = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float y, z;
          up2(v[x], y, z);
          m = max_or_nan(m, max_or_nan(fabsf(y), fabsf(z)));
        }
        return m * inv;
      };
      top[c0 >> 3] = make_float2(largest(a), off0 * inv);
      top[c1 >> 3] = make_float2(largest(b), off1 * inv);
      __syncwarp(group);
      uint32_t scale[2], codes[2], unsure[2];
      bool far[2];  // the scale may be another one
      auto round_chunk = [&](const uint64_t (&v)[4], int second, int c, float off) {
        const float2 t0 = top[c >> 3], t1 = top[(c >> 3) ^ 1];  // of the block's two chunks
        scale[second] = block_scale(max_or_nan(t0.x, t1.x), fmaxf(t0.y, t1.y), far[second]);
        const float s = e4m3_value(scale[second]), r = s > 0.f ? __fdividef(inv, s) : 0.f;
        codes[second] = round8(v, r, off * r > 0.f ? fmaf(off, r, 7.f * kQuot) : 0.f, unsure[second]);  // (quotients up to 6.4)
      };
      round_chunk(a, 0, c0, off0);
      round_chunk(b, 1, c1, off1);
      const bool again = far[0] || far[1];
      if (__any_sync(group, again || (unsure[0] | unsure[1]) != 0)) {  // K only
        Again<D> g = {A, top, A.k + (first + t) * A.k_stride + kh * D, group, places[t], {c0, c1}, inv, {off0, off1}};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int x = 0; x < 4; ++x) g.v[k][x] = k ? b[x] : a[x];
          g.scale[k] = scale[k], g.codes[k] = codes[k], g.unsure[k] = unsure[k], g.far[k] = far[k];
        }
        g.round();
#pragma unroll
        for (int k = 0; k < 2; ++k) scale[k] = g.scale[k], codes[k] = g.codes[k];
      }
      const int row = tk.slot & ((1 << A.page_shift) - 1);
      const int64_t size4 = (int64_t)kv4_unit<D>() << A.page_shift;
      uint8_t* unit = A.kv4 + (((int64_t)(tk.slot >> A.page_shift) * A.Hkv + kh) * 2 + (is_v ? 1 : 0)) * size4;
      auto put = [&](int c, int k) {
        *reinterpret_cast<uint32_t*>(unit + ((((c >> 5) << A.page_shift) + row) << 4) + (c & 31) / 2) = codes[k];
        if (!(c & 8)) unit[((D / 2) << A.page_shift) + row * (D / 16) + (c >> 4)] = (uint8_t)scale[k];
      };
      put(c0, 0);
      put(c1, 1);
      __syncwarp(group);  // tops is the next head's
    }
    __nv_bfloat16* pages = is_v ? A.vp : A.kp;
    if (!kKv4 && !is_q && pages && tk.slot >= 0) {
      const int64_t page = tk.slot >> A.page_shift;
      const int off = tk.slot & ((1 << A.page_shift) - 1);
      __nv_bfloat16* dst = pages + (((page * A.Hkv + kh) << A.page_shift) + off) * D;
      __stcs(reinterpret_cast<uint4*>(dst + c0), x0);
      __stcs(reinterpret_cast<uint4*>(dst + c1), x1);
    }
    t = nt;
    h = nh;
    x0 = y0;
    x1 = y1;
    nt = mt;
    nh = mh;
    y0 = z0;
    y1 = z1;
  }
}

bool aligned(const void* p, size_t a, bool required) {
  if (!p) return !required;
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// The fraction of x >= 0 in units of 2^-64 (exact: a double less its whole part is one, and has no more than 64 bits
// above 2^-64).
uint64_t fraction64(double x) { return (uint64_t)((x - floor(x)) * 0x1p64); }

// f in units of 2^-64 turns: the fraction of f / (2 pi) (whole turns change nothing).  1 / (2 pi) in two doubles and the
// product's rounding error by fma: off by two units at most as long as |f| < 2^30.
uint64_t turns64(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double a = fabs(f), p = a * kHi, e = fma(a, kHi, -p) + a * kLo;
  const uint64_t t = fraction64(p) + (e < 0.0 ? 0 - fraction64(-e) : fraction64(e));
  return f < 0.0 ? 0 - t : t;
}

msa_status norm_rope(const msa_shape& s, const int32_t* cu, int32_t n_seqs, const msa_rope_cfg* cfg, const void* q_in,
                     int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in, int64_t v_stride,
                     const int32_t* positions, void* q, void* k, void* v, const msa_kv_pages* pages,
                     const msa_kv4_pages* kv4, const int32_t* slots, int64_t tokens, cudaStream_t stream) {
  if (!cfg) return MSA_ERR_INVALID_ARG;
  if (cfg->rot_dim < 0 || cfg->rot_dim > s.d_h || !(cfg->eps >= 0.f) || isinf(cfg->eps)) return MSA_ERR_INVALID_ARG;
  if (cfg->norm != 0 && cfg->norm != 1) return MSA_ERR_INVALID_ARG;
  if (cfg->rot_dim % 16) return MSA_ERR_UNSUPPORTED;
  const double theta = cfg->theta > 0.0 ? cfg->theta : 10000.0;
  if (!(cfg->theta == cfg->theta) || isinf(theta) || !isfinite(cfg->rot_scale)) return MSA_ERR_INVALID_ARG;
  if (tokens == 0) return MSA_OK;  // empty tensors need no address
  if (!aligned(q_in, 16, true) || !aligned(k_in, 16, true) || !aligned(v_in, 16, false) || !aligned(q, 16, true) ||
      !aligned(k, 16, false) || !aligned(v, 16, false) || !aligned(positions, 4, false) ||
      !aligned(slots, 4, false) || !aligned(cfg->q_weight, 16, false) || !aligned(cfg->k_weight, 16, false))
    return MSA_ERR_INVALID_ARG;
  if (q_stride < (int64_t)s.Hq * s.d_h || k_stride < (int64_t)s.Hkv * s.d_h ||
      (v_in && v_stride < (int64_t)s.Hkv * s.d_h))
    return MSA_ERR_INVALID_ARG;
  if (q_stride % 8 || k_stride % 8 || (v_in && v_stride % 8)) return MSA_ERR_INVALID_ARG;
  if (!k && !pages && !kv4) return MSA_ERR_INVALID_ARG;  // the keys would go nowhere
  if (v_in ? !v && !pages && !kv4 : v || pages || kv4) return MSA_ERR_INVALID_ARG;  // values come and go together
  // rows move: not in place, nor two outputs in one
  const void* outs[5] = {q, k, v, pages ? pages->k : kv4 ? kv4->data : nullptr, pages ? pages->v : nullptr};
  for (int x = 0; x < 5; ++x) {
    if (!outs[x]) continue;
    if (outs[x] == q_in || outs[x] == k_in || outs[x] == v_in) return MSA_ERR_INVALID_ARG;
    for (int y = 0; y < x; ++y)
      if (outs[x] == outs[y]) return MSA_ERR_INVALID_ARG;
  }
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  if (pages) {
    const msa_status geo = check_page_geometry(pages->num_pages, pages->page_size);
    if (geo != MSA_OK) return geo;
    if (!slots || !aligned(pages->k, 16, true) || !aligned(pages->v, 16, true)) return MSA_ERR_INVALID_ARG;
    a.kp = static_cast<__nv_bfloat16*>(pages->k);
    a.vp = static_cast<__nv_bfloat16*>(pages->v);
    a.slots = slots;
    a.page_shift = __builtin_ctz((unsigned)pages->page_size);
    a.num_pages = pages->num_pages;
  } else if (kv4) {
    const msa_status ok = check_kv4_pages(kv4);
    if (ok != MSA_OK) return ok;
    if (!slots) return MSA_ERR_INVALID_ARG;
    a.kv4 = static_cast<uint8_t*>(kv4->data);
    a.k_inv = 1.f / kv4_scale(kv4->k_scale);
    a.v_inv = 1.f / kv4_scale(kv4->v_scale);
    a.slots = slots;
    a.page_shift = __builtin_ctz((unsigned)kv4->page_size);
    a.num_pages = kv4->num_pages;
  } else if (slots) {
    return MSA_ERR_INVALID_ARG;
  }
  if (tokens >= ((int64_t)1 << 31) - kMaxTokens) return MSA_ERR_UNSUPPORTED;
  for (int i = 0; i < cfg->rot_dim / 2; ++i) {
    const double f = cfg->inv_freq ? cfg->inv_freq[i] : pow(theta, -2.0 * i / cfg->rot_dim);
    if (!isfinite(f)) return MSA_ERR_INVALID_ARG;
    a.turn[i] = turns64(f);
  }
  a.q = static_cast<const __nv_bfloat16*>(q_in);
  a.k = static_cast<const __nv_bfloat16*>(k_in);
  a.v = static_cast<const __nv_bfloat16*>(v_in);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.Hq = s.Hq;
  a.Hkv = s.Hkv;
  a.has_v = v_in != nullptr;
  a.n = s.n;
  a.positions = positions;
  a.q_w = static_cast<const __nv_bfloat16*>(cfg->q_weight);
  a.k_w = static_cast<const __nv_bfloat16*>(cfg->k_weight);
  a.norm = cfg->norm;
  a.rot = cfg->rot_dim;
  a.interleaved = cfg->interleaved;
  a.eps = cfg->eps;
  a.rot_scale = cfg->rot_scale == 0.f ? 1.f : cfg->rot_scale;
  a.qo = static_cast<__nv_bfloat16*>(q);
  a.ko = static_cast<__nv_bfloat16*>(k);
  a.vo = static_cast<__nv_bfloat16*>(v);
  a.err = device_error_word();
  if (!a.err) return MSA_ERR_CUDA;
  // few tokens per CTA while there are few (latency; but heads for every lane), more when they fill the GPU several
  // times over
  const int64_t heads = s.Hq + s.Hkv * (v_in ? 2 : 1), lanes = kThreads / (s.d_h / 16);
  int64_t per = tokens / (152 * kPerSm);
  if (per < lanes / heads) per = lanes / heads;
  a.per_cta = (int)(per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per);
  auto launch = [&](auto kernel, const auto& seqs) {
    const unsigned grid = (unsigned)ceil_div((int64_t)a.tok1 - a.tok0, a.per_cta);
    kernel<<<grid, kThreads, 0, stream>>>(a, seqs);
    note_launch();
    return cudaGetLastError() == cudaSuccess;
  };
  if (!cu) {
    a.tok1 = (int32_t)tokens;
    const bool ok = kv4 ? (s.d_h == 128 ? launch(norm_rope_kernel<128, false, true>, Seqs<false>())
                                        : launch(norm_rope_kernel<64, false, true>, Seqs<false>()))
                        : (s.d_h == 128 ? launch(norm_rope_kernel<128, false, false>, Seqs<false>())
                                        : launch(norm_rope_kernel<64, false, false>, Seqs<false>()));
    return ok ? MSA_OK : MSA_ERR_CUDA;
  }
  Seqs<true> t;
  memset(&t, 0, sizeof(t));
  for (int s0 = 0; s0 < n_seqs; s0 += kMaxBatch) {
    t.count = n_seqs - s0 < kMaxBatch ? n_seqs - s0 : kMaxBatch;
    for (int x = 0; x <= t.count; ++x) t.cu[x] = cu[s0 + x];
    a.tok0 = t.cu[0];
    a.tok1 = t.cu[t.count];
    if (a.tok1 <= a.tok0) continue;
    const bool ok = kv4 ? (s.d_h == 128 ? launch(norm_rope_kernel<128, true, true>, t)
                                        : launch(norm_rope_kernel<64, true, true>, t))
                        : (s.d_h == 128 ? launch(norm_rope_kernel<128, true, false>, t)
                                        : launch(norm_rope_kernel<64, true, false>, t));
    if (!ok) return MSA_ERR_CUDA;
  }
  return MSA_OK;
}

}  // namespace

}  // namespace msa

using namespace msa;

namespace {

msa_status uniform(const msa_shape* shape, const msa_rope_cfg* cfg, const void* q_in, int64_t q_stride,
                   const void* k_in, int64_t k_stride, const void* v_in, int64_t v_stride, const int32_t* positions,
                   void* q, void* k, void* v, const msa_kv_pages* pages, const msa_kv4_pages* kv4,
                   const int32_t* slots, void* stream) {
  const msa_status st = check_shape(shape);
  if (st != MSA_OK) return st;
  return norm_rope(*shape, nullptr, 0, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v, pages,
                   kv4, slots, (int64_t)shape->B * shape->n, (cudaStream_t)stream);
}

msa_status varlen(const msa_shape* shape, const int32_t* cu_seqlens, int32_t n_seqs, const msa_rope_cfg* cfg,
                  const void* q_in, int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in,
                  int64_t v_stride, const int32_t* positions, void* q, void* k, void* v, const msa_kv_pages* pages,
                  const msa_kv4_pages* kv4, const int32_t* slots, void* stream) {
  if (!shape || !cu_seqlens || n_seqs < 1 || cu_seqlens[0] != 0) return MSA_ERR_INVALID_ARG;
  msa_shape s = *shape;
  s.B = 1;
  s.n = 1;
  const msa_status st = check_shape(&s);
  if (st != MSA_OK) return st;
  for (int x = 0; x < n_seqs; ++x)
    if (cu_seqlens[x + 1] < cu_seqlens[x]) return MSA_ERR_INVALID_ARG;
  return norm_rope(s, cu_seqlens, n_seqs, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v,
                   pages, kv4, slots, cu_seqlens[n_seqs], (cudaStream_t)stream);
}

}  // namespace

extern "C" msa_status msa_qk_norm_rope(const msa_shape* shape, const msa_rope_cfg* cfg, const void* q_in,
                                       int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in,
                                       int64_t v_stride, const int32_t* positions, void* q, void* k, void* v,
                                       const msa_kv_pages* pages, const int32_t* slots, void* stream) {
  return uniform(shape, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v, pages, nullptr, slots,
                 stream);
}

extern "C" msa_status msa_qk_norm_rope_varlen(const msa_shape* shape, const int32_t* cu_seqlens, int32_t n_seqs,
                                              const msa_rope_cfg* cfg, const void* q_in, int64_t q_stride,
                                              const void* k_in, int64_t k_stride, const void* v_in, int64_t v_stride,
                                              const int32_t* positions, void* q, void* k, void* v,
                                              const msa_kv_pages* pages, const int32_t* slots, void* stream) {
  return varlen(shape, cu_seqlens, n_seqs, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v,
                pages, nullptr, slots, stream);
}

extern "C" msa_status msa_qk_norm_rope_kv4(const msa_shape* shape, const msa_rope_cfg* cfg, const void* q_in,
                                           int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in,
                                           int64_t v_stride, const int32_t* positions, void* q, void* k, void* v,
                                           const msa_kv4_pages* pages, const int32_t* slots, void* stream) {
  if (!pages || !v_in) return MSA_ERR_INVALID_ARG;
  return uniform(shape, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v, nullptr, pages, slots,
                 stream);
}

extern "C" msa_status msa_qk_norm_rope_varlen_kv4(const msa_shape* shape, const int32_t* cu_seqlens, int32_t n_seqs,
                                                  const msa_rope_cfg* cfg, const void* q_in, int64_t q_stride,
                                                  const void* k_in, int64_t k_stride, const void* v_in,
                                                  int64_t v_stride, const int32_t* positions, void* q, void* k,
                                                  void* v, const msa_kv4_pages* pages, const int32_t* slots,
                                                  void* stream) {
  if (!pages || !v_in) return MSA_ERR_INVALID_ARG;
  return varlen(shape, cu_seqlens, n_seqs, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v,
                nullptr, pages, slots, stream);
}
