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
// What bounds it: HBM, every value read once and written once per
// destination.  A lane holds both members of its pairs (two 16-byte chunks, a
// head in 8 lanes for d_h = 128), so the rotation needs no exchange and the
// norm three shuffles; the cosines of a token are computed once per CTA and
// serve all its heads.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "internal.h"
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

// A lane's 16 values of a head: chunks c0 and c1 of 8.  In the rotated columns
// chunk 0 holds the first and chunk 1 the second members of 8 pairs
// (half-split), or both hold whole pairs (interleaved).
//
// With scalar arithmetic the issue slots were 65 % taken at 5.2 TB/s, so it is in
// packed pairs; and a lane keeps the loads of its next two heads in flight (with one
// the 4 CTAs an SM's registers hold had too little on the way: 162 us).  32K tokens
// of 32 + 8 + 8 heads of 128 into layer and cache take 151 us, 6.2 TB/s (0.92 of the
// measured copy rate), 105K tokens 458 us (0.97), 64 tokens of a decode step 3.5 us.
template <int D, bool kVarlen>
__global__ void __launch_bounds__(kThreads, 4)
    norm_rope_kernel(const __grid_constant__ RopeArgs A, const __grid_constant__ Seqs<kVarlen> T) {
  constexpr int kLanes = D / 16;               // lanes of a head
  constexpr int kHeads = kThreads / kLanes;    // heads in flight per CTA
  // Shared tables hold what a lane reads as two float4, and those of the lanes of a head side by side (no two lanes
  // on one bank): value x of lane l at 4 (l + (x / 4) lanes) + x % 4.
  __shared__ __align__(16) float cosines[kMaxTokens][D / 2], sines[kMaxTokens][D / 2];
  __shared__ __align__(16) float weights[2][2][D / 2];  // [q or k][chunk]
  __shared__ Token toks[kMaxTokens];
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
    if (!is_v) {
      uint64_t a[4], b[4];
      unpack8(x0, a);
      unpack8(x1, b);
      if (A.norm) {
        uint64_t sum = pk2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < 4; ++x) sum = fma2(b[x], b[x], fma2(a[x], a[x], sum));
        float s0, s1;
        up2(sum, s0, s1);
        float ss = s0 + s1;
        const unsigned group = (kLanes == 8 ? 0xFFu : 0xFu) << ((tid & 31) / kLanes * kLanes);
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
    __nv_bfloat16* pages = is_v ? A.vp : A.kp;
    if (!is_q && pages && tk.slot >= 0) {
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
                     const int32_t* slots, int64_t tokens, cudaStream_t stream) {
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
  if (!k && !pages) return MSA_ERR_INVALID_ARG;          // the keys would go nowhere
  if (v_in ? !v && !pages : v || pages) return MSA_ERR_INVALID_ARG;  // values come and go together
  // rows move: not in place, nor two outputs in one
  const void* outs[5] = {q, k, v, pages ? pages->k : nullptr, pages ? pages->v : nullptr};
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
    const bool ok = s.d_h == 128 ? launch(norm_rope_kernel<128, false>, Seqs<false>())
                                 : launch(norm_rope_kernel<64, false>, Seqs<false>());
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
    const bool ok = s.d_h == 128 ? launch(norm_rope_kernel<128, true>, t) : launch(norm_rope_kernel<64, true>, t);
    if (!ok) return MSA_ERR_CUDA;
  }
  return MSA_OK;
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_qk_norm_rope(const msa_shape* shape, const msa_rope_cfg* cfg, const void* q_in,
                                       int64_t q_stride, const void* k_in, int64_t k_stride, const void* v_in,
                                       int64_t v_stride, const int32_t* positions, void* q, void* k, void* v,
                                       const msa_kv_pages* pages, const int32_t* slots, void* stream) {
  const msa_status st = check_shape(shape);
  if (st != MSA_OK) return st;
  return norm_rope(*shape, nullptr, 0, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v, pages,
                   slots, (int64_t)shape->B * shape->n, (cudaStream_t)stream);
}

extern "C" msa_status msa_qk_norm_rope_varlen(const msa_shape* shape, const int32_t* cu_seqlens, int32_t n_seqs,
                                              const msa_rope_cfg* cfg, const void* q_in, int64_t q_stride,
                                              const void* k_in, int64_t k_stride, const void* v_in, int64_t v_stride,
                                              const int32_t* positions, void* q, void* k, void* v,
                                              const msa_kv_pages* pages, const int32_t* slots, void* stream) {
  if (!shape || !cu_seqlens || n_seqs < 1 || cu_seqlens[0] != 0) return MSA_ERR_INVALID_ARG;
  msa_shape s = *shape;
  s.B = 1;
  s.n = 1;
  const msa_status st = check_shape(&s);
  if (st != MSA_OK) return st;
  for (int x = 0; x < n_seqs; ++x)
    if (cu_seqlens[x + 1] < cu_seqlens[x]) return MSA_ERR_INVALID_ARG;
  return norm_rope(s, cu_seqlens, n_seqs, cfg, q_in, q_stride, k_in, k_stride, v_in, v_stride, positions, q, k, v,
                   pages, slots, cu_seqlens[n_seqs], (cudaStream_t)stream);
}
