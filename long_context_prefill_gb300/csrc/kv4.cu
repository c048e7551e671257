// The 4-bit cache: checks of its pages and reading cached tokens back into the
// layer's layout (the prefix of a prompt that continues it).
//
// What bounds the reading: HBM, 9/16 byte in and 2 bytes out a value.  A warp
// takes 16 neighbouring tokens of a head, which lie in one page: one table
// entry, and its codes are runs of 256 bytes.  A lane makes 8 channels of a
// token at a time, so that a token's row leaves in one store of a half warp.
// 128K tokens of 8 heads of 128 105 us, 0.96 of the copy rate; 37 ragged prefixes of up to 9K
// tokens in pages of 16, heads of 64, 48 us, 0.84.
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

bool power_of_two(float s) {
  int e;
  return s == 0.f || (s >= 0x1p-40f && s <= 0x1p40f && frexpf(s, &e) == 0.5f);
}

}  // namespace

msa_status check_kv4_pages(const msa_kv4_pages* p) {
  if (!p) return MSA_ERR_INVALID_ARG;
  const msa_status st = check_page_geometry(p->num_pages, p->page_size);
  if (st != MSA_OK) return st;
  if (!p->data || reinterpret_cast<uintptr_t>(p->data) % 16) return MSA_ERR_INVALID_ARG;
  return power_of_two(p->k_scale) && power_of_two(p->v_scale) ? MSA_OK : MSA_ERR_INVALID_ARG;
}

namespace {

constexpr int kThreads = 256;
constexpr int kRun = 16;  // tokens of a warp

struct GatherArgs {
  const uint8_t* data;
  const int32_t *table, *seq_len;
  __nv_bfloat16 *k, *v;
  int32_t B, Hkv, n, max_pages, num_pages, page_shift, runs;
  float k_scale, v_scale;
  int* err;
};

__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h, float scale) {  // exact: 6 bits times a power of two
  float a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(a), "=f"(b) : "r"(h));
  return pack_bf16x2(a * scale, b * scale);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const GatherArgs A) {
  constexpr int kLanes = D / 8, kTokens = 32 / kLanes;  // lanes of a token, tokens of a warp at a time
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t bh = w / A.runs;
  const int x0 = (int)(w - bh * A.runs) * kRun;
  if (bh >= (int64_t)A.B * A.Hkv) return;
  const int b = (int)(bh / A.Hkv), h = (int)(bh - (int64_t)b * A.Hkv);
  int L = A.seq_len[b];
  if (L < 0 || L > ((int64_t)A.max_pages << A.page_shift)) {
    if (lane == 0 && x0 == 0) atomicCAS(A.err, 0, (int)kErrIndex);
    return;
  }
  L = min(L, A.n);
  if (x0 >= L) return;
  const int page = A.table[(int64_t)b * A.max_pages + (x0 >> A.page_shift)];
  if ((unsigned)page >= (unsigned)A.num_pages) {
    if (lane == 0) atomicCAS(A.err, 0, (int)kErrIndex);
    return;
  }
  const int64_t unit = (int64_t)kv4_unit<D>() << A.page_shift;
  const uint8_t* src = A.data + ((int64_t)page * A.Hkv + h) * 2 * unit;
  const int c = lane % kLanes, t0 = lane / kLanes;  // 8 channels, token
  const int row0 = x0 & ((1 << A.page_shift) - 1);
#pragma unroll
  for (int is_v = 0; is_v < 2; ++is_v, src += unit) {
    uint32_t codes[kRun / kTokens], scale[kRun / kTokens];
#pragma unroll
    for (int y = 0; y < kRun / kTokens; ++y) {  // rows behind the request's end lie in its page too
      const int row = row0 + y * kTokens + t0;
      codes[y] = __ldcs(reinterpret_cast<const uint32_t*>(src + ((((c >> 2) << A.page_shift) + row) << 4) + 4 * (c & 3)));
      scale[y] = src[((D / 2) << A.page_shift) + row * (D / 16) + (c >> 1)];
    }
    __nv_bfloat16* dst = (is_v ? A.v : A.k) + (bh * A.n + x0) * D + 8 * c;
    const float g = is_v ? A.v_scale : A.k_scale;
#pragma unroll
    for (int y = 0; y < kRun / kTokens; ++y) {
      const int t = y * kTokens + t0;
      if (x0 + t >= L) continue;
      uint32_t r[4];
      f16_of_codes(codes[y], f16x2_of_e4m3x2(scale[y] * 0x101u), r);
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = bf16x2_of_f16x2(r[k], g);
      __stcs(reinterpret_cast<uint4*>(dst + (int64_t)t * D), make_uint4(r[0], r[1], r[2], r[3]));
    }
  }
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" msa_status msa_kv4_gather(const msa_shape* shape, const msa_kv4_pages* pages, const int32_t* page_table,
                                     int32_t max_pages, const int32_t* seq_len, void* k, void* v, void* stream) {
  if (!shape) return MSA_ERR_INVALID_ARG;
  msa_status st = check_shape(shape);
  if (st != MSA_OK) return st;
  st = check_kv4_pages(pages);
  if (st != MSA_OK) return st;
  auto bad = [](const void* p, size_t a) { return !p || reinterpret_cast<uintptr_t>(p) % a; };
  if (max_pages < 1 || bad(page_table, 4) || bad(seq_len, 4) || bad(k, 16) || bad(v, 16) || k == v) return MSA_ERR_INVALID_ARG;
  if (k == pages->data || v == pages->data) return MSA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * pages->page_size >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  GatherArgs a;
  a.data = static_cast<const uint8_t*>(pages->data);
  a.table = page_table;
  a.seq_len = seq_len;
  a.k = static_cast<__nv_bfloat16*>(k);
  a.v = static_cast<__nv_bfloat16*>(v);
  a.B = shape->B;
  a.Hkv = shape->Hkv;
  a.n = shape->n;
  a.max_pages = max_pages;
  a.num_pages = pages->num_pages;
  a.page_shift = __builtin_ctz((unsigned)pages->page_size);
  const int64_t most = (int64_t)max_pages * pages->page_size;  // tokens that a request can hold
  a.runs = ceil_div(most < shape->n ? most : shape->n, kRun);
  a.k_scale = kv4_scale(pages->k_scale);
  a.v_scale = kv4_scale(pages->v_scale);
  a.err = device_error_word();
  if (!a.err) return MSA_ERR_CUDA;
  const int64_t ctas = ((int64_t)a.B * a.Hkv * a.runs + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  auto kern = shape->d_h == 128 ? kv4_gather_kernel<128> : kv4_gather_kernel<64>;
  kern<<<(unsigned)ctas, kThreads, 0, (cudaStream_t)stream>>>(a);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}
