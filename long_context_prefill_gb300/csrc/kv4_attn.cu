// Attention of drafted tokens over a paged cache held in 4 bits: the plain
// kernel, one CTA per row, its warps taking keys in turn, joined at the end.
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace msa {

msa_status check_tree_shape(const msa_shape* s);
msa_status check_page_geometry(int32_t num_pages, int32_t page_size);
float effective_scale(const msa_shape& s);

namespace {

constexpr int kWarps = 8;

struct RowArgs {
  int32_t B, Hq, Hkv, n, page_shift, max_pages, num_pages, words, sink, window;
  const int32_t *table, *seq_len, *tree_len, *depth;
  const uint32_t* mask;
  int64_t mask_stride;
  const __nv_bfloat16 *q, *k, *v;
  const uint8_t* data;
  float k_scale, v_scale;
  __nv_bfloat16* o;
  float* lse;
  float scale_log2;
  int* err;
};

template <int D, bool kKv4>
__global__ void __launch_bounds__(32 * kWarps) attn_rows_kernel(const RowArgs A) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int b = (int)(row / ((int64_t)A.Hq * A.n)), hq = (int)(row / A.n % A.Hq), i = (int)(row % A.n);
  const int kvh = hq / (A.Hq / A.Hkv);
  const int L = A.seq_len[b], T = A.tree_len ? A.tree_len[b] : A.n;
  if (T < 0 || T > A.n || L < T || L > ((int64_t)A.max_pages << A.page_shift)) {
    if (threadIdx.x == 0) atomicCAS(A.err, 0, (int)kErrIndex);
    return;
  }
  if (i >= T) return;
  const int C = L - T;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < kPer; ++x) {
    q[x] = __bfloat162float(A.q[row * D + kPer * lane + x]);
    o[x] = 0.f;
  }
  const int e = A.depth ? min(max(A.depth[(int64_t)b * A.n + i], 0), A.n - 1) : i;
  int64_t hole1 = A.window ? (int64_t)C + e - A.window + 1 : 0;  // keys sink .. hole1 - 1 are not seen
  if (A.mask && hole1 > C) hole1 = C;
  for (int j = warp; j < L; j += kWarps) {
    if (j >= A.sink && j < hole1) continue;
    if (j >= C) {
      const int x = j - C;
      if (A.mask ? !(A.mask[b * A.mask_stride + (int64_t)i * A.words + (x >> 5)] >> (x & 31) & 1u) : x > i) continue;
    }
    const int page = A.table[(int64_t)b * A.max_pages + (j >> A.page_shift)], r = j & ((1 << A.page_shift) - 1);
    if ((unsigned)page >= (unsigned)A.num_pages) {
      if (lane == 0) atomicCAS(A.err, 0, (int)kErrIndex);
      continue;
    }
    float k[kPer], v[kPer];
    if constexpr (kKv4) {
      const int64_t unit = (int64_t)kv4_unit<D>() << A.page_shift;
      const uint8_t* u = A.data + ((int64_t)page * A.Hkv + kvh) * 2 * unit;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int c = kPer * lane + x;
        const int64_t at = ((((int64_t)(c >> 5) << A.page_shift) + r) << 4) + (c & 31) / 2;
        const int64_t sc = ((int64_t)(D / 2) << A.page_shift) + r * (D / 16) + c / 16;
        uint32_t y[4];
        f16_of_codes(u[at] >> (4 * (c & 1)) & 15u, f16x2_of_e4m3x2(u[sc]), y);
        k[x] = __half2float(__ushort_as_half((unsigned short)y[0])) * A.k_scale;
        f16_of_codes(u[unit + at] >> (4 * (c & 1)) & 15u, f16x2_of_e4m3x2(u[unit + sc]), y);
        v[x] = __half2float(__ushort_as_half((unsigned short)y[0])) * A.v_scale;
      }
    } else {
      const int64_t at = ((((int64_t)page * A.Hkv + kvh) << A.page_shift) + r) * D + kPer * lane;
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        k[x] = __bfloat162float(A.k[at + x]);
        v[x] = __bfloat162float(A.v[at + x]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < kPer; ++x) s = fmaf(q[x], k[x], s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
    s *= A.scale_log2;
    const float top = fmaxf(m, s), keep = ex2(m - top), p = ex2(s - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = fmaf(p, v[x], o[x] * keep);
  }
  __shared__ float part[kWarps][D], ml[kWarps][2];
#pragma unroll
  for (int x = 0; x < kPer; ++x) part[warp][kPer * lane + x] = o[x];
  if (lane == 0) ml[warp][0] = m, ml[warp][1] = l;
  __syncthreads();
  if (threadIdx.x >= D) return;
  float top = -INFINITY, sum = 0.f, out = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][0]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) {
    const float f = ex2(ml[w][0] - ref);
    sum += f * ml[w][1];
    out += f * part[w][threadIdx.x];
  }
  A.o[row * D + threadIdx.x] = __float2bfloat16(sum == 0.f ? 0.f : out / sum);
  if (threadIdx.x == 0 && A.lse) A.lse[row] = sum == 0.f ? -INFINITY : (top + __log2f(sum)) * 0.69314718055994531f;
}

bool aligned(const void* p, size_t a, bool required) {
  if (!p) return !required;
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

msa_status rows(const msa_shape* shape, const void* q, const msa_kv_pages* pages, const msa_kv4_pages* kv4,
                const int32_t* page_table, int32_t max_pages, const int32_t* seq_len, const int32_t* tree_len,
                const uint32_t* tree_mask, int64_t mask_stride, const msa_tree_window* window, void* o, float* lse,
                void* ws, size_t ws_bytes, size_t need, void* stream) {
  const int32_t num_pages = pages ? pages->num_pages : kv4->num_pages, page_size = pages ? pages->page_size : kv4->page_size;
  if (max_pages < 1) return MSA_ERR_INVALID_ARG;
  if (!aligned(q, 16, true) || !aligned(o, 16, true) || !aligned(page_table, 4, true) || !aligned(seq_len, 4, true) ||
      !aligned(tree_len, 4, false) || !aligned(tree_mask, 4, false) || !aligned(lse, 4, false) || !aligned(ws, 16, true))
    return MSA_ERR_INVALID_ARG;
  if (q == o) return MSA_ERR_INVALID_ARG;
  const int32_t words = (shape->n + 31) / 32;
  if (tree_mask && mask_stride != 0 && mask_stride < (int64_t)shape->n * words) return MSA_ERR_INVALID_ARG;
  if (window && (window->sink < 0 || window->window < 1 || !aligned(window->depth, 4, false) || (window->depth && !tree_mask)))
    return MSA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size * shape->Hkv + 256 >= ((int64_t)1 << 31)) return MSA_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * page_size >= ((int64_t)1 << 31) - 256) return MSA_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MSA_ERR_WORKSPACE_TOO_SMALL;
  RowArgs a;
  memset(&a, 0, sizeof(a));
  a.B = shape->B;
  a.Hq = shape->Hq;
  a.Hkv = shape->Hkv;
  a.n = shape->n;
  a.page_shift = __builtin_ctz((unsigned)page_size);
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.words = words;
  if (window) a.sink = window->sink, a.window = window->window, a.depth = window->depth;
  a.table = page_table;
  a.seq_len = seq_len;
  a.tree_len = tree_len;
  a.mask = tree_mask;
  a.mask_stride = mask_stride;
  a.q = static_cast<const __nv_bfloat16*>(q);
  if (pages) {
    a.k = static_cast<const __nv_bfloat16*>(pages->k);
    a.v = static_cast<const __nv_bfloat16*>(pages->v);
  } else {
    a.data = static_cast<const uint8_t*>(kv4->data);
    a.k_scale = kv4_scale(kv4->k_scale);
    a.v_scale = kv4_scale(kv4->v_scale);
  }
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.scale_log2 = effective_scale(*shape) * 1.4426950408889634f;
  a.err = device_error_word();
  if (!a.err) return MSA_ERR_CUDA;
  auto kern = pages ? (shape->d_h == 128 ? attn_rows_kernel<128, false> : attn_rows_kernel<64, false>)
                    : (shape->d_h == 128 ? attn_rows_kernel<128, true> : attn_rows_kernel<64, true>);
  kern<<<(unsigned)((int64_t)shape->B * shape->Hq * shape->n), 32 * kWarps, 0, (cudaStream_t)stream>>>(a);
  note_launch();
  return cudaGetLastError() == cudaSuccess ? MSA_OK : MSA_ERR_CUDA;
}

}  // namespace

}  // namespace msa

using namespace msa;

extern "C" size_t msa_attn_tree_kv4_workspace(const msa_shape* shape) { return msa_attn_tree_workspace(shape); }

extern "C" msa_status msa_attn_tree_kv4(const msa_shape* shape, const void* q, const msa_kv4_pages* pages,
                                        const int32_t* page_table, int32_t max_pages, const int32_t* seq_len,
                                        const int32_t* tree_len, const uint32_t* tree_mask, int64_t mask_stride,
                                        const msa_tree_window* window, void* o, float* lse, void* ws, size_t ws_bytes,
                                        void* stream) {
  msa_status st = check_tree_shape(shape);
  if (st != MSA_OK) return st;
  st = check_kv4_pages(pages);
  if (st != MSA_OK) return st;
  return rows(shape, q, nullptr, pages, page_table, max_pages, seq_len, tree_len, tree_mask, mask_stride, window, o, lse,
              ws, ws_bytes, msa_attn_tree_kv4_workspace(shape), stream);
}
