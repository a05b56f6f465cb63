// Attention of drafted trees over a cache in 8 bits: entry points and kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_internal.h"
#include "serve.cuh"
#include "serve_args.h"

namespace fa {

struct Serve8Args {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;  // token and head strides, elements
  float* lse;  // [Hq, T] or null
  const uint8_t *kc, *vc;
  long long c_sp, c_sh, c_st;
  const float *ks, *vs;
  long long s_sp, s_sh;
  int block_shift;
  int n_pages, page_shift;
  const int* table;
  long long table_stride;
  int table_width;
  const int* lens;
  const uint32_t* mask;  // null: a chain
  int words;
  const int* cu;
  int B, T, Hq, Hkv, G;
  float scale;
  int* status;
};

template <bool F16>
__device__ __forceinline__ float to_float(uint16_t x) {
  float f;
  if (F16)
    asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(x));
  else
    f = __uint_as_float((uint32_t)x << 16);
  return f;
}
__device__ __forceinline__ float e4m3_float(uint8_t x) {
  float f;
  asm("{\n\t.reg .b32 t;\n\t.reg .b16 l, h;\n\tcvt.rn.f16x2.e4m3x2 t, %1;\n\tmov.b32 {l, h}, t;\n\tcvt.f32.f16 %0, l;\n\t}"
      : "=f"(f)
      : "h"((uint16_t)x));
  return f;
}

// A warp for each row (token, query head): 32 keys at a time, a key a lane for the scores, D / 32 columns
// a lane for O.
template <int D, bool F16>
__global__ void __launch_bounds__(128) tree8_kernel(Serve8Args a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float qs[4][D];
  if (blockIdx.x == 0 && blockIdx.y == 0) check_offsets(a.cu, a.B, a.T, a.status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * 4 + warp, head = blockIdx.y, kvh = head / a.G;
  if (t >= a.T) return;
  const int b = find_sequence(a.cu, a.B, t);
  if (b < 0) return;
  const SeqRange r = seq_range(a.cu, b, a.T, a.status);
  if (t < r.lo || t >= r.hi) return;
  const int len = a.lens[b], L = min(max(len, 0), a.table_width << a.page_shift), n = r.hi - r.lo, me = t - r.lo;
  if (L != len && lane == 0) record_check(a.status, SITE_S_LENGTH);
  for (int c = lane; c < D; c += 32) qs[warp][c] = to_float<F16>(a.q[t * a.q_st + head * a.q_sh + c]);
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  for (int j0 = 0; j0 < L + n; j0 = j0 < L ? min(L, j0 + 32) : j0 + 32) {
    const bool cached = j0 < L;
    const int j = j0 + lane;
    bool seen;
    float s = 0.f, vscale = 1.f;
    const uint8_t* v8 = nullptr;
    if (cached) {
      seen = j < L;
      const int id = seen ? a.table[b * a.table_stride + (j >> a.page_shift)] : 0;
      const int in_page = j & ((1 << a.page_shift) - 1);
      if (seen && (id < 0 || id >= a.n_pages)) {
        record_check(a.status, SITE_S_PAGE);
      } else if (seen) {
        const uint8_t* k8 = a.kc + id * a.c_sp + kvh * a.c_sh + in_page * a.c_st;
        const long long at = id * a.s_sp + kvh * a.s_sh + (in_page >> a.block_shift);
        for (int c = 0; c < D; ++c) s = fmaf(qs[warp][c], e4m3_float(k8[c]), s);
        s *= a.ks[at];
        vscale = a.vs[at];
        v8 = a.vc + id * a.c_sp + kvh * a.c_sh + in_page * a.c_st;
      }
    } else {
      const int i = j - L;
      seen = i < n && (a.mask ? (i >> 5) < a.words && (a.mask[(long long)t * a.words + (i >> 5)] >> (i & 31) & 1) : i <= me);
      if (seen) {
        const uint16_t* k = a.k + (r.lo + i) * a.k_st + kvh * a.k_sh;
        for (int c = 0; c < D; ++c) s = fmaf(qs[warp][c], to_float<F16>(k[c]), s);
      }
    }
    s = seen ? s * a.scale : -INFINITY;
    float top = s;
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float base = top == -INFINITY ? 0.f : top, f = expf(m - base);
    const float p = seen ? expf(s - base) : 0.f;
    m = top;
    l = l * f + p;
    for (int c = 0; c < D / 32; ++c) o[c] *= f;
    for (int x = 0; x < 32; ++x) {
      const float px = __shfl_sync(0xffffffffu, p * vscale, x);
      const unsigned long long row = __shfl_sync(0xffffffffu, (unsigned long long)v8, x);
      if (!__shfl_sync(0xffffffffu, (int)seen, x)) continue;
      if (cached && !row) continue;
      for (int c = 0; c < D / 32; ++c)
        o[c] = fmaf(px, cached ? e4m3_float(reinterpret_cast<const uint8_t*>(row)[lane + 32 * c])
                               : to_float<F16>(a.v[(r.lo + j0 + x - L) * a.v_st + kvh * a.v_sh + lane + 32 * c]), o[c]);
    }
  }
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l != 0.f ? 1.f / l : 0.f;
  for (int c = 0; c < D / 32; ++c) {
    const float x = o[c] * inv;
    a.o[t * a.o_st + head * a.o_sh + lane + 32 * c] = (uint16_t)(F16 ? pack_f16x2(x, x) : pack_bf16x2(x, x));
  }
  if (lane == 0 && a.lse) a.lse[(long long)head * a.T + t] = l != 0.f ? m + logf(l) : -INFINITY;
}

static int launch_serve8(const Serve8Args& a, int d, int dtype, cudaStream_t stream) {
  const dim3 grid((a.T + 3) / 4, a.Hq);
  const auto go = [&](auto kernel) { return launch_pdl("tree8_kernel", kernel, grid, dim3(128), 0, stream, a); };
  if (d == 64) return dtype == FA_FP16 ? go(tree8_kernel<64, true>) : go(tree8_kernel<64, false>);
  return dtype == FA_FP16 ? go(tree8_kernel<128, true>) : go(tree8_kernel<128, false>);
}

}  // namespace fa

using namespace fa::host;

extern "C" {

size_t fa_forward_tree_8bit_workspace_size(int d) {
  return d == 64 || d == 128 ? 256 : 0;
}

int fa_forward_tree_8bit(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                         const fa_pages* cache, const fa_scales* scales, const int32_t* lens, const int32_t* cu_nodes,
                         const uint32_t* mask, int mask_words, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                         void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  int rc = check_sizes(B, T, Hq, Hkv, d, dtype, scale);
  if (rc != FA_OK) return rc;
  if (mask && (mask_words < 1 || mask_words > (1 << 20))) return mask_words < 1 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if ((rc = check_pages(cache, 16)) != FA_OK || (rc = check_scales(scales, cache->page_size)) != FA_OK) return rc;
  for (const fa_rows* r : {q, k, v, o})
    if ((rc = check_rows(r)) != FA_OK) return rc;
  if (!lens || !cu_nodes || !workspace) return FA_ERR_INVALID_ARG;
  if ((lse && !aligned16(lse)) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if (workspace_bytes < fa_forward_tree_8bit_workspace_size(d)) return FA_ERR_INVALID_ARG;
  int err = FA_OK;
  int* status = fa::status_word(&err);
  if (!status) return err;
  fa::Serve8Args a = {};
  a.q = static_cast<const uint16_t*>(q->data);
  a.k = static_cast<const uint16_t*>(k->data);
  a.v = static_cast<const uint16_t*>(v->data);
  a.o = static_cast<uint16_t*>(o->data);
  a.q_st = q->token_stride, a.q_sh = q->head_stride;
  a.k_st = k->token_stride, a.k_sh = k->head_stride;
  a.v_st = v->token_stride, a.v_sh = v->head_stride;
  a.o_st = o->token_stride, a.o_sh = o->head_stride;
  a.lse = lse;
  a.kc = static_cast<const uint8_t*>(cache->k), a.vc = static_cast<const uint8_t*>(cache->v);
  a.c_sp = cache->page_stride, a.c_sh = cache->head_stride, a.c_st = cache->token_stride;
  a.ks = scales->k, a.vs = scales->v, a.s_sp = scales->page_stride, a.s_sh = scales->head_stride;
  a.block_shift = log2_of(scales->block);
  a.n_pages = cache->n_pages, a.page_shift = log2_of(cache->page_size);
  a.table = cache->table, a.table_stride = cache->table_stride, a.table_width = cache->table_width;
  a.lens = lens, a.mask = mask, a.words = mask_words, a.cu = cu_nodes;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
  a.scale = scale;
  a.status = status;
  return fa::launch_serve8(a, d, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
