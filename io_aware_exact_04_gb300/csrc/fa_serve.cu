// Attention of whole prompts and of drafted trees over a cache in pages: entry points and kernels.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "fa_internal.h"
#include "serve.cuh"
#include "tmap.h"

namespace fa {

struct ServeArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;  // token and head strides, elements
  float* lse;  // [Hq, T] or null
  // the cache; prompts have none (table null)
  const uint16_t *kc, *vc;
  long long c_sp, c_sh, c_st;
  int n_pages, page_shift;
  const int* table;
  long long table_stride;
  int table_width;
  const int* lens;
  const uint32_t* mask;  // null: a chain
  int words;
  const int* cu;
  int B, T, Hq, Hkv, G;
  float scale_log2;
  int* status;
};

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t x) {
  return F16 ? __half2float(__ushort_as_half(x)) : __bfloat162float(__ushort_as_bfloat16(x));
}

// One block for each (token, query head): keys in tiles of 128, a key a thread.
template <int D, bool F16>
__global__ void __launch_bounds__(128) serve_rows_kernel(ServeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float qs[D], ps[128], red[4];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  if (t == 0 && h == 0) check_offsets(a.cu, a.B, a.T, a.status);
  const int b = find_sequence(a.cu, a.B, t);
  if (b < 0) return;
  const SeqRange r = seq_range(a.cu, b, a.T, a.status);
  if (t < r.lo || t >= r.hi) return;
  const int kvh = h / a.G, node = t - r.lo, n = r.hi - r.lo;
  int ctx = 0;
  if (a.table) {
    const int cap = a.table_width << a.page_shift;
    ctx = min(max(a.lens[b], 0), cap);
    if (ctx != a.lens[b]) record_check(a.status, SITE_S_LENGTH);
  }
  if (tid < D) qs[tid] = to_f32<F16>(a.q[t * a.q_st + h * a.q_sh + tid]) * a.scale_log2;
  __syncthreads();
  const int total = ctx + (a.mask ? n : node + 1);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = 0; j0 < total; j0 += 128) {
    const int j = j0 + tid;
    bool seen = j < total;
    const uint16_t *kr = nullptr, *vr = nullptr;
    if (seen && j < ctx) {
      const int id = a.table[b * a.table_stride + (j >> a.page_shift)];
      if (id < 0 || id >= a.n_pages) {
        record_check(a.status, SITE_S_PAGE);
      } else {
        const long long off = id * a.c_sp + kvh * a.c_sh + (j & ((1 << a.page_shift) - 1)) * a.c_st;
        kr = a.kc + off;
        vr = a.vc + off;
      }
    } else if (seen) {
      const int i = j - ctx;
      if (a.mask) seen = i < 32 * a.words && (a.mask[(long long)t * a.words + (i >> 5)] >> (i & 31) & 1);
      kr = a.k + (r.lo + i) * a.k_st + kvh * a.k_sh;
      vr = a.v + (r.lo + i) * a.v_st + kvh * a.v_sh;
    }
    float s = -INFINITY;
    if (seen) {
      s = 0.f;
      if (kr)
        for (int c = 0; c < D; ++c) s = fmaf(qs[c], to_f32<F16>(kr[c]), s);
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float base = mn == -INFINITY ? 0.f : mn;
    ps[tid] = exp2f(s - base);
    const float f = exp2f((m == -INFINITY ? base : m) - base);
    __syncthreads();
    l *= f;
    acc *= f;
    m = mn;
    for (int i = 0; i < 128 && j0 + i < total; ++i) {
      const float p = ps[i];
      l += p;
      if (p == 0.f || tid >= D) continue;
      const int jj = j0 + i;
      const uint16_t* row;
      if (jj < ctx) {
        const int id = a.table[b * a.table_stride + (jj >> a.page_shift)];
        if (id < 0 || id >= a.n_pages) continue;
        row = a.vc + id * a.c_sp + kvh * a.c_sh + (jj & ((1 << a.page_shift) - 1)) * a.c_st;
      } else {
        row = a.v + (r.lo + jj - ctx) * a.v_st + kvh * a.v_sh;
      }
      acc = fmaf(p, to_f32<F16>(row[tid]), acc);
    }
    __syncthreads();
  }
  const float o = l != 0.f ? acc / l : 0.f;  // NaN stays NaN
  if (tid < D)
    a.o[t * a.o_st + h * a.o_sh + tid] =
        F16 ? __half_as_ushort(__float2half_rn(o)) : __bfloat16_as_ushort(__float2bfloat16_rn(o));
  if (tid == 0 && a.lse) a.lse[(long long)h * a.T + t] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

static int launch_serve(const ServeArgs& a, int d, int dtype, cudaStream_t stream) {
  const dim3 grid(a.T, a.Hq), block(128);
  if (d == 64) return dtype == FA_FP16 ? launch_pdl("serve_rows_kernel", serve_rows_kernel<64, true>, grid, block, 0, stream, a)
                                       : launch_pdl("serve_rows_kernel", serve_rows_kernel<64, false>, grid, block, 0, stream, a);
  return dtype == FA_FP16 ? launch_pdl("serve_rows_kernel", serve_rows_kernel<128, true>, grid, block, 0, stream, a)
                          : launch_pdl("serve_rows_kernel", serve_rows_kernel<128, false>, grid, block, 0, stream, a);
}

}  // namespace fa

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The largest stride in elements that a tensor map takes (2^40 bytes, exclusive).
constexpr long long kMaxStride = (1LL << 39) - 8;

int check_stride(int64_t s) {
  if (s <= 0 || s % 8 != 0) return FA_ERR_INVALID_ARG;
  return s <= kMaxStride ? FA_OK : FA_ERR_UNSUPPORTED;
}

int check_rows(const fa_rows* r) {
  if (!r || !r->data) return FA_ERR_INVALID_ARG;
  if (!aligned16(r->data)) return FA_ERR_MISALIGNED;
  const int rc = check_stride(r->token_stride);
  return rc != FA_OK ? rc : check_stride(r->head_stride);
}

int check_sizes(int B, int T, int Hq, int Hkv, int d, int dtype, float scale) {
  if (B < 0 || T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_BF16 && dtype != FA_FP16) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hq / Hkv > 128 || Hq > 65535 || B > (1 << 20) || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int check_pages(const fa_pages* c) {
  if (!c || !c->k || !c->v || !c->table) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return FA_ERR_MISALIGNED;
  for (int64_t s : {c->page_stride, c->head_stride, c->token_stride})
    if (const int rc = check_stride(s); rc != FA_OK) return rc;
  if (c->n_pages < 1 || c->table_width < 1 || c->table_stride < c->table_width) return FA_ERR_INVALID_ARG;
  switch (c->page_size) {
    case 16: case 32: case 64: case 128: case 256: break;
    default: return FA_ERR_UNSUPPORTED;
  }
  if ((long long)c->table_width * c->page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int forward(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse, const fa_pages* cache,
            const int32_t* lens, const int32_t* cu, const uint32_t* mask, int words, int B, int T, int Hq, int Hkv, int d,
            int dtype, float scale, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  for (const fa_rows* r : {q, k, v, o})
    if (const int rc = check_rows(r); rc != FA_OK) return rc;
  if (!cu || !workspace || (lse && !aligned16(lse))) return !cu || !workspace ? FA_ERR_INVALID_ARG : FA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if (workspace_bytes < fa_forward_tree_workspace_size(d)) return FA_ERR_INVALID_ARG;
  int err = FA_OK;
  int* status = fa::status_word(&err);
  if (!status) return err;
  fa::ServeArgs a = {};
  a.q = static_cast<const uint16_t*>(q->data);
  a.k = static_cast<const uint16_t*>(k->data);
  a.v = static_cast<const uint16_t*>(v->data);
  a.o = static_cast<uint16_t*>(o->data);
  a.q_st = q->token_stride, a.q_sh = q->head_stride;
  a.k_st = k->token_stride, a.k_sh = k->head_stride;
  a.v_st = v->token_stride, a.v_sh = v->head_stride;
  a.o_st = o->token_stride, a.o_sh = o->head_stride;
  a.lse = lse;
  if (cache) {
    a.kc = static_cast<const uint16_t*>(cache->k);
    a.vc = static_cast<const uint16_t*>(cache->v);
    a.c_sp = cache->page_stride, a.c_sh = cache->head_stride, a.c_st = cache->token_stride;
    a.n_pages = cache->n_pages;
    a.page_shift = log2_of(cache->page_size);
    a.table = cache->table;
    a.table_stride = cache->table_stride;
    a.table_width = cache->table_width;
    a.lens = lens;
    a.mask = mask;
    a.words = words;
  }
  a.cu = cu;
  a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = status;
  return fa::launch_serve(a, d, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

size_t fa_forward_tree_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  int sms = 0;
  if (!fa::sm_count(&sms)) return 0;
  return (size_t)2 * sms * 256 * (d + 1) * 4;
}

int fa_forward_prompt(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                      const int32_t* cu_seqlens, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                      void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  const int rc = check_sizes(B, T, Hq, Hkv, d, dtype, scale);
  if (rc != FA_OK) return rc;
  if (B == 0 || T == 0) return FA_OK;
  return forward(q, k, v, o, lse, nullptr, nullptr, cu_seqlens, nullptr, 0, B, T, Hq, Hkv, d, dtype, scale, workspace,
                 workspace_bytes, stream);
}

int fa_forward_tree(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                    const fa_pages* cache, const int32_t* lens, const int32_t* cu_nodes, const uint32_t* mask,
                    int mask_words, int B, int T, int Hq, int Hkv, int d, int dtype, float scale, void* workspace,
                    size_t workspace_bytes, fa_stream_t stream) {
  int rc = check_sizes(B, T, Hq, Hkv, d, dtype, scale);
  if (rc != FA_OK) return rc;
  if (mask && (mask_words < 1 || mask_words > (1 << 20))) return mask_words < 1 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  rc = check_pages(cache);
  if (rc != FA_OK) return rc;
  if (!lens) return FA_ERR_INVALID_ARG;
  return forward(q, k, v, o, lse, cache, lens, cu_nodes, mask, mask_words, B, T, Hq, Hkv, d, dtype, scale, workspace,
                 workspace_bytes, stream);
}

}  // extern "C"
