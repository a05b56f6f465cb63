// New tokens on their way into the cache: queries and keys rotated by the angles of their positions,
// keys and values written into pages of 16 bits, or of 8 bits with a scale for each block.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>

#include "fa_internal.h"
#include "serve.cuh"
#include "serve_args.h"

namespace fa {

struct RotaryArgs {
  const uint16_t *q, *k, *v;  // q null: none
  uint16_t *qo, *ko;          // ko null: not written
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, ko_st, ko_sh;
  const float* angles;        // null: nothing is rotated
  long long a_stride;
  int positions, dim, interleaved;
  const int* at;
  // the cache; kc null: none. Strides in elements
  uint8_t *kc, *vc;
  long long c_sp, c_sh, c_st;
  int n_pages, page_shift;
  const int* table;
  long long table_stride;
  int table_width;
  float *ks, *vs;             // scales of a cache in 8 bits
  long long s_sp, s_sh;
  int block_shift;
  const int *start, *cu, *rows;
  int B, T, Tkv, Hq, Hkv;
  int splits;                 // warps that share a token's head rows
  long long blocks8;          // blocks of the grid with work in 8 bits; those behind them rotate queries
  int head_groups;
  int* status;
};

// ---------------------------------------------------------------------------------------------
// A thread holds two chunks of 8 elements of a head row, chosen so that a rotation's pairs lie in one
// thread: with halves, chunks p and p + dim / 16; behind the rotated part, neighbours.
struct ChunkPair {
  int c0, c1;
  bool turned;
};
__device__ __forceinline__ ChunkPair chunk_pair(int p, int dim) {
  const int pairs = dim >> 4;
  ChunkPair c;
  c.turned = p < pairs;
  c.c0 = c.turned ? p : 2 * p;
  c.c1 = c.turned ? p + pairs : 2 * p + 1;
  return c;
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (F16) {
      asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
          : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
          : "r"(w[i]));
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = F16 ? pack_f16x2(f[2 * i], f[2 * i + 1]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Cosines and sines of a thread's pairs: with halves the 8 of chunk c0; interleaved the 4 of each chunk.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const RotaryArgs& a, int position, const ChunkPair& cp, Turn* t) {
  const float* row = a.angles + position * a.a_stride;
  const int j0 = a.interleaved ? 4 * cp.c0 : 8 * cp.c0, j1 = a.interleaved ? 4 * cp.c1 : 8 * cp.c0 + 4;
  const float4 x0 = __ldg(reinterpret_cast<const float4*>(row + j0)), x1 = __ldg(reinterpret_cast<const float4*>(row + j1));
  row += a.dim >> 1;
  const float4 y0 = __ldg(reinterpret_cast<const float4*>(row + j0)), y1 = __ldg(reinterpret_cast<const float4*>(row + j1));
  t->c[0] = x0.x, t->c[1] = x0.y, t->c[2] = x0.z, t->c[3] = x0.w, t->c[4] = x1.x, t->c[5] = x1.y, t->c[6] = x1.z, t->c[7] = x1.w;
  t->s[0] = y0.x, t->s[1] = y0.y, t->s[2] = y0.z, t->s[3] = y0.w, t->s[4] = y1.x, t->s[5] = y1.y, t->s[6] = y1.z, t->s[7] = y1.w;
}
// The products are rounded before they are added: what elementary operations give, bit by bit.
__device__ __forceinline__ void turn_pair(float& x1, float& x2, float c, float s) {
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s)), y2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1, x2 = y2;
}
__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const Turn& t, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_pair(x[2 * i], x[2 * i + 1], t.c[i], t.s[i]);
      turn_pair(y[2 * i], y[2 * i + 1], t.c[4 + i], t.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(x[i], y[i], t.c[i], t.s[i]);
  }
}

// The packed token t, by a whole warp: its sequence (or -1: none) and its position among the sequence's
// new tokens. Without offsets every row is a token of sequence 0.
__device__ __forceinline__ int token_of(const RotaryArgs& a, int t, int* i) {
  *i = t;
  if (!a.cu) return 0;
  const int b = find_sequence(a.cu, a.B, t);
  if (b < 0) return -1;
  const SeqRange r = seq_range(a.cu, b, a.T, a.status);
  if (t < r.lo || t >= r.hi) return -1;
  *i = t - r.lo;
  return b;
}

// Share `split` of the head rows of token t, by a warp: queries rotated, and (KV) keys rotated and
// keys and values written into 16-bit pages. D / 16 lanes a row, so that the loads and stores are
// whole sectors; the angles are loaded once for all rows of the warp, four rows' loads at a time.
template <int D, bool F16, bool KV>
__device__ __forceinline__ void rotate_rows(const RotaryArgs& a, int t, int split, int splits) {
  constexpr int LPR = D / 16, RPI = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane / LPR, p = lane % LPR;
  int i;
  const int b = token_of(a, t, &i);
  if (b < 0) return;
  const long long pos = (a.kc ? (long long)a.start[b] : 0) + i;
  const long long place = a.at ? a.at[t] : pos;
  if (place < 0 || place >= a.positions) return record_check(a.status, SITE_S_ANGLE);
  const ChunkPair cp = chunk_pair(p, a.dim);
  Turn tn;
  if (cp.turned) load_turn(a, (int)place, cp, &tn);
  uint16_t *kc = nullptr, *vc = nullptr;
  if (KV && a.kc) {
    if (pos < 0 || pos >= (long long)a.table_width << a.page_shift) {
      record_check(a.status, SITE_S_LENGTH);
    } else {
      const int id = a.table[b * a.table_stride + (pos >> a.page_shift)];
      if (id < 0 || id >= a.n_pages) {
        record_check(a.status, SITE_S_PAGE);
      } else {
        const long long to = id * a.c_sp + (pos & ((1 << a.page_shift) - 1)) * a.c_st;
        kc = reinterpret_cast<uint16_t*>(a.kc) + to;
        vc = reinterpret_cast<uint16_t*>(a.vc) + to;
      }
    }
  }
  const int nq = a.q ? a.Hq : 0, keys = KV ? nq + a.Hkv : nq, all = KV && vc ? keys + a.Hkv : keys;
  constexpr int U = 4;
  for (int j0 = split * RPI; j0 < all; j0 += U * splits * RPI) {
    uint4 x[U], y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * splits * RPI + sub;
      if (j >= all) continue;
      const uint16_t* row = j < nq ? a.q + t * a.q_st + j * a.q_sh
                                   : j < keys ? a.k + t * a.k_st + (j - nq) * a.k_sh : a.v + t * a.v_st + (j - keys) * a.v_sh;
      x[u] = *reinterpret_cast<const uint4*>(row + 8 * cp.c0);
      y[u] = *reinterpret_cast<const uint4*>(row + 8 * cp.c1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * splits * RPI + sub;
      if (j >= all) continue;
      if (j < keys && cp.turned) {
        float f[8], g[8];
        unpack8<F16>(x[u], f);
        unpack8<F16>(y[u], g);
        turn(f, g, tn, a.interleaved);
        x[u] = pack8<F16>(f);
        y[u] = pack8<F16>(g);
      }
      auto put = [&](uint16_t* row) {
        *reinterpret_cast<uint4*>(row + 8 * cp.c0) = x[u];
        *reinterpret_cast<uint4*>(row + 8 * cp.c1) = y[u];
      };
      if (j < nq) {
        put(a.qo + t * a.qo_st + j * a.qo_sh);
      } else if (j < keys) {
        if (a.ko) put(a.ko + t * a.ko_st + (j - nq) * a.ko_sh);
        if (kc) put(kc + (j - nq) * a.c_sh);
      } else {
        put(vc + (j - keys) * a.c_sh);
      }
    }
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(128) rotary_rows_kernel(RotaryArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && a.cu) check_offsets(a.cu, a.B, a.T, a.status);
  const long long w = blockIdx.x * 4LL + (threadIdx.x >> 5);
  const int t = (int)(w / a.splits), split = (int)(w - (long long)t * a.splits);
  if (w < (long long)a.T * a.splits) rotate_rows<D, F16, true>(a, t, split, a.splits);
}

// ---------------------------------------------------------------------------------------------
// A positive finite value as m 2^e with m in [2^23, 2^24).
__device__ __forceinline__ void split_float(float x, uint32_t* m, int* e) {
  const uint32_t u = __float_as_uint(x);
  uint32_t f = u & 0x7fffffu;
  int x2 = (int)(u >> 23) - 150;
  if (u >> 23)
    f |= 0x800000u;
  else
    ++x2;
  const int up = __clz(f) - 8;
  *m = f << up;
  *e = x2 - up;
}
// The least k with most <= 448 scale 2^k (448 = 7 2^6): both exact, so no rounding decides.
__device__ __forceinline__ int growth(float most, float scale) {
  uint32_t m, s;
  int e, f;
  split_float(most, &m, &e);
  split_float(scale, &s, &f);
  return e - f - 8 + (4 * m > 7 * s ? 1 : 8 * m <= 7 * s ? -1 : 0);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // an infinity would saturate: NaN, as the type has none
    const float lo = fabsf(x[2 * i]) <= FLT_MAX ? x[2 * i] * inv : NAN, hi = fabsf(x[2 * i + 1]) <= FLT_MAX ? x[2 * i + 1] * inv : NAN;
    h[i] = e4m3x2(lo, hi);
  }
  return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}
// Eight e4m3 values times a power of two, rounded again.
__device__ __forceinline__ uint2 e4m3x8_scaled(uint2 x, float by) {
  const uint32_t w[2] = {x.x, x.y};
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float lo, hi;
      asm("{\n\t.reg .b32 t;\n\t.reg .b16 l, h;\n\tcvt.rn.f16x2.e4m3x2 t, %2;\n\tmov.b32 {l, h}, t;\n\t"
          "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
          : "=f"(lo), "=f"(hi)
          : "h"((uint16_t)(w[i] >> (16 * k))));
      h[k] = e4m3x2(lo * by, hi * by);
    }
    r[i] = h[0] | h[1] << 16;
  }
  return make_uint2(r[0], r[1]);
}

// The blocks of sequence b that its new tokens touch are numbered from (cu[b] >> block_shift) + 2 b: no
// two sequences' numbers meet, as a sequence of n tokens touches (n >> block_shift) + 2 blocks at most.
// The sequence of number u, by a whole warp, 32 candidates a step.
__device__ __forceinline__ int find_block(const RotaryArgs& a, long long u) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + min(lane * step, n - 1);
    const unsigned below = __ballot_sync(0xffffffffu, (a.cu[i] >> a.block_shift) + 2LL * i <= u);
    if (below == 0) return -1;
    const int at = min((31 - __clz(below)) * step, n - 1);
    n = min(step, n - at);
    lo += at;
  }
  return (a.cu[lo] >> a.block_shift) + 2LL * lo <= u ? lo : -1;
}

// Into 8 bits. A team of block x D / 1024 warps takes one block of one head, of K or of V: a thread two
// pairs of chunks, in registers from the load to the store, so that the block's largest magnitude is
// known before anything is rounded and every row is read once. A CTA has as many teams as fit in eight
// warps (one, where the block is larger), on heads that follow each other.
template <int D, bool F16>
__device__ __forceinline__ void append_block(const RotaryArgs& a, long long unit) {
  constexpr int LPR = D / 16, RPI = 32 / LPR;
  __shared__ float warp_most[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int block = 1 << a.block_shift, wpt = block * D / 1024;
  const int team = warp / wpt, w = warp - team * wpt;
  const long long slot = unit / a.head_groups;
  const int job = (int)(unit - slot * a.head_groups) * max(1, 8 / wpt) + team;  // K of all heads, then V
  const bool is_v = job >= a.Hkv;
  const int h = is_v ? job - a.Hkv : job;
  const int b = find_block(a, slot);
  float f[2][2][8];
  float most = 0.f;
  bool fresh_token[2] = {false, false};
  uint8_t* to = nullptr;
  float* scale = nullptr;
  int first = 0;  // the block's first new token
  const ChunkPair cp = chunk_pair(lane % LPR, is_v ? 0 : a.dim);
  const int place0 = w * 2 * RPI + lane / LPR;  // the thread's tokens in the block: this one and RPI behind it
  if (b >= 0 && job < 2 * a.Hkv) {
    const SeqRange r = seq_range(a.cu, b, a.T, a.status);
    const long long start = a.start[b], end = start + (r.hi - r.lo);
    const long long base = ((start >> a.block_shift) + (slot - ((a.cu[b] >> a.block_shift) + 2LL * b))) << a.block_shift;
    if (r.hi > r.lo && base < end) {
      int id = -1;
      if (base < 0 || base >= (long long)a.table_width << a.page_shift) {
        if (lane == 0) record_check(a.status, SITE_S_LENGTH);
      } else {
        id = a.table[b * a.table_stride + (base >> a.page_shift)];
        if (id < 0 || id >= a.n_pages) {
          if (lane == 0) record_check(a.status, SITE_S_PAGE);
          id = -1;
        }
      }
      const int in_page = (int)(base & ((1 << a.page_shift) - 1));
      if (id >= 0) {
        to = (is_v ? a.vc : a.kc) + id * a.c_sp + h * a.c_sh + in_page * a.c_st;
        scale = (is_v ? a.vs : a.ks) + id * a.s_sp + h * a.s_sh + (in_page >> a.block_shift);
      }
      first = (int)max(0LL, start - base);
      const int last = (int)min((long long)block, end - base);
      uint4 x[2][2];
      int place[2] = {0, 0};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = place0 + u * RPI;
        if (i < first || i >= last) continue;
        const int t = (int)(r.lo + (base + i - start));
        int row = t;
        if (a.rows) {
          row = a.rows[t];
          if (row < 0 || row >= a.Tkv) {
            record_check(a.status, SITE_S_ROW);
            continue;
          }
        }
        if (a.angles) {
          const long long p = a.at ? a.at[t] : base + i;
          if (p < 0 || p >= a.positions) {
            record_check(a.status, SITE_S_ANGLE);
            continue;
          }
          place[u] = (int)p;
        }
        fresh_token[u] = true;
        const uint16_t* from = is_v ? a.v + row * a.v_st + h * a.v_sh : a.k + row * a.k_st + h * a.k_sh;
        x[u][0] = *reinterpret_cast<const uint4*>(from + 8 * cp.c0);
        x[u][1] = *reinterpret_cast<const uint4*>(from + 8 * cp.c1);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!fresh_token[u]) continue;
        unpack8<F16>(x[u][0], f[u][0]);
        unpack8<F16>(x[u][1], f[u][1]);
        if (!is_v && a.angles && cp.turned) {
          Turn tn;
          load_turn(a, place[u], cp, &tn);
          turn(f[u][0], f[u][1], tn, a.interleaved);
        }
        if (!is_v && a.ko) {
          uint16_t* ko = a.ko + (r.lo + (base + place0 + u * RPI - start)) * a.ko_st + h * a.ko_sh;
          *reinterpret_cast<uint4*>(ko + 8 * cp.c0) = pack8<F16>(f[u][0]);
          *reinterpret_cast<uint4*>(ko + 8 * cp.c1) = pack8<F16>(f[u][1]);
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (const float m = fabsf(f[u][c][e]); m <= FLT_MAX) most = fmaxf(most, m);
      }
    }
  }
  float old = 0.f;
  if (scale && first > 0) old = *scale;
  most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
  if (lane == 0) warp_most[warp] = most;
  __syncthreads();
  if (!scale) return;
  for (int k = 0; k < wpt; ++k) most = fmaxf(most, warp_most[team * wpt + k]);
  const bool keeps = old >= FLT_MIN && old <= FLT_MAX;
  int k = most > 0.f ? growth(most, keeps ? old : 1.f) : -118;
  k = max(k, keeps ? 0 : -118);
  const float now = ldexpf(keeps ? old : 1.f, k), inv = 1.f / now;
  if (w == 0 && lane == 0) *scale = now;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = place0 + u * RPI;
    uint8_t* row = to + i * a.c_st;
    if (fresh_token[u]) {
      *reinterpret_cast<uint2*>(row + 8 * cp.c0) = e4m3x8(f[u][0], inv);
      *reinterpret_cast<uint2*>(row + 8 * cp.c1) = e4m3x8(f[u][1], inv);
    } else if (i < first && keeps && k > 0) {
      const float by = ldexpf(1.f, -k);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint2* at = reinterpret_cast<uint2*>(row + 8 * (c ? cp.c1 : cp.c0));
        *at = e4m3x8_scaled(*at, by);
      }
    }
  }
}

template <int D, bool F16, int THREADS>
__global__ void __launch_bounds__(THREADS) append_8bit_kernel(RotaryArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0) check_offsets(a.cu, a.B, a.T, a.status);
  if (blockIdx.x < a.blocks8) {
    append_block<D, F16>(a, blockIdx.x);
  } else {
    const long long w = (blockIdx.x - a.blocks8) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int t = (int)(w / a.splits), split = (int)(w - (long long)t * a.splits);
    if (w < (long long)a.T * a.splits) rotate_rows<D, F16, false>(a, t, split, a.splits);
  }
}

template <int D, bool F16>
static int launch_rotary_d(RotaryArgs a, cudaStream_t stream) {
  int sms = 0;
  if (!sm_count(&sms)) return FA_ERR_CUDA;
  constexpr int RPI = 512 / D;
  const bool eight = a.ks != nullptr;
  const int jobs = (a.q ? a.Hq : 0) + (eight ? 0 : a.Hkv * (a.kc ? 2 : 1));
  // a warp for each token, or more of them while that leaves the SMs idle: 16 warps each
  const int most = std::max(1, (jobs + RPI - 1) / RPI);
  a.splits = (int)std::min<long long>(most, std::max<long long>(1, 16LL * sms / a.T));
  const long long warps = (long long)a.T * a.splits;
  if (!eight) {
    const long long grid = (warps + 3) / 4;
    if (grid > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
    return launch_pdl("rotary_rows_kernel", rotary_rows_kernel<D, F16>, dim3((unsigned)grid), dim3(128), 0, stream, a);
  }
  const int wpt = (D << a.block_shift) / 1024, threads = 32 * std::max(8, wpt), teams = std::max(1, 8 / wpt);
  a.head_groups = (2 * a.Hkv + teams - 1) / teams;
  a.blocks8 = (((long long)a.T >> a.block_shift) + 2LL * a.B) * a.head_groups;
  const long long grid = a.blocks8 + (a.q ? (warps + threads / 32 - 1) / (threads / 32) : 0);
  if (grid > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const auto kernel = threads <= 256 ? append_8bit_kernel<D, F16, 256>
                                     : threads <= 512 ? append_8bit_kernel<D, F16, 512> : append_8bit_kernel<D, F16, 1024>;
  return launch_pdl("append_8bit_kernel", kernel, dim3((unsigned)grid), dim3(threads), 0, stream, a);
}

static int launch_rotary(const RotaryArgs& a, int d, int dtype, cudaStream_t stream) {
  const bool f16 = dtype == FA_FP16;
  if (d == 64) return f16 ? launch_rotary_d<64, true>(a, stream) : launch_rotary_d<64, false>(a, stream);
  return f16 ? launch_rotary_d<128, true>(a, stream) : launch_rotary_d<128, false>(a, stream);
}

}  // namespace fa

namespace {

using namespace fa::host;

void take_cache(const fa_pages* c, const fa_scales* s, fa::RotaryArgs* a) {
  a->kc = static_cast<uint8_t*>(c->k), a->vc = static_cast<uint8_t*>(c->v);
  a->c_sp = c->page_stride, a->c_sh = c->head_stride, a->c_st = c->token_stride;
  a->n_pages = c->n_pages, a->page_shift = log2_of(c->page_size);
  a->table = c->table, a->table_stride = c->table_stride, a->table_width = c->table_width;
  if (s) {
    a->ks = s->k, a->vs = s->v;
    a->s_sp = s->page_stride, a->s_sh = s->head_stride;
    a->block_shift = log2_of(s->block);
  }
}

int check_rotary(const fa_rotary* r, int d) {
  if (!r || !r->angles) return FA_ERR_INVALID_ARG;
  if (!aligned16(r->angles)) return FA_ERR_MISALIGNED;
  if (r->positions < 1 || (r->interleaved != 0 && r->interleaved != 1)) return FA_ERR_INVALID_ARG;
  if (r->dim < 16 || r->dim > d || r->dim % 16 != 0) return FA_ERR_INVALID_ARG;
  if (r->row_stride < r->dim || r->row_stride % 4 != 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

extern "C" {

int fa_cache_append_8bit(const fa_rows* k, const fa_rows* v, const fa_pages* cache, const fa_scales* scales,
                         const int32_t* start, const int32_t* cu, const int32_t* rows, int B, int T, int Tkv, int Hkv, int d,
                         int dtype, fa_stream_t stream) {
  int rc = check_sizes(B, T, Hkv, Hkv, d, dtype, 1.f);
  if (rc != FA_OK) return rc;
  if (Tkv < 0 || (!rows && T != Tkv)) return FA_ERR_INVALID_ARG;
  if (Tkv > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if (Tkv == 0 || !start || !cu) return FA_ERR_INVALID_ARG;  // (rows of nothing)
  for (const fa_rows* r : {k, v})
    if ((rc = check_rows(r)) != FA_OK) return rc;
  if ((rc = check_pages(cache, 16)) != FA_OK || (rc = check_scales(scales, cache->page_size)) != FA_OK) return rc;
  fa::RotaryArgs a = {};
  a.k = static_cast<const uint16_t*>(k->data), a.v = static_cast<const uint16_t*>(v->data);
  a.k_st = k->token_stride, a.k_sh = k->head_stride, a.v_st = v->token_stride, a.v_sh = v->head_stride;
  take_cache(cache, scales, &a);
  a.start = start, a.cu = cu, a.rows = rows;
  a.B = B, a.T = T, a.Tkv = Tkv, a.Hkv = Hkv;
  int err = FA_OK;
  a.status = fa::status_word(&err);
  if (!a.status) return err;
  return fa::launch_rotary(a, d, dtype, reinterpret_cast<cudaStream_t>(stream));
}

int fa_rotary_append(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* q_out, const fa_rows* k_out,
                     const fa_pages* cache, const fa_scales* scales, const fa_rotary* rotary, const int32_t* start,
                     const int32_t* cu, int B, int T, int Hq, int Hkv, int d, int dtype, fa_stream_t stream) {
  if ((q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
  int rc = check_sizes(B, T, q ? Hq : Hkv, Hkv, d, dtype, 1.f);
  if (rc != FA_OK) return rc;
  if (T == 0 || ((cache || cu) && B == 0)) return FA_OK;
  if ((rc = check_rotary(rotary, d)) != FA_OK) return rc;
  for (const fa_rows* r : {q, q_out, k_out})
    if (r && (rc = check_rows(r)) != FA_OK) return rc;
  if ((rc = check_rows(k)) != FA_OK) return rc;
  if (cache) {
    if (!start || !cu) return FA_ERR_INVALID_ARG;
    if ((rc = check_rows(v)) != FA_OK || (rc = check_pages(cache, scales ? 16 : 8)) != FA_OK) return rc;
    if (scales && (rc = check_scales(scales, cache->page_size)) != FA_OK) return rc;
  } else if (!rotary->at || (!q && !k_out)) {
    return FA_ERR_INVALID_ARG;
  }
  fa::RotaryArgs a = {};
  a.k = static_cast<const uint16_t*>(k->data), a.k_st = k->token_stride, a.k_sh = k->head_stride;
  if (q) {
    a.q = static_cast<const uint16_t*>(q->data), a.q_st = q->token_stride, a.q_sh = q->head_stride;
    a.qo = static_cast<uint16_t*>(q_out->data), a.qo_st = q_out->token_stride, a.qo_sh = q_out->head_stride;
  }
  if (k_out) a.ko = static_cast<uint16_t*>(k_out->data), a.ko_st = k_out->token_stride, a.ko_sh = k_out->head_stride;
  if (cache) {
    a.v = static_cast<const uint16_t*>(v->data), a.v_st = v->token_stride, a.v_sh = v->head_stride;
    take_cache(cache, scales, &a);
    a.start = start;
  }
  a.angles = rotary->angles, a.a_stride = rotary->row_stride, a.positions = rotary->positions;
  a.dim = rotary->dim, a.interleaved = rotary->interleaved, a.at = rotary->at;
  a.cu = cu;
  a.B = B, a.T = T, a.Tkv = T, a.Hq = Hq, a.Hkv = Hkv;
  int err = FA_OK;
  a.status = fa::status_word(&err);
  if (!a.status) return err;
  return fa::launch_rotary(a, d, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
