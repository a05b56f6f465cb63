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
#ifdef FA_DEBUG
  int dbg_B;           // batch count B, for the extents the debug build checks against
  int dbg_slack;       // rows taken off those extents (fa_debug_set_check_slack)
#endif
};

// ---------------------------------------------------------------------------------------------
// A thread holds two chunks of 8 elements of a head row, chosen so that a rotation's pairs lie in one thread: with
// halves, chunks p and p + dim / 16; behind the rotated part, the chunks of a row's two halves there. So the lanes of a
// row load and store whole sectors.
struct ChunkPair {
  int c0, c1;
  bool turned;
};
template <int LPR>  // lanes a row
__device__ __forceinline__ ChunkPair chunk_pair(int p, int dim) {
  const int pairs = dim >> 4;
  ChunkPair c;
  c.turned = p < pairs;
  c.c0 = c.turned ? p : pairs + p;
  c.c1 = c.turned ? p + pairs : LPR + p;
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
__device__ __forceinline__ void load_turn(const RotaryArgs& a, const float* row, const ChunkPair& cp, Turn* t) {
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
  if (b < 0 || !FA_CHECK(in_range(t, (long long)a.T - FA_SLACK(a)), a.status, DBG_GLOBAL_LOAD)) return;
  const long long pos = (a.kc ? (long long)a.start[b] : 0) + i;
  const long long place = a.at ? a.at[t] : pos;
  if (place < 0 || place >= a.positions) return record_check(a.status, SITE_S_ANGLE);
  const ChunkPair cp = chunk_pair<LPR>(p, a.dim);
  Turn tn;
  if (cp.turned) load_turn(a, a.angles + place * a.a_stride, cp, &tn);
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
  constexpr int U = KV ? 4 : 2;
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
// The least k >= -118 with most <= 448 2^k, and 2^i for i in [-126, 127].
__device__ __forceinline__ int growth_of_new(float most) {
  const uint32_t u = __float_as_uint(most);
  return max((int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), -118);
}
__device__ __forceinline__ float pow2(int i) { return __uint_as_float((uint32_t)(i + 127) << 23); }
// A block's scale, its reciprocal, and what multiplies the tokens that were there (1: they stay as they are).
struct Rescale {
  float now, inv, by;
};
// A kept scale that is no power of two: not this library's.
__device__ __noinline__ Rescale rescale_any(float old, float most) {
  const int k = most > 0.f ? max(growth(most, old), 0) : 0;
  const float now = ldexpf(old, k);
  return {now, 1.f / now, ldexpf(1.f, -k)};
}
// From the scale as it was (0, as any value that is no scale: none) and the largest magnitude of the new tokens.
__device__ __forceinline__ Rescale rescale(float old, float most) {
  const uint32_t u = __float_as_uint(old);
  const int k = growth_of_new(most);
  if (!(old >= FLT_MIN && old <= FLT_MAX)) return {pow2(k), pow2(-k), 1.f};
  const int e = (int)(u >> 23) - 127;
  if ((u & 0x7fffffu) || e < -118 || e > 120) return rescale_any(old, most);
  const int now = max(e, k);
  return {pow2(now), pow2(-now), pow2(max(e - now, -126))};  // (2^-126 already leaves nothing of an 8-bit value)
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Eight values times inv.
__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
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

// Into 8 bits: a block's share of the heads ("jobs"), of K or of V, by a team of warps each, one after the other. A thread
// holds U pairs of chunks, in registers from the load to the store, so that the block's largest magnitude is known before
// anything is rounded.
//  - TEAM: block x D / (512 U) warps, all of the block at once: every row is read once. A CTA has as many teams as fit
//    (one, where the block is large); the next job's rows are on their way while the last one's are rounded, and
//    finding the sequence and the page, four loads in turn, is done once for all of them.
//  - otherwise, where few tokens a sequence are appended: a warp, which goes over those parts of the block that
//    have new tokens, twice where these are several (a CTA for each job, most of its threads idle: 64 sequences'
//    next tokens took 11.7 us instead of 4.1).
template <int D, bool F16, bool TEAM, int U>
__device__ __forceinline__ void append_block(const RotaryArgs& a, long long unit) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, TOKENS = U * RPI;  // lanes a row, rows at a time, tokens of a warp's part
  __shared__ float warp_most[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wpt = TEAM ? max(1, (D << a.block_shift) / (512 * U)) : 1, teams = (blockDim.x >> 5) / wpt;
  const int team = warp / wpt, w = warp - team * wpt;
  const long long slot = unit / a.head_groups;
  const int share = (int)(unit - slot * a.head_groups);
  const bool is_v = share & 1;
  const int b = find_block(a, slot);
  if (b < 0) return;
  const SeqRange r = seq_range(a.cu, b, a.T, a.status);
  const long long start = a.start[b], end = start + (r.hi - r.lo);
  const int block = 1 << a.block_shift;
  const long long base = ((start >> a.block_shift) + (slot - ((a.cu[b] >> a.block_shift) + 2LL * b))) << a.block_shift;
  if (r.hi <= r.lo || base >= end) return;
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
  const bool puts = !is_v && a.ko, turns = !is_v && a.angles;
  if (id < 0 && !puts) return;
  const int in_page = (int)(base & ((1 << a.page_shift) - 1));
  const int first = (int)max(0LL, start - base), last = (int)min((long long)block, end - base);  // the block's new tokens
  const ChunkPair cp = chunk_pair<LPR>(lane % LPR, is_v ? 0 : a.dim);
  // (debug build) row i of the block, of head h: inside the page, and the page inside the cache
  [[maybe_unused]] auto in_cache = [&](int h, int i) {
    return in_range(h, a.Hkv) && in_range(id, a.n_pages) && in_range(i, block) && in_range(in_page + i, 1LL << a.page_shift);
  };
  uint8_t* const pages = (is_v ? a.vc : a.kc) + id * a.c_sp + in_page * a.c_st;
  float* const scales = (is_v ? a.vs : a.ks) + id * a.s_sp + (in_page >> a.block_shift);
  const long long row_sh = is_v ? a.v_sh : a.k_sh;
  // part `sub`: the thread's rows in head 0 (null: none), their angles, and where the rotated keys go
  const uint16_t* from[U];
  const float* angle[U];
  uint16_t* ko[U];
  auto find_rows = [&](int sub) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = sub * TOKENS + u * RPI + lane / LPR;
      from[u] = nullptr;
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
        angle[u] = a.angles + p * a.a_stride;
      }
      if (!FA_CHECK(in_range(row, (long long)a.Tkv - FA_SLACK(a)) && in_range(t, a.T), a.status, DBG_GLOBAL_LOAD)) continue;
      from[u] = is_v ? a.v + row * a.v_st : a.k + row * a.k_st;
      if (puts) ko[u] = a.ko + t * a.ko_st;
    }
  };
  auto load = [&](int h, uint4 (&to)[U][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!from[u] || !FA_CHECK(in_range(h, a.Hkv), a.status, DBG_GLOBAL_LOAD)) continue;
      const uint16_t* row = from[u] + h * row_sh;
      to[u][0] = *reinterpret_cast<const uint4*>(row + 8 * cp.c0);
      to[u][1] = *reinterpret_cast<const uint4*>(row + 8 * cp.c1);
    }
  };
  // The values of loaded rows, and the largest finite magnitude of the warp's part; the rotated keys go out (put).
  float f[U][2][8];
  auto values = [&](int h, const uint4 (&x)[U][2], bool put) {
    float most = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!from[u]) continue;
      unpack8<F16>(x[u][0], f[u][0]);
      unpack8<F16>(x[u][1], f[u][1]);
      if (turns && cp.turned) {
        Turn tn;
        load_turn(a, angle[u], cp, &tn);
        turn(f[u][0], f[u][1], tn, a.interleaved);
      }
      if (put && puts) {
        uint16_t* row = ko[u] + h * a.ko_sh;
        *reinterpret_cast<uint4*>(row + 8 * cp.c0) = pack8<F16>(f[u][0]);
        *reinterpret_cast<uint4*>(row + 8 * cp.c1) = pack8<F16>(f[u][1]);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(f[u][e >> 3][e & 7]));  // (a NaN is never the larger one)
    }
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    if (most > FLT_MAX) {  // rare: infinities would saturate, and become NaN, as the type has none
      most = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!from[u]) continue;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float& x = f[u][e >> 3][e & 7];
          if (fabsf(x) > FLT_MAX) x = NAN;
          most = fmaxf(most, fabsf(x));
        }
      }
      most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    }
    return most;
  };
  auto scale_of = [&](int h) { return first > 0 && id >= 0 && FA_CHECK(in_cache(h, 0), a.status, DBG_GLOBAL_LOAD) ? scales[h * a.s_sh] : 0.f; };
  Rescale z;
  auto store = [&](int h, int sub) {
    uint8_t* to = pages + h * a.c_sh + (sub * TOKENS + lane / LPR) * a.c_st;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!from[u] || !FA_CHECK(in_cache(h, sub * TOKENS + u * RPI + lane / LPR), a.status, DBG_GLOBAL_STORE)) continue;
      uint8_t* at = to + u * RPI * a.c_st;
      *reinterpret_cast<uint2*>(at + 8 * cp.c0) = e4m3x8(f[u][0], z.inv);
      *reinterpret_cast<uint2*>(at + 8 * cp.c1) = e4m3x8(f[u][1], z.inv);
    }
  };
  auto restate = [&](int h, int sub) {  // the tokens that were there, as their scale grows
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = sub * TOKENS + u * RPI + lane / LPR;
      if (i >= first || !FA_CHECK(in_cache(h, i), a.status, DBG_GLOBAL_STORE)) continue;
      uint4* at = reinterpret_cast<uint4*>(pages + h * a.c_sh + i * a.c_st) + lane % LPR;
      const uint4 v = *at;
      const uint2 lo = e4m3x8_scaled(make_uint2(v.x, v.y), z.by), hi = e4m3x8_scaled(make_uint2(v.z, v.w), z.by);
      *at = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  };
  const int h0 = (share >> 1) * teams + team, step = (a.head_groups >> 1) * teams;
  if (TEAM) {
    find_rows(w);
    uint4 next[U][2];
    if (h0 < a.Hkv) load(h0, next);
    // (the same number of rounds for all teams of the CTA: they meet)
    for (int n = 0, h = h0; h - team < a.Hkv; ++n, h += step) {
      const bool mine = h < a.Hkv;
      float old = 0.f, most = 0.f;
      if (mine) {
        old = scale_of(h);
        most = values(h, next, true);
        if (h + step < a.Hkv) load(h + step, next);
      }
      if (lane == 0) warp_most[n & 1][warp] = most;
      __syncthreads();
      if (!mine || id < 0) continue;
      most = warp_most[n & 1][team * wpt + min(lane, wpt - 1)];
      z = rescale(old, __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most))));
      if (w == 0 && lane == 0 && FA_CHECK(in_cache(h, 0), a.status, DBG_GLOBAL_STORE)) scales[h * a.s_sh] = z.now;
      store(h, w);
      if (z.by < 1.f) restate(h, w);
    }
  } else {
    const int sub0 = first / TOKENS, sub1 = (last - 1) / TOKENS;
    const bool twice = sub0 != sub1;  // the rows are read again, so that the rotated keys, which may take their place, go out then
    uint4 x[U][2];
    for (int h = h0; h < a.Hkv; h += step) {
      const float old = scale_of(h);
      float most = 0.f;
      for (int pass = 0; pass < 2; ++pass) {
        for (int sub = sub0; sub <= sub1; ++sub) {
          if (pass == 0 || twice) {
            find_rows(sub);
            load(h, x);
            most = fmaxf(most, values(h, x, pass == (twice ? 1 : 0)));
          }
          if (pass == 1 && id >= 0) store(h, sub);
        }
        if (pass == 0) {
          if (id < 0 && !twice) break;
          z = rescale(old, most);
          __syncwarp();  // (every lane has read the scale)
          if (lane == 0 && id >= 0 && FA_CHECK(in_cache(h, 0), a.status, DBG_GLOBAL_STORE)) scales[h * a.s_sh] = z.now;
          for (int sub = 0; z.by < 1.f && sub * TOKENS < first; ++sub) restate(h, sub);
        }
      }
    }
  }
}

// U = 0: a warp a job. Two CTAs an SM where the registers allow it: what a round waits for (rows, the team's other warps)
// needs warps, and its instructions, some 300 a warp, are next to the bytes what a long append is bound by, with the
// barrier of all teams of a CTA in every round. 15019 prompt tokens of 8 heads (d = 128, blocks of 64): 28.5 us, of 13.6
// for the bytes; with 32 query heads turned too 69 of 55 (5.4 TB/s). One CTA an SM: 96 with the queries; threads of two
// rows, fewer warps: 78. 64 sequences' next tokens: 4.1 us in a graph (one CTA an SM 5.4, three 6.0).
// Registers: with two CTAs an SM a thread has 64 and spills 64 to 68 bytes; teams of 32 warps with two rows a thread
// (blocks of 256 at d = 128) spill 640 to 752. 8192 tokens of 8 heads take 15.5 us in blocks of 64, 16.9 of 128 and 25.7
// of 256 (at d = 64 9.0, 9.4 and 8.9), of 7.4 (3.7) for the bytes.
template <int D, bool F16, int U, int THREADS>
__global__ void __launch_bounds__(THREADS, U <= 1 ? 2 : 1) append_8bit_kernel(RotaryArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0) check_offsets(a.cu, a.B, a.T, a.status);
  if (blockIdx.x < a.blocks8) {
    append_block<D, F16, U != 0, U ? U : 2>(a, blockIdx.x);
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
  // a warp a job where few tokens a sequence come in, else teams, of which a CTA takes as many jobs in turn as make one
  // wave of two CTAs an SM
  const bool few = a.T <= 16LL * a.B;
  const int pairs = (D << a.block_shift) / 512;  // warps of a team with U = 1
  const int wpt = few ? 1 : pairs <= 16 ? pairs : pairs / 2, threads = 32 * std::max(few ? 8 : 16, wpt), teams = threads / 32 / wpt;
  const long long slots = ((long long)a.T >> a.block_shift) + 2LL * a.B;
  const int rounds = (a.Hkv + teams - 1) / teams;
  a.head_groups = 2 * (few ? rounds : (int)std::min<long long>(rounds, std::max<long long>(1, (long long)sms / slots)));
  a.blocks8 = slots * a.head_groups;
  const long long grid = a.blocks8 + (a.q ? (warps + threads / 32 - 1) / (threads / 32) : 0);
  if (grid > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  const auto kernel = few ? append_8bit_kernel<D, F16, 0, 256>
                          : pairs <= 16 ? append_8bit_kernel<D, F16, 1, 512>
                          : wpt <= 16 ? append_8bit_kernel<D, F16, 2, 512> : append_8bit_kernel<D, F16, 2, 1024>;
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
  FA_DEBUG_ARGS(a, B);
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
  FA_DEBUG_ARGS(a, B);
  int err = FA_OK;
  a.status = fa::status_word(&err);
  if (!a.status) return err;
  return fa::launch_rotary(a, d, dtype, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
