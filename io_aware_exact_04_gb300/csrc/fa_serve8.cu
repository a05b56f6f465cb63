// Attention of decoding and small drafts, few rows a sequence, over a cache in 8 bits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fa_internal.h"
#include "serve.cuh"
#include "serve_tree.h"
#include "tmap.h"

namespace fa {

// ---------------------------------------------------------------------------------------------
// Few rows against many keys: everything is transposed. S^T = K Q^T and O^T = V^T P^T have the keys, or
// the columns of V, as the 128 rows of the tensor core's tile and the query rows as its columns, so that
// decoding does not pay for 128 query rows, and K and V go from the pages through shared memory into the
// tensor core as they are, in 8 bits: no element of the cache is ever converted, which would cost more
// shared-memory traffic than the copy from memory itself.
//
// The other operand is split into 8-bit parts instead, which costs columns of a narrow tile:
//  - q, brought to [2^7, 2^8) by a power of two a row, is q1 + q2 / 16 (+ q3 / 16 in fp16), each the e4m3
//    nearest to what the ones before leave: 8 bits with two parts, all that bf16 has, 11 with three
//    (elements below 2^-10 of the row's largest keep bits down to 2^-21 of that one). q1 K and
//    (q2 + q3) K have columns of their own, as the factor 16 must stay outside.
//  - P, formed 2^11 times its value in fp16 (11 bits; below 2^-25 of the largest, steps of 2^-35 of it), is
//    p1 + p2 + (p3 + p4) / 64, each the e5m2 nearest to what is left (bf16 does without p4). As what is left
//    has a sign, three parts of three bits hold all 11, down to where e5m2, of 2^-16 to 2^15, ends: three parts are off
//    by 2^-21 at most below 2^-10, four by 2^-23 below 2^-12. With fp16's own 2^-25, and as P has up to one bit less
//    than 2^11 where vref is above the largest scale, that is 1.06 2^-31 and 1.25 2^-33 of the row's largest
//    probability (times that scale). (e4m3 would need as many parts and end at 2^-26.) Each has columns of O of
//    its own: one product of N = 3 R or 4 R columns takes 40 to 58 cycles, one of 16 takes 36. The reference
//    maximum moves when it grows by 2^4, so that P stays within 2^15.
//  - The scale of a key's block multiplies its scores, that of its values its probability, which is kept
//    in range by a reference of its own (vref, at least each scale that was met).
//
// The new tokens, in 16 bits, take the same way as tiles of 64 keys: kind::f16 products with Q and P in
// 16 bits, into columns of O of their own (vref = 1 there).
//
// Rows: a row is (token, head of the group), numbered token * G + head; a lane (four warps) has up to RV of
// them, 4, 8 or 16. A work item is 2 RV rows of a sequence and key/value head, RV for each of two lanes, over the same
// tiles of 128 keys; where there are RV rows or fewer both lanes take them and alternate tiles ("dual"),
// and join their results at the end. A kernel for each RV: one with all three has half as much code again, and what an
// item's start and end run through once then no longer stays near the SM (12 heads of 64, 128 contexts of 4096: 211 us,
// with rows in fours alone 171). All tiles of all items form one sequence, of which every CTA
// takes an equal run; items cut between CTAs leave fp32 partial results for serve8_join_kernel.
//
// Roles, 512 threads: warps 0-3 and 4-7 the softmax of lanes 0 and 1, a thread a key, warp 8 the scheduler,
// which loads the pages of K, 14 loads those of V and 15 the scales (one warp for all three took 1100 cycles
// a tile, more than memory does at d = 64), 9 issues S, 10 and 11 O, 12 and 13 split Q.
//
// The softmax needs a maximum over the keys, across its threads, only where a reference moves: for the
// first tile of an item, and where some score passes the reference by more than it may. A vote of the four
// warps says so, taken while P is formed as if nothing moved (with four warps in step, latency bounds a
// tile: a wait costs 100 to 200 cycles, also where its phase has completed). S has two buffers, so that the next one is
// formed meanwhile, and so has P. The layout has R = 16 rows a lane: the columns behind the
// first RV are never looked at, and what stands in them stays in them.
//
// Measured on one GB300: decoding 64 sequences over up to 8192 tokens, 32 heads over 8 of 128: 108 us, 86 % of the copy
// rate (32 of the same length, 8192: 92 us, 86 %; 2048: 34 us, 59 %); 128 over up to 5000, 12 heads of 64: 125 us, 63 %;
// two contexts of 131072, 32 heads over 4 of 128: 50 us, 66 %; drafts of up to 6 nodes over up to 8000, 40 heads over 8:
// 82 us, 45 %. A tile takes 0.70 us at d = 128 with 4 rows a lane, which is memory's time, and 0.44 at d = 64 (memory
// 0.37); with 30 rows, 15 in each lane, it takes 0.88: there the softmax bounds it. An item's start and end take 1.5 us at
// d = 128, 1.9 to 3.4 at d = 64 (256 and 512 sequences) and 5.8 with 30 rows, partly because code is fetched anew: the
// SM's instruction cache answers 94 % of the requests at d = 64, and the one behind it is busy 68 % of the time. The
// first and last 8 us of a call are a chain of loads, conversions and products that wait for each other.
template <int D, bool F16>
struct Serve8Cfg {
  static constexpr int R = 16;
  static constexpr int ROW = D;                      // bytes of a cached row
  static constexpr int KV = 128 * ROW, ENTRY = 2 * KV;
  static constexpr int NEW = 64;                     // keys of a tile of new tokens
  static constexpr int NSUB = D / 64;                // 64-column halves of their rows
  static constexpr int QPARTS = F16 ? 3 : 2;
  static constexpr int Q16 = QPARTS * R * D, QSLOT = Q16 + R * D * 2;
  static constexpr int NQ = 4;                       // slots of Q
  static constexpr int PPARTS = F16 ? 4 : 3;
  static constexpr int PX = 4 * R;                   // P: bytes of a key's row, [p1 | p2 | p3 | p4] of R bytes each; two buffers a lane
  static constexpr int PBYTES = 128 * PX;
  static constexpr int QROW = 16;                    // of a row of Q: factor of its scores, token, place in O (8 bytes)
  static constexpr int MISC = 512 + 256 + 12 * 64 + NQ * R * QROW + 2 * (2 * R + R + R + 4 * R + 4 * (R + 4)) * 4 + 64;
  static constexpr int FIXED = 4 * PBYTES + NQ * QSLOT + MISC;
  static constexpr int NT = (232448 - FIXED) / ENTRY < 12 ? (232448 - FIXED) / ENTRY : 12;
  static constexpr int OFF_P = NT * ENTRY, OFF_Q = OFF_P + 4 * PBYTES, OFF_BAR = OFF_Q + NQ * QSLOT;
  static constexpr int OFF_DESC = OFF_BAR + 512, OFF_SC = OFF_DESC + 256, OFF_QROW = OFF_SC + 12 * 64;
  // of each lane: factor of each row's scores and 11 - its reference, factors of a move; of the item before: reference,
  // sums of each warp
  static constexpr int OFF_ROWC = OFF_QROW + NQ * R * QROW, OFF_FAC = OFF_ROWC + 2 * R * 8, OFF_REF = OFF_FAC + 2 * R * 4;
  static constexpr int OFF_SUM = OFF_REF + 2 * R * 4, OFF_RED = OFF_SUM + 2 * 4 * R * 4;
  static constexpr int OFF_FLAG = OFF_RED + 2 * 4 * (R + 4) * 4, SMEM_BYTES = OFF_FLAG + 64;
  __device__ static constexpr uint32_t tm_s(int t, int u) { return 4u * R * t + 2u * R * u; }
  __device__ static constexpr uint32_t tm_o(int t) { return 8u * R + 4u * R * t; }
  __device__ static constexpr uint32_t tm_n(int t) { return 16u * R + R * t; }  // O of the new tokens
  static constexpr uint32_t TM_COLS = 512;
  static_assert(18 * R <= TM_COLS, "tensor memory");
  static constexpr int THREADS = 512, PRODUCER = 8, S_BOTH = 9, PV0 = 10, PV1 = 11, SPLIT = 12, LOAD_V = 14, SCALES = 15;
  // barriers
  static constexpr int FULL = 0, EMPTY = NT, Q_FULL = 2 * NT, Q_EMPTY = Q_FULL + NQ, S_FULL = Q_EMPTY + NQ, S_FREE = S_FULL + 4,
                       P_READY = S_FREE + 4, O_DONE = P_READY + 4, O_FREE = O_DONE + 4, MERGE = O_FREE + 2, DRAIN = MERGE + 1,
                       GROUP = DRAIN + 1, D_FULL = GROUP + 2, D_EMPTY = D_FULL + 4, BARS = D_EMPTY + 4;
  static_assert(8 * BARS + 12 <= 512, "barrier area");
  static_assert(NT >= 2 && SMEM_BYTES <= 232448, "shared memory");
  static_assert(OFF_P % 1024 == 0 && OFF_Q % 1024 == 0 && QSLOT % 1024 == 0 && Q16 % 1024 == 0 && OFF_BAR % 16 == 0, "alignment");
};

enum { SITE_T8_EMPTY = 80, SITE_T8_FULL, SITE_T8_Q_FULL, SITE_T8_Q_EMPTY, SITE_T8_S_FULL, SITE_T8_S_FREE, SITE_T8_P_READY,
       SITE_T8_O_DONE, SITE_T8_O_FREE, SITE_T8_MERGE, SITE_T8_DESC_FULL, SITE_T8_DESC_EMPTY, SITE_T8_V_FULL, SITE_T8_GROUP };

constexpr float kNoKey = -1e30f;     // reference maximum of a row that has met no key
constexpr float kPLog2 = 11.f, kLagLog2 = 4.f;
constexpr int kMinTiles8 = 2;        // tiles of a CTA where there are few
// An item's start and end cost a CTA as much as some tiles do (1.5 us and 0.70 a tile at d = 128, up to 3.4 and 0.44 at
// d = 64, partly beside the loads of the next one's): the runs are balanced with that many more for each. When drafts and
// decoding at d = 64 took 83 and 133 us with these, they took 88 and 138 with 4 and 8, 88 and 134 with 2 and 4, 84 and 138
// with 5 and 10.
template <int D>
constexpr int kItemTiles = D == 64 ? 5 : 3;
constexpr int kNewBox8 = 16;         // rows of a TMA box of new tokens

// A work item (or the part of it that this CTA computes), as the producer publishes it.
struct Item8 {
  int cnt;     // tiles here; -1: no more items
  int flags;   // 1: dual, 2: the whole item is here (results go straight to O)
  int c0, c1;  // tiles of lanes 0 and 1
  int j0;      // first tile, counted from the item's first
  int nc;      // tiles of cached tokens; tile j >= nc holds the new tokens from 64 (j - nc)
  int L, n;    // cached and new tokens of the sequence
  int row0;    // the sequence's first token among the packed ones
  int r0;      // the item's first row
  int kvh;
  int slot;    // partial result slot
  int b;       // the sequence
};
enum { ITEM8_DUAL = 1, ITEM8_WHOLE = 2 };

// Sizes of sequence b's work, in items of `unit` rows; record: whether invalid device values are recorded.
struct SeqWork8 {
  int row0, n, L, nc, nk, units;
  long long tiles;  // all heads and units, each counted with the nk tiles of the last one, and what an item costs
};
template <int D>
__device__ __forceinline__ SeqWork8 seq_work8(const Serve8BitArgs& a, int lo, int hi, int len, int unit, bool record) {
  SeqWork8 w;
  w.row0 = min(max(lo, 0), a.T);
  const int end = min(max(hi, w.row0), a.T);
  if (record && (w.row0 != lo || end != hi)) record_check(a.status, SITE_S_OFFSETS);
  w.n = end - w.row0;
  w.L = 0;
  if (w.n > 0) {
    w.L = min(max(len, 0), a.table_width << a.page_shift);
    if (record && w.L != len) record_check(a.status, SITE_S_LENGTH);
  }
  w.nc = (w.L + 127) >> 7;
  w.nk = w.nc + ((w.n + 63) >> 6);
  w.units = (w.n * a.G + unit - 1) / unit;
  w.tiles = (long long)w.units * a.Hkv * (w.nk + kItemTiles<D>);
  return w;
}
template <int D>
__device__ __forceinline__ SeqWork8 seq_work8(const Serve8BitArgs& a, int b, int unit, bool record) {
  return seq_work8<D>(a, a.cu[b], a.cu[b + 1], a.lens[b], unit, record);
}

// The run of tiles of CTA c, by a whole warp. Each lane counts the tiles of `chunk` sequences that follow
// each other, four sequences' loads at a time, so that a search looks at one lane's sequences only.
struct Runs8 {
  long long total, base;
  int ctas, rest;  // CTAs with work; the first `rest` of them take a tile more
  long long mine;  // this lane's tiles
  int chunk;
  __device__ long long start(int c) const { return base * c + min(c, rest); }
};
template <int D>
__device__ __forceinline__ Runs8 runs8(const Serve8BitArgs& a, int unit, int grid, bool record) {
  Runs8 r;
  const int lane = threadIdx.x & 31;
  r.chunk = (a.B + 31) >> 5;
  r.mine = 0;
  const int end = min(a.B, (lane + 1) * r.chunk);
  for (int b = lane * r.chunk; b < end; b += 4) {
    int at[5], len[4];
#pragma unroll
    for (int k = 0; k < 5; ++k) at[k] = a.cu[min(b + k, end)];
#pragma unroll
    for (int k = 0; k < 4; ++k) len[k] = a.lens[min(b + k, end - 1)];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (b + k < end) r.mine += seq_work8<D>(a, at[k], at[k + 1], len[k], unit, record).tiles;
  }
  r.total = r.mine;
  for (int o = 16; o; o >>= 1) r.total += __shfl_xor_sync(0xffffffffu, r.total, o);
  r.ctas = r.total < (long long)grid * kMinTiles8 ? max(1, ((int)r.total + kMinTiles8 - 1) / kMinTiles8) : grid;
  r.base = r.total < (1LL << 31) ? (int)r.total / r.ctas : r.total / r.ctas;
  r.rest = (int)(r.total - r.base * r.ctas);
  return r;
}
// The lane whose own tiles hold tile `pos` of all, and their first one; 32: past the end.
__device__ __forceinline__ int lane_with(long long mine, long long pos, long long* first) {
  const int lane = threadIdx.x & 31;
  long long incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  const unsigned past = __ballot_sync(0xffffffffu, *first + incl > pos);
  const int k = past ? __ffs(past) - 1 : 32;
  *first += __shfl_sync(0xffffffffu, k < 32 ? incl - mine : incl, k < 32 ? k : 31);
  return k;
}
// The sequence that tile `pos` of all belongs to, and its first tile; by a whole warp. pos < total.
template <int D>
__device__ __forceinline__ int seek8(const Serve8BitArgs& a, int unit, const Runs8& runs, long long pos, long long* first) {
  *first = 0;
  const int k = lane_with(runs.mine, pos, first);
  if (k == 32) return a.B;
  if (runs.chunk == 1) return k;
  const int end = min(a.B, (k + 1) * runs.chunk);
  for (int b0 = k * runs.chunk; b0 < end; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const int x = lane_with(b < end ? seq_work8<D>(a, b, unit, false).tiles : 0, pos, first);
    if (x < 32) return b0 + x;
  }
  return a.B;
}

// Tiles that the rows [r, r + R) of a sequence need, counted from the first.
__device__ __forceinline__ int tiles_of_rows(const Serve8BitArgs& a, const SeqWork8& w, int r, int R) {
  const int rows = w.n * a.G;
  if (r >= rows) return 0;
  if (a.mask || w.n <= 64) return w.nk;
  return w.nc + ((min(w.n, (min(r + R, rows) - 1) / a.G + 1) + 63) >> 6);
}

__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2_mul64(uint32_t a) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x54005400u));  // 64, 64
  return r;
}
// The two e5m2 nearest to two fp16, as fp16 with the low bytes zero: half a step up in the magnitude's
// bits, and the low bytes off (e5m2 is the upper byte of fp16; ties go away from zero).
__device__ __forceinline__ uint32_t to_e5m2(uint32_t x) { return (x + 0x00800080u) & 0xff00ff00u; }
// The upper bytes of four fp16.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7531); }
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t at, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t at, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
// The offset of 16-byte chunk c of row r in rows of PITCH (64 or 128) bytes, swizzled as TMA and the tensor
// core do: address bits 7 .. exchange with bits 4 ...
template <int PITCH>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  return PITCH == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}
template <int PITCH>
__host__ __device__ constexpr uint32_t desc_hi() {
  return PITCH == 128 ? sdesc_hi(1024) : sdesc_hi_sw64(512);
}
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void e4m3_floats(uint32_t x, float& lo, float& hi) {
  asm("{\n\t.reg .b32 t;\n\t.reg .b16 l, h;\n\tcvt.rn.f16x2.e4m3x2 t, %2;\n\tmov.b32 {l, h}, t;\n\t"
      "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "h"((uint16_t)x));
}
template <bool F16>
__device__ __forceinline__ void halves(uint32_t w, float& lo, float& hi) {
  if (F16) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
  } else {
    lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  }
}
// N columns of the warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "");
  if constexpr (N == 4)
    tmem_ld4(taddr, r);
  else if constexpr (N == 8)
    tmem_ld8(taddr, r);
  else
    tmem_ld16(taddr, r);
}
template <int N>
__device__ __forceinline__ void tmem_stn(uint32_t taddr, const uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16, "");
  if constexpr (N == 4)
    tmem_st4(taddr, r);
  else if constexpr (N == 8)
    tmem_st8(taddr, r);
  else
    tmem_st16(taddr, r);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

template <int D, bool F16, int RV>
__global__ void __launch_bounds__(512, 1)
    serve8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc, Serve8BitArgs a) {
  using C = Serve8Cfg<D, F16>;
  constexpr int R = C::R;
  constexpr int NT = C::NT, NQ = C::NQ;
  // 1024-byte aligned, as the swizzled tiles have to be: there is no room to round the address up
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sbase = smem_u32(sm);
  if (sbase & 1023u) {  // (never seen: the kernel has no static shared memory)
    griddep_wait();
    if (threadIdx.x == 0) {
      record_check(a.status, SITE_S_SMEM);
      a.cuts[2 * blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing for the join to read
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b0 = sbase + C::OFF_BAR;
  auto BAR = [&](int i) { return b0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + 8 * C::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  DevStatus st{a.status, abort_flag};
  int* descs = reinterpret_cast<int*>(sm + C::OFF_DESC);
  float* scales = reinterpret_cast<float*>(sm + C::OFF_SC);  // [entry][K of 8 groups of 16 keys, V of 8]
  struct __align__(16) QRow {
    float factor;  // of the row's scores, to base 2
    int tok;       // its token within the sequence; -1: no row
    long long to;  // head << 40 | packed token
  };
  QRow* qrows = reinterpret_cast<QRow*>(sm + C::OFF_QROW);  // [slot][row]

  if (warp == C::PRODUCER && lane == 0) {
    for (int i = 0; i < NT; ++i) {
      mbar_init(BAR(C::FULL + i), 10);  // K's and V's copies, and each of 8 lanes' scales
      mbar_init(BAR(C::EMPTY + i), 2);  // both issuers of P V, also of a tile that only one of them takes: neither may fall a use behind
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(BAR(C::Q_FULL + i), 2);
      mbar_init(BAR(C::Q_EMPTY + i), 9);  // the issuer of S, and both lanes' warps, also those whose rows are in the other slot
    }
    for (int t = 0; t < 2; ++t) {
      for (int u = 0; u < 2; ++u) {
        mbar_init(BAR(C::S_FULL + 2 * t + u), 1);
        mbar_init(BAR(C::S_FREE + 2 * t + u), 4);
        mbar_init(BAR(C::P_READY + 2 * t + u), 4);
        mbar_init(BAR(C::O_DONE + 2 * t + u), 1);
      }
      mbar_init(BAR(C::O_FREE + t), 8);  // four warps twice, or all eight in a join
      mbar_init(BAR(C::GROUP + t), 4);
    }
    mbar_init(BAR(C::MERGE), 8);
    mbar_init(BAR(C::DRAIN), 3);
    for (int i = 0; i < 4; ++i) {
      mbar_init(BAR(C::D_FULL + i), 1);
      mbar_init(BAR(C::D_EMPTY + i), 15);  // softmax warps, issuers, splitters, loaders
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_kc);
    prefetch_tmap(&tm_vc);
  }
  if (warp == C::PV0) {
    tmem_alloc(smem_u32(tmem_slot), C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // before any access to global memory
  griddep_launch_dependents();

  // Item i of this CTA, for a consumer warp: false when the CTA must give up.
  auto next_item = [&](int i, Item8* it) {
    if (!wait_phase(BAR(C::D_FULL + (i & 3)), (i >> 2) & 1, st, SITE_T8_DESC_FULL)) return false;
    const int4* d = reinterpret_cast<const int4*>(descs + 16 * (i & 3));
    const int4 x = d[0], y = d[1], z = d[2];
    it->b = reinterpret_cast<const int*>(d)[12];
    it->cnt = x.x, it->flags = x.y, it->c0 = x.z, it->c1 = x.w;
    it->j0 = y.x, it->nc = y.y, it->L = y.z, it->n = y.w;
    it->row0 = z.x, it->r0 = z.y, it->kvh = z.z, it->slot = z.w;
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(C::D_EMPTY + (i & 3)));
    return true;
  };
  auto rows_here = [&](const Item8& it, int j) {  // keys of tile j
    return j < it.nc ? min(128, it.L - j * 128) : min(C::NEW, it.n - (j - it.nc) * C::NEW);
  };

  // Loaders: an item's tiles, in the order of the ring. Lane 8 x + g looks after keys 16 g .. of the x-th of four
  // tiles, whose page ids are fetched four tiles ahead.
  const int page = 1 << a.page_shift, prow = min(page, 128), g8 = lane & 7, x8 = lane >> 3;
  auto page_ids = [&](const Item8& it, int k) {  // of the tiles k .. k + 3 of the item's part
    const int j = it.j0 + k + x8, t0 = j * 128 + g8 * 16;
    return j < min(it.j0 + it.cnt, it.nc) && t0 < it.L &&
                   FA_CHECK(in_range(it.b, a.B) && in_range(t0 >> a.page_shift, a.table_width), st, DBG_META) ? a.table[it.b * a.table_stride + (t0 >> a.page_shift)] : 0;
  };
  // K's (kv = 0) or V's copies of the item's tiles, the ring's entries from e on.
  auto load_tiles = [&](const Item8& it, int kv, int* e) {
    int id = 0, id_next = page_ids(it, 0), s = *e % NT;
    uint32_t phase = ((*e / NT) & 1) ^ 1;
    auto next = [&] {
      ++*e;
      if (++s == NT) s = 0, phase ^= 1;
    };
    for (int k = 0; k < it.cnt; ++k, next()) {
      if (!(k & 3)) id = id_next, id_next = page_ids(it, k + 4);
      const int j = it.j0 + k, rows = rows_here(it, j);
      const bool cached = j < it.nc;
      const uint32_t bar = BAR(C::FULL + s), dst0 = sbase + s * C::ENTRY + kv * C::KV;
      const int box = cached ? prow : kNewBox8, boxes = (rows + box - 1) / box;
      if (!wait_phase(BAR(C::EMPTY + s), phase, st, SITE_T8_EMPTY)) return false;
      if (elect_one()) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * (cached ? C::ROW : 2 * D)));
      __syncwarp();
      if (cached) {
        const int in_page = (j * 128 + g8 * 16) & (page - 1);
        const uint32_t dst = dst0 + g8 * 16 * C::ROW;
        if (x8 == (k & 3) && g8 * 16 < rows && (g8 * 16 & (prow - 1)) == 0 && !(kWithhold && *e == 1) &&
            FA_CHECK(smem_in(dst, prow * C::ROW, sbase, sbase + C::OFF_P), st, DBG_TMA_LOAD))
          tma_load_4d(dst, kv ? &tm_vc : &tm_kc, 0, in_page, it.kvh, id >= 0 && id < a.n_pages ? id : a.n_pages, bar);  // outside: zeros
      } else {
        const int r = lane / C::NSUB, c = lane % C::NSUB;
        const uint32_t dst = dst0 + c * (C::NEW * 128) + r * kNewBox8 * 128;
        if (r < boxes && !(kWithhold && *e == 1) && FA_CHECK(smem_in(dst, kNewBox8 * 128, sbase, sbase + C::OFF_P), st, DBG_TMA_LOAD))
          tma_load_3d(dst, kv ? &tm_v : &tm_k, c * 64, it.row0 + (j - it.nc) * C::NEW + r * kNewBox8, it.kvh, bar);
      }
      __syncwarp();
    }
    return true;
  };
  auto let_land = [&](int e) {  // copies in flight, before a CTA that gives up releases its shared memory
    if (!*(volatile int*)abort_flag) return;
    for (int x = max(0, e - NT); x < e; ++x) {
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(BAR(C::FULL + x % NT), (x / NT) & 1) && globaltimer_ns() - t0 < 100000000ull) {
      }
    }
  };

  if (warp == C::PRODUCER || warp == C::LOAD_V) {
    // ------------------------------------------------------------ scheduler and the loads of K; the loads of V
    // (one copy of the loads' code for both: drafts 86 -> 79 us, decoding at d = 64 133 -> 125)
    const int kv = warp == C::LOAD_V;
    int items = 0, e = 0;  // items published, ring entries used
    bool ok = true;
    auto publish = [&](const Item8& it) {
      if (!wait_phase(BAR(C::D_EMPTY + (items & 3)), ((items >> 2) & 1) ^ 1, st, SITE_T8_DESC_EMPTY)) return false;
      if (lane == 0) {
        int4* d = reinterpret_cast<int4*>(descs + 16 * (items & 3));
        d[0] = make_int4(it.cnt, it.flags, it.c0, it.c1);
        d[1] = make_int4(it.j0, it.nc, it.L, it.n);
        d[2] = make_int4(it.row0, it.r0, it.kvh, it.slot);
        reinterpret_cast<int*>(d)[12] = it.b;
        mbar_arrive(BAR(C::D_FULL + (items & 3)));
      }
      __syncwarp();
      ++items;
      return true;
    };
    constexpr int unit = 2 * RV;
    Runs8 runs = {};
    int parts = 0;  // of the item that this CTA is the first to cut
    int4 cut = make_int4(0, 0, 0, 0);
    long long pos = 0, end = 0, first = 0;  // the run's rest; the first tile of sequence b
    int b = 0, p = 0, kvh = 0, x0 = 0;      // the next item: its sequence, rows and head, and how much of it is others'
    bool met = false;                       // sequence b's sizes are known
    SeqWork8 w = {};
    if (!kv) {
      runs = runs8<D>(a, unit, gridDim.x, blockIdx.x == 0);
      if ((int)blockIdx.x < runs.ctas && runs.total > 0) {
        pos = runs.start(blockIdx.x), end = runs.start(blockIdx.x + 1);
        b = seek8<D>(a, unit, runs, pos, &first);
      }
    }
    // The CTA's next item with tiles.
    auto schedule = [&](Item8* it) {
      while (pos < end) {
        if (!met) w = seq_work8<D>(a, b, unit, false);
        const int span = w.nk + kItemTiles<D>;  // an item's share of the run: its costs, then its tiles
        if (!met) {
          // the first item may be cut; from then on they are met from their start
          const long long at = pos - first;
          const int q = at < (1LL << 31) ? (int)at / span : (int)(at / span);
          p = q / a.Hkv, kvh = q - p * a.Hkv, x0 = (int)(at - (long long)q * span);
          met = true;
        }
        if (pos - first >= w.tiles) {
          first += w.tiles;
          ++b;
          met = false;
          continue;
        }
        const int x1 = (int)min((long long)span, x0 + (end - pos));
        const int n0 = tiles_of_rows(a, w, p * unit, RV), n1 = tiles_of_rows(a, w, p * unit + RV, RV), most = max(n0, n1);
        const bool dual = n1 == 0;
        const int j0 = max(0, x0 - kItemTiles<D>), j1 = min(max(0, x1 - kItemTiles<D>), most);
        it->cnt = max(0, j1 - j0);
        it->flags = (dual ? ITEM8_DUAL : 0) | (j0 == 0 && j1 == most ? ITEM8_WHOLE : 0);
        it->c0 = dual ? (it->cnt + 1) >> 1 : max(0, min(j1, n0) - j0);
        it->c1 = dual ? it->cnt >> 1 : it->cnt;
        it->j0 = j0, it->nc = w.nc, it->L = w.L, it->n = w.n, it->row0 = w.row0, it->r0 = p * unit, it->kvh = kvh;
        it->slot = 2 * blockIdx.x + (j0 == 0);
        it->b = b;
        const long long tile0 = pos - x0 + kItemTiles<D>;  // the place of the item's first tile
        if (j0 > 0 && it->cnt > 0 && runs.start(blockIdx.x - 1) <= tile0) {
          // (the first item only) how many CTAs, this one included, hold later parts of it
          const long long end_of_item = tile0 + most;
          for (int k = blockIdx.x + lane; __any_sync(0xffffffffu, k < runs.ctas); k += 32)
            parts += __popc(__ballot_sync(0xffffffffu, k < runs.ctas && runs.start(k) < end_of_item));
          cut = make_int4(it->n * a.G, it->row0, it->r0, it->kvh);
        }
        pos += x1 - x0;
        x0 = 0;
        if (++kvh == a.Hkv) kvh = 0, ++p;
        if (it->cnt > 0) return true;
      }
      return false;
    };
    for (int i = 0; ok; ++i) {
      Item8 it;
      if (kv) {
        if (!next_item(i, &it) || it.cnt < 0) break;
      } else {
        if (!schedule(&it)) break;
        if (!(ok = publish(it))) break;
      }
      ok = load_tiles(it, kv, &e);
    }
    if (!kv) {
      if (lane == 0) {
        a.cuts[2 * blockIdx.x] = make_int4(parts, 0, 0, 0);
        a.cuts[2 * blockIdx.x + 1] = cut;
      }
      if (ok) {
        Item8 it = {};
        it.cnt = -1;
        publish(it);
      }
    }
    let_land(e);
  } else if (warp == C::SCALES) {
    // ------------------------------------------------------------ the loads of the scales
    int e = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      Item8 it;
      if (!next_item(i, &it) || it.cnt < 0) break;
      int id = 0, id_next = page_ids(it, 0);
      for (int k = 0; k < it.cnt; ++k, ++e) {
        if (!(k & 3)) id = id_next, id_next = page_ids(it, k + 4);
        const int j = it.j0 + k, s = e % NT;
        const uint32_t bar = BAR(C::FULL + s);
        if (!(ok = wait_phase(BAR(C::EMPTY + s), ((e / NT) & 1) ^ 1, st, SITE_T8_EMPTY))) break;
        if (j >= it.nc) {
          if (lane == 0) mbar_arrive_n(bar, 8);
        } else if (x8 == (k & 3)) {
          const int t0 = j * 128 + g8 * 16;
          const bool mine = t0 < it.L, there = id >= 0 && id < a.n_pages;
          if (mine && !there) record_check(a.status, SITE_S_PAGE);
          float* to = scales + s * 16 + g8;
          if (mine && there && FA_CHECK(in_range(it.kvh, a.Hkv), st, DBG_GLOBAL_LOAD)) {
            const long long from = id * a.s_sp + it.kvh * a.s_sh + ((t0 & (page - 1)) >> a.block_shift);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(a.ks + from) : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to + 8)), "l"(a.vs + from) : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
          } else {
            to[0] = to[8] = 1.f;
            mbar_arrive(bar);
          }
        }
        __syncwarp();
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= C::SPLIT) {
    // ------------------------------------------------------------ Q in parts
    constexpr int LPR = D / 8, RPI = 32 / LPR, MINE = RV / 2, STEPS = (MINE + RPI - 1) / RPI;  // lanes a row, rows and steps of a warp
    const int half = warp - C::SPLIT, sub = lane / LPR, c = lane % LPR;
    int uq = 0;
    for (int i = 0;; ++i) {
      Item8 it;
      if (!next_item(i, &it) || it.cnt < 0) break;
      const int nq = (it.flags & ITEM8_DUAL) ? 1 : 2, rows = it.n * a.G;
      bool ok = true;
      for (int t = 0; ok && t < nq; ++t, ++uq) {
        const int s = uq % NQ;
        uint4 x[STEPS];
        int toks[STEPS];
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
          const int rr = it.r0 + t * RV + half * MINE + k * RPI + sub, tok = rr / a.G;
          toks[k] = tok;
          x[k] = make_uint4(0, 0, 0, 0);
          if (k * RPI + sub < MINE && rr < rows && FA_CHECK(in_range(it.row0 + tok, a.T - FA_SLACK(a)), st, DBG_GLOBAL_LOAD))
            x[k] = *reinterpret_cast<const uint4*>(a.q + (long long)(it.row0 + tok) * a.q_st +
                                                   (long long)(it.kvh * a.G + rr - tok * a.G) * a.q_sh + 8 * c);
        }
        if (!(ok = wait_phase(BAR(C::Q_EMPTY + s), ((uq / NQ) & 1) ^ 1, st, SITE_T8_Q_EMPTY))) break;
        const uint32_t q8 = sbase + C::OFF_Q + s * C::QSLOT, q16 = q8 + C::Q16;
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
          const uint32_t r = half * MINE + k * RPI + sub;
          const bool mine = k * RPI + sub < MINE;
          if (mine) sts128(q16 + (c >> 3) * (R * 128) + swizzled<128>(r, c & 7), x[k].x, x[k].y, x[k].z, x[k].w);
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
          float f[8], most = 0.f;
#pragma unroll
          for (int y = 0; y < 4; ++y) halves<F16>(w[y], f[2 * y], f[2 * y + 1]);
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            // infinities count as NaN: the parts have none
            if (!(fabsf(f[y]) <= 3.4028235e38f)) f[y] = NAN;
            most = fmaxf(most, fabsf(f[y]));
          }
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          // most 2^-x in [2^7, 2^8)
          const int x2 = max((int)(__float_as_uint(most) >> 23) - 127, -100) - 7;
          const float down = __uint_as_float((uint32_t)(127 - x2) << 23), up = __uint_as_float((uint32_t)(127 + x2) << 23);
          uint32_t part[3][4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float lo = f[2 * y] * down, hi = f[2 * y + 1] * down, bl, bh;
            part[0][y] = e4m3_pair(lo, hi);
            e4m3_floats(part[0][y], bl, bh);
            lo = (lo - bl) * 16.f, hi = (hi - bh) * 16.f;
            part[1][y] = e4m3_pair(lo, hi);
            e4m3_floats(part[1][y], bl, bh);
            part[2][y] = e4m3_pair(lo - bl, hi - bh);
          }
#pragma unroll
          for (int z = 0; z < C::QPARTS; ++z)
            if (mine) sts64(q8 + swizzled<C::ROW>(z * R + r, c >> 1) + (c & 1) * 8, part[z][0] | part[z][1] << 16,
                  part[z][2] | part[z][3] << 16);
          if (c == 0 && mine) {
            const int rr = it.r0 + t * RV + r, tok = toks[k];
            QRow* to = qrows + s * R + r;
            to->factor = rr < rows ? up * a.scale_log2 : 0.f;
            to->tok = rr < rows ? tok : -1;
            to->to = (long long)(it.kvh * a.G + rr - tok * a.G) << 40 | (long long)(it.row0 + tok);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::Q_FULL + s));
      }
      if (!ok) break;
    }
  } else if (warp >= C::S_BOTH) {
    // ------------------------------------------------------------ MMA issuers
    auto commit = [&](uint32_t bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    bool ok = true;
    int e = 0;
    if (warp == C::S_BOTH) {
      // S^T = K Q^T of both lanes, tile after tile in the order of the ring. One copy of the code for both lanes, and loops
      // for the products of new tokens: less code to fetch anew at an item (decoding at d = 64 139 -> 133 us).
      constexpr uint32_t I8 = idesc_e4m3_f32(128, 2 * R, 0, 0), I8X = idesc_e4m3_f32(128, R, 0, 0);
      constexpr uint32_t I16 = F16 ? idesc_f16_f32(128, R, 0, 0) : idesc_bf16_f32(128, R, 0, 0);
      constexpr uint32_t HI = desc_hi<C::ROW>(), HI16 = sdesc_hi(1024);
      const uint32_t ring_lo = sdesc_lo(sbase, 16), q_lo = sdesc_lo(sbase + C::OFF_Q, 16);
      int uq = 0, used0 = 0, used1 = 0;
      for (int i = 0; ok; ++i) {
        Item8 it;
        if (!next_item(i, &it) || it.cnt < 0) break;
        const bool dual = it.flags & ITEM8_DUAL;
        const int nq = dual ? 1 : 2;
        const int slot0 = uq % NQ, slot1 = (uq + 1) % NQ;
        for (int u = uq; ok && u < uq + nq; ++u)
          ok = wait_phase(BAR(C::Q_FULL + u % NQ), (u / NQ) & 1, st, SITE_T8_Q_FULL);
        for (int k = 0; ok && k < it.cnt; ++k, ++e) {
          const int j = it.j0 + k, s = e % NT;
          if (!(ok = wait_phase(BAR(C::FULL + s), (e / NT) & 1, st, SITE_T8_FULL))) break;
          const uint32_t ka = ring_lo + s * (C::ENTRY >> 4);
#pragma unroll 1
          for (int t = dual ? k & 1 : k >= it.c0; t < 2; t += dual ? 2 : 1) {
            const int g = t ? used1++ : used0++, u = g & 1;
            // S of two tiles before is in registers
            if (g > 1 && !(ok = wait_phase(BAR(C::S_FREE + 2 * t + u), ((g >> 1) - 1) & 1, st, SITE_T8_S_FREE))) break;
            tc_fence_after();
            const uint32_t d = tmem + C::tm_s(t, u), qb = q_lo + (t && !dual ? slot1 : slot0) * (C::QSLOT >> 4);
            if (elect_one()) {
              if (j < it.nc) {
#pragma unroll
                for (int x = 0; x < D / 32; ++x) mma8_ss(d, sdesc_join(ka + 2 * x, HI), sdesc_join(qb + 2 * x, HI), I8, x > 0);
                if (F16) {
#pragma unroll
                  for (int x = 0; x < D / 32; ++x)
                    mma8_ss(d + R, sdesc_join(ka + 2 * x, HI), sdesc_join(qb + (2 * R * D >> 4) + 2 * x, HI), I8X, 1);
                }
              } else {
#pragma unroll 1
                for (int x = 0; x < D / 16; ++x) {
                  const uint32_t ko = ((x >> 2) * (C::NEW * 128) + (x & 3) * 32) >> 4;
                  const uint32_t qo = (C::Q16 + (x >> 2) * (R * 128) + (x & 3) * 32) >> 4;
                  mma_ss(d, sdesc_join(ka + ko, HI16), sdesc_join(qb + qo, HI16), I16, x > 0);
                }
              }
              mma_commit(BAR(C::S_FULL + 2 * t + u));
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        for (int u = uq; u < uq + nq; ++u) commit(BAR(C::Q_EMPTY + u % NQ));
        uq += nq;
      }
    } else {
      // O^T += V^T P^T of lane t
      const int t = warp == C::PV1;
      constexpr uint32_t I8 = idesc_e4m3_f32(128, C::PPARTS * R, 1, 1) | 1u << 16;
      constexpr uint32_t I16 = F16 ? idesc_f16_f32(128, R, 1, 1) : idesc_bf16_f32(128, R, 1, 1);
      constexpr uint32_t HIV = desc_hi<C::ROW>(), HIP = desc_hi<C::PX>(), HI16 = sdesc_hi(1024);
      const uint32_t d = tmem + C::tm_o(t), p_lo = sdesc_lo(sbase + C::OFF_P + t * 2 * C::PBYTES, 8192);
      const uint32_t v_lo = sdesc_lo(sbase + C::KV, 8192);
      int g = 0, items = 0;
      for (int i = 0; ok; ++i) {
        Item8 it;
        if (!next_item(i, &it) || it.cnt < 0) break;
        const bool dual = it.flags & ITEM8_DUAL;
        const int tiles = t ? it.c1 : it.c0;
        bool first = true, first_new = true;
        for (int k = 0; ok && k < it.cnt; ++k, ++e) {
          const int s = e % NT;
          // waited for also where the other lane's, and let go by both: the arrival must not count for an earlier use, and
          // a parity tells two uses of the slot apart, not three
          if (!(ok = wait_phase(BAR(C::FULL + s), (e / NT) & 1, st, SITE_T8_V_FULL))) break;
          if (dual ? (k & 1) != t : k >= tiles) {
            if (elect_one()) mbar_arrive(BAR(C::EMPTY + s));
            __syncwarp();
            continue;
          }
          const int j = it.j0 + k, rows = rows_here(it, j);
          const bool cached = j < it.nc;
          if (rows < (cached ? 128 : C::NEW)) {
            // rows past the sequence may hold anything; P is 0 there, but 0 x NaN is not
            uint8_t* v = sm + s * C::ENTRY + C::KV;
            const int pitch = cached ? C::ROW : 128, end = (cached ? 128 : C::NEW) * pitch;
#pragma unroll 1
            for (int at = rows * pitch + lane * 16; at < end; at += 512) {
              *reinterpret_cast<uint4*>(v + at) = make_uint4(0, 0, 0, 0);
              if (D == 128 && !cached) *reinterpret_cast<uint4*>(v + C::NEW * 128 + at) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (!(ok = wait_phase(BAR(C::P_READY + 2 * t + (g & 1)), (g >> 1) & 1, st, SITE_T8_P_READY))) break;
          if (first && items > 0 && !(ok = wait_phase(BAR(C::O_FREE + t), (items - 1) & 1, st, SITE_T8_O_FREE))) break;
          tc_fence_after();
          const uint32_t va = v_lo + s * (C::ENTRY >> 4), pa = p_lo + (g & 1) * (C::PBYTES >> 4);
          if (elect_one()) {
            if (cached) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                mma8_ss(d, sdesc_join(va + x * (32 * C::ROW >> 4), HIV), sdesc_join(pa + x * (32 * C::PX >> 4), HIP), I8, !first || x > 0);
            } else {
#pragma unroll 1
              for (int x = 0; x < 4; ++x)
                mma_ss(tmem + C::tm_n(t), sdesc_join(va + x * (2048 >> 4), HI16), sdesc_join(pa + x * (16 * C::PX >> 4), HIP), I16,
                       !first_new || x > 0);
            }
            mma_commit(BAR(C::O_DONE + 2 * t + (g & 1)));
            mma_commit(BAR(C::EMPTY + s));
          }
          __syncwarp();
          first = false;
          if (!cached) first_new = false;
          ++g;
        }
        items += tiles > 0;
      }
    }
    // every MMA issued has completed before TMEM is released
    commit(BAR(C::DRAIN));
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(BAR(C::DRAIN), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  } else {
    // ------------------------------------------------------------ softmax of lane t, a thread a key
    const int t = warp >> 2, wq = warp & 3, key = wq * 32 + lane;
    const uint32_t tlane = (uint32_t)(wq * 32) << 16;
    float2* rowc = reinterpret_cast<float2*>(sm + C::OFF_ROWC) + t * R;
    float* facs = reinterpret_cast<float*>(sm + C::OFF_FAC) + t * R;
    float* refs = reinterpret_cast<float*>(sm + C::OFF_REF);
    float* sums = reinterpret_cast<float*>(sm + C::OFF_SUM);
    float* red = reinterpret_cast<float*>(sm + C::OFF_RED) + t * 4 * (R + 4);
    volatile int* flags = reinterpret_cast<int*>(sm + C::OFF_FLAG) + 2 * t;
    float* vrefs = reinterpret_cast<float*>(sm + C::OFF_FLAG) + 4;
    if (lane == 0 && wq == 0) flags[0] = flags[1] = 0;  // (read after a phase of GROUP)
    int uq = 0, e0 = 0, g = 0, merges = 0, meets = 0;  // Q slots, ring entries, tiles, joins, phases of GROUP so far
    auto meet_arrive = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::GROUP + t));
    };
    auto meet = [&] {  // the four warps
      meet_arrive();
      return wait_phase(BAR(C::GROUP + t), meets++ & 1, st, SITE_T8_GROUP);
    };
    auto wait_pv = [&](int x) {  // tile x of the lane is in O, its P is read
      return wait_phase(BAR(C::O_DONE + 2 * t + (x & 1)), (x >> 1) & 1, st, SITE_T8_O_DONE);
    };
    auto run_item = [&](const Item8& it) {
      const bool dual = it.flags & ITEM8_DUAL;
      const int slot = (uq + (dual ? 0 : t)) % NQ, steps = t ? it.c1 : it.c0;
      const QRow* qr = qrows + slot * R;
      float l[RV];
#pragma unroll
      for (int r = 0; r < RV; ++r) l[r] = 0.f;
      float vref = 1.1754944e-38f;
      const int stride = dual ? 2 : 1, ahead = dual ? t : 0;
      const int cached_steps = min(steps, max(0, it.nc - it.j0 - ahead + stride - 1) / stride);
      int es = (e0 + ahead) % NT, s = 0;
      auto step = [&](auto of_cache) {
        constexpr bool cached = decltype(of_cache)::value;
        const int j = it.j0 + ahead + s * stride;
        // S is there, and P of the tile that had its buffer before has been read
        const uint32_t s_bar = BAR(C::S_FULL + 2 * t + (g & 1)), p_bar = BAR(C::O_DONE + 2 * t + (g & 1));
        const uint32_t s_ph = (g >> 1) & 1, p_ph = s_ph ^ 1;
        if (g < 2) {
          if (!wait_phase(s_bar, s_ph, st, SITE_T8_S_FULL)) return false;
        } else if (!__all_sync(0xffffffffu, mbar_try_wait(s_bar, s_ph) && mbar_try_wait(p_bar, p_ph))) {
          if (!wait_slow(s_bar, s_ph, st, SITE_T8_S_FULL) || !wait_slow(p_bar, p_ph, st, SITE_T8_O_DONE)) return false;
        }
        tc_fence_after();
        const bool there = key < rows_here(it, j);
        const float kscale = cached ? scales[es * 16 + (key >> 4)] : 1.f;
        const float vscale = cached ? scales[es * 16 + 8 + (key >> 4)] : 1.f;
        const uint32_t ts = tmem + tlane + C::tm_s(t, g & 1);
        uint32_t seen = there ? 0xffffffffu : 0u;  // of the rows
        if (!cached && there) {
          const int nkey = (j - it.nc) * C::NEW + key;  // the new token within its sequence
          seen = 0;
#pragma unroll 1
          for (int r = 0; r < RV; ++r) {
            const int tk = qr[r].tok;
            bool sees = nkey <= tk;
            if (a.mask)
              sees = tk >= 0 && (nkey >> 5) < a.words &&
                     (a.mask[(long long)(it.row0 + tk) * a.words + (nkey >> 5)] >> (nkey & 31) & 1);
            seen |= (uint32_t)sees << r;
          }
        }
        // scores to base 2 without their rows' factors
        auto load_y = [&](float (&y)[RV]) {
          uint32_t x0[RV], x1[RV];
          tmem_ldn<RV>(ts, x0);
          if (cached) tmem_ldn<RV>(ts + R, x1);
          tmem_wait_ld();
          const float k16 = kscale * 0.0625f;
#pragma unroll
          for (int r = 0; r < RV; ++r)
            y[r] = cached ? fmaf(__uint_as_float(x1[r]), k16, __uint_as_float(x0[r]) * kscale) : __uint_as_float(x0[r]);
        };
        // References move: for the first tile, or where a score or a scale has passed its own.
        auto move = [&] {
          float y[RV], mine = 0.f;
          load_y(y);
#pragma unroll
          for (int r = 0; r < RV; ++r) {
            const float f = cached ? qr[r].factor : a.scale_log2;
            const float m = warp_max((seen >> r & 1) ? y[r] * f : -INFINITY);
            if (lane == r) mine = m;
          }
          if (lane < RV) red[wq * (R + 4) + lane] = mine;
          const float vm = warp_max(there && cached ? vscale : 0.f);
          if (lane == 0) red[wq * (R + 4) + R] = vm;
          if (!meet()) return false;
          float v = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) v = fmaxf(v, red[x * (R + 4) + R]);
          const float to = cached && v > vref ? 2.f * v : vref, fv = vref / to;  // (cached tiles come first)
          vref = to;
          if (key < RV) {
            float m = -INFINITY, f = 1.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) m = fmaxf(m, red[x * (R + 4) + key]);
            const bool row = qr[key].tok >= 0;
            // a row that is none never moves; one without a key so far does with the first
            const float nb = s == 0 ? (row ? kPLog2 - kNoKey : kNoKey) : rowc[key].y, ref = kPLog2 - nb;
            if (row && m > ref + kLagLog2) {
              rowc[key] = make_float2(qr[key].factor, kPLog2 - m);
              f = ex2_approx(ref - m);
            } else if (s == 0) {
              rowc[key] = make_float2(qr[key].factor, nb);
            }
            facs[key] = f;
          }
          if (!meet()) return false;
          if (s > 0) {
            if (!wait_pv(g - 1)) return false;
            tc_fence_after();
            const int parts = cached_steps > 0 ? C::PPARTS : 0;  // of O that are there already; then that of new tokens
#pragma unroll 1
            for (int z = 0; z < parts + (s > cached_steps); ++z) {
              const uint32_t at = tmem + tlane + (z < parts ? C::tm_o(t) + z * R : C::tm_n(t));
              uint32_t x[RV];
              tmem_ldn<RV>(at, x);
              tmem_wait_ld();
#pragma unroll
              for (int r = 0; r < RV; ++r) x[r] = __float_as_uint(__uint_as_float(x[r]) * (facs[r] * (z < parts ? fv : 1.f)));
              tmem_stn<RV>(at, x);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int r = 0; r < RV; ++r) l[r] *= facs[r];
          return true;
        };
        bool moves = s == 0, vote = !moves;
        const uint32_t pbuf = sbase + C::OFF_P + (t * 2 + (g & 1)) * C::PBYTES;
        for (;;) {
          if (moves && !move()) return false;
          uint32_t x[RV / 2];
          float p[RV], top = -INFINITY;
          const float w = cached ? vscale / vref : 1.f;
          load_y(p);
#pragma unroll
          for (int r = 0; r < RV; ++r) {
            const float2 rc = rowc[r];
            float tt = fmaf(p[r], cached ? rc.x : a.scale_log2, rc.y);
            if (!(cached ? there : (seen >> r & 1))) tt = -INFINITY;
            top = fmaxf(top, tt);
            p[r] = tt;
          }
          if (vote) {
            const bool grows = __any_sync(0xffffffffu, top > kPLog2 + kLagLog2 || (there && cached && vscale > vref));
            if (grows && lane == 0) flags[meets & 1] = meets + 1;
            meet_arrive();
          } else {
            tc_fence_before();  // S is in registers for good
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::S_FREE + 2 * t + (g & 1)));
          }
#pragma unroll
          for (int r = 0; r < RV / 2; ++r) {
            p[2 * r] = ex2_approx(p[2 * r]);
            p[2 * r + 1] = ex2_approx(p[2 * r + 1]);
            x[r] = cached ? pack_f16x2(p[2 * r] * w, p[2 * r + 1] * w) : pack16<F16>(p[2 * r], p[2 * r + 1]);
          }
          if (vote) {
            const bool ok = wait_phase(BAR(C::GROUP + t), meets & 1, st, SITE_T8_GROUP);
            const bool grows = flags[meets & 1] == meets + 1;
            ++meets;
            if (!ok) return false;
            if (grows) {
              moves = true, vote = false;
              continue;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::S_FREE + 2 * t + (g & 1)));
          }
#pragma unroll
          for (int r = 0; r < RV; ++r) l[r] += p[r];
          if (cached) {
#pragma unroll
            for (int z = 0; z < C::PPARTS; ++z) {
              uint32_t part[RV / 4];
#pragma unroll
              for (int r = 0; r < RV / 4; ++r) {
                const uint32_t lo = to_e5m2(x[2 * r]), hi = to_e5m2(x[2 * r + 1]);
                part[r] = upper_bytes(lo, hi);
                x[2 * r] = h2_sub(x[2 * r], lo);
                x[2 * r + 1] = h2_sub(x[2 * r + 1], hi);
                if (z == 1) x[2 * r] = h2_mul64(x[2 * r]), x[2 * r + 1] = h2_mul64(x[2 * r + 1]);
              }
              if constexpr (RV == 16)
                sts128(pbuf + swizzled<C::PX>(key, z), part[0], part[1], part[2], part[3]);
              else if constexpr (RV == 8)
                sts64(pbuf + swizzled<C::PX>(key, z), part[0], part[1]);
              else
                sts32(pbuf + swizzled<C::PX>(key, z), part[0]);
            }
          } else if (key < C::NEW) {
            if constexpr (RV >= 8) {
#pragma unroll
              for (int c = 0; c < RV / 8; ++c)
                sts128(pbuf + swizzled<C::PX>(key, c), x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            } else {
              sts64(pbuf + swizzled<C::PX>(key, 0), x[0], x[1]);
            }
          }
          break;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::P_READY + 2 * t + (g & 1)));  // (two: P may be two tiles ahead of its product)
        ++s, ++g;
        es += stride;
        if (es >= NT) es -= NT;
        return true;
      };
      while (s < cached_steps)
        if (!step(std::true_type())) return false;
      while (s < steps)
        if (!step(std::false_type())) return false;
      if (steps > 0) {
        if (!wait_pv(g - 1)) return false;
        tc_fence_after();
        // Sums over the warp's keys: groups of 32 / RV lanes end with a row each. Where there are no steps nothing is
        // written here: the other lane may still read what the item before left.
        int row = 0;
#pragma unroll
        for (int o = 16, n = RV / 2; o; o >>= 1, n >>= 1) {
          if (n == 0) {
            l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
            continue;
          }
          const bool up = lane & o;
          row += up ? n : 0;
#pragma unroll
          for (int r = 0; r < n; ++r) {
            const float send = up ? l[r] : l[r + n], keep = up ? l[r + n] : l[r];
            l[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
        if ((lane & (32 / RV - 1)) == 0) sums[(t * 4 + wq) * R + row] = l[0];
        if (key < RV) refs[t * R + key] = kPLog2 - rowc[key].y;
        if (key == 0) vrefs[t] = vref;
      }
      return true;
    };
    // What becomes of an item's results
    auto finish = [&](const Item8& it) {
      const bool dual = it.flags & ITEM8_DUAL, join = dual && it.c1 > 0, whole = it.flags & ITEM8_WHOLE;
      const int slot = (uq + (dual ? 0 : t)) % NQ, steps = t ? it.c1 : it.c0;
      const QRow* qr = qrows + slot * R;
      const long long part0 = (long long)it.slot * (2 * R) + (dual ? 0 : t * RV);
      const int rows = min(RV, it.n * a.G - it.r0 - (dual ? 0 : t * RV));  // 1 at least, where there are steps
      if (steps > 0) {
        // The other lane's results stay as they are until its next product into O, which waits for this lane's
        // arrival below.
        if (join) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(C::MERGE));
          if (!wait_phase(BAR(C::MERGE), merges++ & 1, st, SITE_T8_MERGE)) return false;
          tc_fence_after();
        } else if (!meet()) {
          return false;
        }
        // rows [ra, rb), RG at a time: in a join each lane takes half of them
        constexpr int RG = RV == 16 ? 8 : 4;
        const int half = (rows + 2 * RG - 1) / (2 * RG) * RG, ra = join ? t * half : 0, rb = join && t == 0 ? half : rows;
        const float v0 = vrefs[0], v1 = vrefs[1];
        auto o_free = [&] {  // O is in registers: the issuers may write it again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive_n(BAR(C::O_FREE + t), join ? 1 : 2);
            if (join) mbar_arrive(BAR(C::O_FREE + (t ^ 1)));
          }
        };
        if (ra >= rb) o_free();
#pragma unroll 1
        for (int r0 = ra; r0 < rb; r0 += RG) {
          // weights of both lanes' O for row r0 + lane % RG, and its LSE to base 2
          const int rr = r0 + (lane & (RG - 1));
          const float m0 = refs[(join ? 0 : t) * R + rr], m1 = join ? refs[R + rr] : kNoKey, m = fmaxf(m0, m1);
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            l0 += sums[((join ? 0 : t) * 4 + x) * R + rr];
            if (join) l1 += sums[(4 + x) * R + rr];
          }
          float f0 = ex2_approx(m0 - m), f1 = ex2_approx(m1 - m);
          const int tok = qr[rr].tok;
          float sum = l0 * f0 + l1 * f1;
          // scores of -inf alone, of an infinite query say: no maximum to take off, the row is NaN
          if (sum == 0.f && tok >= 0 &&
              sees_a_key(a.mask, a.words, it.row0 + tok, tok, it.n, it.j0 < it.nc, max(0, it.j0 - it.nc) * C::NEW,
                         (it.j0 + it.cnt - it.nc) * C::NEW))
            sum = NAN;
          const float inv = sum != 0.f ? 1.f / sum : 0.f;  // 0: no key; NaN stays NaN
          f0 *= inv, f1 *= inv;
          const long long token = qr[rr].to & 0xffffffffffll, head = qr[rr].to >> 40;
          if (wq == 0 && lane < RG && rr < rb && tok >= 0) {
            const float lse2 = sum != 0.f ? m - kPLog2 + lg2_approx(sum) : -INFINITY;
            if (!whole) {
              if (FA_CHECK(in_range(part0 + rr, a.part_rows), st, DBG_GLOBAL_STORE)) a.part_lse[part0 + rr] = lse2;
            } else if (a.lse && FA_CHECK(in_range(token, a.T - FA_SLACK(a)), st, DBG_GLOBAL_STORE)) {
              a.lse[head * a.T + token] = lse2 * 0.6931471805599453f;
            }
          }
          float o[RG] = {};
          if (key < D) {
#pragma unroll 1
            for (int u = 0; u < 1 + join; ++u) {
              uint32_t x[C::PPARTS][RG], y[RG];
              const int of = join ? u : t, first = it.j0 + (dual ? of : 0), last = dual ? it.j0 + it.cnt - 1 - ((it.cnt - 1 - of) & 1)
                                                                                     : it.j0 + steps - 1;
              const bool old = first < it.nc, fresh = last >= it.nc;  // that lane's tiles: cached ones, new ones
              const float v = of ? v1 : v0;
#pragma unroll
              for (int z = 0; z < C::PPARTS; ++z) tmem_ldn<RG>(tmem + tlane + C::tm_o(of) + r0 + z * R, x[z]);
              tmem_ldn<RG>(tmem + tlane + C::tm_n(of) + r0, y);
              tmem_wait_ld();
#pragma unroll
              for (int r = 0; r < RG; ++r) {
                float low = __uint_as_float(x[2][r]);
                if (F16) low += __uint_as_float(x[C::PPARTS - 1][r]);
                low = fmaf(low, 0.015625f, __uint_as_float(x[0][r]) + __uint_as_float(x[1][r]));
                // (what was never written is not looked at)
                const float all = (old ? low * v : 0.f) + (fresh ? __uint_as_float(y[r]) : 0.f);
                o[r] = fmaf(all, __shfl_sync(0xffffffffu, u ? f1 : f0, r), o[r]);
              }
            }
          }
          if (r0 + RG >= rb) o_free();
          if (key >= D) continue;
          if (whole) {
            // even threads write the even rows of two columns each, odd threads the odd rows
            uint16_t* const row = a.o + token * a.o_st + head * a.o_sh;  // of this lane's rr
            const long long mine = tok >= 0 && FA_CHECK(in_range(token, a.T - FA_SLACK(a)), st, DBG_GLOBAL_STORE) ? (long long)row : 0;
#pragma unroll
            for (int r = 0; r < RG; r += 2) {
              const float got = __shfl_xor_sync(0xffffffffu, (lane & 1) ? o[r] : o[r + 1], 1);
              const uint32_t y = (lane & 1) ? pack16<F16>(got, o[r + 1]) : pack16<F16>(o[r], got);
              const long long to = __shfl_sync(0xffffffffu, mine, r + (lane & 1));
              if (to) *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(to) + (key & ~1)) = y;
            }
          } else {
#pragma unroll
            for (int r = 0; r < RG; ++r)
              if (__shfl_sync(0xffffffffu, tok, r) >= 0 && FA_CHECK(in_range(part0 + r0 + r, a.part_rows), st, DBG_GLOBAL_STORE))
                a.part_o[(part0 + r0 + r) * D + key] = o[r];
          }
        }
      } else if (!dual && key < RV && qr[key].tok >= 0 && FA_CHECK(in_range(part0 + key, a.part_rows), st, DBG_GLOBAL_STORE)) {
        a.part_lse[part0 + key] = -INFINITY;  // (a cut item only) none of this part's keys concerns these rows
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::Q_EMPTY + slot));
      return true;
    };
    for (int i = 0;; ++i) {
      Item8 it;
      if (!next_item(i, &it) || it.cnt < 0) break;
      const bool dual = it.flags & ITEM8_DUAL;
      // both slots of a pair, and the other lane's let go at once: a barrier's parity tells two uses of a slot apart, not
      // three, so none may be left out, nor be two uses ahead of a wait for it
      bool ok = true;
      for (int u = uq; ok && u < uq + (dual ? 1 : 2); ++u)
        ok = wait_phase(BAR(C::Q_FULL + u % NQ), (u / NQ) & 1, st, SITE_T8_Q_FULL);
      if (!ok) break;
      if (!dual && lane == 0) mbar_arrive(BAR(C::Q_EMPTY + (uq + (t ^ 1)) % NQ));
      if (!run_item(it) || !finish(it)) break;
      uq += dual ? 1 : 2;
      e0 += it.cnt;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::PV0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Joins the partial results of the items, `unit` rows each, that CTA boundaries cut: block (x, y) takes rows
// [16 y, 16 y + 16) of the item that boundary x + 1 is the first to cut, a group of D / 4 threads a row.
// Latency bounds it: a long sequence has a part in many CTAs, so the group reads as many parts' LSEs at once as it
// has threads, and eight parts' rows (one after the other, joining two contexts of 131072 tokens took 15 us).
template <int D, bool F16>
__global__ void __launch_bounds__(4 * D) serve8_join_kernel(Serve8BitArgs a, int unit) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x + 1;
  const int parts = a.cuts[2 * c].x + 1;  // part 0: CTA c - 1's last item; then the first items of c, c + 1, ..
  if (parts == 1) return;
  const int4 cut = a.cuts[2 * c + 1];  // rows of the sequence, its first token, the item's first row, head
  constexpr int LPR = D / 4;
  const int sub = threadIdx.x % LPR, row = blockIdx.y * 16 + threadIdx.x / LPR, rr = cut.z + row;
  const int tok = rr / a.G;
  auto at = [&](int k) { return (long long)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * (2 * Serve8Cfg<D, F16>::R) + row; };
  const bool there = row < unit && rr < cut.x &&
                     FA_CHECK(in_range(at(0), a.part_rows) && in_range(at(parts - 1), a.part_rows), a.status, DBG_GLOBAL_LOAD) &&
                     FA_CHECK(in_range(cut.y + tok, a.T - FA_SLACK(a)) && in_range(cut.w, a.Hkv), a.status, DBG_GLOBAL_STORE);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < parts; k0 += LPR) {
    const int k = k0 + sub, n = min(LPR, parts - k0);
    const float s = there && k < parts ? a.part_lse[at(k)] : -INFINITY;  // (-inf: nothing was written there)
    float top = s;
#pragma unroll
    for (int x = LPR / 2; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(top, m);
    const float base = top == -INFINITY ? 0.f : top, f = ex2_approx(m - base), w = s == s ? ex2_approx(s - base) : s;
    l *= f, o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    m = top;
    for (int x0 = 0; x0 < n; x0 += 8) {
      float4 v[8];
      float wx[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        wx[x] = __shfl_sync(0xffffffffu, w, min(x0 + x, n - 1), LPR);
        if (x0 + x >= n) wx[x] = 0.f;
        v[x] = wx[x] != 0.f ? *reinterpret_cast<const float4*>(a.part_o + at(k0 + x0 + x) * D + 4 * sub) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        l += wx[x];
        o.x = fmaf(wx[x], v[x].x, o.x), o.y = fmaf(wx[x], v[x].y, o.y), o.z = fmaf(wx[x], v[x].z, o.z), o.w = fmaf(wx[x], v[x].w, o.w);
      }
    }
  }
  if (!there) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int h = cut.w * a.G + rr - tok * a.G;
  const long long token = cut.y + tok;
  *reinterpret_cast<uint2*>(a.o + token * a.o_st + h * a.o_sh + 4 * sub) =
      make_uint2(pack16<F16>(o.x * inv, o.y * inv), pack16<F16>(o.z * inv, o.w * inv));
  if (sub == 0 && a.lse)
    a.lse[(long long)h * a.T + token] = (l != 0.f ? m + lg2_approx(l) : -INFINITY) * 0.6931471805599453f;
}

template <int D, bool F16, int RV>
static int launch_serve8_d(const fa_rows* k, const fa_rows* v, const fa_pages* c, Serve8BitArgs a, cudaStream_t stream) {
  using C = Serve8Cfg<D, F16>;
  const auto type = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mk, mv, mkc, mvc;
  auto map3 = [&](CUtensorMap* m, const fa_rows* r) {
    const cuuint64_t dims[3] = {D, (cuuint64_t)a.T, (cuuint64_t)a.Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)r->token_stride * 2, (cuuint64_t)r->head_stride * 2};
    const cuuint32_t box[3] = {64, kNewBox8, 1};
    return make_tmap_strided(m, r->data, type, 3, dims, strides, box);
  };
  auto map4 = [&](CUtensorMap* m, const void* p) {
    const cuuint64_t dims[4] = {D, (cuuint64_t)c->page_size, (cuuint64_t)a.Hkv, (cuuint64_t)c->n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c->token_stride, (cuuint64_t)c->head_stride, (cuuint64_t)c->page_stride};
    const cuuint32_t box[4] = {D, (cuuint32_t)std::min(c->page_size, 128), 1, 1};
    return make_tmap_strided(m, p, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, dims, strides, box,
                             D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (!map3(&mk, k) || !map3(&mv, v) || !map4(&mkc, c->k) || !map4(&mvc, c->v))
    return cuda_fail("cuTensorMapEncodeTiled", 0, "tensor map rejected");
  const auto kernel = serve8_kernel<D, F16, RV>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute", (int)e, cudaGetErrorName(e));
  int sms = 0;
  if (!sm_count(&sms)) return FA_ERR_CUDA;
  // slots of its own in the workspace, which fa_forward_tree_workspace_size measures for slots of 256 rows
  static_assert(2 * C::R <= 256, "the workspace");
  a.part_rows = 2LL * sms * 2 * C::R;
  a.part_lse = a.part_o + a.part_rows * D;
  a.cuts = reinterpret_cast<int4*>(a.part_lse + a.part_rows);
  const int rc = launch_pdl("serve8_kernel", kernel, dim3(sms), dim3(C::THREADS), C::SMEM_BYTES, stream, mk, mv, mkc, mvc, a);
  if (rc != FA_OK || sms < 2) return rc;
  return launch_pdl("serve8_join_kernel", serve8_join_kernel<D, F16>, dim3(sms - 1, (2 * RV + 15) / 16), dim3(4 * D), 0, stream, a, 2 * RV);
}

template <int D, bool F16>
static int launch_serve8_rows(const fa_rows* k, const fa_rows* v, const fa_pages* c, const Serve8BitArgs& a, cudaStream_t stream) {
  // The rows of a sequence are on the device; their average decides. Up to an average of 16, sequences with up to twice as
  // many still have one item a head; above it, where averages of up to 32 come here too, those with up to 32 rows. Others
  // have more, and their context is read once for each. Whatever the distribution, that makes no more than 2 B items a
  // head: a part of a prompt among decoding sequences, or a batch of mostly empty ones, costs at most what two decoding
  // batches of B over its length do. 256 sequences over 4096 tokens, 32 heads over 8 of 128: 128 tokens of one and one of
  // each other 414 us (the kernel for many rows 1055), 64 tokens of four and none of the others 167 (49).
  const long long rows = (long long)a.T * a.G;
  if (rows <= 4LL * a.B) return launch_serve8_d<D, F16, 4>(k, v, c, a, stream);
  if (rows <= 8LL * a.B) return launch_serve8_d<D, F16, 8>(k, v, c, a, stream);
  return launch_serve8_d<D, F16, 16>(k, v, c, a, stream);
}

int launch_serve8(const fa_rows* k, const fa_rows* v, const fa_pages* cache, Serve8BitArgs a, int d, int dtype,
                  cudaStream_t stream) {
  const bool f16 = dtype == FA_FP16;
  if (d == 64) return f16 ? launch_serve8_rows<64, true>(k, v, cache, a, stream) : launch_serve8_rows<64, false>(k, v, cache, a, stream);
  return f16 ? launch_serve8_rows<128, true>(k, v, cache, a, stream) : launch_serve8_rows<128, false>(k, v, cache, a, stream);
}

}  // namespace fa
