// Attention of whole prompts and of drafted trees over a cache in pages: entry points and kernels.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fa_internal.h"
#include "serve.cuh"
#include "serve_args.h"
#include "serve_tree.h"
#include "tmap.h"

namespace fa {

// Key tiles that a CTA of the tree kernel takes where there are few (the last one may take one less), and
// rows of a TMA box of new tokens there (a draft seldom fills a tile of 128).
constexpr int kMinTiles = 2;
constexpr int kNewBox = 16;

// ---------------------------------------------------------------------------------------------
// One persistent kernel for prompts and for trees over a cache.
//
// Rows: a query tile holds the rows (token, head of the group) of NPT = 128 / G tokens of one
// key/value head, so that its keys are read once for the whole group. A work item is a pair of
// such tiles, one for each of two query lanes (warpgroups 0 and 1), over the key tiles of its
// sequence: first the cached tokens, 128 a tile, then the new ones. Where an item has one query
// tile only, both lanes take it and alternate key tiles ("dual"), and join the two results out of
// tensor memory at the end, each for half of the columns.
//
// Roles, 384 threads: warps 0-3 and 4-7 the softmax of lanes 0 and 1 (a thread a row), warp 9
// the TMA producer and scheduler, warps 8 and 10 the issuers of O += P V of lanes 0 and 1, warp
// 11 the issuer of S = Q K^T of both (with one issuer a lane for both products, decoding 64
// sequences over up to 8192 tokens took 210 us instead of 176). The producer
// runs ahead: it publishes items in a ring of four descriptors, loads Q into two slots and K and
// V tiles alternately into one ring of NSLOT slots (224 KB with Q). A page is one TMA box, the
// lanes of the producer warp issuing one each. All rings and barrier phases run on across items.
//
// Trees (PAGED): all key tiles of all items form one sequence, of which every CTA takes an equal
// run, whatever the lengths; an item cut between CTAs leaves fp32 partial results, which
// serve_join_kernel joins. Prompts: whole items, longest first in the snake order.
//
// Rounding: scores, maxima, sums and O are fp32; P is rounded to the inputs' type for the product
// with V (the tensor core takes both operands in one type), its sum is not; O is rounded once.
// fp16 has all its bits down to 2^-14 and none below 2^-25, so there P is formed 2^9 times its value,
// and the reference maximum moves when it grows by 2^6 (bf16: 2^8), so that P stays within 2^15: a
// probability keeps its bits down to 2^-23 of the row's largest and is off by 2^-34 of it at most below that
// (2^-25 without the factor: 8000 keys with 3e-4 of the weight beside one of value 0 gave O off by a fifth).
// A factor of 2^11 with a growth of 2^4 costs fp16 1-3 % where queries are four times as large, this one 0-1 %.
// l carries the factor with it, O = P V / l does not, and the LSE takes it off.
//
// Measured on one GB300, in a graph: prompts of 8192 + 590 + 13 tokens, 16 heads over 2 of 128: 186 us,
// 1480 TFLOP/s, 77 % of the measured bf16 peak, the tensor pipe busy 78 % of the cycles (16 over 4 of 64:
// 142 us, 970 TFLOP/s, busy 51 %: a lane's one score buffer makes softmax and S wait for each other);
// decoding 64 sequences over up to 8192 tokens, 32 heads over 8 of 128: 169 us, 6.4 TB/s, 95 % of the
// measured copy rate (97 us, 82 %, at d = 64 and 174 us, 92 %, with pages of 16 tokens, where the
// producer's issue bounds it); 512 sequences over up to 500 tokens: 194 us, 44 % (12 heads of 64: 239 us, 27 %):
// an item's start and end; 64 trees of up to 64 nodes over up to 32768 tokens: 960 us, bound by the
// tensor pipe (81-84 % busy) beside memory at 76 %.
//
// A cache in 8 bits (C8): the pages arrive in a ring of their own, and four more warps (12-15) turn them into tiles
// of fp16 (exactly) in the ring that the products read, so that all else is as it is. A converter thread takes
// 16 elements of one key at a time, the lanes of a quarter-warp eight keys that follow each other, which the
// swizzled rows of both sides spread over all banks. The products are fp16 for bf16 queries too: e4m3 to fp16 is one
// instruction for two elements, to bf16 four (with it, the trees below took 398 us). The converters bring the
// queries, and the keys and values of new tokens, to fp16 with a power of two for each 32 rows that takes their
// largest element to [2^14, 2^15): elements keep their bits down to 2^-28 of that one. They load the new tokens
// too, as they meet all entries of the ring in order.
// Scales: that of a key's block of 16 multiplies its scores within the exponential's argument, and the block's
// maximum; that of a value's adds its logarithm there, so that P is formed with it, and the sum l takes it out
// again by blocks. A reference (vref, twice the largest so far) keeps P in range; O keeps up with it as it does
// with the maximum. It takes one bit of P's range: what is below 2^-22 of the row's largest probability (times the
// largest scale) is off by 2^-33 of it.
// 32 trees of up to 64 nodes over up to 16384 tokens, 32 heads over 8 of 128: 311 us, 730 TFLOP/s, the tensor pipe busy
// 48 % of the cycles: a step of 64 keys takes both lanes' softmax some 1850. That is longer than in 16 bits, by the work
// on the scales of each 16 keys, in 128 registers a thread: where rows are many, a cache of half the size is read more
// slowly. The same calls over 8 bits and over 16, 32 heads over 8 of 128, bf16 (fp16): 32 trees of 32 to 64 nodes over
// 2000 to 16384 tokens 322 and 249 us (298 and 256), 8 times 512 tokens over 8192 608 and 430 (497 and 432), 8 times
// 2048 over 32768 8775 and 6994 (7541 and 7370).
template <int D, bool C8 = false>
struct ServeCfg {
  static constexpr int NSUB = D / 64;
  static constexpr int SUB_BYTES = 128 * 128, Q_BYTES = NSUB * SUB_BYTES;
  static constexpr int TK = C8 ? 64 : 128, TK_LOG2 = C8 ? 6 : 7;  // keys of a tile
  // what an item's start and end cost, in tiles, as the runs are balanced (an item's change of 15000 cycles stands beside
  // 1200 to 1900 a tile with C8)
  static constexpr int ITEM_TILES = C8 ? 10 : 0;
  static constexpr int KSUB_BYTES = TK * 128, TILE_BYTES = NSUB * KSUB_BYTES;
  static constexpr int NSLOT = C8 ? (D == 64 ? 10 : 6) : D == 64 ? 12 : 5;
  static constexpr int STAGE = TK * D, NS8 = C8 ? (D == 64 ? 12 : 6) : 0;  // pages of 8 bits
  // tiles whose scales are kept: more than have an entry in either ring, or have not been met by the softmax
  static constexpr int SCALES = C8 ? 16 : 0;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_R = 2 * Q_BYTES;
  static constexpr int OFF_S8 = OFF_R + NSLOT * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_S8 + NS8 * STAGE, BAR_AREA = C8 ? 2048 : 512;
  static constexpr int OFF_DESC = OFF_BAR + BAR_AREA;  // 4 x 16 ints
  static constexpr int OFF_ML = OFF_DESC + 256;    // m and l of both lanes' rows, for the join of a dual item
  static constexpr int OFF_SC = OFF_ML + 2048;     // [tile][K of 4 groups of 16 keys, V of 4]
  static constexpr int SMEM_BYTES = OFF_SC + SCALES * 32;
  // A key tile is taken in HPT steps of KT keys. The softmax must find S of the next step ready
  // when it ends one, so S may not wait for PV of the step before. TMEM has room for that in two
  // ways: d = 64 keeps P apart from S (one step a tile; S is free once it is in registers);
  // d = 128, where O takes half the columns, takes a tile as two halves; even and odd steps of a
  // lane have a buffer each, P over its own S, and S is formed two steps ahead.
  static constexpr bool SEP_P = D == 64 && !C8;
  static constexpr int KT = SEP_P ? 128 : 64, HPT = TK / KT;
  __device__ static constexpr int buf(int g) { return SEP_P ? 0 : g & 1; }            // of a lane's step g
  __device__ static constexpr uint32_t phase(int g) { return (SEP_P ? g : g >> 1) & 1; }  // of its barriers
  __device__ static constexpr uint32_t tm_s(int t, int u) { return 128u * t + 64u * u; }
  __device__ static constexpr uint32_t tm_p(int t, int u) { return SEP_P ? 256u + 64u * t : tm_s(t, u); }
  __device__ static constexpr uint32_t tm_o(int t) { return SEP_P ? 384u + 64u * t : 256u + (uint32_t)D * t; }
  static constexpr uint32_t TM_COLS = 512;
  static constexpr int THREADS = C8 ? 512 : 384;
  // with few rows the softmax is warps 0 and 4, on the scheduler of warp 8: the least busy role there
  static constexpr int PV0 = 8, PRODUCER = 9, PV1 = 10, S_BOTH = 11;
  // barriers
  static constexpr int FULL = 0, EMPTY = NSLOT, Q_FULL = 2 * NSLOT, Q_EMPTY = Q_FULL + 2, S_FULL = Q_EMPTY + 2,
                       P_READY = S_FULL + 4, O_DONE = P_READY + 4, S_FREE = O_DONE + 4, O_FREE = S_FREE + 2,
                       MERGE = O_FREE + 2, DRAIN = MERGE + 1, D_FULL = DRAIN + 1, D_EMPTY = D_FULL + 4,
                       FULL8 = D_EMPTY + 4, EMPTY8 = FULL8 + NS8, Q_RAW = EMPTY8 + NS8, NEW_RAW = Q_RAW + 2 * C8,
                       BARS = NEW_RAW + NSLOT * C8;
  // behind the barriers: three words, and with C8 vref of both lanes, the factors of 32 rows of each Q slot, and
  // those of 32 keys, K and V, of the last new tiles
  static constexpr int OFF_VREF = 8 * BARS + 12, OFF_QF = OFF_VREF + 8, OFF_NSC = (OFF_QF + 32 + 15) / 16 * 16;
  static_assert((C8 ? OFF_NSC + SCALES * 16 : 8 * BARS + 12) <= BAR_AREA, "barrier area");
  static_assert(!C8 || (NSLOT % 2 == 0 && NS8 % 2 == 0), "K and V have slots of their own");
  static_assert(SMEM_BYTES <= 232448, "shared memory above 227 KB");
};

enum { SITE_SW_EMPTY = 60, SITE_SW_Q_FULL, SITE_SW_Q_EMPTY, SITE_SW_K_FULL, SITE_SW_V_FULL, SITE_SW_S_FREE,
       SITE_SW_P_READY, SITE_SW_O_FREE, SITE_SW_S_FULL, SITE_SW_O_DONE, SITE_SW_MERGE, SITE_SW_DESC_FULL,
       SITE_SW_DESC_EMPTY, SITE_SW_FULL8, SITE_SW_EMPTY8 };

// A work item (or the part of it that this CTA computes), as the producer publishes it.
struct ServeItem {
  int cnt;     // key tiles here; -1: no more items
  int flags;   // 1: dual, 2: the whole item is here (results go straight to O)
  int c0, c1;  // key tiles of lanes 0 and 1
  int j0;      // first key tile, counted from the item's first
  int nc;      // tiles of cached tokens; tile j >= nc holds the new tokens from 128 (j - nc)
  int L, n;    // cached and new tokens of the sequence
  int row0;    // the sequence's first row among the packed tokens
  int tok0;    // the pair's first token within the sequence
  int kvh;
  int slot;    // partial result slot
  int s0, s1;  // steps of lanes 0 and 1 (a half of a tile with no key in it is no step)
  int cnt_all; // (not published) key tiles of the whole item
};
enum { ITEM_DUAL = 1, ITEM_WHOLE = 2 };

// Sizes of sequence b's work, in items of `unit` tokens; record: whether invalid device values are
// recorded.
struct SeqWork {
  int row0, n, L, nc, nk, units;
  long long tiles;  // all heads and units, each counted with the nk tiles of the last one
};
template <bool PAGED, int TL, int EX>
__device__ __forceinline__ SeqWork seq_sizes(const ServeArgs& a, int lo, int hi, int len, int unit, bool record) {
  SeqWork w;
  w.row0 = min(max(lo, 0), a.T);
  const int end = min(max(hi, w.row0), a.T);
  if (record && (w.row0 != lo || end != hi)) record_check(a.status, SITE_S_OFFSETS);
  w.n = end - w.row0;
  w.L = 0;
  if (PAGED && w.n > 0) {
    w.L = min(max(len, 0), a.table_width << a.page_shift);
    if (record && w.L != len) record_check(a.status, SITE_S_LENGTH);
  }
  w.nc = (w.L + (1 << TL) - 1) >> TL;
  w.nk = w.nc + ((w.n + (1 << TL) - 1) >> TL);
  w.units = (w.n + unit - 1) / unit;
  w.tiles = (long long)w.units * a.Hkv * (w.nk + EX);
  return w;
}
template <bool PAGED, int TL, int EX>
__device__ __forceinline__ SeqWork seq_work(const ServeArgs& a, int b, int unit, bool record) {
  return seq_sizes<PAGED, TL, EX>(a, a.cu[b], a.cu[b + 1], PAGED ? a.lens[b] : 0, unit, record);
}

__device__ __forceinline__ long long warp_sum(long long x) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Trees: the run of key tiles of CTA c, by a whole warp. Each lane counts the tiles of `chunk` sequences
// that follow each other, four sequences' loads at a time, so that the search below looks at a lane's
// sequences only (a block of 32 sequences after the other, both took up to 15 us for 512 sequences).
struct ServeRuns {
  long long total, base;
  int ctas, rest;        // CTAs with work; the first `rest` of them take a tile more
  long long mine;        // this lane's tiles
  int chunk;
  __device__ long long start(int c) const { return base * c + min(c, rest); }
};
template <int TL, int EX>
__device__ __forceinline__ ServeRuns serve_runs(const ServeArgs& a, int unit, int grid, bool record) {
  ServeRuns r;
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
      if (b + k < end) r.mine += seq_sizes<true, TL, EX>(a, at[k], at[k + 1], len[k], unit, record).tiles;
  }
  r.total = warp_sum(r.mine);
  r.ctas = r.total < (long long)grid * kMinTiles ? max(1, ((int)r.total + kMinTiles - 1) / kMinTiles) : grid;
  r.base = r.total < (1LL << 31) ? (int)r.total / r.ctas : r.total / r.ctas;  // the short division costs a fifth
  r.rest = (int)(r.total - r.base * r.ctas);
  return r;
}
// The lane whose own tiles hold tile `pos` of all, and their first one; 32: past the end.
__device__ __forceinline__ int lane_of(long long mine, long long pos, long long* first) {
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
template <int TL, int EX>
__device__ __forceinline__ int serve_seek(const ServeArgs& a, int unit, const ServeRuns& runs, long long pos,
                                          long long* first) {
  *first = 0;
  const int k = lane_of(runs.mine, pos, first);
  if (k == 32) return a.B;
  if (runs.chunk == 1) return k;
  const int end = min(a.B, (k + 1) * runs.chunk);
  for (int b0 = k * runs.chunk; b0 < end; b0 += 32) {
    const int b = b0 + (threadIdx.x & 31);
    const int x = lane_of(b < end ? seq_work<true, TL, EX>(a, b, unit, false).tiles : 0, pos, first);
    if (x < 32) return b0 + x;
  }
  return a.B;
}

// Key tiles that query tile u (tokens [u npt, ..)) of a sequence needs, counted from the first.
template <int TL>
__device__ __forceinline__ int tiles_of(const SeqWork& w, int u, int npt, bool tree) {
  if (u * npt >= w.n) return 0;
  return w.nc + ((min(tree ? w.n : (u + 1) * npt, w.n) + (1 << TL) - 1) >> TL);
}

// Prompts: the tokens of an item, by a whole warp. Two query tiles share the keys that an item loads;
// but with few items the longest one alone may outlast the even share of all key tiles, and items
// of one tile, whose keys both lanes divide, take half as long: 16 prompts of up to 2048 tokens, 16 / 8
// heads of 128, take 30 us so and 31.4 in pairs, four of up to 200, 12 heads of 64, 6.6 and 7.5; prompts
// of 8192 + 590 + 13, 16 / 2 heads, where the share is longer than any item, 249 and 186.
__device__ __forceinline__ int prompt_unit(const ServeArgs& a, int npt, int grid, bool record) {
  long long tiles = 0;
  int longest = 0;
  for (int b0 = threadIdx.x & 31; b0 < a.B; b0 += 128) {  // four sequences' loads at a time
    int lo[4], hi[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int b = min(b0 + 32 * k, a.B - 1);
      lo[k] = a.cu[b], hi[k] = a.cu[b + 1];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (b0 + 32 * k >= a.B) break;
      const SeqWork w = seq_sizes<false, 7, 0>(a, lo[k], hi[k], 0, 2 * npt, record);
      tiles += (w.tiles + (long long)w.units * a.Hkv) / 2;  // item p of a sequence has about (p + 1) nk / units
      longest = max(longest, w.nk);
    }
  }
  tiles = warp_sum(tiles);
  longest = __reduce_max_sync(0xffffffffu, longest);
  return tiles < (long long)longest * grid ? npt : 2 * npt;
}
// The items of all prompts, longest first: level p holds the p-th items of all sequences that have
// one, in the order of the sequences. Used by a whole warp; the item counts of the first 128
// sequences stay in registers (read again for every item, they made the search longer than an
// ordinary item's work). A CTA asks for ascending items, so that a search goes on where the last one
// ended; starting anew each time, 1024 prompts of up to 200 tokens took 2925 us instead of 329.
struct PromptItems {
  static constexpr int KEPT = 4;
  const ServeArgs& a;
  int unit, total, mine[KEPT];
  int level, end;   // the last item's level, and the items of that level and up
  int b0, before;   // the block of sequences that holds it, and the items before that block's
  __device__ PromptItems(const ServeArgs& args, int u) : a(args), unit(u) {
    int most = 0;
#pragma unroll
    for (int k = 0; k < KEPT; ++k) {
      mine[k] = units(32 * k);
      most = max(most, mine[k]);
    }
    int x = 0;
#pragma unroll 4
    for (int b = 32 * KEPT; b < a.B; b += 32) {
      const int n = units(b);
      x += n;
      most = max(most, n);
    }
#pragma unroll
    for (int k = 0; k < KEPT; ++k) x += mine[k];
    total = __reduce_add_sync(0xffffffffu, x);
    level = __reduce_max_sync(0xffffffffu, most);  // above the first item's
    end = b0 = before = 0;
  }
  __device__ int units(int from) const {
    const int b = from + (threadIdx.x & 31);
    return b < a.B ? seq_work<false, 7, 0>(a, b, unit, false).units : 0;
  }
  __device__ int above(int l) const {  // items of that level and up
    int x = 0;
#pragma unroll
    for (int k = 0; k < KEPT; ++k) x += max(0, mine[k] - l);
#pragma unroll 4
    for (int b = 32 * KEPT; b < a.B; b += 32) x += max(0, units(b) - l);
    return __reduce_add_sync(0xffffffffu, x);
  }
  // Sequence and level of item i < total, not before the last one asked for.
  __device__ void find(int i, int* b, int* l) {
    if (i >= end) {  // a lower level: doubling steps down to above(lo) > i >= above(hi), then halves
      int hi = level, lo = level, n_hi = end, n_lo = end;
      for (int step = 1; n_lo <= i && lo > 0; step *= 2) {
        hi = lo, n_hi = n_lo;
        lo = max(0, lo - step);
        n_lo = above(lo);
      }
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, n = above(mid);
        if (n > i) lo = mid, n_lo = n; else hi = mid, n_hi = n;
      }
      level = lo, end = n_lo;
      b0 = 0, before = n_hi;
    }
    *l = level;
    for (; b0 < a.B; b0 += 32) {
      int u = 0;
#pragma unroll
      for (int k = 0; k < KEPT; ++k)
        if (b0 == 32 * k) u = mine[k];
      if (b0 >= 32 * KEPT) u = units(b0);
      unsigned m = __ballot_sync(0xffffffffu, u > level);
      const int k = __popc(m);
      if (i - before < k) {
        for (int left = i - before; left; --left) m &= m - 1;
        *b = b0 + __ffs(m) - 1;
        return;
      }
      before += k;
    }
  }
};

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// Sixteen e4m3 as two 16-byte chunks of fp16, exactly.
__device__ __forceinline__ void widen16(const uint4& x, uint4* lo, uint4* hi) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r[i]) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
  *lo = make_uint4(r[0], r[1], r[2], r[3]);
  *hi = make_uint4(r[4], r[5], r[6], r[7]);
}
// Rows of bf16 in swizzled tiles of 64 columns to fp16 in place, by a warp: eight from `first` on, and eight more every
// `stride`, below `end`; times a power of two that takes their largest finite element to [2^14, 2^15). Returns what
// undoes the factor. (Rows behind them are nobody's, or masked, or, of V, zeroed before the product.)
// Loops of few instructions: the code runs once an item, and fetching it anew is what it takes (unrolled, 32 rows of
// 128 columns took 10000 cycles between the loops of the products, against 2600 at the start).
template <int NSUB, int SUB_BYTES>
__device__ __forceinline__ float to_fp16_rows(uint8_t* tile, int first, int stride, int end) {
  const int lane = threadIdx.x & 31;
  // a step: 4 rows, 8 chunks each; two steps and NSUB columns of them, then the next eight rows
  const int steps = (max(0, end - first) + stride - 1) / stride * 2 * NSUB;
  auto row_of = [&](int y) { return first + stride * (y / (2 * NSUB)) + y / NSUB % 2 * 4 + (lane >> 3); };
  auto place = [&](int y) { return reinterpret_cast<uint4*>(tile + y % NSUB * SUB_BYTES + sw128_offset(row_of(y), lane & 7)); };
  uint32_t most2 = 0;  // two magnitudes, as whole numbers
#pragma unroll 1
  for (int y = 0; y < steps; ++y) {
    const uint4 x = *place(y);
    if (row_of(y) >= end) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w) & 0x7fff7fffu;
      most2 = __vmaxu2(most2, w & __vcmpltu2(w, 0x7f807f80u));
    }
  }
  const uint32_t most = __reduce_max_sync(0xffffffffu, max(most2 & 0xffffu, most2 >> 16));
  const int e = max((int)(most >> 7) - 127, -100) - 14;  // 2^-e times the largest lies in [2^14, 2^15)
  const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 1
  for (int y = 0; y < steps; ++y) {
    uint4* at = place(y);
    uint4 x = *at;
    auto half2 = [&](uint32_t w) { return pack_f16x2(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down); };
    x.x = half2(x.x), x.y = half2(x.y), x.z = half2(x.z), x.w = half2(x.w);
    *at = x;
  }
  return up;
}

template <int D, bool F16, bool PAGED, bool C8 = false>
__global__ void __launch_bounds__(C8 ? 512 : 384, 1)
    serve_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kc,
                 const __grid_constant__ CUtensorMap tm_vc, std::conditional_t<C8, Serve8BitArgs, ServeArgs> a) {
  using C = ServeCfg<D, C8>;
  constexpr bool H = C8 || F16;         // the products are fp16
  constexpr bool TURN = C8 && !F16;     // the converters bring Q, and K and V of new tokens, to fp16
  constexpr float P_LOG2 = H ? 9.f : 0.f, LAG_LOG2 = H ? 6.f : 8.f;
  // 1024-byte aligned, as the swizzled tiles have to be: there is no room to round the address up
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sbase = smem_u32(sm);
  if (sbase & 1023u) {  // (never seen: the kernel has no static shared memory)
    griddep_wait();
    if (threadIdx.x == 0) {
      record_check(a.status, SITE_S_SMEM);
      if (PAGED) a.cuts[2 * blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing for the join to read
    }
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t b0 = sbase + C::OFF_BAR;
  auto BAR = [&](int i) { return b0 + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + 8 * C::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  volatile int* loading = reinterpret_cast<int*>(tmem_slot + 2);  // ring entries whose loads have begun
  float* vrefs = reinterpret_cast<float*>(sm + C::OFF_BAR + C::OFF_VREF);  // (C8) of both lanes, for the join
  float* qfs = reinterpret_cast<float*>(sm + C::OFF_BAR + C::OFF_QF);      // [slot][32 rows each]
  float* nscales = reinterpret_cast<float*>(sm + C::OFF_BAR + C::OFF_NSC);  // [new tile][K of 32 keys each, V]
  float* scales = reinterpret_cast<float*>(sm + C::OFF_SC);
  DevStatus st{a.status, abort_flag};
  int* descs = reinterpret_cast<int*>(sm + C::OFF_DESC);
  const int npt = 128 / a.G;  // tokens of a query tile

  if (warp == C::PRODUCER && lane == 0) {
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(BAR(C::FULL + i), C8 ? 4 : 1);  // (two converters twice, or, of K of new tokens, all four)
      mbar_init(BAR(C::EMPTY + i), 2);  // V: both issuers; K: its issuer twice
    }
    for (int i = 0; i < C::NS8; ++i) {
      mbar_init(BAR(C::FULL8 + i), i & 1 ? 1 : 9);  // the copies, and with K each of 8 lanes' scale
      mbar_init(BAR(C::EMPTY8 + i), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(BAR(C::Q_FULL + t), TURN ? 4 : 1);
      if (C8) mbar_init(BAR(C::Q_RAW + t), 1);
      mbar_init(BAR(C::Q_EMPTY + t), TURN ? 9 : 1);  // the issuer of S (and all softmax warps)
      for (int h = 0; h < 2; ++h) {
        mbar_init(BAR(C::S_FULL + 2 * t + h), 1);
        mbar_init(BAR(C::P_READY + 2 * t + h), 4);
        mbar_init(BAR(C::O_DONE + 2 * t + h), 1);
      }
      mbar_init(BAR(C::S_FREE + t), 4);
      mbar_init(BAR(C::O_FREE + t), 8);  // four warps twice, or all eight in a join
    }
    for (int i = 0; i < (C8 ? C::NSLOT : 0); ++i) mbar_init(BAR(C::NEW_RAW + i), 1);
    mbar_init(BAR(C::MERGE), 8);
    mbar_init(BAR(C::DRAIN), 3);
    for (int i = 0; i < 4; ++i) {
      mbar_init(BAR(C::D_FULL + i), 1);
      mbar_init(BAR(C::D_EMPTY + i), C8 ? 15 : 11);  // softmax warps, issuers and converters
    }
    *abort_flag = 0;
    *loading = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    if (PAGED) {
      prefetch_tmap(&tm_kc);
      prefetch_tmap(&tm_vc);
    }
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

  // Steps that lane t takes in the item's tile j: those halves in which some row of its query tile
  // sees a key.
  const bool tree = PAGED && a.mask != nullptr;
  auto steps_in = [&](const ServeItem& it, int t, int j) {
    if (C::HPT == 1) return 1;
    const int last = it.tok0 + ((it.flags & ITEM_DUAL) ? 1 : t + 1) * npt;  // past the lane's last token
    const int keys = j < it.nc ? it.L - j * 128 : (tree ? it.n : min(it.n, last)) - (j - it.nc) * 128;
    return keys > C::KT ? 2 : 1;
  };

  // Item i of this CTA, for a consumer warp: false when the CTA must give up.
  auto next_item = [&](int i, ServeItem* it) {
    if (!wait_phase(BAR(C::D_FULL + (i & 3)), (i >> 2) & 1, st, SITE_SW_DESC_FULL)) return false;
    const int4* d = reinterpret_cast<const int4*>(descs + 16 * (i & 3));
    const int4 x = d[0], y = d[1], z = d[2], w = d[3];
    it->cnt = x.x, it->flags = x.y, it->c0 = x.z, it->c1 = x.w;
    it->j0 = y.x, it->nc = y.y, it->L = y.z, it->n = y.w;
    it->row0 = z.x, it->tok0 = z.y, it->kvh = z.z, it->slot = z.w;
    it->s0 = w.x, it->s1 = w.y;
    __syncwarp();
    if (lane == 0) mbar_arrive(BAR(C::D_EMPTY + (i & 3)));
    return true;
  };

  if (warp == C::PRODUCER) {
    // ------------------------------------------------------------ scheduler and TMA producer
    int items = 0, uq = 0, e = 0;  // items published, Q slots and ring entries (C8: tiles of 8 bits) used
    bool ok = true;
    auto publish = [&](const ServeItem& it) {
      if (!wait_phase(BAR(C::D_EMPTY + (items & 3)), ((items >> 2) & 1) ^ 1, st, SITE_SW_DESC_EMPTY)) return false;
      if (lane == 0) {
        int4* d = reinterpret_cast<int4*>(descs + 16 * (items & 3));
        d[0] = make_int4(it.cnt, it.flags, it.c0, it.c1);
        d[1] = make_int4(it.j0, it.nc, it.L, it.n);
        d[2] = make_int4(it.row0, it.tok0, it.kvh, it.slot);
        d[3] = make_int4(it.s0, it.s1, 0, 0);
        mbar_arrive(BAR(C::D_FULL + (items & 3)));
      }
      __syncwarp();
      ++items;
      return true;
    };
    // Loads the item's query tiles and its key tiles [j0, j0 + cnt).
    auto run_item = [&](const ServeItem& it, int b) {
      if (!publish(it)) return false;
      // page ids of a tile: lane (box r, column block c) = r NSUB + c, and lane 16 + r NSUB + c
      const int prow = min(1 << a.page_shift, C::TK);  // rows of a page's box
      const int r = (lane & 15) / C::NSUB, c = lane % C::NSUB;
      auto page_of = [&](int j) {
        if (C8) {  // lane (kv, g) = 4 kv + g: of 16 keys
          const int t0 = j * 64 + (lane & 3) * 16;
          return lane < 8 && j < min(it.j0 + it.cnt, it.nc) && t0 < it.L ? a.table[b * a.table_stride + (t0 >> a.page_shift)] : 0;
        }
        const int pg = (j * 128 + r * prow) >> a.page_shift;
        const bool there = j < it.j0 + it.cnt && j < it.nc && r * prow < 128 && j * 128 + r * prow < it.L;
        return there ? a.table[b * a.table_stride + pg] : 0;
      };
      int id = PAGED ? page_of(it.j0) : 0;
      const int nq = (it.flags & ITEM_DUAL) ? 1 : 2;
      for (int t = 0; t < nq; ++t, ++uq) {
        const uint32_t qf = BAR((TURN ? C::Q_RAW : C::Q_FULL) + (uq & 1));
        if (!wait_phase(BAR(C::Q_EMPTY + (uq & 1)), ((uq >> 1) & 1) ^ 1, st, SITE_SW_Q_EMPTY)) return false;
        if (elect_one()) mbar_arrive_expect_tx(qf, (uint32_t)(npt * a.G * 128 * C::NSUB));
        __syncwarp();
        const uint32_t dst = sbase + C::OFF_Q + (uq & 1) * C::Q_BYTES;
        if (lane < C::NSUB)
          tma_load_3d(dst + lane * C::SUB_BYTES, &tm_q, lane * 64, it.kvh * a.G, it.row0 + it.tok0 + t * npt, qf);
        __syncwarp();
      }
      int j = it.j0;
      if constexpr (C8) {
        // K and V of a tile in one go, a lane for 16 keys: their scale, and the box that begins with them
        const int kv = (lane >> 2) & 1, g = lane & 3, page_size = 1 << a.page_shift;
        for (; j < min(it.j0 + it.cnt, it.nc); ++j, ++e) {
          const int id_next = page_of(j + 1), rows = min(64, it.L - j * 64), boxes = (rows + prow - 1) / prow;
          const int sk = (2 * e) % C::NS8, sv = sk + 1;
          const uint32_t ph = ((2 * e / C::NS8) & 1) ^ 1;
          if (!wait_phase(BAR(C::EMPTY8 + sk), ph, st, SITE_SW_EMPTY8) || !wait_phase(BAR(C::EMPTY8 + sv), ph, st, SITE_SW_EMPTY8))
            return false;
          const int t0 = j * 64 + g * 16, in_page = t0 & (page_size - 1);
          const bool mine = lane < 8 && g * 16 < rows, there = id >= 0 && id < a.n_pages;
          if (mine && !there) record_check(a.status, SITE_S_PAGE);
          if (elect_one()) {
            mbar_arrive_expect_tx(BAR(C::FULL8 + sk), (uint32_t)(boxes * prow * D));
            mbar_arrive_expect_tx(BAR(C::FULL8 + sv), (uint32_t)(boxes * prow * D));
          }
          __syncwarp();
          float* to = scales + e % C::SCALES * 8 + lane;
          if (mine && there && FA_CHECK(in_range(it.kvh, a.Hkv), st, DBG_GLOBAL_LOAD)) {
            const float* from = (kv ? a.vs : a.ks) + id * a.s_sp + it.kvh * a.s_sh + (in_page >> a.block_shift);
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(BAR(C::FULL8 + sk)) : "memory");
          } else if (lane < 8) {
            *to = kv ? 0.f : 1.f;  // nothing there: its probabilities are 0, and stay out of vref
            mbar_arrive(BAR(C::FULL8 + sk));
          }
          const uint32_t dst = sbase + C::OFF_S8 + (kv ? sv : sk) * C::STAGE + g * 16 * D;
          if (mine && (g * 16 & (prow - 1)) == 0 && !(kWithhold && e == 1) &&
              FA_CHECK(smem_in(dst, prow * D, sbase + C::OFF_S8, sbase + C::OFF_BAR), st, DBG_TMA_LOAD))
            tma_load_4d(dst, kv ? &tm_vc : &tm_kc, 0, in_page, it.kvh, there ? id : a.n_pages, BAR(C::FULL8 + (kv ? sv : sk)));
          __syncwarp();
          id = id_next;
        }
        return true;
      }
      // With few rows and small boxes this warp is the slowest: K and V of a tile in one go then, a lane for
      // each box (decoding 64 sequences of up to 8192 tokens took 112 us a slot at a time and takes 100 at
      // d = 64, 190 and 177 at d = 128 with pages of 16 tokens). Few tiles an item gain nothing by it, nor
      // do larger boxes at d = 128, where the ring has five slots and is full.
      if (PAGED && (D == 64 || a.page_shift == 4) && it.cnt >= 8 && it.n <= 16 && it.n * a.G <= 16) {
        for (; j < min(it.j0 + it.cnt, it.nc); ++j, e += 2) {
          const int id_next = page_of(j + 1), boxes = (min(128, it.L - j * 128) + prow - 1) / prow;
          const bool mine = (lane & 15) < boxes * C::NSUB;
          int page = id;
          if (mine && (id < 0 || id >= a.n_pages)) {
            record_check(a.status, SITE_S_PAGE);
            page = a.n_pages;
          }
          const int s0 = e % C::NSLOT, s1 = (e + 1) % C::NSLOT, s = lane < 16 ? s0 : s1;
          if (!wait_phase(BAR(C::EMPTY + s0), ((e / C::NSLOT) & 1) ^ 1, st, SITE_SW_EMPTY) ||
              !wait_phase(BAR(C::EMPTY + s1), (((e + 1) / C::NSLOT) & 1) ^ 1, st, SITE_SW_EMPTY))
            return false;
          if (elect_one()) {
            *loading = e + 2;
            mbar_arrive_expect_tx(BAR(C::FULL + s0), (uint32_t)(boxes * prow * 128 * C::NSUB));
            mbar_arrive_expect_tx(BAR(C::FULL + s1), (uint32_t)(boxes * prow * 128 * C::NSUB));
          }
          __syncwarp();
          const uint32_t dst = sbase + C::OFF_R + s * C::TILE_BYTES + c * C::KSUB_BYTES + r * prow * 128;
          if (mine && !(kWithhold && (e >> 1) == 1) &&
              FA_CHECK(smem_in(dst, prow * 128, sbase + C::OFF_R, sbase + C::OFF_BAR), st, DBG_TMA_LOAD))
            tma_load_4d(dst, lane < 16 ? &tm_kc : &tm_vc, c * 64, j * 128 & ((1 << a.page_shift) - 1) & ~127, it.kvh, page,
                        BAR(C::FULL + s));
          __syncwarp();
          id = id_next;
        }
      }
      for (; j < it.j0 + it.cnt; ++j) {
        const int id_next = PAGED ? page_of(j + 1) : 0;
        const bool cached = PAGED && j < it.nc;
        const int k0 = cached ? j * 128 : (j - it.nc) * 128;
        const int rows = min(128, (cached ? it.L : it.n) - k0);
        const int box = cached ? prow : PAGED ? kNewBox : 128;
        const int boxes = (rows + box - 1) / box;
        int page = id;
        if (cached && lane < boxes * C::NSUB && (id < 0 || id >= a.n_pages)) {
          record_check(a.status, SITE_S_PAGE);
          page = a.n_pages;  // outside the tensor: reads as zeros
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++e) {
          const int s = e % C::NSLOT;
          const uint32_t bar = BAR(C::FULL + s);
          if (!wait_phase(BAR(C::EMPTY + s), ((e / C::NSLOT) & 1) ^ 1, st, SITE_SW_EMPTY)) return false;
          if (elect_one()) {
            *loading = e + 1;
            mbar_arrive_expect_tx(bar, (uint32_t)(boxes * box * 128 * C::NSUB));
          }
          __syncwarp();
          if (kWithhold && (e >> 1) == 1) continue;  // test build: this copy never arrives
          const uint32_t dst = sbase + C::OFF_R + s * C::TILE_BYTES + c * C::KSUB_BYTES + r * box * 128;
          if (lane < boxes * C::NSUB &&
              FA_CHECK(smem_in(dst, box * 128, sbase + C::OFF_R, sbase + C::OFF_BAR), st, DBG_TMA_LOAD)) {
            if (cached)
              tma_load_4d(dst, kv ? &tm_vc : &tm_kc, c * 64, k0 & ((1 << a.page_shift) - 1) & ~127, it.kvh, page, bar);
            else
              tma_load_3d(dst, kv ? &tm_v : &tm_k, c * 64, it.row0 + k0 + r * box, it.kvh, bar);
          }
          __syncwarp();
        }
        id = id_next;
      }
      return true;
    };
    auto make_item = [&](const SeqWork& w, int unit, int kvh, int p, int j0, int j1, ServeItem* it) {
      const int u = unit == npt ? p : 2 * p;  // first query tile
      const int n0 = tiles_of<C::TK_LOG2>(w, u, npt, tree), n1 = unit == npt ? 0 : tiles_of<C::TK_LOG2>(w, u + 1, npt, tree);
      const int nmax = max(n0, n1);
      const bool dual = n1 == 0;
      j1 = min(j1, nmax);
      it->cnt = max(0, j1 - j0);
      it->cnt_all = nmax;
      it->flags = (dual ? ITEM_DUAL : 0) | (j0 == 0 && j1 == nmax ? ITEM_WHOLE : 0);
      it->c0 = dual ? (it->cnt + 1) >> 1 : max(0, min(j1, n0) - j0);
      it->c1 = dual ? it->cnt >> 1 : it->cnt;
      it->j0 = j0, it->nc = w.nc, it->L = w.L, it->n = w.n, it->row0 = w.row0, it->tok0 = p * unit, it->kvh = kvh;
      it->slot = 2 * blockIdx.x + (j0 == 0);
      it->s0 = it->c0 * C::HPT, it->s1 = it->c1 * C::HPT;
      if (C::HPT > 1) {  // only the last cached tile and a lane's last tile may have a half less
        for (int t = 0; t < 2; ++t) {
          int* steps = t ? &it->s1 : &it->s0;
          const int end = dual ? j0 + it->cnt : j0 + (t ? it->c1 : it->c0);  // past the lane's tiles
          auto mine = [&](int j) { return j >= j0 && j < end && (!dual || ((j - j0) & 1) == t); };
          const int lc = w.nc - 1, ln = (dual || t == 0 ? n0 : n1) - 1;
          if (mine(lc)) *steps -= 2 - steps_in(*it, t, lc);
          if (ln != lc && mine(ln)) *steps -= 2 - steps_in(*it, t, ln);
        }
      }
    };
    ServeItem it;
    if (PAGED) {
      const int unit = 2 * npt;
      const ServeRuns runs = serve_runs<C::TK_LOG2, C::ITEM_TILES>(a, unit, gridDim.x, blockIdx.x == 0);
      int parts = 0;  // of the item that this CTA is the first to cut
      int4 cut = make_int4(0, 0, 0, 0);
      if ((int)blockIdx.x < runs.ctas && runs.total > 0) {
        long long pos = runs.start(blockIdx.x), first = 0;
        const long long end = runs.start(blockIdx.x + 1);
        int b = serve_seek<C::TK_LOG2, C::ITEM_TILES>(a, unit, runs, pos, &first);
        while (ok && pos < end) {
          const SeqWork w = seq_work<PAGED, C::TK_LOG2, C::ITEM_TILES>(a, b, unit, false);
          // the first item may be cut; from then on they are met from their start
          const int span = w.nk + C::ITEM_TILES;  // an item's share of the run: its costs, then its tiles
          const long long at = pos - first;
          const int q = at < (1LL << 31) ? (int)at / max(span, 1) : (int)(at / span);
          int p = q / a.Hkv, kvh = q - p * a.Hkv, x0 = (int)(at - (long long)q * span);
          bool again = false;  // the last item was whole, and this one differs in its head only
          while (ok && pos < end && pos - first < w.tiles) {
            const int x1 = (int)min((long long)span, x0 + (end - pos));
            const int j0 = max(0, x0 - C::ITEM_TILES), j1 = max(0, x1 - C::ITEM_TILES);
            if (again && j1 == w.nk)
              it.kvh = kvh;
            else
              make_item(w, unit, kvh, p, j0, j1, &it);
            const long long tile0 = pos - x0 + C::ITEM_TILES;  // the place of the item's first tile
            if (j0 > 0 && it.cnt > 0 && runs.start(blockIdx.x - 1) <= tile0) {
              // (the first item only) how many CTAs, this one included, hold later parts of it
              const long long end_of_item = tile0 + it.cnt_all;
              for (int k = blockIdx.x + lane; __any_sync(0xffffffffu, k < runs.ctas); k += 32)
                parts += __popc(__ballot_sync(0xffffffffu, k < runs.ctas && runs.start(k) < end_of_item));
              cut = make_int4(it.n, it.row0, it.tok0, it.kvh);
            }
            if (it.cnt > 0) ok = run_item(it, b);
            pos += x1 - x0;
            again = j0 == 0 && j1 == w.nk;
            x0 = 0;
            if (++kvh == a.Hkv) kvh = 0, ++p, again = false;
          }
          first += w.tiles;
          ++b;
        }
      }
      if (lane == 0) {
        a.cuts[2 * blockIdx.x] = make_int4(parts, 0, 0, 0);
        a.cuts[2 * blockIdx.x + 1] = cut;
      }
    } else {
      const int unit = prompt_unit(a, npt, gridDim.x, blockIdx.x == 0);
      PromptItems items_of(a, unit);
      for (long long round = 0; ok; ++round) {
        const int G = gridDim.x, c = blockIdx.x;
        const long long i = round * G + ((round & 1) ? G - 1 - c : c);
        int b = 0, p = 0;
        if (i >= (long long)items_of.total * a.Hkv) break;  // later rounds lie past the end too
        items_of.find((int)(i / a.Hkv), &b, &p);
        const SeqWork w = seq_work<PAGED, C::TK_LOG2, C::ITEM_TILES>(a, b, unit, false);
        make_item(w, unit, (int)(i % a.Hkv), p, 0, w.nk, &it);
        ok = run_item(it, b);
      }
    }
    if (ok) {
      it.cnt = -1;
      ok = publish(it);
    }
    if constexpr (C8) asm volatile("cp.async.wait_all;" ::: "memory");
    if (*(volatile int*)abort_flag) {
      // let copies already in flight land before the CTA's shared memory is released
      const int ring = C8 ? C::NS8 : C::NSLOT, full = C8 ? C::FULL8 : C::FULL, used = C8 ? 2 * e : e;
      for (int x = max(0, used - ring); x < used; ++x) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(BAR(full + x % ring), (x / ring) & 1) && globaltimer_ns() - t0 < 100000000ull) {
        }
      }
      for (int x = max(0, uq - 2); x < uq; ++x) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(BAR((TURN ? C::Q_RAW : C::Q_FULL) + (x & 1)), (x >> 1) & 1) && globaltimer_ns() - t0 < 100000000ull) {
        }
      }
    }
  } else if (C8 && warp >= 12) {
    // ------------------------------------------------------------ converters, and the loads of new tokens
    if constexpr (C8) {
      const int cw = warp - 12;
      // Warps 12 and 13 take K, 14 and 15 V, half of the keys each: the slots of K (even) and V are rings of their own.
      constexpr int NS8 = C8 ? C::NS8 : 2;
      const int kv = cw >> 1, half = cw & 1;
      int x = 0, uq = 0, news = 0, slot = kv;  // tiles of 8 bits, Q slots and new tiles so far
      uint32_t phase = 1, raw = 0;             // of the slot's EMPTY; of each slot's NEW_RAW
      bool ok = true;
      for (int i = 0; ok; ++i) {
        ServeItem it;
        if (!next_item(i, &it) || it.cnt < 0) break;
        if (TURN) {
          const int nq = (it.flags & ITEM_DUAL) ? 1 : 2;
          for (int t = 0; ok && t < nq; ++t, ++uq) {
            if (!(ok = wait_phase(BAR(C::Q_RAW + (uq & 1)), (uq >> 1) & 1, st, SITE_SW_Q_FULL))) break;
            const int toks = min(npt, it.n - it.tok0 - t * npt);  // (rows behind them may be other sequences')
            const float up = to_fp16_rows<C::NSUB, C::SUB_BYTES>(sm + C::OFF_Q + (uq & 1) * C::Q_BYTES, 8 * cw, 32, toks * a.G);
            if (lane == 0) qfs[(uq & 1) * 4 + cw] = up;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::Q_FULL + (uq & 1)));
          }
        }
        for (int j = it.j0; ok && j < it.j0 + it.cnt; ++j) {
          const uint32_t full = BAR(C::FULL + slot);
          uint8_t* to = sm + C::OFF_R + slot * C::TILE_BYTES;
          if (j < it.nc) {
            const int s8 = (2 * x + kv) % NS8;
            if (!(ok = wait_phase(BAR(C::FULL8 + s8), ((2 * x + kv) / NS8) & 1, st, SITE_SW_FULL8))) break;
            if (!(ok = wait_phase(BAR(C::EMPTY + slot), phase, st, SITE_SW_EMPTY))) break;
            if (!FA_CHECK(smem_in(smem_u32(to), C::TILE_BYTES, sbase + C::OFF_R, sbase + C::OFF_S8) &&
                              smem_in(sbase + C::OFF_S8 + s8 * C::STAGE, C::STAGE, sbase + C::OFF_S8, sbase + C::OFF_BAR),
                          st, DBG_SMEM)) {
              ok = false;
              break;
            }
            const uint8_t* from = sm + C::OFF_S8 + s8 * C::STAGE;
            const int c0 = lane >> 3;
#pragma unroll
            for (int y = 0; y < 4 * (D / 64); ++y) {
              const uint32_t key = half * 32 + (y & 3) * 8 + (lane & 7), c = c0 + 4 * (y >> 2);
              const uint32_t at = D == 128 ? key * 128 + ((c ^ (key & 7)) << 4) : key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
              uint4 lo, hi;
              widen16(*reinterpret_cast<const uint4*>(from + at), &lo, &hi);
              uint8_t* sub = to + (c >> 2) * C::KSUB_BYTES;
              *reinterpret_cast<uint4*>(sub + sw128_offset(key, 2 * (c & 3))) = lo;
              *reinterpret_cast<uint4*>(sub + sw128_offset(key, 2 * (c & 3) + 1)) = hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_n(full, 2);
              mbar_arrive(BAR(C::EMPTY8 + s8));
            }
            ++x;
          } else {
            const int k0 = (j - it.nc) * 64, rows = min(64, it.n - k0), boxes = (rows + kNewBox - 1) / kNewBox;
            if (!(ok = wait_phase(BAR(C::EMPTY + slot), phase, st, SITE_SW_EMPTY))) break;
            const uint32_t landed = BAR(C::NEW_RAW + slot);
            if (half == 0) {
              if (elect_one()) mbar_arrive_expect_tx(landed, (uint32_t)(boxes * kNewBox * 128 * C::NSUB));
              __syncwarp();
              const int r = lane / C::NSUB, c = lane % C::NSUB;
              const uint32_t dst = smem_u32(to) + c * C::KSUB_BYTES + r * kNewBox * 128;
              if (lane < boxes * C::NSUB && FA_CHECK(smem_in(dst, kNewBox * 128, sbase + C::OFF_R, sbase + C::OFF_S8), st, DBG_TMA_LOAD))
                tma_load_3d(dst, kv ? &tm_v : &tm_k, c * 64, it.row0 + k0 + r * kNewBox, it.kvh, landed);
              __syncwarp();
            }
            if (!(ok = wait_phase(landed, raw >> slot & 1, st, SITE_SW_FULL8))) break;
            raw ^= 1u << slot;
            if (TURN) {
              const float up = to_fp16_rows<C::NSUB, C::KSUB_BYTES>(to, half * 32, 8, min(rows, half * 32 + 32));
              if (lane == 0) nscales[news % C::SCALES * 4 + kv * 2 + half] = up;
              fence_proxy_async_smem();
              __syncwarp();
            }
            // S of the tile finds the factors of both: K's entry is full when V is there too (K's slot has been given up
            // by the tile that had V's before, as this one has been waited for)
            if (lane == 0) {
              mbar_arrive_n(full, kv ? 2 : 1);
              if (kv) mbar_arrive(BAR(C::FULL + slot - 1));
            }
            ++news;
          }
          slot += 2;
          if (slot >= C::NSLOT) slot = kv, phase ^= 1;
        }
      }
      if (*(volatile int*)abort_flag && half == 0) {  // as the producer does: copies of new tokens land first
        // (those whose waits gave up; where another wait did, none is in flight)
        for (int y = kv; y < C::NSLOT; y += 2) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(BAR(C::NEW_RAW + y), raw >> y & 1) && globaltimer_ns() - t0 < 10000000ull) {
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ MMA issuers
    constexpr uint32_t IDESC_S = H ? idesc_f16_f32(128, C::KT, 0, 0) : idesc_bf16_f32(128, C::KT, 0, 0);
    constexpr uint32_t IDESC_O = H ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
    constexpr uint32_t HI = sdesc_hi(1024), TILE16 = C::TILE_BYTES >> 4, Q16 = C::Q_BYTES >> 4, HALF16 = (C::KT * 128) >> 4;
    auto commit = [&](uint32_t bar) {
      if (elect_one()) mma_commit(bar);
      __syncwarp();
    };
    // A place in the ring of K and V tiles. A barrier's parity tells two uses of a slot apart, not
    // three: a warp that releases only K or only V, which take turns in a slot at d = 128, may wait for
    // a use only when the slot's use before it has landed. Within an item that follows from the steps
    // before (the use before lies two or three tiles back, and this warp has waited for a product
    // that reads it); for an item's first tiles, and for those of which its lane computes nothing,
    // `landed` looks whether the load has begun, which it does once that use is over.
    struct Place {
      int entry, slot;
      uint32_t parity;
      __device__ void skip(int entries) {  // fewer than NSLOT
        entry += entries;
        slot += entries;
        if (slot >= C::NSLOT) slot -= C::NSLOT, parity ^= 1;
      }
    };
    int begun = 0;  // of `loading`, when last looked at
    // (C8: K and V have slots of their own, and every warp waits for all uses in order.)
    auto landed = [&](const Place& p, bool steady, int site) {
      if (!C8 && !steady && begun <= p.entry) {
        const uint64_t t0 = globaltimer_ns();
        for (uint32_t spins = 1;; ++spins) {
          begun = *loading;
          if (__all_sync(0xffffffffu, begun > p.entry)) break;
          bool give_up = false;
          if ((spins & 63u) == 0) {
            if (*(volatile int*)abort_flag || *(volatile int*)st.word == FA_ERR_TIMEOUT) {
              *(volatile int*)abort_flag = 1;
              give_up = true;
            } else if (globaltimer_ns() - t0 > kWaitLimitNs) {
              record_error(st, FA_ERR_TIMEOUT, site);
              give_up = true;
            }
          }
          if (__any_sync(0xffffffffu, give_up)) return false;
        }
      }
      return wait_phase(BAR(C::FULL + p.slot), p.parity, st, site);
    };
    bool ok = true;
    if (warp == C::S_BOTH) {
      // S = Q K^T of both lanes, tile after tile in the order of the ring
      const uint32_t q_lo = sdesc_lo(sbase + C::OFF_Q, 16), k_lo = sdesc_lo(sbase + C::OFF_R, 16);
      Place ks = {0, 0, 0};
      int uq = 0, g0 = 0, g1 = 0;  // Q slots and steps of both lanes so far
      for (int i = 0; ok; ++i) {
        ServeItem it;
        if (!next_item(i, &it) || it.cnt < 0) break;
        const bool dual = it.flags & ITEM_DUAL;
        const int nq = dual ? 1 : 2;
        for (int u = uq; ok && u < uq + nq; ++u)
          ok = wait_phase(BAR(C::Q_FULL + (u & 1)), (u >> 1) & 1, st, SITE_SW_Q_FULL);
        const uint32_t qa0 = q_lo + (uq & 1) * Q16, qa1 = q_lo + ((uq + nq - 1) & 1) * Q16;
        auto form_s = [&](int t, int g, uint32_t qa, uint32_t ka) {
          const uint32_t d = tmem + C::tm_s(t, C::buf(g));
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * C::SUB_BYTES + (k & 3) * 32) >> 4, koff = ((k >> 2) * C::KSUB_BYTES + (k & 3) * 32) >> 4;
            if (elect_one()) mma_ss(d, sdesc_join(qa + off, HI), sdesc_join(ka + koff, HI), IDESC_S, k > 0);
          }
          commit(BAR(C::S_FULL + 2 * t + C::buf(g)));
        };
        auto issue_s = [&](int t, int g, uint32_t qa, uint32_t ka) {
          // S(g) goes over S(g - 1), once it is in registers (d = 64), or over P(g - 2), once PV has read it
          if (C::SEP_P ? g > 0 : g > 1) {
            if (C::SEP_P ? !wait_phase(BAR(C::S_FREE + t), (g - 1) & 1, st, SITE_SW_S_FREE)
                         : !wait_phase(BAR(C::O_DONE + 2 * t + C::buf(g)), C::phase(g - 2), st, SITE_SW_O_DONE))
              return false;
          }
          tc_fence_after();
          form_s(t, g, qa, ka);
          return true;
        };
        // up to three phases at once: a wait for each costs some 200 cycles even where all have completed
        auto wait_for = [&](uint32_t x, uint32_t px, uint32_t y, uint32_t py, uint32_t z, uint32_t pz) {
          if (__all_sync(0xffffffffu, mbar_try_wait(x, px) && mbar_try_wait(y, py) && mbar_try_wait(z, pz))) return true;
          return wait_slow(x, px, st, SITE_SW_K_FULL) && wait_slow(y, py, st, SITE_SW_O_DONE) &&
                 wait_slow(z, pz, st, SITE_SW_O_DONE);
        };
        for (int k = 0; ok && k < it.cnt; ++k) {
          const int j = it.j0 + k;
          const int h0 = (dual ? (k & 1) : k >= it.c0) ? 0 : steps_in(it, 0, j);
          const int h1 = (dual ? !(k & 1) : k >= it.c1) ? 0 : steps_in(it, 1, j);
          const uint32_t ka = k_lo + ks.slot * TILE16, kb = BAR(C::FULL + ks.slot);
          const uint32_t o0 = BAR(C::O_DONE + C::buf(g0)), o1 = BAR(C::O_DONE + 2 + C::buf(g1));
          if (!C::SEP_P && k >= 4 && h0 == 2 && h1 == 2) {
            // the ordinary tile of two lanes
            if (!(ok = wait_for(kb, ks.parity, o0, C::phase(g0 - 2), o1, C::phase(g1 - 2)))) break;
            tc_fence_after();
            form_s(0, g0++, qa0, ka);
            form_s(1, g1++, qa1, ka);
            const uint32_t n0 = BAR(C::O_DONE + C::buf(g0)), n1 = BAR(C::O_DONE + 2 + C::buf(g1));
            if (!(ok = wait_for(n0, C::phase(g0 - 2), n0, C::phase(g0 - 2), n1, C::phase(g1 - 2)))) break;
            tc_fence_after();
            form_s(0, g0++, qa0, ka + HALF16);
            form_s(1, g1++, qa1, ka + HALF16);
          } else {
            if (!(ok = landed(ks, k >= 4, SITE_SW_K_FULL))) break;
            for (int h = 0; ok && h < max(h0, h1); ++h) {
              if (h < h0) ok = issue_s(0, g0++, qa0, ka + h * HALF16);
              if (ok && h < h1) ok = issue_s(1, g1++, qa1, ka + h * HALF16);
            }
          }
          if (elect_one()) {
            mma_commit(BAR(C::EMPTY + ks.slot));
            mbar_arrive(BAR(C::EMPTY + ks.slot));
          }
          __syncwarp();
          ks.skip(2);
        }
        for (int u = uq; u < uq + nq; ++u) commit(BAR(C::Q_EMPTY + (u & 1)));
        uq += nq;
      }
    } else {
      // O += P V of lane t
      const int t = warp == C::PV1;
      const uint32_t v_lo = sdesc_lo(sbase + C::OFF_R, C::KSUB_BYTES);
      Place vs = {1, 1, 0};
      int used = 0, g = 0;  // this lane's items and steps so far
      for (int i = 0; ok; ++i) {
        ServeItem it;
        if (!next_item(i, &it) || it.cnt < 0) break;
        const bool dual = it.flags & ITEM_DUAL;
        const int tiles = t ? it.c1 : it.c0;
        bool first = true;
        for (int k = 0; ok && k < it.cnt; ++k) {
          if (!(ok = landed(vs, k >= 4 && (dual || k < tiles), SITE_SW_V_FULL))) break;
          if (dual ? (k & 1) != t : k >= tiles) {  // the other lane's
            if (elect_one()) mbar_arrive(BAR(C::EMPTY + vs.slot));
            __syncwarp();
            vs.skip(2);
            continue;
          }
          const int j = it.j0 + k;
          const int rows = j < it.nc ? it.L - j * C::TK : it.n - (j - it.nc) * C::TK;
          const int halves = steps_in(it, t, j);
          if (rows < halves * C::KT) {
            // rows past the sequence may hold anything; P is 0 there, but 0 x NaN is not
            uint8_t* v = sm + C::OFF_R + vs.slot * C::TILE_BYTES + rows * 128;
            const int chunks = (halves * C::KT - rows) * 8;
            for (int z = lane; z < chunks * C::NSUB; z += 32)
              *reinterpret_cast<uint4*>(v + z / chunks * C::KSUB_BYTES + z % chunks * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          for (int h = 0; h < halves; ++h, ++g, first = false) {
            if (!(ok = wait_phase(BAR(C::P_READY + 2 * t + C::buf(g)), C::phase(g), st, SITE_SW_P_READY))) break;
            if (first && used > 0 && !(ok = wait_phase(BAR(C::O_FREE + t), (used - 1) & 1, st, SITE_SW_O_FREE))) break;
            tc_fence_after();
            const uint32_t va = v_lo + vs.slot * TILE16 + h * HALF16;
            const uint32_t d = tmem + C::tm_o(t), pa = tmem + C::tm_p(t, C::buf(g));
#pragma unroll
            for (int q = 0; q < C::KT / 16; ++q)
              if (elect_one()) mma_ts(d, pa + q * 8, sdesc_join(va + q * (2048 >> 4), HI), IDESC_O, !first || q > 0);
            commit(BAR(C::O_DONE + 2 * t + C::buf(g)));
          }
          if (!ok) break;
          commit(BAR(C::EMPTY + vs.slot));
          vs.skip(2);
        }
        used += tiles > 0;
      }
    }
    // every MMA issued has completed before TMEM is released
    commit(BAR(C::DRAIN));
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(BAR(C::DRAIN), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
    }
  } else {
    // ------------------------------------------------------------ softmax of lane t
    const int t = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;
    const int rn = row / a.G, rg = row - rn * a.G;  // token and head of the row within its tile
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const float sl2 = a.scale_log2;
    float* ml = reinterpret_cast<float*>(sm + C::OFF_ML);
    int st0 = 0, st1 = 0, merges = 0;  // steps of both lanes and joins of dual items so far
    int tiles8 = 0, news = 0, uq = 0;  // (C8) cached and new tiles, Q slots so far
    for (int i = 0;; ++i) {
      ServeItem it;
      if (!next_item(i, &it) || it.cnt < 0) break;
      const bool dual = it.flags & ITEM_DUAL, whole = it.flags & ITEM_WHOLE;
      const int steps = t ? it.s1 : it.s0, before = t ? st1 : st0;
      const int tok = it.tok0 + (dual ? 0 : t * npt) + rn;
      const bool valid = rn < npt && tok < it.n;
      const bool any = __any_sync(0xffffffffu, valid);
      float m_run = -INFINITY, l_run = 0.f, vref = 0.f;  // vref: (C8) to base 2
      bool ok = true;
      // (C8) of scores: what undoes the factor of the row's Q; there with the first S, and kept until this arrival
      float qf = 1.f;
      const int qslot = (uq + (dual ? 0 : t)) & 1;
      auto q_read = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::Q_EMPTY + qslot));
      };
      // Every use of both slots is waited for, in order, and the other lane's let go at once: the arrival may not count
      // for the use before, nor may a slot be two uses ahead of a wait for it.
      if (TURN) {
        for (int y = uq; ok && y < uq + (dual ? 1 : 2); ++y)
          ok = wait_phase(BAR(C::Q_FULL + (y & 1)), (y >> 1) & 1, st, SITE_SW_Q_FULL);
        if (!ok) break;
        if (!dual && lane == 0) mbar_arrive(BAR(C::Q_EMPTY + (qslot ^ 1)));
        if (steps == 0) q_read();
      }
      const int tok_first = __shfl_sync(0xffffffffu, tok, 0);  // the warp's tokens ascend with its rows
      auto wait_pv = [&](int lane_t, int g) {  // PV of that lane's step g has landed in O
        return wait_phase(BAR(C::O_DONE + 2 * lane_t + C::buf(g)), C::phase(g), st, SITE_SW_O_DONE);
      };
      const int stride = dual ? 2 : 1;
      int js = it.j0 + (dual ? t : 0), hs = 0, halves = steps_in(it, t, js);  // the step's key tile and half
      constexpr int KT = C::KT;
      auto begin_step = [&](int s) {  // its key tile and half; S is there
        if (C::HPT == 1 ? s > 0 && ++hs == halves : hs == halves) {
          hs = 0;
          js += stride;
          halves = steps_in(it, t, js);
        }
        return wait_phase(BAR(C::S_FULL + 2 * t + C::buf(before + s)), C::phase(before + s), st, SITE_SW_S_FULL);
      };
      auto s_in_registers = [&] {
        if (C::SEP_P) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(C::S_FREE + t));
        }
      };
      auto end_step = [&](int s, bool rescale, float f) {  // P is on its way; O of row `lane` takes the factor f
        if (rescale) {
          if (!C::SEP_P) {
            if (!wait_pv(t, before + s - 1)) return false;
            tc_fence_after();
          }
          const uint32_t tO = tmem + lane_off + C::tm_o(t);
          uint32_t r[32];
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            tmem_ld32(tO + q * 32, r);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * f);
            tmem_st32(tO + q * 32, r);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::P_READY + 2 * t + C::buf(before + s)));
        return true;
      };
      if (C8 || !(PAGED && any && it.n <= 16 && it.n * a.G <= 16)) {
        for (int s = 0; s < steps; ++s, hs += C::HPT > 1) {
          const int u = C::buf(before + s);
          if (!(ok = begin_step(s))) break;
          if (TURN && s == 0) {
            qf = qfs[qslot * 4 + (row >> 3 & 3)];
            q_read();
          }
          if (!any) {  // no row here: P stays what it is, its rows of O are nobody's
            __syncwarp();
            if (C::SEP_P) {
              if (lane == 0) mbar_arrive(BAR(C::S_FREE + t));
            }
            // d = 64: S of this tile may be there before the other warps have written P of the one
            // before: an arrival now would count for that one
            if (C::SEP_P && s > 0 && !(ok = wait_pv(t, before + s - 1))) break;
            if (lane == 0) mbar_arrive(BAR(C::P_READY + 2 * t + u));
            continue;
          }
          tc_fence_after();
          float f = 1.f, fv = 1.f;  // of O and l, and of O alone
          bool rescale = false;
          float sv[KT], ks[C8 ? KT / 16 : 1], w[C8 ? KT / 16 : 1];
          {
            uint32_t r[KT / 32][32];
#pragma unroll
            for (int q = 0; q < KT / 32; ++q) tmem_ld32(tmem + lane_off + C::tm_s(t, u) + q * 32, r[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < KT / 32; ++q)
#pragma unroll
              for (int x = 0; x < 32; ++x) sv[q * 32 + x] = __uint_as_float(r[q][x]);
          }
          s_in_registers();
          if constexpr (C8) {
            constexpr int GR = KT / 16;  // (4)
            float vs[GR];
            if (js < it.nc) {
              const float4* sc = reinterpret_cast<const float4*>(scales + (tiles8 + js - it.j0) % C::SCALES * 8);
              const float4 k4 = sc[0], v4 = sc[1];
              ks[0] = k4.x, ks[1] = k4.y, ks[2] = k4.z, ks[3] = k4.w;
              vs[0] = v4.x, vs[1] = v4.y, vs[2] = v4.z, vs[3] = v4.w;
            } else if (TURN) {
              const float4 f4 = reinterpret_cast<const float4*>(nscales)[(news + js - max(it.nc, it.j0)) % C::SCALES];
              ks[0] = ks[1] = f4.x, ks[2] = ks[3] = f4.y, vs[0] = vs[1] = f4.z, vs[2] = vs[3] = f4.w;
            } else {
#pragma unroll
              for (int x = 0; x < GR; ++x) ks[x] = vs[x] = 1.f;
            }
            // the reference of the values' scales, to base 2
            const float vtop = lg2_approx(fmax3(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]), 1.1754944e-38f));
            if (s == 0) {
              vref = vtop + 1.f;
            } else if (vtop > vref) {
              rescale = true, fv = ex2_approx(vref - (vtop + 1.f));
              vref = vtop + 1.f;
            }
#pragma unroll
            for (int x = 0; x < GR; ++x) {
              // Not 0, as -inf times it has to stay -inf: of zeros, or where there are no rows, qf and a key's factor are
              // 2^-114 each, and a block's scale 2^-118, so that their product is what has to be kept from 0.
              ks[x] = fmaxf(ks[x] * (sl2 * qf), 1.1754944e-38f);
              // not below 2^-40: what is that small adds nothing to O, but to the sum
              w[x] = fmaxf(lg2_approx(vs[x]) - vref, -40.f);
            }
          }
          if (tree && js >= it.nc) {
            const int k0 = (js - it.nc) * C::TK + hs * KT;
            const uint32_t* words = a.mask + (long long)(it.row0 + tok) * a.words;
            uint32_t w[KT / 32];
#pragma unroll
            for (int q = 0; q < KT / 32; ++q) {
              const int left = it.n - k0 - 32 * q;  // nodes from this word on
              w[q] = valid && left > 0 && (k0 >> 5) + q < a.words ? words[(k0 >> 5) + q] : 0u;
              if (left > 0 && left < 32) w[q] &= (1u << left) - 1;
            }
#pragma unroll
            for (int x = 0; x < KT; ++x)
              if (!(w[x >> 5] >> (x & 31) & 1)) sv[x] = -INFINITY;
          } else {
            // keys [0, lim) of the step are seen, by the warp's first row fewest
            const int k0 = js * C::TK + hs * KT - (js < it.nc ? it.L : it.nc * C::TK);
            if (js < it.nc ? k0 > -KT : min(it.n, tok_first + 1) < k0 + KT) {
              const int lim = js < it.nc ? -k0 : min(it.n, tok + 1) - k0;
#pragma unroll
              for (int x = 0; x < KT; ++x)
                if (x >= lim) sv[x] = -INFINITY;
            }
          }
          float m_tile;
          if constexpr (C8) {
            m_tile = -INFINITY;
#pragma unroll
            for (int x = 0; x < KT / 16; ++x) {
              float pm[2] = {fmax3(sv[16 * x], sv[16 * x + 1], sv[16 * x + 2]), fmax3(sv[16 * x + 3], sv[16 * x + 4], sv[16 * x + 5])};
#pragma unroll
              for (int y = 6; y < 14; y += 4) {
                pm[0] = fmax3(pm[0], sv[16 * x + y], sv[16 * x + y + 1]);
                pm[1] = fmax3(pm[1], sv[16 * x + y + 2], sv[16 * x + y + 3]);
              }
              m_tile = fmaxf(m_tile, ks[x] * fmax3(fmaxf(pm[0], pm[1]), sv[16 * x + 14], sv[16 * x + 15]));
            }
          } else {
            float pm[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) pm[y] = sv[y];
#pragma unroll
            for (int x = 4; x < KT - 4; x += 8)
#pragma unroll
              for (int y = 0; y < 4; ++y) pm[y] = fmax3(pm[y], sv[x + 2 * y], sv[x + 2 * y + 1]);
            const float mx = fmax3(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]),
                                   fmax3(sv[KT - 4], sv[KT - 3], fmaxf(sv[KT - 2], sv[KT - 1])));
            m_tile = mx * sl2;
          }
          // the reference maximum moves only when it grows by more than 2^LAG_LOG2; O and l share it
          if (s == 0) {
            m_run = m_tile;
          } else {
            const bool grow = valid && m_tile > m_run + LAG_LOG2;
            rescale |= __any_sync(0xffffffffu, grow);
            if (grow) {
              f = ex2_approx(m_run - m_tile);
              m_run = m_tile;
            }
          }
          const float nbase = P_LOG2 - (m_run == -INFINITY ? 0.f : m_run);
          const uint64_t sl2x2 = f2_pack(sl2, sl2), nbase2 = f2_pack(nbase, nbase);
          [[maybe_unused]] uint64_t ks2, nb2, sum16;
          [[maybe_unused]] float l_step = 0.f;
          uint64_t ps2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
          uint32_t pk[KT / 32][16];
          const uint32_t tP = tmem + lane_off + C::tm_p(t, u);
#pragma unroll
          for (int q = 0; q < KT / 32; ++q) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float x0, x1;
              if constexpr (C8) {  // w P, whose sums over 16 keys are divided by w again
                if ((x & 7) == 0) {
                  const float nb = nbase + w[2 * q + (x >> 3)];
                  ks2 = f2_pack(ks[2 * q + (x >> 3)], ks[2 * q + (x >> 3)]);
                  nb2 = f2_pack(nb, nb);
                }
                f2_unpack(f2_fma(f2_pack(sv[q * 32 + 2 * x], sv[q * 32 + 2 * x + 1]), ks2, nb2), x0, x1);
              } else {
                f2_unpack(f2_fma(f2_pack(sv[q * 32 + 2 * x], sv[q * 32 + 2 * x + 1]), sl2x2, nbase2), x0, x1);
              }
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              if constexpr (C8) {
                sum16 = (x & 7) == 0 ? f2_pack(p0, p1) : f2_add(sum16, f2_pack(p0, p1));
                if ((x & 7) == 7) {
                  float lo, hi;
                  f2_unpack(sum16, lo, hi);
                  l_step = fmaf(lo + hi, ex2_approx(-w[2 * q + (x >> 3)]), l_step);
                }
              } else {
                ps2[x & 1] = f2_add(ps2[x & 1], f2_pack(p0, p1));
              }
              pk[q][x] = pack2<H>(p0, p1);
            }
            if (C::SEP_P && q == 1) {
              if (s > 0) {  // PV of the tile before has read P (across items its epilogue waited for that)
                if (!(ok = wait_pv(t, before + s - 1))) break;
                tc_fence_after();
              }
              tmem_st16(tP, pk[0]);
              tmem_st16(tP + 16, pk[1]);
            }
            if (!C::SEP_P || q >= 2) tmem_st16(tP + q * 16, pk[q]);
          }
          if (!ok) break;
          float ps[4];
          f2_unpack(ps2[0], ps[0], ps[1]);
          f2_unpack(ps2[1], ps[2], ps[3]);
          l_run = l_run * f + (C8 ? l_step : (ps[0] + ps[1]) + (ps[2] + ps[3]));
          if (!(ok = end_step(s, rescale, C8 ? f * fv : f))) break;
        }
      } else {
        // Decoding and small drafts: up to 16 rows, in the first warp's lanes. A thread of it takes a quarter
        // of the keys of rows lane / 4 and lane / 4 + 8 rather than all of row `lane`: with the exponentials
        // of 32 rows a warp, decoding 512 sequences of up to 500 tokens took 332 us at d = 64 (12 heads)
        // instead of 255, and 217 at d = 128 (32 / 8 heads) instead of 209.
        const int tok_few[2] = {(lane >> 2) / a.G, ((lane >> 2) + 8) / a.G};
        float m_few[2] = {-INFINITY, -INFINITY}, l_few[2] = {0.f, 0.f};
        for (int s = 0; s < steps; ++s, hs += C::HPT > 1) {
          const int u = C::buf(before + s);
          if (!(ok = begin_step(s))) break;
          tc_fence_after();
          uint32_t r[KT / 64][32];
#pragma unroll
          for (int q = 0; q < KT / 64; ++q) tmem_ld_rows16(tmem + lane_off + C::tm_s(t, u) + q * 64, r[q]);
          tmem_wait_ld();
          s_in_registers();
          uint32_t pk[KT / 64][16];
          float fh[2] = {1.f, 1.f};
          bool grow = false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (h == 1 && it.n * a.G <= 8) {
#pragma unroll
              for (int y = 0; y < KT / 8; ++y) pk[y >> 3][2 * (y & 7) + 1] = 0;
              break;
            }
            float x[KT / 4];
#pragma unroll
            for (int y = 0; y < KT / 8; ++y) {
              x[2 * y] = __uint_as_float(r[y >> 3][4 * (y & 7) + 2 * h]);
              x[2 * y + 1] = __uint_as_float(r[y >> 3][4 * (y & 7) + 2 * h + 1]);
            }
            const int token = tok_few[h], c0 = 2 * (lane & 3);
            if (js >= it.nc) {  // at most 16 new tokens
              uint32_t seen = tree ? (token < it.n ? a.mask[(long long)(it.row0 + token) * a.words] : 0u)
                                   : (2u << min(token, 30)) - 1;
              seen &= (1u << it.n) - 1;
#pragma unroll
              for (int y = 0; y < KT / 8; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (y >= 4 || !(seen >> (8 * y + c0 + e) & 1)) x[2 * y + e] = -INFINITY;
            } else if (it.L - js * 128 - hs * KT < KT) {
              const int lim = it.L - js * 128 - hs * KT - c0;
#pragma unroll
              for (int y = 0; y < KT / 8; ++y)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (8 * y + e >= lim) x[2 * y + e] = -INFINITY;
            }
            float pm[2] = {x[0], x[1]};
#pragma unroll
            for (int y = 2; y < KT / 4 - 2; y += 4)
#pragma unroll
              for (int e = 0; e < 2; ++e) pm[e] = fmax3(pm[e], x[y + 2 * e], x[y + 2 * e + 1]);
            float mx = fmax3(fmaxf(pm[0], pm[1]), x[KT / 4 - 2], x[KT / 4 - 1]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_tile = mx * sl2;
            float& m = m_few[h];
            if (s == 0) {
              m = m_tile;
            } else if (token < it.n && m_tile > m + LAG_LOG2) {
              grow = true;
              fh[h] = ex2_approx(m - m_tile);
              m = m_tile;
            }
            const float nbase = P_LOG2 - (m == -INFINITY ? 0.f : m);
            const uint64_t sl2x2 = f2_pack(sl2, sl2), nbase2 = f2_pack(nbase, nbase);
            uint64_t ps2 = f2_pack(0.f, 0.f);
#pragma unroll
            for (int y = 0; y < KT / 8; ++y) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(x[2 * y], x[2 * y + 1]), sl2x2, nbase2), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              ps2 = f2_add(ps2, f2_pack(p0, p1));
              pk[y >> 3][2 * (y & 7) + h] = pack2<F16>(p0, p1);
            }
            float ps0, ps1;
            f2_unpack(ps2, ps0, ps1);
            l_few[h] = l_few[h] * fh[h] + (ps0 + ps1);
          }
          if (C::SEP_P && s > 0) {
            if (!(ok = wait_pv(t, before + s - 1))) break;
            tc_fence_after();
          }
#pragma unroll
          for (int q = 0; q < KT / 64; ++q) tmem_st_rows16(tmem + lane_off + C::tm_p(t, u) + q * 32, pk[q]);
          const bool rescale = __any_sync(0xffffffffu, grow);
          float f = 1.f;
          if (rescale) {
            const float fa = __shfl_sync(0xffffffffu, fh[0], 4 * (lane & 7));
            const float fb = __shfl_sync(0xffffffffu, fh[1], 4 * (lane & 7));
            f = lane < 8 ? fa : fb;
          }
          if (!(ok = end_step(s, rescale, f))) break;
        }
        // maximum and sum of row `lane`
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float l = l_few[h];
          l += __shfl_xor_sync(0xffffffffu, l, 1);
          l += __shfl_xor_sync(0xffffffffu, l, 2);
          const float mr = __shfl_sync(0xffffffffu, m_few[h], 4 * (lane & 7)), lr = __shfl_sync(0xffffffffu, l, 4 * (lane & 7));
          if ((lane >> 3) == h) m_run = mr, l_run = lr;
        }
      }
      if (ok && steps > 0) ok = wait_pv(t, before + steps - 1);
      if (!ok) break;
      tc_fence_after();
      const bool join = dual && it.c1 > 0;
      float f0 = 1.f, f1 = 0.f;  // weights of this lane's O and of the other's
      if (join) {
        ml[256 * t + row] = m_run;
        ml[256 * t + 128 + row] = l_run;
        if (C8 && row == 0) vrefs[t] = vref;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::MERGE));
        if (!wait_phase(BAR(C::MERGE), merges & 1, st, SITE_SW_MERGE) ||
            !wait_pv(t ^ 1, t ? st0 + it.s0 - 1 : st1 + it.s1 - 1))
          break;
        tc_fence_after();
        const float* other = ml + 256 * (t ^ 1) + row;
        const float m = fmaxf(m_run, other[0]), base = m == -INFINITY ? 0.f : m;
        f0 = ex2_approx(m_run - base);
        f1 = ex2_approx(other[0] - base);
        l_run = l_run * f0 + other[128] * f1;
        m_run = m;
        ++merges;
      }
      st0 += it.s0;
      st1 += it.s1;
      if (C8) {
        const int here = max(0, min(it.nc - it.j0, it.cnt));
        tiles8 += here, news += it.cnt - here, uq += dual ? 1 : 2;
      }
      if (dual && t == 1 && !join) continue;  // lane 0 has all of them
      if constexpr (C8) {  // scores of -inf alone, of an infinite query say: no maximum to take off, the row is NaN
        if (l_run == 0.f && valid && steps > 0 &&
            sees_a_key(a.mask, a.words, it.row0 + tok, tok, it.n, it.j0 < it.nc, max(0, it.j0 - it.nc) * C::TK,
                       (it.j0 + it.cnt - it.nc) * C::TK))
          l_run = NAN;
      }
      // l = 0: no key; NaN stays NaN
      const float inv = l_run != 0.f ? 1.f / l_run : 0.f;
      const float lse2 = l_run != 0.f ? m_run - P_LOG2 + lg2_approx(l_run) : -INFINITY;
      const long long part = (long long)it.slot * 256 + (dual ? 0 : t * 128) + row;
      if (steps == 0) {  // (a cut item only) none of this part's keys concerns this tile
        if (valid && FA_CHECK(in_range(part, a.part_rows), st, DBG_GLOBAL_STORE)) a.part_lse[part] = -INFINITY;
        continue;
      }
      const int head = it.kvh * a.G + rg;
      const long long token = it.row0 + tok;
      f0 *= inv;
      f1 *= inv;
      if (C8) {
        f0 *= exp2f(vref);
        if (join) f1 *= exp2f(vrefs[t ^ 1]);
      }
      const bool write = valid && FA_CHECK(whole ? in_range(token, a.T - FA_SLACK(a)) : in_range(part, a.part_rows), st, DBG_GLOBAL_STORE);
      uint16_t* orow = a.o + token * a.o_st + head * a.o_sh;
      float* prow = a.part_o + part * D;
      // in a join each lane takes half of the columns
      const int q0 = join ? t * (D / 64) : 0, q1 = join ? q0 + D / 64 : D / 32;
      if (any) {
#pragma unroll 1
        for (int q = q0; q < q1; ++q) {
          uint32_t r[32];
          float v[32];
          tmem_ld32(tmem + lane_off + C::tm_o(t) + q * 32, r);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = __uint_as_float(r[x]) * f0;
          if (join) {
            tmem_ld32(tmem + lane_off + C::tm_o(t ^ 1) + q * 32, r);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = fmaf(__uint_as_float(r[x]), f1, v[x]);
          }
          if (q == q1 - 1) {  // O is in registers: the issuers may write it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_n(BAR(C::O_FREE + t), join ? 1 : 2);
              if (join) mbar_arrive(BAR(C::O_FREE + (t ^ 1)));
            }
          }
          // a thread writes a row: whole sectors where the rows allow it
          if (write && whole) {
            uint32_t y[2][8];
#pragma unroll
            for (int x = 0; x < 16; ++x) y[x >> 3][x & 7] = pack2<F16>(v[2 * x], v[2 * x + 1]);
            if (a.o_wide) {
              store_32b(orow + q * 32, y[0]);
              store_32b(orow + q * 32 + 16, y[1]);
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint4*>(orow + q * 32 + x * 8) =
                    make_uint4(y[x >> 1][(x & 1) * 4], y[x >> 1][(x & 1) * 4 + 1], y[x >> 1][(x & 1) * 4 + 2],
                               y[x >> 1][(x & 1) * 4 + 3]);
            }
          } else if (write) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t y[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) y[z] = __float_as_uint(v[8 * x + z]);
              store_32b(prow + q * 32 + x * 8, y);
            }
          }
        }
        if (write && q0 == 0) {
          if (!whole)
            a.part_lse[part] = lse2;
          else if (a.lse)
            a.lse[(long long)head * a.T + token] = lse2 * 0.6931471805599453f;
        }
      } else if (lane == 0) {
        mbar_arrive_n(BAR(C::O_FREE + t), join ? 1 : 2);
        if (join) mbar_arrive(BAR(C::O_FREE + (t ^ 1)));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::PV0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

// Joins the partial results of the items that CTA boundaries cut: block (x, y) takes rows
// [32 y, 32 y + 32) of the item that boundary x + 1 is the first to cut. A warp a row at d = 128,
// half a warp at d = 64; the parts' weights come from their LSEs, as between key tiles. Latency
// bounds it: a record says whether there is a cut, and most blocks end there (finding the cuts again
// in every block took 2 us more).
template <int D, bool F16>
__global__ void __launch_bounds__(256) serve_join_kernel(ServeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int npt = 128 / a.G, c = blockIdx.x + 1;
  const int parts = a.cuts[2 * c].x + 1;  // part 0: CTA c - 1's last item; then the first items of c, c + 1, ..
  if (parts == 1) return;
  const int4 cut = a.cuts[2 * c + 1];  // tokens of the sequence, its first row, the item's first token, head
  constexpr int LPR = D / 4;  // lanes a row
  const int sub = threadIdx.x % LPR;
  for (int row = blockIdx.y * 32 + threadIdx.x / LPR; row < blockIdx.y * 32 + 32; row += 256 / LPR) {
    const int rr = row & 127, rn = rr / a.G, rg = rr - rn * a.G;
    const int tok = cut.z + (row >> 7) * npt + rn;
    if (rn >= npt || tok >= cut.x) continue;
    auto at = [&](int k) { return (long long)(k == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + k)) * 256 + row; };
    if (!FA_CHECK(in_range(at(0), a.part_rows) && in_range(at(parts - 1), a.part_rows), a.status, DBG_GLOBAL_LOAD) ||
        !FA_CHECK(in_range(cut.y + tok, a.T - FA_SLACK(a)) && in_range(cut.w, a.Hkv), a.status, DBG_GLOBAL_STORE))
      continue;
    float m = -INFINITY;
    for (int k = 0; k < parts; ++k) m = fmaxf(m, a.part_lse[at(k)]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) {
      const float s = a.part_lse[at(k)];
      if (s == -INFINITY) continue;  // nothing was written there
      const float w = ex2_approx(s - base);
      const float4 x = *reinterpret_cast<const float4*>(a.part_o + at(k) * D + 4 * sub);
      l += w;
      o.x = fmaf(w, x.x, o.x), o.y = fmaf(w, x.y, o.y), o.z = fmaf(w, x.z, o.z), o.w = fmaf(w, x.w, o.w);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int h = cut.w * a.G + rg;
    const long long token = cut.y + tok;
    *reinterpret_cast<uint2*>(a.o + token * a.o_st + h * a.o_sh + 4 * sub) =
        make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
    if (sub == 0 && a.lse)
      a.lse[(long long)h * a.T + token] = (l != 0.f ? m + lg2_approx(l) : -INFINITY) * 0.6931471805599453f;
  }
}

template <int D, bool F16, bool PAGED, bool C8 = false>
static int launch_serve_d(std::conditional_t<C8, Serve8BitArgs, ServeArgs> a, cudaStream_t stream) {
  using C = ServeCfg<D, C8>;
  const auto type = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap mq, mk, mv, mkc = {}, mvc = {};
  auto map3 = [&](CUtensorMap* m, const uint16_t* p, long long st, long long sh, bool heads_inner, int heads, int box1,
                  int box2) {
    const cuuint64_t T = (cuuint64_t)a.T, H = (cuuint64_t)heads, sT = (cuuint64_t)st * 2, sH = (cuuint64_t)sh * 2;
    const cuuint64_t dims[3] = {D, heads_inner ? H : T, heads_inner ? T : H};
    const cuuint64_t strides[2] = {heads_inner ? sH : sT, heads_inner ? sT : sH};
    const cuuint32_t box[3] = {64, (cuuint32_t)box1, (cuuint32_t)box2};
    return make_tmap_strided(m, p, type, 3, dims, strides, box);
  };
  auto map4 = [&](CUtensorMap* m, const uint16_t* p) {
    const int page = 1 << a.page_shift;
    const cuuint64_t dims[4] = {D, (cuuint64_t)page, (cuuint64_t)a.Hkv, (cuuint64_t)a.n_pages};
    const cuuint64_t elem = C8 ? 1 : 2;
    const cuuint64_t strides[3] = {(cuuint64_t)a.c_st * elem, (cuuint64_t)a.c_sh * elem, (cuuint64_t)a.c_sp * elem};
    const cuuint32_t box[4] = {C8 ? D : 64, (cuuint32_t)std::min(page, C::TK), 1, 1};
    return make_tmap_strided(m, p, C8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type, 4, dims, strides, box,
                             C8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  };
  const int box = PAGED ? kNewBox : 128;
  if (!map3(&mq, a.q, a.q_st, a.q_sh, true, a.Hq, a.G, 128 / a.G) || !map3(&mk, a.k, a.k_st, a.k_sh, false, a.Hkv, box, 1) ||
      !map3(&mv, a.v, a.v_st, a.v_sh, false, a.Hkv, box, 1) || (PAGED && (!map4(&mkc, a.kc) || !map4(&mvc, a.vc))))
    return cuda_fail("cuTensorMapEncodeTiled", 0, "tensor map rejected");
  const auto kernel = serve_kernel<D, F16, PAGED, C8>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute", (int)e, cudaGetErrorName(e));
  int sms = 0;
  if (!sm_count(&sms)) return FA_ERR_CUDA;
  int grid = sms;
  if (!PAGED) {  // no more CTAs than there may be items of one query tile
    const int npt = 128 / a.G;
    grid = (int)std::min<long long>(sms, ((a.T + npt - 1) / npt + (long long)a.B) * a.Hkv);
  }
  int rc = launch_pdl("serve_kernel", kernel, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, stream, mq, mk, mv, mkc, mvc, a);
  if (rc != FA_OK || !PAGED || grid < 2) return rc;
  return launch_pdl("serve_join_kernel", serve_join_kernel<D, F16>, dim3(grid - 1, 8), dim3(256), 0, stream,
                    static_cast<const ServeArgs&>(a));
}

static int launch_serve(const ServeArgs& a, int d, int dtype, cudaStream_t stream) {
  const bool f16 = dtype == FA_FP16, paged = a.table != nullptr;
#define FA_SERVE(DD, FF) (paged ? launch_serve_d<DD, FF, true>(a, stream) : launch_serve_d<DD, FF, false>(a, stream))
  if (d == 64) return f16 ? FA_SERVE(64, true) : FA_SERVE(64, false);
  return f16 ? FA_SERVE(128, true) : FA_SERVE(128, false);
#undef FA_SERVE
}

}  // namespace fa

namespace {

using namespace fa::host;

int forward(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse, const fa_pages* cache,
            const fa_scales* scales, const int32_t* lens, const int32_t* cu, const uint32_t* mask, int words, int B, int T,
            int Hq, int Hkv, int d, int dtype, float scale, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  for (const fa_rows* r : {q, k, v, o})
    if (const int rc = check_rows(r); rc != FA_OK) return rc;
  if (!cu || (cache && !workspace)) return FA_ERR_INVALID_ARG;
  if ((lse && !aligned16(lse)) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if (cache && workspace_bytes < fa_forward_tree_workspace_size(d)) return FA_ERR_INVALID_ARG;
  int err = FA_OK;
  int* status = fa::status_word(&err);
  if (!status) return err;
  fa::Serve8BitArgs a = {};
  a.q = static_cast<const uint16_t*>(q->data);
  a.k = static_cast<const uint16_t*>(k->data);
  a.v = static_cast<const uint16_t*>(v->data);
  a.o = static_cast<uint16_t*>(o->data);
  a.q_st = q->token_stride, a.q_sh = q->head_stride;
  a.k_st = k->token_stride, a.k_sh = k->head_stride;
  a.v_st = v->token_stride, a.v_sh = v->head_stride;
  a.o_st = o->token_stride, a.o_sh = o->head_stride;
  a.lse = lse;
  a.o_wide = (reinterpret_cast<uintptr_t>(o->data) & 31u) == 0 && o->token_stride % 16 == 0 && o->head_stride % 16 == 0;
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
  FA_DEBUG_ARGS(a, B);
  int sms = 0;
  if (!fa::sm_count(&sms)) return FA_ERR_CUDA;
  a.part_rows = 2LL * sms * 256;
  a.part_o = static_cast<float*>(workspace);
  a.part_lse = a.part_o + a.part_rows * d;
  a.cuts = reinterpret_cast<int4*>(a.part_lse + a.part_rows);
  a.status = status;
  const auto st = reinterpret_cast<cudaStream_t>(stream);
  if (!scales) return fa::launch_serve(a, d, dtype, st);
  a.ks = scales->k, a.vs = scales->v, a.s_sp = scales->page_stride, a.s_sh = scales->head_stride;
  a.block_shift = log2_of(scales->block);
  // Few rows a sequence on the average (the lengths are on the device) have a kernel of their own; in fp16 more parts of P
  // and Q cost it more. 32 sequences of some 30 rows, there and here: at d = 128, 8 heads, 122 and 168 us over 8192 tokens
  // and 42 and 49 over 1024 (fp16 128 and 159, 46 and 44); at d = 64 in bf16 72 and 82 over 4096 (8 heads), 45 both over
  // 700 (12 heads); in fp16, 12 heads, 106 and 112 over 4096, but 46 and 37 over 700.
  const long long few = d == 64 && dtype == FA_FP16 ? 16 : 32;
  if ((long long)T * a.G <= few * B) return fa::launch_serve8(k, v, cache, a, d, dtype, st);
  const bool f16 = dtype == FA_FP16;
  if (d == 64) return f16 ? fa::launch_serve_d<64, true, true, true>(a, st) : fa::launch_serve_d<64, false, true, true>(a, st);
  return f16 ? fa::launch_serve_d<128, true, true, true>(a, st) : fa::launch_serve_d<128, false, true, true>(a, st);
}

}  // namespace

extern "C" {

size_t fa_forward_tree_workspace_size(int d) {
  if (d != 64 && d != 128) return 0;
  int sms = 0;
  if (!fa::sm_count(&sms)) return 0;
  return (size_t)2 * sms * 256 * (d + 1) * 4 + (size_t)sms * 2 * sizeof(int4);
}

int fa_forward_prompt(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                      const int32_t* cu_seqlens, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                      fa_stream_t stream) {
  const int rc = check_sizes(B, T, Hq, Hkv, d, dtype, scale);
  if (rc != FA_OK) return rc;
  if (B == 0 || T == 0) return FA_OK;
  return forward(q, k, v, o, lse, nullptr, nullptr, nullptr, cu_seqlens, nullptr, 0, B, T, Hq, Hkv, d, dtype, scale, nullptr, 0,
                 stream);
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
  return forward(q, k, v, o, lse, cache, nullptr, lens, cu_nodes, mask, mask_words, B, T, Hq, Hkv, d, dtype, scale,
                 workspace, workspace_bytes, stream);
}

size_t fa_forward_tree_8bit_workspace_size(int d) { return fa_forward_tree_workspace_size(d); }

int fa_forward_tree_8bit(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, float* lse,
                         const fa_pages* cache, const fa_scales* scales, const int32_t* lens, const int32_t* cu_nodes,
                         const uint32_t* mask, int mask_words, int B, int T, int Hq, int Hkv, int d, int dtype, float scale,
                         void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  int rc = check_sizes(B, T, Hq, Hkv, d, dtype, scale);
  if (rc != FA_OK) return rc;
  if (mask && (mask_words < 1 || mask_words > (1 << 20))) return mask_words < 1 ? FA_ERR_INVALID_ARG : FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if ((rc = check_pages(cache, 16)) != FA_OK || (rc = check_scales(scales, cache->page_size)) != FA_OK) return rc;
  if (!lens) return FA_ERR_INVALID_ARG;
  return forward(q, k, v, o, lse, cache, scales, lens, cu_nodes, mask, mask_words, B, T, Hq, Hkv, d, dtype, scale, workspace,
                 workspace_bytes, stream);
}

}  // extern "C"
