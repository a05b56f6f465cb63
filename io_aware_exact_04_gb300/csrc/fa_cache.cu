// The cache in pages: tokens written into their pages, slots updated (forked, trimmed, freed,
// grown), pages compacted; and the visibility bits of a drafted tree.
#include <cuda_runtime.h>

#include <algorithm>

#include "fa_internal.h"
#include "serve.cuh"

namespace fa {

// ---------------------------------------------------------------------------------------------
// Bits of a tree: node i sees itself and what its parent sees. A block takes a sequence, 256 nodes
// after the other: a thread walks the chain of one node as long as it stays among these (in shared
// memory, as a step of the walk waits for the one before; every step goes to a smaller index, so that
// it ends whatever the parents are), and the rest of the row is that of the first ancestor before
// them, which is written already. So a step walks 256 nodes at most and copies a row, however long
// the chains are: a chain of 32768 nodes takes 14 ms, 64 trees of 64 nodes 2.1 us. Walked to its root
// by every node the chain took 873 ms; steps of 128 nodes took half again as long for trees of 256
// to 4096 nodes, steps of 512 longer for chains of up to 128.
constexpr int kTreeNodes = 256;
__global__ void __launch_bounds__(kTreeNodes) tree_mask_kernel(const int* parents, const int* cu, uint32_t* mask, int words,
                                                               int B, int T, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int parent[kTreeNodes];
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const SeqRange r = seq_range(cu, b, T, status);
  const int n = r.hi - r.lo;
  if (n > 32 * words && threadIdx.x == 0) record_check(status, SITE_S_WORDS);
  for (int c0 = 0; c0 < n; c0 += kTreeNodes) {
    const int i = c0 + threadIdx.x, w0 = c0 >> 5;
    if (i < n) parent[threadIdx.x] = parents[r.lo + i];
    __syncthreads();  // also: the rows of the nodes before are written
    uint32_t bits[kTreeNodes / 32] = {};
    int before = -1;  // the first ancestor before c0
    for (int j = i < n ? i : -1; j >= c0;) {
#pragma unroll
      for (int q = 0; q < kTreeNodes / 32; ++q) bits[q] |= ((j - c0) >> 5) == q ? 1u << (j & 31) : 0u;
      const int p = parent[j - c0];
      if (p >= j) record_check(status, SITE_S_PARENT);
      if (p < 0 || p >= j) break;
      if (p < c0) before = p;
      j = p;
    }
    if (i < n) {
      uint32_t* row = mask + (long long)(r.lo + i) * words + w0;
#pragma unroll
      for (int q = 0; q < kTreeNodes / 32; ++q)
        if (w0 + q < words) row[q] = bits[q];
    }
    if (c0 > 0 || words > kTreeNodes / 32) {
      // the other words of the warp's 32 rows, 32 words a step in the order of the rows, four steps' loads at a time
      const int first = c0 + (threadIdx.x & ~31), rows = min(32, n - first);
      const int dk = 32 / words, dw = 32 - dk * words;
      int k = lane / words, w = lane - k * words;
      for (long long left = (long long)rows * words; left > 0; left -= 4 * 32) {
        uint32_t x[4], *to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int of = __shfl_sync(0xffffffffu, before, k & 31);
          const bool mine = k < rows && (w < w0 || w >= w0 + kTreeNodes / 32);
          to[u] = mine ? mask + (long long)(r.lo + first + k) * words + w : nullptr;
          x[u] = mine && w < w0 && of >= 0 ? mask[(long long)(r.lo + of) * words + w] : 0;
          k += dk, w += dw;
          if (w >= words) ++k, w -= words;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (to[u]) *to[u] = x[u];
      }
    }
    __syncthreads();  // the parents have been read
  }
}

// ---------------------------------------------------------------------------------------------
struct AppendArgs {
  const uint16_t *k, *v;
  long long k_st, k_sh, v_st, v_sh;
  uint16_t *kc, *vc;
  long long c_sp, c_sh, c_st;
  int n_pages, page_shift;
  const int* table;
  long long table_stride;
  int table_width;
  const int *start, *cu, *rows;
  int B, T, Tkv, Hkv;
  int* status;
};

// A warp for each token: its head rows are whole lines on both sides, 16 bytes a lane. The longest
// prompts (72 MB moved) take 10.3 us, the measured copy rate; a step's accepted tokens 3.5 us, the
// latency of finding the sequence, its page and the row.
template <int D>
__global__ void __launch_bounds__(128) cache_append_kernel(AppendArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (blockIdx.x == 0) check_offsets(a.cu, a.B, a.T, a.status);
  if (t >= a.T) return;
  const int b = find_sequence(a.cu, a.B, t);
  if (b < 0) return;
  const SeqRange r = seq_range(a.cu, b, a.T, a.status);
  if (t < r.lo || t >= r.hi) return;
  const long long pos = (long long)a.start[b] + (t - r.lo);
  if (pos < 0 || pos >= (long long)a.table_width << a.page_shift) return record_check(a.status, SITE_S_LENGTH);
  const int id = a.table[b * a.table_stride + (pos >> a.page_shift)];
  if (id < 0 || id >= a.n_pages) return record_check(a.status, SITE_S_PAGE);
  const int row = a.rows ? a.rows[t] : t;
  if (row < 0 || row >= a.Tkv) return record_check(a.status, SITE_S_ROW);
  const long long to = id * a.c_sp + (pos & ((1 << a.page_shift) - 1)) * a.c_st;
  for (int i = lane; i < a.Hkv * (D / 8); i += 32) {
    const int h = i / (D / 8), c = i % (D / 8) * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(a.k + row * a.k_st + h * a.k_sh + c);
    const uint4 y = *reinterpret_cast<const uint4*>(a.v + row * a.v_st + h * a.v_sh + c);
    *reinterpret_cast<uint4*>(a.kc + to + h * a.c_sh + c) = x;
    *reinterpret_cast<uint4*>(a.vc + to + h * a.c_sh + c) = y;
  }
}

// ---------------------------------------------------------------------------------------------
// Slots and pages: a plan, made by one cluster of eight CTAs (the counts of all pages have to be
// complete before the free ones are numbered; a cluster's barrier costs less than another launch:
// compacting a small pool took 44 us of the host with five launches and 39 beside it with two), and its
// execution by the whole GPU. Each phase of the plan waits for L2: 10-12 us in all. Workspace, in
// ints: head [64], uses [n_pages], pages [n_pages] (new pages, or where a page goes), slots [slots] x 2,
// copies [slots] x 3, moves [n_pages] x 2, the table as it was.
struct PoolArgs {
  uint8_t* data;
  long long plane_bytes;
  int planes, n_pages, Hkv, page_shift, row_bytes;
  int *table, *lens;
  int slots, width;
  const int *src, *fresh;  // update only
  int* info;
  int* status;
  int *head, *uses, *pages, *slot, *copies, *moves, *old;
  float* scales;  // of a pool in 8 bits, else null: [planes][n_pages][Hkv][blocks]
  long long scale_plane;
  int blocks, block_shift;
};
constexpr int kPlanCtas = 8, kPlanThreads = 1024;
enum { H_ERR = 0, H_NEED, H_FREE, H_COPIES, H_MOVES, H_COUNT = 8, H_HOLES = 16, H_HIGH = 24 };  // the last three: one a CTA
constexpr int kWasUsed = 1 << 30;

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// All CTAs of the cluster, and what they wrote to global memory.
__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void pool_error(const PoolArgs& a, int site) {
  a.head[H_ERR] = 1;
  record_check(a.status, site);
}

// The sum over the block's threads below this one, and the block's total.
__device__ __forceinline__ int block_scan(int x, int* total, int* sh) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int y = x;
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  if (lane == 31) sh[w] = y;
  __syncthreads();
  if (w == 0) {
    int v = sh[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += z;
    }
    sh[lane] = v;
  }
  __syncthreads();
  *total = sh[31];
  const int before = y - x + (w ? sh[w - 1] : 0);
  __syncthreads();
  return before;
}

// Of slot s, by a warp: its pages are marked as used, its table row is kept and, for an update,
// the pages that it will share are counted.
template <bool UPDATE>
__device__ void mark_slot(const PoolArgs& a, int s) {
  const int lane = threadIdx.x & 31, cap = a.width << a.page_shift;
  const int len = a.lens[s];
  if (len < 0 || len > cap) return pool_error(a, SITE_S_LENGTH);
  const int n = pages_of(len, a.page_shift);
  for (int j = lane; j < n; j += 32) {
    const int id = a.table[(long long)s * a.width + j];
    if (UPDATE) a.old[(long long)s * a.width + j] = id;
    if (id < 0 || id >= a.n_pages) {
      pool_error(a, SITE_S_PAGE);
      continue;
    }
    atomicOr(&a.uses[id], kWasUsed);
  }
  if (!UPDATE) return;
  const int t = a.src[s], want = a.fresh[s];
  if (t < 0 || t >= a.slots) return pool_error(a, SITE_S_SLOT);
  if (want < 0 || want > cap) return pool_error(a, SITE_S_LENGTH);
  const int keep = min(want, min(max(a.lens[t], 0), cap));
  const int shared = (keep >> a.page_shift) + (t == s && (keep & ((1 << a.page_shift) - 1)) != 0);
  for (int j = lane; j < shared; j += 32) {
    const int id = a.table[(long long)t * a.width + j];
    if (id >= 0 && id < a.n_pages) atomicAdd(&a.uses[id], 1);
  }
}

// How many pages each slot keeps, where its new ones start, and which partly kept pages are copied;
// by one CTA.
__device__ void plan_slots(const PoolArgs& a, int* sh) {
  int need = 0, copies = 0, total;
  for (int s0 = 0; s0 < a.slots; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    int mine = 0, copy = 0, kept = 0, part = 0, page = 0;
    if (s < a.slots) {
      const int t = a.src[s], keep = min(a.fresh[s], a.lens[t]);
      part = keep & ((1 << a.page_shift) - 1);
      kept = keep >> a.page_shift;
      if (part) {
        page = a.table[(long long)t * a.width + kept];
        copy = !(t == s && (__ldcg(&a.uses[page]) & (kWasUsed - 1)) == 1);
        kept += !copy;
      }
      mine = pages_of(a.fresh[s], a.page_shift) - kept;
    }
    const int before = block_scan(mine, &total, sh);
    if (s < a.slots) {
      a.slot[2 * s] = kept;
      a.slot[2 * s + 1] = need + before;
    }
    need += total;  // at most slots x width
    const int at = block_scan(copy, &total, sh);
    if (copy) {
      int* c = a.copies + 3 * (copies + at);
      c[0] = s, c[1] = page, c[2] = part;
    }
    copies += total;
  }
  if (threadIdx.x == 0) {
    a.info[0] = need;
    a.head[H_NEED] = need;
    a.head[H_COPIES] = copies;
  }
}

template <bool UPDATE>
__global__ void __launch_bounds__(kPlanThreads) pool_plan_kernel(PoolArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int sh[32];
  const int tid = threadIdx.x, rank = blockIdx.x, warp = tid >> 5;  // the grid is one cluster
  // this CTA's share of the pages
  const int chunk = (a.n_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(a.n_pages, rank * chunk), hi = min(a.n_pages, lo + chunk);
  for (int p = lo + tid; p < hi; p += kPlanThreads) a.uses[p] = 0;
  if (rank == 0 && tid < 8) a.head[tid] = 0;
  cluster_sync();
  for (int s = rank * 32 + warp; s < a.slots; s += 32 * kPlanCtas) mark_slot<UPDATE>(a, s);
  cluster_sync();
  if (__ldcg(&a.head[H_ERR])) {  // (the same for every CTA)
    if (rank == 0 && tid < 2) a.info[tid] = -1;
    return;
  }
  // pages in use of each share, then what lies before this one
  int total, n = 0;
  for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    n += __syncthreads_count(p < hi && __ldcg(&a.uses[p]) != 0);
  }
  if (tid == 0) a.head[H_COUNT + rank] = n;
  if (UPDATE && rank == kPlanCtas - 1) plan_slots(a, sh);
  cluster_sync();
  int used = 0, used_before = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int x = __ldcg(&a.head[H_COUNT + r]);
    used += x;
    used_before += r < rank ? x : 0;
  }
  if (UPDATE) {  // the free pages, ascending
    int at = lo - used_before;
    for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
      const int p = p0 + tid;
      const int is_free = p < hi && __ldcg(&a.uses[p]) == 0;
      const int before = block_scan(is_free, &total, sh);
      if (is_free) a.pages[at + before] = p;
      at += total;
    }
    if (rank == 0 && tid == 0) a.info[1] = a.head[H_FREE] = a.n_pages - used;
    return;
  }
  // compaction: pages in use at or past `used` move to free ones below it
  int holes = 0, high = 0;
  for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const bool in_use = p < hi && __ldcg(&a.uses[p]) != 0;
    holes += __syncthreads_count(p < hi && p < used && !in_use);
    high += __syncthreads_count(p >= used && in_use);
  }
  if (tid == 0) a.head[H_HOLES + rank] = holes, a.head[H_HIGH + rank] = high;
  cluster_sync();
  int at_hole = 0, at_high = 0, moves = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int x = __ldcg(&a.head[H_HOLES + r]), y = __ldcg(&a.head[H_HIGH + r]);
    at_hole += r < rank ? x : 0;
    at_high += r < rank ? y : 0;
    moves += y;
  }
  for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const bool in_use = p < hi && __ldcg(&a.uses[p]) != 0;
    const int hole = p < hi && p < used && !in_use, goes = p >= used && in_use;
    int before = block_scan(hole, &total, sh);
    if (hole) a.moves[2 * (at_hole + before) + 1] = p;
    at_hole += total;
    before = block_scan(goes, &total, sh);
    if (goes) a.moves[2 * (at_high + before)] = p;
    if (p < hi) a.pages[p] = goes ? -1 - (at_high + before) : p;
    at_high += total;
  }
  if (rank == 0 && tid == 0) {
    a.info[0] = used;
    a.info[1] = moves;
    a.head[H_MOVES] = moves;
  }
}

// A warp copies up to kCopyChunks x 512 bytes, all loads before the stores: with four blocks of eight
// warps an SM, 128 KB of loads in flight there.
constexpr int kCopyChunks = 8, kCopyBytes = kCopyChunks * 512;
__device__ __forceinline__ void warp_copy(uint8_t* to, const uint8_t* from, int bytes) {
  const int lane = threadIdx.x & 31, n = bytes / 16;
  const uint4* f = reinterpret_cast<const uint4*>(from);
  uint4* t = reinterpret_cast<uint4*>(to);
  uint4 x[kCopyChunks];
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c)
    if (c * 32 + lane < n) x[c] = __ldcs(f + c * 32 + lane);
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c)
    if (c * 32 + lane < n) __stcs(t + c * 32 + lane, x[c]);
}

// The table rows (a warp each), then the kept rows of the pages that are copied: a warp a plane, head
// and kCopyBytes. Memory bounds it where much is copied: 256 slots and 51 MB in 11 us.
__global__ void __launch_bounds__(256) update_apply_kernel(PoolArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (a.head[H_ERR] || a.head[H_NEED] > a.head[H_FREE]) return;
  const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
  for (int s = warp; s < a.slots; s += warps) {
    const int kept = a.slot[2 * s], off = a.slot[2 * s + 1], want = a.fresh[s], n = pages_of(want, a.page_shift);
    const int* row = a.old + (long long)a.src[s] * a.width;
    for (int j = lane; j < a.width; j += 32)
      a.table[(long long)s * a.width + j] = j < kept ? row[j] : j < n ? a.pages[off + j - kept] : -1;
    if (lane == 0) a.lens[s] = want;
  }
  const int head_bytes = a.row_bytes << a.page_shift;  // one head's rows of a page: at most 64 KB
  const int parts = (head_bytes + kCopyBytes - 1) / kCopyBytes;
  const long long units = (long long)a.head[H_COPIES] * a.planes * a.Hkv * parts;
  for (long long u = warp; u < units; u += warps) {
    const int part = (int)(u % parts), h = (int)(u / parts % a.Hkv);
    const long long v = u / parts / a.Hkv;
    const int x = (int)(v % a.planes), c = (int)(v / a.planes);
    const int s = a.copies[3 * c], of = a.copies[3 * c + 1], bytes = a.copies[3 * c + 2] * a.row_bytes - part * kCopyBytes;
    if (bytes <= 0) continue;
    const int to = a.pages[a.slot[2 * s + 1]];  // the slot's first new page
    uint8_t* plane = a.data + x * a.plane_bytes + part * kCopyBytes;
    warp_copy(plane + ((long long)to * a.Hkv + h) * head_bytes, plane + ((long long)of * a.Hkv + h) * head_bytes,
              min(bytes, kCopyBytes));
    if (part == 0 && a.scales) {  // of the blocks that hold kept tokens: at most 16
      float* x8 = a.scales + x * a.scale_plane;
      if (lane <= (a.copies[3 * c + 2] - 1) >> a.block_shift)
        x8[((long long)to * a.Hkv + h) * a.blocks + lane] = x8[((long long)of * a.Hkv + h) * a.blocks + lane];
    }
  }
}

// The table, then the moved pages, a warp a plane and kCopyBytes: 4.04 GB in 641 us, 93 % of the measured
// copy rate (one 16-byte load in flight a thread: 717 us).
__global__ void __launch_bounds__(256) compact_apply_kernel(PoolArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  if (a.head[H_ERR]) return;
  const int lane = threadIdx.x & 31, warps = gridDim.x * 8;
  const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
  for (int s = warp; s < a.slots; s += warps) {
    const int n = pages_of(a.lens[s], a.page_shift);
    for (int j = lane; j < n; j += 32) {
      int* e = &a.table[(long long)s * a.width + j];
      const int g = a.pages[*e];
      if (g < 0) *e = a.moves[2 * (-1 - g) + 1];
    }
  }
  const long long page_bytes = ((long long)a.row_bytes << a.page_shift) * a.Hkv;
  const long long parts = (page_bytes + kCopyBytes - 1) / kCopyBytes;
  const long long units = a.head[H_MOVES] * parts * a.planes;
  for (long long u = warp; u < units; u += warps) {
    const long long part = u % parts, v = u / parts;
    const int x = (int)(v % a.planes), m = (int)(v / a.planes);
    uint8_t* plane = a.data + x * a.plane_bytes + part * kCopyBytes;
    warp_copy(plane + a.moves[2 * m + 1] * page_bytes, plane + a.moves[2 * m] * page_bytes,
              (int)min(page_bytes - part * kCopyBytes, (long long)kCopyBytes));
    if (part == 0 && a.scales) {
      const long long n = (long long)a.Hkv * a.blocks;
      float* x8 = a.scales + x * a.scale_plane;
      for (long long i = lane; i < n; i += 32) x8[a.moves[2 * m + 1] * n + i] = x8[a.moves[2 * m] * n + i];
    }
  }
}

static int launch_pool(bool update, const PoolArgs& a, cudaStream_t stream) {
  int sms = 0;
  if (!sm_count(&sms)) return FA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kPlanCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = update ? cudaLaunchKernelEx(&cfg, pool_plan_kernel<true>, a) : cudaLaunchKernelEx(&cfg, pool_plan_kernel<false>, a);
  if (e != cudaSuccess) return cuda_fail("pool_plan_kernel", (int)e, cudaGetErrorName(e));
  const int rc = check_launch("pool_plan_kernel");
  if (rc != FA_OK) return rc;
  return update ? launch_pdl("update_apply_kernel", update_apply_kernel, dim3(4 * sms), dim3(256), 0, stream, a)
                : launch_pdl("compact_apply_kernel", compact_apply_kernel, dim3(4 * sms), dim3(256), 0, stream, a);
}

}  // namespace fa

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct PoolLayout {
  long long uses, pages, slot, copies, moves, old, total;  // in ints
};
PoolLayout pool_layout(long long n_pages, long long slots, long long width) {
  PoolLayout l;
  l.uses = 64;
  l.pages = l.uses + (n_pages + 63) / 64 * 64;
  l.slot = l.pages + (n_pages + 63) / 64 * 64;
  l.copies = l.slot + 2 * slots;
  l.moves = l.copies + 3 * slots;
  l.old = l.moves + 2 * n_pages;
  l.total = l.old + slots * width;
  return l;
}

bool pool_sizes_ok(long long n_pages, long long slots, long long width) {
  return n_pages >= 1 && slots >= 1 && width >= 1 && n_pages <= (1 << 28) && slots <= (1 << 20) && width <= (1 << 26) &&
         slots * width <= (1 << 28);
}

int check_pool(const fa_pool* p, const fa_pool_scales* scales, int elem, const int32_t* info, const void* workspace,
               size_t bytes, fa::PoolArgs* a) {
  if (!p || !p->data || !p->table || !p->lens || !info || !workspace) return FA_ERR_INVALID_ARG;
  if (!aligned16(p->data)) return FA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if (p->planes < 1 || p->Hkv < 1 || p->plane_stride < 0) return FA_ERR_INVALID_ARG;
  if (p->n_pages < 1 || p->slots < 1 || p->table_width < 1) return FA_ERR_INVALID_ARG;
  switch (p->page_size) {
    case 16: case 32: case 64: case 128: case 256: break;
    default: return FA_ERR_UNSUPPORTED;
  }
  if ((p->d != 64 && p->d != 128) || p->planes > (1 << 20) || p->Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (!pool_sizes_ok(p->n_pages, p->slots, p->table_width) || (long long)p->table_width * p->page_size > (1 << 30))
    return FA_ERR_UNSUPPORTED;
  const long long plane = (long long)p->n_pages * p->Hkv * p->page_size * p->d;
  if (p->plane_stride % (16 / elem) != 0 || (p->planes > 1 && p->plane_stride < plane)) return FA_ERR_INVALID_ARG;
  if (elem == 1) {
    if (!scales || !scales->data || scales->blocks < 1 || scales->plane_stride < 0) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(scales->data) & 3u) != 0) return FA_ERR_MISALIGNED;
    a->block_shift = 4;
    while ((p->page_size >> a->block_shift) > scales->blocks) ++a->block_shift;
    if ((long long)scales->blocks << a->block_shift != p->page_size) return FA_ERR_UNSUPPORTED;
    if (p->planes > 1 && scales->plane_stride < (long long)p->n_pages * p->Hkv * scales->blocks) return FA_ERR_INVALID_ARG;
    a->scales = scales->data, a->scale_plane = scales->plane_stride, a->blocks = scales->blocks;
  }
  if (bytes < fa_cache_workspace_size(p->n_pages, p->slots, p->table_width)) return FA_ERR_INVALID_ARG;
  int err = FA_OK;
  a->status = fa::status_word(&err);
  if (!a->status) return err;
  a->data = static_cast<uint8_t*>(p->data);
  a->plane_bytes = p->plane_stride * elem;
  a->planes = p->planes, a->n_pages = p->n_pages, a->Hkv = p->Hkv, a->row_bytes = elem * p->d;
  a->page_shift = 0;
  while ((1 << a->page_shift) < p->page_size) ++a->page_shift;
  a->table = p->table, a->lens = p->lens, a->slots = p->slots, a->width = p->table_width;
  a->info = const_cast<int32_t*>(info);
  const PoolLayout l = pool_layout(p->n_pages, p->slots, p->table_width);
  int* w = static_cast<int*>(const_cast<void*>(workspace));
  a->head = w, a->uses = w + l.uses, a->pages = w + l.pages, a->slot = w + l.slot, a->copies = w + l.copies;
  a->moves = w + l.moves, a->old = w + l.old;
  return FA_OK;
}

int update_pool(const fa_pool* pool, const fa_pool_scales* scales, int elem, const int32_t* src, const int32_t* new_lens,
                int32_t* info, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  fa::PoolArgs a = {};
  const int rc = check_pool(pool, scales, elem, info, workspace, workspace_bytes, &a);
  if (rc != FA_OK) return rc;
  if (!src || !new_lens) return FA_ERR_INVALID_ARG;
  a.src = src, a.fresh = new_lens;
  return fa::launch_pool(true, a, reinterpret_cast<cudaStream_t>(stream));
}

int compact_pool(const fa_pool* pool, const fa_pool_scales* scales, int elem, int32_t* info, void* workspace,
                 size_t workspace_bytes, fa_stream_t stream) {
  fa::PoolArgs a = {};
  const int rc = check_pool(pool, scales, elem, info, workspace, workspace_bytes, &a);
  return rc != FA_OK ? rc : fa::launch_pool(false, a, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int fa_tree_mask(const int32_t* parents, const int32_t* cu_nodes, uint32_t* mask, int mask_words, int B, int T,
                 fa_stream_t stream) {
  if (B < 0 || T < 0 || mask_words < 1) return FA_ERR_INVALID_ARG;
  if (B > (1 << 20) || T > (1 << 30) || mask_words > (1 << 20)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if (!parents || !cu_nodes || !mask) return FA_ERR_INVALID_ARG;
  int err = FA_OK;
  int* status = fa::status_word(&err);
  if (!status) return err;
  return fa::launch_pdl("tree_mask_kernel", fa::tree_mask_kernel, dim3(B), dim3(fa::kTreeNodes), 0,
                        reinterpret_cast<cudaStream_t>(stream), parents, cu_nodes, mask, mask_words, B, T, status);
}

int fa_cache_append(const fa_rows* k, const fa_rows* v, const fa_pages* cache, const int32_t* start, const int32_t* cu,
                    const int32_t* rows, int B, int T, int Tkv, int Hkv, int d, fa_stream_t stream) {
  if (B < 0 || T < 0 || Tkv < 0 || Hkv < 1 || (!rows && T != Tkv)) return FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Hkv > 65535 || B > (1 << 20) || T > (1 << 30) || Tkv > (1 << 30)) return FA_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return FA_OK;
  if (Tkv == 0) return FA_ERR_INVALID_ARG;  // rows of nothing
  if (!cache || !cache->k || !cache->v || !cache->table || !start || !cu) return FA_ERR_INVALID_ARG;
  if (!aligned16(cache->k) || !aligned16(cache->v)) return FA_ERR_MISALIGNED;
  for (const fa_rows* r : {k, v}) {
    if (!r || !r->data) return FA_ERR_INVALID_ARG;
    if (!aligned16(r->data)) return FA_ERR_MISALIGNED;
    if (r->token_stride <= 0 || r->token_stride % 8 || r->head_stride <= 0 || r->head_stride % 8) return FA_ERR_INVALID_ARG;
  }
  for (int64_t s : {cache->page_stride, cache->head_stride, cache->token_stride})
    if (s <= 0 || s % 8) return FA_ERR_INVALID_ARG;
  if (cache->n_pages < 1 || cache->table_width < 1 || cache->table_stride < cache->table_width) return FA_ERR_INVALID_ARG;
  switch (cache->page_size) {
    case 16: case 32: case 64: case 128: case 256: break;
    default: return FA_ERR_UNSUPPORTED;
  }
  if ((long long)cache->table_width * cache->page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  fa::AppendArgs a;
  a.k = static_cast<const uint16_t*>(k->data), a.v = static_cast<const uint16_t*>(v->data);
  a.k_st = k->token_stride, a.k_sh = k->head_stride, a.v_st = v->token_stride, a.v_sh = v->head_stride;
  a.kc = static_cast<uint16_t*>(cache->k), a.vc = static_cast<uint16_t*>(cache->v);
  a.c_sp = cache->page_stride, a.c_sh = cache->head_stride, a.c_st = cache->token_stride;
  a.n_pages = cache->n_pages;
  a.page_shift = 0;
  while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
  a.table = cache->table, a.table_stride = cache->table_stride, a.table_width = cache->table_width;
  a.start = start, a.cu = cu, a.rows = rows;
  a.B = B, a.T = T, a.Tkv = Tkv, a.Hkv = Hkv;
  int err = FA_OK;
  a.status = fa::status_word(&err);
  if (!a.status) return err;
  const dim3 grid((T + 3) / 4);
  const auto st = reinterpret_cast<cudaStream_t>(stream);
  return d == 64 ? fa::launch_pdl("cache_append_kernel", fa::cache_append_kernel<64>, grid, dim3(128), 0, st, a)
                 : fa::launch_pdl("cache_append_kernel", fa::cache_append_kernel<128>, grid, dim3(128), 0, st, a);
}

size_t fa_cache_workspace_size(int n_pages, int slots, int table_width) {
  if (!pool_sizes_ok(n_pages, slots, table_width)) return 0;
  return (size_t)pool_layout(n_pages, slots, table_width).total * 4;
}

int fa_cache_update(const fa_pool* pool, const int32_t* src, const int32_t* new_lens, int32_t* info, void* workspace,
                    size_t workspace_bytes, fa_stream_t stream) {
  return update_pool(pool, nullptr, 2, src, new_lens, info, workspace, workspace_bytes, stream);
}

int fa_cache_compact(const fa_pool* pool, int32_t* info, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return compact_pool(pool, nullptr, 2, info, workspace, workspace_bytes, stream);
}

int fa_cache_update_8bit(const fa_pool* pool, const fa_pool_scales* scales, const int32_t* src, const int32_t* new_lens,
                         int32_t* info, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return update_pool(pool, scales, 1, src, new_lens, info, workspace, workspace_bytes, stream);
}

int fa_cache_compact_8bit(const fa_pool* pool, const fa_pool_scales* scales, int32_t* info, void* workspace,
                          size_t workspace_bytes, fa_stream_t stream) {
  return compact_pool(pool, scales, 1, info, workspace, workspace_bytes, stream);
}

}  // extern "C"
