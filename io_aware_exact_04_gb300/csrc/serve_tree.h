// What the kernels of prompts and trees get, in 16 and in 8 bits.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {

struct ServeArgs {
  const uint16_t *q, *k, *v;
  uint16_t* o;
  long long q_st, q_sh, k_st, k_sh, v_st, v_sh, o_st, o_sh;  // token and head strides, elements
  float* lse;  // [Hq, T] or null
  int o_wide;  // every row of o is 32-byte aligned
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
  // Workspace, of fa_forward_tree_workspace_size bytes: two slots of rows for each CTA, then the cuts. A slot has 256
  // rows, lane 1's from 128 on. The few-row kernel of fa_serve8.cu divides the same bytes into slots of 32, lane 1's
  // rows following lane 0's.
  float* part_o;    // O normalised by its own l
  float* part_lse;  // their LSEs, base 2 (-inf: no key, O not written)
  long long part_rows;
  int4* cuts;       // two for each CTA, of the item that it is the first to cut: {later parts (0: none), ..},
                    // {tokens of the sequence, its first row, the item's first token, key/value head}, or of the
                    // few-row kernel {rows of the sequence (tokens times heads of the group), its first token, the
                    // item's first row, key/value head}
  int* status;
#ifdef FA_DEBUG
  int dbg_B;           // batch count B, for the extents the debug build checks against
  int dbg_slack;       // rows taken off those extents (fa_debug_set_check_slack)
#endif
};

// Over a cache in 8 bits: its scales. (Strides and tensor maps count its elements, bytes.)
struct Serve8BitArgs : ServeArgs {
  const float *ks, *vs;
  long long s_sp, s_sh;
  int block_shift;
};

// Trees over a cache in 8 bits with few rows a sequence (fa_serve8.cu). a: as for the kernels of fa_serve.cu.
int launch_serve8(const fa_rows* k, const fa_rows* v, const fa_pages* cache, Serve8BitArgs a, int d, int dtype,
                  cudaStream_t stream);

}  // namespace fa
