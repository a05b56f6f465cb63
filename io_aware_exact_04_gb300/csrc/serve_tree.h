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
  float* part_o;    // workspace: two slots of 256 rows for each CTA, O normalised by its own l
  float* part_lse;  // their LSEs, base 2 (-inf: no key, O not written)
  long long part_rows;
  int4* cuts;       // two for each CTA, of the item that it is the first to cut: {later parts (0: none), ..},
                    // {tokens of the sequence, its first row, the item's first token, key/value head}
  int* status;
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
