// host.h — host-side helpers of the entry points (defined in api.cu): the
// current device's error word and SM count, the checks and the tensor maps
// that every call uses.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include "../../include/pkv.h"

namespace pkv {

unsigned int* err_word();                 // of the current device; nullptr on failure
int sm_count();                           // of the current device; 0 on failure
int block_log2(int block_size);           // -1 for sizes the kernels do not take
int page_shift(int block_size);           // log2 of the 16-token pages per block
bool page_rows_fit(int num_blocks, int Hkv, int block_size, int max_blocks_per_seq);
bool make_kv_tmap(CUtensorMap* m, const void* base, pkv_dtype dt, int D, int Hkv, int num_blocks,
                  int ppb_shift);
bool make_q_tmap(CUtensorMap* m, const void* q, int D, int Hq, int G, int q_tile, int rows);
bool aligned16(const void* p);
bool valid_dtypes(pkv_dtype q, pkv_dtype kv);

}  // namespace pkv
