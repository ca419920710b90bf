// decode_ext_wide.cu — decode attention over block scales or with modified
// scores in its whole-context shape: one CTA of kDecodeWideWarps warps per
// (sequence, KV head), as planned by wide_decode in plan.h (head_dim 64, 128).
#include "decode_ext_kernel.cuh"

namespace pkv {

pkv_status launch_decode_ext_wide(const DecodeExtParams& p, int head_dim, pkv_dtype q_dtype,
                                  pkv_dtype kv_dtype, bool block_scaled, const CUtensorMap& tmK,
                                  const CUtensorMap& tmV, cudaStream_t stream) {
  if (head_dim == 128)
    return launch_decode_ext_d<128, kDecodeWideWarps>(p, q_dtype, kv_dtype, block_scaled, tmK,
                                                      tmV, stream);
  if (head_dim == 64)
    return launch_decode_ext_d<64, kDecodeWideWarps>(p, q_dtype, kv_dtype, block_scaled, tmK, tmV,
                                                     stream);
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
