// decode_ext.cu — decode attention over block scales or with modified scores,
// CTAs of kDecodeWarps warps (decode_ext_kernel.cuh); whole-context plans go to
// decode_ext_wide.cu.
#include "decode_ext_kernel.cuh"

namespace pkv {

pkv_status launch_decode_ext(const DecodeExtParams& p, int head_dim, pkv_dtype q_dtype,
                             pkv_dtype kv_dtype, bool block_scaled, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, cudaStream_t stream) {
  if (p.base.wide)
    return launch_decode_ext_wide(p, head_dim, q_dtype, kv_dtype, block_scaled, tmK, tmV, stream);
  if (head_dim == 256)
    return launch_decode_ext_d<256, kDecodeWarps>(p, q_dtype, kv_dtype, block_scaled, tmK, tmV,
                                                  stream);
  if (head_dim == 128)
    return launch_decode_ext_d<128, kDecodeWarps>(p, q_dtype, kv_dtype, block_scaled, tmK, tmV,
                                                  stream);
  return launch_decode_ext_d<64, kDecodeWarps>(p, q_dtype, kv_dtype, block_scaled, tmK, tmV,
                                               stream);
}

}  // namespace pkv
