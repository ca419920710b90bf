// prefill_mod.cu — the tensor-core chunked prefill (prefill_tc_kernel.cuh) with
// modified scores over 16-bit caches and E4M3 caches with a scale per head.
#include "prefill_tc_kernel.cuh"

namespace pkv {

template <int D>
static pkv_status launch_d(const PrefillExtParams& p, pkv_dtype q_dtype, pkv_dtype kv_dtype,
                           const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                           cudaStream_t stream) {
  if (kv_dtype == PKV_BF16)
    return launch_tc_ext<D, KV_BF16, true, kTcModScores>(p, tmQ, tmK, tmV, stream);
  if (kv_dtype == PKV_F16)
    return launch_tc_ext<D, KV_F16, false, kTcModScores>(p, tmQ, tmK, tmV, stream);
  return q_dtype == PKV_BF16
             ? launch_tc_ext<D, KV_E4M3, true, kTcModScores>(p, tmQ, tmK, tmV, stream)
             : launch_tc_ext<D, KV_E4M3, false, kTcModScores>(p, tmQ, tmK, tmV, stream);
}

pkv_status launch_prefill_mod(const PrefillExtParams& p, int head_dim, pkv_dtype q_dtype,
                              pkv_dtype kv_dtype, const CUtensorMap& tmQ,
                              const CUtensorMap& tmK, const CUtensorMap& tmV,
                              cudaStream_t stream) {
  if (head_dim == 256) return launch_d<256>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream);
  if (head_dim == 128) return launch_d<128>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream);
  return launch_d<64>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream);
}

}  // namespace pkv
