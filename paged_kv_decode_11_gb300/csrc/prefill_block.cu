// prefill_block.cu — the tensor-core chunked prefill (prefill_tc_kernel.cuh) over
// E4M3 blocks with a scale per block and KV head, with and without modified
// scores.
#include "prefill_tc_kernel.cuh"

namespace pkv {

template <int D, int MODE>
static pkv_status launch_q(const PrefillExtParams& p, pkv_dtype q_dtype, const CUtensorMap& tmQ,
                           const CUtensorMap& tmK, const CUtensorMap& tmV, cudaStream_t stream) {
  return q_dtype == PKV_BF16
             ? launch_tc_ext<D, KV_E4M3, true, MODE>(p, tmQ, tmK, tmV, stream)
             : launch_tc_ext<D, KV_E4M3, false, MODE>(p, tmQ, tmK, tmV, stream);
}

pkv_status launch_prefill_block(const PrefillExtParams& p, int head_dim, pkv_dtype q_dtype,
                                const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                const CUtensorMap& tmV, cudaStream_t stream) {
  const bool mod = p.cap_log2 != 0.f || p.slopes != nullptr || p.window > 0 ||
                   p.prefix_lens != nullptr;
  constexpr int kBoth = kTcBlockScales | kTcModScores;
  if (head_dim == 256)
    return mod ? launch_q<256, kBoth>(p, q_dtype, tmQ, tmK, tmV, stream)
               : launch_q<256, kTcBlockScales>(p, q_dtype, tmQ, tmK, tmV, stream);
  if (head_dim == 128)
    return mod ? launch_q<128, kBoth>(p, q_dtype, tmQ, tmK, tmV, stream)
               : launch_q<128, kTcBlockScales>(p, q_dtype, tmQ, tmK, tmV, stream);
  return mod ? launch_q<64, kBoth>(p, q_dtype, tmQ, tmK, tmV, stream)
             : launch_q<64, kTcBlockScales>(p, q_dtype, tmQ, tmK, tmV, stream);
}

}  // namespace pkv
