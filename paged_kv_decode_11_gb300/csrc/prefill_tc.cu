// prefill_tc.cu — the tensor-core chunked prefill (prefill_tc_kernel.cuh) for
// paged_attn_prefill_chunk and paged_attn_varlen: which launch a call takes.
#include "prefill_tc_kernel.cuh"

namespace pkv {

// SMs of device `dev`, read once; 0 on failure.
static int prefill_tc_sms(int dev) {
  static std::atomic<int> sms[64];
  int n = sms[dev].load();
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    sms[dev].store(n);
  }
  return n;
}

// One CTA per query tile when that fills at least half of the GPU (or other
// work shares it); otherwise a cluster of two per tile, each taking half of
// the key tiles. Beside a decode grid (may_split false), the 64-key tiles.
template <int D, int KV, bool QBF16>
static pkv_status launch_prefill_tc_t(const PrefillParams& p, const CUtensorMap& tmQ,
                                      const CUtensorMap& tmK, const CUtensorMap& tmV,
                                      cudaStream_t stream,
                                      bool may_split) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
  const int n_sms = prefill_tc_sms(dev);
  if (n_sms == 0) return PKV_ERR_CUDA;
  PrefillParams q = p;
  q.q_tile = kTcRows / p.G;
  const int64_t ctas = (int64_t)((q.max_q_len + q.q_tile - 1) / q.q_tile) * q.Hkv * q.num_seqs;
  if (!may_split)
    return PrefillTcLaunch<D, KV, QBF16, 1, false, kTcPlain>::launch(q, tmQ, tmK, tmV, stream, dev);
  if (2 * ctas <= n_sms)
    return PrefillTcLaunch<D, KV, QBF16, 2, true, kTcPlain>::launch(q, tmQ, tmK, tmV, stream, dev);
  return PrefillTcLaunch<D, KV, QBF16, 1, true, kTcPlain>::launch(q, tmQ, tmK, tmV, stream, dev);
}

template <int D>
static pkv_status launch_prefill_tc_d(const PrefillParams& p, pkv_dtype q_dtype,
                                      pkv_dtype kv_dtype, const CUtensorMap& tmQ,
                                      const CUtensorMap& tmK, const CUtensorMap& tmV,
                                      cudaStream_t stream,
                                      bool may_split) {
  if (kv_dtype == PKV_BF16)
    return launch_prefill_tc_t<D, KV_BF16, true>(p, tmQ, tmK, tmV, stream, may_split);
  if (kv_dtype == PKV_F16)
    return launch_prefill_tc_t<D, KV_F16, false>(p, tmQ, tmK, tmV, stream, may_split);
  if constexpr (D <= 128) {
    return q_dtype == PKV_BF16
               ? launch_prefill_tc_t<D, KV_E4M3, true>(p, tmQ, tmK, tmV, stream, may_split)
               : launch_prefill_tc_t<D, KV_E4M3, false>(p, tmQ, tmK, tmV, stream, may_split);
  }
  return PKV_ERR_UNSUPPORTED;
}

bool prefill_tc_supported(int head_dim, pkv_dtype kv_dtype) {
  if (kv_dtype == PKV_FP8_E4M3) return head_dim == 64 || head_dim == 128;
  return head_dim == 64 || head_dim == 128 || head_dim == 256;
}

pkv_status launch_prefill_tc(const PrefillParams& p, int head_dim, pkv_dtype q_dtype,
                             pkv_dtype kv_dtype, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, cudaStream_t stream, bool may_split) {
  if (head_dim == 256)
    return launch_prefill_tc_d<256>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream, may_split);
  if (head_dim == 128)
    return launch_prefill_tc_d<128>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream, may_split);
  return launch_prefill_tc_d<64>(p, q_dtype, kv_dtype, tmQ, tmK, tmV, stream, may_split);
}

}  // namespace pkv
