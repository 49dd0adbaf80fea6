// Decode over 8-bit caches: planning, and the kernels of bf16 contexts (those
// of fp32 contexts compile beside them, in decode_q8_f32.cu).
#include "decode_q8_impl.cuh"

namespace fkv {

cudaError_t decode_q8_launch_f32(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);

namespace {

template <int D>
size_t q8_shape(const DecodeArgs& a, int* warps) {
  *warps = a.nsrc == 2 ? Q8Shape<D, 2>::W : Q8Shape<D, 1>::W;
  return a.nsrc == 2 ? q8_smem_bytes<D, 2>(a.batch, a.group)
                     : q8_smem_bytes<D, 1>(a.batch, a.group);
}

}  // namespace

cudaError_t decode_q8_plan(const DecodeArgs& a, int num_sms, DecodePlan* plan) {
  size_t smem = 0;
  int W = 0;
  if (a.group != 1 && a.group != 2 && a.group != 4) return cudaErrorNotSupported;
  switch (a.head_dim) {
    case 64: smem = q8_shape<64>(a, &W); break;
    case 80: smem = q8_shape<80>(a, &W); break;
    case 96: smem = q8_shape<96>(a, &W); break;
    case 128: smem = q8_shape<128>(a, &W); break;
    default: return cudaErrorNotSupported;
  }
  const long long rows = (long long)a.batch * a.kv_heads * a.max_seq;
  long long ctas = a.num_ctas > 0 ? a.num_ctas : num_sms;
  // small calls (by the rows that the context's caches hold: the workspace is
  // asked for once, whatever the calls' windows and lengths): CTAs of 8 rows a
  // warp, which take whole units where they can
  // (fused, 64 channels, us with 8, 16 and 64 rows a warp: 128 units of 100 rows
  // 6.6, 8.4, 12.2; 64 of 300 7.4, 7.3, 10.7; 2 of 256 6.9, 6.8, 8.5)
  const long long by_rows = (rows + 8LL * W - 1) / (8LL * W);
  if (a.num_ctas <= 0) ctas = ctas < by_rows ? ctas : by_rows;
  if (ctas < 1) ctas = 1;
  plan->ctas = (int)ctas;
  plan->warps_per_cta = W;
  plan->smem_bytes = smem;
  const size_t units = (size_t)a.batch * a.kv_heads;
  const size_t slots = (size_t)ctas + units;   // a CTA's partial of unit u: slot CTA + u
  plan->partial_bytes = (slots * a.group * partial_stride(a.head_dim) * sizeof(float) + 15) / 16 * 16;
  plan->workspace_bytes = plan->partial_bytes + units * a.group * sizeof(unsigned long long);
  return cudaSuccess;
}

cudaError_t decode_q8_launch(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
  return a.is_f32 ? decode_q8_launch_f32(a, plan, stream) : q8_by_dim<__nv_bfloat16>(a, plan, stream);
}

}  // namespace fkv
