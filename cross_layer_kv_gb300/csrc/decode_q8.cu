// Decode over 8-bit caches: planning, and the kernels of bf16 contexts (those
// of fp32 contexts compile beside them, in decode_q8_f32.cu).
#include "decode_q8_impl.cuh"

namespace fkv {

cudaError_t decode_q8_launch_f32(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream);

namespace {

template <int D, int NSRC, int G, bool F32>
void q8_shape(int B, size_t* smem, int* warps) {
  *smem = q8_smem_bytes<D, NSRC, G, F32>(B);
  *warps = Q8Shape<NSRC, G, F32>::W;
}

template <int D, int NSRC, bool F32>
void q8_shape_g(const DecodeArgs& a, size_t* smem, int* warps) {
  if (a.group == 1) q8_shape<D, NSRC, 1, F32>(a.batch, smem, warps);
  if (a.group == 2) q8_shape<D, NSRC, 2, F32>(a.batch, smem, warps);
  if (a.group == 4) q8_shape<D, NSRC, 4, F32>(a.batch, smem, warps);
}

template <int D>
void q8_shape_d(const DecodeArgs& a, size_t* smem, int* warps) {
  if (a.is_f32)
    a.nsrc == 2 ? q8_shape_g<D, 2, true>(a, smem, warps) : q8_shape_g<D, 1, true>(a, smem, warps);
  else
    a.nsrc == 2 ? q8_shape_g<D, 2, false>(a, smem, warps) : q8_shape_g<D, 1, false>(a, smem, warps);
}

}  // namespace

cudaError_t decode_q8_plan(const DecodeArgs& a, int num_sms, DecodePlan* plan) {
  size_t smem = 0;
  int W = 0;
  switch (a.head_dim) {
    case 64: q8_shape_d<64>(a, &smem, &W); break;
    case 80: q8_shape_d<80>(a, &smem, &W); break;
    case 96: q8_shape_d<96>(a, &smem, &W); break;
    case 128: q8_shape_d<128>(a, &smem, &W); break;
    default: return cudaErrorNotSupported;
  }
  if (W == 0) return cudaErrorNotSupported;
  const long long rows = (long long)a.batch * a.kv_heads * a.max_seq;
  long long ctas = a.num_ctas > 0 ? a.num_ctas : num_sms;
  const long long by_rows = (rows + 64LL * W - 1) / (64LL * W);
  if (a.num_ctas <= 0) ctas = ctas < by_rows ? ctas : by_rows;
  if (ctas < 1) ctas = 1;
  plan->ctas = (int)ctas;
  plan->warps_per_cta = W;
  plan->smem_bytes = smem;
  const size_t units = (size_t)a.batch * a.kv_heads;
  const size_t slots = (size_t)ctas * W + units;
  plan->partial_bytes = (slots * a.group * partial_stride(a.head_dim) * sizeof(float) + 15) / 16 * 16;
  plan->workspace_bytes = plan->partial_bytes + units * sizeof(unsigned long long);
  return cudaSuccess;
}

cudaError_t decode_q8_launch(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
  return a.is_f32 ? decode_q8_launch_f32(a, plan, stream) : q8_by_dim<__nv_bfloat16>(a, plan, stream);
}

}  // namespace fkv
