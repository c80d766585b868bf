// The quantised decodes' merge kernel over partials that a test makes: one KV head of two query heads, head_dim 128.
#include "../paged_kv_attention_10_gb300/csrc/quant_decode.cuh"

struct Any {
  static constexpr int kDim = 128;
};

// warps: of a query head, 1 or 8.  The grid is that of a decode of num_ctas CTAs over kv_lens [batch].
extern "C" int merge(int batch, int num_ctas, int warps, const int* kv_lens, const float* part_o, const float* part_lse,
                     int* unit_first, int* unit_last, void* out, float* lse, unsigned* err_word) {
  pkv::QuantDecodeArgs a = {};
  a.batch = batch;
  a.num_q_heads = 2;
  a.num_kv_heads = a.HC = a.nhg = 1;
  a.group = 2;
  a.kv_lens = kv_lens;
  a.part_o = const_cast<float*>(part_o);
  a.part_lse = const_cast<float*>(part_lse);
  a.unit_first = unit_first;
  a.unit_last = unit_last;
  a.out = (__nv_bfloat16*)out;
  a.lse = lse;
  a.err_word = err_word;
  a.num_parts = num_ctas + batch;
  const dim3 grid((unsigned)batch, (unsigned)((2 * warps + 7) / 8));
  if (warps == 8) pkv::quant_decode_merge_kernel<Any, 8><<<grid, 256>>>(a);
  else pkv::quant_decode_merge_kernel<Any, 1><<<grid, 256>>>(a);
  return cudaDeviceSynchronize();
}
