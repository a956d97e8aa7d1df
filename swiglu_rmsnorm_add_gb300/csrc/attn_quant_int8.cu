// Decode attention over a cache in 8 bits, bf16 and fp16 queries.
#include "attn_quant_impl.cuh"

namespace sra {
cudaError_t launch_attn_quant_int8(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) { return qattn::launch_format<false, KV_INT8>(a, p, s); }
unsigned int quant_attn_wait_timeouts_int8() { return qattn::unit_wait_timeouts(); }
}  // namespace sra
