// Decode attention over a cache in 8 bits, fp32 queries.
#include "attn_quant_impl.cuh"

namespace sra {
cudaError_t launch_attn_quant_int8_f32(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) { return qattn::launch_format<true, KV_INT8>(a, p, s); }
unsigned int quant_attn_wait_timeouts_int8_f32() { return qattn::unit_wait_timeouts(); }
}  // namespace sra
