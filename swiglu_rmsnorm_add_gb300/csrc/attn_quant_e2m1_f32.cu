// Decode attention over a cache in 4 bits, fp32 queries.
#include "attn_quant_impl.cuh"

namespace sra {
cudaError_t launch_attn_quant_e2m1_f32(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) { return qattn::launch_format<true, KV_E2M1>(a, p, s); }
unsigned int quant_attn_wait_timeouts_e2m1_f32() { return qattn::unit_wait_timeouts(); }
}  // namespace sra
