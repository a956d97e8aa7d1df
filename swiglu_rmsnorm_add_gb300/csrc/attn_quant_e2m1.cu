// Decode attention over a cache in 4 bits, bf16 and fp16 queries.
#include "attn_quant_impl.cuh"

namespace sra {
cudaError_t launch_attn_quant_e2m1(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) { return qattn::launch_format<false, KV_E2M1>(a, p, s); }
unsigned int quant_attn_wait_timeouts_int8();
unsigned int quant_attn_wait_timeouts_e2m1_f32();
unsigned int quant_attn_wait_timeouts_int8_f32();
unsigned int quant_attn_wait_timeouts() {
    return qattn::unit_wait_timeouts() + quant_attn_wait_timeouts_int8() + quant_attn_wait_timeouts_e2m1_f32() +
           quant_attn_wait_timeouts_int8_f32();
}
}  // namespace sra
