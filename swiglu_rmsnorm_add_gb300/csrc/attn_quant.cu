// Decode attention over a KV cache held in 4 or 8 bits (format: kv_format.cuh).
//
//   o = sum_t softmax_t(scale * q . K_t) V_t over a request's tokens, K_t and V_t the values that the cache holds.
//
// A CTA takes a (request, kv head) pair, 16 tokens at a time: codes become fp32 in shared memory, a thread takes
// a (query head, token) score, the running maximum and sum of the softmax are kept for each head, and the threads
// that own output columns add p V.
#include "kv_format.cuh"

namespace sra {
namespace qattn {

constexpr int kThreads = 128, kTok = 16;

template <typename T, int FMT, int HD>
__global__ void __launch_bounds__(kThreads) decode_kernel(QuantAttnArgs a) {
    constexpr int R = kvq::row_bytes(FMT, HD), CODES = kvq::code_bytes(FMT, HD), WORDS = FMT == KV_E2M1 ? 1 : 2;
    constexpr int COLS = HD > kThreads ? HD / kThreads : 1;
    __shared__ float qs[8][HD], ks[kTok][HD + 1], vs[kTok][HD], ps[8][kTok], m_run[8], l_run[8], corr[8];
    pdl_enter();
    const int64_t b = blockIdx.x / a.n_kv;
    const int kvh = static_cast<int>(blockIdx.x - b * a.n_kv), G = a.group, BS = a.block_size;
    int64_t len = a.seq_lens[b];
    const int64_t cap = a.max_blocks * BS;
    if ((len < 0 || len > cap) && kvh == 0 && threadIdx.x == 0 && a.err) atomicAdd(a.err, 1);
    len = len < 0 ? 0 : (len > cap ? cap : len);
    for (int i = threadIdx.x; i < G * HD; i += kThreads)
        qs[i / HD][i % HD] = to_f32(static_cast<const T*>(a.q)[b * a.qs + static_cast<int64_t>(kvh) * G * HD + i]);
    if (threadIdx.x < 8) m_run[threadIdx.x] = -INFINITY, l_run[threadIdx.x] = 0.0f;
    float acc[8][COLS];
#pragma unroll
    for (int g = 0; g < 8; ++g)
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[g][c] = 0.0f;
    for (int64_t t0 = 0; t0 < len; t0 += kTok) {
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * kTok * (HD / 8); i += kThreads) {
            const int plane = i / (kTok * (HD / 8)), rest = i - plane * kTok * (HD / 8);
            const int t = rest / (HD / 8), d = (rest - t * (HD / 8)) * 8;
            const int64_t tok = t0 + t;
            const int32_t page = tok < len ? a.table[b * a.max_blocks + tok / BS] : -1;
            const bool ok = page >= 0 && page < a.num_blocks;
            if (!ok && tok < len && tok % BS == 0 && i == t * (HD / 8) && kvh == 0 && a.err) atomicAdd(a.err, 1);
            uint32_t v[4] = {0, 0, 0, 0};
            if (ok) {
                const uint8_t* row = static_cast<const uint8_t*>(a.cache) + plane * a.plane_bytes +
                                     ((static_cast<int64_t>(page) * a.n_kv + kvh) * BS + tok % BS) * R;
                uint32_t w[WORDS];
#pragma unroll
                for (int j = 0; j < WORDS; ++j) w[j] = reinterpret_cast<const uint32_t*>(row + d * WORDS / 2)[j];
                kvq::decode8<FMT>(w, kvq::scale_pair(row[CODES + d / kvq::kGroup]), v);
            }
            float* dst = plane ? &vs[t][d] : &ks[t][d];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __half2 h;
                memcpy(&h, &v[j], 4);
                const float2 f = __half22float2(h);
                dst[2 * j] = f.x, dst[2 * j + 1] = f.y;
            }
        }
        __syncthreads();
        const int g = threadIdx.x / kTok, t = threadIdx.x % kTok;
        const int64_t tok = t0 + t;
        bool valid = tok < len && g < G;
        if (valid) {
            const int32_t page = a.table[b * a.max_blocks + tok / BS];
            valid = page >= 0 && page < a.num_blocks;
        }
        float s = -INFINITY;
        if (valid) {
            float d0 = 0.0f;
            for (int d = 0; d < HD; ++d) d0 = fmaf(qs[g][d], ks[t][d], d0);
            s = d0 * a.scale_log2;
        }
        float mx = s;
        for (int o = kTok / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_old = m_run[g], m_new = fmaxf(m_old, mx);
        // (no score above -inf yet: those weigh nothing; a NaN stays one)
        const float p = valid ? exp2f(s - (m_new == -INFINITY ? 0.0f : m_new)) : 0.0f;
        float sum = p;
        for (int o = kTok / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncwarp();
        ps[g][t] = p;
        if (t == 0) {
            const float c = m_new == -INFINITY ? 1.0f : exp2f(m_old - m_new);
            corr[g] = c;
            l_run[g] = l_run[g] * c + sum;
            m_run[g] = m_new;
        }
        __syncthreads();
        const int n = static_cast<int>(len - t0 < kTok ? len - t0 : kTok);
        for (int gg = 0; gg < G; ++gg)
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const int d = threadIdx.x + c * kThreads;
                if (d < HD) {
                    float x = acc[gg][c] * corr[gg];
                    for (int k = 0; k < n; ++k) x = fmaf(ps[gg][k], vs[k][d], x);
                    acc[gg][c] = x;
                }
            }
    }
    __syncthreads();
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const int d = threadIdx.x + c * kThreads;
            if (d < HD)
                static_cast<T*>(a.out)[b * a.os + (static_cast<int64_t>(kvh) * G + g) * HD + d] =
                    from_f32<T>(l_run[g] != 0.0f ? acc[g][c] / l_run[g] : 0.0f);
        }
}

template <typename T, int FMT>
cudaError_t launch(const QuantAttnArgs& a, const QuantAttnPlan& p, cudaStream_t s) {
    auto kernel = p.head_dim == 64 ? decode_kernel<T, FMT, 64> : p.head_dim == 128 ? decode_kernel<T, FMT, 128> : decode_kernel<T, FMT, 256>;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(a.B * a.n_kv)), dim3(kThreads), 0, s, p.pdl, 1, a);
}

}  // namespace qattn

cudaError_t launch_attention_quant(const QuantAttnArgs& a, const QuantAttnPlan& p, int dtype, cudaStream_t s) {
    using namespace qattn;
    const bool e = p.format == KV_E2M1;
    switch (dtype) {
        case DT_F32: return e ? launch<float, KV_E2M1>(a, p, s) : launch<float, KV_INT8>(a, p, s);
        case DT_F16: return e ? launch<__half, KV_E2M1>(a, p, s) : launch<__half, KV_INT8>(a, p, s);
        case DT_BF16: return e ? launch<__nv_bfloat16, KV_E2M1>(a, p, s) : launch<__nv_bfloat16, KV_INT8>(a, p, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace sra
