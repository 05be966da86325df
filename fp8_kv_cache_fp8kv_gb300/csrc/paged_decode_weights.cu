// A decode step that adds up each cached token's attention weight, the measure by
// which fp8kv_evict keeps tokens.
//
// A token's probabilities are known only when the sums over the whole context
// are, so the streaming decode (stream_decode.cuh, WS = true) also writes its
// scores, 4 g bytes a token and kv head beside the 2 d bytes of its codes, and each
// query head's softmax reference m and 1 / l.  A second kernel then reads them back
// (from L2: a launch's scores stay within 64 MiB):
//     weights_t = old_t decay + sum_h 2^(s_ht - m_h) / l_h,
// one thread a token, so the sum has one order and the result one value.
// Reading K again instead would cost d bytes a token (128, against 8 g = 32 at g = 4).
// Measured (GB300, 8 x 20K, 32 over 8 heads of 128, E4M3): 74.1 us, 4.5 TB/s, of
// which the second kernel about 10 (fp8kv_paged_decode alone 59.6); 1 x 4096 10.7 us
// (9.2).  Four tokens a thread: 73.3 and 12.5 us.
#include "stream_decode.cuh"

namespace fp8kv {

// G query heads a unit, U units a cache head (2 where g = 16 runs as two of 8).
template <int G, int U>
__global__ void __launch_bounds__(256) add_weights_kernel(const DecodeArgs a) {
    __shared__ float2 soft[G * U];
    __shared__ uint32_t err;
    const int tid = threadIdx.x, b = blockIdx.z, hk = blockIdx.y;
    const int Hc = a.num_kv_heads / U;
    griddep_launch_dependents();
    const int L = clamp_len(ld_input(a.seq_lens + b), a.max_seq_len);   // (final: read by the decode before)
    const int lo = first_token(L, a.window), base = lo / kBS * kBS;
    const int t = base + blockIdx.x * 256 + tid;
    const bool in = t >= lo && t < L;
    int id = in ? ld_input(a.block_tables + static_cast<int64_t>(b) * a.max_blocks_per_seq + t / kBS) : -1;
    if (id >= a.num_blocks) id = -1;                                    // (the decode reports it)
    griddep_wait();
    if (base + blockIdx.x * 256 >= L) return;
    // (one thread asks: every warp's read of the one word made the 8 x 20K call 5 us longer)
    if (tid == 255) err = *reinterpret_cast<volatile uint32_t*>(a.err);
    if (tid < G * U) soft[tid] = a.softmax[static_cast<int64_t>(b) * a.num_q_heads + hk * G * U + tid];
    __syncthreads();
    if (id < 0 || err == FP8KV_ERR_TIMEOUT) return;                     // (the decode was skipped: no scores)
    float* w = a.weights + (static_cast<int64_t>(id) * Hc + hk) * kBS + t % kBS;
    const float old = t == L - 1 ? 0.f : *w * a.decay;
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float* s = a.scores + (static_cast<int64_t>(b * a.num_kv_heads + hk * U + u) * a.score_tokens + (t - base)) * G;
        float x[G];
        if constexpr (G >= 4) {
#pragma unroll
            for (int i = 0; i < G / 4; ++i) {
                const float4 y = *(reinterpret_cast<const float4*>(s) + i);
                x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i) x[i] = s[i];
        }
#pragma unroll
        for (int i = 0; i < G; ++i) sum = fmaf(fast_exp2(x[i] - soft[u * G + i].x), soft[u * G + i].y, sum);
    }
    *w = old + sum;
}

template <int G, int U>
static cudaError_t launch_add(const DecodeArgs& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.score_tokens + 255) / 256), static_cast<unsigned>(a.num_kv_heads / U),
                       static_cast<unsigned>(a.batch));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, add_weights_kernel<G, U>, a);
}

template <int ES, bool E5M2>
static cudaError_t launch_decode(int head_dim, int G, const DecodeArgs& a, int ctas, cudaStream_t s) {
    return head_dim == 64    ? launch_stream_g<64, ES, E5M2, false, true>(G, a, ctas, s)
           : head_dim == 128 ? launch_stream_g<128, ES, E5M2, false, true>(G, a, ctas, s)
                             : launch_stream_g<256, ES, E5M2, false, true>(G, a, ctas, s);
}

cudaError_t launch_stream_weights(int head_dim, int G, int es, bool e5m2, const DecodeArgs& a, int ctas, cudaStream_t s) {
    const cudaError_t e = es == 2 ? launch_decode<2, false>(head_dim, G, a, ctas, s)
                          : e5m2  ? launch_decode<1, true>(head_dim, G, a, ctas, s)
                                  : launch_decode<1, false>(head_dim, G, a, ctas, s);
    if (e != cudaSuccess || a.score_tokens == 0) return e;
    if (a.kv_shift) return launch_add<8, 2>(a, s);
    switch (G) {
        case 1: return launch_add<1, 1>(a, s);
        case 2: return launch_add<2, 1>(a, s);
        case 4: return launch_add<4, 1>(a, s);
        case 8: return launch_add<8, 1>(a, s);
        default: return launch_add<16, 1>(a, s);
    }
}

}  // namespace fp8kv
