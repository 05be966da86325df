// The streaming decode over a block-scaled E4M3 cache: one K and one V scale
// for every (page, kv head), the granularity below the per-tensor and per-head
// scales of gpusmith.com, "FP8 KV Cache Quantization: Capacity Gains and
// Accuracy Risk", "Scales and calibration".
//
// The kernel is stream_decode_kernel (stream_decode.cuh) with BS = true.  With
// c_t the codes and ks, vs the scales of key t's page, in log2 units,
//     s_t = sm (q . ck_t) ks,   w_t = 2^(s_t + log2 vs - m),
//     out = sum_t w_t cv_t / sum_t (w_t / vs),
// m the largest s_t + log2 vs: the scales are the multiplier and the addend of
// one FMA a score, and the row sum takes a factor a page.  They are read from
// HBM with the pages: 8 bytes beside a page's 32 d bytes, as 4-byte cp.async
// copies in the stage's own group.
//
// What bounds it is what bounds the kernel without them (stream_decode.cuh): HBM
// and the fixed cost of a step.  8 x 20K, 32 over 8 heads, d = 128: 62.2 us, 329 MB
// at 5.3 TB/s (59.5 with one scale per tensor and the append fused in); 1 x 128K,
// 64 over 8 heads: 50.4 us, 5.3 TB/s; 1 x 4096: 9.4 us; 9 sequences behind a window
// of 128: 13.4 us.
#include "stream_decode.cuh"

namespace fp8kv {

cudaError_t launch_stream_block(int head_dim, int G, const DecodeArgs& a, int ctas, cudaStream_t s) {
    return head_dim == 64    ? launch_stream_g<64, 1, false, true>(G, a, ctas, s)
           : head_dim == 128 ? launch_stream_g<128, 1, false, true>(G, a, ctas, s)
                             : launch_stream_g<256, 1, false, true>(G, a, ctas, s);
}

}  // namespace fp8kv
