// linear_fp8.cu -- which kernel of qmoe_linear_fp8 takes a call.
#include "linear_fp8.cuh"

namespace qmoe {

cudaError_t linear_fp8_prepare() { return linear_pair_prepare(); }

// Up to 16 tokens go to mma.sync, whose CTAs read W once and wait for nothing else (W of
// 2048 x 5120, one token: 3.3 us, 9 on a pair of CTAs; of 2048 x 40000, 16 tokens: 24, 32).
// Beyond, x is widened again in every CTA of 16 features, and the sizes decide, by what the
// kernels were measured to take in us: a start, and so much a block of k for each wave of
// CTAs or pairs.
//                                   mma.sync   pairs, 128 features   pairs, 256
//   K 4096  N  2048   64 tokens       8.1           14.6                21.2
//   K 2048  N  5120   32              7.4            9.4                13.1
//                     64             12.8            9.5                13.2
//                    400             60             15.8                14.2
//                   1500              -             28.7                23.9
//   K 2000  N  1003  100              5.9            9.2                13.3
//                    777             26              9.6                13.8
//                   3000              -             16.7                14.5
//   K  512  N  2048  100              5.3            5.8                 7.4
//                    192              9.5            5.7                 7.6
cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    if (a.T <= 16) return launch_linear_few(a, st);
    auto waves = [](int64_t work, int at_once) { return (double)((work + at_once - 1) / at_once); };
    const double kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int64_t ctas = (int64_t)((a.N + LF_ROWS - 1) / LF_ROWS) * ((a.T + 63) / 64), token_tiles = (a.T + 255) / 256;
    const double few = 2.0 + (a.T <= 32 ? waves(ctas, 2 * num_sms) * (0.3 + 0.11 * kb) : waves(ctas, num_sms) * (0.9 + 0.17 * kb));
    const double p128 = 3.7 + 0.33 * kb * waves(token_tiles * ((a.N + 127) / 128), num_sms / 2);
    const double p256 = 4.7 + 0.52 * kb * waves(token_tiles * ((a.N + 255) / 256), num_sms / 2);
    if (few <= p128 && few <= p256 && a.T <= 64 * 65535) return launch_linear_few(a, st);   // a grid's second size
    return launch_linear_pair(a, p128 < p256 ? 128 : 256, num_sms, st);
}

}  // namespace qmoe
