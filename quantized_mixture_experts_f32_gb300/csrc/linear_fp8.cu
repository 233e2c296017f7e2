// linear_fp8.cu -- which kernel of qmoe_linear_fp8 takes a call.
#include "linear_fp8.cuh"

namespace qmoe {

cudaError_t linear_fp8_prepare() { return linear_pair_prepare(); }

// Up to 16 tokens go to mma.sync, whose CTAs read W once and wait for nothing else (W of
// 2048 x 5120, one token: 3.3 us, 9 on a pair of CTAs; of 2048 x 40000, 16 tokens: 24, 32).
// Beyond, the sizes decide, by what the kernels were measured to take in us: a start, and
// so much a CTA and block of k that an SM takes, or a block of k for each wave of pairs.
//                                   mma.sync   pairs, 128 features   pairs, 256
//   K  4096  N 2048   64 tokens       7.9           14.4                20.3
//                    160             17.7           14.5                20.6
//   K  2048  N 5120   32              7.3            9.1                12.4
//                     64             11.3            9.4                12.6
//                    400             54             15.4                13.5
//                   1500              -             28.7                23.9
//   K  2000  N 1003  100              5.6            9.0                12.7
//                    200              8.2            9.1                12.9
//                    777             24              9.4                13.2
//                   3000              -             16.7                14.5
//   K 16384  N  512  256             22             45                  66
//   K   512  N 2048  100              4.5            5.7                 7.1
//                    192              6.5            5.7                 7.3
//   K   256  N  256 2000              7.0            5.0                 6.4
cudaError_t launch_linear_fp8(const LinearArgs& a, int num_sms, cudaStream_t st) {
    if (a.T <= 16) return launch_linear_few(a, st);
    auto waves = [](int64_t work, int at_once) { return (double)((work + at_once - 1) / at_once); };
    const double kb = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int group = linear_few_group(a.T);
    const int64_t token_tiles = (a.T + 255) / 256, ctas = (int64_t)((a.N + LF_ROWS - 1) / LF_ROWS) * ((a.T + group - 1) / group);
    const double each = group == 16 ? 0.35 + 0.057 * kb : 0.45 + 0.095 * kb;
    const double few = 2.0 + each * (ctas < num_sms ? 1.0 : (double)ctas / num_sms);
    const double p128 = 3.7 + 0.33 * kb * waves(token_tiles * ((a.N + 127) / 128), num_sms / 2);
    const double p256 = 4.7 + 0.52 * kb * waves(token_tiles * ((a.N + 255) / 256), num_sms / 2);
    if (few <= p128 && few <= p256 && a.T <= 32 * 65535) return launch_linear_few(a, st);   // a grid's second size
    return launch_linear_pair(a, p128 < p256 ? 128 : 256, num_sms, st);
}

}  // namespace qmoe
