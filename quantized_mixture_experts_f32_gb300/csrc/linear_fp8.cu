// linear_fp8.cu -- which kernel of qmoe_linear_fp8 takes a call.
#include <math.h>

#include "linear_fp8.cuh"

namespace qmoe {

// Up to 16 tokens go to mma.sync, whose CTAs read W once and wait for nothing else (W of
// 2048 x 5120, one token: 3.3 us, 9 on a pair of CTAs; of 2048 x 40000, 16 tokens: 21, 32).
// Beyond, the sizes decide, by what the kernels were measured to take in us: a start, and
// so much a CTA and block of k that an SM takes, or a block of k for each wave of pairs.
//                                 mma.sync  pairs, 256 features  128   k shared by 2     3     4
//   K  4096  N 2048   64 tokens     7.9           20.3          14.4       10.8   10.1  17.5
//                    256           24.9           20.6          14.6       11.4   10.6  18.8
//                    500           43                           14.6       11.7   20.8  28.3
//   K  2048  N 5120   32            7.3           12.4           9.1
//                     64           11.3           12.6           9.4
//                    400           54             13.5          15.4
//                   1500            -             23.9          28.7
//   K  2000  N 1003  100            5.7           12.7           9.0        8.2    8.5   7.9
//                    200            8.1           12.9           9.1        8.4    8.7   8.0
//                    777           24             13.2           9.4        8.8   17.3  22.8
//                   3000            -             14.5          16.7
//   K 16384  N  512   30            9.5                         44         25.6   19.6  15.9
//                    256           22.3           66            45         26.6   20.4  16.8
//                   1000           80                           46         27.1   21.2  33.9
//   K   512  N 2048  100            4.5            7.1           5.7
//                    192            6.5            7.3           5.7
//   K   256  N  256 2000            7.0            6.4           5.0
LinearChoice linear_fp8_choice(int T, int K, int N, int num_sms) {
    if (T <= 16) return {0, 1};
    auto waves = [](int64_t work, int at_once) { return (double)((work + at_once - 1) / at_once); };
    const double kb = (K + FP8_BLOCK - 1) / FP8_BLOCK;
    const int group = linear_few_group(T);
    const int64_t token_tiles = (T + 255) / 256, ctas = (int64_t)((N + LF_ROWS - 1) / LF_ROWS) * ((T + group - 1) / group);
    const double each = group == 16 ? 0.35 + 0.057 * kb : 0.45 + 0.095 * kb;
    const double few = 2.0 + each * (ctas < num_sms ? 1.0 : (double)ctas / num_sms);
    const double p128 = 3.7 + 0.33 * kb * waves(token_tiles * ((N + 127) / 128), num_sms / 2);
    const double p256 = 4.7 + 0.52 * kb * waves(token_tiles * ((N + 255) / 256), num_sms / 2);
    // a tile's k shared by 2, 3 or 4 pairs, where such clusters fit the GPU at once (36, 21 and 15 on
    // 152 SMs): 5.2 us, 0.3 a pair, and its blocks of k, in groups of four
    const int64_t tiles = token_tiles * ((N + 127) / 128), groups = ((int64_t)kb + 3) / 4;
    double split = 1e30;
    int parts = 1;
    for (int p = 2; p <= 4; ++p) {
        if (tiles > (p == 2 ? num_sms / 4 - 2 : num_sms / (p == 3 ? 7 : 10)) || groups < p) break;
        const double t = 5.2 + 0.3 * p + 0.33 * 4.0 * (double)((groups + p - 1) / p);
        if (t < split) {
            split = t;
            parts = p;
        }
    }
    const double pairs = fmin(fmin(p128, p256), split);
    if (few <= pairs && T <= 32 * 65535) return {0, 1};       // a grid's second size
    if (split < p128 && split < p256) return {128, parts};
    return {p128 < p256 ? 128 : 256, 1};
}

cudaError_t launch_linear_fp8(const LinearArgs& a, const LinearRun& run) {
    const LinearChoice c = linear_fp8_choice(a.T, a.K, a.N, run.num_sms);
    return c.tile ? launch_linear_pair(a, c.tile, c.parts, run) : launch_linear_few(a, run.num_sms, run.st);
}

}  // namespace qmoe
