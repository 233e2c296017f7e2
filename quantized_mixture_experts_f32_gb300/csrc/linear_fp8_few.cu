// linear_fp8_few.cu -- qmoe_linear_fp8 for a few tokens, on mma.sync (m16n8k16, F16).
//
// The call is W's bytes and latency, so everything that costs a wait is left out: codes go
// from global memory through registers into the products (E4M3 is exact in F16, the
// products in fp32), W's 16 rows as the first operand, eight tokens as the second.
// tcgen05 would need W in shared memory, TMEM taken and given back, and three hand-overs.
// A lane loads 16 neighbouring codes of a row; which k a product's position means is
// free as long as both operands agree, so they serve four products of 16 as they lie.
//
// One token, W of 2048 x 5120: 3.3 us, 3.1 TB/s (2048 x 40000: 16.1 us, 5.1 TB/s; x 151936:
// 52.5 us, 5.9 TB/s), bound by one chain of load, products and join.  Long rows are that chain
// several times, as k is not shared by CTAs and a warp's next loads begin behind its products:
// 8192 x 8192 from HBM 16.4 us (10.0 for W's bytes), 16384 x 512 7.5 us on 32 CTAs (1.3), x 128 7.2.
// 64 tokens, 4096 x 2048: 8.0 us (8.4 with a residual), bound by its loads' latency with two CTAs an SM (21%
// of the warps; long_scoreboard 5.9 an issue, math_pipe_throttle 0.8, tensor pipe 22%).  Copies by
// cp.async (9.2 when this took 8.0), products on E4M3 directly (12.9, emulated) and 32 features a CTA (15.2) were no faster.
#include "linear_fp8.cuh"

namespace qmoe {

namespace {

constexpr int LF_WARPS = 8;                   // of a CTA: 16 features, k dealt between them

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 codes -> eight pairs in F16
__device__ __forceinline__ void widen16(const uint4& u, uint32_t (&h)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = kv4_u(kv4_scale2(w[i] & 0xffffu));
        h[2 * i + 1] = kv4_u(kv4_scale2(w[i] >> 16));
    }
}

// (out of line: it keeps the products' registers to themselves, 3.35 -> 3.25 us one token, 2048 x 5120)
__device__ __noinline__ float activate1(float z, int act) {
    float v[1] = {z};
    activate(v, act);
    return v[0];
}

// CTAs that an SM holds
constexpr int lf_ctas(int nt, int u) { return nt == 4 ? 2 : (nt == 1 ? 4 : 3) - (u == 2); }

// NT tiles of eight tokens.  A warp takes every eighth block of k, U at a time, with all
// their loads on the way before the first is used.
template <int NT, int U>
__global__ void __launch_bounds__(LF_WARPS * 32, lf_ctas(NT, U)) linear_few_kernel(const LinearArgs a, bool ahead) {
    __shared__ float part[LF_WARPS][NT * 8][LF_ROWS];
    if (ahead && threadIdx.x < LF_ROWS && blockIdx.y == 0) {  // W's rows into L2, whatever runs before
        const uint8_t* row = a.w + (size_t)min((int)blockIdx.x * LF_ROWS + (int)threadIdx.x, a.N - 1) * a.K;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row), "r"(a.K) : "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int t0 = (int)blockIdx.y * 8 * NT;                  // this CTA's tokens
    const int n0 = (int)blockIdx.x * LF_ROWS, kb_all = (a.K + FP8_BLOCK - 1) / FP8_BLOCK;
    const uint8_t* w0 = a.w + (size_t)min(n0 + g, a.N - 1) * a.K;
    const uint8_t* w1 = a.w + (size_t)min(n0 + g + 8, a.N - 1) * a.K;
    const float* ws = a.ws + (size_t)(n0 / FP8_BLOCK) * kb_all;
    float z[NT][4] = {};
    for (int kb0 = warp; kb0 < kb_all; kb0 += U * LF_WARPS) {
        uint4 wa[U][2], wb[U][2], x[U][2][NT];
        float s[U], xs[U][NT][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * LF_WARPS;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kb * FP8_BLOCK + h * 64 + c * 16;
                const bool in = k < a.K;
                wa[u][h] = in ? ld_stream(w0 + k) : make_uint4(0, 0, 0, 0);
                wb[u][h] = in ? ld_stream(w1 + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    x[u][h][j] = in ? __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)min(t0 + 8 * j + g, a.T - 1) * a.K + k))
                                    : make_uint4(0, 0, 0, 0);
            }
            const int at = min(kb, kb_all - 1);
            s[u] = __ldg(ws + at);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) xs[u][j][i] = __ldg(a.xs + (size_t)min(t0 + 8 * j + 2 * c + i, a.T - 1) * kb_all + at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb0 + u * LF_WARPS >= kb_all) break;          // the same for the whole warp
            float d[NT][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[8], q[8], r[8];
                widen16(wa[u][h], p);
                widen16(wb[u][h], q);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    widen16(x[u][h][j], r);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) mma_f16(d[j], p[i], q[i], p[i + 1], q[i + 1], r[i], r[i + 1]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[j][i] = fmaf(d[j][i], s[u] * xs[u][j][i & 1], z[j][i]);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][8 * j + 2 * c + (i & 1)][g + 8 * (i >> 1)] = z[j][i];
    __syncthreads();
    // the warps' sums in their order
    const int rows = min(8 * NT, a.T - t0);
    for (int i = (int)threadIdx.x; i < LF_ROWS * rows; i += LF_WARPS * 32) {
        const int t = i / LF_ROWS, f = i % LF_ROWS, n = n0 + f;
        if (n >= a.N) continue;
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < LF_WARPS; ++k) v += part[k][t][f];
        if (a.bias) v += a.bias[n];
        if (a.act) v = activate1(v, a.act);
        put_one(a, t0 + t, n, v);
    }
}

}  // namespace

// Groups of 16 tokens up to 32, of 32 beyond: more CTAs against W read (from L2) again.
// In us, groups of 16 / 32 / 64 tokens:
//   K 4096  N 2048   32 tokens   5.5   5.8   7.6      64 tokens    9.6    8.2    8.0
//   K 2048  N 5120               7.3   7.4  11.6                  12.2   11.2   12.9
//   K 2000  N 1003               2.8   3.9   4.8                   3.9    4.1    5.5
//
// Up to 32 tokens two blocks of k at a time, or one with one more CTA an SM where that saves a
// wave of CTAs.  In us: 16 tokens 2048 x 5120 5.9 / 4.85, x 40000 24.2 / 21.3, one token x 40000
// 17.3 / 16.1, x 151936 56 / 52.5; where it saves none 4096 x 2048 4.3 / 5.2, 8192 x 8192 19.3 / 21.2
// (16 tokens), 2048 x 5120 3.35 / 3.9 (one).
//
// Where all CTAs run at once they ask for their rows of W before they wait for the kernel before
// (W from HBM, in us: one token 2048 x 5120 4.1 -> 3.3, 4096 x 2048 4.3 -> 3.95, 64 tokens 9.1 ->
// 8.4); in several waves it only adds requests (8192 x 8192, one token 15.9 -> 16.9).
cudaError_t launch_linear_few(const LinearArgs& a, int num_sms, cudaStream_t st) {
    const unsigned group = (unsigned)linear_few_group(a.T);
    const dim3 block(LF_WARPS * 32), grid((unsigned)((a.N + LF_ROWS - 1) / LF_ROWS), ((unsigned)a.T + group - 1) / group);
    const uint64_t ctas = (uint64_t)grid.x * grid.y;
    auto waves = [&](int u) { return (ctas - 1) / ((uint64_t)lf_ctas((int)group / 8, u) * (uint64_t)num_sms) + 1; };
    const int u = group == 32 || waves(1) < waves(2) ? 1 : 2;
    const bool ahead = waves(u) == 1;
    if (group == 8)
        return u == 1 ? launch_pdl(linear_few_kernel<1, 1>, grid, block, 0, st, a, ahead) : launch_pdl(linear_few_kernel<1, 2>, grid, block, 0, st, a, ahead);
    if (group == 16)
        return u == 1 ? launch_pdl(linear_few_kernel<2, 1>, grid, block, 0, st, a, ahead) : launch_pdl(linear_few_kernel<2, 2>, grid, block, 0, st, a, ahead);
    return launch_pdl(linear_few_kernel<4, 1>, grid, block, 0, st, a, ahead);
}

}  // namespace qmoe
