// kv4_attn.cu -- causal GQA attention of a ragged batch of tokens over the paged
// 4-bit cache.
//
// Row (token i of the N new ones of a sequence of len positions, q head h) sees
// the positions p <= len - N + i:  z_p = scale q.k_p, o = sum softmax(z)_p v_p.
#include <math.h>

#include "kv4.cuh"
#include "ptx_sync.cuh"

namespace qmoe {

namespace {

constexpr int AS_THREADS = 128;

// one CTA per (token row, q head), warp w owns positions w, w+4, ...; lane l holds
// the elements 2 l + 64 j, 2 l + 64 j + 1
__global__ void __launch_bounds__(AS_THREADS) kv4_attention_simple(const Kv4AttnArgs a) {
    pdl_wait();
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hd = a.s.hd, n2 = hd / 64, g = h / (a.s.nq / a.s.nkv);
    int s = -1;
    Kv4Seq q{0, 0, 0};
    for (int i = 0; i < a.n_seqs; ++i) {
        Kv4Seq r;
        if (!kv4_seq(a, i, r)) {
            if (threadIdx.x == 0) atomicExch(a.status, ST_DEVICE_CHECK);
        } else if (row >= r.q0 && row < r.q0 + r.n) {
            s = i;
            q = r;
        }
    }
    if (s < 0) return;
    const int seen = max(0, q.len - q.n + (row - q.q0) + 1);
    float2 qv[4], acc[4];
    for (int j = 0; j < n2; ++j) {
        const size_t at = (size_t)row * a.q_stride + (size_t)h * hd + 2 * lane + 64 * j;
        qv[j] = make_float2(kv4_load(a.q, at, a.q_t), kv4_load(a.q, at + 1, a.q_t));
        acc[j] = make_float2(0.f, 0.f);
    }
    const float kscale = a.scale * a.c.kg[g];
    float m = -INFINITY, l = 0.f;
    for (int p = warp; p < seen; p += AS_THREADS / 32) {
        const int pg = a.table[(size_t)s * a.s.width + p / a.s.page];
        if (pg < 0 || pg >= a.s.n_pages) {
            if (lane == 0) atomicExch(a.status, ST_DEVICE_CHECK);
            continue;
        }
        const size_t at = ((size_t)pg * a.s.nkv + g) * a.s.page + p % a.s.page;
        float z = 0.f;
        for (int j = 0; j < n2; ++j) {
            const float2 c = e2m1x2_f2(a.c.kc[at * (hd / 2) + lane + 32 * j]);
            z += (qv[j].x * c.x + qv[j].y * c.y) * e4m3_f(a.c.ks[at * (hd / 16) + (lane + 32 * j) / 8]);
        }
        z = group_sum<32>(z) * kscale;
        const float mn = fmaxf(m, z);
        const float corr = m == -INFINITY ? 0.f : expf(m - mn), e = expf(z - mn);
        l = l * corr + e;
        m = mn;
        for (int j = 0; j < n2; ++j) {
            const float2 c = e2m1x2_f2(a.c.vc[at * (hd / 2) + lane + 32 * j]);
            const float sv = e * e4m3_f(a.c.vs[at * (hd / 16) + (lane + 32 * j) / 8]);
            acc[j].x = acc[j].x * corr + sv * c.x;
            acc[j].y = acc[j].y * corr + sv * c.y;
        }
    }
    __shared__ float sm[AS_THREADS / 32], sl[AS_THREADS / 32], so[AS_THREADS / 32][256];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    for (int j = 0; j < n2; ++j) {
        so[warp][2 * lane + 64 * j] = acc[j].x;
        so[warp][2 * lane + 64 * j + 1] = acc[j].y;
    }
    __syncthreads();
    float mt = -INFINITY, lt = 0.f;
    for (int w = 0; w < AS_THREADS / 32; ++w) mt = fmaxf(mt, sm[w]);
    for (int w = 0; w < AS_THREADS / 32; ++w) lt += sl[w] == 0.f ? 0.f : sl[w] * expf(sm[w] - mt);
    const float inv = lt > 0.f ? a.c.vg[g] / lt : 0.f;
    for (int d = threadIdx.x; d < hd; d += AS_THREADS) {
        float o = 0.f;
        for (int w = 0; w < AS_THREADS / 32; ++w) o += sl[w] == 0.f ? 0.f : so[w][d] * expf(sm[w] - mt);
        kv4_store(a.out, (size_t)row * a.out_stride + (size_t)h * hd + d, a.out_t, o * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)row * a.s.nq + h] = lt > 0.f ? mt + logf(lt) : -INFINITY;
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t st) {
    return launch_pdl(kv4_attention_simple, dim3(a.n_tokens, a.s.nq), dim3(AS_THREADS), 0, st, a);
}

}  // namespace qmoe
