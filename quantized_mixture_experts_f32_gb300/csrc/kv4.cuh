// kv4.cuh -- the paged 4-bit KV cache: what its kernels and the C ABI share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lowbit.cuh"
#include "pdl.cuh"

namespace qmoe {

enum : int { KV4_F32 = 0, KV4_F16 = 1, KV4_BF16 = 2 };

// Geometry of every layer's cache and the table that maps positions to pages.
struct Kv4Shape {
    int nq, nkv, hd, page, n_pages, width;   // width: columns of the block table
    int page_log2;
};

// One layer's cache.  codes [n_pages][nkv][page][hd/2], scales [n_pages][nkv][page][hd/16]
struct Kv4Cache {
    uint8_t* kc;
    uint8_t* ks;
    uint8_t* vc;
    uint8_t* vs;
    const float* kg;
    const float* vg;
};

struct Kv4PlanArgs {
    int n, page, n_pages, width, cap;
    const int32_t* seq_len;
    const int32_t* new_len;
    int32_t* table;
    int32_t* free_pages;
    const int32_t* n_free;
    int32_t* seq_len_out;
    int32_t* n_free_out;
    int32_t* cu;
    int32_t* positions;
    int64_t* slots;
    unsigned* arrive;     // zero between launches
    int* status;
};
cudaError_t kv4_plan_prepare();           // shared-memory limits, once a device
cudaError_t launch_kv4_plan(const Kv4PlanArgs& a, int num_sms, cudaStream_t st);

struct Kv4AppendArgs {
    Kv4Shape s;
    Kv4Cache c;
    const void* k;
    const void* v;
    int dtype, n_tokens;
    int64_t k_stride, v_stride;   // elements between rows
    const int64_t* slots;
    float* k_hat;
    float* v_hat;
    int* status;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t st);

struct Kv4AttnArgs {
    Kv4Shape s;
    Kv4Cache c;
    const void* q;
    int q_t, out_t;
    int64_t q_stride, out_stride;
    int n_seqs, n_tokens, max_new;
    const int32_t* cu;
    const int32_t* seq_len;
    const int32_t* table;
    float scale;
    void* out;
    float* lse;
    int* status;
};
// Attention: sequences of at most few_rows rows (new tokens x heads of a group) by
// launch_kv4_decode, the others by launch_kv4_extend.  The two may run side by side, so
// each has its own workspace, zero between launches but for the parts.
struct Kv4Work {
    float *parts, *ext_parts;          // parts of items that several CTAs share
    unsigned *arrive, *ext_arrive;     // [kv4_arrive_words] each: arrival counters of those items
    unsigned* ext_total;               // pieces the prompt kernel works on, while it does
    int num_sms;
    unsigned long long stall_ns;       // test hook: parts of split items are handed over this much later
};
constexpr int KV4_FEW_ROWS = 16;       // few_rows at least
size_t kv4_decode_part_floats(int hd, int num_sms);
size_t kv4_extend_part_floats(int hd, int num_sms, long long max_rows);   // rows: tokens x heads of a group
cudaError_t kv4_decode_prepare();
cudaError_t kv4_extend_prepare();
// behind: launched right after launch_kv4_extend on the stream
cudaError_t launch_kv4_decode(const Kv4AttnArgs& a, int few_rows, bool behind, const Kv4Work& w, cudaStream_t st);
cudaError_t launch_kv4_extend(const Kv4AttnArgs& a, int few_rows, const Kv4Work& w, cudaStream_t st);
int kv4_arrive_words(int num_sms);
cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, const Kv4Work& w, cudaStream_t st);

// What qmoe_step_kv4 needs of a handle.
struct Kv4View {
    Kv4Shape s;
    Kv4Work w;
    int* status;
    unsigned long long* stall_ns;      // of the next attention, zeroed by whoever launches it
    cudaStream_t stream;
    int device, max_seqs, max_tokens;
};

// A sequence's part of a call: rows q0 .. q0+n-1 are its last n of len positions.
// False (and ok cleared) where the device arrays hold values out of range.
struct Kv4Seq {
    int q0, n, len;
};
__device__ __forceinline__ bool kv4_seq(const Kv4AttnArgs& a, int s, Kv4Seq& r) {
    r.q0 = a.cu[s];
    const int q1 = a.cu[s + 1];
    r.len = a.seq_len[s];
    const bool good = r.q0 >= 0 && q1 >= r.q0 && q1 <= a.n_tokens && q1 - r.q0 <= a.max_new && r.len >= 0 &&
                      (int64_t)r.len <= (int64_t)a.s.width * a.s.page;
    r.n = good ? q1 - r.q0 : 0;
    if (!good) r.len = 0;
    return good;
}

}  // namespace qmoe
