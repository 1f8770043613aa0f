// Token mixers: parameters shared by the C-ABI layer and the kernels, and
// the device helpers that read a batch description.
#pragma once

#include <atomic>

#include "lmoe_internal.cuh"

namespace lmoe {

constexpr int kAttnCtrlBytes = 4096;   // control block at the start of a mixer's workspace
constexpr int kSms = 148;              // SMs of a B200

// Raise a kernel's dynamic shared-memory limit, once per device (calls from
// several host threads may meet here).
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(Kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

struct KvParams {
    // shape
    int Hq, Hk, G, D, fmt;      // G = Hq / Hk query heads per key head
    int page_log2;
    // cache
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int n_pages;
    // batch
    const int32_t* q_start;
    const int32_t* kv_len;
    const int32_t* table;
    int n_seqs, table_stride, n_tokens, max_new;
    Ctrl* ctrl;
};

// The new tokens of one sequence; n < 0: the sequence is left out.
struct SeqRows {
    int q0, n, kv;
};

__device__ __forceinline__ SeqRows seq_rows(const KvParams& p, int s) {
    SeqRows r;
    r.q0 = __ldg(p.q_start + s);
    const int q1 = __ldg(p.q_start + s + 1);
    r.kv = __ldg(p.kv_len + s);
    r.n = q1 - r.q0;
    if (r.q0 < 0 || q1 < r.q0 || q1 > p.n_tokens || r.n > p.max_new || r.kv < 0 ||
        (long long)r.kv > ((long long)p.table_stride << p.page_log2)) {
        set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
        r.n = -1;
    }
    return r;
}

// First row of a page and head in the scale arrays (times D: in the codes).
__device__ __forceinline__ size_t page_row(const KvParams& p, int page, int head) {
    return ((size_t)page * p.Hk + head) << p.page_log2;
}

struct AttendParams : KvParams {
    const uint16_t* q;
    size_t q_stride;
    float scale_log2;      // softmax scale * log2(e)
    int causal, window;
    uint16_t* out;
    float* lse;
    int4* cuts;            // per CTA: the item it began and others go on with
    float* part;           // parts of items cut between CTAs
    int h0, Hn;            // key heads of this launch
    char* img;             // images of key tiles [sequence][head of the launch][tile]
    int img_tiles;
};

struct DeltaParams {
    int H, Hq, group, DK, DV, l2norm;
    const int32_t* q_start;
    const int32_t* src;
    const int32_t* dst;
    int n_seqs, n_states, n_tokens, max_new;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    size_t qs, ks, vs;
    const float* log_decay;
    const float* beta;
    float scale;
    float* states;
    uint16_t* out;
    Ctrl* ctrl;
    char* chunk_ws;        // per-chunk matrices of the chunked form
};

cudaError_t run_kv_append(const KvParams& p, const uint16_t* k, const uint16_t* v, size_t k_stride, size_t v_stride,
                          cudaStream_t st);
cudaError_t run_kv_read(const KvParams& p, uint16_t* k, uint16_t* v, size_t k_stride, size_t v_stride,
                        cudaStream_t st);
size_t attend_ws_bytes(int D);
cudaError_t run_attend(AttendParams p, void* ws, cudaStream_t st);
size_t delta_chunk_ws_bytes(int H, int n_tokens, int n_seqs, int max_new);
cudaError_t run_delta(const DeltaParams& p, cudaStream_t st);

}  // namespace lmoe
