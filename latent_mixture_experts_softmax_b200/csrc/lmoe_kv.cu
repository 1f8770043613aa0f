// The 8-bit paged KV cache: rows quantised as they are written, and read
// back.  Layout and rules: include/lmoe.h.
//
// Both kernels are copies with a little arithmetic, bound by HBM: a write
// reads 2 bytes an element and stores 1 (and 4 a row), a read the reverse.
// A row's D elements are spread over D / 8 lanes, 16 bytes of bf16 each, so
// a row's maximum is a few shuffles and every access of a warp is whole
// 32-byte sectors.

#include "lmoe_mixers.cuh"

namespace lmoe {

namespace {

constexpr int kThreads = 256;

// Row r's sequence: the first s with q_start[s + 1] > r; n_seqs if none.
__device__ __forceinline__ int seq_of_row(const KvParams& p, int r) {
    int lo = 0, hi = p.n_seqs;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.q_start + mid + 1) > r) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Place of token row r in the cache: >= 0 the row in the scale arrays of key
// head 0, -1 the row is to be left alone, -2 the token has no place (a
// negative position, or a page that is not there).
__device__ __forceinline__ long long place_of_row(const KvParams& p, int r) {
    const int s = seq_of_row(p, r);
    if (s >= p.n_seqs) return -1;
    const SeqRows q = seq_rows(p, s);
    if (q.n < 0 || r < q.q0 || r >= q.q0 + q.n) return -1;
    const int pos = q.kv - q.n + (r - q.q0);
    if (pos < 0) return -2;
    const int page = __ldg(p.table + (size_t)s * p.table_stride + (pos >> p.page_log2));
    if (page < 0 || page >= p.n_pages) {
        set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
        return -2;
    }
    return (long long)page_row(p, page, 0) + (pos & ((1 << p.page_log2) - 1));
}

__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// One row of D elements per D / 8 lanes; grid.y: 0 keys, 1 values.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvParams p, const uint16_t* __restrict__ kx,
                                                        const uint16_t* __restrict__ vx, size_t k_stride,
                                                        size_t v_stride) {
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x % LANES;
    const size_t item = (size_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int tok = (int)(item / p.Hk), head = (int)(item % p.Hk);
    const bool is_v = blockIdx.y == 1;
    const long long place = tok < p.n_tokens ? place_of_row(p, tok) : -1;
    uint4 w = make_uint4(0, 0, 0, 0);
    if (place >= 0) {
        const uint16_t* src = is_v ? vx + (size_t)tok * v_stride : kx + (size_t)tok * k_stride;
        w = ldg_stream(reinterpret_cast<const uint4*>(src + (size_t)head * D + lane * 8));
    }
    // max |x| as bf16 bits (their order is that of the magnitudes, NaN last)
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (place < 0) return;
    float a = bf16_bits_to_f32(m);
    constexpr float kTop = FMT == LMOE_KV_INT8 ? 127.f : 448.f;
    float scale = __fdiv_rn(a, kTop);
    uint32_t c[2] = {0, 0};
    if (m >= 0x7f80u) {                       // infinity or NaN
        scale = __int_as_float(0x7fffffff);
        set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
    } else if (a < 0x1p-100f) {
        scale = 1.f;
    } else {
        // code = round(top * x / a).  top * x is exact (8 + 7 bits), so the
        // correctly rounded quotient decides as exact arithmetic does: a
        // quotient that is no tie is at least 2^-9 of a step away from one.
        // Rows beyond 2^64 are scaled down by a power of two first, so that
        // the product stays finite.
        const float f = a > 0x1p64f ? 0x1p-64f : 1.f;
        a *= f;
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = bf16x2_to_f32x2(u[i]);
            y[2 * i] = __fdiv_rn(x.x * f * kTop, a);
            y[2 * i + 1] = __fdiv_rn(x.y * f * kTop, a);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (FMT == LMOE_KV_INT8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i] |= (uint32_t)(__float2int_rn(y[4 * i + j]) & 0xff) << (8 * j);
            } else {
                c[i] = e4m3x2_of(y[4 * i], y[4 * i + 1]) | e4m3x2_of(y[4 * i + 2], y[4 * i + 3]) << 16;
            }
        }
    }
    const size_t row = (size_t)place + ((size_t)head << p.page_log2);
    *reinterpret_cast<uint2*>((is_v ? p.v : p.k) + row * D + lane * 8) = make_uint2(c[0], c[1]);
    if (lane == 0) (is_v ? p.vs : p.ks)[row] = scale;
}

// One row per D / 8 lanes, as above.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvParams p, uint16_t* __restrict__ ky, uint16_t* __restrict__ vy,
                                                      size_t k_stride, size_t v_stride) {
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x % LANES;
    const size_t item = (size_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    const int tok = (int)(item / p.Hk), head = (int)(item % p.Hk);
    const bool is_v = blockIdx.y == 1;
    if (tok >= p.n_tokens) return;
    const long long place = place_of_row(p, tok);
    if (place == -1) return;
    uint32_t o[4] = {0, 0, 0, 0};
    if (place >= 0) {
        const size_t row = (size_t)place + ((size_t)head << p.page_log2);
        const float scale = __ldg((is_v ? p.vs : p.ks) + row);
        const uint2 c = __ldg(reinterpret_cast<const uint2*>((is_v ? p.v : p.k) + row * D + lane * 8));
        float y[8];
        if (FMT == LMOE_KV_INT8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (float)(int8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        } else {
            float lo[4], hi[4];
            e4m3x4_to_f32x4(c.x, lo);
            e4m3x4_to_f32x4(c.y, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) { y[i] = lo[i]; y[4 + i] = hi[i]; }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = (uint32_t)f32_to_bf16_bits(y[2 * i] * scale) | (uint32_t)f32_to_bf16_bits(y[2 * i + 1] * scale) << 16;
    }
    uint16_t* dst = is_v ? vy + (size_t)tok * v_stride : ky + (size_t)tok * k_stride;
    *reinterpret_cast<uint4*>(dst + (size_t)head * D + lane * 8) = make_uint4(o[0], o[1], o[2], o[3]);
}

dim3 row_grid(const KvParams& p) {
    const size_t rows = (size_t)p.n_tokens * p.Hk, per = kThreads / (p.D / 8);
    return dim3((unsigned)((rows + per - 1) / per), 2);
}

}  // namespace

cudaError_t run_kv_append(const KvParams& p, const uint16_t* k, const uint16_t* v, size_t k_stride, size_t v_stride,
                          cudaStream_t st) {
    const dim3 g = row_grid(p);
    auto go = [&](auto kernel) { kernel<<<g, kThreads, 0, st>>>(p, k, v, k_stride, v_stride); };
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) i8 ? go(k_kv_append<64, LMOE_KV_INT8>) : go(k_kv_append<64, LMOE_KV_E4M3>);
    else if (p.D == 128) i8 ? go(k_kv_append<128, LMOE_KV_INT8>) : go(k_kv_append<128, LMOE_KV_E4M3>);
    else i8 ? go(k_kv_append<256, LMOE_KV_INT8>) : go(k_kv_append<256, LMOE_KV_E4M3>);
    return cudaGetLastError();
}

cudaError_t run_kv_read(const KvParams& p, uint16_t* k, uint16_t* v, size_t k_stride, size_t v_stride,
                        cudaStream_t st) {
    const dim3 g = row_grid(p);
    auto go = [&](auto kernel) { kernel<<<g, kThreads, 0, st>>>(p, k, v, k_stride, v_stride); };
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) i8 ? go(k_kv_read<64, LMOE_KV_INT8>) : go(k_kv_read<64, LMOE_KV_E4M3>);
    else if (p.D == 128) i8 ? go(k_kv_read<128, LMOE_KV_INT8>) : go(k_kv_read<128, LMOE_KV_E4M3>);
    else i8 ? go(k_kv_read<256, LMOE_KV_INT8>) : go(k_kv_read<256, LMOE_KV_E4M3>);
    return cudaGetLastError();
}

}  // namespace lmoe
