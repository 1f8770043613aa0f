// The 8-bit paged KV cache: rows quantised as they are written, and read
// back.  Layout and rules: include/lmoe.h.
//
// Both kernels are copies with a little arithmetic, bound by HBM: a write
// reads 2 bytes an element and stores 1 (and 4 a row), a read the reverse.
// A block takes some tokens, looks up their places once (a search, the
// sequence's lengths and its page: four loads one behind the other, which a
// thread per row paid for every 16 bytes), and then moves their rows, four
// 8-element pieces in flight per thread.  A row's D elements are spread over
// D / 8 lanes, 16 bytes of bf16 each, so a row's maximum is a few shuffles and
// every access of a warp is whole 32-byte sectors.

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

// To the nearest number of 20 significant bits.
__device__ __forceinline__ float bits20(float x) { return __uint_as_float((__float_as_uint(x) + 8u) & ~15u); }

constexpr int kPieces = 4;        // pieces in flight per thread
constexpr int kMaxTokens = 64;    // tokens of a block

// Places of the block's tokens.
__device__ __forceinline__ void find_places(const KvParams& p, long long (&place)[kMaxTokens], int tok0, int n) {
    if ((int)threadIdx.x < n) place[threadIdx.x] = place_of_row(p, tok0 + threadIdx.x);
    __syncthreads();
}

// grid.x: runs of `tokens` tokens; grid.y: 0 keys, 1 values.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvParams p, const uint16_t* __restrict__ kx,
                                                        const uint16_t* __restrict__ vx, size_t k_stride,
                                                        size_t v_stride, int tokens) {
    constexpr int LANES = D / 8;
    __shared__ long long s_place[kMaxTokens];
    const bool is_v = blockIdx.y == 1;
    const int tok0 = blockIdx.x * tokens, n = min(tokens, p.n_tokens - tok0);
    find_places(p, s_place, tok0, n);
    const uint16_t* src = is_v ? vx : kx;
    const size_t stride = is_v ? v_stride : k_stride;
    uint8_t* codes = is_v ? p.v : p.k;
    float* scales = is_v ? p.vs : p.ks;
    const int total = n * p.Hk * LANES, lane = threadIdx.x % LANES;
    for (int base = 0; base < total; base += kThreads * kPieces) {
        uint4 w[kPieces];
        long long row[kPieces];                // the row in the scale arrays, -1: none
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            // (every load has a place to read, so that none waits for a condition)
            const int r = min(base + i * kThreads + (int)threadIdx.x, total - LANES + lane) / LANES;
            const int tok = r / p.Hk, head = r - tok * p.Hk;
            const long long place = s_place[tok];
            row[i] = place >= 0 && base + i * kThreads + (int)threadIdx.x < total
                         ? place + ((long long)head << p.page_log2) : -1;
            w[i] = ldg_stream(reinterpret_cast<const uint4*>(src + (size_t)(tok0 + tok) * stride + (size_t)head * D + lane * 8));
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            // max |x| as bf16 bits (their order is that of the magnitudes, NaN last)
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) m = max(m, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (row[i] < 0) continue;
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
                // code = round(top * x / a).  top * x is exact (8 + 7 bits).  The
                // quotient is a tie of the codes' grid or at least 2^-16 of itself
                // away from one (x = X 2^i, a = A 2^j with X, A < 2^8, top < 2^7
                // or 7 2^6: what separates it from a tie is a whole number over a
                // product of two of these).  The product with the reciprocal is
                // within 2^-22 of it, and rounded to 20 bits it stands on the
                // tie, or on the quotient's side of it.  (Prompts of 16358
                // tokens, 50 MB: 19 us; 23 us with a division each.)  Rows
                // beyond 2^64 are scaled down by a power of two first, so that the
                // product stays finite.
                const float f = a > 0x1p64f ? 0x1p-64f : 1.f;
                const float inv = __frcp_rn(a * f);
                float y[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = bf16x2_to_f32x2(u[j]);
                    y[2 * j] = bits20(x.x * f * kTop * inv);
                    y[2 * j + 1] = bits20(x.y * f * kTop * inv);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (FMT == LMOE_KV_INT8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[j] |= (uint32_t)(__float2int_rn(y[4 * j + e]) & 0xff) << (8 * e);
                    } else {
                        c[j] = e4m3x2_of(y[4 * j], y[4 * j + 1]) | e4m3x2_of(y[4 * j + 2], y[4 * j + 3]) << 16;
                    }
                }
            }
            *reinterpret_cast<uint2*>(codes + row[i] * D + lane * 8) = make_uint2(c[0], c[1]);
            if (lane == 0) scales[row[i]] = scale;
        }
    }
}

// The same grid; a piece is 16 elements (half the requests of 8, and whole
// 32-byte stores a lane: 24.7 us before for a prefix of 32768 tokens).
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvParams p, uint16_t* __restrict__ ky, uint16_t* __restrict__ vy,
                                                      size_t k_stride, size_t v_stride, int tokens) {
    constexpr int LANES = D / 16;
    __shared__ long long s_place[kMaxTokens];
    const bool is_v = blockIdx.y == 1;
    const int tok0 = blockIdx.x * tokens, n = min(tokens, p.n_tokens - tok0);
    find_places(p, s_place, tok0, n);
    uint16_t* dst = is_v ? vy : ky;
    const size_t stride = is_v ? v_stride : k_stride;
    const uint8_t* codes = is_v ? p.v : p.k;
    const float* scales = is_v ? p.vs : p.ks;
    const int total = n * p.Hk * LANES, lane = threadIdx.x % LANES;
    for (int base = 0; base < total; base += kThreads * kPieces) {
        uint4 c[kPieces];
        float scale[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int r = min(base + i * kThreads + (int)threadIdx.x, total - LANES + lane) / LANES;
            const int tok = r / p.Hk, head = r - tok * p.Hk;
            const long long place = s_place[tok];      // (without one: row 0 is read and dropped)
            const size_t row = place >= 0 ? (size_t)place + ((size_t)head << p.page_log2) : 0;
            scale[i] = __ldg(scales + row);
            c[i] = ldg_stream(reinterpret_cast<const uint4*>(codes + row * D + lane * 16));
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int idx = base + i * kThreads + (int)threadIdx.x;
            if (idx >= total) continue;
            const int r = idx / LANES, tok = r / p.Hk, head = r - tok * p.Hk;
            const long long place = s_place[tok];
            if (place == -1) continue;
            const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[4];
                if (FMT == LMOE_KV_INT8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = (float)(int8_t)(w[j] >> (8 * e));
                } else {
                    e4m3x4_to_f32x4(w[j], y);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[2 * j + e]) : "f"(y[2 * e + 1] * scale[i]), "f"(y[2 * e] * scale[i]));
                    if (place < 0) o[2 * j + e] = 0;
                }
            }
            uint4* to = reinterpret_cast<uint4*>(dst + (size_t)(tok0 + tok) * stride + (size_t)head * D + lane * 16);
            to[0] = make_uint4(o[0], o[1], o[2], o[3]);
            to[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

// Tokens of a block: two rounds of pieces, or fewer where the tokens are too
// few to fill the SMs with that.
int block_tokens(const KvParams& p) {
    const int fill = 2 * kThreads * kPieces / (p.Hk * (p.D / 8)), spread = (p.n_tokens + kSms - 1) / kSms;
    const int n = fill < spread ? fill : spread;
    return n < 1 ? 1 : n > kMaxTokens ? kMaxTokens : n;
}

}  // namespace

cudaError_t run_kv_append(const KvParams& p, const uint16_t* k, const uint16_t* v, size_t k_stride, size_t v_stride,
                          cudaStream_t st) {
    const int tokens = block_tokens(p);
    const dim3 g((unsigned)((p.n_tokens + tokens - 1) / tokens), 2);
    auto go = [&](auto kernel) { kernel<<<g, kThreads, 0, st>>>(p, k, v, k_stride, v_stride, tokens); };
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) i8 ? go(k_kv_append<64, LMOE_KV_INT8>) : go(k_kv_append<64, LMOE_KV_E4M3>);
    else if (p.D == 128) i8 ? go(k_kv_append<128, LMOE_KV_INT8>) : go(k_kv_append<128, LMOE_KV_E4M3>);
    else i8 ? go(k_kv_append<256, LMOE_KV_INT8>) : go(k_kv_append<256, LMOE_KV_E4M3>);
    return cudaGetLastError();
}

cudaError_t run_kv_read(const KvParams& p, uint16_t* k, uint16_t* v, size_t k_stride, size_t v_stride,
                        cudaStream_t st) {
    const int tokens = block_tokens(p);
    const dim3 g((unsigned)((p.n_tokens + tokens - 1) / tokens), 2);
    auto go = [&](auto kernel) { kernel<<<g, kThreads, 0, st>>>(p, k, v, k_stride, v_stride, tokens); };
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) i8 ? go(k_kv_read<64, LMOE_KV_INT8>) : go(k_kv_read<64, LMOE_KV_E4M3>);
    else if (p.D == 128) i8 ? go(k_kv_read<128, LMOE_KV_INT8>) : go(k_kv_read<128, LMOE_KV_E4M3>);
    else i8 ? go(k_kv_read<256, LMOE_KV_INT8>) : go(k_kv_read<256, LMOE_KV_E4M3>);
    return cudaGetLastError();
}

}  // namespace lmoe
