// The gated delta rule: S <- a S + b k (v - a k^T S), out = scale S^T q, per
// head, with the state S [head_k][head_v] in fp32.
//
// k_delta_step is the recurrence.  A warp owns 8 columns of a head's state
// in registers (a lane: 2 columns of DK / 8 rows), so a token is two dot
// products and one rank-one update in a warp, with shuffles among the lanes
// that share columns and no exchange between warps.  For a few tokens the
// state's bytes, read and written once, bound it.

#include "lmoe_mixers.cuh"

namespace lmoe {

namespace {

constexpr int kStepWarps = 8;
constexpr int kStepTokens = 8;     // tokens staged at a time

struct DeltaRows {
    int q0, n, src, dst;           // n < 0: the sequence is left out
};

__device__ __forceinline__ DeltaRows delta_rows(const DeltaParams& p, int s) {
    DeltaRows r;
    r.q0 = __ldg(p.q_start + s);
    const int q1 = __ldg(p.q_start + s + 1);
    r.src = __ldg(p.src + s);
    r.dst = __ldg(p.dst + s);
    r.n = q1 - r.q0;
    if (r.q0 < 0 || q1 < r.q0 || q1 > p.n_tokens || r.n > p.max_new || r.src < -1 || r.src >= p.n_states ||
        r.dst < -1 || r.dst >= p.n_states) {
        set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
        r.n = -1;
    }
    return r;
}

// A CTA: 64 columns of a head's state.
template <int DK>
__global__ void __launch_bounds__(kStepWarps * 32) k_delta_step(DeltaParams p) {
    constexpr int KR = DK / 8;                 // state rows of a lane
    constexpr int KS = KR + 4;                 // stride of a lane group's rows in shared memory (banks)
    __shared__ float s_k[kStepTokens][8 * KS], s_q[kStepTokens][8 * KS];
    __shared__ float s_a[kStepTokens], s_b[kStepTokens];
    const int cb = blockIdx.x % (p.DV / 64), sh = blockIdx.x / (p.DV / 64);
    const int s = sh / p.H, h = sh % p.H, hq = h / p.group;
    const DeltaRows r = delta_rows(p, s);
    if (r.n < 0) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kg = lane >> 2, c0 = cb * 64 + warp * 8 + (lane & 3) * 2;   // rows kg * KR .., columns c0, c0 + 1
    float S[KR][2];
    if (r.src >= 0) {
        const float* src = p.states + (((size_t)r.src * p.H + h) * DK + kg * KR) * p.DV + c0;
#pragma unroll
        for (int i = 0; i < KR; ++i) {
            const float2 v = *reinterpret_cast<const float2*>(src + (size_t)i * p.DV);
            S[i][0] = v.x;
            S[i][1] = v.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < KR; ++i) S[i][0] = S[i][1] = 0.f;
    }
    for (int t0 = 0; t0 < r.n; t0 += kStepTokens) {
        const int nt = min(kStepTokens, r.n - t0);
        __syncthreads();
        for (int j = warp; j < 2 * nt; j += kStepWarps) {
            const int tok = j >> 1;
            const bool isq = j & 1;
            const uint16_t* x = isq ? p.q + (size_t)(r.q0 + t0 + tok) * p.qs : p.k + (size_t)(r.q0 + t0 + tok) * p.ks;
            x += (size_t)hq * DK;
            float v[DK / 32], sum = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 64; ++i) {
                const float2 f = bf16x2_to_f32x2(__ldg(reinterpret_cast<const uint32_t*>(x) + lane * (DK / 64) + i));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
                sum = fmaf(f.x, f.x, fmaf(f.y, f.y, sum));
            }
            float f = isq ? p.scale : 1.f;
            if (p.l2norm) f *= 1.f / sqrtf(warp_sum(sum) + 1e-6f);
            float* dst = isq ? s_q[tok] : s_k[tok];
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) {
                const int d = lane * (DK / 32) + i;
                dst[(d / KR) * KS + d % KR] = v[i] * f;
            }
        }
        if (threadIdx.x < nt) {
            const size_t at = (size_t)(r.q0 + t0 + threadIdx.x) * p.H + h;
            s_a[threadIdx.x] = expf(p.log_decay[at]);
            s_b[threadIdx.x] = p.beta[at];
        }
        __syncthreads();
        for (int j = 0; j < nt; ++j) {
            const size_t row = (size_t)(r.q0 + t0 + j);
            const float2 v = bf16x2_to_f32x2(
                __ldg(reinterpret_cast<const uint32_t*>(p.v + row * p.vs + (size_t)h * p.DV + c0)));
            const float a = s_a[j], b = s_b[j];
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int i = 0; i < KR; ++i) {
                const float k = s_k[j][kg * KS + i];
                S[i][0] *= a;
                S[i][1] *= a;
                x0 = fmaf(k, S[i][0], x0);
                x1 = fmaf(k, S[i][1], x1);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                x0 += __shfl_xor_sync(0xffffffffu, x0, o);
                x1 += __shfl_xor_sync(0xffffffffu, x1, o);
            }
            const float u0 = (v.x - x0) * b, u1 = (v.y - x1) * b;
            x0 = x1 = 0.f;
#pragma unroll
            for (int i = 0; i < KR; ++i) {
                const float k = s_k[j][kg * KS + i], q = s_q[j][kg * KS + i];
                S[i][0] = fmaf(k, u0, S[i][0]);
                S[i][1] = fmaf(k, u1, S[i][1]);
                x0 = fmaf(q, S[i][0], x0);
                x1 = fmaf(q, S[i][1], x1);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                x0 += __shfl_xor_sync(0xffffffffu, x0, o);
                x1 += __shfl_xor_sync(0xffffffffu, x1, o);
            }
            if (kg == 0)
                *reinterpret_cast<uint32_t*>(p.out + (row * p.H + h) * p.DV + c0) =
                    (uint32_t)f32_to_bf16_bits(x0) | (uint32_t)f32_to_bf16_bits(x1) << 16;
        }
    }
    if (r.dst >= 0 && (r.n > 0 || r.dst != r.src)) {
        float* dst = p.states + (((size_t)r.dst * p.H + h) * DK + kg * KR) * p.DV + c0;
#pragma unroll
        for (int i = 0; i < KR; ++i)
            *reinterpret_cast<float2*>(dst + (size_t)i * p.DV) = make_float2(S[i][0], S[i][1]);
    }
}

}  // namespace

size_t delta_chunk_ws_bytes(int H, int DK, int DV, int n_tokens, int n_seqs, int max_new) { return 0; }

cudaError_t run_delta(const DeltaParams& p, cudaStream_t st) {
    const unsigned g = (unsigned)((size_t)p.n_seqs * p.H * (p.DV / 64));
    if (p.DK == 64) k_delta_step<64><<<g, kStepWarps * 32, 0, st>>>(p);
    else k_delta_step<128><<<g, kStepWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lmoe
