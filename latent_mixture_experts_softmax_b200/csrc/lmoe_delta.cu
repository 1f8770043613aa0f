// The gated delta rule: S <- a S + b k (v - a k^T S), out = scale S^T q, per
// head, with the state S [head_k][head_v] in fp32.
//
// k_delta_step is the recurrence.  A warp owns 8 columns of a head's state
// in registers (a lane: 2 columns of DK / 8 rows), so a token is two dot
// products and one rank-one update in a warp, with shuffles among the lanes
// that share columns and no exchange between warps.  For a few tokens the
// state's bytes, read and written once, bound it.
//
// The chunked form, for longer sequences: within a chunk of 32 tokens with
// log decays G_i summed from its start (D_ij = exp(G_i - G_j)), the tokens'
// updates u solve a unit lower triangular system,
//   u_i + sum_{j<i} b_i D_ij (k_i k_j) u_j = b_i (v_i - exp(G_i) k_i S),
// so with T its inverse and P_ij = scale D_ij (q_i k_j), j <= i,
//   U = T (b V - b exp(G) K S),  out = scale exp(G) Q S + P U,
//   S <- exp(G_C) S + (exp(G_C - G) K)^T U.
// k_delta_chunks makes T, P and the factors of every chunk, k_delta_scan
// walks a sequence's chunks with S.  Products run on mma.sync m16n8k16 in
// bf16 (matrices of 32 rows are too small for a tcgen05 tile): q and k are
// exact operands as they come, what is held in fp32 (S, T, P, U) enters as
// the sum of two bf16 terms, 2^-17 of its size, with fp32 sums; row norms
// and decays are applied outside the products.

#include "lmoe_mixers.cuh"
#include "lmoe_sm100.cuh"

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


// ---------------------------------------------------------------------------
// chunked form
// ---------------------------------------------------------------------------

constexpr int kC = 32;                       // tokens of a chunk

// What k_delta_chunks leaves of a chunk and head.  A fragment: 16 bytes per
// lane, an m16 x k16 operand; tiles (0, 0), (1, 0), (1, 1) of the 32 x 32.
struct ChunkData {
    uint4 t[3][2][32];                       // [tile][high, low][lane]
    uint4 p[3][2][32];
    float4 f[kC];                            // b, b exp(G) |k|^-1, scale exp(G) |q|^-1, exp(G_C - G) |k|^-1
    float4 last;                             // exp(G_C)
};

__host__ __device__ __forceinline__ int chunks_of(int n) { return (n + kC - 1) / kC; }

// Chunks of the sequences before s, and the sequence's rows; every thread of
// the block takes part.  A sequence whose chunks do not fit the workspace
// (sequences that share rows) is left out.
__device__ DeltaRows chunk_rows(const DeltaParams& p, int s, int slots, int* base) {
    __shared__ int s_sum;
    __syncthreads();
    if (threadIdx.x == 0) s_sum = 0;
    __syncthreads();
    int mine = 0;
    for (int i = threadIdx.x; i < s; i += blockDim.x) mine += chunks_of(max(0, delta_rows(p, i).n));
    mine = (int)__reduce_add_sync(0xffffffffu, (unsigned)mine);
    if ((threadIdx.x & 31) == 0) atomicAdd(&s_sum, mine);
    __syncthreads();
    *base = s_sum;
    DeltaRows r = delta_rows(p, s);
    if (r.n > 0 && ((long long)*base + chunks_of(r.n) > slots || *base < 0)) {
        set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
        r.n = -1;
    }
    return r;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(sm100::smem_u32(p)));
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], const void* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(sm100::smem_u32(p)));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two fp32 numbers as the sum of two bf16 terms each.
__device__ __forceinline__ void split2(float x, float y, uint32_t& high, uint32_t& low) {
    high = pack_bf16(x, y);
    const float2 h = bf16x2_to_f32x2(high);
    low = pack_bf16(x - h.x, y - h.y);
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows of a chunk (n_here of them, zeros behind) of one head to shared memory.
template <int DK>
__device__ __forceinline__ void load_rows(uint16_t (*dst)[DK + 8], const uint16_t* src, size_t stride, int n_here, int nt) {
    for (int i = threadIdx.x; i < kC * DK / 8; i += nt) {
        const int r = i / (DK / 8), c = i % (DK / 8) * 8;
        if (r < n_here) cp_async16(&dst[r][c], src + (size_t)r * stride + c);
        else *reinterpret_cast<uint4*>(&dst[r][c]) = make_uint4(0, 0, 0, 0);
    }
}

constexpr int kPrepThreads = 128;

// Block (chunk, head, sequence).
template <int DK>
__global__ void __launch_bounds__(kPrepThreads) k_delta_chunks(DeltaParams p, int slots) {
    __shared__ __align__(16) uint16_t sk[kC][DK + 8], sq[kC][DK + 8];
    __shared__ __align__(16) float sa[kC][kC + 4], sp[kC][kC + 4];
    __shared__ float s_rk[kC], s_rq[kC], s_b[kC], s_gh[kC], s_gl[kC];
    sm100::grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y, hq = h / p.group;
    for (int s = blockIdx.z; s < p.n_seqs; s += gridDim.z) {
        int base;
        const DeltaRows r = chunk_rows(p, s, slots, &base);
        if (r.n <= 0 || (int)blockIdx.x >= chunks_of(r.n)) continue;
        const int row0 = r.q0 + blockIdx.x * kC, n_here = min(kC, r.n - (int)blockIdx.x * kC);
        load_rows<DK>(sk, p.k + (size_t)row0 * p.ks + (size_t)hq * DK, p.ks, n_here, kPrepThreads);
        load_rows<DK>(sq, p.q + (size_t)row0 * p.qs + (size_t)hq * DK, p.qs, n_here, kPrepThreads);
        cp_async_commit();
        if (warp == 0) {
            // decays: a sum in two parts, multiples of 1/8 (exact) and the
            // rest (small), so that differences of large sums stay exact
            const size_t at = (size_t)(row0 + min(lane, n_here - 1)) * p.H + h;
            float gt = lane < n_here ? p.log_decay[at] : 0.f;
            if (gt < -128.f) gt = -128.f;                        // (-infinity too: e^-128 is 0 in fp32)
            float gh = rintf(gt * 8.f) * 0.125f, gl = gt - gh;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float yh = __shfl_up_sync(0xffffffffu, gh, o), yl = __shfl_up_sync(0xffffffffu, gl, o);
                if (lane >= o) { gh += yh; gl += yl; }
            }
            s_gh[lane] = gh;
            s_gl[lane] = gl;
            s_b[lane] = lane < n_here ? p.beta[at] : 0.f;
        }
        cp_async_wait<0>();
        __syncthreads();
        // norms: four threads a row
        {
            const int row = threadIdx.x >> 2;
            float nk = 0.f, nq = 0.f;
#pragma unroll
            for (int i = 0; i < DK / 8; ++i) {
                const float2 a = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sk[row][2 * (t + 4 * i)]));
                const float2 b = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sq[row][2 * (t + 4 * i)]));
                nk = fmaf(a.x, a.x, fmaf(a.y, a.y, nk));
                nq = fmaf(b.x, b.x, fmaf(b.y, b.y, nq));
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                nk += __shfl_xor_sync(0xffffffffu, nk, o);
                nq += __shfl_xor_sync(0xffffffffu, nq, o);
            }
            if (t == 0) {
                s_rk[row] = p.l2norm ? 1.f / sqrtf(nk + 1e-6f) : 1.f;
                s_rq[row] = p.scale * (p.l2norm ? 1.f / sqrtf(nq + 1e-6f) : 1.f);
            }
        }
        __syncthreads();
        // K K^T (warps 0, 1) and Q K^T (2, 3), 16 rows a warp
        {
            const int m = warp & 1;
            const bool isq = warp >> 1;
            const uint16_t(*a_rows)[DK + 8] = isq ? sq : sk;
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t a[4], b[2][4];
                ldm4(a, &a_rows[16 * m + (lane & 15)][16 * k + (lane >> 4) * 8]);
                // rows of K are columns of the product: n16 x k16 of two n-tiles
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ldm4(b[j], &sk[16 * j + (lane & 7) + (lane >> 4) * 8][16 * k + ((lane >> 3) & 1) * 8]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_bf16(acc[j], a, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * m + g + 8 * (i >> 1), col = 8 * j + 2 * t + (i & 1);
                    const float d = expf((s_gh[row] - s_gh[col]) + (s_gl[row] - s_gl[col]));
                    if (isq) sp[row][col] = col <= row ? acc[j][i] * d * s_rq[row] * s_rk[col] : 0.f;
                    else sa[row][col] = col < row ? acc[j][i] * d * s_b[row] * s_rk[row] * s_rk[col] : 0.f;
                }
        }
        __syncthreads();
        ChunkData* out = reinterpret_cast<ChunkData*>(p.chunk_ws) + ((size_t)(base + blockIdx.x) * p.H + h);
        auto put = [&](uint4 (*dst)[2][32], const float (*m)[kC + 4], int tile) {
            const int r0 = tile ? 16 : 0, c0 = tile == 2 ? 16 : 0;
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = *reinterpret_cast<const float2*>(&m[r0 + g + 8 * (i & 1)][c0 + 2 * t + 8 * (i >> 1)]);
                split2(x.x, x.y, hi[i], lo[i]);
            }
            dst[tile][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            dst[tile][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        };
        if (warp == 0) {
            // column `lane` of the inverse, from the top
            float x[kC];
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                float y[4] = {i == lane ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < i; j += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(&sa[i][j]);      // (zeros from column i on)
                    y[0] = fmaf(-a.x, x[j], y[0]);
                    if (j + 1 < i) y[1] = fmaf(-a.y, x[j + 1], y[1]);
                    if (j + 2 < i) y[2] = fmaf(-a.z, x[j + 2], y[2]);
                    if (j + 3 < i) y[3] = fmaf(-a.w, x[j + 3], y[3]);
                }
                x[i] = (y[0] + y[1]) + (y[2] + y[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kC; ++i) sa[i][lane] = x[i];
            __syncwarp();
            for (int i = 0; i < 3; ++i) put(out->t, sa, i);
        } else {
            put(out->p, sp, warp - 1);
            if (warp == 1) {
                const float e = expf(s_gh[lane] + s_gl[lane]), b = s_b[lane];
                const float w = expf((s_gh[kC - 1] - s_gh[lane]) + (s_gl[kC - 1] - s_gl[lane]));
                out->f[lane] = make_float4(b, b * e * s_rk[lane], e * s_rq[lane], w * s_rk[lane]);
                if (lane == kC - 1) out->last = make_float4(e, 0.f, 0.f, 0.f);
            }
        }
    }
}

constexpr int kScanThreads = 256;
constexpr int kN = 32;                       // state columns of a block

template <int DK>
struct Scan {
    uint16_t k[2][kC][DK + 8], q[2][kC][DK + 8];
    uint16_t s[2][DK][kN + 8];               // the state, high and low terms
    uint16_t r[2][kC][kN + 8];               // right-hand sides
    uint16_t u[2][kC][kN + 8];
    uint16_t w[2][kC][kN + 8];               // exp(G_C - G) |k|^-1 U
};

// Block: kN columns of a head's state.  A warp has a 16 x 8 tile of the
// chunk's rows (K S and Q S, then U, then out) and 16 rows of the state (or,
// for head_k 64, half the columns of 16 rows), in fp32 registers from the
// first chunk to the last.
template <int DK>
__global__ void __launch_bounds__(kScanThreads, 2) k_delta_scan(DeltaParams p, int slots) {
    extern __shared__ __align__(16) char smem[];
    Scan<DK>& sm = *reinterpret_cast<Scan<DK>*>(smem);
    constexpr int MT = DK / 16, NP = 8 / MT, NT = kN / 8 / NP;       // state: row tiles, column parts, 8-column tiles of a part
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = p.DV / kN;
    const int cb = blockIdx.x % nb, sh = blockIdx.x / nb, s = sh / p.H, h = sh % p.H, hq = h / p.group;
    int base;
    const DeltaRows r = chunk_rows(p, s, slots, &base);
    if (r.n < 0) return;
    const int m = warp & 1, nt = warp >> 1;                          // tile of the chunk's rows
    const int sm_row = (warp % MT) * 16, sn = (warp / MT) * NT;      // state rows, first 8-column tile
    const int n_chunks = chunks_of(r.n);
    const size_t state_at = ((size_t)h * DK + sm_row) * p.DV + cb * kN;
    float S[NT][4];
    {
        const float* src = r.src >= 0 ? p.states + (size_t)r.src * p.H * DK * p.DV + state_at : nullptr;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 x = src ? *reinterpret_cast<const float2*>(src + (size_t)(g + 8 * i) * p.DV + (sn + j) * 8 + 2 * t)
                                     : make_float2(0.f, 0.f);
                S[j][2 * i] = x.x;
                S[j][2 * i + 1] = x.y;
            }
    }
    auto store_state = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t hi, lo;
                split2(S[j][2 * i], S[j][2 * i + 1], hi, lo);
                *reinterpret_cast<uint32_t*>(&sm.s[0][sm_row + g + 8 * i][(sn + j) * 8 + 2 * t]) = hi;
                *reinterpret_cast<uint32_t*>(&sm.s[1][sm_row + g + 8 * i][(sn + j) * 8 + 2 * t]) = lo;
            }
    };
    sm100::grid_dep_wait();                  // the chunks' data is written
    const ChunkData* data = reinterpret_cast<const ChunkData*>(p.chunk_ws) + ((size_t)base * p.H + h);
    auto load_chunk = [&](int c, int b) {
        const int row0 = r.q0 + c * kC, n_here = min(kC, r.n - c * kC);
        load_rows<DK>(sm.k[b], p.k + (size_t)row0 * p.ks + (size_t)hq * DK, p.ks, n_here, kScanThreads);
        load_rows<DK>(sm.q[b], p.q + (size_t)row0 * p.qs + (size_t)hq * DK, p.qs, n_here, kScanThreads);
        cp_async_commit();
    };
    // a thread's values of a chunk, read a chunk ahead: factors and v of rows
    // g and g + 8 of its tile, fragments of T and P
    struct Ahead {
        float4 f[2];
        uint32_t v[2];
        uint4 t[2][2], p[2][2];
        float last;
    };
    const size_t vcol = (size_t)h * p.DV + cb * kN + nt * 8 + 2 * t;
    auto fetch = [&](Ahead& a, int c) {
        const ChunkData* d = data + (size_t)c * p.H;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = 16 * m + g + 8 * i;
            a.f[i] = __ldg(&d->f[row]);
            // (past the last token: its row, weighed with b = 0)
            a.v[i] = __ldg(reinterpret_cast<const uint32_t*>(p.v + (size_t)(r.q0 + min(c * kC + row, r.n - 1)) * p.vs + vcol));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)          // (m = 0 has one tile; it reads it twice and uses it once)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                a.t[k][o] = __ldg(&d->t[m ? 1 + k : 0][o][lane]);
                a.p[k][o] = __ldg(&d->p[m ? 1 + k : 0][o][lane]);
            }
        a.last = __ldg(&d->last.x);
    };
    // c += M B with M from fragments (high and low), B from two terms in shared memory
    auto tri = [&](float (&acc)[4], const uint4 (&f)[2][2], const uint16_t (*b)[kC][kN + 8]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k > m) continue;
            uint32_t x[4];                   // k16 x n8: high 0-7, 8-15, low 0-7, 8-15
            ldm4t(x, &b[lane >> 4][16 * k + (lane & 15)][nt * 8]);
            const uint32_t hi[4] = {f[k][0].x, f[k][0].y, f[k][0].z, f[k][0].w};
            const uint32_t lo[4] = {f[k][1].x, f[k][1].y, f[k][1].z, f[k][1].w};
            mma_bf16(acc, hi, x[0], x[1]);
            mma_bf16(acc, hi, x[2], x[3]);
            mma_bf16(acc, lo, x[0], x[1]);
        }
    };
    Ahead cur;
    if (n_chunks) {
        load_chunk(0, 0);
        fetch(cur, 0);
        store_state();
    }
    for (int c = 0; c < n_chunks; ++c) {
        const int b = c & 1;
        cp_async_wait<0>();
        __syncthreads();                     // the state and this chunk's rows are there; the other buffer is free
        Ahead next;
        const int cn = min(c + 1, n_chunks - 1);
        if (c + 1 < n_chunks) load_chunk(c + 1, b ^ 1);
        fetch(next, cn);
        // ---- K S, Q S
        float ks[2][4], qs[2][4];            // high, low term of S
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[o][i] = qs[o][i] = 0.f;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            uint32_t a[4], aq[4], x[4];
            ldm4(a, &sm.k[b][16 * m + (lane & 15)][16 * k + (lane >> 4) * 8]);
            ldm4(aq, &sm.q[b][16 * m + (lane & 15)][16 * k + (lane >> 4) * 8]);
            ldm4t(x, &sm.s[lane >> 4][16 * k + (lane & 15)][nt * 8]);
            mma_bf16(ks[0], a, x[0], x[1]);
            mma_bf16(qs[0], aq, x[0], x[1]);
            mma_bf16(ks[1], a, x[2], x[3]);
            mma_bf16(qs[1], aq, x[2], x[3]);
        }
        // ---- right-hand sides
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 v = bf16x2_to_f32x2(cur.v[i]);
            uint32_t hi, lo;
            split2(fmaf(-cur.f[i].y, ks[0][2 * i] + ks[1][2 * i], cur.f[i].x * v.x),
                   fmaf(-cur.f[i].y, ks[0][2 * i + 1] + ks[1][2 * i + 1], cur.f[i].x * v.y), hi, lo);
            *reinterpret_cast<uint32_t*>(&sm.r[0][16 * m + g + 8 * i][nt * 8 + 2 * t]) = hi;
            *reinterpret_cast<uint32_t*>(&sm.r[1][16 * m + g + 8 * i][nt * 8 + 2 * t]) = lo;
        }
        __syncthreads();
        // ---- U
        float u[4] = {0.f, 0.f, 0.f, 0.f};
        tri(u, cur.t, sm.r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t hi, lo;
            split2(u[2 * i], u[2 * i + 1], hi, lo);
            *reinterpret_cast<uint32_t*>(&sm.u[0][16 * m + g + 8 * i][nt * 8 + 2 * t]) = hi;
            *reinterpret_cast<uint32_t*>(&sm.u[1][16 * m + g + 8 * i][nt * 8 + 2 * t]) = lo;
            split2(cur.f[i].w * u[2 * i], cur.f[i].w * u[2 * i + 1], hi, lo);
            *reinterpret_cast<uint32_t*>(&sm.w[0][16 * m + g + 8 * i][nt * 8 + 2 * t]) = hi;
            *reinterpret_cast<uint32_t*>(&sm.w[1][16 * m + g + 8 * i][nt * 8 + 2 * t]) = lo;
        }
        __syncthreads();
        // ---- the state, and to shared memory for the next chunk
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][i] *= cur.last;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t a[4];                   // K^T: 16 state rows x 16 tokens
            ldm4t(a, &sm.k[b][16 * k + (lane & 7) + (lane >> 4) * 8][sm_row + ((lane >> 3) & 1) * 8]);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                uint32_t x[4];
                ldm4t(x, &sm.w[lane >> 4][16 * k + (lane & 15)][(sn + j) * 8]);
                mma_bf16(S[j], a, x[0], x[1]);
                mma_bf16(S[j], a, x[2], x[3]);
            }
        }
        store_state();
        // ---- out
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = cur.f[i >> 1].z * (qs[0][i] + qs[1][i]);
        tri(o, cur.p, sm.u);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = c * kC + 16 * m + g + 8 * i;
            if (row < r.n)
                *reinterpret_cast<uint32_t*>(p.out + (size_t)(r.q0 + row) * p.H * p.DV + vcol) = pack_bf16(o[2 * i], o[2 * i + 1]);
        }
        cur = next;
    }
    if (r.dst >= 0 && (r.n > 0 || r.dst != r.src)) {
        float* dst = p.states + (size_t)r.dst * p.H * DK * p.DV + state_at;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<float2*>(dst + (size_t)(g + 8 * i) * p.DV + (sn + j) * 8 + 2 * t) =
                    make_float2(S[j][2 * i], S[j][2 * i + 1]);
    }
}

// More new tokens than this per sequence run the chunked form.
constexpr int kStepTokensMax = 16;

int chunk_slots(int n_tokens, int n_seqs) {
    const long long n = (long long)n_tokens / kC + n_seqs;
    return n > 0x7fffffff ? 0x7fffffff : (int)n;
}

template <int DK>
cudaError_t run_chunks(const DeltaParams& p, cudaStream_t st) {
    const int slots = chunk_slots(p.n_tokens, p.n_seqs);
    const int z = p.n_seqs < 65535 ? p.n_seqs : 65535;
    k_delta_chunks<DK><<<dim3(chunks_of(p.max_new), p.H, z), kPrepThreads, 0, st>>>(p, slots);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = allow_smem<k_delta_scan<DK>>(sizeof(Scan<DK>));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((size_t)p.n_seqs * p.H * (p.DV / kN)));
    cfg.blockDim = dim3(kScanThreads);
    cfg.dynamicSmemBytes = sizeof(Scan<DK>);
    cfg.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_delta_scan<DK>, p, slots);
}

}  // namespace

size_t delta_chunk_ws_bytes(int H, int n_tokens, int n_seqs, int max_new) {
    return max_new <= kStepTokensMax ? 0 : sizeof(ChunkData) * (size_t)chunk_slots(n_tokens, n_seqs) * H;
}

cudaError_t run_delta(const DeltaParams& p, cudaStream_t st) {
    if (p.max_new > kStepTokensMax) return p.DK == 64 ? run_chunks<64>(p, st) : run_chunks<128>(p, st);
    const unsigned g = (unsigned)((size_t)p.n_seqs * p.H * (p.DV / 64));
    if (p.DK == 64) k_delta_step<64><<<g, kStepWarps * 32, 0, st>>>(p);
    else k_delta_step<128><<<g, kStepWarps * 32, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lmoe
