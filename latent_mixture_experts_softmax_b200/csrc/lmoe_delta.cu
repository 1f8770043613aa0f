// The gated delta rule: S <- a S + b k (v - a k^T S), out = scale S^T q, per
// head, with the state S [head_k][head_v] in fp32.
//
// All of it in the chunked form: within a chunk of C tokens with log decays
// G_i summed from its start (D_ij = exp(G_i - G_j)), the tokens' updates u
// solve a unit lower triangular system,
//   u_i + sum_{j<i} b_i D_ij (k_i k_j) u_j = b_i (v_i - exp(G_i) k_i S),
// so with T its inverse and P_ij = scale D_ij (q_i k_j), j <= i,
//   U = T (b V - b exp(G) K S),  out = scale exp(G) Q S + P U,
//   S <- exp(G_C) S + (exp(G_C - G) K)^T U.
// Products run on mma.sync m16n8k16 in bf16 (matrices of 16 and 32 rows are
// too small for a tcgen05 tile): q and k are exact operands as they come.
// What is held in fp32 and goes into the state (S in K S, T, the right-hand
// sides, U) enters as the sum of three bf16 terms, all 24 bits (of three terms
// by three, the products below 2^-24 are left out); what only goes into the
// outputs, which are bf16, as two (2^-16 of its size).  Sums
// are fp32, and the tensor cores, which truncate where they add, never add to
// the state itself: S exp(G_C) + delta is one rounded fma an element.  (With
// two terms throughout, the state was 2.6e-6 of its size off after prompts of
// 4096 tokens; so it is 1.3e-7, as with the recurrence in fp32.)  Row norms
// and decays are applied outside the products.  The state is held transposed:
// with S^T as the first operand a result's registers are the next product's
// operand as they are.
//
// A number that is not finite must not reach the tokens before it: the zeros
// above T's and P's diagonals are factors of the products like any other.  So
// where an update U is not finite, k_delta_scan makes the outputs anew from
// right-hand sides and updates that are cut off at the first token that is not,
// a column at a time (the column's state is lost as it should be);
// k_delta_short falls back on the recurrence.
//
// k_delta_short takes a few tokens (one chunk of up to 16) in one launch,
// bound by the state's bytes, read and written once.  (The plain recurrence,
// two dot products and a rank-one update a token in fp32, spends 16
// instructions an element of the state on four tokens where this spends 5,
// and took 28 us for four tokens of 16 sequences and 32 heads, 67 MB of
// states; this takes 25.)
// For longer sequences k_delta_chunks makes T, P and the factors of every
// chunk of 32, and k_delta_scan walks a sequence's chunks with S: 267 us for
// one prompt of 4096 tokens, 32 heads of 128 x 128.

#include "lmoe_mixers.cuh"
#include "lmoe_sm100.cuh"

namespace lmoe {

namespace {

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

constexpr int kC = 32;                       // tokens of a chunk

// What k_delta_chunks leaves of a chunk and head.  T and P as the second
// operand of a product: tile (k, j), 16 x 8, holds rows 8 j .. of the matrix at
// columns 16 k .. (tiles that are not zero: 0..3 = (0, j), 4, 5 = (1, 2), (1, 3)),
// 16 bytes a lane: the two registers of the high terms, then of the next; of T
// the lowest terms too.
struct ChunkData {
    uint4 t[6][32], p[6][32];
    uint2 tl[6][32];
    float b[kC], kf[kC], qf[kC], wf[kC];     // b, b exp(G) |k|^-1, scale exp(G) |q|^-1, exp(G_C - G) |k|^-1
    float last[4];                           // exp(G_C)
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
    asm(
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
// As the sum of three: every bit.
__device__ __forceinline__ void split3(float x, float y, uint32_t& high, uint32_t& mid, uint32_t& low) {
    high = pack_bf16(x, y);
    const float2 h = bf16x2_to_f32x2(high);
    split2(x - h.x, y - h.y, mid, low);
}
__device__ __forceinline__ void split_a(const float (&x)[4], const float (&y)[4], uint32_t (&a)[3][4]) {
    split3(x[0], x[1], a[0][0], a[1][0], a[2][0]);
    split3(x[2], x[3], a[0][1], a[1][1], a[2][1]);
    split3(y[0], y[1], a[0][2], a[1][2], a[2][2]);
    split3(y[2], y[3], a[0][3], a[1][3], a[2][3]);
}
// The two terms of 16 rows x 16 columns of results as a first operand.
__device__ __forceinline__ void split_a(const float (&x)[4], const float (&y)[4], uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(x[0], x[1], hi[0], lo[0]);
    split2(x[2], x[3], hi[1], lo[1]);
    split2(y[0], y[1], hi[2], lo[2]);
    split2(y[2], y[3], hi[3], lo[3]);
}
// acc += A B from three terms each: the six products that count, small first.
__device__ __forceinline__ void mul3(float (&acc)[4], const uint32_t (&a)[3][4], const uint4& b, const uint2& bl) {
    mma_bf16(acc, a[2], b.x, b.y);
    mma_bf16(acc, a[1], b.z, b.w);
    mma_bf16(acc, a[0], bl.x, bl.y);
    mma_bf16(acc, a[1], b.x, b.y);
    mma_bf16(acc, a[0], b.z, b.w);
    mma_bf16(acc, a[0], b.x, b.y);
}
// A lane's results of J tiles of 8 tokens: tokens 8 j + 2 t + (i & 1) of the
// columns i >> 1.
template <int J>
__device__ __forceinline__ bool not_finite(const float (&x)[J][4]) {
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = fmaf(x[j][i], 0.f, z[i]);
    return (z[0] + z[1]) + (z[2] + z[3]) != 0.f;
}
// The first token of each column that is not finite (or rounds to a bf16 that
// is not), where it comes before at[].
template <int J>
__device__ __forceinline__ int2 first_bad(const float (&x)[J][4], int t, int2 at) {
    int f[2] = {at.x, at.y};
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(fabsf(x[j][i]) < 0x1.ffp127f)) f[i >> 1] = min(f[i >> 1], 8 * j + 2 * t + (i & 1));
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) f[c] = min(f[c], __shfl_xor_sync(0xffffffffu, f[c], o));
    return make_int2(f[0], f[1]);
}
// `with` from token at[] on.
template <int J>
__device__ __forceinline__ void cut_off(float (&x)[J][4], int t, int2 at, float with) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * j + 2 * t + (i & 1) >= (i < 2 ? at.x : at.y)) x[j][i] = with;
}

// An 8 x 8 matrix of 16-bit numbers, two a lane, transposed: pairs of tokens
// of a column become pairs of columns of a token.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}
// 16 bytes, or as many zeros, which arrive like a copy.
__device__ __forceinline__ void cp_async16_or_zeros(void* dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// W elements of each of ROWS rows (n_here there, zeros behind) to shared memory.
template <int W, int STRIDE, int ROWS = kC>
__device__ __forceinline__ void load_rows(uint16_t* dst, const uint16_t* src, size_t stride, int n_here, int nt) {
#pragma unroll
    for (int i0 = 0; i0 < ROWS * W / 8; i0 += nt) {
        const int i = i0 + threadIdx.x;
        if (ROWS * W / 8 % nt && i >= ROWS * W / 8) break;
        const int r = i / (W / 8), c = i % (W / 8) * 8;
        if (r < n_here) cp_async16(dst + r * STRIDE + c, src + (size_t)r * stride + c);
        else *reinterpret_cast<uint4*>(dst + r * STRIDE + c) = make_uint4(0, 0, 0, 0);
    }
}

// The same by one warp: a lane has a column of pieces.  The zeros are copies
// too: the arrival on the stage's barrier covers a lane's copies, not what it
// stores itself.
template <int W, int STRIDE>
__device__ __forceinline__ void rows_async(uint16_t* dst, const uint16_t* src, size_t stride, int n_here, int lane) {
    constexpr int PC = W / 8, RP = 32 / PC;      // pieces of a row, rows of a pass
    const int row = lane / PC, c = lane % PC * 8;
    dst += row * STRIDE + c;
    const uint16_t* first = src;
    src += row * stride + c;
    if (n_here == kC) {
#pragma unroll
        for (int i = 0; i < kC / RP; ++i) cp_async16(dst + i * RP * STRIDE, src + i * RP * stride);
    } else {
        for (int i = 0; i < kC / RP; ++i) {
            const bool some = row + i * RP < n_here;
            cp_async16_or_zeros(dst + i * RP * STRIDE, some ? src + i * RP * stride : first, some);
        }
    }
}

constexpr int kPrepThreads = 128;

// e^x for x <= 0.  The product is rounded by |x| 2^-24, which moves e^x by less
// than 2^-25 in all.
__device__ __forceinline__ float exp_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Block (chunk, head of q and k, sequence).  K K^T and Q K^T once, then two of
// the heads that share them at a time, two warps each: one for T, one for P
// and the factors.
template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 6) k_delta_chunks(DeltaParams p, int slots) {
    __shared__ __align__(16) uint16_t sk[kC][DK + 8], sq[kC][DK + 8];
    __shared__ __align__(16) float kk[kC][kC + 4], qk[kC][kC + 4], sa[2][kC][kC + 4];
    __shared__ float s_rk[kC], s_rq[kC], s_gh[4][kC], s_gl[4][kC];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int hq = blockIdx.y;
    for (int s = blockIdx.z; s < p.n_seqs; s += gridDim.z) {
        int base;
        const DeltaRows r = chunk_rows(p, s, slots, &base);
        if (r.n <= 0 || (int)blockIdx.x >= chunks_of(r.n)) continue;
        const int row0 = r.q0 + blockIdx.x * kC, n_here = min(kC, r.n - (int)blockIdx.x * kC);
        load_rows<DK, DK + 8>(&sk[0][0], p.k + (size_t)row0 * p.ks + (size_t)hq * DK, p.ks, n_here, kPrepThreads);
        load_rows<DK, DK + 8>(&sq[0][0], p.q + (size_t)row0 * p.qs + (size_t)hq * DK, p.qs, n_here, kPrepThreads);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        // norms of q, four threads a row (those of k are the diagonal of K K^T)
        {
            const int row = threadIdx.x >> 2;
            float nq = 0.f;
            if (p.l2norm) {
#pragma unroll
                for (int i = 0; i < DK / 8; ++i) {
                    const float2 b = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sq[row][2 * (t + 4 * i)]));
                    nq = fmaf(b.x, b.x, fmaf(b.y, b.y, nq));
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) nq += __shfl_xor_sync(0xffffffffu, nq, o);
            }
            if (t == 0) s_rq[row] = p.scale * (p.l2norm ? 1.f / sqrtf(nq + 1e-6f) : 1.f);
        }
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
                // rows of K are columns of the product: two n-tiles
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ldm4(b[j], &sk[16 * j + (lane & 7) + (lane >> 4) * 8][16 * k + ((lane >> 3) & 1) * 8]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_bf16(acc[j], a, b[j >> 1][2 * (j & 1)], b[j >> 1][2 * (j & 1) + 1]);
            }
            float(*dst)[kC + 4] = isq ? qk : kk;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2*>(&dst[16 * m + g + 8 * i][8 * j + 2 * t]) = make_float2(acc[j][2 * i], acc[j][2 * i + 1]);
        }
        __syncthreads();
        const float rk = p.l2norm ? 1.f / sqrtf(kk[lane][lane] + 1e-6f) : 1.f;
        if (warp == 0) s_rk[lane] = rk;
        __syncthreads();
        for (int hh = warp >> 1; hh < p.group; hh += 2) {
            const int h = hq * p.group + hh;
            ChunkData* out = reinterpret_cast<ChunkData*>(p.chunk_ws) + ((size_t)(base + blockIdx.x) * p.H + h);
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
            const float b = lane < n_here ? p.beta[at] : 0.f;
            float* xh = s_gh[warp];
            float* xl = s_gl[warp];
            __syncwarp();
            xh[lane] = gh;
            xl[lane] = gl;
            __syncwarp();
            if (!(warp & 1)) {
                // the first token with a number that is not finite: its row of A T11
                // below would meet the zeros of earlier rows of T22
                bool bad = !(fabsf(b) < INFINITY) || !(gt < INFINITY);
                if (!(kk[lane][lane] < INFINITY))
                    for (int i = 0; i < DK; ++i) bad |= (sk[lane][i] & 0x7fffu) >= 0x7f80u;
                const unsigned bads = __ballot_sync(0xffffffffu, bad);
                const int first = bads ? __ffs(bads) - 1 : kC;
                float(*m)[kC + 4] = sa[warp >> 1];
                const float br = b * rk;
#pragma unroll 8
                for (int i = 0; i < kC; ++i) {                   // column `lane` of b_i D_ij (k_i k_j)
                    const float d = exp_of((xh[i] - gh) + (xl[i] - gl));
                    const float bi = __shfl_sync(0xffffffffu, br, i);
                    const float y = kk[i][lane] * (bi * rk) * d;     // (every lane: a branch here waits for its load)
                    m[i][lane] = lane < i ? y : 0.f;
                }
                __syncwarp();
                // the inverse by blocks of 16: T11 and T22 a column a lane,
                // from the top, then T21 = -T22 A21 T11
                {
                    const int o = lane & 16, cj = lane & 15;
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float y[4] = {i == cj ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < i; j += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(&m[o + i][o + j]);   // (zeros from column i on)
                            y[0] = fmaf(-a.x, x[j], y[0]);
                            if (j + 1 < i) y[1] = fmaf(-a.y, x[j + 1], y[1]);
                            if (j + 2 < i) y[2] = fmaf(-a.z, x[j + 2], y[2]);
                            if (j + 3 < i) y[3] = fmaf(-a.w, x[j + 3], y[3]);
                        }
                        x[i] = (y[0] + y[1]) + (y[2] + y[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) m[o + i][lane] = x[i];
                    __syncwarp();
                    // (A21 T11 stands in the upper right block, which no tile holds)
                    const int rb = o >> 1;
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = m[i][cj];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(&m[16 + rb + i][j]);
                            y[0] = fmaf(a.x, x[j], y[0]);
                            y[1] = fmaf(a.y, x[j + 1], y[1]);
                            y[2] = fmaf(a.z, x[j + 2], y[2]);
                            y[3] = fmaf(a.w, x[j + 3], y[3]);
                        }
                        m[rb + i][16 + cj] = 16 + rb + i < first ? (y[0] + y[1]) + (y[2] + y[3]) : 0.f;
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = m[i][16 + cj];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(&m[16 + rb + i][16 + j]);
                            y[0] = fmaf(-a.x, x[j], y[0]);
                            y[1] = fmaf(-a.y, x[j + 1], y[1]);
                            y[2] = fmaf(-a.z, x[j + 2], y[2]);
                            y[3] = fmaf(-a.w, x[j + 3], y[3]);
                        }
                        m[16 + rb + i][cj] = (y[0] + y[1]) + (y[2] + y[3]);
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int tile = 0; tile < 6; ++tile) {
                    const int k = tile >> 2, j = tile < 4 ? tile : tile - 2;
                    const float2 u0 = *reinterpret_cast<const float2*>(&m[8 * j + g][16 * k + 2 * t]);
                    const float2 u1 = *reinterpret_cast<const float2*>(&m[8 * j + g][16 * k + 2 * t + 8]);
                    uint4 w;
                    uint2 l;
                    split3(u0.x, u0.y, w.x, w.z, l.x);
                    split3(u1.x, u1.y, w.y, w.w, l.y);
                    out->t[tile][lane] = w;
                    out->tl[tile][lane] = l;
                }
            } else {
                const float e = exp_of(gh + gl);
                const float w = exp_of((xh[kC - 1] - gh) + (xl[kC - 1] - gl));
                out->b[lane] = b;
                out->kf[lane] = b * e * rk;
                out->qf[lane] = e * s_rq[lane];
                out->wf[lane] = w * rk;
                if (lane == kC - 1) *reinterpret_cast<float4*>(out->last) = make_float4(e, 0.f, 0.f, 0.f);
#pragma unroll
                for (int tile = 0; tile < 6; ++tile) {
                    const int k = tile >> 2, j = tile < 4 ? tile : tile - 2, i = 8 * j + g;
                    float u[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int col = 16 * k + 2 * t + (c & 1) + 8 * (c >> 1);
                        const float d = exp_of((xh[i] - xh[col]) + (xl[i] - xl[col]));
                        const float y = qk[i][col] * (s_rq[i] * s_rk[col]) * d;
                        u[c] = col <= i ? y : 0.f;
                    }
                    uint4 x;
                    split2(u[0], u[1], x.x, x.z);
                    split2(u[2], u[3], x.y, x.w);
                    out->p[tile][lane] = x;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// a few tokens
// ---------------------------------------------------------------------------

constexpr int kFew = 16;                     // tokens, at most
constexpr int kShortThreads = 128;
constexpr int kShortN = 64;                  // state columns of a block, 16 a warp

// Block: 64 columns of a head's state.  Its loads are issued first and arrive
// while the chunk's matrices are made.
template <int DK>
__global__ void __launch_bounds__(kShortThreads, 4) k_delta_short(DeltaParams p) {
    constexpr int NT = DK / 8;
    __shared__ __align__(16) uint16_t sk[kFew][DK + 8], sq[kFew][DK + 8], sv[kFew][kShortN + 8];
    __shared__ __align__(16) float kk[kFew][kFew + 4], qk[kFew][kFew + 4], sa[kFew][kFew + 4];
    __shared__ __align__(16) uint4 s_t[2][32], s_p[2][32];
    __shared__ uint2 s_tl[2][32];
    __shared__ __align__(16) float s_b[kFew], s_kf[kFew], s_qf[kFew], s_wf[kFew];
    __shared__ float s_rk[kFew], s_rq[kFew], s_gh[2][kFew], s_gl[2][kFew], s_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int nb = p.DV / kShortN, cb = blockIdx.x % nb, sh = blockIdx.x / nb;
    const int s = sh / p.H, h = sh % p.H, hq = h / p.group;
    const DeltaRows r = delta_rows(p, s);
    if (r.n < 0) return;
    // element (column g + 8 i, row 8 j + 2 t + e) of this warp's 16 columns
    const size_t state_at = ((size_t)h * DK + 2 * t) * p.DV + cb * kShortN + warp * 16 + g;
    float S[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][i] = 0.f;
    if (r.src >= 0) {
        const float* src = p.states + (size_t)r.src * p.H * DK * p.DV + state_at;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][i] = src[(8 * j + (i & 1)) * p.DV + 8 * (i >> 1)];
    }
    if (r.n > 0) {
        load_rows<DK, DK + 8, kFew>(&sk[0][0], p.k + (size_t)r.q0 * p.ks + (size_t)hq * DK, p.ks, r.n, kShortThreads);
        load_rows<DK, DK + 8, kFew>(&sq[0][0], p.q + (size_t)r.q0 * p.qs + (size_t)hq * DK, p.qs, r.n, kShortThreads);
        load_rows<kShortN, kShortN + 8, kFew>(&sv[0][0], p.v + (size_t)r.q0 * p.vs + (size_t)h * p.DV + cb * kShortN, p.vs, r.n,
                                              kShortThreads);
        cp_async_commit();
        // ---- decays (warps 0 and 1; a lane a token), as in k_delta_chunks
        float gh = 0.f, gl = 0.f, b = 0.f;
        if (warp < 2) {
            const size_t at = (size_t)(r.q0 + min(lane, r.n - 1)) * p.H + h;
            float gt = lane < r.n ? p.log_decay[at] : 0.f;
            b = lane < r.n ? p.beta[at] : 0.f;
            if (gt < -128.f) gt = -128.f;
            gh = rintf(gt * 8.f) * 0.125f;
            gl = gt - gh;
#pragma unroll
            for (int o = 1; o < kFew; o <<= 1) {
                const float yh = __shfl_up_sync(0xffffffffu, gh, o), yl = __shfl_up_sync(0xffffffffu, gl, o);
                if (lane >= o) { gh += yh; gl += yl; }
            }
            if (lane < kFew) {
                s_gh[warp][lane] = gh;
                s_gl[warp][lane] = gl;
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        // ---- K K^T (warp 0), Q K^T (1), norms of q (2)
        if (warp < 2) {
            const uint16_t(*a_rows)[DK + 8] = warp ? sq : sk;
            float acc[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                uint32_t a[4], y[4];
                ldm4(a, &a_rows[lane & 15][16 * k + (lane >> 4) * 8]);
                ldm4(y, &sk[(lane & 7) + (lane >> 4) * 8][16 * k + ((lane >> 3) & 1) * 8]);
                mma_bf16(acc[0], a, y[0], y[1]);
                mma_bf16(acc[1], a, y[2], y[3]);
            }
            float(*dst)[kFew + 4] = warp ? qk : kk;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2*>(&dst[g + 8 * i][8 * j + 2 * t]) = make_float2(acc[j][2 * i], acc[j][2 * i + 1]);
        } else if (warp == 2) {
            const int row = lane >> 1;
            float nq = 0.f;
#pragma unroll 8
            for (int i = 0; i < DK / 4; ++i) {
                const float2 x = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sq[row][2 * ((lane & 1) + 2 * i)]));
                nq = fmaf(x.x, x.x, fmaf(x.y, x.y, nq));
            }
            nq += __shfl_xor_sync(0xffffffffu, nq, 1);
            if (!(lane & 1)) s_rq[row] = p.scale * (p.l2norm ? 1.f / sqrtf(nq + 1e-6f) : 1.f);
        }
        __syncthreads();
        // ---- T (warp 0), P and factors (warp 1)
        if (warp < 2) {
            const float* xh = s_gh[warp];
            const float* xl = s_gl[warp];
            const int tok = lane & 15;
            gh = xh[tok];
            gl = xl[tok];
            b = __shfl_sync(0xffffffffu, b, tok);
            const float rk = p.l2norm ? 1.f / sqrtf(kk[tok][tok] + 1e-6f) : 1.f;
            if (warp == 0) {
                const float br = b * rk;
                float x[kFew];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kFew; ++i) {             // column `tok` of b_i D_ij (k_i k_j)
                    const float bi = __shfl_sync(0xffffffffu, br, i);
                    const float y = kk[i][tok] * (bi * rk) * exp_of((xh[i] - gh) + (xl[i] - gl));
                    x[i] = tok < i ? y : 0.f;
                }
                __syncwarp();
                if (lane < kFew)
#pragma unroll
                    for (int i = 0; i < kFew; ++i) sa[i][lane] = x[i];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kFew; ++i) {             // and of the inverse, from the top
                    float y[4] = {i == tok ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < i; j += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(&sa[i][j]);          // (zeros from column i on)
                        y[0] = fmaf(-a.x, x[j], y[0]);
                        if (j + 1 < i) y[1] = fmaf(-a.y, x[j + 1], y[1]);
                        if (j + 2 < i) y[2] = fmaf(-a.z, x[j + 2], y[2]);
                        if (j + 3 < i) y[3] = fmaf(-a.w, x[j + 3], y[3]);
                    }
                    x[i] = (y[0] + y[1]) + (y[2] + y[3]);
                }
                __syncwarp();
                if (lane < kFew)
#pragma unroll
                    for (int i = 0; i < kFew; ++i) sa[i][lane] = x[i];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 u0 = *reinterpret_cast<const float2*>(&sa[8 * j + g][2 * t]);
                    const float2 u1 = *reinterpret_cast<const float2*>(&sa[8 * j + g][2 * t + 8]);
                    uint4 w;
                    uint2 l;
                    split3(u0.x, u0.y, w.x, w.z, l.x);
                    split3(u1.x, u1.y, w.y, w.w, l.y);
                    s_t[j][lane] = w;
                    s_tl[j][lane] = l;
                }
            } else {
                const float e = exp_of(gh + gl), w = exp_of((xh[kFew - 1] - gh) + (xl[kFew - 1] - gl));
                if (lane < kFew) {
                    s_b[lane] = b;
                    s_kf[lane] = b * e * rk;
                    s_qf[lane] = e * s_rq[lane];
                    s_wf[lane] = w * rk;
                    s_rk[lane] = rk;
                    if (lane == kFew - 1) s_last = e;
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int i = 8 * j + g;
                    float u[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int col = 2 * t + (c & 1) + 8 * (c >> 1);
                        const float d = exp_of((xh[i] - xh[col]) + (xl[i] - xl[col]));
                        const float y = qk[i][col] * (s_rq[i] * s_rk[col]) * d;
                        u[c] = col <= i ? y : 0.f;
                    }
                    uint4 x;
                    split2(u[0], u[1], x.x, x.z);
                    split2(u[2], u[3], x.y, x.w);
                    s_p[j][lane] = x;
                }
            }
        }
        __syncthreads();
        // ---- (K S)^T, (Q S)^T: 16 columns x 16 tokens
        float ks[2][4], qs[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[j][i] = qs[j][i] = 0.f;
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            uint32_t a[3][4], bk[4], bq[4];
            split_a(S[2 * k], S[2 * k + 1], a);
            const int col = 16 * k + ((lane >> 3) & 1) * 8;
            ldm4(bk, &sk[(lane & 7) + (lane >> 4) * 8][col]);
            ldm4(bq, &sq[(lane & 7) + (lane >> 4) * 8][col]);
#pragma unroll
            for (int o = 0; o < 3; ++o)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mma_bf16(ks[j], a[o], bk[2 * j], bk[2 * j + 1]);
                    if (o < 2) mma_bf16(qs[j], a[o], bq[2 * j], bq[2 * j + 1]);
                }
        }
        // ---- right-hand sides over K S, U^T
        float u[2][4], o[2][4];
        uint32_t v[4], hi[4], lo[4];
        ldm4t(v, &sv[lane & 15][warp * 16 + (lane >> 4) * 8]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 bb = *reinterpret_cast<const float2*>(&s_b[8 * j + 2 * t]);
            const float2 f = *reinterpret_cast<const float2*>(&s_kf[8 * j + 2 * t]);
            const float2 q = *reinterpret_cast<const float2*>(&s_qf[8 * j + 2 * t]);
            const float2 v0 = bf16x2_to_f32x2(v[j]), v1 = bf16x2_to_f32x2(v[2 + j]);
            ks[j][0] = fmaf(-f.x, ks[j][0], bb.x * v0.x);
            ks[j][1] = fmaf(-f.y, ks[j][1], bb.y * v0.y);
            ks[j][2] = fmaf(-f.x, ks[j][2], bb.x * v1.x);
            ks[j][3] = fmaf(-f.y, ks[j][3], bb.y * v1.y);
            o[j][0] = q.x * qs[j][0];
            o[j][1] = q.y * qs[j][1];
            o[j][2] = q.x * qs[j][2];
            o[j][3] = q.y * qs[j][3];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[j][i] = 0.f;
        }
        uint32_t a[3][4];
        split_a(ks[0], ks[1], a);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 f = s_t[j][lane];
            const uint2 l = s_tl[j][lane];
            mul3(u[j], a, f, l);
        }
        if (__builtin_expect(__any_sync(0xffffffffu, not_finite(u)), 0)) {
            // numbers that are not finite: the recurrence itself, a token after the other
            const size_t col = (size_t)h * p.DV + cb * kShortN + warp * 16 + g + 8 * t;
            for (int i = 0; i < r.n; ++i) {
                const float decay = exp_of(i ? (s_gh[0][i] - s_gh[0][i - 1]) + (s_gl[0][i] - s_gl[0][i - 1]) : s_gh[0][0] + s_gl[0][0]);
                const float rk = s_rk[i], b = s_b[i];
                float y[2] = {0.f, 0.f};
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float2 f = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sk[i][8 * j + 2 * t]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[j][e] *= decay;
                        y[e >> 1] = fmaf(e & 1 ? f.y : f.x, S[j][e], y[e >> 1]);
                    }
                }
                float z[2] = {0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    y[c] += __shfl_xor_sync(0xffffffffu, y[c], 1);
                    y[c] += __shfl_xor_sync(0xffffffffu, y[c], 2);
                    y[c] = b * rk * (bf16_bits_to_f32(sv[i][warp * 16 + g + 8 * c]) - rk * y[c]);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const float2 f = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sk[i][8 * j + 2 * t]));
                    const float2 q = bf16x2_to_f32x2(*reinterpret_cast<const uint32_t*>(&sq[i][8 * j + 2 * t]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[j][e] = fmaf(e & 1 ? f.y : f.x, y[e >> 1], S[j][e]);
                        z[e >> 1] = fmaf(e & 1 ? q.y : q.x, S[j][e], z[e >> 1]);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    z[c] += __shfl_xor_sync(0xffffffffu, z[c], 1);
                    z[c] += __shfl_xor_sync(0xffffffffu, z[c], 2);
                }
                if (t < 2) p.out[(size_t)(r.q0 + i) * p.H * p.DV + col] = f32_to_bf16_bits((t ? z[1] : z[0]) * s_rq[i]);
            }
        } else {
            // ---- out^T
            split_a(u[0], u[1], hi, lo);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 f = s_p[j][lane];
                mma_bf16(o[j], hi, f.x, f.y);
                mma_bf16(o[j], hi, f.z, f.w);
                mma_bf16(o[j], lo, f.x, f.y);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t y = transposed(pack_bf16(o[j][2 * i], o[j][2 * i + 1]));
                    const int row = 8 * j + g;
                    if (row < r.n)
                        *reinterpret_cast<uint32_t*>(p.out + ((size_t)(r.q0 + row) * p.H + h) * p.DV + cb * kShortN + warp * 16 + 8 * i +
                                                     2 * t) = y;
                }
            // ---- the state
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 f = *reinterpret_cast<const float2*>(&s_wf[8 * j + 2 * t]);
                u[j][0] *= f.x;
                u[j][1] *= f.y;
                u[j][2] *= f.x;
                u[j][3] *= f.y;
            }
            split_a(u[0], u[1], a);
            const float last = s_last;
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
                uint32_t bk[4];
                ldm4t(bk, &sk[lane & 15][16 * j + (lane >> 4) * 8]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int o = 2; o >= 0; --o) mma_bf16(d, a[o], bk[2 * i], bk[2 * i + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) S[2 * j + i][e] = fmaf(S[2 * j + i][e], last, d[e]);
                }
            }
        }
    }
    if (r.dst >= 0 && (r.n > 0 || r.dst != r.src)) {
        float* dst = p.states + (size_t)r.dst * p.H * DK * p.DV + state_at;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[(8 * j + (i & 1)) * p.DV + 8 * (i >> 1)] = S[j][i];
    }
}

// ---------------------------------------------------------------------------
// a sequence's chunks
// ---------------------------------------------------------------------------

constexpr int kScanThreads = 160;           // four warps compute, the fifth loads
constexpr uint64_t kWaitLimit = 4000000000ull;   // SM cycles per barrier wait (about 2 s)
constexpr int kN = 32;                       // state columns of a block
constexpr int kStages = 3;

// (P U)^T of a chunk's tokens 16 hf .. 16 hf + 15 from updates that are not all
// finite: right-hand sides and updates are cut off at each column's first token
// that is not.
struct Rhs {
    float y[4][4];
};
struct Outputs {
    float o[2][4];
};
__device__ __forceinline__ void times_p(float (&o)[2][4], const float (&u)[4][4], const ChunkData& d, int hf, int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (k > hf) continue;
        uint32_t hi[4], lo[4];
        split_a(u[2 * k], u[2 * k + 1], hi, lo);
        uint4 f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) f[j] = d.p[k ? 4 + j : 2 * hf + j][lane];
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_bf16(o[j], hi, f[j].x, f[j].y);
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_bf16(o[j], hi, f[j].z, f[j].w);
#pragma unroll
        for (int j = 0; j < 2; ++j) mma_bf16(o[j], lo, f[j].x, f[j].y);
    }
}
__device__ __noinline__ Outputs outputs_cut_off(Rhs r, const ChunkData& d, int hf, int lane) {
    const int t = lane & 3;
    Outputs x;
    float u[4][4];
    int2 cut = first_bad(r.y, t, make_int2(kC, kC));
    cut_off(r.y, t, cut, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[j][i] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t a[3][4];
        split_a(r.y[2 * k], r.y[2 * k + 1], a);
#pragma unroll
        for (int j = 2 * k; j < 4; ++j) mul3(u[j], a, d.t[k ? j + 2 : j][lane], d.tl[k ? j + 2 : j][lane]);
    }
    cut = first_bad(u, t, cut);              // (rows of T from there on; sums that overflowed)
    cut_off(u, t, cut, 0.f);
    times_p(x.o, u, d, hf, lane);
    cut_off(x.o, t, make_int2(cut.x - 16 * hf, cut.y - 16 * hf), __int_as_float(0x7fffffff));
    return x;
}

template <int DK>
struct Scan {
    struct Stage {
        uint16_t k[kC][DK + 8], q[kC][DK + 8], v[kC][kN + 8];
        ChunkData d;
    } st[kStages];
    float4 part[4][6][32];                   // a warp's share of K S and Q S for its partner
    uint64_t full[kStages], empty[kStages];
    uint64_t wrote[2], read[2];              // shares of the two warps of a group
    int abort;
};

// Block: kN columns of a head's state.  Two warps hold 16 columns, half of the
// state's rows each, in fp32 registers from the first chunk to the last; they
// add up their shares of K S and Q S through shared memory, both compute U,
// and each updates its rows of S and writes half of the tokens.  The chain of
// a chunk's steps bounds it (3500 cycles, of which its 180 products take 1440;
// 4700 with two blocks on an SM), so all that is not on it is done by the
// fifth warp, which keeps two chunks ahead.
template <int DK>
__global__ void __launch_bounds__(kScanThreads, 2) k_delta_scan(DeltaParams p, int slots) {
    extern __shared__ __align__(16) char smem[];
    Scan<DK>& sm = *reinterpret_cast<Scan<DK>*>(smem);
    constexpr int KH = DK / 2, NT = KH / 8;                          // state rows of a warp, 8-row tiles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int gp = warp >> 1, hf = warp & 1;
    const int nb = p.DV / kN;
    const int cb = blockIdx.x % nb, sh = blockIdx.x / nb, s = sh / p.H, h = sh % p.H, hq = h / p.group;
    int base;
    const DeltaRows r = chunk_rows(p, s, slots, &base);
    if (r.n < 0) return;
    const int n_chunks = chunks_of(r.n);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            sm100::mbar_init(&sm.full[i], 32);
            sm100::mbar_init(&sm.empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            sm100::mbar_init(&sm.wrote[i], 2);
            sm100::mbar_init(&sm.read[i], 2);
        }
        sm.abort = 0;
        sm100::fence_barrier_init();
    }
    __syncthreads();
    volatile int* abort = &sm.abort;
    if (warp == 4) {
        const ChunkData* data = reinterpret_cast<const ChunkData*>(p.chunk_ws) + ((size_t)base * p.H + h);
        int c = 0;
        for (int st = 0, ph = 1; c < n_chunks; ++c, st = st + 1 < kStages ? st + 1 : 0, ph ^= st == 0) {
            const bool ok = sm100::mbar_wait(&sm.empty[st], ph, abort, kWaitLimit);
            if (!__all_sync(0xffffffffu, ok)) break;
            typename Scan<DK>::Stage& x = sm.st[st];
            const int n_here = min(kC, r.n - c * kC);
            const size_t row0 = (size_t)r.q0 + (size_t)c * kC;
            rows_async<DK, DK + 8>(&x.k[0][0], p.k + row0 * p.ks + (size_t)hq * DK, p.ks, n_here, lane);
            rows_async<DK, DK + 8>(&x.q[0][0], p.q + row0 * p.qs + (size_t)hq * DK, p.qs, n_here, lane);
            rows_async<kN, kN + 8>(&x.v[0][0], p.v + row0 * p.vs + (size_t)h * p.DV + cb * kN, p.vs, n_here, lane);
            const char* d = reinterpret_cast<const char*>(data + (size_t)c * p.H) + 16 * lane;
            char* xd = reinterpret_cast<char*>(&x.d) + 16 * lane;
            constexpr int kWhole = sizeof(ChunkData) / 512;
#pragma unroll
            for (int i = 0; i < kWhole; ++i) cp_async16(xd + 512 * i, d + 512 * i);
            if (lane < (int)(sizeof(ChunkData) % 512 / 16)) cp_async16(xd + 512 * kWhole, d + 512 * kWhole);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(&sm.full[st])) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        return;
    }
    // element (column g + 8 i, row 8 j + 2 t + e) of this warp's tile
    const size_t state_at = ((size_t)h * DK + hf * KH + 2 * t) * p.DV + cb * kN + gp * 16 + g;
    float S[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[j][i] = 0.f;
    if (r.src >= 0) {
        const float* src = p.states + (size_t)r.src * p.H * DK * p.DV + state_at;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) S[j][i] = src[(size_t)(8 * j + (i & 1)) * p.DV + 8 * (i >> 1)];
    }
    bool dead = false;
    for (int c = 0, st = 0, ph = 0; c < n_chunks; ++c, st = st + 1 < kStages ? st + 1 : 0, ph ^= st == 0) {
        dead = !sm100::mbar_wait(&sm.full[st], ph, abort, kWaitLimit);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        const typename Scan<DK>::Stage& x = sm.st[st];
        // ---- this warp's share of (K S)^T and (Q S)^T: 16 columns x 32 tokens
        float ks[4][4], qs[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[j][i] = qs[j][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KH / 16; ++k) {
            uint32_t a[3][4];
            split_a(S[2 * k], S[2 * k + 1], a);
            const int col = hf * KH + 16 * k + ((lane >> 3) & 1) * 8;
            uint32_t bk[2][4], bq[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ldm4(bk[j], &x.k[16 * j + (lane & 7) + (lane >> 4) * 8][col]);
                ldm4(bq[j], &x.q[16 * j + (lane & 7) + (lane >> 4) * 8][col]);
            }
            // (products that add to the same sums stand far apart here and below)
#pragma unroll
            for (int o = 0; o < 3; ++o)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma_bf16(ks[j], a[o], bk[j >> 1][2 * (j & 1)], bk[j >> 1][2 * (j & 1) + 1]);
                    if (o < 2) mma_bf16(qs[j], a[o], bq[j >> 1][2 * (j & 1)], bq[j >> 1][2 * (j & 1) + 1]);
                }
        }
        // ---- the partner's share: all of K S, and Q S of the tokens this warp writes
        dead = c > 0 && !sm100::mbar_wait(&sm.read[gp], (c - 1) & 1, abort, kWaitLimit);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.part[warp][j][lane] = make_float4(ks[j][0], ks[j][1], ks[j][2], ks[j][3]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 y = hf ? make_float4(qs[j][0], qs[j][1], qs[j][2], qs[j][3])
                                : make_float4(qs[2 + j][0], qs[2 + j][1], qs[2 + j][2], qs[2 + j][3]);
            sm.part[warp][4 + j][lane] = y;
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sm.wrote[gp]);
        // (what the next steps read, while the partner's share is on its way)
        uint32_t v[2][4];
        uint4 ft[6];
#pragma unroll
        for (int j = 0; j < 2; ++j) ldm4t(v[j], &x.v[16 * j + (lane & 15)][gp * 16 + (lane >> 4) * 8]);
#pragma unroll
        for (int j = 0; j < 6; ++j) ft[j] = x.d.t[j][lane];
        dead = !sm100::mbar_wait(&sm.wrote[gp], c & 1, abort, kWaitLimit);
        dead = __any_sync(0xffffffffu, dead);
        if (dead) break;
        float o[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 y = sm.part[warp ^ 1][j][lane];
            ks[j][0] += y.x;
            ks[j][1] += y.y;
            ks[j][2] += y.z;
            ks[j][3] += y.w;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 y = sm.part[warp ^ 1][4 + j][lane];
            const float2 f = *reinterpret_cast<const float2*>(&x.d.qf[16 * hf + 8 * j + 2 * t]);
            o[j][0] = f.x * ((hf ? qs[2 + j][0] : qs[j][0]) + y.x);
            o[j][1] = f.y * ((hf ? qs[2 + j][1] : qs[j][1]) + y.y);
            o[j][2] = f.x * ((hf ? qs[2 + j][2] : qs[j][2]) + y.z);
            o[j][3] = f.y * ((hf ? qs[2 + j][3] : qs[j][3]) + y.w);
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sm.read[gp]);
        // ---- right-hand sides, over K S
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            // v^T: columns gp * 16 + g (+ 8), tokens 16 j + 2 t .. and 8 on
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 b = *reinterpret_cast<const float2*>(&x.d.b[16 * j + 8 * i + 2 * t]);
                const float2 f = *reinterpret_cast<const float2*>(&x.d.kf[16 * j + 8 * i + 2 * t]);
                const float2 v0 = bf16x2_to_f32x2(v[j][i]), v1 = bf16x2_to_f32x2(v[j][2 + i]);
                float(&y)[4] = ks[2 * j + i];
                y[0] = fmaf(-f.x, y[0], b.x * v0.x);
                y[1] = fmaf(-f.y, y[1], b.y * v0.y);
                y[2] = fmaf(-f.x, y[2], b.x * v1.x);
                y[3] = fmaf(-f.y, y[3], b.y * v1.y);
            }
        }
        // ---- U^T
        float u[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[j][i] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t a[3][4];
            split_a(ks[2 * k], ks[2 * k + 1], a);
            const uint4* f = ft + 2 * k;
            uint2 l[4];
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) l[j] = x.d.tl[k ? j + 2 : j][lane];
            // (mul3, of up to four tiles side by side)
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[2], f[j].x, f[j].y);
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[1], f[j].z, f[j].w);
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[0], l[j].x, l[j].y);
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[1], f[j].x, f[j].y);
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[0], f[j].z, f[j].w);
#pragma unroll
            for (int j = 2 * k; j < 4; ++j) mma_bf16(u[j], a[0], f[j].x, f[j].y);
        }
        // ---- the state
        const float last = x.d.last[0];
        uint32_t w[2][3][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float y[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float2 f = *reinterpret_cast<const float2*>(&x.d.wf[16 * k + 8 * j + 2 * t]);
                y[j][0] = f.x * u[2 * k + j][0];
                y[j][1] = f.y * u[2 * k + j][1];
                y[j][2] = f.x * u[2 * k + j][2];
                y[j][3] = f.y * u[2 * k + j][3];
            }
            split_a(y[0], y[1], w[k]);
        }
#pragma unroll
        for (int j0 = 0; j0 < NT; j0 += 4) {             // 32 rows of the state at a time
            uint32_t bk[2][2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ldm4t(bk[k][j], &x.k[16 * k + (lane & 15)][hf * KH + 8 * j0 + 16 * j + (lane >> 4) * 8]);
            float d[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) d[j][i] = 0.f;
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_bf16(d[j], w[k][o], bk[k][j >> 1][2 * (j & 1)], bk[k][j >> 1][2 * (j & 1) + 1]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) S[j0 + j][i] = fmaf(S[j0 + j][i], last, d[j][i]);
        }
        // ---- out^T of 16 tokens
        float pu[2][4];
        times_p(pu, u, x.d, hf, lane);
        if (__builtin_expect(__any_sync(0xffffffffu, not_finite(u)), 0)) {
            // (the state is NaN in these columns, as it has to be; outputs before are not)
            Rhs r;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) r.y[j][i] = ks[j][i];
            const Outputs y = outputs_cut_off(r, x.d, hf, lane);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) pu[j][i] = y.o[j][i];      // (NaN from there on)
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] += pu[j][i];
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&sm.empty[st]);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t y = transposed(pack_bf16(o[j][2 * i], o[j][2 * i + 1]));
                const int row = c * kC + 16 * hf + 8 * j + g;
                if (row < r.n)
                    *reinterpret_cast<uint32_t*>(p.out + ((size_t)(r.q0 + row) * p.H + h) * p.DV + cb * kN + gp * 16 + 8 * i + 2 * t) = y;
            }
    }
    if (dead) {
        if (lane == 0) set_status(p.ctrl, LMOE_ERR_TIMEOUT);
        return;
    }
    if (r.dst >= 0 && (r.n > 0 || r.dst != r.src)) {
        float* dst = p.states + (size_t)r.dst * p.H * DK * p.DV + state_at;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[(size_t)(8 * j + (i & 1)) * p.DV + 8 * (i >> 1)] = S[j][i];
    }
}

int chunk_slots(int n_tokens, int n_seqs) {
    const long long n = (long long)n_tokens / kC + n_seqs;
    return n > 0x7fffffff ? 0x7fffffff : (int)n;
}

template <int DK>
cudaError_t run_chunks(const DeltaParams& p, cudaStream_t st) {
    const int slots = chunk_slots(p.n_tokens, p.n_seqs);
    const int z = p.n_seqs < 65535 ? p.n_seqs : 65535;
    k_delta_chunks<DK><<<dim3(chunks_of(p.max_new), p.H / p.group, z), kPrepThreads, 0, st>>>(p, slots);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = allow_smem<k_delta_scan<DK>>(sizeof(Scan<DK>));
    if (e != cudaSuccess) return e;
    // (Not overlapped with the chunks' kernel: blocks that start while it
    // drains gather two to an SM on the first SMs to empty, which are then the
    // last to finish: 394 us for one sequence of 4096 tokens instead of 275.)
    k_delta_scan<DK><<<(unsigned)((size_t)p.n_seqs * p.H * (p.DV / kN)), kScanThreads, sizeof(Scan<DK>), st>>>(p, slots);
    return cudaGetLastError();
}

}  // namespace

size_t delta_chunk_ws_bytes(int H, int n_tokens, int n_seqs, int max_new) {
    return max_new <= kFew ? 0 : sizeof(ChunkData) * (size_t)chunk_slots(n_tokens, n_seqs) * H;
}

cudaError_t run_delta(const DeltaParams& p, cudaStream_t st) {
    if (p.max_new > kFew) return p.DK == 64 ? run_chunks<64>(p, st) : run_chunks<128>(p, st);
    const unsigned g = (unsigned)((size_t)p.n_seqs * p.H * (p.DV / kShortN));
    if (p.DK == 64) k_delta_short<64><<<g, kShortThreads, 0, st>>>(p);
    else k_delta_short<128><<<g, kShortThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace lmoe
