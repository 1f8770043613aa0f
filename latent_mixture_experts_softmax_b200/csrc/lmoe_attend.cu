// Attention of new tokens over the 8-bit paged cache: the kernel for few
// query rows per key head (decode steps and verify windows), and the kernel
// that joins results cut between CTAs.
//
// Mathematics.  For one key head the query rows are the pairs (new token,
// query head of its group); with codes c_j and scales a_j (keys), b_j
// (values),
//   t_j = scale log2(e) a_j (q . ck_j) + log2(b_j),   p_j = 2^(t_j - m),
//   out = sum_j p_j cv_j / sum_j p_j (1 / b_j)
// (the second sum in a unit that keeps it inside fp32, kSumUnit; rows of zeros
// enter it by their bare score, kZeroDrop).
// Folding the value's scale into the exponent keeps the second product in
// fp16 whatever the scales are: p is below 2^16 (kMaxP) and the codes are
// exact in fp16 (integers up to 127, E4M3 values), so the only rounding is
// that of p to fp16 (half a step, 2^-11).  Queries are scaled by a power of
// two per row, their largest into [1, 2): exact in fp16 down to 2^-17 of it,
// smaller elements (fp16's subnormals) off by up to 2^-25; sums are fp32.
//
// What bounds it: the bytes of the codes, each read once (64 tokens of a batch
// over up to 16K cached ones: 130 us, 4.5 TB/s), up to 8 rows; with 32 rows
// and head_dim 256 the latency of one block of eight warps an SM (32 tokens
// over up to 128K: 267 us, 2.4 TB/s).  The products run
// on mma.sync m16n8k16 with the tokens as M (S^T = K Q^T) and the query rows
// as N, so 8 rows cost one instruction per 16 tokens and 16 columns, and
// neither product needs a transposed copy of the codes: both sums run over
// permuted index orders that make a lane's operand bytes contiguous in the
// stored rows (16-byte loads straight to registers, converted there).
//
// Split: the work of all (sequence, key head, row tile) items is laid out on
// one line in units of 128 tokens and cut into equal pieces, one per CTA
// whatever the lengths; the 8 warps of a CTA take 16-token steps in turn and
// join their results through shared memory.  An item cut between CTAs leaves
// its parts in the workspace for k_attend_join, which adds them in order.

#include "lmoe_attend.cuh"
#include "lmoe_sm100.cuh"

namespace lmoe {

namespace {

using namespace sm100;
using namespace attend;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = kFewRows;
constexpr float kNull = 0x1p127f;       // stands for the inverse of a scale of 0

// ---------------------------------------------------------------------------
// arithmetic
// ---------------------------------------------------------------------------

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ---------------------------------------------------------------------------
// few query rows
// ---------------------------------------------------------------------------

// D, code format, NR tiles of 8 query rows, NS warps that share a step: each
// sums the scores over D / NS of the columns, which they add up through shared
// memory, and holds D / NS of the output columns, which bounds the
// accumulators to 128 registers.
template <int D, int FMT, int NR, int NS>
struct Few {
    static_assert(NS == 1 || (NS == 2 && D == 256), "a lane's 16 bytes of each half of a value row");
    static constexpr int kRows = 8 * NR;
    static constexpr int kGroups = kWarps / NS;
    static constexpr int kSteps = D / 16;              // K steps of the score product
    static constexpr int kOwn = kSteps / NS;           // those of a warp
    static constexpr int kKw = kOwn;                   // words of a key row per lane
    static constexpr int kVw = D / 32 / NS;            // words of a value row per lane
    static constexpr int kTiles = 2 * kVw;             // M tiles of the output product per warp
    static constexpr int kOut = kTiles * 4 * NR;       // accumulators
    static constexpr bool kQInRegs = kOwn * 2 * NR <= 32;
    static constexpr size_t kQBytes = (size_t)kSteps * NR * 32 * 8;
    static constexpr size_t kJoinBytes = (size_t)(kGroups / 2) * NS * kOut * 32 * 4;
    static constexpr size_t kShareBytes = NS == 2 ? (size_t)2 * kWarps * 4 * NR * 32 * 4 : 0;
    static constexpr size_t kSmem = kQBytes + kJoinBytes + kShareBytes;
    static constexpr int kCtasPerSm = kOut <= 32 ? 2 : 1;   // 128 or 255 registers a thread
};

template <int D, int FMT, int NR, int NS>
__global__ void __launch_bounds__(kThreads, Few<D, FMT, NR, NS>::kCtasPerSm)
    k_attend_few(AttendParams p, Plan pl) {
    using C = Few<D, FMT, NR, NS>;
    extern __shared__ __align__(16) char smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem);                       // query fragments [step][NR][lane]
    float* jbuf = reinterpret_cast<float*>(smem + C::kQBytes);
    float4* share = reinterpret_cast<float4*>(smem + C::kQBytes + C::kJoinBytes);     // [2][warp][NR][lane]
    __shared__ float s_qscale[kMaxRows];
    __shared__ int s_pos[kMaxRows];
    __shared__ float s_m[kWarps][kMaxRows], s_l[kWarps][kMaxRows];

    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int grp = warp / NS, hs = warp % NS;
    const Line line = find_unit(p, pl, gridDim.x, [&](const Line& l) { return l.chunk * blockIdx.x; });
    const long long x_begin = line.chunk * blockIdx.x;
    long long x = x_begin;
    const long long x_end = min(line.total, x + line.chunk);
    if (x >= x_end) {
        if (threadIdx.x == 0) p.cuts[blockIdx.x].x = -1;
        return;
    }
    Item it;
    it.seek(p, pl, line, x);
    const int page_mask = (1 << p.page_log2) - 1;

    for (;;) {
        const int u0 = (int)(x - it.begin);
        const int u1 = (int)min((long long)it.tile.units, x_end - it.begin);
        const int r0 = it.rt * C::kRows, n_rows = min(C::kRows, it.rows.n * p.G - r0);
        const int first = it.rows.kv - it.rows.n;

        // ---- queries: rows scaled by a power of two into fp16, as fragments
        __syncthreads();
        for (int r = warp; r < C::kRows; r += kWarps) {
            float v[D / 32];
            float a = 0.f;
            const int row = r0 + r;
            if (r < n_rows) {
                const uint16_t* src = p.q + (size_t)(it.rows.q0 + row / p.G) * p.q_stride +
                                      (size_t)(it.head * p.G + row % p.G) * D + lane * (D / 32);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const float2 f = bf16x2_to_f32x2(__ldg(reinterpret_cast<const uint32_t*>(src) + i));
                    v[2 * i] = f.x;
                    v[2 * i + 1] = f.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 32; ++i) v[i] = 0.f;
            }
            bool bad = false;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                a = fmaxf(a, fabsf(v[i]));
                bad |= !(fabsf(v[i]) <= 3.4e38f);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            bad = __any_sync(0xffffffffu, bad);
            // 2^e with a 2^-e in [1, 2); the exponent is kept where both
            // powers are normal
            int e = (int)(__float_as_uint(a) >> 23) - 127;
            e = min(max(e, -100), 126);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
            // element d of a row: step (d / 64) * 4 + (d / 4) % 4 and lane t = (d / 16) % 4
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = lane * (D / 32) + i;
                const int step = (d >> 6) * 4 + ((d >> 2) & 3), tt = (d >> 4) & 3;
                __half* f = reinterpret_cast<__half*>(qf + ((size_t)step * NR + (r >> 3)) * 32 + (r & 7) * 4 + tt);
                f[d & 3] = __float2half_rn(bad ? 0.f : v[i] * down);
            }
            if (lane == 0) {
                s_qscale[r] = bad ? __int_as_float(0x7fffffff) : up * p.scale_log2;
                s_pos[r] = first + row / p.G;
            }
        }
        __syncthreads();

        float qscale[NR][2];
        uint2 q_reg[C::kQInRegs ? C::kOwn : 1][NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            qscale[r][0] = s_qscale[8 * r + 2 * t];
            qscale[r][1] = s_qscale[8 * r + 2 * t + 1];
            if (C::kQInRegs) {
#pragma unroll
                for (int k = 0; k < C::kOwn; ++k) q_reg[k][r] = qf[((size_t)(hs * C::kOwn + k) * NR + r) * 32 + lane];
            }
        }

        float o[C::kTiles][NR][4];
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int j = 0; j < C::kTiles; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][r][i] = 0.f;
            m[r][0] = m[r][1] = -INFINITY;
            l[r][0] = l[r][1] = 0.f;
        }

        // ---- the piece's 16-token steps, this warp's in turn
        const int st_end = min(it.tile.step1, it.tile.step0 + u1 * C::kGroups);
        int st = it.tile.step0 + u0 * C::kGroups + grp;
        const int32_t* table = p.table + (size_t)it.s * p.table_stride;
        // rows all of whose tokens every query row sees need no mask
        const int pos_lo = p.causal ? first + r0 / p.G : it.rows.kv - 1;
        const int pos_hi = first + (r0 + n_rows - 1) / p.G;
        const int win_lo = p.window ? pos_hi - p.window : -1;

        uint32_t kw[2][C::kKw], vw[4][C::kVw];
        float ks[2], vs[2];
        bool ok = false;            // the step's page exists
        size_t row = 0;
        auto locate = [&](int step, bool& good) -> size_t {
            const int tok = step << 4;
            const int page = __ldg(table + (tok >> p.page_log2));
            good = page >= 0 && page < p.n_pages;
            if (!good) set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
            return page_row(p, good ? page : 0, it.head) + (tok & page_mask);
        };
        auto load_k = [&](size_t base) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* src = p.k + (base + g + 8 * h) * D + hs * (D / NS) + t * 16;
#pragma unroll
                for (int i = 0; i < D / 64 / NS; ++i) {
                    const uint4 v = ldg_stream(reinterpret_cast<const uint4*>(src + i * 64));
                    kw[h][4 * i] = v.x;
                    kw[h][4 * i + 1] = v.y;
                    kw[h][4 * i + 2] = v.z;
                    kw[h][4 * i + 3] = v.w;
                }
                ks[h] = __ldg(p.ks + base + g + 8 * h);
                vs[h] = __ldg(p.vs + base + g + 8 * h);
            }
        };
        auto load_v = [&](size_t base) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint8_t* src = p.v + (base + 2 * t + (h & 1) + 8 * (h >> 1)) * D;
                if (D == 64) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + g * 8));
                    vw[h][0] = v.x;
                    vw[h][1] = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < C::kVw / 4; ++i) {
                        const uint4 v = ldg_stream(reinterpret_cast<const uint4*>(src + ((hs + i) * 8 + g) * 16));
                        vw[h][4 * i] = v.x;
                        vw[h][4 * i + 1] = v.y;
                        vw[h][4 * i + 2] = v.z;
                        vw[h][4 * i + 3] = v.w;
                    }
                }
            }
        };
        size_t row_next = 0;
        bool ok_next = false;
        int odd = 0;
        if (st < st_end) {
            row = locate(st, ok);
            load_k(row);
            load_v(row);
            if (st + C::kGroups < st_end) row_next = locate(st + C::kGroups, ok_next);
        }
        for (; st < st_end; st += C::kGroups) {
            const bool more = st + C::kGroups < st_end;
            // scores, tokens x rows
            float s[NR][4];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][i] = 0.f;
#pragma unroll
            for (int k = 0; k < C::kOwn; ++k) {
                uint32_t a[4];
                codes_to_f16<FMT>(biased<FMT>(kw[0][k]), a[0], a[2]);
                codes_to_f16<FMT>(biased<FMT>(kw[1][k]), a[1], a[3]);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const uint2 b = C::kQInRegs ? q_reg[C::kQInRegs ? k : 0][r] : qf[((size_t)(hs * C::kOwn + k) * NR + r) * 32 + lane];
                    mma_f16(s[r], a, b.x, b.y);
                }
            }
            if (NS == 2) {           // (both add the same two numbers; the next step uses the other half of the buffer)
                float4* mine = share + (((size_t)odd * kWarps + warp) * NR) * 32 + lane;
                const float4* other = share + (((size_t)odd * kWarps + (warp ^ 1)) * NR) * 32 + lane;
#pragma unroll
                for (int r = 0; r < NR; ++r) mine[r * 32] = make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
                named_bar_sync(1 + grp, 64);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float4 y = other[r * 32];
                    s[r][0] += y.x;
                    s[r][1] += y.y;
                    s[r][2] += y.z;
                    s[r][3] += y.w;
                }
                odd ^= 1;
            }
            const float k0 = ks[0], k1 = ks[1];
            // scales that are no numbers from 0 on make a score NaN (a row stored
            // as NaN) or belong to places that are masked below; 0 and 1 may be
            // rows of zeros (looking for them in this order costs a batch of 64
            // single tokens nothing; as part of the branches for masks or for m: 4%)
            const bool zeros = __any_sync(0xffffffffu, vs[0] == 0.f || vs[0] == 1.f || vs[1] == 0.f || vs[1] == 1.f);
            float lv0 = vs[0] < INFINITY ? __log2f(vs[0]) : __int_as_float(0x7fffffff);
            float lv1 = vs[1] < INFINITY ? __log2f(vs[1]) : __int_as_float(0x7fffffff);
            const float iv0 = fminf(fabsf(__frcp_rn(vs[0]) * kSumUnit), kNull), iv1 = fminf(fabsf(__frcp_rn(vs[1]) * kSumUnit), kNull);
            if (__builtin_expect(zeros, 0)) {            // the bare score
                lv0 = vs[0] == 0.f ? 0.f : lv0;
                lv1 = vs[1] == 0.f ? 0.f : lv1;
            }
            const int tok = st << 4;
            const bool whole = ok && tok + 15 <= min(pos_lo, it.rows.kv - 1) && tok > win_lo;
            const bool ok_now = ok;
            if (more) {
                load_k(row_next);
                ok = ok_next;
            }
            float top = -INFINITY;
            bool grow = false;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                s[r][0] = fmaf(s[r][0] * k0, qscale[r][0], lv0);
                s[r][1] = fmaf(s[r][1] * k0, qscale[r][1], lv0);
                s[r][2] = fmaf(s[r][2] * k1, qscale[r][0], lv1);
                s[r][3] = fmaf(s[r][3] * k1, qscale[r][1], lv1);
            }
            if (!whole) {
                const int t0 = tok + g, t1 = t0 + 8;
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tk = i < 2 ? t0 : t1, pos = s_pos[8 * r + 2 * t + (i & 1)];
                        bool seen = ok_now && tk < it.rows.kv;
                        if (p.causal) seen = seen && tk <= pos && (!p.window || tk > pos - p.window);
                        if (!seen) s[r][i] = -INFINITY;
                    }
                // codes behind the last token may be anything, a NaN code too
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (!ok_now || tok + 2 * t + (h & 1) + 8 * (h >> 1) >= it.rows.kv)
#pragma unroll
                        for (int i = 0; i < C::kVw; ++i) vw[h][i] = 0u;
            }
            bool z0 = false, z1 = false;                 // rows g and g + 8 are zeros
            if (__builtin_expect(zeros, 0)) {
                // bit g * 4 + t of any[h] tells of codes in row 2 t + (h & 1) + 8 (h >> 1).
                // (The other warp's columns are read here: a barrier of the two would
                // hang where a row behind the last token, which another call may be
                // writing, shows one of them a scale of 1.)
                uint32_t any[4];
                bool here = true;
                const uint8_t* others = NS == 2 ? p.v + locate(st, here) * D + ((hs ^ 1) * 8 + g) * 16 : nullptr;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < C::kVw; ++i) w |= vw[h][i];
                    if (NS == 2) {
                        const uint4 y = ldg_stream(reinterpret_cast<const uint4*>(others + (2 * t + (h & 1) + 8 * (h >> 1)) * D));
                        w |= y.x | y.y | y.z | y.w;
                    }
                    any[h] = __ballot_sync(0xffffffffu, (FMT == LMOE_KV_INT8 ? w : w & 0x7f7f7f7fu) != 0);
                }
                const uint32_t row_g = 0x11111111u << (g >> 1);
                z0 = iv0 == kNull || (iv0 == kSumUnit && !((g & 1 ? any[1] : any[0]) & row_g));
                z1 = iv1 == kNull || (iv1 == kSumUnit && !((g & 1 ? any[3] : any[2]) & row_g));
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < 2 ? z0 : z1) s[r][i] -= kZeroDrop;
            }
            // m is raised rarely, so most steps skip the exchange between
            // lanes and the rescaling
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top = fmaxf(s[r][i], s[r][i + 2]);
                    grow |= top > m[r][i] + kMaxP;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float n = fmaxf(s[r][i], s[r][i + 2]);
                        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
                        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
                        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16));
                        n = fmaxf(n - kRaiseP, m[r][i]);
                        const float h = m[r][i] == n ? 1.f : ex2(0.5f * (m[r][i] - n)), f = h * h;
                        m[r][i] = n;
                        l[r][i] = twice(l[r][i], h);
#pragma unroll
                        for (int j = 0; j < C::kTiles; ++j) {
                            o[j][r][i] *= f;
                            o[j][r][i + 2] *= f;
                        }
                    }
            }
            if (__builtin_expect(zeros, 0)) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < 2 ? z0 : z1) {
                            const float mm = m[r][i & 1] == -INFINITY ? 0.f : m[r][i & 1];
                            l[r][i & 1] += ex2(s[r][i] + kZeroDrop - mm) * kSumUnit;
                            s[r][i] = -INFINITY;
                        }
            }
            uint32_t pb[NR][2];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float m0 = m[r][0] == -INFINITY ? 0.f : m[r][0], m1 = m[r][1] == -INFINITY ? 0.f : m[r][1];
                const float p0 = ex2(s[r][0] - m0), p1 = ex2(s[r][1] - m1), p2 = ex2(s[r][2] - m0), p3 = ex2(s[r][3] - m1);
                l[r][0] = fmaf(p0, iv0, fmaf(p2, iv1, l[r][0]));
                l[r][1] = fmaf(p1, iv0, fmaf(p3, iv1, l[r][1]));
                const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
                pb[r][0] = movmatrix(*reinterpret_cast<const uint32_t*>(&h0));
                pb[r][1] = movmatrix(*reinterpret_cast<const uint32_t*>(&h1));
            }
            // output, columns x rows
#pragma unroll
            for (int w = 0; w < C::kVw; ++w) {
                const uint32_t v0 = biased<FMT>(vw[0][w]), v1 = biased<FMT>(vw[1][w]), v2 = biased<FMT>(vw[2][w]),
                               v3 = biased<FMT>(vw[3][w]);
                uint32_t a[2][4];
                codes_to_f16<FMT>(prmt(v0, v1, 0x5140), a[0][0], a[0][1]);
                codes_to_f16<FMT>(prmt(v2, v3, 0x5140), a[0][2], a[0][3]);
                codes_to_f16<FMT>(prmt(v0, v1, 0x7362), a[1][0], a[1][1]);
                codes_to_f16<FMT>(prmt(v2, v3, 0x7362), a[1][2], a[1][3]);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma_f16(o[2 * w + j][r], a[j], pb[r][0], pb[r][1]);
            }
            if (more) {
                load_v(row_next);
                if (st + 2 * C::kGroups < st_end) row_next = locate(st + 2 * C::kGroups, ok_next);
            }
        }

        // ---- join the warps
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[r][i] += __shfl_xor_sync(0xffffffffu, l[r][i], d);
                if (g == 0 && hs == 0) {
                    s_m[grp][8 * r + 2 * t + i] = m[r][i];
                    s_l[grp][8 * r + 2 * t + i] = l[r][i];
                }
            }
        __syncthreads();
        float ltot[NR][2], mtot[NR][2];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rr = 8 * r + 2 * t + i;
                float n = -INFINITY;
#pragma unroll
                for (int w = 0; w < C::kGroups; ++w) n = fmaxf(n, s_m[w][rr]);
                const float nn = n == -INFINITY ? 0.f : n;
                float sum = 0.f;
#pragma unroll
                for (int w = 0; w < C::kGroups; ++w) sum += twice(s_l[w][rr], ex2(0.5f * (s_m[w][rr] - nn)));
                mtot[r][i] = n;
                ltot[r][i] = sum;
                const float f = ex2(m[r][i] - nn);
#pragma unroll
                for (int j = 0; j < C::kTiles; ++j) {
                    o[j][r][i] *= f;
                    o[j][r][i + 2] *= f;
                }
            }
#pragma unroll
        for (int h = C::kGroups / 2; h > 0; h >>= 1) {
            if (grp >= h && grp < 2 * h) {
                float* b = jbuf + ((size_t)((grp - h) * NS + hs) * C::kOut) * 32 + lane;
#pragma unroll
                for (int j = 0; j < C::kTiles; ++j)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) b[((j * NR + r) * 4 + i) * 32] = o[j][r][i];
            }
            __syncthreads();
            if (grp < h) {
                const float* b = jbuf + ((size_t)(grp * NS + hs) * C::kOut) * 32 + lane;
#pragma unroll
                for (int j = 0; j < C::kTiles; ++j)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[j][r][i] += b[((j * NR + r) * 4 + i) * 32];
            }
            __syncthreads();
        }
        if (grp == 0) {
            const bool cut = u0 > 0 || u1 < it.tile.units;
            // lane (g, t): rows 2t, 2t + 1 of each 8, columns per word w, tile
            // pair j and half: the bytes it read of a value row
            float* part = p.part + ((size_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * part_floats(C::kRows, D);
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int rr = 8 * r + 2 * t + i;
                    if (rr >= n_rows) continue;
                    const Norm norm = cut ? Norm{1.f, 1.f} : norm_of(ltot[r][i]);
                    const size_t orow = (size_t)(it.rows.q0 + (r0 + rr) / p.G) * p.Hq + it.head * p.G + (r0 + rr) % p.G;
#pragma unroll
                    for (int w = 0; w < C::kVw; ++w) {
                        const int d = D == 64 ? g * 8 + 4 * w : ((hs + (w >> 2)) * 8 + g) * 16 + 4 * (w & 3);
                        float y[4] = {o[2 * w][r][i], o[2 * w][r][i + 2], o[2 * w + 1][r][i], o[2 * w + 1][r][i + 2]};
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = y[e] * norm.inv * norm.post;
                        if (cut) {
                            *reinterpret_cast<float4*>(part + (size_t)rr * D + d) = make_float4(y[0], y[1], y[2], y[3]);
                        } else {
                            const uint2 b = make_uint2(
                                (uint32_t)f32_to_bf16_bits(y[0]) | (uint32_t)f32_to_bf16_bits(y[1]) << 16,
                                (uint32_t)f32_to_bf16_bits(y[2]) | (uint32_t)f32_to_bf16_bits(y[3]) << 16);
                            *reinterpret_cast<uint2*>(p.out + orow * D + d) = b;
                        }
                    }
                    if (g == 0 && hs == 0) {
                        if (cut) {
                            part[(size_t)C::kRows * D + rr] = mtot[r][i];
                            part[(size_t)C::kRows * (D + 1) + rr] = ltot[r][i];
                        } else if (p.lse) {
                            p.lse[orow] = lse_of(mtot[r][i], ltot[r][i]);
                        }
                    }
                }
        }
        x = it.begin + u1;
        if (x >= x_end || !it.next(p, pl)) break;
    }
    if (threadIdx.x == 0) {
        const Cut c = it.begin >= x_begin ? cut_of(line, it, x_end) : Cut{-1, 0, 0, 0};
        p.cuts[blockIdx.x] = make_int4(c.s, c.head, c.rt, c.last);
    }
}

// ---------------------------------------------------------------------------
// items cut between CTAs
// ---------------------------------------------------------------------------

constexpr int kJoinThreads = 128;

// Block (c, b): rows of the item that CTA c began and others went on with.
// FEW: one row a block, whose four warps take parts in turn (an item of few
// rows may be spread over all CTAs); else four rows a warp side by side (an
// item of many rows has few parts).  A lane looks at a part's reference and
// sum, so that one load's time covers them all (one part after the other, a
// prompt's join took 19 us).  Parts are added in a fixed order.
template <int D, bool FEW>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(AttendParams p, int rows) {
    constexpr int V = D / 32, RW = FEW ? 1 : 4, PS = FEW ? 4 : 1;   // rows of a warp, warps that share their parts
    __shared__ float s_o[FEW ? 4 : 1][FEW ? D : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dep_wait();
    const int4 cut = p.cuts[blockIdx.x];
    if (cut.x < 0) return;
    const int c = blockIdx.x, np = cut.w - c + 1;
    const SeqRows sr = seq_rows(p, cut.x);
    const int r0 = cut.z * rows, n_rows = min(rows, sr.n * p.G - r0);
    const int rr0 = FEW ? blockIdx.y : blockIdx.y * 16 + warp * 4;
    if (rr0 >= n_rows) return;                  // a whole block (FEW), or the warp's rows
    const size_t pf = part_floats(rows, D);
    auto part = [&](int k) { return p.part + ((size_t)(c + k) * 2 + (k == 0 ? 1 : 0)) * pf; };
    int rr[RW];                                 // (past the last row: that row again)
    float m[RW], l[RW], o[RW][V];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        rr[i] = min(rr0 + i, n_rows - 1);
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[i][v] = 0.f;
    }
    // (FEW: a warp's first two parts are on their way before the references
    // are known: a single token's join is nothing but such waits)
    float ahead[FEW ? 2 : 1][V];
    if (FEW) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float* s = part(min(warp + PS * u, np - 1)) + (size_t)rr[0] * D + lane;
#pragma unroll
            for (int v = 0; v < V; ++v) ahead[u][v] = s[32 * v];
        }
    }
    for (int k0 = 0; k0 < np; k0 += 32) {
        const float* q = part(min(k0 + lane, np - 1)) + (size_t)rows * D;
#pragma unroll
        for (int i = 0; i < RW; ++i) m[i] = fmaxf(m[i], q[rr[i]]);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    for (int k0 = 0; k0 < np; k0 += 32) {
        const float* q = part(min(k0 + lane, np - 1)) + (size_t)rows * D;
        float f[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const float d = q[rr[i]] - (m[i] == -INFINITY ? 0.f : m[i]);
            f[i] = k0 + lane < np ? ex2(d) : 0.f;
            const float y = twice(q[rows + rr[i]], ex2(0.5f * d));
            l[i] = k0 + lane < np ? l[i] + y : l[i];
        }
        const int n = min(32, np - k0);
        int j = FEW ? warp : 0;
        if (FEW && k0 == 0) {
#pragma unroll
            for (int u = 0; u < 2; ++u, j += PS) {
                const float w = __shfl_sync(0xffffffffu, f[0], j);       // (0 past the last part)
#pragma unroll
                for (int v = 0; v < V; ++v) o[0][v] = j < np ? fmaf(w, ahead[u][v], o[0][v]) : o[0][v];
            }
        }
#pragma unroll 2
        for (; j < n; j += PS) {
            const float* s = part(k0 + j);
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                const float w = __shfl_sync(0xffffffffu, f[i], j);
#pragma unroll
                for (int v = 0; v < V; ++v) o[i][v] = fmaf(w, s[(size_t)rr[i] * D + lane + 32 * v], o[i][v]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
    if (FEW) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[warp][lane + 32 * v] = o[0][v];
        __syncthreads();
        if (warp) return;
#pragma unroll
        for (int v = 0; v < V; ++v)
            o[0][v] = (s_o[0][lane + 32 * v] + s_o[1][lane + 32 * v]) + (s_o[2][lane + 32 * v] + s_o[3][lane + 32 * v]);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const Norm norm = norm_of(l[i]);
        const size_t orow = (size_t)(sr.q0 + (r0 + rr[i]) / p.G) * p.Hq + cut.y * p.G + (r0 + rr[i]) % p.G;
#pragma unroll
        for (int v = 0; v < V; ++v) p.out[orow * D + lane + 32 * v] = f32_to_bf16_bits(o[i][v] * norm.inv * norm.post);
        if (lane == 0 && p.lse) p.lse[orow] = lse_of(m[i], l[i]);
    }
}

}  // namespace

// Starts while the attention kernel drains, and waits for it on the device.
cudaError_t attend::launch_join(const AttendParams& p, int rows, int n_ctas, bool few, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(n_ctas, few ? rows : rows / 16);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = 1;
    if (p.D == 64) return cudaLaunchKernelEx(&cfg, few ? k_attend_join<64, true> : k_attend_join<64, false>, p, rows);
    if (p.D == 128) return cudaLaunchKernelEx(&cfg, few ? k_attend_join<128, true> : k_attend_join<128, false>, p, rows);
    return cudaLaunchKernelEx(&cfg, few ? k_attend_join<256, true> : k_attend_join<256, false>, p, rows);
}

namespace {

template <int D, int FMT, int NR, int NS>
cudaError_t launch_few(const AttendParams& p, cudaStream_t st) {
    using C = Few<D, FMT, NR, NS>;
    const Plan pl{C::kRows, 4, C::kGroups, 0};
    constexpr int kCtas = kSms * C::kCtasPerSm;
    cudaError_t e = allow_smem<k_attend_few<D, FMT, NR, NS>>(C::kSmem);
    if (e != cudaSuccess) return e;
    k_attend_few<D, FMT, NR, NS><<<kCtas, kThreads, C::kSmem, st>>>(p, pl);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_join(p, C::kRows, kCtas, true, st);
}

// Rows of a sequence and key head, by their bound.  30 rows of head_dim 128 over
// 8 x 4096 (4 x 32768) tokens take 57 (98) us here, 66 (162) in the kernel for
// many rows; 65 rows 82 (186) against 66 (162).  Of 40 rows, two row tiles here
// would take 64 (137) against 66 (162): the switch stands at one tile.
template <int D, int FMT>
cudaError_t launch_rows(const AttendParams& p, cudaStream_t st) {
    const long long rows = (long long)p.max_new * p.G;
    if (rows <= 8) return launch_few<D, FMT, 1, 1>(p, st);
    if (rows <= 16) return launch_few<D, FMT, 2, 1>(p, st);
    if (rows <= 32) return launch_few<D, FMT, 4, D == 256 ? 2 : 1>(p, st);
    return launch_many(p, st);
}

}  // namespace

static size_t parts_bytes(int D) {
    const size_t few = kMaxCtas * part_floats(kFewRows, D), many = kSms * part_floats(many_rows(D), D);
    return (2 * 4 * (few > many ? few : many) + 255) & ~(size_t)255;
}

size_t attend_ws_bytes(int D) { return kCutBytes + parts_bytes(D) + kImageBytes; }

cudaError_t run_attend(AttendParams p, void* ws, cudaStream_t st) {
    p.cuts = static_cast<int4*>(ws);
    p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kCutBytes);
    p.img = static_cast<char*>(ws) + kCutBytes + parts_bytes(p.D);
    p.img_tiles = 0;
    p.h0 = 0;
    p.Hn = p.Hk;
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) return i8 ? launch_rows<64, LMOE_KV_INT8>(p, st) : launch_rows<64, LMOE_KV_E4M3>(p, st);
    if (p.D == 128) return i8 ? launch_rows<128, LMOE_KV_INT8>(p, st) : launch_rows<128, LMOE_KV_E4M3>(p, st);
    return i8 ? launch_rows<256, LMOE_KV_INT8>(p, st) : launch_rows<256, LMOE_KV_E4M3>(p, st);
}

}  // namespace lmoe
