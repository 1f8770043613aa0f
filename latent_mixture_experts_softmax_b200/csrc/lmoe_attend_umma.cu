// Attention over the 8-bit paged cache, many query rows per key head: prompt
// chunks.
//
// The mathematics is that of the kernel for few rows (lmoe_attend.cu); the
// products run on tcgen05 (kind::f16, fp32 accumulators in tensor memory).
// What bounds it: the softmax warps' own chain.  Of about 2900 cycles a tile of
// 64 tokens and 256 rows (head_dim 128), a warp takes 640 to scale its scores,
// 780 for the exponentials and sums (two warps of a scheduler share 1024 of
// the exponential unit), 300 for votes and the rare change of the reference,
// and the rest waits for barriers; the tensor core needs 1024, at the pace at
// which shared memory gives it Q, K and V.  4096 causal tokens of 20 heads take
// 156 us (550 TFLOP/s), 2048 tokens over 32768 of head_dim 256 713 us (934
// TFLOP/s; the card runs that power-capped).
//
// A CTA (one per SM) holds query tiles of 128 rows as fp16 in shared memory
// (two for head_dim 64 and 128, one for 256) and walks the keys in tiles of
// 64 tokens:
//   softmax      eight warps: a thread owns a row; S comes from tensor memory, P
//                goes back over it as the A operand.  Four warps have a query
//                tile each; where there is one tile, they take its key tiles in
//                turn, handing on the row's reference.  (Warps that meet in
//                every tile do the exponentials at the same time, and the units
//                for those stand still in between.)
//   keys, values the operands of a tile: a key row is K-major as it is stored,
//                and the same layout read as MN-major is the value operand, so
//                neither is transposed.  One thread each fetches them as images
//                (k_attend_images) that were laid out once for all row tiles;
//                where few row tiles read a key tile (launch_groups), four
//                warps each read the codes (registers, a tile ahead) and write
//                them as fp16 with the 128-byte swizzle.
//   issue        a warp per query tile: S = Q K^T and O += P V (one warp for both
//                would make each wait for the other's probabilities)
// Four score buffers let S run two tiles ahead of the sums.  The row's
// reference m is raised as in the kernel for few rows, and to a whole number,
// so that what it rescales changes by a power of two.
//
// Work is cut into equal pieces of the line of (item, key tile) units as in
// the kernel for few rows, one piece per CTA; cut items are joined after it.

#include "lmoe_attend.cuh"
#include "lmoe_sm100.cuh"

namespace lmoe {

namespace {

using namespace sm100;
using namespace attend;

constexpr int kExtra = 6;                        // loading the queries and writing the sums, in key tiles
constexpr uint64_t kWaitLimit = 4000000000ull;   // SM cycles per barrier wait (about 2 s)
constexpr uint64_t kDrainLimit = 20000000ull;    // and per wait for a copy in flight after one gave up

template <int D, bool IMG>
struct Many {
    static constexpr int NQ = D == 256 ? 1 : 2;       // query tiles of 128 rows
    static constexpr int TK = 64;                     // tokens of a key tile
    static constexpr int NST = D == 256 ? 2 : 4;      // stages of keys, and of values
    static constexpr int kRows = NQ * 128;
    static constexpr int kKeyWarp = 8, kValueWarp = kKeyWarp + (IMG ? 1 : 4),
                         kMmaWarp = kValueWarp + (IMG ? 1 : 4);
    static constexpr int kThreads = (kMmaWarp + NQ) * 32;
    static constexpr size_t kQBytes = 128 * D * 2;    // one query tile
    static constexpr size_t kOpBytes = TK * D * 2;    // one stage of keys or values
    // per token: key scale, log2 and inverse of the value scale; then a bit per
    // token whose value row is all zeros
    static constexpr size_t kScaleBytes = 3 * TK * 4 + 16;
    // keys, values, scales of a tile, in whole lines of 128 bytes (copies from
    // other addresses cost prompts 2%, and 5% with head_dim 256)
    static constexpr size_t kImage = 2 * kOpBytes + (kScaleBytes + 127) / 128 * 128;
    static constexpr size_t kSmem = 1024 + NQ * kQBytes + 2 * NST * kOpBytes + 4 * kScaleBytes + 512;
    static constexpr uint32_t kColO = 256;            // tensor memory: scores from 0 ((NB q + b) * TK), sums from 256 (q * D)
};

// MN-major operand: 64 elements of N (128 bytes, swizzled) by 8 of K per
// 1024-byte atom; atoms of the next 8 K follow, the next 64 N are lbo away.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
    d |= (uint64_t)(lbo >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

constexpr uint32_t kTransposeB = 1u << 16;   // instruction descriptor: B is MN-major

// Products and commits are issued by a whole warp, converged, one elected lane
// of it: 48 cycles for M 128, N 64, K 16 (shared memory's pace), where a
// single lane in a divergent branch needs 60 to 100 to get one out.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Whether a value row's codes are all zeros (nearly every other row shows in
// its first 16 bytes).
template <int D, int FMT>
__device__ __forceinline__ bool zero_codes(const uint8_t* row) {
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(row) + i);
        const uint32_t w = u.x | u.y | u.z | u.w;
        if (FMT == LMOE_KV_INT8 ? w : w & 0x7f7f7f7fu) return false;
    }
    return true;
}

// What the softmax needs of token `tok` of a tile, whose place is `row` (a warp
// has 32 tokens).  A place without one weighs nothing, nor does a value row of
// zeros but in the sum; a value scale that is no number from 0 on makes its
// token's scores NaN.
template <int D, int FMT>
__device__ __forceinline__ void token_scales(const AttendParams& p, bool some, size_t row, float ks, float vs, float* sc, int tok) {
    constexpr int TK = image_tokens(D);
    const bool fine = vs > 0.f && vs < INFINITY;
    const bool zero = some && (vs == 0.f || (vs == 1.f && zero_codes<D, FMT>(p.v + row * D)));
    sc[tok] = some ? ks * p.scale_log2 : 0.f;
    sc[TK + tok] = !some || zero ? -INFINITY : fine ? __log2f(vs) : __int_as_float(0x7fffffff);
    sc[2 * TK + tok] = some && fine ? __frcp_rn(vs) * kSumUnit : 1.f;
    const uint32_t bits = __ballot_sync(0xffffffffu, zero);
    if ((tok & 31) == 0) reinterpret_cast<uint32_t*>(sc + 3 * TK)[tok >> 5] = bits;
}

// The CTA's piece of the line, item by item.
struct Walk {
    Item it;
    long long x, x_end;
    int u0, u1;       // units of the item in this piece
    int t0, t1;       // its key tiles
    int n_rows;

    __device__ void open(const AttendParams& p, const Plan& pl) {
        u0 = (int)(x - it.begin);
        u1 = (int)min((long long)it.tile.units, x_end - it.begin);
        t0 = it.tile.step0 + max(0, u0 - pl.extra);
        t1 = it.tile.step0 + max(0, u1 - pl.extra);
        t1 = min(t1, it.tile.step1);
        n_rows = min(pl.rows, it.rows.n * p.G - it.rt * pl.rows);
    }
    __device__ bool next(const AttendParams& p, const Plan& pl) {
        x = it.begin + u1;
        if (x >= x_end || !it.next(p, pl)) return false;
        open(p, pl);
        return true;
    }
};

template <int D, int FMT, bool IMG>
__global__ void __launch_bounds__(Many<D, IMG>::kThreads, 1) k_attend_many(AttendParams p, Plan pl) {
    using C = Many<D, IMG>;
    constexpr int NQ = C::NQ, TK = C::TK, NST = C::NST;
    constexpr int kStLog2 = NST == 2 ? 1 : 2;
    constexpr int NB = 4 / NQ;                   // score buffers of a query tile
    constexpr int kBufLog2 = NB == 4 ? 2 : 1;
    constexpr bool CH = NQ == 1;                 // two groups of softmax warps take one query tile's key tiles in turn
    constexpr int PW = IMG ? TK : 32;            // columns of a piece (registers: 168 a thread, or 96)
    __shared__ float s_m[2][CH ? 128 : 1];       // reference a key tile left, by the tile's parity
    __shared__ float s_scale[CH ? 128 : 1], s_l[2][CH ? 128 : 1];
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + (-smem_u32(smem_raw) & 1023);
    char* sq = smem;
    char* sk = sq + NQ * C::kQBytes;
    char* sv = sk + NST * C::kOpBytes;
    float* ssc = reinterpret_cast<float*>(sv + NST * C::kOpBytes);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(ssc) + 4 * C::kScaleBytes);
    uint64_t* k_full = bars;         // [NST] keys of a stage written
    uint64_t* v_full = bars + 4;     // [NST]
    uint64_t* k_empty = bars + 8;    // [NST] read by the tensor core (commit)
    uint64_t* v_empty = bars + 12;   // [NST]
    uint64_t* sc_full = bars + 16;   // [4] scales of a stage written
    uint64_t* sc_free = bars + 20;   // [4] and read
    uint64_t* s_full = bars + 24;    // [NB q + b] scores of a buffer done (commit)
    uint64_t* p_full = bars + 28;    // [NB q + b] probabilities written (4 warps)
    uint64_t* o_done = bars + 32;    // [NB q + b] sums updated from a buffer's probabilities (commit)
    uint64_t* pair = bars + 36;      // [quad] CH: the two warps of a row meet
    uint64_t* q_full = bars + 45;    // [q] query tile written
    uint64_t* chain = bars + 41;     // [quad] CH: the reference of a key tile is known
    uint64_t* final_bar = bars + 40;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 47);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&k_full[i], IMG ? 1 : 4);
            mbar_init(&v_full[i], IMG ? 1 : 4);
            mbar_init(&k_empty[i], NQ);
            mbar_init(&v_empty[i], NQ);
            mbar_init(&sc_full[i], IMG ? 1 : 4);
            mbar_init(&sc_free[i], CH ? 4 : 8);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&pair[i], 2);
            mbar_init(&chain[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&q_full[i], CH ? 8 : 4);
        mbar_init(final_bar, NQ);
        *abort_flag = 0;
        p.cuts[blockIdx.x] = make_int4(-1, 0, 0, 0);
        fence_barrier_init();
    }
    if (warp == C::kMmaWarp) {
        __syncwarp();
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    grid_dep_launch();
    tc_fence_before();
    __syncwarp();
    const Line line = find_unit(p, pl, gridDim.x, [&](const Line& l) { return l.chunk * blockIdx.x; });
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const long long x_begin = line.chunk * blockIdx.x;
    Walk w;
    w.x = x_begin;
    w.x_end = min(line.total, x_begin + line.chunk);
    bool more = w.x < w.x_end;
    if (more) {
        w.it.seek(p, pl, line, w.x);
        w.open(p, pl);
    }
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity & 1, abort_flag, kWaitLimit); };

    if (warp < 8) {
        // ------------------------------------------------------ softmax
        const int half = warp >> 2, quad = warp & 3, row = threadIdx.x & 127;
        const int q = CH ? 0 : half;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const uint32_t tO = tmem + lanes + C::kColO + q * D;
        uint32_t n = 0, cnt = 0;     // key tiles of the CTA, and those of this query tile
        uint32_t met = 0;            // meetings of the two warps of a row
        bool dead = false;
        auto meet = [&]() {          // false: given up
            __syncwarp();
            if (lane == 0) mbar_arrive(&pair[quad]);
            const bool ok = wait(&pair[quad], met++);
            return !__any_sync(0xffffffffu, !ok);
        };
        // The sums with key tile i (of this query tile) in them.  A wait by
        // parity is sound while the barrier is at most one phase behind: with a
        // barrier per score buffer the sums of tile i - NB have to be done,
        // which the scores that this warp waited for last imply (they were
        // issued after those sums).
        auto wait_sums = [&](uint32_t i) {
            const bool ok = wait(&o_done[NB * q + (i & (NB - 1))], i >> kBufLog2);
            return !__any_sync(0xffffffffu, !ok);
        };
        // 16 bytes of a row of the query tile's place (fp16 queries, later bf16 sums)
        auto place = [&](int rw, int ch) {
            return reinterpret_cast<uint4*>(sq + q * C::kQBytes + (32 * quad + rw) * 128 + (ch >> 3) * (128 * 128) +
                                            (((ch & 7) ^ (rw & 7)) << 4));
        };
        while (more && !dead) {
            const int r = q * 128 + row, row0 = w.it.rt * C::kRows;
            const bool some = w.t0 < w.t1;
            // this thread's row: token and head (past the last row: that row)
            const int tok = (row0 + min(r, w.n_rows - 1)) / p.G, gh = row0 + min(r, w.n_rows - 1) - tok * p.G;
            const int pos = w.it.rows.kv - w.it.rows.n + tok;
            const unsigned long long orow = (unsigned long long)(w.it.rows.q0 + tok) * p.Hq + w.it.head * p.G + gh;
            float m = -INFINITY, l = 0.f;
            if (q * 128 >= w.n_rows) {                           // a query tile without rows only lets the scales go
                for (int t = w.t0; t < w.t1 && !dead; ++t, ++n) {
                    dead = !wait(&sc_full[n & 3], n >> 2);
                    dead = __any_sync(0xffffffffu, dead);
                    if (!dead && lane == 0) mbar_arrive(&sc_free[n & 3]);
                }
                if (!dead) more = w.next(p, pl);
                continue;
            }
            if (some) {
                if (CH) {
                    dead = !meet();      // both have stored the last item's sums from the tile's place
                    if (dead) break;
                }
                // the warp's rows as fp16, each scaled by a power of two (past
                // the last row: a copy of it, so that no load is conditional);
                // the two warps of a quarter take every other pass
                constexpr int LPR = D / 8, RPL = 32 / LPR;       // lanes of a row, rows of a pass
                const unsigned long long from =
                    (unsigned long long)(w.it.rows.q0 + tok) * p.q_stride + (unsigned long long)(w.it.head * p.G + gh) * D;
                float scale = 0.f;
#pragma unroll 4
                for (int i = CH ? half : 0; i < LPR; i += CH ? 2 : 1) {
                    const int rw = i * RPL + lane / LPR, ch = lane % LPR;
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.q + __shfl_sync(0xffffffffu, from, rw)) + ch);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    uint32_t mb = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) mb = max(mb, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
                    const bool bad = mb >= 0x7f80u;
                    const int e = min(max((int)(mb >> 7) - 127, -100), 126);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    const float up = bad ? __int_as_float(0x7fffffff) : __uint_as_float((uint32_t)(127 + e) << 23);
                    if (CH) {
                        if (ch == 0) s_scale[32 * quad + rw] = up;
                    } else {
#pragma unroll
                        for (int j = 0; j < RPL; ++j) {
                            const float y = __shfl_sync(0xffffffffu, up, j * LPR);
                            if (lane == i * RPL + j) scale = y;
                        }
                    }
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = bf16x2_to_f32x2(u[j]);
                        const __half2 hh = __floats2half2_rn(f.x * down, f.y * down);
                        h[j] = bad ? 0u : *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    *place(rw, ch) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[q]);
                if (CH) {
                    dead = !meet();
                    if (dead) break;
                    scale = s_scale[row];
                }
                const f2 scale2 = pack2(scale, scale);

                for (int t = w.t0; t < w.t1; ++t, ++n, ++cnt) {
                    if (CH && (int)(n & 1) != half) continue;
                    const int st = n & 3, b = NB * q + (cnt & (NB - 1));
                    const float4* ks = reinterpret_cast<const float4*>(ssc + st * (C::kScaleBytes / 4));
                    dead = !wait(&sc_full[st], n >> 2);
                    const uint2 zeros = *reinterpret_cast<const uint2*>(ks + 3 * TK / 4);
                    dead = dead || !wait(&s_full[b], cnt >> kBufLog2);
                    dead = __any_sync(0xffffffffu, dead);
                    if (dead) break;
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t tS = tmem + lanes + b * TK;
                    const int tok0 = t * TK;
                    // keys this row sees: columns lo .. hi - 1
                    const int hi = p.causal ? pos + 1 - tok0 : TK;
                    const int lo = p.window ? pos + 1 - p.window - tok0 : 0;
                    const bool mask = __any_sync(0xffffffffu, hi < TK || lo > 0);
                    uint32_t x[PW];
                    auto exponents = [&](int c) {        // piece c of t_j
#pragma unroll
                        for (int i = 0; i < PW / 32; ++i)
                            tmem_ld_32x32b_x32(tS + PW * c + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * i));
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < PW / 4; ++i) {
                            const float4 k4 = ks[PW / 4 * c + i], b4 = ks[TK / 4 + PW / 4 * c + i];
                            uint32_t* y = x + 4 * i;
                            const float2 z0 = unpack2(fma2(mul2(pack2(__uint_as_float(y[0]), __uint_as_float(y[1])), pack2(k4.x, k4.y)), scale2, pack2(b4.x, b4.y)));
                            const float2 z1 = unpack2(fma2(mul2(pack2(__uint_as_float(y[2]), __uint_as_float(y[3])), pack2(k4.z, k4.w)), scale2, pack2(b4.z, b4.w)));
                            y[0] = __float_as_uint(z0.x);
                            y[1] = __float_as_uint(z0.y);
                            y[2] = __float_as_uint(z1.x);
                            y[3] = __float_as_uint(z1.y);
                        }
                        if (mask) {
#pragma unroll
                            for (int i = 0; i < PW; ++i)
                                if (PW * c + i < lo || PW * c + i >= hi) x[i] = 0xff800000u;
                        }
                    };
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < TK / PW; ++c) {
                        exponents(c);
                        float a = -INFINITY;
#pragma unroll
                        for (int i = 0; i < PW; i += 4) {
                            top = fmaxf(fmaxf(top, __uint_as_float(x[i])), __uint_as_float(x[i + 1]));
                            a = fmaxf(fmaxf(a, __uint_as_float(x[i + 2])), __uint_as_float(x[i + 3]));
                        }
                        top = fmaxf(top, a);
                    }
                    float was = m;                       // the reference of the tile before
                    if (__builtin_expect(zeros.x | zeros.y, 0)) {
                        // tokens whose value row is all zeros (their exponents are -infinity)
                        auto each = [&](auto f) {
#pragma unroll 1
                            for (unsigned long long z = (unsigned long long)zeros.y << 32 | zeros.x; z; z &= z - 1) {
                                const int c = __ffsll(z) - 1;
                                __syncwarp();
                                const float y = tmem_ld_32x32b_x1(tS + c);
                                f(c < lo || c >= hi ? -INFINITY : y * reinterpret_cast<const float*>(ks)[c] * scale);
                            }
                        };
                        float ztop = -INFINITY;
                        each([&](float y) { ztop = fmaxf(ztop, y - kZeroDrop); });
                        if (ztop > m + kMaxP) {          // as below for all of the tile
                            const float n = ceilf(ztop) - kRaiseP;
                            l = twice(l, ex2(0.5f * (m - n)));
                            m = n;
                        }
                        each([&](float y) { l += ex2(y - (m == -INFINITY ? 0.f : m)) * kSumUnit; });
                        top = fmaxf(top, ztop);
                    }
                    if (CH) {
                        was = -INFINITY;
                        if (t > w.t0) {
                            dead = !wait(&chain[quad], n - 1);
                            dead = __any_sync(0xffffffffu, dead);
                            if (dead) break;
                            was = s_m[(n - 1) & 1][row];
                        }
                    }
                    float now = was;
                    const bool grow = __any_sync(0xffffffffu, top > was + kMaxP);
                    if (grow) now = fmaxf(was, ceilf(top) - kRaiseP);
                    if (CH) {
                        s_m[n & 1][row] = now;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&chain[quad]);
                    }
                    if (__any_sync(0xffffffffu, m != now)) {     // (CH: also where the other warp has raised it)
                        l = m == now ? l : twice(l, ex2(0.5f * (m - now)));
                        m = now;
                    }
                    if (grow && t > w.t0) {              // the sums of the earlier tiles are in tensor memory
                        const float f = was == now ? 1.f : ex2(was - now);
                        dead = !wait_sums(cnt - 1);
                        if (dead) break;
                        tc_fence_after();
                        __syncwarp();
#pragma unroll 1
                        for (int d = 0; d < D / 32; ++d) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(tO + 32 * d, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st_32x32b_x32(tO + 32 * d, o);
                        }
                    }
                    const float mm = m == -INFINITY ? 0.f : -m;
                    const f2 m2 = pack2(mm, mm);
                    f2 l2 = pack2(0.f, 0.f), l3 = pack2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < TK / PW; ++c) {
                        if (!IMG) exponents(c);          // (fewer registers: gone through twice)
#pragma unroll
                        for (int g = 0; g < PW / 32; ++g) {
                            uint32_t ph[16];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float4 i4 = ks[TK / 2 + PW / 4 * c + 8 * g + i];
                                const uint32_t* y = x + 32 * g + 4 * i;
                                const float2 y0 = unpack2(add2(pack2(__uint_as_float(y[0]), __uint_as_float(y[1])), m2));
                                const float2 y1 = unpack2(add2(pack2(__uint_as_float(y[2]), __uint_as_float(y[3])), m2));
                                const float p0 = ex2(y0.x), p1 = ex2(y0.y), p2 = ex2(y1.x), p3 = ex2(y1.y);
                                l2 = fma2(pack2(p0, p1), pack2(i4.x, i4.y), l2);
                                l3 = fma2(pack2(p2, p3), pack2(i4.z, i4.w), l3);
                                const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
                                ph[2 * i] = *reinterpret_cast<const uint32_t*>(&h0);
                                ph[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                            }
                            tmem_st_32x32b_x16(tS + 16 * (c * (PW / 32) + g), ph);
                        }
                    }
                    const float2 la = unpack2(l2), lb = unpack2(l3);
                    l += (la.x + la.y) + (lb.x + lb.y);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&p_full[b]);
                        mbar_arrive(&sc_free[st]);
                    }
                }
                if (dead) break;
                if (CH) {
                    dead = !wait(&chain[quad], n - 1);
                    dead = __any_sync(0xffffffffu, dead);
                    if (dead) break;
                    const float now = s_m[(n - 1) & 1][row];
                    s_l[half][row] = l = m == now ? l : twice(l, ex2(0.5f * (m - now)));
                    m = now;
                    dead = !meet();
                    if (dead) break;
                    l = s_l[0][row] + s_l[1][row];
                }
                dead = !wait_sums(cnt - 1);
                if (dead) break;
                tc_fence_after();
                __syncwarp();
            }
            // sums out (CH: a warp has half of its rows' columns)
            constexpr int SP = CH ? 2 : 1;
            const int part_of = CH ? half : 0;
            const bool cut = w.u0 > 0 || w.u1 < w.it.tile.units;
            const bool live = r < w.n_rows;
            float* part = p.part + ((size_t)blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0)) * part_floats(C::kRows, D);
            const int last = w.n_rows - 1 - q * 128 - 32 * quad;     // the warp's last row
            if (last >= 0) {
                const Norm norm = cut ? Norm{1.f, 1.f} : norm_of(l);
#pragma unroll 1
                for (int c = part_of * (D / 32 / SP); c < (part_of + 1) * (D / 32 / SP); ++c) {
                    uint32_t o[32];
                    if (some) {
                        tmem_ld_32x32b_x32(tO + 32 * c, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
                    if (live && cut) {
                        float4* d = reinterpret_cast<float4*>(part + (size_t)r * D + 32 * c);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    } else if (live) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {            // through the query tile's place, for whole-row stores
                            uint32_t h[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float2 y = unpack2(mul2(mul2(pack2(__uint_as_float(o[8 * i + 2 * j]), __uint_as_float(o[8 * i + 2 * j + 1])),
                                                                   pack2(norm.inv, norm.inv)), pack2(norm.post, norm.post)));
                                h[j] = bf16x2_of(y.x, y.y);
                            }
                            *place(lane, 4 * c + i) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                    __syncwarp();
                }
                if (!cut) {
                    constexpr int LPR = D / 8 / SP, RPL = 32 / LPR;
#pragma unroll 4
                    for (int i = 0; i < LPR; ++i) {
                        const int rw = min(i * RPL + lane / LPR, last), ch = part_of * LPR + lane % LPR;   // (the last row: repeated)
                        const unsigned long long at = __shfl_sync(0xffffffffu, orow, rw);
                        *(reinterpret_cast<uint4*>(p.out + at * D) + ch) = *place(rw, ch);
                    }
                    __syncwarp();
                }
                if (live && part_of == 0) {
                    if (cut) {
                        part[(size_t)C::kRows * D + r] = m;
                        part[(size_t)C::kRows * (D + 1) + r] = l;
                    } else if (p.lse) {
                        p.lse[orow] = lse_of(m, l);
                    }
                }
            }
            tc_fence_before();      // O has been read before the next item's first P is announced
            if (threadIdx.x == 0) {
                const bool goes_on = w.u0 == 0 && w.u1 < w.it.tile.units;
                const Cut c = goes_on ? cut_of(line, w.it, w.x_end) : Cut{-1, 0, 0, 0};
                p.cuts[blockIdx.x] = make_int4(c.s, c.head, c.rt, c.last);   // the last item's stands
            }
            more = w.next(p, pl);
        }
    } else if (IMG && warp < C::kMmaWarp) {
        // ------------------------------------------------------ images
        if (lane == 0) {
            const bool keys = warp == C::kKeyWarp;
            uint32_t n = 0;
            bool dead = false, half = false;     // half: the scales of tile n are on their way
            grid_dep_wait();                     // the images are written
            while (more && !dead) {
                const char* img = p.img + ((size_t)w.it.s * p.Hn + (w.it.head - p.h0)) * p.img_tiles * C::kImage;
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const char* src = img + (size_t)t * C::kImage;
                    const int st = n & (NST - 1);
                    const uint32_t ph = (n >> kStLog2) ^ 1;
                    if (keys) {
                        dead = !wait(&sc_free[n & 3], (n >> 2) ^ 1);
                        if (dead) break;
                        mbar_arrive_expect_tx(&sc_full[n & 3], (uint32_t)C::kScaleBytes);
                        bulk_load(ssc + (n & 3) * (C::kScaleBytes / 4), src + 2 * C::kOpBytes, (uint32_t)C::kScaleBytes, &sc_full[n & 3]);
                        half = true;
                        dead = !wait(&k_empty[st], ph);
                        if (dead) break;
                        half = false;
                        mbar_arrive_expect_tx(&k_full[st], (uint32_t)C::kOpBytes);
                        bulk_load(sk + st * C::kOpBytes, src, (uint32_t)C::kOpBytes, &k_full[st]);
                    } else {
                        dead = !wait(&v_empty[st], ph);
                        if (dead) break;
                        mbar_arrive_expect_tx(&v_full[st], (uint32_t)C::kOpBytes);
                        bulk_load(sv + st * C::kOpBytes, src + C::kOpBytes, (uint32_t)C::kOpBytes, &v_full[st]);
                    }
                }
                if (!dead) more = w.next(p, pl);
            }
            // the copies in flight end before the CTA does, after an abort too
            volatile int no_abort = 0;
            uint64_t* full = keys ? k_full : v_full;
            for (uint32_t i = n > NST ? n - NST : 0; i < n; ++i)
                mbar_wait(&full[i & (NST - 1)], (i >> kStLog2) & 1, &no_abort, kDrainLimit);
            if (keys)
                for (uint32_t i = n > 3 ? n - 3 : 0; i < n + (half ? 1 : 0); ++i)
                    mbar_wait(&sc_full[i & 3], (i >> 2) & 1, &no_abort, kDrainLimit);
        }
        __syncwarp();
    } else if (!IMG && warp < C::kMmaWarp) {
        // ------------------------------------------------------ keys, values
        const bool keys = warp < C::kValueWarp;
        const uint8_t* codes = keys ? p.k : p.v;
        char* ring = keys ? sk : sv;
        uint64_t* full = keys ? k_full : v_full;
        uint64_t* empty = keys ? k_empty : v_empty;
        const int tid = threadIdx.x & 127;
        // eight lanes: four 16-byte pieces of two rows, whose swizzled places
        // then cover all banks
        constexpr int BLKS = D / 64;             // 64-column blocks of a row
        constexpr int RPP = 32 / BLKS;           // rows of a pass
        constexpr int PASSES = TK / RPP;
        const int c4 = tid & 3, blk = (tid >> 3) % BLKS, r_first = (tid >> 3) / BLKS * 2 + ((tid >> 2) & 1);
        const int page_mask = (1 << p.page_log2) - 1;
        struct Raw {
            uint4 v[PASSES];
            float ksc, vsc;
            uint32_t row;                        // this thread's token, in the scale arrays (caches of 2^32 rows fit no card)
            uint32_t none;                       // bit i: row i of this thread holds no token, bit 31: its scales
        };
        uint32_t pid = ~0u;                      // lane i: page of tokens 16 i .. of the next tile
        int tok0 = 0, there = 0, head = 0;       // its first token, rows that hold a token (0: no such tile)
        int t = w.t0;
        auto settle = [&]() {                    // to the next key tile there is
            while (more && t >= w.t1) {
                more = w.next(p, pl);
                t = w.t0;
            }
        };
        // pages are looked up a tile before their rows are read
        auto locate = [&]() {
            tok0 = t * TK;
            there = more ? min(w.it.rows.kv - tok0, TK) : 0;
            head = w.it.head;
            // (lanes past the last token look up the tile's first page)
            pid = more ? __ldg(p.table + (size_t)w.it.s * p.table_stride +
                               ((tok0 + (16 * lane < there ? 16 * lane : 0)) >> p.page_log2)) : 0;
        };
        // Every load has a place to read: one that is not due reads the
        // cache's first row, and its result is dropped.  (Under a condition
        // the compiler waits for each load before it issues the next.)
        auto fetch = [&](Raw& raw) {
            long long at = -1;                   // lane i: first row of tokens 16 i .. in the scale arrays
            if (16 * lane < there) {
                if (pid >= (uint32_t)p.n_pages) set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
                else at = (long long)page_row(p, (int)pid, head) + ((tok0 + 16 * lane) & page_mask);
            }
            const uint8_t* src = codes + blk * 64 + c4 * 16;
            raw.none = 0;
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const int r = r_first + i * RPP;
                const long long first = __shfl_sync(0xffffffffu, at, RPP >= 16 ? r >> 4 : i * RPP >> 4);
                const bool good = first >= 0 && r < there;
                raw.none |= good ? 0u : 1u << i;
                raw.v[i] = ldg_stream(reinterpret_cast<const uint4*>(src + (good ? (first + (r & 15)) * D : 0ll)));
            }
            const long long first = __shfl_sync(0xffffffffu, at, (tid & (TK - 1)) >> 4);
            const bool good = keys && first >= 0 && tid < there;
            raw.none |= good ? 0u : 1u << 31;
            raw.row = good ? (uint32_t)first + (tid & 15) : 0;
            raw.ksc = __ldg(p.ks + raw.row);
            raw.vsc = __ldg(p.vs + raw.row);
        };
        Raw cur;
        settle();
        bool have = more;                        // a tile is on its way to `cur`
        locate();
        fetch(cur);
        ++t;
        settle();
        locate();
        for (uint32_t n = 0; have; ++n) {
            Raw next;                            // (a copy, whose moves wait for the loads at the end of the pass)
            have = more;
            fetch(next);
            ++t;
            settle();
            locate();
            const int st = n & (NST - 1);
            const uint32_t ph = (n >> kStLog2) ^ 1;
            bool dead = !wait(&empty[st], ph) || (keys && !wait(&sc_free[n & 3], (n >> 2) ^ 1));
            dead = __any_sync(0xffffffffu, dead);
            if (dead) break;
            if (keys && tid < TK)
                token_scales<D, FMT>(p, !(cur.none >> 31), cur.row, cur.ksc, cur.vsc, ssc + (n & 3) * (C::kScaleBytes / 4), tid);
            if (cur.none << 1) {                 // codes behind the last token may be anything, a NaN code too
#pragma unroll
                for (int i = 0; i < PASSES; ++i)
                    if (cur.none >> i & 1) cur.v[i] = make_uint4(0, 0, 0, 0);
            }
            char* dst = ring + st * C::kOpBytes + blk * (TK * 128) + r_first * 128;
            const int o0 = ((2 * c4) ^ (r_first & 7)) << 4;     // (a pass is a multiple of eight rows)
#pragma unroll
            for (int i = 0; i < PASSES; ++i) {
                const uint32_t u[4] = {cur.v[i].x, cur.v[i].y, cur.v[i].z, cur.v[i].w};
                uint32_t h[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) codes_to_f16<FMT>(biased<FMT>(u[j]), h[2 * j], h[2 * j + 1]);
                char* d = dst + i * RPP * 128;
                *reinterpret_cast<uint4*>(d + o0) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(d + (o0 ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&full[st]);
                if (keys) mbar_arrive(&sc_full[n & 3]);
            }
            cur = next;
        }
    } else {
        // ------------------------------------------------------ issue
        {
            const uint32_t idesc_s = idesc_f16(128, TK, 0), idesc_o = idesc_f16(128, D, 0) | kTransposeB;
            const uint64_t q_desc = sdesc_k128(smem_u32(sq)), k_desc = sdesc_k128(smem_u32(sk)),
                           v_desc = sdesc_mn128(smem_u32(sv), TK * 128);
            const int q = warp - C::kMmaWarp;
            const uint32_t tS = tmem + NB * q * TK, tO = tmem + C::kColO + q * D;
            auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
            uint32_t n = 0, ns = 0, np = 0, items = 0;       // tiles of the CTA, scores and sums issued, items
            bool ok = true;
            auto score = [&](uint32_t k) {
                const int st = k & (NST - 1), b = ns & (NB - 1);
                ok = wait_all(&k_full[st], k >> kStLog2);
                if (!ok) return;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    mma_ss(tS + b * TK, q_desc + ((q * C::kQBytes + (i >> 2) * (128 * 128) + (i & 3) * 32) >> 4),
                           k_desc + ((st * C::kOpBytes + (i >> 2) * (TK * 128) + (i & 3) * 32) >> 4), idesc_s, i > 0);
                commit(&s_full[NB * q + b]);
                commit(&k_empty[st]);
                ++ns;
            };
            while (more && ok) {
                const int J = w.t1 - w.t0;
                if (q * 128 >= w.n_rows) {               // no rows: lets the stages go as they come
                    for (int j = 0; j < J && ok; ++j, ++n) {
                        const int st = n & (NST - 1);
                        ok = wait_all(&k_full[st], n >> kStLog2) && wait_all(&v_full[st], n >> kStLog2);
                        if (ok && lane == 0) {
                            mbar_arrive(&k_empty[st]);
                            mbar_arrive(&v_empty[st]);
                        }
                    }
                } else if (J > 0) {
                    ok = wait_all(&q_full[q], items++);
                    // scores run two tiles ahead of the sums.  Two buffers: those of tile j + 2 follow the sums of
                    // tile j, whose P their buffer held; four: they go before them
                    for (int j = -2; j < J && ok; ++j) {
                        const bool ahead = j + 2 < J;
                        const uint32_t k = n + (j < 0 ? j + 2 : 2);
                        if (ahead && (NB == 4 || j < 0)) score(k);
                        if (j < 0 || !ok) continue;
                        const int st = n & (NST - 1), b = np & (NB - 1);
                        ok = wait_all(&v_full[st], n >> kStLog2) && wait_all(&p_full[NB * q + b], np >> kBufLog2);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < TK / 16; ++i)
                            mma_ts(tO, tS + b * TK + i * 8, v_desc + ((st * C::kOpBytes + i * 2048) >> 4), idesc_o, j > 0 || i > 0);
                        commit(&o_done[NB * q + b]);
                        commit(&v_empty[st]);
                        ++np;
                        if (ahead && NB == 2) score(k);
                        ++n;
                    }
                }
                if (ok) more = w.next(p, pl);
            }
            // every MMA done before tensor memory is freed, even after an abort
            commit(final_bar);
            volatile int no_abort = 0;
            mbar_wait(final_bar, 0, &no_abort, kWaitLimit);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    if (warp == C::kMmaWarp) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) set_status(p.ctrl, LMOE_ERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// images
// ---------------------------------------------------------------------------

// Block (tile, head, sequence): the shared-memory image of a key tile -- keys
// and values as swizzled fp16 operands, then per token key scale times
// softmax scale, log2 and inverse of the value scale -- as the key and value
// warps above write it.
template <int D, int FMT>
__global__ void __launch_bounds__(256) k_attend_images(AttendParams p) {
    using C = Many<D, true>;
    constexpr int TK = C::TK, BLKS = D / 64, RPP = 64 / BLKS;      // rows of a pass
    sm100::grid_dep_launch();
    const SeqRows r = seq_rows(p, blockIdx.z);
    if (r.n <= 0) return;
    const int first = r.kv - r.n, lo = p.window ? (int)max(0ll, (long long)first - p.window + 1) : 0;
    const int tok0 = blockIdx.x * TK;
    if (tok0 >= r.kv || tok0 + TK <= lo) return;
    const int head = p.h0 + blockIdx.y;
    char* img = p.img + (((size_t)blockIdx.z * p.Hn + blockIdx.y) * p.img_tiles + blockIdx.x) * C::kImage;
    const int32_t* table = p.table + (size_t)blockIdx.z * p.table_stride;
    const int page_mask = (1 << p.page_log2) - 1;
    const int c4 = threadIdx.x & 3, blk = (threadIdx.x >> 3) % BLKS;
    const int r_first = (threadIdx.x >> 3) / BLKS * 2 + ((threadIdx.x >> 2) & 1);
    auto place = [&](int tok) -> long long {                       // row in the scale arrays; -1: none
        if (tok >= r.kv) return -1;
        const int page = __ldg(table + (tok >> p.page_log2));
        if (page < 0 || page >= p.n_pages) {
            set_status(p.ctrl, LMOE_ERR_DEVICE_CHECK);
            return -1;
        }
        return (long long)page_row(p, page, head) + (tok & page_mask);
    };
#pragma unroll
    for (int i = 0; i < TK / RPP; ++i) {
        const int row = r_first + i * RPP;
        const long long at = place(tok0 + row);
        uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (at >= 0) {
            raw[0] = ldg_stream(reinterpret_cast<const uint4*>(p.k + at * D + blk * 64 + c4 * 16));
            raw[1] = ldg_stream(reinterpret_cast<const uint4*>(p.v + at * D + blk * 64 + c4 * 16));
        }
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const uint32_t u[4] = {raw[o].x, raw[o].y, raw[o].z, raw[o].w};
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) codes_to_f16<FMT>(biased<FMT>(u[j]), h[2 * j], h[2 * j + 1]);
            char* d = img + o * C::kOpBytes + blk * (TK * 128) + row * 128;
            const int o0 = ((2 * c4) ^ (row & 7)) << 4;
            *reinterpret_cast<uint4*>(d + o0) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(d + (o0 ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
    }
    if (threadIdx.x < TK) {
        const long long at = place(tok0 + threadIdx.x);
        token_scales<D, FMT>(p, at >= 0, (size_t)at, at >= 0 ? __ldg(p.ks + at) : 0.f, at >= 0 ? __ldg(p.vs + at) : 0.f,
                             reinterpret_cast<float*>(img + 2 * C::kOpBytes), threadIdx.x);
    }
}

template <int D, int FMT, bool IMG>
cudaError_t launch(const AttendParams& p, cudaStream_t st) {
    using C = Many<D, IMG>;
    static_assert(C::kRows == many_rows(D) && C::kImage == image_bytes(D) && C::TK == image_tokens(D), "sizes");
    const Plan pl{C::kRows, 6, 1, kExtra};
    cudaError_t e = allow_smem<k_attend_many<D, FMT, IMG>>(C::kSmem);
    if (e != cudaSuccess) return e;
    // over the images' kernel: it starts while that one runs, and its loaders wait for it
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kSms);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = a;
    cfg.numAttrs = IMG ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, k_attend_many<D, FMT, IMG>, p, pl);
    if (e != cudaSuccess) return e;
    return launch_join(p, C::kRows, kSms, false, st);
}

// Images pay where several row tiles read a key tile, and go in groups of
// sequences, or of heads of one sequence, that fit the workspace (and L2).  A
// sequence that may be too long for them, even one head of it, is converted
// on the way.  The lengths are on the device, so this goes by the page table's
// width: 248,512 tokens for head_dim 64, 127,552 for 128, 64,640 for 256.
template <int D, int FMT>
cudaError_t launch_groups(AttendParams p, cudaStream_t st) {
    const long long tiles = (((long long)p.table_stride << p.page_log2) + image_tokens(D) - 1) / image_tokens(D);
    const long long fit = (long long)(kImageBytes / image_bytes(D)) / tiles;      // (sequence, head) pairs of a group
    const long long rows = (long long)p.max_new * p.G;
    const bool brief = rows > many_rows(D) && tiles * image_tokens(D) <= kImageTokens && (long long)p.n_seqs * p.Hk <= fit;
    if (fit < 1 || (rows <= kImageRowTiles * many_rows(D) && !brief)) return launch<D, FMT, false>(p, st);
    const int heads = (int)(fit < p.Hk ? fit : p.Hk);
    const int seqs = (int)(fit / heads < p.n_seqs ? fit / heads : p.n_seqs);
    AttendParams g = p;
    g.img_tiles = (int)tiles;
    for (int s = 0; s < p.n_seqs; s += seqs) {
        g.n_seqs = p.n_seqs - s < seqs ? p.n_seqs - s : seqs;
        g.q_start = p.q_start + s;
        g.kv_len = p.kv_len + s;
        g.table = p.table + (size_t)s * p.table_stride;
        for (int h = 0; h < p.Hk; h += heads) {
            g.h0 = h;
            g.Hn = p.Hk - h < heads ? p.Hk - h : heads;
            // (a grid's y and z end at 65535; fit is far below)
            k_attend_images<D, FMT><<<dim3((unsigned)tiles, g.Hn, g.n_seqs), 256, 0, st>>>(g);
            cudaError_t e = cudaGetLastError();
            if (e == cudaSuccess) e = launch<D, FMT, true>(g, st);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t attend::launch_many(const AttendParams& p, cudaStream_t st) {
    const bool i8 = p.fmt == LMOE_KV_INT8;
    if (p.D == 64) return i8 ? launch_groups<64, LMOE_KV_INT8>(p, st) : launch_groups<64, LMOE_KV_E4M3>(p, st);
    if (p.D == 128) return i8 ? launch_groups<128, LMOE_KV_INT8>(p, st) : launch_groups<128, LMOE_KV_E4M3>(p, st);
    return i8 ? launch_groups<256, LMOE_KV_INT8>(p, st) : launch_groups<256, LMOE_KV_E4M3>(p, st);
}

}  // namespace lmoe
