// Attention over the 8-bit paged cache, many query rows per key head: prompt
// chunks.
//
// The mathematics is that of the kernel for few rows (lmoe_attend.cu); the
// products run on tcgen05 (kind::f16, fp32 accumulators in tensor memory).
// What bounds it: the tensor cores (4 D flops per row and key) and, close
// behind, the exponentials (one per row and key, 16 a cycle and SM).
//
// A CTA (one per SM) holds query tiles of 128 rows as fp16 in shared memory
// (two for head_dim 64 and 128, one for 256) and walks the keys in tiles of
// 64 tokens:
//   softmax      eight warps: a thread has a row of each query tile and half of
//                the columns; S comes from tensor memory, P goes back over it
//                as the A operand.  (Two rows a thread share the loads of the
//                tokens' constants: shared memory, which feeds the tensor core
//                as well, is what runs out first.)
//   keys, values four warps each read the codes of a tile (registers, one tile
//                ahead) and write them as fp16 operands with the 128-byte
//                swizzle; a key row is K-major as it is stored, and the same
//                layout read as MN-major is the value operand, so neither is
//                transposed.
//   issue        one thread: S = Q K^T and O += P V
// Two score buffers per query tile let the next S run ahead of the softmax.  The row's
// reference m is raised as in the kernel for few rows, and to a whole number,
// so that what it rescales (O, and the P of the tile's earlier pieces)
// changes by a power of two: the scores are gone
// through once, and the loop stays small enough for the instruction caches
// (a form that held a tile's scores in registers, unrolled, spent a third of
// its time waiting for instructions).
//
// Work is cut into equal pieces of the line of (item, key tile) units as in
// the kernel for few rows, one piece per CTA; cut items are joined after it.

#include "lmoe_attend.cuh"
#include "lmoe_sm100.cuh"

namespace lmoe {

namespace {

using namespace sm100;
using namespace attend;

constexpr int kExtra = 4;                        // loading the queries and writing the sums, in key tiles
constexpr uint64_t kWaitLimit = 4000000000ull;   // SM cycles per barrier wait (about 2 s)
constexpr uint64_t kDrainLimit = 20000000ull;    // and per wait for a copy in flight after one gave up

template <int D, bool IMG>
struct Many {
    static constexpr int NQ = D == 256 ? 1 : 2;       // query tiles of 128 rows
    static constexpr int TK = 64;                     // tokens of a key tile
    static constexpr int NST = D == 256 ? 2 : 4;      // stages of keys, and of values
    static constexpr int kRows = NQ * 128;
    static constexpr int kKeyWarp = 8, kValueWarp = kKeyWarp + (IMG ? 1 : 4),
                         kMmaWarp = kValueWarp + (IMG ? 0 : 4);
    static constexpr int kThreads = (kMmaWarp + 1) * 32;
    static constexpr size_t kQBytes = 128 * D * 2;    // one query tile
    static constexpr size_t kOpBytes = TK * D * 2;    // one stage of keys or values
    static constexpr size_t kScaleBytes = 3 * TK * 4; // per token: key scale, log2 and inverse of the value scale
    static constexpr size_t kImage = 2 * kOpBytes + kScaleBytes;   // keys, values, scales of a tile
    static constexpr size_t kSmem = 1024 + NQ * kQBytes + 2 * NST * kOpBytes + 4 * kScaleBytes + 512;
    static constexpr uint32_t kColO = 256;            // tensor memory: scores from 0 ((2 q + b) * TK), sums from 256 (q * D)
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
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Contiguous bytes (16-byte aligned, a multiple of 16) to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

// Pairs of fp32 in one instruction.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// What the softmax needs of a token.  A place without one weighs nothing; a
// value scale that is no positive number makes its token's scores NaN.
__device__ __forceinline__ void token_scales(const AttendParams& p, bool some, float ks, float vs, float* sc, int TK) {
    const bool fine = vs > 0.f && vs < INFINITY;
    sc[0] = some ? ks * p.scale_log2 : 0.f;
    sc[TK] = !some ? -INFINITY : fine ? __log2f(vs) : __int_as_float(0x7fffffff);
    sc[2 * TK] = some && fine ? __frcp_rn(vs) : 1.f;
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
    constexpr int CW = TK / 2;                   // columns of a softmax warp
    constexpr int PW = IMG ? CW : 16;            // columns of a piece (registers: 168 a thread, or 96)
    __shared__ float s_row[2][2][NQ][128];       // exchange between the two warps of a row
    __shared__ float s_scale[NQ][128];
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
    uint64_t* sc_free = bars + 16;   // [4] scales of a stage read (8 warps)
    uint64_t* s_full = bars + 20;    // [b] scores of a buffer done (commit)
    uint64_t* p_full = bars + 22;    // [b] probabilities written (8 warps)
    uint64_t* o_done = bars + 24;    // sums updated (commit)
    uint64_t* q_full = bars + 25;    // query tiles written (8 warps)
    uint64_t* sc_full = bars + 32;   // [4] scales of a stage written
    uint64_t* pair = bars + 36;      // [4] the two warps of a row
    uint64_t* final_bar = bars + 40;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 41);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&k_full[i], IMG ? 1 : 4);
            mbar_init(&v_full[i], IMG ? 1 : 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&sc_full[i], IMG ? 1 : 4);
            mbar_init(&sc_free[i], 8);
            mbar_init(&pair[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 8);
        }
        mbar_init(o_done, 1);
        mbar_init(q_full, 8);
        mbar_init(final_bar, 1);
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
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        const uint32_t tO = tmem + lanes + C::kColO;
        uint32_t n = 0;              // key tiles of the CTA
        uint32_t met = 0;            // meetings of the two warps of a row
        bool dead = false;
        auto meet = [&]() {          // false: given up
            __syncwarp();
            if (lane == 0) mbar_arrive(&pair[quad]);
            const bool ok = wait(&pair[quad], met++);
            return !__any_sync(0xffffffffu, !ok);
        };
        // 16 bytes of a row of a query tile's place (fp16 queries, later bf16 sums)
        auto place = [&](int q, int rw, int ch) {
            return reinterpret_cast<uint4*>(sq + q * C::kQBytes + (32 * quad + rw) * 128 + (ch >> 3) * (128 * 128) +
                                            (((ch & 7) ^ (rw & 7)) << 4));
        };
        while (more && !dead) {
            const int nq = w.n_rows > 128 ? NQ : 1;      // query tiles with rows
            const int row0 = w.it.rt * C::kRows;
            float m[NQ], l[NQ];
            f2 m2[NQ];               // -m twice; 0 while m is -infinity
            int pos[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                m[q] = -INFINITY;
                l[q] = 0.f;
                m2[q] = 0ull;
                pos[q] = w.it.rows.kv - w.it.rows.n + (row0 + q * 128 + row) / p.G;
            }
            const bool some = w.t0 < w.t1;
            if (some) {
                dead = !meet();      // both have stored the last item's sums from the tiles' places
                if (dead) break;
                // rows as fp16, each scaled by a power of two (past the last
                // row: a copy of it, so that no load is conditional); the two
                // warps take a tile each, or every other pass
                constexpr int LPR = D / 8, RPL = 32 / LPR;       // lanes of a row, rows of a pass
                const int qt = NQ == 2 ? half : 0;
#pragma unroll 4
                for (int i = NQ == 2 ? 0 : half; i < LPR; i += 3 - NQ) {
                    const int rw = i * RPL + lane / LPR, ch = lane % LPR;
                    const int id = row0 + min(qt * 128 + 32 * quad + rw, w.n_rows - 1);
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                                              p.q + (size_t)(w.it.rows.q0 + id / p.G) * p.q_stride +
                                              (size_t)(w.it.head * p.G + id % p.G) * D) + ch);
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    uint32_t mb = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) mb = max(mb, max(u[j] & 0x7fffu, (u[j] >> 16) & 0x7fffu));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
                    const bool bad = mb >= 0x7f80u;
                    const int e = min(max((int)(mb >> 7) - 127, -100), 126);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    if (ch == 0)
                        s_scale[qt][32 * quad + rw] =
                            bad ? __int_as_float(0x7fffffff) : __uint_as_float((uint32_t)(127 + e) << 23);
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = bf16x2_to_f32x2(u[j]);
                        const __half2 hh = __floats2half2_rn(f.x * down, f.y * down);
                        h[j] = bad ? 0u : *reinterpret_cast<const uint32_t*>(&hh);
                    }
                    *place(qt, rw, ch) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
                dead = !meet();
                if (dead) break;
                f2 scale2[NQ];
#pragma unroll
                for (int q = 0; q < NQ; ++q) scale2[q] = pack2(s_scale[q][row], s_scale[q][row]);

                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const int st = n & 3, b = n & 1;
                    dead = !wait(&sc_full[st], n >> 2) || !wait(&s_full[b], n >> 1);
                    dead = __any_sync(0xffffffffu, dead);
                    if (dead) break;
                    tc_fence_after();
                    __syncwarp();
                    const uint32_t tS = tmem + lanes + b * TK;       // (query tile q: 2 q TK on)
                    const float4* ks = reinterpret_cast<const float4*>(ssc + st * (C::kScaleBytes / 4) + half * CW);
                    const int tok0 = t * TK + half * CW;
                    // keys a row sees: columns lo .. hi - 1
                    int hi[NQ], lo[NQ];
                    bool edge = false;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        hi[q] = p.causal ? pos[q] + 1 - tok0 : CW;
                        lo[q] = p.window ? pos[q] + 1 - p.window - tok0 : 0;
                        edge |= hi[q] < CW || lo[q] > 0;
                    }
                    const bool mask = __any_sync(0xffffffffu, edge);
                    f2 l2[NQ];
#pragma unroll
                    for (int q = 0; q < NQ; ++q) l2[q] = pack2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < CW / PW; ++c, ks += PW / 4) {
                        uint32_t x[NQ][PW];
#pragma unroll
                        for (int q = 0; q < NQ; ++q)
#pragma unroll
                            for (int i = 0; i < PW / 16; ++i)
                                tmem_ld_32x32b_x16(tS + 2 * q * TK + half * CW + PW * c + 16 * i,
                                                   *reinterpret_cast<uint32_t(*)[16]>(x[q] + 16 * i));
                        tmem_ld_wait();
                        float top[NQ];
#pragma unroll
                        for (int q = 0; q < NQ; ++q) top[q] = -INFINITY;
                        // the tokens' constants come from shared memory, whose
                        // bandwidth the tensor core's operands need most of:
                        // one load serves both query tiles
#pragma unroll
                        for (int i = 0; i < PW / 4; ++i) {
                            const float4 k4 = ks[i], b4 = ks[TK / 4 + i];
#pragma unroll
                            for (int q = 0; q < NQ; ++q) {
                                uint32_t* y = x[q] + 4 * i;
                                const float2 z0 = unpack2(fma2(mul2(pack2(__uint_as_float(y[0]), __uint_as_float(y[1])), pack2(k4.x, k4.y)), scale2[q], pack2(b4.x, b4.y)));
                                const float2 z1 = unpack2(fma2(mul2(pack2(__uint_as_float(y[2]), __uint_as_float(y[3])), pack2(k4.z, k4.w)), scale2[q], pack2(b4.z, b4.w)));
                                y[0] = __float_as_uint(z0.x);
                                y[1] = __float_as_uint(z0.y);
                                y[2] = __float_as_uint(z1.x);
                                y[3] = __float_as_uint(z1.y);
                            }
                        }
                        if (mask) {
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
#pragma unroll
                                for (int i = 0; i < PW; ++i)
                                    if (i < lo[q] - PW * c || i >= hi[q] - PW * c) x[q][i] = 0xff800000u;
                        }
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
#pragma unroll
                            for (int i = 0; i < PW; i += 2)
                                top[q] = fmaxf(fmaxf(top[q], __uint_as_float(x[q][i])), __uint_as_float(x[q][i + 1]));
                            s_row[met & 1][half][q][row] = top[q];
                        }
                        const int slot = met & 1;
                        dead = !meet();
                        if (dead) break;
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            top[q] = fmaxf(top[q], s_row[slot][half ^ 1][q][row]);
                            if (!__any_sync(0xffffffffu, top[q] > m[q] + kMaxP) || q >= nq) continue;
                            const float mn = fmaxf(m[q], ceilf(top[q]) - kRaiseP);
                            const float f = m[q] == mn ? 1.f : ex2(m[q] - mn);
                            m[q] = mn;
                            m2[q] = mn == -INFINITY ? 0ull : pack2(-mn, -mn);
                            l[q] *= f;
                            l2[q] = mul2(l2[q], pack2(f, f));
                            if (t > w.t0) {       // the sums of the earlier tiles are in tensor memory
                                dead = !wait(o_done, n - 1);
                                dead = __any_sync(0xffffffffu, dead);
                                if (dead) break;
                                tc_fence_after();
                                __syncwarp();
#pragma unroll 1
                                for (int d = half * (D / 32); d < (half + 1) * (D / 32); ++d) {
                                    uint32_t o[16];
                                    tmem_ld_32x32b_x16(tO + q * D + 16 * d, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                    tmem_st_32x32b_x16(tO + q * D + 16 * d, o);
                                }
                            }
                            const __half2 fh = __float2half2_rn(f);
#pragma unroll 1
                            for (int d = 0; d < c * (PW / 16); ++d) {      // P of the earlier pieces
                                const uint32_t at = tS + 2 * q * TK + half * CW + 8 * d;
                                uint32_t o[8];
                                tmem_ld_32x32b_x8(at, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&o[i]), fh);
                                    o[i] = *reinterpret_cast<const uint32_t*>(&h);
                                }
                                tmem_st_32x32b_x8(at, o);
                            }
                        }
                        if (dead) break;
#pragma unroll
                        for (int g = 0; g < PW / 16; ++g) {
                            uint32_t ph[NQ][8];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 i4 = ks[TK / 2 + 4 * g + i];
#pragma unroll
                                for (int q = 0; q < NQ; ++q) {
                                    const uint32_t* y = x[q] + 16 * g + 4 * i;
                                    const float2 y0 = unpack2(add2(pack2(__uint_as_float(y[0]), __uint_as_float(y[1])), m2[q]));
                                    const float2 y1 = unpack2(add2(pack2(__uint_as_float(y[2]), __uint_as_float(y[3])), m2[q]));
                                    const float p0 = ex2(y0.x), p1 = ex2(y0.y), p2 = ex2(y1.x), p3 = ex2(y1.y);
                                    l2[q] = fma2(pack2(p0, p1), pack2(i4.x, i4.y), l2[q]);
                                    l2[q] = fma2(pack2(p2, p3), pack2(i4.z, i4.w), l2[q]);
                                    const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
                                    ph[q][2 * i] = *reinterpret_cast<const uint32_t*>(&h0);
                                    ph[q][2 * i + 1] = *reinterpret_cast<const uint32_t*>(&h1);
                                }
                            }
#pragma unroll
                            for (int q = 0; q < NQ; ++q)
                                tmem_st_32x32b_x8(tS + 2 * q * TK + half * CW + 8 * (c * (PW / 16) + g), ph[q]);
                        }
                    }
                    if (dead) break;
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        const float2 ls = unpack2(l2[q]);
                        l[q] += ls.x + ls.y;
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&p_full[b]);
                        mbar_arrive(&sc_free[st]);
                    }
                }
                if (dead) break;
                const int slot = met & 1;
#pragma unroll
                for (int q = 0; q < NQ; ++q) s_row[slot][half][q][row] = l[q];
                dead = !meet();
                if (dead) break;
#pragma unroll
                for (int q = 0; q < NQ; ++q) l[q] += s_row[slot][half ^ 1][q][row];
                dead = !wait(o_done, n - 1);
                dead = __any_sync(0xffffffffu, dead);
                if (dead) break;
                tc_fence_after();
                __syncwarp();
            }
            // sums out: a warp has half of a row's columns
            const bool cut = w.u0 > 0 || w.u1 < w.it.tile.units;
            float* part = p.part + ((size_t)blockIdx.x * 2 + (w.u0 == 0 ? 1 : 0)) * part_floats(C::kRows, D);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const int r = q * 128 + row, last = w.n_rows - 1 - q * 128 - 32 * quad;    // the warp's last row
                const bool live = r < w.n_rows;
                if (last < 0) continue;
                const float inv = cut ? 1.f : l[q] == 0.f ? 0.f : 1.f / l[q];
#pragma unroll 1
                for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
                    uint32_t o[32];
                    if (some) {
                        tmem_ld_32x32b_x32(tO + q * D + 32 * c, o);
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
                            for (int j = 0; j < 4; ++j)
                                h[j] = (uint32_t)f32_to_bf16_bits(__uint_as_float(o[8 * i + 2 * j]) * inv) |
                                       (uint32_t)f32_to_bf16_bits(__uint_as_float(o[8 * i + 2 * j + 1]) * inv) << 16;
                            *place(q, lane, 4 * c + i) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                    __syncwarp();
                }
                if (!cut) {
                    constexpr int LPR = D / 16, RPL = 32 / LPR;
#pragma unroll 4
                    for (int i = 0; i < LPR; ++i) {
                        const int rw = min(i * RPL + lane / LPR, last), ch = half * LPR + lane % LPR;   // (the last row: repeated)
                        const int id = row0 + q * 128 + 32 * quad + rw;
                        const size_t at = (size_t)(w.it.rows.q0 + id / p.G) * p.Hq + w.it.head * p.G + id % p.G;
                        *(reinterpret_cast<uint4*>(p.out + at * D) + ch) = *place(q, rw, ch);
                    }
                    __syncwarp();
                }
                if (live && half == 0) {
                    const int id = row0 + r;
                    if (cut) {
                        part[(size_t)C::kRows * D + r] = m[q];
                        part[(size_t)C::kRows * (D + 1) + r] = l[q];
                    } else if (p.lse) {
                        p.lse[(size_t)(w.it.rows.q0 + id / p.G) * p.Hq + w.it.head * p.G + id % p.G] =
                            l[q] == 0.f ? -INFINITY : (m[q] + log2f(l[q])) * 0.6931471805599453f;
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
            uint32_t n = 0;
            bool dead = false;
            int half = 0;                        // of tile n on their way: 1 the keys, 2 the scales too
            while (more && !dead) {
                const char* img = p.img + ((size_t)w.it.s * p.Hn + (w.it.head - p.h0)) * p.img_tiles * C::kImage;
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    const char* src = img + (size_t)t * C::kImage;
                    const int st = n & (NST - 1);
                    const uint32_t ph = (n >> kStLog2) ^ 1;
                    dead = !wait(&k_empty[st], ph);
                    if (dead) break;
                    mbar_arrive_expect_tx(&k_full[st], (uint32_t)C::kOpBytes);
                    bulk_load(sk + st * C::kOpBytes, src, (uint32_t)C::kOpBytes, &k_full[st]);
                    half = 1;
                    dead = !wait(&sc_free[n & 3], (n >> 2) ^ 1);
                    if (dead) break;
                    mbar_arrive_expect_tx(&sc_full[n & 3], (uint32_t)C::kScaleBytes);
                    bulk_load(ssc + (n & 3) * (C::kScaleBytes / 4), src + 2 * C::kOpBytes, (uint32_t)C::kScaleBytes, &sc_full[n & 3]);
                    half = 2;
                    dead = !wait(&v_empty[st], ph);
                    if (dead) break;
                    half = 0;
                    mbar_arrive_expect_tx(&v_full[st], (uint32_t)C::kOpBytes);
                    bulk_load(sv + st * C::kOpBytes, src + C::kOpBytes, (uint32_t)C::kOpBytes, &v_full[st]);
                }
                if (!dead) more = w.next(p, pl);
            }
            // the copies in flight end before the CTA does, after an abort too
            volatile int no_abort = 0;
            for (uint32_t i = n > NST ? n - NST : 0; i < n; ++i) {
                mbar_wait(&k_full[i & (NST - 1)], (i >> kStLog2) & 1, &no_abort, kDrainLimit);
                mbar_wait(&v_full[i & (NST - 1)], (i >> kStLog2) & 1, &no_abort, kDrainLimit);
                mbar_wait(&sc_full[i & 3], (i >> 2) & 1, &no_abort, kDrainLimit);
            }
            if (half > 0) mbar_wait(&k_full[n & (NST - 1)], (n >> kStLog2) & 1, &no_abort, kDrainLimit);
            if (half > 1) mbar_wait(&sc_full[n & 3], (n >> 2) & 1, &no_abort, kDrainLimit);
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
            raw.ksc = __ldg(p.ks + (good ? first + (tid & 15) : 0ll));
            raw.vsc = __ldg(p.vs + (good ? first + (tid & 15) : 0ll));
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
                token_scales(p, !(cur.none >> 31), cur.ksc, cur.vsc, ssc + (n & 3) * (C::kScaleBytes / 4) + tid, TK);
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
            auto scores = [&](int q, int b, int st) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_ss(tmem + (2 * q + b) * TK, q_desc + ((q * C::kQBytes + (k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                           k_desc + ((st * C::kOpBytes + (k >> 2) * (TK * 128) + (k & 3) * 32) >> 4), idesc_s, k > 0);
            };
            // (each half's P lies over its own scores)
            auto sums = [&](int q, int b, int st, bool first) {
#pragma unroll
                for (int k = 0; k < TK / 16; ++k)
                    mma_ts(tmem + C::kColO + q * D, tmem + (2 * q + b) * TK + (k >> 1) * (TK / 2) + (k & 1) * 8,
                           v_desc + ((st * C::kOpBytes + k * 2048) >> 4), idesc_o, !first || k > 0);
            };
            auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
            uint32_t n = 0, items = 0;
            bool ok = true, issued = false;
            while (more && ok) {
                const int J = w.t1 - w.t0, nq = w.n_rows > 128 ? NQ : 1;
                if (J > 0) {
                    ok = wait_all(q_full, items++);
                    // scores run two tiles ahead of the sums: those of tile j + 2 follow the sums of tile j, whose P
                    // their buffer held, and are done while the softmax works on tile j + 1
                    for (int j = -2; j < J && ok; ++j) {
                        if (j >= 0) {
                            const int st = n & (NST - 1);
                            ok = wait_all(&v_full[st], n >> kStLog2) && wait_all(&p_full[n & 1], n >> 1);
                            if (!ok) break;
                            tc_fence_after();
                            sums(0, n & 1, st, j == 0);
                            if (nq == 2) sums(NQ - 1, n & 1, st, j == 0);
                            commit(o_done);
                            commit(&v_empty[st]);
                        }
                        if (j + 2 < J) {
                            const uint32_t k = n + (j < 0 ? j + 2 : 2);
                            const int st = k & (NST - 1);
                            ok = wait_all(&k_full[st], k >> kStLog2);
                            if (!ok) break;
                            tc_fence_after();
                            issued = true;
                            scores(0, k & 1, st);
                            if (nq == 2) scores(NQ - 1, k & 1, st);
                            commit(&s_full[k & 1]);
                            commit(&k_empty[st]);
                        }
                        if (j >= 0) ++n;
                    }
                }
                if (ok) more = w.next(p, pl);
            }
            if (issued) {
                // every MMA done before tensor memory is freed, even after an abort
                commit(final_bar);
                volatile int no_abort = 0;
                mbar_wait(final_bar, 0, &no_abort, kWaitLimit);
            }
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
    const SeqRows r = seq_rows(p, blockIdx.z);
    if (r.n <= 0) return;
    const int first = r.kv - r.n, lo = p.window ? max(0, first - p.window + 1) : 0;
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
        token_scales(p, at >= 0, at >= 0 ? __ldg(p.ks + at) : 0.f, at >= 0 ? __ldg(p.vs + at) : 0.f,
                     reinterpret_cast<float*>(img + 2 * C::kOpBytes) + threadIdx.x, TK);
    }
}

template <int D, int FMT, bool IMG>
cudaError_t launch(const AttendParams& p, cudaStream_t st) {
    using C = Many<D, IMG>;
    static_assert(C::kRows == many_rows(D) && C::kImage == image_bytes(D) && C::TK == image_tokens(D), "sizes");
    const Plan pl{C::kRows, 6, 1, kExtra};
    cudaError_t e = allow_smem<k_attend_many<D, FMT, IMG>>(C::kSmem);
    if (e != cudaSuccess) return e;
    k_attend_many<D, FMT, IMG><<<kSms, C::kThreads, C::kSmem, st>>>(p, pl);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_join(p, C::kRows, kSms, false, st);
}

// Images pay where several row tiles read a key tile, and go in groups of
// sequences, or of heads of one sequence, that fit the workspace (and L2).  A
// sequence that may be too long for them, even one head of it, is converted
// on the way.
template <int D, int FMT>
cudaError_t launch_groups(AttendParams p, cudaStream_t st) {
    const long long tiles = (((long long)p.table_stride << p.page_log2) + image_tokens(D) - 1) / image_tokens(D);
    const long long fit = (long long)(kImageBytes / image_bytes(D)) / tiles;      // (sequence, head) pairs of a group
    if ((long long)p.max_new * p.G <= kImageRowTiles * many_rows(D) || fit < 1) return launch<D, FMT, false>(p, st);
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
