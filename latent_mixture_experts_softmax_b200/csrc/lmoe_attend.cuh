// Attention over the 8-bit paged cache: what the kernel for few query rows,
// the kernel for many and the joining of cut items share -- the line of work
// units, the parts of cut items and the decoding of codes.
#pragma once

#include "lmoe_mixers.cuh"

namespace lmoe {
namespace attend {

constexpr int kMaxCtas = 2 * kSms;
// Probabilities are p = 2^(t - m): m is raised when a t passes it by kMaxP, to
// kRaiseP below the largest t.  P fits fp16 (2^16) with room, most key tiles
// leave m as it is, and a p as small as 2^-126 still counts in the sum of a
// row whose values' scales differ by 2^120.
constexpr float kMaxP = 15.75f, kRaiseP = 6.f;
// Sums of exponentials are kept as l = sum p kSumUnit / b over the value scales
// b.  The cache stores rows of 2^-100 to 2^128, b from 2^-109 to 2^121; with p up
// to 2^16, 2^18 keys of the smallest scale stay below 2^127, and the unit over
// a scale keeps its 24 bits up to b = 2^109 (12 at the largest).
constexpr float kSumUnit = 0x1p-17f;
// Value rows of zeros (scale 0, or codes of zeros under the scale 1 that the
// cache stores with them) have no size, so their scale says nothing about the
// reference: left in t, one of them among rows of 1e-8 pushed the others'
// probabilities out of fp16.  They stay out of the products, and enter the sum
// as 2^(s - m) with the bare score s in fp32, which has room for s far above m
// (2^18 keys at kMaxP + kZeroDrop, in kSumUnit: 2^123).  Towards m they count as
// t = s - kZeroDrop.
constexpr float kZeroDrop = 106.f;
constexpr int kFewRows = 32;            // query rows of an item of the kernel for few rows, at most

// ---------------------------------------------------------------------------
// the line of work units
// ---------------------------------------------------------------------------

struct Plan {
    int rows;          // query rows of a row tile
    int step_log2;     // tokens of a step
    int groups;        // steps of a unit
    int extra;         // units of a row tile besides those of its steps
};

struct Tile {
    int step0, step1;  // steps the row tile reads
    int units;         // at least one, so that empty tiles are written too
};

__device__ __forceinline__ Tile tile_of(const AttendParams& p, const Plan& pl, const SeqRows& s, int rt) {
    const int r0 = rt * pl.rows, r1 = min(r0 + pl.rows, s.n * p.G);
    const int first = s.kv - s.n;
    int lo = 0, hi = s.kv;
    if (p.causal) {
        hi = min(hi, first + (r1 - 1) / p.G + 1);
        if (p.window) lo = (int)max(0ll, (long long)first + r0 / p.G - p.window + 1);
    }
    hi = max(hi, lo);
    Tile t;
    t.step0 = lo >> pl.step_log2;
    t.step1 = hi > lo ? ((hi - 1) >> pl.step_log2) + 1 : t.step0;
    t.units = max(1, (t.step1 - t.step0 + pl.groups - 1) / pl.groups) + pl.extra;
    return t;
}

__device__ __forceinline__ int n_row_tiles(const AttendParams& p, const Plan& pl, const SeqRows& s) {
    return s.n <= 0 ? 0 : (int)(((long long)s.n * p.G + pl.rows - 1) / pl.rows);
}

// Units of one head of a sequence, all lanes of a warp together.
__device__ __forceinline__ long long head_units(const AttendParams& p, const Plan& pl, const SeqRows& s) {
    long long u = 0;
    for (int rt = threadIdx.x & 31, n = n_row_tiles(p, pl, s); rt < n; rt += 32) u += tile_of(p, pl, s, rt).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}

// The same for each lane's own sequence (s >= n_seqs: 0).
__device__ __forceinline__ long long lane_units(const AttendParams& p, const Plan& pl, int s) {
    SeqRows r{0, -1, 0};
    if (s < p.n_seqs) r = seq_rows(p, s);
    const int n = n_row_tiles(p, pl, r);
    long long u = 0;
    if (n <= 2)
        for (int rt = 0; rt < n; ++rt) u += tile_of(p, pl, r, rt).units;
    for (unsigned todo = __ballot_sync(0xffffffffu, n > 2); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
        const SeqRows o{__shfl_sync(0xffffffffu, r.q0, from), __shfl_sync(0xffffffffu, r.n, from),
                        __shfl_sync(0xffffffffu, r.kv, from)};
        const long long v = head_units(p, pl, o);
        if ((threadIdx.x & 31) == from) u = v;
    }
    return u;
}

struct Line {
    long long total, chunk;   // units, and units per CTA
    int seq;                  // the sequence holding unit x, its first unit, and the units of a head of it
    long long base, per_head;
};

// Where unit x of the line lies: the CTA sums every sequence's units, a run
// of sequences per thread.  x(total) gives the unit wanted once the total is
// known; at or past the end: seq = n_seqs.
template <class F>
__device__ Line find_unit(const AttendParams& p, const Plan& pl, int n_ctas, F x_of) {
    __shared__ long long s_sum[32];
    __shared__ long long s_base, s_head;
    __shared__ int s_seq;
    const int nt = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.n_seqs + nt - 1) / nt;
    const int a = (int)min((long long)p.n_seqs, (long long)threadIdx.x * per), b = min(p.n_seqs, a + per);
    long long mine = 0, first = 0;
    for (int i = 0; i < per; ++i) {
        const long long u = lane_units(p, pl, a + i < b ? a + i : p.n_seqs);
        if (i == 0) first = u;
        mine += u * p.Hn;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_sum[warp] = inc;
    if (threadIdx.x == 0) { s_seq = p.n_seqs; s_base = s_head = 0; }
    __syncthreads();
    Line l;
    l.total = 0;
    long long before = inc - mine;
    for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += s_sum[w];
        l.total += s_sum[w];
    }
    l.chunk = max(1ll, (l.total + n_ctas - 1) / n_ctas);
    const long long x = x_of(l);
    if (__any_sync(0xffffffffu, x >= before && x < before + mine)) {
        for (int i = 0; i < per; ++i) {
            const long long u = i == 0 ? first : lane_units(p, pl, a + i < b ? a + i : p.n_seqs);
            if (x >= before && x < before + u * p.Hn) {
                s_seq = a + i;
                s_base = before;
                s_head = u;
            }
            before += u * p.Hn;
        }
    }
    __syncthreads();
    l.seq = s_seq;
    l.base = s_base;
    l.per_head = s_head;
    return l;
}

// One item of the line, and how to go on to the next.
struct Item {
    int s, head, rt;
    SeqRows rows;
    Tile tile;
    long long begin;          // first unit

    __device__ void load(const AttendParams& p, const Plan& pl) { tile = tile_of(p, pl, rows, rt); }
    // The item of the line that holds unit x (all lanes of a warp together).
    __device__ bool seek(const AttendParams& p, const Plan& pl, const Line& l, long long x) {
        s = l.seq;
        if (s >= p.n_seqs) return false;
        rows = seq_rows(p, s);
        const int h = (int)((x - l.base) / l.per_head);
        head = p.h0 + h;
        begin = l.base + h * l.per_head;
        const int n = n_row_tiles(p, pl, rows), lane = threadIdx.x & 31;
        for (rt = 0;; rt += 32) {
            const long long u = rt + lane < n ? tile_of(p, pl, rows, rt + lane).units : 0;
            long long inc = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned in = __ballot_sync(0xffffffffu, x < begin + inc);
            const int at = in ? __ffs(in) - 1 : 31;
            if (in) {
                begin += __shfl_sync(0xffffffffu, inc - u, at);
                rt += at;
                break;
            }
            begin += __shfl_sync(0xffffffffu, inc, 31);
            if (rt + 32 >= n) return false;      // (x lies in the sequence, so this is not reached)
        }
        load(p, pl);
        return true;
    }
    __device__ bool next(const AttendParams& p, const Plan& pl) {
        begin += tile.units;
        if (++rt >= n_row_tiles(p, pl, rows)) {
            rt = 0;
            if (++head >= p.h0 + p.Hn) {
                head = p.h0;
                do {
                    if (++s >= p.n_seqs) return false;
                    rows = seq_rows(p, s);
                } while (n_row_tiles(p, pl, rows) == 0);
            }
        }
        load(p, pl);
        return true;
    }
};

// Floats of one part of a cut item: rows * D sums, then m and l per row.
__host__ __device__ constexpr size_t part_floats(int rows, int D) { return (size_t)rows * (D + 2); }

// A CTA whose last item goes on in the next CTAs: the item, and the last CTA
// that has a part of it; s < 0: none.  Its own part is the CTA's second, the
// others' parts are their first.
struct Cut {
    int s, head, rt, last;
};

__device__ __forceinline__ Cut cut_of(const Line& l, const Item& it, long long x_end) {
    if (it.begin + it.tile.units <= x_end) return Cut{-1, 0, 0, 0};
    return Cut{it.s, it.head, it.rt, (int)((it.begin + it.tile.units - 1) / l.chunk)};
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x h^2 with h = 2^(d / 2), for d down to twice the exponents' range: a sum of
// rows of zeros can stand that far above its reference.
__device__ __forceinline__ float twice(float x, float h) { return x * h * h; }

// What makes an item's sums its outputs, sums * inv * post: the power of two
// apart keeps inv a normal number.  A row without keys (l = 0) gets zeros.
struct Norm {
    float inv, post;
};
__device__ __forceinline__ Norm norm_of(float l) {
    const bool large = l > 1.f;
    return Norm{l == 0.f ? 0.f : (large ? kSumUnit * 0x1p43f : kSumUnit) / l, large ? 0x1p-43f : 1.f};
}

// log(sum of exponentials) from the reference and the sum.  The sum's exponent
// is taken apart, so that what cancels against m is a whole number.
__device__ __forceinline__ float lse_of(float m, float l) {
    if (l == 0.f) return -INFINITY;
    if (!(l < INFINITY)) return l;
    const bool tiny = l < 0x1p-100f;
    const uint32_t u = __float_as_uint(tiny ? l * 0x1p60f : l);
    const int e = (int)(u >> 23) - 127 + (tiny ? 17 - 60 : 17);          // (17: kSumUnit)
    return ((m + (float)e) + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u))) * 0.6931471805599453f;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of a word as fp16: lo = bytes 0, 1, hi = bytes 2, 3.  int8: the
// byte plus 128 under the exponent of 1024 is 1152 + code, minus 1152.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (FMT == LMOE_KV_INT8) {
        lo = hsub2(prmt(w, 0x64646464u, 0x4140), 0x64806480u);
        hi = hsub2(prmt(w, 0x64646464u, 0x4342), 0x64806480u);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    }
}

template <int FMT>
__device__ __forceinline__ uint32_t biased(uint32_t w) { return FMT == LMOE_KV_INT8 ? w ^ 0x80808080u : w; }

// Query rows of an item of the kernel for many rows: two tensor-core tiles of
// 128, or one where the accumulators of one fill tensor memory's half.
__host__ __device__ constexpr int many_rows(int D) { return D == 256 ? 128 : 256; }

// Images of key tiles: tokens of a tile, bytes (keys and values in fp16, three
// floats and a bit a token), and what a workspace holds of them: half of L2.
__host__ __device__ constexpr int image_tokens(int) { return 64; }
__host__ __device__ constexpr size_t image_bytes(int D) { return (size_t)image_tokens(D) * (4 * D + 12) + 128; }
constexpr size_t kImageBytes = 64u << 20;
// Images are made for more row tiles than kImageRowTiles, and for two to four
// where the contexts are brief and one group takes all (300 rows over 8000
// tokens of head_dim 64: 89 us converted on the way, 69 us with images; 480
// rows over 65536 tokens of head_dim 128: 202 and 572 us).
constexpr int kImageRowTiles = 4, kImageTokens = 8192;

constexpr size_t kCutBytes = 8192;      // kMaxCtas records of 16 bytes
static_assert(kMaxCtas * 16 <= kCutBytes, "cut records");

cudaError_t launch_join(const AttendParams& p, int rows, int n_ctas, bool few, cudaStream_t st);
cudaError_t launch_many(const AttendParams& p, cudaStream_t st);

}  // namespace attend
}  // namespace lmoe
