// gdn_kv_attn, few rows a request (decode, drafted tokens): softmax attention over the paged
// 8-bit cache, bound by the cache's bytes.
//
// Rows: the query tokens of a request times the query heads that share a KV head, 16 to a tile
// (row R is token R / G, head R % G). A unit of work is (request, KV head, row tile); its cost is
// its kv tiles of 128 tokens. All units' tiles form one line, cut into equal shares, one a block
// (each block finds its share from the lengths, on the device): a long context is spread over
// many blocks and short ones share one, whatever the mix, with nothing planned on the host. A unit
// cut by a share's end leaves a partial (m, l, O) in the workspace, and kv_attn_join_kernel adds
// the parts of each cut unit in order. Short contexts are not cut, and few of them get a cluster of
// eight blocks each (launch_kv_attn has the rules and what each side measured).
//
// Inside a block each of the four warps runs its own stream of 32-token steps with its own online
// softmax: K and V codes come by TMA into the warp's ring (one lane issues, nobody else is waited
// for). K's codes are the B operand of mma.m16n8k32 as they are where queries and output are bf16
// (queries as two e4m3 parts), and go to fp16 in registers otherwise (e4m3 fits fp16 exactly; queries
// as one or two fp16 parts); V's always do. The block scale, a power of two, multiplies the scores in
// fp32; V's is carried as the unit of the accumulators (O is kept in units of the current block's V
// scale and multiplied by the ratio, exactly, when it changes, down to 2^-64 of the largest), so no operand is
// rounded for it.
// Queries are divided by a power of two for each row so that the parts hold them. The weights are
// one fp16 part, and two where the output is fp32.
//
// The contraction index of an MMA may be permuted as long as both operands agree: a lane's
// 16-byte load of 16 key coordinates feeds its k-steps, and V's token pairs come from two rows'
// words by byte permutes. Rows of the 128-byte-swizzled tiles are taken in an order in which the
// eight lanes of a quarter-warp hit different banks.
//
// Measured (one B200): 64 requests of 128 to 16384 tokens, 32 query and 8 KV heads, d = 128, 441 MB:
// 105 us (4.2 TB/s); a block's loop alone moves 5.7 TB/s, the rest is units' starts and ends (8 thousand
// cycles each) and blocks that end apart. Warp-level MMA is enough here: with K's codes as an operand
// the tensor pipe is 40 % busy. Two blocks an SM (255 registers) hold 128 KB of copies in flight, and
// three stages a warp reached the rate of a plain copy loop; more and smaller shares (two a block) were
// slower (115 us), as were whole parts of units for few long contexts (73.5 against 71.6 us).
#include <algorithm>

#include "kv_attn.cuh"

namespace gdn {
namespace {
using namespace ptx;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStep = 32;                   // tokens of a warp's step
constexpr int kTile = kStep * kWarps;       // tokens of a block's tile
constexpr int kRows = 16;
constexpr float kNegInf = -__builtin_huge_valf();
// A row's reference is kBias below the largest exponent of the step that moves it, and its exponents may pass it by
// kSlack: fp16 holds weights up to 2^15, and starts to lose the small ones 2^-14 below 1. With the weights that high
// in its range, what is lost is below 2^-32 of the largest weight (one part) or 2^-44 (two).
constexpr float kBias = 7.f, kSlack = 15.f, kDown = 0x1p-15f;      // kDown: 2^-kSlack
constexpr float kLowPart = 4096.f;          // the second part of a weight is this much larger

template <int D> struct Smem {
    static constexpr int kBlocks = D == 128 ? 2 : 3;         // blocks an SM holds (registers)
    static constexpr int kStages = D == 128 ? 3 : 4;
    static constexpr int kStepBytes = kStep * D;             // K or V codes of a step
    static constexpr int kStageBytes = 2 * kStepBytes;
    static constexpr int kRing = kStages * kStageBytes;      // per warp
    static constexpr int kMergeRow = D + 4;                  // floats; rows of the cross-warp merge, over the rings
    static constexpr int kMerge = kWarps * kRows * kMergeRow * 4;
    static constexpr int kData = kWarps * kRing > kMerge ? kWarps * kRing : kMerge;
    static constexpr int kBytes = kData + 1024;              // slack to align to 1024
};

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ld_cluster_v2(uint32_t a, float (&r)[4]) {
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(r[0]), "=f"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ld_cluster_v4(uint32_t a, float (&r)[4]) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]) : "r"(a) : "memory");
}
// the same for an e4m3 query: D += A (16 x 32, e4m3) B (32 x 8, e4m3)
__device__ __forceinline__ void mma16832(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the two e4m3 codes in the low half -> fp16 pair (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t w) {
    uint32_t h;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
    return h;
}
// x as two fp16 parts: hi + lo = x to 22 bits (|x| within fp16's normal range)
__device__ __forceinline__ void split_h2(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = pack_h2(x - f.x, y - f.y);
}
// a weight as two fp16 parts: hi + lo / kLowPart = x to 2^-23, and to 2^-37 below fp16's range. What is left of a weight
// of up to 2^15 is at most 2^3, so lo is at most 2^15 too.
__device__ __forceinline__ void split_weight(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = pack_h2((x - f.x) * kLowPart, (y - f.y) * kLowPart);
}
// (a, b) += (x, y) + (xl, yl) / kLowPart, two-wide
__device__ __forceinline__ void add_parts(float &a, float &b, float x, float y, float xl, float yl) {
    asm("{\n\t.reg .b64 s, t, u, c;\n\t"
        "mov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tmov.b64 u, {%4, %5};\n\tmov.b64 c, {%6, %6};\n\t"
        "fma.rn.f32x2 t, u, c, t;\n\t"
        "add.rn.f32x2 s, s, t;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y), "f"(xl), "f"(yl), "f"(1.f / kLowPart));
}
// How queries enter Q K^T. kF8: as two e4m3 parts (bf16 queries with a bf16 output: the codes of K are then an
// operand as they are); kF16, kF16x2: as one or two fp16 parts, K's codes converted.
enum QKind { kF8, kF16, kF16x2 };

// A warp's row state while a unit runs, and its steps.
// HV: block scales of a step (2 where blocks hold 16 tokens)
template <int D, QKind QK, bool PSPLIT, int HV>
struct Worker {
    static constexpr int KS = QK == kF8 ? D / 32 : D / 16;     // k-steps of Q K^T
    static constexpr int NT = D / 8;                           // n-tiles of P V
    uint32_t qa[KS][4], ql[QK == kF16 ? 1 : KS][4];            // queries, high and low parts
    float o[NT][4];
    float m[2], l[2], rf[2];       // rows g and g + 8: reference of the exponents, this lane's part of the sum, score factor
    int hi[2], lo[2];              // positions a row sees: lo .. hi
    float vu;                      // V scale that the accumulators are in units of (0: none yet)
    float floor;                   // the smallest unit they may fall to (see enter)
    bool saw_nan;                  // a NaN of V was taken out of an edge step

    __device__ __forceinline__ static int token_of(int n) { return D == 128 ? (n & 1) * 4 + (n >> 1) : n; }

    __device__ __forceinline__ void scale_o(float f0, float f1) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            o[i][0] *= f0; o[i][1] *= f0; o[i][2] *= f1; o[i][3] *= f1;
        }
    }

    // The accumulators' unit becomes that of a block of V scale vs; returned is the factor that they need for it. The unit
    // never falls more than 2^64 below the largest scale met (floor), so that sums of 2^40 in units of that one stay
    // finite: a block of zeros has the scale 2^-100. Nor does it fall below 2^-100, the smallest that append makes. What
    // a smaller scale lacks goes into its block's weights (step).
    __device__ __forceinline__ float enter(float vs) {
        const float unit = fmaxf(vs, floor), f = vu == 0.f ? 1.f : vu / unit;
        vu = unit;
        floor = fmaxf(floor, vs * 0x1p-64f);
        return f;
    }

    // Queries of row g + 8 r from this lane's D / 4 coordinates (lane c: coordinates 16 (c + 4 half) + 0 .. 15).
    __device__ __forceinline__ void set_query(int r, const float (&f)[D / 4], float scale_log2) {
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(f[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // a power of two 2^e: |q| 2^-e < 2 for fp16 parts, <= 448 for e4m3 ones
        const uint32_t u = __float_as_uint(mx);
        int e = static_cast<int>(u >> 23) - 127;
        if (QK == kF8) e += ((u & 0x7fffffu) > 0x600000u ? 1 : 0) - 8;
        e = mx == 0.f || u >= 0x7f800000u ? 0 : min(max(e, -100), 126);
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        rf[r] = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        if constexpr (QK == kF8) {
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int half = 0; half < 2; ++half) {         // coordinates 8 s + 4 half + 0 .. 3
                    float y[4], z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = f[8 * s + 4 * half + i] * inv;
                        if (fabsf(y[i]) > 448.f) y[i] = __int_as_float(0x7fffffff);      // an infinite query shows as NaN
                    }
                    const uint32_t h = e4m3x4(y);
                    uint32_t lo2, hi2;
                    e4m3_to_h2(h, lo2, hi2);
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&lo2));
                    const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&hi2));
                    z[0] = y[0] - p.x; z[1] = y[1] - p.y; z[2] = y[2] - q.x; z[3] = y[3] - q.y;
                    qa[s][r + 2 * half] = h;
                    ql[s][r + 2 * half] = e4m3x4(z);
                }
        } else {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    y[i] = f[4 * s + i] * inv;
                    // an infinite query shows as NaN (as two parts it does so by itself): scores of -inf alone would pass
                    // for a row that sees nothing
                    if (QK == kF16 && fabsf(y[i]) > 65504.f) y[i] = __int_as_float(0x7fffffff);
                }
                if constexpr (QK == kF16x2) {
                    split_h2(y[0], y[1], qa[s][r], ql[s][r]);
                    split_h2(y[2], y[3], qa[s][r + 2], ql[s][r + 2]);
                } else {
                    qa[s][r] = pack_h2(y[0], y[1]);
                    qa[s][r + 2] = pack_h2(y[2], y[3]);
                }
            }
        }
    }

    __device__ __forceinline__ void no_query(int r) {
        rf[r] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qa[s][r] = qa[s][r + 2] = 0u;
            if constexpr (QK != kF16) ql[s][r] = ql[s][r + 2] = 0u;
        }
    }

    // One step: 32 tokens from position t0. sk, sv: shared addresses of the codes; ks, vs: scales of the step's halves;
    // edge: some row does not see some token; tok: tokens that exist and some row sees (bit i: t0 + i).
    __device__ __forceinline__ void step(uint32_t sk, uint32_t sv, int t0, const float (&ks)[HV], const float (&vs)[HV],
                                         uint32_t tok, bool edge) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        // (the four token groups side by side: a group's own products are a chain)
        float x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
            uint32_t w[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 8 * j + token_of(g), swz = D == 128 ? (r & 7) : ((r >> 1) & 3);
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(w[j][0]), "=r"(w[j][1]), "=r"(w[j][2]), "=r"(w[j][3])
                             : "r"(sk + r * D + (((c + 4 * half) ^ swz) << 4)));
            }
            if constexpr (QK == kF8) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16832(x[j], qa[2 * half + i], w[j][2 * i], w[j][2 * i + 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16832(x[j], ql[2 * half + i], w[j][2 * i], w[j][2 * i + 1]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b0[4], b1[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) e4m3_to_h2(w[j][i], b0[j], b1[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma16816(x[j], qa[4 * half + i], b0[j], b1[j]);
                    if constexpr (QK == kF16x2) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma16816(x[j], ql[4 * half + i], b0[j], b1[j]);
                    }
                }
            }
        }
        // Base-2 exponents against the row's reference m; elements 0, 1: row g, tokens token_of(2c), token_of(2c + 1),
        // 2, 3: row g + 8. The reference moves only when an exponent passes kSlack, so that most steps neither reduce over
        // the row's lanes nor touch the accumulators.
        auto sees = [&](int j, int i) {
            const int t = 8 * j + token_of(2 * c + (i & 1));
            return ((tok >> t) & 1u) && t0 + t <= hi[i >> 1] && t0 + t >= lo[i >> 1];
        };
        const bool none[2] = {m[0] == kNegInf, m[1] == kNegInf};      // rows without a reference yet
        float top = kNegInf;
        {
            const float base[2] = {none[0] ? 0.f : m[0], none[1] ? 0.f : m[1]};
            float rk[HV][2];
#pragma unroll
            for (int b = 0; b < HV; ++b) {
                rk[b][0] = rf[0] * ks[b];
                rk[b][1] = rf[1] * ks[b];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = fmaf(x[j][i], rk[HV == 1 ? 0 : j >> 1][i >> 1], -base[i >> 1]);
        }
        if (edge) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = sees(j, i) ? x[j][i] : kNegInf;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])));
        // the accumulators' factors: of the references, and of V's unit
        float f[2] = {1.f, 1.f};
        const float floor1 = HV == 1 ? floor : fmaxf(floor, vs[0] * 0x1p-64f);       // of the step's second half
        const bool far = vs[0] < floor || vs[HV - 1] < floor1;
        const bool move = __any_sync(0xffffffffu, top > kSlack || none[0] || none[1] || far);
        if (move) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = kNegInf;
#pragma unroll
                for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fmaxf(x[j][2 * r], x[j][2 * r + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                if (mx > (none[r] ? kNegInf : kBias)) {
                    const float by = mx - kBias;
                    f[r] = none[r] ? 0.f : ex2(-by);
                    m[r] = none[r] ? by : m[r] + by;
#pragma unroll
                    for (int j = 0; j < 4; ++j) { x[j][2 * r] -= by; x[j][2 * r + 1] -= by; }
                }
                l[r] *= f[r];
            }
            if (far) {      // rare: weights smaller by what the unit does not hold, but whole in the rows' sums
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float s = vs[HV == 1 ? 0 : j >> 1], fl = j < 2 ? floor : floor1;
                    const float lack = s < fl ? log2f(s) - log2f(fl) : 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        l[i >> 1] += ex2(x[j][i]) - ex2(x[j][i] + lack);
                        x[j][i] += lack;
                    }
                }
            }
        }
        if (move || vs[0] != vu) {
            const float u = enter(vs[0]);
            scale_o(f[0] * u, f[1] * u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[j][i] = ex2(x[j][i]);
                l[i >> 1] += x[j][i];
            }
        // P V for NH halves at a time, 16 tokens each. An fp32 output takes both where they have one V scale: the tensor
        // core's own running sum truncates, so each such sum starts anew and is added in fp32.
        constexpr int NH = PSPLIT && HV == 1 ? 2 : 1, W = D / 32;      // W: words a lane takes of a row
#pragma unroll
        for (int h0 = 0; h0 < 2; h0 += NH) {
            if constexpr (HV == 2) {
                if (h0 == 1 && vs[1] != vu) {
                    const float u = enter(vs[1]);
                    scale_o(u, u);
                }
            }
            uint32_t p[NH][4], pl[NH][4], v[NH][4][W];
#pragma unroll
            for (int k = 0; k < NH; ++k) {
                const int hf = h0 + k;
                float(&xa)[4] = x[2 * hf], (&xb)[4] = x[2 * hf + 1];
                if constexpr (PSPLIT) {
                    split_weight(xa[0], xa[1], p[k][0], pl[k][0]);
                    split_weight(xa[2], xa[3], p[k][1], pl[k][1]);
                    split_weight(xb[0], xb[1], p[k][2], pl[k][2]);
                    split_weight(xb[2], xb[3], p[k][3], pl[k][3]);
                } else {
                    p[k][0] = pack_h2(xa[0], xa[1]); p[k][1] = pack_h2(xa[2], xa[3]);
                    p[k][2] = pack_h2(xb[0], xb[1]); p[k][3] = pack_h2(xb[2], xb[3]);
                }
                // this lane's four V rows of the half: k = 2c, 2c + 1, 2c + 8, 2c + 9
                const int ra = 16 * hf + token_of(2 * c), rb = 16 * hf + token_of(2 * c + 1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = (i & 1 ? rb : ra) + (i >> 1) * 8;
                    uint32_t(&vr)[W] = v[k][i];
                    if constexpr (D == 128) {
                        const int ch = (g & 1) * 4 + (g >> 1);
                        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                     : "=r"(vr[0]), "=r"(vr[1]), "=r"(vr[2]), "=r"(vr[3])
                                     : "r"(sv + r * D + ((ch ^ (r & 7)) << 4)));
                    } else {
                        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];"
                                     : "=r"(vr[0]), "=r"(vr[1])
                                     : "r"(sv + r * D + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8));
                    }
                }
                if (edge) {
                    // Rows that do not exist hold anything, and 0 * NaN would reach rows that do not see the NaN: both are
                    // taken out, and a NaN is noted (the rows it belongs to are found when the unit is done).
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = (i & 1 ? rb : ra) + (i >> 1) * 8;
                        const uint32_t keep = (tok >> r) & 1u ? 0xffffffffu : 0u;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const uint32_t isnan = __vcmpeq4(v[k][i][w] & 0x7f7f7f7fu, 0x7f7f7f7fu) & keep;
                            saw_nan |= isnan != 0u;
                            v[k][i][w] &= keep & ~isnan;
                        }
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // column 4 w + q of the lane's chunk: the two rows' bytes side by side, then as fp16 pair
                    const uint32_t sel = q | ((4 + q) << 4);
                    float(&acc)[4] = o[4 * w + q];
                    float t[4] = {0.f, 0.f, 0.f, 0.f}, tl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < NH; ++k) {
                        const uint32_t b0 = e4m3x2_to_h2(__byte_perm(v[k][0][w], v[k][1][w], sel));
                        const uint32_t b1 = e4m3x2_to_h2(__byte_perm(v[k][2][w], v[k][3][w], sel));
                        if constexpr (PSPLIT) {
                            mma16816(tl, pl[k], b0, b1);
                            mma16816(t, p[k], b0, b1);
                        } else {
                            mma16816(acc, p[k], b0, b1);
                        }
                    }
                    // (blocks of 16 tokens have twice as many of these sums: two-wide, 64 requests of fp32 queries 146 us against
                    // 151; with larger blocks that was slower, 118 us against 115 for bf16 queries)
                    if constexpr (PSPLIT && HV == 2) {
#pragma unroll
                        for (int r = 0; r < 4; r += 2) add_parts(acc[r], acc[r + 1], t[r], t[r + 1], tl[r], tl[r + 1]);
                    } else if constexpr (PSPLIT) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[r] += fmaf(tl[r], 1.f / kLowPart, t[r]);
                    }
                }
        }
    }
};

template <int D, QKind QK, bool PSPLIT, int HV, typename IT>
__global__ void __launch_bounds__(kThreads, Smem<D>::kBlocks)
kv_attn_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const AttnArgs a) {
    using S = Smem<D>;
    using W = Worker<D, QK, PSPLIT, HV>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t s_bar[kWarps][S::kStages];
    __shared__ Share s_share;
    __shared__ float s_ml[kWarps][kRows][2];
    __shared__ __align__(8) float s_fin[kRows][2];     // a cluster's blocks: m and l of this block's rows
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int G = a.Hq / a.Hkv;

    cudaTriggerProgrammaticLaunchCompletion();     // the join kernel's blocks may take their places; they wait there
    if (lane == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(&s_bar[warp][i], 1);
        fence_mbar_init();
    }
    const int cs = a.cluster, rank = blockIdx.x % cs;
    find_share<kThreads>(a, blockIdx.x / cs, gridDim.x / cs, &s_share);      // ends with a block barrier
    const Share sh = s_share;
    CutUnit cut{};
    if (sh.begin >= sh.end) {
        if (tid == 0) a.cuts[blockIdx.x] = cut;
        return;
    }
    const uint32_t ring = smem_u32(smem) + warp * S::kRing;
    uint32_t phase = 0;                     // parity bit of each stage
    uint32_t live = 0;                      // stages with copies in flight
    bool ok = true;                         // this warp's copies arrive
    constexpr int br = kStep / HV;          // rows of a TMA box

    int n = sh.n;
    long long off = sh.off, left = sh.end - sh.begin;
    bool first_unit = true;
    ReqWork rw = request_work(a, n);
    while (left > 0) {
        if (off >= rw.work) {
            off -= rw.work;
            rw = request_work(a, ++n);
            continue;
        }
        // the unit (head, row tile) and its part of this share
        const int cost = cs > 1 ? 1 : rw.tiles + kUnitCost;
        const int unit = static_cast<int>(off < 0x7fffffff ? static_cast<unsigned>(off) / static_cast<unsigned>(cost) : off / cost);
        const int at = static_cast<int>(off - static_cast<long long>(unit) * cost);
        int take = static_cast<int>(min(left, static_cast<long long>(cost - at)));
        if (a.whole) {                      // a share takes the units that start in it, to their ends
            if (at > 0) {
                off += take;
                left -= take;
                continue;
            }
            take = cost;
        }
        int tile0 = max(0, at - kUnitCost), ntile = max(0, at + take - kUnitCost) - tile0;
        off += take;
        left -= take;
        if (cs > 1) {                       // this block's part of the cluster's unit; it may be none
            tile0 = rank * rw.tiles / cs;
            ntile = (rank + 1) * rw.tiles / cs - tile0;
        } else if (ntile == 0) {
            continue;                       // the share ends before the unit's first tile
        }
        const int h = unit / rw.row_tiles, rt = unit - h * rw.row_tiles;
        const int rows = rw.qlen * G;
        const int p_first = rw.kv - rw.qlen + rt * kRows / G;
        const int p_last = rw.kv - rw.qlen + min(rt * kRows + kRows - 1, rows - 1) / G;
        // tokens of this part that some row sees
        const int t_lo = max((rw.tile0 + tile0) * kTile, a.window > 0 ? max(0, max(p_first, -1) - a.window + 1) / kTile * kTile : 0);
        const int t_hi = min((rw.tile0 + tile0 + ntile) * kTile, p_last + 1);

        W w;
        const int *table = a.table + static_cast<long long>(n) * a.max_blocks;
        // block numbers and scales of the warp's next 32 steps, one step a lane
        struct Bank {
            int blk[HV];
            float ksc[HV], vsc[HV];
        } cur, nxt;
        auto fetch_blocks = [&](Bank &bank, int step0) {
#pragma unroll
            for (int b = 0; b < HV; ++b) {
                const int t = t_lo + (step0 + lane) * kTile + warp * kStep + b * br;
                bank.blk[b] = -1;
                bank.ksc[b] = bank.vsc[b] = 1.f;
                if (t < t_hi) {
                    const int id = in_bounds(t >> a.bs_log2, a.max_blocks, a.err) ? table[t >> a.bs_log2] : -1;
                    if (id >= 0 && id < a.num_blocks) {
                        bank.blk[b] = id;
                        bank.ksc[b] = a.k_scale[static_cast<long long>(id) * a.Hkv + h];
                        bank.vsc[b] = a.v_scale[static_cast<long long>(id) * a.Hkv + h];
                    } else {
                        atomicOr(a.err, kErrBadSeqlens);
                    }
                }
            }
        };
        auto issue = [&](int i, int stage, const Bank &bank) {           // copies of step i
            const int t = t_lo + i * kTile + warp * kStep;
            int id[HV], boxes = 0;
#pragma unroll
            for (int b = 0; b < HV; ++b) {
                id[b] = __shfl_sync(0xffffffffu, bank.blk[b], i & 31);
                boxes += id[b] >= 0 ? 1 : 0;
            }
            if (lane == 0 && boxes > 0) {
                uint64_t *bar = &s_bar[warp][stage];
                mbar_arrive_expect_tx(bar, 2 * boxes * br * D);
#pragma unroll
                for (int b = 0; b < HV; ++b)
                    if (id[b] >= 0) {
                        const uint32_t dst = ring + stage * S::kStageBytes + b * br * D;
                        const int row = ((id[b] * a.Hkv + h) << a.bs_log2) + (HV == 1 ? t & (a.bs - 1) : 0);
                        tma_load_2d(dst, &mk, bar, 0, row);
                        tma_load_2d(dst + S::kStepBytes, &mv, bar, 0, row);
                    }
            }
            return boxes > 0;
        };
        // steps of this warp: those that start before t_hi
        const int nstep = t_hi > t_lo + warp * kStep ? (t_hi - t_lo - warp * kStep + kTile - 1) / kTile : 0;
        // queries, in fragment order: coordinates 16 (c + 4 half) + 4 i + 0 .. 3 of rows g and g + 8. Their loads go out
        // before the block numbers' and are used after the first copies are under way.
        float qf[2][D / 4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int R = rt * kRows + g + 8 * r;
            const bool in = R < rows;
            const int tok = R / G;
            const IT *qp = static_cast<const IT *>(a.q) + (rw.row0 + tok) * a.q_stride +
                           static_cast<long long>(h * G + (R - tok * G)) * D;
#pragma unroll
            for (int half = 0; half < D / 64; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i) load4(in ? qp + 16 * (c + 4 * half) + 4 * i : nullptr, &qf[r][16 * half + 4 * i]);
            w.hi[r] = in ? rw.kv - rw.qlen + tok : -1;
            w.lo[r] = a.window > 0 ? max(w.hi[r], -1) - a.window + 1 : 0;      // (rows before position 0 see nothing anyway)
            w.m[r] = kNegInf;
            w.l[r] = 0.f;
        }
        fetch_blocks(cur, 0);
        nxt = cur;
        for (int i = 0; i < min(nstep, S::kStages - 1); ++i)
            if (ok && issue(i, i, cur)) live |= 1u << i;

        const int nrows = min(kRows, rows - rt * kRows);        // rows of this tile
        w.set_query(0, qf[0], a.scale_log2);
        if (nrows > 8) w.set_query(1, qf[1], a.scale_log2);
        else w.no_query(1);
#pragma unroll
        for (int i = 0; i < W::NT; ++i) w.o[i][0] = w.o[i][1] = w.o[i][2] = w.o[i][3] = 0.f;
        w.vu = 0.f;
        w.floor = 0x1p-100f;
        w.saw_nan = false;

        const int lo_last = a.window > 0 ? max(p_last, -1) - a.window + 1 : 0;
        const int lo_first = a.window > 0 ? max(0, max(p_first, -1) - a.window + 1) : 0;      // no row sees a position before it
        struct Step {
            int t;
            float ks[HV], vs[HV];
            uint32_t tok;          // tokens that exist and some row sees
            bool edge;             // some row does not see some token
        };
        auto look = [&](int i) {
            Step x;
            x.t = t_lo + i * kTile + warp * kStep;
            if ((i & 31) == 0 && i > 0) cur = nxt;
            if ((i & 31) == 8 && i + 24 < nstep) fetch_blocks(nxt, i + 24);
            x.tok = 0u;
#pragma unroll
            for (int b = 0; b < HV; ++b) {
                x.ks[b] = __shfl_sync(0xffffffffu, cur.ksc[b], i & 31);
                x.vs[b] = __shfl_sync(0xffffffffu, cur.vsc[b], i & 31);
                const int id = __shfl_sync(0xffffffffu, cur.blk[b], i & 31);
                if (id >= 0) x.tok |= (HV == 1 ? 0xffffffffu : 0xffffu) << (16 * b);
            }
            if (t_hi - x.t < kStep) x.tok &= (1u << (t_hi - x.t)) - 1u;
            if (x.t < lo_first) x.tok = lo_first - x.t < kStep ? x.tok & (0xffffffffu << (lo_first - x.t)) : 0u;
            if (HV == 2) {         // a half with nothing to see leaves V's unit alone
                if ((x.tok & 0xffffu) == 0u) x.vs[0] = x.vs[HV - 1];
                else if ((x.tok >> 16) == 0u) x.vs[HV - 1] = x.vs[0];
            }
            x.edge = x.tok != 0xffffffffu || x.t + kStep - 1 > p_first || x.t < lo_last;
            return x;
        };
        int st = 0, nst = (S::kStages - 1) % S::kStages;      // stages of step i and of the one sent out beside it
        auto turn = [&](int i) {            // sends a later step's copies out, waits for this one's
            __syncwarp();
            const int nx = i + S::kStages - 1;
            if (nx < nstep && ok && issue(nx, nst, (nx >> 5) == (i >> 5) ? cur : nxt)) live |= 1u << nst;
            if (ok && (live & (1u << st))) {
                const uint32_t par = (phase >> st) & 1u;
                if (!bounded_wait(&s_bar[warp][st], par, a.wait_limit)) {
                    // gave up: reported, and the copy still in flight is waited for (with the drain's limit)
                    // before its buffer is used again
                    if (lane == 0) atomicOr(a.err, kErrWaitTimeout);
                    ok = bounded_wait(&s_bar[warp][st], par, kDrainLimitCycles);
                }
                ok = __all_sync(0xffffffffu, ok);
                phase ^= 1u << st;
                live ^= 1u << st;
            }
            const uint32_t sk = ring + st * S::kStageBytes;
            nst = st;
            st = st + 1 == S::kStages ? 0 : st + 1;
            return sk;
        };
        for (int i = 0; i < nstep; ++i) {
            const Step x = look(i);
            const uint32_t sk = turn(i);
            if (ok && x.tok != 0u) w.step(sk, sk + S::kStepBytes, x.t, x.ks, x.vs, x.tok, x.edge);
        }
        // A copy that did not come even within the drain's limit: the others in flight are waited for as well, before their
        // buffers are used for the merge or the block ends, and this warp sends no more.
        if (!ok) {
            for (int i = 0; i < S::kStages; ++i)
                if (live & (1u << i)) bounded_wait(&s_bar[warp][i], (phase >> i) & 1u, kDrainLimitCycles);
            live = 0;
        }

        // ---- the four warps' parts of each row, against references kSlack higher: weights up to 1, so that the sums of
        // weights times values are finite wherever the tokens' number times the largest value is
        const float out_unit = w.vu * kDown;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 1);
            w.l[r] += __shfl_xor_sync(0xffffffffu, w.l[r], 2);
            if (c == 0) {
                s_ml[warp][g + 8 * r][0] = w.m[r] + kSlack;
                s_ml[warp][g + 8 * r][1] = w.l[r] * kDown;
            }
        }
        const bool nans = __syncthreads_or(w.saw_nan);      // (and every warp is through its ring)
        float *mg = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (g + 8 * r >= nrows) break;
            float *row = mg + (warp * kRows + g + 8 * r) * S::kMergeRow;
            // n-tile i: column 2c is coordinate x0 + i, column 2c + 1 coordinate x1 + i
            const int x0 = 16 * c, x1 = D == 128 ? 64 + 16 * c : 16 * c + 8;
#pragma unroll
            for (int i = 0; i < W::NT; i += 4) {
                *reinterpret_cast<float4 *>(row + x0 + i) = make_float4(w.o[i][2 * r] * out_unit, w.o[i + 1][2 * r] * out_unit,
                                                                        w.o[i + 2][2 * r] * out_unit, w.o[i + 3][2 * r] * out_unit);
                *reinterpret_cast<float4 *>(row + x1 + i) =
                    make_float4(w.o[i][2 * r + 1] * out_unit, w.o[i + 1][2 * r + 1] * out_unit, w.o[i + 2][2 * r + 1] * out_unit,
                                w.o[i + 3][2 * r + 1] * out_unit);
            }
        }
        __syncthreads();
        const bool whole = tile0 == 0 && ntile == rw.tiles;
        // a block leaves at most two parts: the end of a unit begun by another block (slot 0), and the start
        // of one that another ends (slot 1; a middle piece goes to slot 0)
        float *part = whole ? nullptr : a.ws + (2ll * blockIdx.x + (first_unit && tile0 > 0 ? 0 : 1)) * part_floats(D);
        // a row at a time to a warp (two at d = 64), four columns a lane
        constexpr int RPW = 128 / D, LPR = 32 / RPW;
#pragma unroll
        for (int q = 0; q < kRows / (kWarps * RPW); ++q) {
            const int r = (q * kWarps + warp) * RPW + lane / LPR, x = (lane % LPR) * 4;
            if (r >= nrows) break;
            float mm = kNegInf;
#pragma unroll
            for (int p = 0; p < kWarps; ++p) mm = fmaxf(mm, s_ml[p][r][0]);
            const float base = mm == kNegInf ? 0.f : mm;
            float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < kWarps; ++p) {
                const float f = ex2(s_ml[p][r][0] - base);
                const float4 v = *reinterpret_cast<const float4 *>(mg + (p * kRows + r) * S::kMergeRow + x);
                ll = fmaf(s_ml[p][r][1], f, ll);
                acc[0] = fmaf(v.x, f, acc[0]);
                acc[1] = fmaf(v.y, f, acc[1]);
                acc[2] = fmaf(v.z, f, acc[2]);
                acc[3] = fmaf(v.w, f, acc[3]);
            }
            const int R = rt * kRows + r;
            if (nans) {        // rare: the row's own positions are looked through for NaN in these columns
                const int pos = rw.kv - rw.qlen + R / G, lo = a.window > 0 ? max(0, max(pos, -1) - a.window + 1) : 0;
                for (int t = max(t_lo, lo); t < min(t_hi, pos + 1); ++t) {
                    const int id = table[t >> a.bs_log2];
                    if (id < 0 || id >= a.num_blocks) continue;
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(
                        a.v_codes + ((((static_cast<long long>(id) * a.Hkv + h) << a.bs_log2) + (t & (a.bs - 1))) * D + x));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (((v >> (8 * k)) & 0x7fu) == 0x7fu) acc[k] = __int_as_float(0x7fffffff);
                }
            }
            if (cs > 1) {
                // (only this lane reads these four values of part 0)
                *reinterpret_cast<float4 *>(mg + r * S::kMergeRow + x) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                if (x == 0) { s_fin[r][0] = mm; s_fin[r][1] = ll; }
            } else if (whole) {
                store_row<4>(a, rw.row0 + R / G, h * G + R % G, D, x, acc, ll, mm);
            } else {
                if (x == 0) { part[r] = mm; part[kRows + r] = ll; }
                *reinterpret_cast<float4 *>(part + 2 * kRows + r * D + x) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
        }
        if (cs > 1) {
            // the cluster's parts of each row, in block order, rows in turn over the blocks
            cluster_sync();
            for (int r = rank + cs * warp; r < nrows; r += cs * kWarps) {
                if (lane >= D / 4) break;
                const int x = 4 * lane, R = rt * kRows + r;
                const uint32_t fin = smem_u32(&s_fin[r][0]), row = smem_u32(mg + r * S::kMergeRow + x);
                float mm = kNegInf, ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
                for (int p = 0; p < cs; ++p) {
                    float v[4], ml[4];
                    ld_cluster_v2(mapa_shared(fin, p), ml);
                    ld_cluster_v4(mapa_shared(row, p), v);
                    const float mn = fmaxf(mm, ml[0]), base = mn == kNegInf ? 0.f : mn;
                    const float f = ex2(mm - base), fp = ex2(ml[0] - base);
                    mm = mn;
                    ll = ll * f + ml[1] * fp;
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] = acc[i] * f + v[i] * fp;
                }
                store_row<4>(a, rw.row0 + R / G, h * G + R % G, D, x, acc, ll, mm);
            }
            cluster_sync();                     // nobody leaves, or takes copies, while its parts are read
        } else if (tile0 == 0 && ntile < rw.tiles)      // begun here, ended in a later share
            cut = CutUnit{rw.row0, h, rt, nrows,
                          static_cast<int>((sh.end + rw.tiles - ntile - 1) / sh.per) - static_cast<int>(blockIdx.x) + 1};
        // the rings take copies again: what was read and written through the generic proxy comes before them
        fence_proxy_async();
        __syncthreads();
        first_unit = false;
    }
    if (tid == 0) a.cuts[blockIdx.x] = cut;
}

// Adds the parts of the units that were cut: block (c, y) takes four rows of the unit that starts in share c
// and ends in a later one (the main kernel has noted which). A row's parts are taken in turn by kJoinWarps
// warps, whose sums are added in warp order, so the order is fixed.
constexpr int kJoinRows = 4, kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinRows * kJoinWarps) kv_attn_join_kernel(const AttnArgs a) {
    constexpr int CPL = D / 32;            // columns of a lane
    __shared__ float s_ml[kJoinRows][kJoinWarps][2];
    __shared__ float s_o[kJoinRows][kJoinWarps][D];
    cudaGridDependencySynchronize();
    const int blk = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const CutUnit cu = a.cuts[blk];
    const int rr = warp / kJoinWarps, pw = warp % kJoinWarps;
    const int r = blockIdx.y * kJoinRows + rr;
    if (cu.parts == 0 || blockIdx.y * kJoinRows >= cu.rows) return;

    float m = kNegInf, l = 0.f, o[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int p = pw; p < cu.parts; p += kJoinWarps) {
        const float *q = a.ws + (2ll * (blk + p) + (p == 0 ? 1 : 0)) * part_floats(D);
        const float mp = q[r], lp = q[kRows + r];
        float x[CPL];
        const float *qo = q + 2 * kRows + r * D + lane * CPL;
        if constexpr (D == 128) *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(qo);
        else *reinterpret_cast<float2 *>(x) = *reinterpret_cast<const float2 *>(qo);
        const float mn = fmaxf(m, mp), base = mn == kNegInf ? 0.f : mn;
        const float f = ex2(m - base), fp = ex2(mp - base);
        m = mn;
        l = l * f + lp * fp;
#pragma unroll
        for (int i = 0; i < CPL; ++i) o[i] = o[i] * f + x[i] * fp;
    }
    if (lane == 0) { s_ml[rr][pw][0] = m; s_ml[rr][pw][1] = l; }
#pragma unroll
    for (int i = 0; i < CPL; ++i) s_o[rr][pw][lane * CPL + i] = o[i];
    __syncthreads();
    if (pw != 0 || lane >= D / 4 || r >= cu.rows) return;
    float mm = kNegInf, ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int q = 0; q < kJoinWarps; ++q) mm = fmaxf(mm, s_ml[rr][q][0]);
    const float base = mm == kNegInf ? 0.f : mm;
#pragma unroll
    for (int q = 0; q < kJoinWarps; ++q) {
        const float f = ex2(s_ml[rr][q][0] - base);
        ll = fmaf(s_ml[rr][q][1], f, ll);
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(s_o[rr][q][4 * lane + i], f, acc[i]);
    }
    const int G = a.Hq / a.Hkv, R = cu.row_tile * kRows + r;
    store_row<4>(a, cu.row0 + R / G, cu.head * G + R % G, D, 4 * lane, acc, ll, mm);
}

template <int D, QKind QK, bool PSPLIT, typename IT>
gdn_status_t launch_t(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, cudaStream_t stream) {
    auto kern = a.bs == 16 ? kv_attn_kernel<D, QK, PSPLIT, 2, IT> : kv_attn_kernel<D, QK, PSPLIT, 1, IT>;
    if (!ensure_smem_limit(reinterpret_cast<const void *>(kern), Smem<D>::kBytes)) return GDN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    if (a.cluster > 1) {
        cfg.gridDim = dim3(static_cast<unsigned>(a.blocks));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Smem<D>::kBytes;
        cfg.stream = stream;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = static_cast<unsigned>(a.cluster);
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, mk, mv, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    kern<<<grid, kThreads, Smem<D>::kBytes, stream>>>(mk, mv, a);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    if (a.whole) return GDN_OK;            // nothing to join
    cfg.gridDim = dim3(static_cast<unsigned>(grid), kRows / kJoinRows);
    cfg.blockDim = dim3(32 * kJoinRows * kJoinWarps);
    cfg.stream = stream;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D>, a) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int D>
gdn_status_t launch_d(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int grid, bool in_f32,
                      bool out_f32, cudaStream_t stream) {
    if (in_f32) return out_f32 ? launch_t<D, kF16x2, true, float>(mk, mv, a, grid, stream)
                               : launch_t<D, kF16x2, false, float>(mk, mv, a, grid, stream);
    return out_f32 ? launch_t<D, kF16, true, __nv_bfloat16>(mk, mv, a, grid, stream)
                   : launch_t<D, kF8, false, __nv_bfloat16>(mk, mv, a, grid, stream);
}

}  // namespace

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();      // tc_gdn.cu

bool make_cache_map(CUtensorMap *m, const void *ptr, long long rows, int d, int box_rows) {
    EncodeTiledFn encode = encode_fn();
    if (!encode) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(box_rows)}, one[2] = {1, 1};
    return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static int kv_attn_grid(int d) {
    const int sms = sm_count();
    return (sms > 0 ? sms : 148) * (d == 128 ? Smem<128>::kBlocks : Smem<64>::kBlocks);
}

size_t kv_attn_ws_bytes(int N, int d) {
    return static_cast<size_t>(kv_attn_grid(d)) * (2 * part_floats(d) * sizeof(float) + sizeof(CutUnit)) +
           (static_cast<size_t>(N) * sizeof(int) + 15) / 16 * 16;
}

// kv_prompt.cu: requests of more than a.many_rows rows (bf16 in and out); redo: (N) ints, zeroed by it
gdn_status_t launch_kv_prompt(const void *kc, const void *vc, const AttnArgs &a, int d, int *redo, cudaStream_t stream);

constexpr int kManyRows = 64, kManyRowsPerSm128 = 40, kManyRowsPerSm64 = 58;
constexpr int kWholeTokens = 256, kWholeTokensMany = 1024;
constexpr int kClusterTokens = 8 * kTile;

gdn_status_t launch_kv_attn(const void *kc, const void *vc, AttnArgs a, int d, bool in_f32, bool out_f32,
                            cudaStream_t stream) {
    a.v_codes = static_cast<const uint8_t *>(vc);
    a.err = device_error_word();
    if (!a.err) return GDN_ERR_CUDA;
    a.wait_limit = wait_limit_cycles();
    const long long rows = static_cast<long long>(a.num_blocks) * a.Hkv * a.bs;
    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, kc, rows, d, std::min(a.bs, kStep)) || !make_cache_map(&mv, vc, rows, d, std::min(a.bs, kStep)))
        return GDN_ERR_CUDA;
    const int grid = kv_attn_grid(d), sms = grid / (d == 128 ? Smem<128>::kBlocks : Smem<64>::kBlocks);
    a.cuts = reinterpret_cast<CutUnit *>(a.ws + grid * 2 * part_floats(d));
    // Contexts (or windows) that the table bounds to kWholeTokens are not cut, nor those up to kWholeTokensMany where there
    // are units for half the blocks: no join, and fewer units begun (8 KV heads, d = 128, cut / not cut: one request of
    // 100 tokens 10.5 / 8.7 us, 32 of 700 23.9 / 18.7 us, but one of 700 10.7 / 15.5 us)
    const long long most = static_cast<long long>(a.max_blocks) * a.bs;
    const long long seen = a.window > 0 ? std::min(most, static_cast<long long>(a.window) + std::min<long long>(a.max_q, kManyRows) + 127)
                                        : most;
    a.whole = seen <= kWholeTokens || (seen <= kWholeTokensMany && 2ll * a.N * a.Hkv >= grid) ? 1 : 0;
    // Few units of up to kClusterTokens, a kv tile for each of eight blocks: a cluster of eight for each unit, whose parts are
    // added through distributed shared memory (one launch, no workspace). One request of 700 tokens, 8 KV heads, d =
    // 128: 8.9 us against 9.5 cut and joined, and 2 us less on the host; with one tile in all (7.6 us whole against
    // 8.6), two tiles a block (10.5 against 10.2) or clusters of two for more units (11.8 against 10.3) it is slower.
    a.cluster = 1;
    if (seen > kTile && seen <= kClusterTokens && static_cast<long long>(a.max_q) * (a.Hq / a.Hkv) <= kManyRows) {
        const long long units = (static_cast<long long>(a.T) * (a.Hq / a.Hkv) / kRows + a.N) * a.Hkv;      // at most
        if (8 * units <= sms) {
            a.cluster = 8;
            a.blocks = static_cast<int>(8 * units);
        }
    }
    int *redo = reinterpret_cast<int *>(a.cuts + grid);
    a.redo = redo;
    a.many_rows = 0;
    // The many-rows kernel walks a context with one block per 256 rows, this one spreads it over the device: the former pays
    // from rows for a good part of the SMs on (at one token from each other request, the most that the prompts can have).
    // Many / few rows, one prompt: d = 128, 4096 rows 40 / 30 us over 1024 tokens and 88 / 68 over 4096, 8192 rows 40 / 48
    // and 89 / 118; d = 64, 8192 rows 35 / 33 and 82 / 80, 16384 rows 36 / 52 and 84 / 145.
    const long long prompt_rows = static_cast<long long>(a.T - std::min(a.T, a.N - 1)) * a.Hq;
    if (!in_f32 && !out_f32 && static_cast<long long>(a.max_q) * (a.Hq / a.Hkv) > kManyRows &&
        prompt_rows >= static_cast<long long>(sms) * (d == 128 ? kManyRowsPerSm128 : kManyRowsPerSm64)) {
        a.many_rows = kManyRows;
        const gdn_status_t st = launch_kv_prompt(kc, vc, a, d, redo, stream);
        if (st != GDN_OK) return st;
    }
    return d == 128 ? launch_d<128>(mk, mv, a, grid, in_f32, out_f32, stream)
                    : launch_d<64>(mk, mv, a, grid, in_f32, out_f32, stream);
}

}  // namespace gdn
