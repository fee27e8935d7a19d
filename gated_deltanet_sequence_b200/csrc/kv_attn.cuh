// Shared by the kernels of gdn_kv_attn: arguments, the shares of the work line, row outputs.
#pragma once
#include "tc_kernels.cuh"
#include "tc_ptx.cuh"

namespace gdn {

// A unit that a share begins and a later one ends (parts == 0: none), for the join.
struct CutUnit {
    long long row0;
    int head, row_tile, rows, parts;
};

struct AttnArgs {
    const void *q;
    long long q_stride;
    const float *k_scale, *v_scale;
    const uint8_t *v_codes;
    const int *table, *cu, *kv_lens;
    void *o;
    float *lse, *ws;
    CutUnit *cuts;
    int N, T, Hq, Hkv, num_blocks, bs, bs_log2, max_blocks, max_q, window, out_bf16;
    float scale_log2;          // scale * log2(e): scores are kept as base-2 exponents
    int whole;                 // units are not cut (and not joined)
    int cluster, blocks;       // blocks of a unit (1: shares of the line instead), and of the launch then
    // requests of more rows than this belong to the many-rows kernel (0: it is not used), but for those it left
    int many_rows;
    const int *redo;           // (N), nullable: requests that the many-rows kernel left
    unsigned *err;
    long long wait_limit;
};

// A 2-D TMA map over the cache as (rows, d) bytes; boxes of box_rows whole rows, swizzled over their width.
bool make_cache_map(CUtensorMap *m, const void *ptr, long long rows, int d, int box_rows);

// A box of such a map, to shared memory.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1)
        : "memory");
}
// four e4m3 codes -> two fp16 pairs (exact)
__device__ __forceinline__ void e4m3_to_h2(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
// four values -> four e4m3 codes, nearest even (NaN stays NaN)
__device__ __forceinline__ uint32_t e4m3x4(const float (&y)[4]) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(y[1]), "f"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(y[3]), "f"(y[2]));
    return a | (static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Floats of one partial: m and l of 16 rows, then their O.
__host__ __device__ constexpr long long part_floats(int d) { return 32 + 16ll * d; }

// What a unit costs beside its tiles (its queries, the warps' merge, its rows), in tiles. Without it the shares of
// short contexts took longest.
constexpr int kUnitCost = 3;

// A request's part of the work line: (Hkv x row_tiles) units of kUnitCost + `tiles` places, a place for each kv tile
// (128 tokens) from tile0 on. A request with rows has one tile at least, so that every unit's rows are written.
struct ReqWork {
    long long row0;     // first token row
    int qlen, kv, row_tiles, tiles, tile0;
    long long work;
    bool bad, many;
};
__device__ __forceinline__ ReqWork request_work(const AttnArgs &a, int n, bool many_kernel = false) {
    ReqWork w;
    const int c0 = a.cu[n], c1 = a.cu[n + 1];
    w.row0 = c0;
    w.qlen = c1 - c0;
    w.kv = a.kv_lens[n];
    const bool bad = c0 < 0 || c1 < c0 || c1 > a.T || w.qlen > a.max_q || w.kv < 0 ||
                     w.kv > static_cast<long long>(a.max_blocks) * a.bs;
    if (bad) w.qlen = 0;
    w.many = !bad && a.many_rows > 0 && static_cast<long long>(w.qlen) * (a.Hq / a.Hkv) > a.many_rows;
    if (w.many && !many_kernel && !a.redo[n]) w.qlen = 0;
    w.row_tiles = static_cast<int>((static_cast<long long>(w.qlen) * (a.Hq / a.Hkv) + 15) / 16);
    w.tile0 = 0;
    if (a.window > 0) w.tile0 = static_cast<int>(max(0ll, static_cast<long long>(w.kv) - w.qlen - a.window + 1) / 128);
    w.tiles = max(1, (w.kv + 127) / 128 - w.tile0);
    w.work = static_cast<long long>(a.Hkv) * w.row_tiles * (a.cluster > 1 ? 1 : w.tiles + kUnitCost);
    w.bad = bad;
    return w;
}

// Block `blk`'s share of the line of `nblocks` equal shares: tiles begin .. end - 1, of which the first is tile
// `off` of request n's.
struct Share {
    long long begin, end, off, per;
    int n;
};
// All THREADS threads call it; *out is shared memory and may be read afterwards.
template <int THREADS>
__device__ __forceinline__ void find_share(const AttnArgs &a, int blk, int nblocks, Share *out) {
    __shared__ long long s_sum[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_thread = (a.N + THREADS - 1) / THREADS;
    const int n0 = min(a.N, tid * per_thread), n1 = min(a.N, n0 + per_thread);
    long long own = 0;
    for (int n = n0; n < n1; ++n) {
        const ReqWork w = request_work(a, n);
        if (w.bad && blk == 0) atomicOr(a.err, kErrBadSeqlens);
        own += w.work;
    }
    long long inc = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    if (lane == 31) s_sum[warp] = inc;
    __syncthreads();
    long long before = inc - own, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    const long long per = max(1ll, (total + nblocks - 1) / nblocks);
    const long long begin = min(total, per * blk), end = min(total, begin + per);
    if (tid == 0) {
        out->begin = begin;
        out->end = end;
        out->per = per;
    }
    if (begin < end && begin >= before && begin < before + own) {
        long long at = before;
        int n = n0;
        for (; n < n1; ++n) {
            const long long w = request_work(a, n).work;
            if (begin < at + w) break;
            at += w;
        }
        out->n = n;
        out->off = begin - at;
    }
    __syncthreads();
}

// Whether phase `parity` is complete, without suspending the thread.
__device__ __forceinline__ bool mbar_test_wait(uint32_t b, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(b), "r"(parity)
        : "memory");
    return ok != 0;
}
// Wait for phase `parity`, at most about `limit` cycles. The first look does not suspend the thread, so that a
// limit shorter than the hardware's own suspension is kept too.
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity, long long limit) {
    const uint32_t b = ptx::smem_u32(bar);
    if (mbar_test_wait(b, parity)) return true;
    const long long t0 = clock64();
    do {
        if (clock64() - t0 > limit) return false;
    } while (!ptx::mbar_try_wait(b, parity));
    return true;
}

// 4 values of a row as fp32 (zeros for a null pointer)
__device__ __forceinline__ void load4(const float *p, float *f) {
    const float4 x = p ? __ldg(reinterpret_cast<const float4 *>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float *f) {
    const uint2 x = p ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
    f[0] = __uint_as_float(x.x << 16); f[1] = __uint_as_float(x.x & 0xffff0000u);
    f[2] = __uint_as_float(x.y << 16); f[3] = __uint_as_float(x.y & 0xffff0000u);
}

// Columns x .. x + N - 1 of the row (token, head): acc / l, zero where nothing was seen; column 0's thread
// writes lse = ln 2 (m + log2 l).
template <int N>
__device__ __forceinline__ void store_row(const AttnArgs &a, long long token, int head, int d, int x, const float (&acc)[N],
                                          float l, float m) {
    static_assert(N % 4 == 0, "whole vectors");
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const bool none = l == 0.f;
    const long long at = (token * a.Hq + head) * d + x;
    if (!in_bounds(at + N - 1, static_cast<long long>(a.T) * a.Hq * d, a.err)) return;
    if (a.out_bf16) {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(a.o) + at;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(none ? 0.f : acc[i] * inv, none ? 0.f : acc[i + 1] * inv);
            const __nv_bfloat162 q = __floats2bfloat162_rn(none ? 0.f : acc[i + 2] * inv, none ? 0.f : acc[i + 3] * inv);
            uint2 w;
            w.x = *reinterpret_cast<const uint32_t *>(&p);
            w.y = *reinterpret_cast<const uint32_t *>(&q);
            *reinterpret_cast<uint2 *>(o + i) = w;
        }
    } else {
        float *o = static_cast<float *>(a.o) + at;
#pragma unroll
        for (int i = 0; i < N; i += 4)
            st_global4(o + i, none ? make_float4(0.f, 0.f, 0.f, 0.f)
                                   : make_float4(acc[i] * inv, acc[i + 1] * inv, acc[i + 2] * inv, acc[i + 3] * inv));
    }
    if (x == 0 && a.lse)
        a.lse[token * a.Hq + head] = none ? -__builtin_huge_valf() : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace gdn
