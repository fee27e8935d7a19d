// gdn_kv_append: new K and V rows into the paged 8-bit cache, one power-of-two scale for each
// block of tokens and head.
//
//   scale = 2^e, the smallest with max |x| <= 448 * 2^e;   code = e4m3(x / scale)
// The scale is a power of two because e4m3 is a float: its relative step does not depend on the
// scale, so a finer scale would buy less than a binade of range, while with powers of two x /
// scale and the rescaling of codes already there are exact (until they fall below the smallest
// normal, 2^-6), and appending a prompt in pieces gives what appending it at once gives.
//
// The unit of work is a run: consecutive rows that go to consecutive cache rows of one block,
// for one head of K or V. One pass: the run's values stay in registers between the maximum and
// the codes. A block of 256 threads looks over R rows and takes the runs that start there: runs
// that a warp holds in a few registers (decode: one row) go one to a warp, longer ones (prompts)
// to the whole block. DRAM bytes bound it: rows in, codes out. 24 prompts of 157 to 4096 rows, 16 heads, d =
// 128 (386 MB): 82 us, 4.7 TB/s; a run's codes wait for its maximum, so a block's next run is loaded
// meanwhile (without that, and one head a block, 186 us).
#include "common.cuh"
#include "tc_kernels.cuh"

namespace gdn {
namespace {

constexpr int kAppThreads = 256, kAppWarps = kAppThreads / 32;
constexpr int kMaxRows = 64, kMaxBs = 128;
constexpr int kMaskWords = (kMaxRows + kMaxBs + 31) / 32;
constexpr int kScaleExpMin = -100;
constexpr int kWarpSteps = 4;   // a warp's run: at most 4 chunks of 8 values a lane

struct AppArgs {
    const void *x[2];
    long long stride[2];
    uint8_t *cache[2];
    float *scale[2];
    const int *slot;
    int T, H, bs_log2, num_blocks;
    int R, HG;                 // rows and heads of a block
};

// 8 values (one chunk) of a row, as fp32
template <typename IT> struct Chunk;
template <> struct Chunk<__nv_bfloat16> {
    uint4 w;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
    // bits of the largest magnitude, as fp32 (NaN and infinities count)
    __device__ __forceinline__ uint32_t top() const {
        const uint32_t m = 0x7fff7fffu;
        const uint32_t t = __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
        return max(t & 0xffff0000u, t << 16);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};
template <> struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const float4 *>(p));
        b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ uint32_t top() const {
        float f[8];
        get(f);
        uint32_t t = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(f[i]) & 0x7fffffffu);
        return t;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// bits of the largest finite magnitude: for runs that hold NaN or an infinity, where top() says that
constexpr uint32_t kInfBits = 0x7f800000u;
template <typename IT>
__device__ __noinline__ uint32_t finite_top(const Chunk<IT> &c) {
    float f[8];
    c.get(f);
    uint32_t m = 0u;
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = __float_as_uint(f[i]) & 0x7fffffffu;
        m = u < kInfBits ? max(m, u) : m;
    }
    return m;
}

// exponent of the smallest power of two s, >= 2^kScaleExpMin, with amax <= 448 s: amax = 1.f *
// 2^(E - 127) and 448 = 1.75 * 2^8
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return amax > 0.f ? max(e, kScaleExpMin) : kScaleExpMin;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// two fp32 -> two e4m3 (nearest even; beyond 448 to 448; NaN to NaN), lo in the low byte
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w)));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Codes of a chunk, at cache[at]; inv is a power of two, so the products are exact. odd: the run holds NaN or an
// infinity; an infinity would be taken to 448 and is stored as NaN instead, so that it shows.
template <typename IT>
__device__ __forceinline__ void store_codes(uint8_t *cache, long long at, long long n, const Chunk<IT> &c, float inv, bool odd,
                                            unsigned *err) {
    if (!in_bounds(at, n - 7, err)) return;
    float f[8];
    c.get(f);
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(f[i]) == __uint_as_float(kInfBits)) f[i] = __int_as_float(0x7fffffff);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint64_t x[2], y;                    // two-wide products
        asm("mov.b64 %0, {%1, %1};" : "=l"(y) : "f"(inv));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            asm("mov.b64 %0, {%1, %2};" : "=l"(x[k]) : "f"(f[4 * i + 2 * k]), "f"(f[4 * i + 2 * k + 1]));
            asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x[k]) : "l"(y));
        }
        // both pairs' codes into one word
        asm("{\n\t.reg .f32 a, b, c, d;\n\t.reg .b16 p, q;\n\t"
            "mov.b64 {a, b}, %1;\n\tmov.b64 {c, d}, %2;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 p, b, a;\n\tcvt.rn.satfinite.e4m3x2.f32 q, d, c;\n\t"
            "mov.b32 %0, {p, q};\n\t}"
            : "=r"(w[i])
            : "l"(x[0]), "l"(x[1]));
    }
    *reinterpret_cast<uint2 *>(cache + at) = make_uint2(w[0], w[1]);
}

// The scale of a run's block: fresh blocks take what the run needs, others the larger of that
// and their own.
__device__ __forceinline__ float run_scale(float amax, bool fresh, float old) {
    const float fit = exp2i(scale_exp(amax));
    return fresh || !(old >= fit) ? fit : old;
}

// Codes of the block's earlier rows, `bytes` of them, times ratio (a power of two below 1);
// threads t of nt.
__device__ __forceinline__ void rescale_codes(uint8_t *p, int bytes, float ratio, int t, int nt) {
    for (int i = t * 8; i < bytes; i += nt * 8) {
        uint2 w = *reinterpret_cast<const uint2 *>(p + i);
        uint32_t u[2] = {w.x, w.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 a = from_e4m3x2(u[j] & 0xffffu), b = from_e4m3x2(u[j] >> 16);
            u[j] = to_e4m3x2(a.x * ratio, a.y * ratio) | (to_e4m3x2(b.x * ratio, b.y * ratio) << 16);
        }
        *reinterpret_cast<uint2 *>(p + i) = make_uint2(u[0], u[1]);
    }
}

// MB: the largest block size (64 or 128): a thread holds MB * D / 8 / 256 chunks of a long run, twice (the next item's
// values are on their way while one is reduced and coded).
template <int D, int MB, typename IT>
__global__ void __launch_bounds__(kAppThreads, (MB == 64 && sizeof(IT) == 2 ? 4 : 2))
kv_append_kernel(const AppArgs a, unsigned *__restrict__ err) {
    constexpr int CPR = D / 8;                           // chunks a row
    constexpr int STEPS = MB * CPR / kAppThreads;        // chunks a thread of a block's longest run
    __shared__ int s_slot[kMaxRows + kMaxBs];
    __shared__ uint32_t s_brk[kMaskWords];
    __shared__ int s_long[kMaxRows], s_short[kMaxRows], s_nlong, s_nshort;
    __shared__ uint32_t s_max[2][kAppWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h0 = blockIdx.y * a.HG, nh = min(a.HG, a.H - h0), z = blockIdx.z, bs = 1 << a.bs_log2;
    const long long r0 = static_cast<long long>(blockIdx.x) * a.R;
    const int nslots = a.num_blocks << a.bs_log2;
    const IT *x = static_cast<const IT *>(z ? a.x[1] : a.x[0]);
    const long long stride = z ? a.stride[1] : a.stride[0];
    uint8_t *cache = z ? a.cache[1] : a.cache[0];
    float *scale = z ? a.scale[1] : a.scale[0];
    const long long ncodes = static_cast<long long>(nslots) * a.H * D;      // (bounds checks of the debug build)

    // slots of this block's rows and of the rows a run may reach past them; a bit where a run starts
    // (or a row that is skipped, or the end)
    const int span = a.R + bs;
    if (tid == 0) s_nlong = s_nshort = 0;
    for (int base = 0; base < ((span + 31) & ~31); base += kAppThreads) {
        const int i = base + tid;
        const long long r = r0 + i;
        int s = -1, prev = -1;
        if (i < span && r < a.T) {
            s = a.slot[r];
            if (r > 0) prev = a.slot[r - 1];
            if (s < -1 || s >= nslots) {
                if (i < a.R && h0 == 0 && z == 0) atomicOr(err, kErrBadSeqlens);
                s = -1;
            }
        }
        const bool starts = s < 0 || prev < 0 || s != prev + 1 || (s & (bs - 1)) == 0 || r == 0;
        if (i < span) s_slot[i] = s;
        const unsigned bits = __ballot_sync(0xffffffffu, starts);
        if (lane == 0 && (base >> 5) + warp < kMaskWords) s_brk[(base >> 5) + warp] = bits;
    }
    __syncthreads();
    if (tid < a.R && s_slot[tid] >= 0 && ((s_brk[tid >> 5] >> (tid & 31)) & 1u)) {
        // rows to the next start: at most bs, since a block's first row starts a run
        int w = tid >> 5;
        uint32_t m = (tid & 31) == 31 ? 0u : s_brk[w] & (0xfffffffeu << (tid & 31));
        while (m == 0 && 32 * (w + 1) < span) m = s_brk[++w];
        const int end = m ? min(32 * w + __ffs(m) - 1, span) : span;
        const int len = end - tid;
        const int id = tid | (len << 8);
        if (len * CPR <= 32 * kWarpSteps) s_short[atomicAdd(&s_nshort, 1)] = id;
        else s_long[atomicAdd(&s_nlong, 1)] = id;
    }
    __syncthreads();

    // ---- long runs, head by head: the whole block. Items (run, head) in order; `it` holds an item's place.
    struct Item {
        int run, head;
    };
    const int nlong = s_nlong, nshort = s_nshort * nh;
    auto next = [&](Item &it) {
        if (++it.head == nh) {
            it.head = 0;
            ++it.run;
        }
    };
    auto load_long = [&](const Item &it, Chunk<IT> (&c)[STEPS]) {
        const int run = s_long[it.run], i0 = run & 255, len = run >> 8;
        const IT *row = x + (r0 + i0 + tid / CPR) * stride + (h0 + it.head) * D + (tid % CPR) * 8;
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
            if (tid / CPR + j * (kAppThreads / CPR) < len) c[j].load(row + j * (kAppThreads / CPR) * stride);
            else c[j].zero();
        }
    };
    int turn = 0;
    auto block_max = [&](uint32_t v) {
        v = __reduce_max_sync(0xffffffffu, v);
        if (lane == 0) s_max[turn][warp] = v;
        __syncthreads();      // (and the item before is through with the other s_max)
        v = __reduce_max_sync(0xffffffffu, s_max[turn][lane & (kAppWarps - 1)]);
        turn ^= 1;
        return v;
    };
    auto code_long = [&](const Item &it, const Chunk<IT> (&c)[STEPS]) {
        const int run = s_long[it.run], i0 = run & 255, len = run >> 8;
        const int slot = s_slot[i0], off = slot & (bs - 1);
        const long long bh = static_cast<long long>(slot >> a.bs_log2) * a.H + h0 + it.head;
        const float old = off > 0 ? scale[bh] : 0.f;
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < STEPS; ++j) m = max(m, c[j].top());
        m = block_max(m);
        const bool odd = m >= kInfBits;
        if (odd) {                // rare: the scale goes by the finite ones
            m = 0u;
#pragma unroll
            for (int j = 0; j < STEPS; ++j) m = max(m, finite_top(c[j]));
            m = block_max(m);
        }
        const float sc = run_scale(__uint_as_float(m), off == 0, old);
        const float inv = exp2i(127 - static_cast<int>(__float_as_uint(sc) >> 23));
        const long long blk0 = (bh << a.bs_log2) * D;          // the block's first code
#pragma unroll
        for (int j = 0; j < STEPS; ++j)
            if (tid / CPR + j * (kAppThreads / CPR) < len)
                store_codes(cache, blk0 + off * D + (tid + j * kAppThreads) * 8, ncodes, c[j], inv, odd, err);
        if (off > 0 && sc != old && in_bounds(blk0 + off * D - 1, ncodes, err))
            rescale_codes(cache + blk0, off * D, old * inv, tid, kAppThreads);
        // everyone has read the old scale: each did before the barrier above
        if (tid == 0 && (off == 0 || sc != old)) scale[bh] = sc;
    };
    {
        Chunk<IT> c[STEPS], ahead[STEPS];
        Item it{0, 0};
        if (nlong > 0) load_long(it, ahead);
        while (it.run < nlong) {
            const Item now = it;
#pragma unroll
            for (int j = 0; j < STEPS; ++j) c[j] = ahead[j];
            next(it);
            if (it.run < nlong) load_long(it, ahead);
            code_long(now, c);
        }
    }

    // ---- short runs: one, of one head, to a warp
    for (int e = warp; e < nshort; e += kAppWarps) {
        const int run = s_short[e / nh], i0 = run & 255, len = run >> 8;
        const int slot = s_slot[i0], off = slot & (bs - 1), h = h0 + e % nh;
        const long long bh = static_cast<long long>(slot >> a.bs_log2) * a.H + h;
        const float old = off > 0 ? scale[bh] : 0.f;
        Chunk<IT> w[kWarpSteps];
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < kWarpSteps; ++j) {
            const int id = lane + j * 32;
            if (id < len * CPR) w[j].load(x + (r0 + i0 + id / CPR) * stride + h * D + (id % CPR) * 8);
            else w[j].zero();
        }
#pragma unroll
        for (int j = 0; j < kWarpSteps; ++j) m = max(m, w[j].top());
        m = __reduce_max_sync(0xffffffffu, m);
        const bool odd = m >= kInfBits;
        if (odd) {
            m = 0u;
#pragma unroll
            for (int j = 0; j < kWarpSteps; ++j) m = max(m, finite_top(w[j]));
            m = __reduce_max_sync(0xffffffffu, m);
        }
        const float sc = run_scale(__uint_as_float(m), off == 0, old);
        const float inv = exp2i(127 - static_cast<int>(__float_as_uint(sc) >> 23));
        const long long blk0 = (bh << a.bs_log2) * D;          // the block's first code
#pragma unroll
        for (int j = 0; j < kWarpSteps; ++j) {
            const int id = lane + j * 32;
            if (id < len * CPR) store_codes(cache, blk0 + off * D + id * 8, ncodes, w[j], inv, odd, err);
        }
        if (off > 0 && sc != old && in_bounds(blk0 + off * D - 1, ncodes, err))
            rescale_codes(cache + blk0, off * D, old * inv, lane, 32);
        __syncwarp();
        if (lane == 0 && (off == 0 || sc != old)) scale[bh] = sc;
    }
}

template <int D, typename IT>
void launch_app(const AppArgs &a, dim3 grid, unsigned *err, cudaStream_t stream) {
    if (a.bs_log2 <= 6) kv_append_kernel<D, 64, IT><<<grid, kAppThreads, 0, stream>>>(a, err);
    else kv_append_kernel<D, 128, IT><<<grid, kAppThreads, 0, stream>>>(a, err);
}

}  // namespace

gdn_status_t launch_kv_append(const void *k, const void *v, long long ks, long long vs, const int *slot, void *kc,
                              void *vc, float *ksc, float *vsc, int T, int H, int d, int num_blocks, int block_size,
                              gdn_dtype_t in_dtype, cudaStream_t stream) {
    unsigned *err = device_error_word();
    if (!err) return GDN_ERR_CUDA;
    int lg = 0;
    while ((1 << lg) < block_size) ++lg;
    AppArgs a{{k, v}, {ks, vs}, {static_cast<uint8_t *>(kc), static_cast<uint8_t *>(vc)}, {ksc, vsc}, slot, T, H, lg,
              num_blocks, 0, 0};
    // Prompts: 64 rows and four heads a block, whose items follow each other without a pause. Few rows: 8 rows and one
    // head, for more blocks.
    a.R = T >= 4096 ? kMaxRows : kAppWarps;
    a.HG = T >= 4096 ? 4 : 1;
    const dim3 grid(static_cast<unsigned>((T + a.R - 1) / a.R), static_cast<unsigned>((H + a.HG - 1) / a.HG), 2);
    if (in_dtype == GDN_F32) {
        if (d == 128) launch_app<128, float>(a, grid, err, stream);
        else launch_app<64, float>(a, grid, err, stream);
    } else {
        if (d == 128) launch_app<128, __nv_bfloat16>(a, grid, err, stream);
        else launch_app<64, __nv_bfloat16>(a, grid, err, stream);
    }
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
