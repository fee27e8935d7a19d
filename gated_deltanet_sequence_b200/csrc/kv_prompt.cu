// gdn_kv_attn, many rows a request (a prompt's chunk), bf16 queries and output: the same attention on the
// tensor cores' tcgen05 path.
//
// A block takes 256 rows (row R: token R / G, query head R % G of one KV head) as two groups of 128, each a
// 128-row UMMA tile, and walks the 128-token tiles of the cache that some row sees:
//   S = Q K^T   kind::f8f6f4: the cache's codes are the operand as TMA brings them; queries are the sum of
//               two e4m3 parts (row scaled by a power of two), so two products into one accumulator
//   P = 2^(S rk - m)   rk: row and block scale; m: a reference that moves only when a tile's weights sum past
//               kMaxSum, so that the accumulators are rarely rescaled; P as fp16 over S in tensor memory
//   O += P V    kind::f16: V's codes converted to fp16 in shared memory once for both groups, times the
//               block's scale over the unit's largest (a power of two: exact)
// Scores cannot be in fp32 here (two e4m3 parts hold a bf16 query exactly down to 2^-9 of its row's largest
// element, and within 2^-18 of it below), which is why other types take the few-rows kernel.
//
// What bounds it: per tile and group the two products take 1024 cycles of the tensor pipe and the 16384
// exponentials 1024 of the special-function units, so the two groups' softmax and products are interleaved:
// one group's exponentials run under the other's products. Four requests of 1000 to 2048 rows over 2048 to
// 6000 tokens, 32 query and 8 KV heads, d = 128 (428 GFLOP): 500 to 514 us, 850 TFLOP/s; the few-rows
// kernel takes 3417 us. A half tile takes 2200 cycles, of which 950 are waits, votes and tensor-memory
// turnarounds and 1270 the weights; neither pipe is the limit (without the exponentials 459 us).
//
// Warps: 0 K tiles and scales, 1-2 UMMA issue (2: tensor memory too), 3 V tiles, 4-7 V conversion, 8-11 and 12-15 the groups.
// Tensor memory: S (and P over it) of each group, O of each group, 512 columns at d = 128.
//
// Two inputs do not fit this scheme, and their request is left to the few-rows kernel, which runs after
// this one and computes it again: V scales of one unit more than 2^12 apart (fp16 would lose the small ones),
// and NaN codes in V (0 * NaN would reach rows that do not see them).
#include <algorithm>

#include "kv_attn.cuh"
#include "tc_ctl.cuh"

namespace gdn {
namespace {
using namespace ptx;

constexpr int kThreads = 512;
constexpr int kTok = 128, kHalf = 64;     // tokens of a tile; scores and weights go half by half
constexpr int kGroupRows = 128, kUnitRows = 256;
constexpr int kKStages = 3, kVStages = 3, kCStages = 2, kKsSlots = 8;   // K and V codes, fp16 V, K scales
constexpr float kMaxSum = 16384.f;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kMinScale = 7.888609052210118e-31f;      // 2^-100: a block of zeros
constexpr float kSpread = 4096.f;
constexpr float kMinNormal = 1.1754943508222875e-38f;    // 2^-126

enum : int {
    B_Q = 0,          // 8 warps: queries written
    B_KF = 1,         // [3] K tile in
    B_KE = 4,         // [3] both groups' products with it done
    B_VF = 7,         // [3] V codes in
    B_VE = 10,        // [3] converted
    B_CF = 13,        // [2] fp16 V written
    B_CE = 15,        // [2] both groups' products with it done
    B_S = 17,         // [2 groups][2 halves] scores done
    B_P = 21,         // [2 groups][2 halves] weights written, accumulators rescaled
    B_O = 25,         // [2 groups][2 halves] P V done
    B_END = 29,       // [2 groups] everything issued is done
    B_KS = 31,        // [8] K scales of a tile written
    B_VU = 39,        // V's unit known
    kNumBars = 40
};

template <int D> struct Lay {
    static constexpr uint32_t kTile8 = kTok * D, kTile16 = kTok * D * 2;
    static constexpr uint32_t OFF_Q = 0;                                  // [group][hi, lo] 128 x D
    static constexpr uint32_t OFF_K = 4 * kGroupRows * D;
    static constexpr uint32_t OFF_V8 = OFF_K + kKStages * kTile8;
    static constexpr uint32_t OFF_V = OFF_V8 + kVStages * kTile8;         // halves of 64 columns, 128 rows x 128 B
    static constexpr uint32_t OFF_KS = OFF_V + kCStages * kTile16;        // K scales of 16-token groups, and which exist
    static constexpr uint32_t OFF_BAR = OFF_KS + kKsSlots * 9 * 4;
    static constexpr uint32_t kBytes = OFF_BAR + kNumBars * 8 + 64;
    static constexpr uint32_t kAlloc = kBytes + 1024;
    static_assert(OFF_K % 1024 == 0 && OFF_V8 % 1024 == 0 && OFF_V % 1024 == 0 && OFF_BAR % 8 == 0, "alignment");
    static_assert(kAlloc <= 232448, "shared memory");
    static constexpr uint32_t TM_S = 0, TM_O = 256;                       // + 128 (S), + D (O) for the second group
};

// D[tmem] (+)= A[smem] B[smem]^T, e4m3 operands, fp32 accumulation
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);   // e4m3: 0
}
// K-major tile of D-byte rows: 128-byte swizzle at D = 128, 64-byte at D = 64
template <int D> __device__ __forceinline__ uint64_t kdesc(uint32_t addr) {
    uint64_t d = sdesc_sw128(addr, 16, 8 * D);
    if (D == 64) d = (d & ~(7ull << 61)) | (4ull << 61);
    return d;
}
// byte offset of 16-byte chunk c of row r in such a tile
template <int D> __device__ __forceinline__ uint32_t kswz(uint32_t r, uint32_t c) {
    return D == 128 ? sw128(r, c) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}
// Wait for this thread's tensor-memory loads; the values are tied to it, so that no use is moved before it.
__device__ __forceinline__ void tmem_wait_ld32(float (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                   "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                   "+f"(r[30]), "+f"(r[31])::"memory");
}
// Two fp32 values in a register pair, and Blackwell's two-wide fp32 instructions on them.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void e4m3_to_h2(uint32_t w, __half2 &lo, __half2 &hi) {
    uint32_t a, b;
    gdn::e4m3_to_h2(w, a, b);
    lo = *reinterpret_cast<const __half2 *>(&a);
    hi = *reinterpret_cast<const __half2 *>(&b);
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

// The request and row tile (of 256 rows) that block `idx` takes: tiles in falling order of the kv tile they end in, so
// that the longest units start first whatever the requests' lengths are, and the last blocks to run are the shortest
// (by request, the SMs that got one unit more than others took 15 % longer than the mean). A request's row tiles end
// later and later, so those that end in kv tile E or later are its last ones, counted in closed form; E is found by
// bisection over all requests.
struct Unit {
    int n, rt;
};
struct Rows {
    int rows, tiles, p0;     // rows (0: not for this kernel), row tiles, position of the first row
};
__device__ __forceinline__ Rows unit_rows(const AttnArgs &a, int n) {
    const ReqWork w = request_work(a, n, true);
    const int rows = w.many ? w.qlen * (a.Hq / a.Hkv) : 0;
    return Rows{rows, (rows + kUnitRows - 1) / kUnitRows, w.kv - w.qlen};
}
// first row tile of the request that ends in kv tile e or later (rows.tiles: none)
__device__ __forceinline__ int first_from(const Rows &q, int e, int G) {
    if (e <= 0) return 0;                // (rows before position 0 count as tile 0's)
    const long long need = static_cast<long long>(G) * (static_cast<long long>(e) * kTok - q.p0);     // last row >= need
    if (need <= 0) return 0;
    const long long t = (need + kUnitRows) / kUnitRows - 1;
    if (t < q.tiles - 1) return static_cast<int>(t);
    return q.rows - 1 >= need ? max(q.tiles - 1, 0) : q.tiles;
}
// Every warp finds it for itself (no barrier); lane i looks at requests i, i + 32, ...
__device__ __forceinline__ bool find_unit(const AttnArgs &a, int idx, Unit *out) {
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    const Rows none{0, 0, 0};
    const Rows q0 = lane < a.N ? unit_rows(a, lane) : none, q1 = lane + 32 < a.N ? unit_rows(a, lane + 32) : none;
    auto req = [&](int n) { return n == lane ? q0 : n == lane + 32 ? q1 : n < a.N ? unit_rows(a, n) : none; };
    auto from = [&](int e) {             // row tiles that end in kv tile e or later
        int c = (q0.tiles - first_from(q0, e, G)) + (q1.tiles - first_from(q1, e, G));
        for (int n = lane + 64; n < a.N; n += 32) {
            const Rows q = unit_rows(a, n);
            c += q.tiles - first_from(q, e, G);
        }
        return __reduce_add_sync(0xffffffffu, c);
    };
    // the largest e with more than idx tiles from it on
    int lo = 0, hi = a.max_blocks * a.bs / kTok + 1;
    if (from(0) <= idx) return false;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from(mid) > idx) lo = mid;
        else hi = mid;
    }
    int at = idx - from(lo + 1);         // among those that end in kv tile lo, in request order
    for (int base = 0; base < a.N; base += 32) {
        const Rows q = req(base + lane);
        const int f = first_from(q, lo, G), own = first_from(q, lo + 1, G) - f;
        int inc = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, at < inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            out->n = base + src;
            out->rt = __shfl_sync(0xffffffffu, f + at - (inc - own), src);
            return true;
        }
        at -= __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kv_prompt_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const AttnArgs a,
                 int *__restrict__ redo) {
    using L = Lay<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kNumBars);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    float *s_ks = reinterpret_cast<float *>(smem + L::OFF_KS);                       // [slot][8]
    uint32_t *s_have = reinterpret_cast<uint32_t *>(s_ks + kKsSlots * 8);            // [slot]
    __shared__ float s_vrange[4][2], s_vu;
    const Ctl ctl{bars, abort_flag, a.err, a.wait_limit};
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.Hq / a.Hkv, h = blockIdx.x % a.Hkv;

    if (tid == 0) {
        for (int b = 0; b < kNumBars; ++b)
            mbar_init(&bars[b], b == B_Q                                                          ? 8
                                : (b >= B_VE && b < B_CE) || (b >= B_P && b < B_O)                ? 4
                                : (b >= B_KE && b < B_VF) || (b >= B_CE && b < B_S)               ? 2
                                                                                                  : 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&mk);
        prefetch_tmap(&mv);
    }
    Unit u{};
    if (!find_unit(a, blockIdx.x / a.Hkv, &u)) return;
    const ReqWork rw = request_work(a, u.n, true);
    const int rows = rw.qlen * G, p0 = rw.kv - rw.qlen;
    // positions of each group's first and last row, and its tiles
    int pf[2], pl[2], ta[2], tb[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int r0 = u.rt * kUnitRows + g * kGroupRows, r1 = min(r0 + kGroupRows, rows) - 1;
        pf[g] = p0 + r0 / G;
        pl[g] = r1 >= r0 ? p0 + r1 / G : -1;
        tb[g] = pl[g] >= 0 ? pl[g] / kTok + 1 : 0;
        ta[g] = a.window > 0 ? min(tb[g], max(0, max(pf[g], -1) - a.window + 1) / kTok) : 0;
    }
    if (tb[1] == 0) ta[1] = tb[1] = tb[0];               // no rows: after the other's tiles
    if (tb[0] == 0) ta[0] = tb[0] = ta[1];
    const int t_a = ta[0], nt = tb[1] - ta[0];           // tiles t_a .. t_a + nt - 1
    const int t_hi = max(pl[0], pl[1]) + 1;
    const int *table = a.table + static_cast<long long>(u.n) * a.max_blocks;

    if (warp == 2) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // a warp's wait: most phases are complete when they are looked at, and the abort flag is looked at only in the others
    auto wait = [&](int b, uint32_t parity) {
        const bool now = mbar_test_wait(smem_u32(&bars[b]), parity);
        if (__all_sync(0xffffffffu, now)) return true;
        const bool ok = now || (!ctl.aborted() && (bounded_wait(&bars[b], parity, ctl.limit) || ctl.give_up()));
        return __all_sync(0xffffffffu, ok) != 0;
    };
    // The groups keep a row's 128 scores in registers: 256 threads take 192 each, the other 256 64 (65536 in all, what
    // the block was launched with)
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0 || warp == 3) {
        // ================================================================ TMA: K and its scales (warp 0), V (warp 3)
        const bool is_k = warp == 0;
        const CUtensorMap *map = is_k ? &mk : &mv;
        const int full = is_k ? B_KF : B_VF, empty = is_k ? B_KE : B_VE;
        const uint32_t ring = sb + (is_k ? L::OFF_K : L::OFF_V8);
        static_assert(kKStages == kVStages, "one ring depth");
        const int bl = a.bs >> 4;                        // 16-token groups of a block
        auto look = [&](int j) {                         // block of this lane's 16-token group of tile j
            const int t = (t_a + j) * kTok + 16 * lane;
            const int id = lane < 8 && j < nt && t < t_hi && in_bounds(t >> a.bs_log2, a.max_blocks, a.err) ? table[t >> a.bs_log2] : -1;
            return id < a.num_blocks ? id : -1;
        };
        int id_next = look(0), last = -1;
        bool ok = true;
        for (int j = 0; j < nt && ok; ++j) {
            const int id = id_next, t = (t_a + j) * kTok + 16 * lane, sl = j % kKStages;
            const float ks = is_k && id >= 0 ? a.k_scale[static_cast<long long>(id) * a.Hkv + h] : 1.f;
            id_next = look(j + 1);
            const bool box = id >= 0 && lane % bl == 0;
            const uint32_t boxes = __ballot_sync(0xffffffffu, box), have = __ballot_sync(0xffffffffu, id >= 0);
            const int row = ((id * a.Hkv + h) << a.bs_log2) + (t & (a.bs - 1));
            if (j >= kKStages) ok = wait(empty + sl, (j / kKStages - 1) & 1);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&bars[full + sl], __popc(boxes) * a.bs * D);
            __syncwarp();
            if (box) tma_load_2d(ring + sl * L::kTile8 + 16 * lane * D, map, &bars[full + sl], 0, row);
            if (is_k) {
                if (lane < 8) s_ks[(j % kKsSlots) * 8 + lane] = ks;
                if (lane == 0) s_have[j % kKsSlots] = have;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[B_KS + j % kKsSlots]);
            }
            last = j;
        }
        // never leave a copy in flight past the end of the block
        for (int j = max(0, last - kKStages + 1); j <= last; ++j) ctl.drain(full + j % kKStages, (j / kKStages) & 1);
    } else if (warp < 3) {
        // ================================================================ UMMA issue, a warp for each group
        // The whole warp runs the loop and one elected lane issues: in code the compiler knows to be uniform the
        // descriptors live in uniform registers (issued by a lane of a divergent branch, an instruction took 130
        // cycles for the pipe's 65). A wait costs a warp about 200 cycles even when there is nothing to wait for; with
        // a warp for each group, one group's products run meanwhile.
        const int g = warp - 1;
        constexpr uint32_t kIdS = idesc_e4m3(128, kHalf), kIdO = idesc_f16(128, D, false, true);
        const bool leader = elect_one();
        const uint32_t tsg = tmem + L::TM_S + g * 128, tog = tmem + L::TM_O + g * D;
        const uint64_t dq = kdesc<D>(sb + L::OFF_Q + g * 2 * kGroupRows * D), dk = kdesc<D>(sb + L::OFF_K);
        const uint64_t dv = sdesc_sw128(sb + L::OFF_V, 16384, 1024);
        const int j0 = ta[g] - t_a, j1 = tb[g] - t_a;    // this group's tiles
        auto scores = [&](int j, int hf) {               // S[hf] = Q K_j[hf]^T
            const uint64_t kd = dk + (j % kKStages) * (L::kTile8 >> 4) + ((hf * kHalf * D) >> 4);
            if (leader) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk)
                        mma_f8(tsg + hf * kHalf, dq + ((part * kGroupRows * D + kk * 32) >> 4), kd + 2 * kk, kIdS, part + kk > 0);
                mma_commit(&bars[B_S + 2 * g + hf]);
            }
            __syncwarp();
        };
        bool ok = nt > 0 && wait(B_Q, 0);
        // Tile by tile and half by half: P V, then the scores that take the same half of the next tile. These wait for the P V
        // just issued, which reads the weights in their place; meanwhile the group works on the other half.
        for (int j = -1; j < nt && ok; ++j) {
            const bool pv = j >= j0 && j < j1, qk = j + 1 >= j0 && j + 1 < j1;
            const int par = (j - j0) & 1;
            if (j >= 0) ok = wait(B_CF + j % kCStages, (j / kCStages) & 1);
            if (ok && j + 1 < nt) ok = wait(B_KF + (j + 1) % kKStages, ((j + 1) / kKStages) & 1);
            const uint64_t vd = dv + (j % kCStages) * (L::kTile16 >> 4);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (pv && ok) {
                    ok = wait(B_P + 2 * g + hf, par);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kHalf / 16; ++kk)
                            mma_f16_ts(tog, tsg + hf * kHalf + kk * 8, vd + (hf * (kHalf / 16) + kk) * 128, kIdO,
                                       j > j0 || hf > 0 || kk > 0);
                        mma_commit(&bars[B_O + 2 * g + hf]);
                    }
                    __syncwarp();
                }
                if (hf == 1 && ok && j >= 0 && leader) mma_commit(&bars[B_CE + j % kCStages]);   // through with V
                if (qk && ok) {
                    if (pv) ok = wait(B_O + 2 * g + hf, par);
                    if (!ok) break;
                    tc_fence_after();
                    scores(j + 1, hf);
                }
            }
            if (ok && j + 1 < nt && leader) mma_commit(&bars[B_KE + (j + 1) % kKStages]);        // through with K
            __syncwarp();
        }
        if (leader) {
            mma_commit(&bars[B_END + g]);
            ctl.drain(B_END + g, 0);
        }
    } else if (warp >= 4 && warp < 8) {
        // ================================================================ V: codes -> fp16, a token a thread
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        const int tk = tid - 128;
        // Its block's number is loaded two tiles ahead and the block's scale one tile ahead, both used no sooner: a load
        // that an instruction of the same tile waited for would hold up the conversion (1300 cycles a tile).
        auto block_of = [&](int j) {
            const int t = (t_a + j) * kTok + tk;
            return j < nt && t < t_hi && in_bounds(t >> a.bs_log2, a.max_blocks, a.err) ? table[t >> a.bs_log2] : -1;
        };
        auto scale_of = [&](int id) {
            return id >= 0 && id < a.num_blocks ? a.v_scale[static_cast<long long>(id) * a.Hkv + h] : -1.f;
        };
        // V's largest scale here is the unit that V is converted in; the smallest has to be within kSpread of it, or fp16
        // would lose its block. A block of zeros has the smallest scale that there is, which says nothing here; whether it is
        // one is seen when it is converted.
        float vu;
        {
            float mx = kMinScale, mn = __int_as_float(0x7f800000);
            const int b1 = (t_hi + a.bs - 1) >> a.bs_log2;
            for (int b = ((t_a * kTok) >> a.bs_log2) + tk; b < b1; b += 128) {
                const int id = table[b];
                if (id < 0 || id >= a.num_blocks) { atomicOr(a.err, kErrBadSeqlens); continue; }
                const float s = a.v_scale[static_cast<long long>(id) * a.Hkv + h];
                mx = fmaxf(mx, s);
                if (s > kMinScale) mn = fminf(mn, s);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            }
            if (lane == 0) { s_vrange[warp - 4][0] = mx; s_vrange[warp - 4][1] = mn; }
            named_bar(1, 128);
            vu = fmaxf(fmaxf(s_vrange[0][0], s_vrange[1][0]), fmaxf(s_vrange[2][0], s_vrange[3][0]));
            mn = fminf(fminf(s_vrange[0][1], s_vrange[1][1]), fminf(s_vrange[2][1], s_vrange[3][1]));
            if (tk == 0) {
                if (vu > kSpread * mn) redo[u.n] = 1;
                s_vu = vu;
                mbar_arrive(&bars[B_VU]);
            }
        }
        const float inv_vu = 1.f / vu;
        float s_next = scale_of(block_of(0));             // negative: the token does not exist
        int id_next = block_of(1);
        bool ok = true, leave = false;                    // leave: something that fp16 does not hold
        for (int j = 0; j < nt && ok; ++j) {
            const int sl = j % kVStages, csl = j % kCStages;
            const float s_raw = s_next;
            s_next = scale_of(id_next);
            id_next = block_of(j + 2);
            ok = wait(B_VF + sl, (j / kVStages) & 1);
            if (ok && j >= kCStages) ok = wait(B_CE + csl, (j / kCStages - 1) & 1);
            if (!ok) break;
            const bool e = s_raw >= 0.f;
            const float s = fmaxf(s_raw, 0.f) * inv_vu;   // exact: powers of two
            const __half2 f = __float2half2_rn(s);
            __half2 probe = __float2half2_rn(0.f);
            const uint8_t *src = smem + L::OFF_V8 + sl * L::kTile8;
            if (e && s < 1.f / kSpread) {                 // the smallest scale: a block of zeros, unless it holds something
                uint32_t any = 0u;
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(src + kswz<D>(tk, c));
                    any |= (w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
                }
                leave |= any != 0u;
            }
            uint8_t *dst = smem + L::OFF_V + csl * L::kTile16;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint4 w = *reinterpret_cast<const uint4 *>(src + kswz<D>(tk, c));
                if (!e) w = make_uint4(0u, 0u, 0u, 0u);  // rows that do not exist hold anything
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __half2 lo, hi;
                    e4m3_to_h2(x[i], lo, hi);
                    lo = __hmul2(lo, f);
                    hi = __hmul2(hi, f);
                    probe = __hfma2(lo, __float2half2_rn(0.f), probe);
                    probe = __hfma2(hi, __float2half2_rn(0.f), probe);
                    y[2 * i] = h2u(lo);
                    y[2 * i + 1] = h2u(hi);
                }
                // 16 columns: two chunks of the 64-column half c / 4
                uint8_t *half = dst + (c >> 2) * 16384;
                *reinterpret_cast<uint4 *>(half + sw128(tk, (2 * c) & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4 *>(half + sw128(tk, (2 * c + 1) & 7)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
            leave |= __half2float(__low2half(probe)) != 0.f || __half2float(__high2half(probe)) != 0.f;
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[B_CF + csl]);
                mbar_arrive(&bars[B_VE + sl]);
            }
        }
        if (leave) redo[u.n] = 1;
    } else if (warp >= 8) {
        // ================================================================ a group's rows, one a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int g = (warp - 8) >> 2, r = tid - 256 - g * 128;
        const int R = u.rt * kUnitRows + g * kGroupRows + r;
        const bool in = R < rows;
        const int tok = R / G;
        const long long token = rw.row0 + tok;
        const int head = h * G + (R - tok * G);
        const uint32_t trow = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + trow + L::TM_S + g * 128, to = tmem + trow + L::TM_O + g * D;
        float rf;
        {
            const uint4 *qp = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + token * a.q_stride +
                                                              static_cast<long long>(head) * D);
            uint4 w[D / 8];
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                w[i] = in ? __ldg(qp + i) : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x[k] << 16)), fabsf(__uint_as_float(x[k] & 0xffff0000u))));
            }
            const uint32_t ub = __float_as_uint(mx);
            int e = static_cast<int>(ub >> 23) - 127 - 8 + ((ub & 0x7fffffu) > 0x600000u ? 1 : 0);
            e = mx == 0.f || ub >= 0x7f800000u ? 0 : min(max(e, -100), 126);
            // the score factor is kept positive (a negative scale goes into the query), so that a column group's
            // largest product is also its largest score
            const float inv = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), a.scale_log2);
            rf = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            uint8_t *qh = smem + L::OFF_Q + g * 2 * kGroupRows * D, *ql = qh + kGroupRows * D;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t x0 = k < 2 ? (k == 0 ? w[2 * c].x : w[2 * c].z) : (k == 2 ? w[2 * c + 1].x : w[2 * c + 1].z);
                    const uint32_t x1 = k < 2 ? (k == 0 ? w[2 * c].y : w[2 * c].w) : (k == 2 ? w[2 * c + 1].y : w[2 * c + 1].w);
                    float y[4] = {__uint_as_float(x0 << 16) * inv, __uint_as_float(x0 & 0xffff0000u) * inv,
                                  __uint_as_float(x1 << 16) * inv, __uint_as_float(x1 & 0xffff0000u) * inv};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (fabsf(y[i]) > 448.f) y[i] = __int_as_float(0x7fffffff);      // an infinite query shows as NaN
                    hi[k] = e4m3x4(y);
                    __half2 p, q;
                    e4m3_to_h2(hi[k], p, q);
                    const float2 pf2 = __half22float2(p), qf2 = __half22float2(q);
                    const float z[4] = {y[0] - pf2.x, y[1] - pf2.y, y[2] - qf2.x, y[3] - qf2.y};
                    lo[k] = e4m3x4(z);
                }
                *reinterpret_cast<uint4 *>(qh + kswz<D>(r, c)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4 *>(ql + kswz<D>(r, c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_Q]);
        }
        const int hi = in ? p0 + tok : -1, lo = a.window > 0 ? max(hi, -1) - a.window + 1 : 0;
        const int lo_last = a.window > 0 ? max(pl[g], -1) - a.window + 1 : 0;
        float m = kNegInf, l = 0.f;
        int done = 0;                                    // tiles of this group so far
        bool ok = true;
        for (int i = 2 * ta[g]; i < 2 * tb[g] && ok; ++i) {              // half tiles
            const int tile = i >> 1, hf = i & 1, j = tile - t_a, t0 = i * kHalf, slot = j % kKsSlots;
            done = tile - ta[g];
            ok = wait(B_KS + slot, (j / kKsSlots) & 1) && wait(B_S + 2 * g + hf, done & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t have = (s_have[slot] >> (4 * hf)) & 0xfu, tsh = ts + hf * kHalf;
            const bool edge = have != 0xfu || t0 + kHalf - 1 > pf[g] || t0 < lo_last;
            const int c_hi = hi - t0, c_lo = lo - t0;    // columns this row sees
            float k[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) k[q] = fmaxf(rf * s_ks[slot * 8 + 4 * hf + q], kMinNormal);   // never 0: -inf stays -inf
            // Weights against the row's reference m. m is the largest exponent of the row's first half tile with something
            // to see, and stays while a half tile's weights sum to at most kMaxSum (then none of them is beyond
            // fp16): the sum is there anyway, so most half tiles need no maximum, and their accumulators no rescaling.
            uint32_t p[kHalf / 2];
            float sum;
            auto mask = [&](float (&s)[32], int ch) {
#pragma unroll
                for (int c = 32 * ch; c < 32 * ch + 32; ++c)
                    s[c & 31] = c <= c_hi && c >= c_lo && ((have >> (c >> 4)) & 1u) ? s[c & 31] : kNegInf;
            };
            auto weights = [&]() {                       // 32 scores at a time, the next 32 on their way
                const float base = m == kNegInf ? 0.f : m;
                float s[2][32];
                uint64_t part[2] = {0, 0};               // two running sums each
                tmem_ld32(tsh, s[0]);
#pragma unroll
                for (int ch = 0; ch < kHalf / 32; ++ch) {
                    float(&cur)[32] = s[ch & 1];
                    tmem_wait_ld32(cur);
                    if (ch < kHalf / 32 - 1) tmem_ld32(tsh + 32 * (ch + 1), s[(ch + 1) & 1]);
                    if (edge) mask(cur, ch);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float kk = k[2 * ch + (c >> 4)];
                        const uint64_t x = fma2(pair(cur[c], cur[c + 1]), pair(kk, kk), pair(-base, -base));
                        const uint64_t e = pair(ex2(lo2(x)), ex2(hi2(x)));
                        part[(c >> 1) & 1] = add2(part[(c >> 1) & 1], e);
                        p[16 * ch + (c >> 1)] = pack_h2(lo2(e), hi2(e));
                    }
                }
                const uint64_t t = add2(part[0], part[1]);
                sum = lo2(t) + hi2(t);
            };
            const bool none = m == kNegInf;
            weights();
            if (__any_sync(0xffffffffu, (none && in) || sum > kMaxSum)) {
                float top = kNegInf, f = 1.f;
#pragma unroll 1
                for (int ch = 0; ch < kHalf / 32; ++ch) {
                    float s[32];
                    tmem_ld32(tsh + 32 * ch, s);
                    tmem_wait_ld32(s);
                    if (edge) mask(s, ch);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float x[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = fmaxf(s[16 * q + c], s[16 * q + 8 + c]);
#pragma unroll
                        for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
                            for (int c = 0; c < w; ++c) x[c] = fmaxf(x[c], x[c + w]);
                        if (x[0] > kNegInf) top = fmaxf(top, x[0] * fmaxf(rf * s_ks[slot * 8 + 4 * hf + 2 * ch + q], kMinNormal));
                    }
                }
                if (top > m) {
                    f = none ? 0.f : ex2(m - top);
                    m = top;
                    l *= f;
                }
                if (i > 2 * ta[g]) {                     // rescale the row's accumulators: P V before this must be done
                    const int b = i - 1;
                    ok = wait(B_O + 2 * g + (b & 1), ((b >> 1) - ta[g]) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < D / 16; ++ch) {
                        float o[16];
                        tmem_ld16(to + 16 * ch, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 16; ++c) o[c] *= f;
                        tmem_st16(to + 16 * ch, o);
                    }
                }
                weights();
            }
            tmem_st16u(tsh, p);
            tmem_st16u(tsh + 16, p + 16);
            l += sum;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[B_P + 2 * g + hf]);
        }
        done = tb[g] - ta[g];
        if (ok && done > 0) ok = wait(B_O + 2 * g + 1, (done - 1) & 1);
        tc_fence_after();
        ok = ok && wait(B_VU, 0);
        const float inv = l == 0.f ? 0.f : s_vu / l;
        __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.o) + (token * a.Hq + head) * D;
        if (ok) {
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
                float o[32];
                if (done > 0) {
                    tmem_ld32(to + 32 * ch, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(l == 0.f ? 0.f : o[i + 2 * k] * inv,
                                                                       l == 0.f ? 0.f : o[i + 2 * k + 1] * inv);
                        w[k] = *reinterpret_cast<const uint32_t *>(&b);
                    }
                    if (in && in_bounds((token * a.Hq + head) * D + 32 * ch + i + 7, static_cast<long long>(a.T) * a.Hq * D, a.err))
                        *reinterpret_cast<uint4 *>(op + 32 * ch + i) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (in && a.lse) a.lse[token * a.Hq + head] = l == 0.f ? kNegInf : 0.6931471805599453f * (m + log2f(l));
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

template <int D>
gdn_status_t launch_t(const CUtensorMap &mk, const CUtensorMap &mv, const AttnArgs &a, int *redo, cudaStream_t stream) {
    auto kern = kv_prompt_kernel<D>;
    if (!ensure_smem_limit(reinterpret_cast<const void *>(kern), Lay<D>::kAlloc)) return GDN_ERR_CUDA;
    // no more units than this, whatever the lengths are: a request that comes here has more than many_rows rows
    const long long all = static_cast<long long>(a.T) * (a.Hq / a.Hkv);
    const long long units = (all / kUnitRows + std::min<long long>(a.N, all / a.many_rows)) * a.Hkv;
    if (units > 2147483647ll) return GDN_ERR_UNSUPPORTED;
    if (units == 0) return GDN_OK;         // fewer rows in all than one such request has
    if (cudaMemsetAsync(redo, 0, static_cast<size_t>(a.N) * sizeof(int), stream) != cudaSuccess) return GDN_ERR_CUDA;
    kern<<<static_cast<unsigned>(units), kThreads, Lay<D>::kAlloc, stream>>>(mk, mv, a, redo);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

gdn_status_t launch_kv_prompt(const void *kc, const void *vc, const AttnArgs &a, int d, int *redo, cudaStream_t stream) {
    const long long rows = static_cast<long long>(a.num_blocks) * a.Hkv * a.bs;
    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, kc, rows, d, a.bs) || !make_cache_map(&mv, vc, rows, d, a.bs)) return GDN_ERR_CUDA;
    return d == 128 ? launch_t<128>(mk, mv, a, redo, stream) : launch_t<64>(mk, mv, a, redo, stream);
}

}  // namespace gdn
