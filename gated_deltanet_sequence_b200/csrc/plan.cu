// gdn_plan_batch: block tables, slot maps and packed offsets of a serving step.
//
// All integer work on a few thousand values, so the time is launches and dependent steps, not
// bytes. One block scans the requests (a shuffle scan, 1024 requests a turn), returns finished
// requests' blocks to the free list, takes new ones off it, and for steps of up to
// kInlineTokens tokens fills the per-token arrays as well; a larger step's tokens are filled by
// a second kernel over every SM. Lists of varying length (the table entries of finished
// requests, the new entries, the tokens) are walked flat: item i belongs to the request whose
// prefix range holds i, found by binary search in shared memory. That keeps one long prompt
// among many short ones from being one thread's loop. 256 requests of a decode step: 6.9 us; 24 prompts of
// 19500 tokens: 8.4 us (graph replays).
#include "common.cuh"
#include "tc_kernels.cuh"

namespace gdn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxN = 8192;

struct PlanArgs {
    const int *ctx, *add;
    int *table, *free_list, *free_count;
    int *cu, *kv, *pos, *seq, *slot, *info;
    int N, max_blocks, num_blocks, bs_log2, T;
};

// Exclusive block-wide prefix of x over kPlanThreads threads; *total: the sum. Meets twice.
template <typename V>
__device__ __forceinline__ V block_prefix(V x, V *total) {
    __shared__ V warp_sum[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    V inc = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
    }
    if (lane == 31) warp_sum[w] = inc;
    __syncthreads();
    V s = warp_sum[lane];
    const V own = s;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const V before = __shfl_sync(0xffffffffu, s - own, w);
    __syncthreads();
    return before + inc - x;
}

// The request whose range [pre[n], pre[n + 1]) holds i (0 <= i < pre[N]).
__device__ __forceinline__ int find_range(const int *pre, int N, int i) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void plan_token(const PlanArgs &a, const int *cu, int total, int t, bool may_be_short,
                                           unsigned *err) {
    int n = -1, p = -1, slot = -1;
    if (t < total) {
        n = find_range(cu, a.N, t);
        p = a.kv[n] - (cu[n + 1] - t);
        const long long at = static_cast<long long>(n) * a.max_blocks + (p >> a.bs_log2);
        const int b = in_bounds(at, static_cast<long long>(a.N) * a.max_blocks, err) ? a.table[at] : -1;
        if (b >= 0 && b < a.num_blocks) slot = (b << a.bs_log2) + (p & ((1 << a.bs_log2) - 1));
        else if (b >= a.num_blocks || !may_be_short) atomicOr(err, kErrBadSeqlens);
    }
    a.pos[t] = p;
    a.seq[t] = n;
    a.slot[t] = slot;
}

template <bool INLINE_TOKENS>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, unsigned *__restrict__ err) {
    extern __shared__ int sm[];
    int *tok = sm, *blk = sm + a.N + 1, *gone = blk + a.N + 1;   // prefixes of tokens and blocks; finished requests
    __shared__ int s_kvmax;
    if (!INLINE_TOKENS) cudaTriggerProgrammaticLaunchCompletion();   // the token kernel may take its place; it waits below
    const int tid = threadIdx.x, bs = 1 << a.bs_log2;
    const long long cap = static_cast<long long>(a.max_blocks) << a.bs_log2;
    int count = *a.free_count;
    if (count < 0 || count > a.num_blocks) {
        if (tid == 0) atomicOr(err, kErrBadSeqlens);
        count = 0;
    }
    if (tid == 0) s_kvmax = 0;
    __syncthreads();

    // ---- offsets: tokens and new table entries of each request. This is the only look at ctx: it may be kv itself (a step
    // that takes its cached lengths from the plan of the one before), so what follows takes the new tokens off kv.
    long long tokens = 0;
    int entries = 0, ngone = 0;
    for (int base = 0; base < a.N; base += kPlanThreads) {
        const int n = base + tid;
        int c = 0, add = 0, e = 0, kv = 0;
        bool fin = false;
        if (n < a.N) {
            c = a.ctx[n];
            add = a.add[n];
            fin = add == -1;
            if (add < -1 || (!fin && (c < 0 || static_cast<long long>(c) + add > cap))) {
                atomicOr(err, kErrBadSeqlens);
                c = add = 0;
            }
            if (fin) c = add = 0;
            kv = c + add;
            e = ((kv + bs - 1) >> a.bs_log2) - ((c + bs - 1) >> a.bs_log2);
        }
        long long sum;
        const long long before = tokens + block_prefix<long long>(add, &sum);
        // two counts in one prefix: new entries (low 32 bits; at most 2^27 a turn) and finished requests
        unsigned long long both;
        const unsigned long long pre =
            block_prefix<unsigned long long>(static_cast<unsigned>(e) | (static_cast<unsigned long long>(fin) << 48),
                                             &both);
        if (n < a.N) {
            tok[n] = static_cast<int>(min(before, 2147483647LL));
            blk[n] = entries + static_cast<int>(pre & 0xffffffffu);
            if (fin) gone[ngone + static_cast<int>(pre >> 48)] = n;
            a.kv[n] = kv;
            if (kv > 0) atomicMax(&s_kvmax, kv);
        }
        tokens += sum;
        entries += static_cast<int>(both & 0xffffffffu);
        ngone += static_cast<int>(both >> 48);
    }
    if (tokens > a.T) {     // uniform: the step does not fit its token grid, so it brings none
        __syncthreads();    // everyone's length is in s_kvmax
        if (tid == 0) { atomicOr(err, kErrBadSeqlens); s_kvmax = 0; }
        __syncthreads();
        tokens = 0;
        entries = 0;
        for (int n = tid; n < a.N; n += kPlanThreads) {
            const int c = a.kv[n] > 0 ? a.kv[n] - a.add[n] : 0;      // (0: finished, out of range, or nothing cached or new)
            tok[n] = 0;
            blk[n] = 0;
            a.kv[n] = c;
            if (c > 0) atomicMax(&s_kvmax, c);
        }
    }
    if (tid == 0) {
        tok[a.N] = static_cast<int>(tokens);
        blk[a.N] = entries;
    }
    __syncthreads();
    for (int n = tid; n <= a.N; n += kPlanThreads) a.cu[n] = tok[n];

    // ---- finished requests' blocks go on top of the free list, in (request, block) order
    const long long rows = static_cast<long long>(ngone) * a.max_blocks;
    const long long entry_count = static_cast<long long>(a.N) * a.max_blocks;      // (bounds checks of the debug build)
    for (long long base = 0; base < rows; base += 4 * kPlanThreads) {      // four entries a thread
        const long long i0 = base + 4 * tid;
        int b[4], have = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            b[k] = -1;
            if (i0 + k < rows) {
                const int g = static_cast<int>((i0 + k) / a.max_blocks);
                const long long place = static_cast<long long>(gone[g]) * a.max_blocks + (i0 + k - static_cast<long long>(g) * a.max_blocks);
                if (!in_bounds(place, entry_count, err)) continue;
                int *entry = a.table + place;
                b[k] = *entry;
                if (b[k] != -1) *entry = -1;
                if (b[k] < -1 || b[k] >= a.num_blocks) { atomicOr(err, kErrBadSeqlens); b[k] = -1; }
            }
            have += b[k] >= 0 ? 1 : 0;
        }
        int pushed;
        int at = count + block_prefix<int>(have, &pushed);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (b[k] >= 0) {
                if (at < a.num_blocks) {
                    if (in_bounds(at, a.num_blocks, err)) a.free_list[at] = b[k];
                }
                else atomicOr(err, kErrBadSeqlens);
                ++at;
            }
        count = min(count + pushed, a.num_blocks);
    }
    __syncthreads();

    // ---- new blocks come off it in the same order, all of them or none
    auto new_entry = [&](int i) {
        const int n = find_range(blk, a.N, i);
        const int first = (a.kv[n] - (tok[n + 1] - tok[n]) + bs - 1) >> a.bs_log2;
        const long long place = static_cast<long long>(n) * a.max_blocks + first + (i - blk[n]);
        return a.table + (in_bounds(place, entry_count, err) ? place : 0);
    };
    int want = 0, missing = 0;
    if (entries > kPlanThreads) {
        for (int base = 0; base < entries; base += kPlanThreads) {
            const int i = base + tid;
            want += __syncthreads_count(i < entries && *new_entry(i) < 0);
        }
        missing = max(0, want - count);
    }
    int taken = 0;
    for (int base = 0; base < entries && missing == 0; base += kPlanThreads) {
        const int i = base + tid;
        int *entry = i < entries ? new_entry(i) : nullptr;
        const bool need = entry && *entry < 0;
        int sum;
        const int r = block_prefix<int>(need ? 1 : 0, &sum);
        if (entries <= kPlanThreads) missing = max(0, sum - count);
        if (need && missing == 0) {
            const int place = count - 1 - taken - r;
            const int b = in_bounds(place, a.num_blocks, err) ? a.free_list[place] : -1;
            if (b >= 0 && b < a.num_blocks) *entry = b;
            else atomicOr(err, kErrBadSeqlens);
        }
        taken += sum;
    }
    if (missing == 0) count -= taken;
    __syncthreads();
    if (tid == 0) {
        *a.free_count = count;
        a.info[0] = static_cast<int>(tokens);
        a.info[1] = s_kvmax;
        a.info[2] = missing;
        a.info[3] = count;
    }
    if (INLINE_TOKENS)
        for (int t = tid; t < a.T; t += kPlanThreads)
            plan_token(a, tok, static_cast<int>(tokens), t, missing > 0, err);
}

__global__ void __launch_bounds__(256) plan_tokens_kernel(const PlanArgs a, unsigned *__restrict__ err) {
    cudaGridDependencySynchronize();
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t < a.T) plan_token(a, a.cu, a.cu[a.N], t, a.info[2] > 0, err);
}

}  // namespace

constexpr int kInlineTokens = 4096;

gdn_status_t launch_plan(const int *ctx, const int *add, int N, int *table, int max_blocks, int *free_list,
                         int *free_count, int num_blocks, int block_size, int T, int *cu, int *kv, int *pos, int *seq,
                         int *slot, int *info, cudaStream_t stream) {
    unsigned *err = device_error_word();
    if (!err) return GDN_ERR_CUDA;
    int lg = 0;
    while ((1 << lg) < block_size) ++lg;
    const PlanArgs a{ctx, add, table, free_list, free_count, cu, kv, pos, seq, slot, info, N, max_blocks, num_blocks, lg, T};
    const unsigned smem = static_cast<unsigned>((3 * N + 2) * sizeof(int));
    const bool one = T <= kInlineTokens;
    const void *fn = one ? reinterpret_cast<const void *>(plan_kernel<true>) : reinterpret_cast<const void *>(plan_kernel<false>);
    if (smem > 48 * 1024 && !ensure_smem_limit(fn, (3 * kPlanMaxN + 2) * sizeof(int))) return GDN_ERR_CUDA;
    if (one) {
        plan_kernel<true><<<1, kPlanThreads, smem, stream>>>(a, err);
        return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    }
    plan_kernel<false><<<1, kPlanThreads, smem, stream>>>(a, err);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(T) + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, plan_tokens_kernel, a, err) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
