// C-ABI entry points of the serving calls: argument validation and dispatch.
#include <math.h>

#include "kv_attn.cuh"

namespace gdn {
gdn_status_t launch_plan(const int *ctx, const int *add, int N, int *table, int max_blocks, int *free_list,
                         int *free_count, int num_blocks, int block_size, int T, int *cu, int *kv, int *pos, int *seq,
                         int *slot, int *info, cudaStream_t stream);
gdn_status_t launch_kv_append(const void *k, const void *v, long long ks, long long vs, const int *slot, void *kc,
                              void *vc, float *ksc, float *vsc, int T, int H, int d, int num_blocks, int block_size,
                              gdn_dtype_t in_dtype, cudaStream_t stream);
size_t kv_attn_ws_bytes(int N, int d);
gdn_status_t launch_kv_attn(const void *kc, const void *vc, AttnArgs a, int d, bool in_f32, bool out_f32,
                            cudaStream_t stream);
gdn_status_t launch_decode_slots(const void *q, const void *k, const void *v, long long qs, long long ks, long long vs,
                                 const float *beta, const float *g, float *state, const int *slots, const int *cu,
                                 void *o, int N, int T, int Hk, int Hv, int n_slots, int dk, int dv, float scale,
                                 gdn_dtype_t in_dtype, const FwdOpts &oo, cudaStream_t stream);
bool set_fwd_opts(const gdn_fwd_opts_t &opts, bool has_g, FwdOpts *oo);   // api.cu
}  // namespace gdn

namespace {

bool al(const void *p, unsigned n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool al_opt(const void *p, unsigned n) { return !p || al(p, n); }
bool dtype_ok(gdn_dtype_t t) { return t == GDN_F32 || t == GDN_BF16; }
long long esize(gdn_dtype_t t) { return t == GDN_BF16 ? 2 : 4; }
bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128; }
bool head_ok(int d) { return d == 64 || d == 128; }
constexpr long long kMaxRows = 1ll << 30, kInt = 2147483647ll;
// Positions of gdn_kv_attn: its kernels look a few thousand positions past a context's end in 32 bits.
constexpr long long kMaxContext = kInt - 65535;
// rows of `width` elements, `stride` apart, T of them: 16-byte vectors stay aligned and offsets fit
bool stride_ok(long long stride, long long width, gdn_dtype_t t) {
    return stride >= width && stride <= (1ll << 40) && (stride * esize(t)) % 16 == 0;
}

}  // namespace

extern "C" {

gdn_status_t gdn_plan_batch(const int *ctx_lens, const int *new_lens, int N, int *block_table, int max_blocks,
                            int *free_list, int *free_count, int num_blocks, int block_size, int T, int *cu_seqlens,
                            int *kv_lens, int *positions, int *seq_ids, int *slot_map, int *info, void *cuda_stream) {
    if (N < 1 || T < 0 || max_blocks < 1 || num_blocks < 1) return GDN_ERR_INVALID_ARG;
    if (!al(ctx_lens, 4) || !al(new_lens, 4) || !al(block_table, 4) || !al(free_list, 4) || !al(free_count, 4) ||
        !al(cu_seqlens, 4) || !al(kv_lens, 4) || !al(info, 4))
        return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!al(positions, 4) || !al(seq_ids, 4) || !al(slot_map, 4))) return GDN_ERR_INVALID_ARG;
    if (!block_size_ok(block_size) || N > 8192 || T > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * block_size > kInt || static_cast<long long>(max_blocks) * block_size > kInt)
        return GDN_ERR_INVALID_ARG;
    return gdn::launch_plan(ctx_lens, new_lens, N, block_table, max_blocks, free_list, free_count, num_blocks,
                            block_size, T, cu_seqlens, kv_lens, positions, seq_ids, slot_map, info,
                            static_cast<cudaStream_t>(cuda_stream));
}

gdn_status_t gdn_kv_append(const void *k, const void *v, long long k_stride, long long v_stride, const int *slot_map,
                           void *k_cache, void *v_cache, float *k_scale, float *v_scale, int T, int Hkv, int d,
                           int num_blocks, int block_size, gdn_dtype_t in_dtype, void *cuda_stream) {
    if (T < 0 || Hkv < 1 || num_blocks < 1 || !dtype_ok(in_dtype)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(d) || !block_size_ok(block_size) || Hkv > 65535 || T > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * block_size > kInt) return GDN_ERR_INVALID_ARG;
    if (!al(k_cache, 16) || !al(v_cache, 16) || !al(k_scale, 4) || !al(v_scale, 4)) return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    const long long width = static_cast<long long>(Hkv) * d;
    if (!al(k, 16) || !al(v, 16) || !al(slot_map, 4) || !stride_ok(k_stride, width, in_dtype) ||
        !stride_ok(v_stride, width, in_dtype))
        return GDN_ERR_INVALID_ARG;
    return gdn::launch_kv_append(k, v, k_stride, v_stride, slot_map, k_cache, v_cache, k_scale, v_scale, T, Hkv, d,
                                 num_blocks, block_size, in_dtype, static_cast<cudaStream_t>(cuda_stream));
}

size_t gdn_kv_attn_workspace_bytes(int N, int T, int Hq, int Hkv, int d, int max_q_len) {
    if (N < 1 || T < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || !head_ok(d) || max_q_len < 1) return 0;
    return gdn::kv_attn_ws_bytes(N, d);
}

gdn_status_t gdn_kv_attn(const void *q, long long q_stride, const void *k_cache, const void *v_cache,
                         const float *k_scale, const float *v_scale, const int *block_table, const int *cu_seqlens,
                         const int *kv_lens, void *o, float *lse, void *workspace, size_t workspace_bytes, int N, int T,
                         int Hq, int Hkv, int d, int num_blocks, int block_size, int max_blocks, int max_q_len,
                         int window, float scale, gdn_dtype_t in_dtype, gdn_dtype_t out_dtype, void *cuda_stream) {
    if (N < 1 || T < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || num_blocks < 1 || max_blocks < 1 || max_q_len < 1 ||
        window < 0 || !isfinite(scale) || !dtype_ok(in_dtype) || !dtype_ok(out_dtype))
        return GDN_ERR_INVALID_ARG;
    if (!head_ok(d) || !block_size_ok(block_size) || Hq > 65535 || T > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_blocks) * Hkv * block_size > kInt ||
        static_cast<long long>(max_blocks) * block_size > kMaxContext)
        return GDN_ERR_INVALID_ARG;
    if (!al(k_cache, 16) || !al(v_cache, 16) || !al(k_scale, 4) || !al(v_scale, 4) || !al(block_table, 4) ||
        !al(cu_seqlens, 4) || !al(kv_lens, 4) || !al_opt(lse, 4) || !al(workspace, 16) ||
        workspace_bytes < gdn_kv_attn_workspace_bytes(N, T, Hq, Hkv, d, max_q_len))
        return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    if (!al(q, 16) || !al(o, 16) || !stride_ok(q_stride, static_cast<long long>(Hq) * d, in_dtype))
        return GDN_ERR_INVALID_ARG;
    gdn::AttnArgs a{};
    a.q = q;
    a.q_stride = q_stride;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.table = block_table;
    a.cu = cu_seqlens;
    a.kv_lens = kv_lens;
    a.o = o;
    a.lse = lse;
    a.ws = static_cast<float *>(workspace);
    a.N = N;
    a.T = T;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.num_blocks = num_blocks;
    a.bs = block_size;
    while ((1 << a.bs_log2) < block_size) ++a.bs_log2;
    a.max_blocks = max_blocks;
    a.max_q = max_q_len;
    // a window that no context outgrows is none
    a.window = window >= static_cast<long long>(max_blocks) * block_size ? 0 : window;
    a.out_bf16 = out_dtype == GDN_BF16 ? 1 : 0;
    a.scale_log2 = scale * 1.4426950408889634f;
    return gdn::launch_kv_attn(k_cache, v_cache, a, d, in_dtype == GDN_F32, out_dtype == GDN_F32,
                               static_cast<cudaStream_t>(cuda_stream));
}

gdn_status_t gdn_decode_slots(const void *q, const void *k, const void *v, long long q_stride, long long k_stride,
                              long long v_stride, const float *beta, const float *g, float *state, const int *slots,
                              const int *cu_seqlens, void *o, int N, int T, int Hk, int Hv, int n_slots, int dk, int dv,
                              float scale, gdn_dtype_t in_dtype, const gdn_fwd_opts_t *opts, void *cuda_stream) {
    if (N < 1 || T < 0 || Hk < 1 || Hv < Hk || Hv % Hk != 0 || n_slots < 1 || !isfinite(scale) || !dtype_ok(in_dtype))
        return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens && T != N) return GDN_ERR_INVALID_ARG;
    gdn::FwdOpts oo{false, nullptr, false, gdn::kXNormNone, nullptr, 0.f};
    if (opts && !gdn::set_fwd_opts(*opts, g != nullptr, &oo)) return GDN_ERR_INVALID_ARG;
    if (!head_ok(dk) || !head_ok(dv) || Hv > 65535 || T > kMaxRows) return GDN_ERR_UNSUPPORTED;
    if (!al(state, 16) || !al(slots, 4) || !al_opt(cu_seqlens, 4) || !al_opt(beta, 4) || !al_opt(g, 4))
        return GDN_ERR_INVALID_ARG;
    if (T == 0) return GDN_OK;
    if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(o, 16)) return GDN_ERR_INVALID_ARG;
    const long long wk = static_cast<long long>(Hk) * dk, wv = static_cast<long long>(Hv) * dv, most = 1ll << 40;
    if (q_stride < wk || k_stride < wk || v_stride < wv || q_stride > most || k_stride > most || v_stride > most)
        return GDN_ERR_INVALID_ARG;
    return gdn::launch_decode_slots(q, k, v, q_stride, k_stride, v_stride, beta, g, state, slots, cu_seqlens, o, N, T, Hk,
                                    Hv, n_slots, dk, dv, scale, in_dtype, oo, static_cast<cudaStream_t>(cuda_stream));
}

}  // extern "C"
