// gdn_decode_slots: the decode step's recurrence over a pool of states, several tokens a request.
//
// Per token and value head, with S the head's dk x dv state and q' = scale q (page
// "【CS336】lecture4", section "继续改进：GDN"; the arithmetic of the one-token step):
//   sk = (diag(alpha) S)^T k,  sq = (diag(alpha) S)^T q'     one pass over S
//   u  = beta (v - sk)   (u = v without the delta term),   o = sq + (q'.k) u
//   S <- diag(alpha) S + k u^T                               alpha one value, or one per key row
// The state's traffic bounds it: 8 dk dv bytes a head and request however many tokens the
// request brings, so one block keeps its head's state in registers from the first token to the
// last. Thread t owns 4 consecutive value columns of DK / RG key rows, RG rows apart, so every
// warp-wide state access is a contiguous run of 256 or 512 bytes. A token costs two block
// meetings: one when its operands are in shared memory, one when the partial column sums are;
// the next token's operands are fetched before the first of them, so that a drafted run of
// tokens does not wait for memory at each. Every block looks through the slots before its own
// request's, so that a slot named twice is found on the device and no two blocks update one state.
// One token of 256 requests, 32 heads of 128 x 128 (1.08 GB): 173 us, 6.2 TB/s; up to six tokens of 48
// requests, 16 heads of 64 x 128 (40 MB): 16.2 us.
#include "common.cuh"
#include "tc_kernels.cuh"

namespace gdn {
namespace {

constexpr int kSlotThreads = 256;

struct SlotArgs {
    long long qs, ks, vs;          // elements between token rows
    const float *beta, *g;
    float *state;
    const int *slots, *cu;
    void *o;
    int T, Hk, Hv, n_slots;
    float scale;
    int vec, out_bf16, xnorm;
    const float *dskip, *xw;
    float xeps;
};

template <int DK, int DV, typename IT, bool DELTA>
__global__ void __launch_bounds__(kSlotThreads, DK * DV == 16384 ? 2 : DK * DV == 8192 ? 3 : 4)
decode_slots_kernel(const IT *__restrict__ q, const IT *__restrict__ k, const IT *__restrict__ v, const SlotArgs a,
                    unsigned *__restrict__ err) {
    constexpr int CG = DV / 4, RG = kSlotThreads / CG, RPT = DK / RG;
    static_assert(RPT >= 1 && RG * RPT == DK && DK <= kSlotThreads && DV <= kSlotThreads, "bad tiling");
    __shared__ float s_k[2][DK], s_q[2][DK], s_a[2][DK], s_v[2][DV];
    __shared__ float red_k[DELTA ? RG : 1][DV], red_q[RG][DV];
    __shared__ float s_qk[2];

    const int n = blockIdx.x, h = blockIdx.y;
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG;
    const int slot = a.slots[n];
    int t0 = n, t1 = n + 1;
    if (a.cu) { t0 = a.cu[n]; t1 = a.cu[n + 1]; }
    if (slot == -1) return;
    if (slot < -1 || slot >= a.n_slots || t0 < 0 || t1 < t0 || t1 > a.T) {
        if (tid == 0 && h == 0) atomicOr(err, kErrBadSeqlens);
        return;
    }
    if (t0 == t1) return;

    float *S = a.state + (static_cast<long long>(slot) * a.Hv + h) * (DK * DV);
    if (!in_bounds((static_cast<long long>(slot) * a.Hv + h + 1) * (DK * DV) - 1, static_cast<long long>(a.n_slots) * a.Hv * DK * DV, err))
        return;
    float4 st[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) st[i] = ld_global4(S + (rg + RG * i) * DV + 4 * cg);
    bool twice = false;
    for (int m = tid; m < n; m += kSlotThreads) twice |= a.slots[m] == slot;

    const int kh = h / (a.Hv / a.Hk);
    float rk = 0.f, rq = 0.f, rv = 0.f, ra = 1.f, alpha_n = 1.f, beta_n = 1.f;   // the token fetched ahead
    auto fetch = [&](int t) {
        const long long th = static_cast<long long>(t) * a.Hv + h;
        if (tid < DK) {
            rk = ld_in(k + t * a.ks + kh * DK + tid);
            rq = ld_in(q + t * a.qs + kh * DK + tid);
            if (a.vec) ra = a.g[th * DK + tid];
        }
        if (tid < DV) rv = ld_in(v + t * a.vs + h * DV + tid);
        if (a.g && !a.vec) alpha_n = a.g[th];
        if (DELTA) beta_n = a.beta[th];
    };
    fetch(t0);
    if (__syncthreads_or(twice)) {
        if (tid == 0 && h == 0) atomicOr(err, kErrBadSeqlens);
        return;
    }
    for (int t = t0; t < t1; ++t) {
        const int p = (t - t0) & 1;
        if (tid < DK) {
            s_k[p][tid] = rk;
            s_q[p][tid] = a.scale * rq;
            s_a[p][tid] = a.vec ? expf(ra) : 1.f;
        }
        if (tid < DV) s_v[p][tid] = rv;
        const float alpha = a.g && !a.vec ? expf(alpha_n) : 1.f;
        const float bt = beta_n;
        if (t + 1 < t1) fetch(t + 1);
        __syncthreads();

        float4 pk = make_float4(0.f, 0.f, 0.f, 0.f), pq = pk;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int j = rg + RG * i;
            const float aj = a.vec ? s_a[p][j] : alpha;
            st[i].x *= aj; st[i].y *= aj; st[i].z *= aj; st[i].w *= aj;
            const float kj = s_k[p][j], qj = s_q[p][j];
            if (DELTA) {
                pk.x = fmaf(st[i].x, kj, pk.x); pk.y = fmaf(st[i].y, kj, pk.y);
                pk.z = fmaf(st[i].z, kj, pk.z); pk.w = fmaf(st[i].w, kj, pk.w);
            }
            pq.x = fmaf(st[i].x, qj, pq.x); pq.y = fmaf(st[i].y, qj, pq.y);
            pq.z = fmaf(st[i].z, qj, pq.z); pq.w = fmaf(st[i].w, qj, pq.w);
        }
        if (DELTA) *reinterpret_cast<float4 *>(&red_k[rg][4 * cg]) = pk;
        *reinterpret_cast<float4 *>(&red_q[rg][4 * cg]) = pq;
        if (tid >= kSlotThreads - 32) {
            float x = 0.f;
            for (int j = tid & 31; j < DK; j += 32) x = fmaf(s_q[p][j], s_k[p][j], x);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if ((tid & 31) == 0) s_qk[p] = x;
        }
        __syncthreads();

        float u[4], ov[4];
        {
            float sk[4] = {0.f, 0.f, 0.f, 0.f};
            if (DELTA) {
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    const float4 x = *reinterpret_cast<const float4 *>(&red_k[r][4 * cg]);
                    sk[0] += x.x; sk[1] += x.y; sk[2] += x.z; sk[3] += x.w;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float vc = s_v[p][4 * cg + c];
                u[c] = DELTA ? bt * (vc - sk[c]) : vc;
            }
        }
        if (rg == 0) {
            float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                const float4 x = *reinterpret_cast<const float4 *>(&red_q[r][4 * cg]);
                sq[0] += x.x; sq[1] += x.y; sq[2] += x.z; sq[3] += x.w;
            }
            const float qk = s_qk[p];
#pragma unroll
            for (int c = 0; c < 4; ++c) ov[c] = fmaf(qk, u[c], sq[c]);
            if (a.dskip)
#pragma unroll
                for (int c = 0; c < 4; ++c) ov[c] = fmaf(a.dskip[h * DV + 4 * cg + c], s_v[p][4 * cg + c], ov[c]);
            if (a.xnorm != kXNormNone) {    // over the DV values of the row, 4 in each of lanes 0 .. CG-1
                constexpr unsigned mask = CG >= 32 ? 0xffffffffu : ((1u << CG) - 1u);
                if (a.xnorm == kXNormLayer) {
                    float s1 = (ov[0] + ov[1]) + (ov[2] + ov[3]);
#pragma unroll
                    for (int off = CG / 2; off > 0; off >>= 1) s1 += __shfl_xor_sync(mask, s1, off);
#pragma unroll
                    for (int c = 0; c < 4; ++c) ov[c] -= s1 * (1.f / DV);
                }
                float s2 = (ov[0] * ov[0] + ov[1] * ov[1]) + (ov[2] * ov[2] + ov[3] * ov[3]);
#pragma unroll
                for (int off = CG / 2; off > 0; off >>= 1) s2 += __shfl_xor_sync(mask, s2, off);
                const float rs = rsqrtf(s2 * (1.f / DV) + a.xeps);
#pragma unroll
                for (int c = 0; c < 4; ++c) ov[c] *= rs * (a.xw ? a.xw[h * DV + 4 * cg + c] : 1.f);
            }
            const long long at = (static_cast<long long>(t) * a.Hv + h) * DV + 4 * cg;
            const bool o_in = in_bounds(at + 3, static_cast<long long>(a.T) * a.Hv * DV, err);
            if (o_in && a.out_bf16) {
                __nv_bfloat162 lo = __floats2bfloat162_rn(ov[0], ov[1]), hi = __floats2bfloat162_rn(ov[2], ov[3]);
                uint2 w;
                w.x = *reinterpret_cast<const uint32_t *>(&lo);
                w.y = *reinterpret_cast<const uint32_t *>(&hi);
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + at) = w;
            } else if (o_in) {
                st_global4(static_cast<float *>(a.o) + at, make_float4(ov[0], ov[1], ov[2], ov[3]));
            }
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float kj = s_k[p][rg + RG * i];
            st[i].x = fmaf(kj, u[0], st[i].x); st[i].y = fmaf(kj, u[1], st[i].y);
            st[i].z = fmaf(kj, u[2], st[i].z); st[i].w = fmaf(kj, u[3], st[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) st_global4(S + (rg + RG * i) * DV + 4 * cg, st[i]);
}

template <int DK, int DV, typename IT>
gdn_status_t launch_slots_t(const void *q, const void *k, const void *v, const SlotArgs &a, int N, cudaStream_t stream) {
    unsigned *err = device_error_word();
    if (!err) return GDN_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(N), static_cast<unsigned>(a.Hv));
    const IT *q_ = static_cast<const IT *>(q), *k_ = static_cast<const IT *>(k), *v_ = static_cast<const IT *>(v);
    if (a.beta) decode_slots_kernel<DK, DV, IT, true><<<grid, kSlotThreads, 0, stream>>>(q_, k_, v_, a, err);
    else decode_slots_kernel<DK, DV, IT, false><<<grid, kSlotThreads, 0, stream>>>(q_, k_, v_, a, err);
    return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename IT>
gdn_status_t launch_slots_dt(const void *q, const void *k, const void *v, const SlotArgs &a, int N, int dk, int dv,
                             cudaStream_t stream) {
    if (dk == 128 && dv == 128) return launch_slots_t<128, 128, IT>(q, k, v, a, N, stream);
    if (dk == 128 && dv == 64) return launch_slots_t<128, 64, IT>(q, k, v, a, N, stream);
    if (dk == 64 && dv == 128) return launch_slots_t<64, 128, IT>(q, k, v, a, N, stream);
    return launch_slots_t<64, 64, IT>(q, k, v, a, N, stream);
}

}  // namespace

gdn_status_t launch_decode_slots(const void *q, const void *k, const void *v, long long qs, long long ks, long long vs,
                                 const float *beta, const float *g, float *state, const int *slots, const int *cu,
                                 void *o, int N, int T, int Hk, int Hv, int n_slots, int dk, int dv, float scale,
                                 gdn_dtype_t in_dtype, const FwdOpts &oo, cudaStream_t stream) {
    const SlotArgs a{qs, ks, vs, beta, g, state, slots, cu, o, T, Hk, Hv, n_slots, scale, oo.gate_per_key ? 1 : 0,
                     oo.bf16 ? 1 : 0, oo.xnorm, oo.dskip, oo.xw, oo.xeps};
    return in_dtype == GDN_F32 ? launch_slots_dt<float>(q, k, v, a, N, dk, dv, stream)
                               : launch_slots_dt<__nv_bfloat16>(q, k, v, a, N, dk, dv, stream);
}

}  // namespace gdn
