// One step of the recurrence for rows whose states sit in slots of a pool (declared in
// include/ssm_scan.h as ssm_selective_state_update_slots): the sequential mode of the Mamba
// "architecture-details" page, section "Parallel Algorithm", as ssm_selective_state_update, with
// an index between a row and its state.
//
//   dt = softplus(delta + bias), h = exp(dt A) h + dt u B, out = (sum_n C h + D u) silu(z)
//
// HBM-bound: each state is read and written once, so the work beside that is kept small (below).
// CTAs of two warps, each of one row: 248 rows x 4096 channels x 16 states in 30.7 us (4.5 TB/s); timed
// beside one another 29.9 us, 30.8 with four rows a warp, whose one read of A costs registers and so
// loads in flight, and 33.8 with eight warps.  248 rows x 32 heads x 64 channels x 128 states 93 us
// (5.6 TB/s), 4 of them 3.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // f32x2 operations, ex2_approx, softplus1, silu1, window_reduce
#include "slots.h"
#include "ssm_scan.h"

namespace {

using ssm::aligned_to;
using ssm::all_aligned;
using ssm::ex2_approx;
using ssm::kLog2e;
constexpr int kThreads = 64;
constexpr int64_t kMaxGridY = 65535;

struct StepParams {
    float* states;
    const void *u, *delta, *B, *C, *z;
    const float *A, *D, *bias;
    const int* slots;
    void* out;
    int64_t batch, n_slots, slot_stride;
    uint32_t dim, nheads, ngroups, head_dim, group_dim, warps_per_group;
    int softplus;
};

template <typename T> __device__ __forceinline__ float ld_io(const T* p);
template <> __device__ __forceinline__ float ld_io<float>(const float* p) { return __ldg(p); }
template <> __device__ __forceinline__ float ld_io<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <typename T> __device__ __forceinline__ void st_io(T* p, float v);
template <> __device__ __forceinline__ void st_io<float>(float* p, float v) { *p = v; }
template <> __device__ __forceinline__ void st_io<__nv_bfloat16>(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// four consecutive B or C values
template <typename T> __device__ __forceinline__ float4 ld4(const T* p);
template <> __device__ __forceinline__ float4 ld4<float>(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
template <> __device__ __forceinline__ float4 ld4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

// A warp's share: CHW channels, IT = CHW (N/4) / 32 pieces of 16 bytes per lane.  N/4 = TPC
// neighbouring lanes hold a channel's states; over the IT pieces a lane meets IT channels.  What
// belongs to a channel alone (dt, the skip and the gate) is computed by the lane that owns it,
// the one that the reduce-scatter of y leaves its sum with, and dt, dt u go round by shuffles.
template <int N>
struct StepCfg {
    static constexpr int TPC = N / 4;
    static constexpr int IT = N == 8 ? 2 : 4;
    static constexpr int GRP = 32 / TPC;               // channels of one piece per warp
    static constexpr int CHW = IT * GRP;
    static constexpr int OWN = TPC / IT;               // lanes that share a channel's ownership
};

template <typename T, int N, bool HEAD>
__global__ void __launch_bounds__(kThreads) state_update_slots_kernel(const StepParams p) {
    using SC = StepCfg<N>;
    constexpr int TPC = SC::TPC, IT = SC::IT, GRP = SC::GRP, CHW = SC::CHW, OWN = SC::OWN;
    const int lane = threadIdx.x & 31, grp = lane / TPC, j = lane % TPC;
    const uint32_t wid = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t g = wid / p.warps_per_group;         // a warp's channels belong to one group
    if (g >= p.ngroups) return;
    const uint32_t c0 = wid % p.warps_per_group * CHW;
    const uint32_t d0 = g * p.group_dim + c0;
    const uint32_t nch = p.group_dim - c0 < (uint32_t)CHW ? p.group_dim - c0 : (uint32_t)CHW;
    const uint32_t own = GRP * (j / OWN) + grp;         // the lane's own channel
    const bool writes = own < nch && j % OWN == 0;
    const uint32_t d = d0 + (own < nch ? own : 0u);     // lanes past the last channel keep to the shuffles
    const uint32_t hd = HEAD ? d / p.head_dim : d;
    for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int slot = p.slots ? __ldg(p.slots + b) : (int)b;
        const ssm::SlotKind kind = ssm::slot_kind(slot, p.n_slots);
        if (kind == ssm::kSlotPad) continue;
        const bool live = kind == ssm::kSlotLive;
        float* hp = p.states + (live ? slot : 0) * p.slot_stride + ((int64_t)d0 + grp) * N + 4 * j;
        float4 h[IT], a[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t c = GRP * i + grp;
            h[i] = live && c < nch ? __ldcs(reinterpret_cast<const float4*>(hp + GRP * i * N)) : make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (!HEAD)
                a[i] = __ldg(reinterpret_cast<const float4*>(p.A + (int64_t)(d0 + (c < nch ? c : 0u)) * N) + j);
        }
        const int64_t bc = (b * p.ngroups + g) * N + 4 * j;
        const float4 bb = ld4<T>(static_cast<const T*>(p.B) + bc);
        const float4 cc = ld4<T>(static_cast<const T*>(p.C) + bc);
        const float u = ld_io<T>(static_cast<const T*>(p.u) + b * p.dim + d);
        const float z = p.z ? ld_io<T>(static_cast<const T*>(p.z) + b * p.dim + d) : 0.f;
        const float x = ld_io<T>(static_cast<const T*>(p.delta) + b * p.nheads + hd) + (p.bias ? __ldg(p.bias + hd) : 0.f);
        const float dt = p.softplus ? ssm::softplus1(x) : x;
        const float du = dt * u;
        const float s = dt * kLog2e;
        const float dv = HEAD ? ex2_approx(s * __ldg(p.A + hd)) : s;     // the decay itself, or dt log2 e
        float y[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int from = (lane & ~(TPC - 1)) + i * OWN;
            const float2 d2 = ssm::dup2(__shfl_sync(0xffffffffu, dv, from));
            const float2 u2 = ssm::dup2(__shfl_sync(0xffffffffu, du, from));
            float2 e0 = d2, e1 = d2;
            if constexpr (!HEAD) {
                e0 = ssm::mul2(d2, make_float2(a[i].x, a[i].y));
                e1 = ssm::mul2(d2, make_float2(a[i].z, a[i].w));
                e0 = make_float2(ex2_approx(e0.x), ex2_approx(e0.y));
                e1 = make_float2(ex2_approx(e1.x), ex2_approx(e1.y));
            }
            const float2 h0 = ssm::fma2(e0, make_float2(h[i].x, h[i].y), ssm::mul2(u2, make_float2(bb.x, bb.y)));
            const float2 h1 = ssm::fma2(e1, make_float2(h[i].z, h[i].w), ssm::mul2(u2, make_float2(bb.z, bb.w)));
            if (live && (uint32_t)(GRP * i + grp) < nch)
                __stcs(reinterpret_cast<float4*>(hp + GRP * i * N), make_float4(h0.x, h0.y, h1.x, h1.y));
            const float2 q = ssm::fma2(make_float2(cc.x, cc.y), h0, ssm::mul2(make_float2(cc.z, cc.w), h1));
            y[i] = q.x + q.y;
        }
        int off;
        ssm::window_reduce<IT, TPC>(y, j, off);
        if (writes) {
            float o = fmaf(p.D ? __ldg(p.D + d) : 0.f, u, y[0]);
            if (p.z) o *= ssm::silu1(z);
            st_io<T>(static_cast<T*>(p.out) + b * p.dim + d, live ? o : __int_as_float(0x7FC00000));
        }
    }
}

template <typename T, int N>
int launch_n(StepParams p, cudaStream_t s) {
    using SC = StepCfg<N>;
    constexpr int64_t kWarps = kThreads / 32;
    p.warps_per_group = (uint32_t)((p.group_dim + SC::CHW - 1) / SC::CHW);
    const int64_t bx = ((int64_t)p.warps_per_group * p.ngroups + kWarps - 1) / kWarps;
    const dim3 g((unsigned)bx, (unsigned)(p.batch < kMaxGridY ? p.batch : kMaxGridY));
    if (p.nheads != p.dim) state_update_slots_kernel<T, N, true><<<g, kThreads, 0, s>>>(p);
    else state_update_slots_kernel<T, N, false><<<g, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T>
int launch(const StepParams& p, int64_t N, cudaStream_t s) {
    switch (N) {
        case 8: return launch_n<T, 8>(p, s);
        case 16: return launch_n<T, 16>(p, s);
        case 32: return launch_n<T, 32>(p, s);
        case 64: return launch_n<T, 64>(p, s);
        case 128: return launch_n<T, 128>(p, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

}  // namespace

extern "C" int ssm_selective_state_update_slots(const ssm_dims_t* dims, float* states, const int32_t* slots,
                                                int64_t n_slots, int64_t slot_stride, const void* u, const void* delta,
                                                const float* A, const void* B, const void* C, const float* D,
                                                const void* z, const float* delta_bias, int softplus, void* out,
                                                ssm_stream_t stream) {
    if (!dims) return SSM_ERR_INVALID_ARG;
    const ssm_dims_t& d = *dims;
    if (d.batch < 0 || d.dim <= 0 || d.dstate <= 0 || d.nheads <= 0 || d.ngroups <= 0 || d.reserved != 0)
        return SSM_ERR_INVALID_ARG;
    if (d.seqlen != 1 || d.dim % d.nheads || d.dim % d.ngroups) return SSM_ERR_INVALID_ARG;
    if (d.io_dtype != SSM_F32 && d.io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (d.batch > 0x7FFFFFFF || d.dim > (1 << 24) || n_slots < 0 || n_slots > 0x7FFFFFFF) return SSM_ERR_INVALID_ARG;
    const int64_t N = d.dstate;
    if (N != 8 && N != 16 && N != 32 && N != 64 && N != 128) return SSM_ERR_UNSUPPORTED;
    if (d.batch == 0) return SSM_OK;
    if (!states || !u || !delta || !A || !B || !C || !out) return SSM_ERR_INVALID_ARG;
    if (slot_stride < d.dim * N) return SSM_ERR_INVALID_ARG;
    const uintptr_t esz = d.io_dtype == SSM_BF16 ? 2 : 4;
    if (!all_aligned(esz, {u, delta, B, C, z, out}) || !all_aligned(4, {states, slots, A, D, delta_bias}))
        return SSM_ERR_INVALID_ARG;
    // four states move as one 16-byte (state, A, fp32 B and C) or 8-byte (bf16 B and C) piece
    if (!aligned_to(states, 16) || slot_stride % 4 || !aligned_to(B, 4 * esz) || !aligned_to(C, 4 * esz) ||
        (d.nheads == d.dim && !aligned_to(A, 16)))
        return SSM_ERR_UNSUPPORTED;
    StepParams p{};
    p.states = states; p.u = u; p.delta = delta; p.B = B; p.C = C; p.z = z;
    p.A = A; p.D = D; p.bias = delta_bias; p.slots = slots; p.out = out;
    p.batch = d.batch; p.n_slots = n_slots; p.slot_stride = slot_stride;
    p.dim = (uint32_t)d.dim; p.nheads = (uint32_t)d.nheads; p.ngroups = (uint32_t)d.ngroups;
    p.head_dim = (uint32_t)(d.dim / d.nheads); p.group_dim = (uint32_t)(d.dim / d.ngroups);
    p.softplus = softplus ? 1 : 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return d.io_dtype == SSM_BF16 ? launch<__nv_bfloat16>(p, N, s) : launch<float>(p, N, s);
}
