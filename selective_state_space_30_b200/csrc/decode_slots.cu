// One step of the recurrence for rows whose states sit in slots of a pool (declared in
// include/ssm_scan.h as ssm_selective_state_update_slots): the sequential mode of the Mamba
// "architecture-details" page, section "Parallel Algorithm", as ssm_selective_state_update, with
// an index between a row and its state.
//
//   dt = softplus(delta + bias), h = exp(dt A) h + dt u B, out = (sum_n C h + D u) silu(z)
//
// HBM-bound: each state is read and written once.  A thread holds four states of one channel for
// K rows at a time, so one read of A serves K rows and K independent 16-byte state loads are in
// flight per thread; N/4 neighbouring lanes hold a channel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // ex2_approx, softplus1, silu1
#include "slots.h"
#include "ssm_scan.h"

namespace {

using ssm::ex2_approx;
using ssm::kLog2e;
constexpr int kThreads = 256;
constexpr int kMaxGridY = 65535;

struct StepParams {
    float* states;
    const void *u, *delta, *B, *C, *z;
    const float *A, *D, *bias;
    const int* slots;
    void* out;
    int64_t batch, n_slots, slot_stride;
    uint32_t dim, nheads, ngroups, head_dim, group_dim;
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

template <typename T, int N, int K, bool HEAD>
__global__ void __launch_bounds__(kThreads) state_update_slots_kernel(const StepParams p) {
    constexpr uint32_t TPC = N / 4;
    constexpr uint32_t CH = kThreads / TPC;            // channels per CTA
    const uint32_t dc = blockIdx.x * CH + threadIdx.x / TPC;
    const bool live = dc < p.dim;                      // lanes past the last channel keep to the shuffles
    const uint32_t d = live ? dc : p.dim - 1;
    const uint32_t n0 = 4u * (threadIdx.x % TPC);
    const uint32_t hd = HEAD ? d / p.head_dim : d;
    const uint32_t g = p.ngroups == 1 ? 0u : d / p.group_dim;
    float4 a;
    if constexpr (HEAD) {
        const float ah = __ldg(p.A + hd) * kLog2e;
        a = make_float4(ah, ah, ah, ah);
    } else {
        a = __ldg(reinterpret_cast<const float4*>(p.A + (int64_t)d * N + n0));
        a.x *= kLog2e; a.y *= kLog2e; a.z *= kLog2e; a.w *= kLog2e;
    }
    const float bias = p.bias ? __ldg(p.bias + hd) : 0.f;
    const float Dd = p.D ? __ldg(p.D + d) : 0.f;
    for (int64_t b0 = (int64_t)blockIdx.y * K; b0 < p.batch; b0 += (int64_t)gridDim.y * K) {
        float4 h[K], bb[K], cc[K];
        float u[K], x[K], z[K];
        float* hp[K];
        ssm::SlotKind kind[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t b = b0 + k;
            const int slot = b < p.batch ? (p.slots ? __ldg(p.slots + b) : (int)b) : -1;
            kind[k] = ssm::slot_kind(slot, p.n_slots);
            hp[k] = p.states + (kind[k] == ssm::kSlotLive ? slot : 0) * p.slot_stride + (int64_t)d * N + n0;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            h[k] = kind[k] == ssm::kSlotLive ? __ldcs(reinterpret_cast<const float4*>(hp[k])) : make_float4(0.f, 0.f, 0.f, 0.f);
            // padding rows read row 0's inputs, which are there, and write nothing
            const int64_t b = kind[k] == ssm::kSlotPad ? 0 : b0 + k;
            const int64_t bc = (b * p.ngroups + g) * N + n0;
            bb[k] = ld4<T>(static_cast<const T*>(p.B) + bc);
            cc[k] = ld4<T>(static_cast<const T*>(p.C) + bc);
            u[k] = ld_io<T>(static_cast<const T*>(p.u) + b * p.dim + d);
            x[k] = ld_io<T>(static_cast<const T*>(p.delta) + b * p.nheads + hd);
            z[k] = p.z ? ld_io<T>(static_cast<const T*>(p.z) + b * p.dim + d) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float xb = x[k] + bias;
            const float dt = p.softplus ? ssm::softplus1(xb) : xb;
            const float du = dt * u[k];
            if constexpr (HEAD) {
                const float da = ex2_approx(dt * a.x);
                h[k].x = fmaf(da, h[k].x, du * bb[k].x);
                h[k].y = fmaf(da, h[k].y, du * bb[k].y);
                h[k].z = fmaf(da, h[k].z, du * bb[k].z);
                h[k].w = fmaf(da, h[k].w, du * bb[k].w);
            } else {
                h[k].x = fmaf(ex2_approx(dt * a.x), h[k].x, du * bb[k].x);
                h[k].y = fmaf(ex2_approx(dt * a.y), h[k].y, du * bb[k].y);
                h[k].z = fmaf(ex2_approx(dt * a.z), h[k].z, du * bb[k].z);
                h[k].w = fmaf(ex2_approx(dt * a.w), h[k].w, du * bb[k].w);
            }
            if (live && kind[k] == ssm::kSlotLive) __stcs(reinterpret_cast<float4*>(hp[k]), h[k]);
            float y = fmaf(cc[k].x, h[k].x, fmaf(cc[k].y, h[k].y, fmaf(cc[k].z, h[k].z, cc[k].w * h[k].w)));
#pragma unroll
            for (uint32_t m = TPC / 2; m >= 1; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
            if (live && n0 == 0 && kind[k] != ssm::kSlotPad) {
                y = fmaf(Dd, u[k], y);
                if (p.z) y *= ssm::silu1(z[k]);
                if (kind[k] == ssm::kSlotBad) y = __int_as_float(0x7FC00000);
                st_io<T>(static_cast<T*>(p.out) + (b0 + k) * p.dim + d, y);
            }
        }
    }
}

template <typename T, int N, int K>
int launch_k(const StepParams& p, cudaStream_t s) {
    constexpr int64_t CH = kThreads / (N / 4);
    const int64_t bx = (p.dim + CH - 1) / CH;
    const int64_t rows = (p.batch + K - 1) / K;
    const dim3 g((unsigned)bx, (unsigned)(rows < kMaxGridY ? rows : kMaxGridY));
    if (p.nheads != p.dim) state_update_slots_kernel<T, N, K, true><<<g, kThreads, 0, s>>>(p);
    else state_update_slots_kernel<T, N, K, false><<<g, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T, int N>
int launch_n(const StepParams& p, cudaStream_t s) {
    // four rows per thread once one row each would give every SM its fill of CTAs
    const int64_t ctas = (p.dim * (N / 4) + kThreads - 1) / kThreads * p.batch;
    return ctas >= 4 * 148 * 8 ? launch_k<T, N, 4>(p, s) : launch_k<T, N, 1>(p, s);
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

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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
    for (const void* t : {u, delta, z, static_cast<const void*>(out)})
        if (!aligned_to(t, esz)) return SSM_ERR_INVALID_ARG;
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
