// Gradients of the causal depthwise convolution (declared in include/ssm_scan.h as
// ssm_causal_conv1d_bwd), the backward pass of ssm_causal_conv1d_fwd.
//
//   v[t]  = bias + sum_{k<W} w[k] x[t-W+1+k]              (recomputed)
//   dv[t] = dout[t] act'(v[t]),   silu'(v) = s (1 + v (1 - s)), s = 1 / (1 + exp(-v))
//   dx[t] = sum_k w[k] dv[t+W-1-k],   dw[k] = sum_{b,t} dv[t] x[t-W+1+k],   dbias = sum_{b,t} dv[t]
//
// HBM-bound: x and dout are read once and dx is written once.  A warp walks a stretch of one
// row from its end to its start, 32 16-byte pieces at a time: the inputs before a piece come
// from the lane below, the dv behind it from the lane above, and lane 31's from the tile before.
// dw and dbias stay in registers for the stretch; each warp writes one partial and a second
// kernel adds the partials in a fixed order, so the gradients repeat bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // ex2_approx, rcp_approx
#include "ssm_scan.h"

namespace {

constexpr int kMaxWidth = 4;
constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct ConvBwd {
    const void *x, *dout;
    const float *w, *bias;
    void* dx;
    float* part;            // [batch * n_seg][dim][W + 1]
    int64_t rows, dim, seqlen;
    int64_t tiles, tiles_per_seg, n_seg;
    int silu;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Tokens [t, t + V) of a row; those outside [0, L) read as zero and are not accessed.
template <typename T>
__device__ __forceinline__ void load_tokens(const T* row, int64_t t, int64_t L, float* v) {
    constexpr int V = 16 / sizeof(T);
    const T* p = row + t;
    if (t >= 0 && t + V <= L && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
        if constexpr (sizeof(T) == 4) {
            v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
            v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = t + e >= 0 && t + e < L ? to_f<T>(p[e]) : 0.f;
    }
}

// dv of one token
__device__ __forceinline__ float dact(float v, float g, int silu) {
    if (!silu) return g;
    const float s = ssm::rcp_approx(1.f + ssm::ex2_approx(-kLog2e * v));
    return g * s * fmaf(v, 1.f - s, 1.f);
}

template <typename T, int W>
__global__ void __launch_bounds__(32 * kWarps) conv1d_bwd_kernel(const ConvBwd p) {
    constexpr int V = 16 / sizeof(T), H = W - 1;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (id >= p.rows * p.n_seg) return;
    const int64_t r = id / p.n_seg, seg = id % p.n_seg, d = r % p.dim, L = p.seqlen;
    const T* x = static_cast<const T*>(p.x) + r * L;
    const T* go = static_cast<const T*>(p.dout) + r * L;
    T* dx = static_cast<T*>(p.dx) + r * L;
    // pieces sit on dx's 16-byte grid: the row's first one may start up to V-1 tokens early
    const int m = (int)((reinterpret_cast<uintptr_t>(dx) & 15u) / sizeof(T));
    float w[W], dw[W], db = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = __ldg(p.w + d * W + k);
        dw[k] = 0.f;
    }
    const float bias = p.bias ? __ldg(p.bias + d) : 0.f;
    const int64_t first = seg * p.tiles_per_seg;
    const int64_t end = first + p.tiles_per_seg < p.tiles ? first + p.tiles_per_seg : p.tiles;

    // dv of the W-1 tokens behind the stretch, on lanes 0 .. W-2, then on every lane
    float behind[H > 0 ? H : 1];
    {
        const int64_t t = end * 32 * V - m + lane;
        float g = 0.f;
        if (lane < H && t < L) {
            float v = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const int64_t s = t - H + k;
                if (s >= 0) v = fmaf(w[k], to_f<T>(x[s]), v);
            }
            g = dact(v, to_f<T>(go[t]), p.silu);
        }
#pragma unroll
        for (int k = 0; k < H; ++k) behind[k] = __shfl_sync(0xffffffffu, g, k);
    }
    for (int64_t tile = end - 1; tile >= first; --tile) {
        const int64_t t = (tile * 32 + lane) * V - m;
        float xv[H + V], dv[V + H];                   // tokens t - H .. t + V - 1; t .. t + V + H - 1
        load_tokens<T>(x, t, L, xv + H);
        load_tokens<T>(go, t, L, dv);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            xv[k] = __shfl_up_sync(0xffffffffu, xv[V + k], 1);
            const int64_t s = t - H + k;
            if (lane == 0) xv[k] = s >= 0 && s < L ? to_f<T>(x[s]) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float v = bias;
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[k], xv[e + k], v);
            dv[e] = dact(v, dv[e], p.silu);
        }
#pragma unroll
        for (int k = 0; k < H; ++k) {
            dv[V + k] = __shfl_down_sync(0xffffffffu, dv[k], 1);
            if (lane == 31) dv[V + k] = behind[k];
            behind[k] = __shfl_sync(0xffffffffu, dv[k], 0);
        }
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                a = fmaf(w[k], dv[e + H - k], a);
                dw[k] = fmaf(dv[e], xv[e + k], dw[k]);
            }
            db += dv[e];
            o[e] = a;
        }
        if (t >= 0 && t + V <= L) {
            uint4 q;
            if constexpr (sizeof(T) == 4) {
                q = make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3]));
            } else {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                    u[i] = *reinterpret_cast<const uint32_t*>(&b2);
                }
                q = make_uint4(u[0], u[1], u[2], u[3]);
            }
            *reinterpret_cast<uint4*>(dx + t) = q;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (t + e >= 0 && t + e < L) dx[t + e] = from_f<T>(o[e]);
        }
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) {
        db += __shfl_xor_sync(0xffffffffu, db, s);
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k] += __shfl_xor_sync(0xffffffffu, dw[k], s);
    }
    if (lane == 0) {
        float* o = p.part + (((r / p.dim) * p.n_seg + seg) * p.dim + d) * (W + 1);
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = dw[k];
        o[W] = db;
    }
}

// Adds the partials of each weight and bias gradient in a fixed order: eight threads an output,
// each every eighth partial, joined in order.
__global__ void __launch_bounds__(256) conv1d_bwd_sum_kernel(const float* part, int64_t n_part, int64_t dim, int width,
                                                             float* dw, float* dbias) {
    __shared__ float s[8][32];
    const int64_t n = dim * (width + 1), i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float a = 0.f;
    if (i < n)
        for (int64_t q = threadIdx.y; q < n_part; q += 8) a += __ldcg(part + q * n + i);
    s[threadIdx.y][threadIdx.x] = a;
    __syncthreads();
    if (threadIdx.y == 0 && i < n) {
#pragma unroll
        for (int q = 1; q < 8; ++q) a += s[q][threadIdx.x];
        const int64_t d = i / (width + 1), k = i % (width + 1);
        if (k < width) dw[d * width + k] = a;
        else if (dbias) dbias[d] = a;
    }
}

struct Plan {
    int64_t tiles, tiles_per_seg, n_seg;
};

// Rows are cut into stretches where there are too few of them to fill the machine (64 warps on
// each of 148 SMs); the shape alone decides, so the sums' order is the shape's.
Plan plan_of(int64_t batch, int64_t dim, int64_t seqlen, int io_dtype) {
    const int64_t V = io_dtype == SSM_BF16 ? 8 : 4;
    Plan q;
    q.tiles = (seqlen + V - 1 + 32 * V - 1) / (32 * V);
    const int64_t rows = batch * dim, want = 148 * 64;
    int64_t n = rows > 0 ? (want + rows - 1) / rows : 1;
    if (n > q.tiles) n = q.tiles;
    if (n < 1) n = 1;
    q.tiles_per_seg = (q.tiles + n - 1) / n;
    q.n_seg = q.tiles_per_seg > 0 ? (q.tiles + q.tiles_per_seg - 1) / q.tiles_per_seg : 1;
    return q;
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_shape(int64_t batch, int64_t dim, int64_t seqlen, int32_t width, int32_t io_dtype) {
    if (batch < 0 || dim <= 0 || seqlen < 0) return SSM_ERR_INVALID_ARG;
    if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (width < 1 || width > kMaxWidth) return SSM_ERR_UNSUPPORTED;
    if (dim > (1 << 24) || seqlen > ((int64_t)1 << 40) || batch > ((int64_t)1 << 46) / dim ||
        (seqlen > 0 && batch * dim > ((int64_t)1 << 46) / seqlen))
        return SSM_ERR_INVALID_ARG;
    return SSM_OK;
}

template <typename T, int W>
int launch(const ConvBwd& p, cudaStream_t s) {
    const int64_t ctas = (p.rows * p.n_seg + kWarps - 1) / kWarps;
    if (ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    conv1d_bwd_kernel<T, W><<<(unsigned)ctas, 32 * kWarps, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T>
int launch_t(const ConvBwd& p, int width, cudaStream_t s) {
    switch (width) {
        case 1: return launch<T, 1>(p, s);
        case 2: return launch<T, 2>(p, s);
        case 3: return launch<T, 3>(p, s);
        case 4: return launch<T, 4>(p, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

}  // namespace

extern "C" int ssm_causal_conv1d_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen, int32_t width,
                                                    int32_t io_dtype, size_t* bytes) {
    if (!bytes) return SSM_ERR_INVALID_ARG;
    const int rc = check_shape(batch, dim, seqlen, width, io_dtype);
    if (rc != SSM_OK) return rc;
    *bytes = seqlen == 0 ? 0 : (size_t)(batch * plan_of(batch, dim, seqlen, io_dtype).n_seg * dim * (width + 1)) * 4;
    return SSM_OK;
}

extern "C" int ssm_causal_conv1d_bwd(int64_t batch, int64_t dim, int64_t seqlen, int32_t width, int32_t io_dtype,
                                     const void* x, const float* w, const float* bias, int silu, const void* dout,
                                     void* dx, float* dw, float* dbias, void* workspace, size_t workspace_bytes,
                                     ssm_stream_t stream) {
    size_t need = 0;
    const int rc = ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, width, io_dtype, &need);
    if (rc != SSM_OK) return rc;
    if (!w || !dw) return SSM_ERR_INVALID_ARG;
    if (need > 0 && (!x || !dout || !dx || !workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
    const uintptr_t esz = io_dtype == SSM_BF16 ? 2 : 4;
    if (!aligned_to(x, esz) || !aligned_to(dout, esz) || !aligned_to(dx, esz) || !aligned_to(workspace, 4))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int64_t n_part = 0;
    if (need > 0) {
        const Plan q = plan_of(batch, dim, seqlen, io_dtype);
        ConvBwd p{};
        p.x = x; p.dout = dout; p.w = w; p.bias = bias; p.dx = dx; p.part = static_cast<float*>(workspace);
        p.rows = batch * dim; p.dim = dim; p.seqlen = seqlen;
        p.tiles = q.tiles; p.tiles_per_seg = q.tiles_per_seg; p.n_seg = q.n_seg;
        p.silu = silu ? 1 : 0;
        const int r = io_dtype == SSM_BF16 ? launch_t<__nv_bfloat16>(p, width, s) : launch_t<float>(p, width, s);
        if (r != SSM_OK) return r;
        n_part = batch * q.n_seg;
    }
    // with no tokens every gradient is an empty sum
    const int64_t n = dim * (width + 1);
    conv1d_bwd_sum_kernel<<<(unsigned)((n + 31) / 32), dim3(32, 8), 0, s>>>(static_cast<const float*>(workspace), n_part,
                                                                           dim, width, dw, dbias);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
