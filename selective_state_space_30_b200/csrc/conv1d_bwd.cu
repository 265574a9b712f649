// Gradients of the causal depthwise convolution (declared in include/ssm_scan.h as
// ssm_causal_conv1d_bwd), the backward pass of ssm_causal_conv1d_fwd.
//
//   v[t]  = bias + sum_{k<W} w[k] x[t-W+1+k]              (recomputed)
//   dv[t] = dout[t] act'(v[t]),   silu'(v) = s (1 + v (1 - s)), s = 1 / (1 + exp(-v))
//   dx[t] = sum_k w[k] dv[t+W-1-k],   dw[k] = sum_{b,t} dv[t] x[t-W+1+k],   dbias = sum_{b,t} dv[t]
//
// HBM-bound: x and dout are read once and dx is written once.  A warp walks a stretch of two
// rows from its end to its start, 32 16-byte pieces at a time: the inputs before a piece come
// from the lane below, the dv behind it from the lane above, and lane 31's from the tile before.
// dw and dbias stay in registers over a warp's stretches and are added over the CTA's warps in
// order; where a channel is split over CTAs a second kernel adds their partials, in order too, so
// the gradients repeat bit for bit.
//
// Measured on one B200: 8 x 1536 x 2048 bf16, width 4, 42 us (3.6 TB/s; 23 us of HBM time), issue
// 55 % busy with 14 of 64 warps an SM (128 registers hold two rows and the loads ahead); three CTAs an
// SM with 84 registers 61 us.  2 x 768 x 1021 fp32, width 3, 6.5 us in a graph with four warps a pair of
// channels (beside one another 6.9, 8.7 with eight, 9.6 with partials and a second kernel).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // f32x2 operations, ex2_approx, rcp_approx
#include "slots.h"           // all_aligned
#include "ssm_scan.h"

namespace {

using ssm::all_aligned;

constexpr int kMaxWidth = 4;
constexpr int kWarps = 8;

struct ConvBwd {
    const void *x, *dout;
    const float *w, *bias;
    void* dx;
    float *dw, *dbias;
    float* part;            // [n_split][dim][W + 1] where a channel's sums are split over CTAs
    int64_t batch, dim, seqlen;
    int64_t tiles_per_seg, n_seg, n_split;
    int silu;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// dv of two tokens
template <bool SILU>
__device__ __forceinline__ float2 dact2(float2 v, float2 g) {
    if (!SILU) return g;
    const float2 a = ssm::mul2(v, ssm::dup2(-ssm::kLog2e));
    const float2 q = ssm::add2(make_float2(ssm::ex2_approx(a.x), ssm::ex2_approx(a.y)), ssm::dup2(1.f));
    const float2 s = make_float2(ssm::rcp_approx(q.x), ssm::rcp_approx(q.y));
    const float2 c = ssm::fma2(s, ssm::dup2(-1.f), ssm::dup2(1.f));
    return ssm::mul2(ssm::mul2(g, s), ssm::fma2(v, c, ssm::dup2(1.f)));
}

// One 16-byte piece of x and of dout, and of x the 8 (bf16) or 16 (fp32) bytes before it.
template <typename T>
struct Piece {
    static constexpr int PW = sizeof(T) == 2 ? 2 : 4;
    uint4 x, g;
    uint32_t before[PW];
};

template <typename T, int CNT>
__device__ __forceinline__ void unpack(const uint32_t* w, float* v) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < CNT; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// Tokens t .. of a row as 32-bit words; those outside [0, L) read as zero and are not accessed.
template <typename T, int WORDS>
__device__ __forceinline__ void gather(const T* row, int64_t t, int64_t L, uint32_t* w) {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = t + i >= 0 && t + i < L ? __float_as_uint(row[t + i]) : 0u;
        } else {
            const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
            const int64_t a = t + 2 * i;
            const uint32_t lo = a >= 0 && a < L ? r[a] : 0u, hi = a + 1 >= 0 && a + 1 < L ? r[a + 1] : 0u;
            w[i] = lo | hi << 16;
        }
    }
}

// As load_piece, for rows that start on the 16-byte grid: lanes behind the row's end hold zeros.
template <typename T>
__device__ __forceinline__ Piece<T> load_aligned(const T* x, const T* go, bool in, bool before) {
    Piece<T> p = {};
    if (in) {
        p.x = __ldg(reinterpret_cast<const uint4*>(x));
        p.g = __ldg(reinterpret_cast<const uint4*>(go));
        if (before) {
            if constexpr (sizeof(T) == 2) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(x - 4));
                p.before[0] = q.x; p.before[1] = q.y;
            } else {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(x - 4));
                p.before[0] = q.x; p.before[1] = q.y; p.before[2 % Piece<T>::PW] = q.z; p.before[3 % Piece<T>::PW] = q.w;
            }
        }
    }
    return p;
}

// The lane's pieces of a tile; lane 0's earlier tokens too (the others take theirs from the lane
// below).  `whole`: the tile lies inside the row, on the 16-byte grid (t > 0 is then at least V).
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* x, const T* go, int64_t t, int64_t L, bool whole, int lane) {
    constexpr int V = 16 / sizeof(T), PW = Piece<T>::PW;
    Piece<T> p;
#pragma unroll
    for (int i = 0; i < PW; ++i) p.before[i] = 0u;
    if (whole) {
        p.x = __ldg(reinterpret_cast<const uint4*>(x + t));
        p.g = __ldg(reinterpret_cast<const uint4*>(go + t));
        if (lane == 0 && t > 0) {
#pragma unroll
            for (int i = 0; i < PW; i += 2) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(x + t - V / 2 * (PW / 2)) + i / 2);
                p.before[i] = q.x;
                p.before[i + 1] = q.y;
            }
        }
    } else {
        uint32_t w[4];
        gather<T, 4>(x, t, L, w);
        p.x = make_uint4(w[0], w[1], w[2], w[3]);
        gather<T, 4>(go, t, L, w);
        p.g = make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) gather<T, PW>(x, t - 4, L, p.before);
    }
    return p;
}

// A warp walks two rows, of neighbouring channels: they are the two halves of every f32x2
// operation, so that a value sits in one register pair for all the taps that meet it.  (Rows off
// the 16-byte grid have their pieces at different tokens; the arithmetic is the same.)
// ALIGNED: every row of x, dout and dx starts on the 16-byte grid.
template <typename T, int W, bool ALIGNED, bool SILU>
__global__ void __launch_bounds__(32 * kWarps, 2) conv1d_bwd_kernel(const ConvBwd p) {
    constexpr int V = 16 / sizeof(T), H = W - 1, PW = Piece<T>::PW;
    __shared__ float sums[kWarps][2 * (W + 1)];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = blockDim.x / 32;
    const int64_t d0 = blockIdx.x / p.n_split * 2, split = blockIdx.x % p.n_split, L = p.seqlen;
    const bool both = d0 + 1 < p.dim;                 // an odd last channel pairs with itself and writes once
    const int64_t d[2] = {d0, both ? d0 + 1 : d0};
    float2 w[W], dw[W], db = ssm::dup2(0.f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
        w[k] = make_float2(__ldg(p.w + d[0] * W + k), __ldg(p.w + d[1] * W + k));
        dw[k] = ssm::dup2(0.f);
    }
    const float2 bias = p.bias ? make_float2(__ldg(p.bias + d[0]), __ldg(p.bias + d[1])) : ssm::dup2(0.f);
    // the pair's stretches, one after the other over the warps of its CTAs
    for (int64_t item = split * warps + warp; item < p.batch * p.n_seg; item += p.n_split * warps) {
        const int64_t seg = item % p.n_seg, b = item / p.n_seg;
        const T *x[2], *go[2];
        T* dx[2];
        int m[2];
        bool grid[2];
        int64_t tiles[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int64_t row = (b * p.dim + d[r]) * L;
            x[r] = static_cast<const T*>(p.x) + row;
            go[r] = static_cast<const T*>(p.dout) + row;
            dx[r] = static_cast<T*>(p.dx) + row;
            // pieces sit on dx's 16-byte grid: the row's first one may start up to V-1 tokens early
            m[r] = ALIGNED ? 0 : (int)((reinterpret_cast<uintptr_t>(dx[r]) & 15u) / sizeof(T));
            grid[r] = ((reinterpret_cast<uintptr_t>(x[r]) ^ reinterpret_cast<uintptr_t>(dx[r])) & 15u) == 0 &&
                      ((reinterpret_cast<uintptr_t>(go[r]) ^ reinterpret_cast<uintptr_t>(dx[r])) & 15u) == 0;
            // the row's own tiles end where its tokens do, which may be one tile earlier than another row's
            tiles[r] = (L + m[r] + 32 * V - 1) / (32 * V);
        }
        const int64_t all = tiles[0] > tiles[1] ? tiles[0] : tiles[1];
        const int64_t first_end = (tiles[0] < tiles[1] ? tiles[0] : tiles[1]) - 1;
        const int64_t tile0 = seg * p.tiles_per_seg, tile1 = tile0 + p.tiles_per_seg < all ? tile0 + p.tiles_per_seg : all;
        auto load = [&](int r, int64_t tile) {
            if constexpr (ALIGNED) {
                // both rows alike: only the row's last tile has lanes behind its end
                const int64_t o = (tile * 32 + lane) * V;
                const bool in = tile + 1 < tile1 || o < L;
                return load_aligned<T>(x[r] + o, go[r] + o, in, lane == 0 && tile > 0);
            }
            const int64_t t = tile * 32 * V - m[r];
            if (tile >= tiles[r]) return Piece<T>{};      // this row ends a tile before the other
            return load_piece<T>(x[r], go[r], t + lane * V, L, grid[r] && t >= 0 && t + 32 * V <= L, lane);
        };
        Piece<T> next[2] = {};
        if (tile1 > tile0) {
            next[0] = load(0, tile1 - 1);
            next[1] = load(1, tile1 - 1);
        }
        // dv of the W-1 tokens behind the stretch, on lanes 0 .. W-2, then on every lane
        float2 behind[H > 0 ? H : 1];
        {
            float g[2] = {0.f, 0.f};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t t = tile1 * 32 * V - m[r] + lane;
                if (lane < H && t < L) {
                    float v = r ? bias.y : bias.x;
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        const int64_t s = t - H + k;
                        if (s >= 0) v = fmaf(r ? w[k].y : w[k].x, to_f<T>(x[r][s]), v);
                    }
                    g[r] = dact2<SILU>(ssm::dup2(v), ssm::dup2(to_f<T>(go[r][t]))).x;
                }
            }
#pragma unroll
            for (int k = 0; k < H; ++k)
                behind[k] = make_float2(__shfl_sync(0xffffffffu, g[0], k), __shfl_sync(0xffffffffu, g[1], k));
        }
        for (int64_t tile = tile1 - 1; tile >= tile0; --tile) {
            const Piece<T> cur[2] = {next[0], next[1]};
            if (tile > tile0) {
                next[0] = load(0, tile - 1);
                next[1] = load(1, tile - 1);
            }
            // Behind a row's end dv is zero, and the inputs that its sums would meet there, the last ones of the
            // row, read as zero too: an infinity or a NaN among them stays out of the taps that it does not
            // belong to.  (With silu it is in dv of the last token, and so in every tap.)
            const bool tail = !SILU && tile >= first_end;
            int left[2] = {V, V};                         // the lane's tokens ahead of the end
            if (tail) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int64_t n = L - ((tile * 32 + lane) * V - m[r]);
                    left[r] = n < V ? (int)(n > 0 ? n : 0) : V;
                }
            }
            // tokens t - 4 .. t + V - 1 of x; t .. t + V + H - 1 of dv
            float2 xv[4 + V], dv[V + H];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t xw[4] = {cur[r].x.x, cur[r].x.y, cur[r].x.z, cur[r].x.w};
                const uint32_t gw[4] = {cur[r].g.x, cur[r].g.y, cur[r].g.z, cur[r].g.w};
                uint32_t bw[PW];
#pragma unroll
                for (int i = 0; i < PW; ++i) {
                    bw[i] = __shfl_up_sync(0xffffffffu, xw[4 - PW + i], 1);
                    if (lane == 0) bw[i] = cur[r].before[i];
                    if (!SILU && ALIGNED && left[r] == 0) bw[i] = 0u;
                }
                float xb[4], xc[V], gc[V];
                unpack<T, 4>(bw, xb);
                unpack<T, V>(xw, xc);
                unpack<T, V>(gw, gc);
#pragma unroll
                for (int e = 0; e < 4; ++e) (r ? xv[e].y : xv[e].x) = xb[e];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    (r ? xv[4 + e].y : xv[4 + e].x) = xc[e];
                    (r ? dv[e].y : dv[e].x) = gc[e];
                }
            }
            float2* xh = xv + 4 - H;                      // xh[e + k] meets w[k] at token e
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (!ALIGNED && tail) {
#pragma unroll
                    for (int k = 0; k < H; ++k) {
                        if (e >= left[0]) xh[e + k].x = 0.f;
                        if (e >= left[1]) xh[e + k].y = 0.f;
                    }
                }
                float2 v = bias;
#pragma unroll
                for (int k = 0; k < W; ++k) v = ssm::fma2(w[k], xh[e + k], v);
                dv[e] = dact2<SILU>(v, dv[e]);
                db = ssm::add2(db, dv[e]);
#pragma unroll
                for (int k = 0; k < W; ++k) dw[k] = ssm::fma2(dv[e], xh[e + k], dw[k]);
            }
#pragma unroll
            for (int k = 0; k < H; ++k) {
                dv[V + k] = make_float2(__shfl_down_sync(0xffffffffu, dv[k].x, 1), __shfl_down_sync(0xffffffffu, dv[k].y, 1));
                if (lane == 31) dv[V + k] = behind[k];
                behind[k] = make_float2(__shfl_sync(0xffffffffu, dv[k].x, 0), __shfl_sync(0xffffffffu, dv[k].y, 0));
            }
            float2 o[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                o[e] = ssm::mul2(w[H], dv[e]);
#pragma unroll
                for (int k = 0; k < H; ++k) o[e] = ssm::fma2(w[k], dv[e + H - k], o[e]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t t = (tile * 32 + lane) * V - m[r];
                if (r && !both) break;
                if (ALIGNED ? tile + 1 < tile1 || t < L : t >= 0 && t + V <= L) {
                    uint32_t u[4];
                    if constexpr (sizeof(T) == 4) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(r ? o[i].y : o[i].x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __nv_bfloat162 b2 = r ? __floats2bfloat162_rn(o[2 * i].y, o[2 * i + 1].y)
                                                        : __floats2bfloat162_rn(o[2 * i].x, o[2 * i + 1].x);
                            u[i] = *reinterpret_cast<const uint32_t*>(&b2);
                        }
                    }
                    *reinterpret_cast<uint4*>(dx[r] + t) = make_uint4(u[0], u[1], u[2], u[3]);
                } else if (!ALIGNED) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (t + e >= 0 && t + e < L) dx[r][t + e] = from_f<T>(r ? o[e].y : o[e].x);
                }
            }
        }
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) {
        db = ssm::add2(db, make_float2(__shfl_xor_sync(0xffffffffu, db.x, s), __shfl_xor_sync(0xffffffffu, db.y, s)));
#pragma unroll
        for (int k = 0; k < W; ++k)
            dw[k] = ssm::add2(dw[k], make_float2(__shfl_xor_sync(0xffffffffu, dw[k].x, s),
                                                 __shfl_xor_sync(0xffffffffu, dw[k].y, s)));
    }
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            sums[warp][k] = dw[k].x;
            sums[warp][W + 1 + k] = dw[k].y;
        }
        sums[warp][W] = db.x;
        sums[warp][2 * W + 1] = db.y;
    }
    __syncthreads();
    if (threadIdx.x < (both ? 2 : 1) * (W + 1)) {
        float a = sums[0][threadIdx.x];
#pragma unroll
        for (int q = 1; q < kWarps; ++q)
            if (q < warps) a += sums[q][threadIdx.x];
        const int r = threadIdx.x / (W + 1), k = threadIdx.x % (W + 1);
        if (p.n_split > 1) p.part[(split * p.dim + d0 + r) * (W + 1) + k] = a;
        else if (k < W) p.dw[(d0 + r) * W + k] = a;
        else if (p.dbias) p.dbias[d0 + r] = a;
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
    int64_t tiles_per_seg, n_seg, n_split;
    int warps;              // of a CTA
};

// A pair of channels is one CTA's, whose sums then need no second kernel, of eight warps or of four,
// whichever walk fewer tiles after one another (2 x 768 x 1021 fp32, 384 pairs: four warps in one round
// 6.9 us, eight in two 8.7; 8 x 1536 x 2048 bf16: three rounds of 8 tiles against two of 16).  Where few
// pairs leave SMs idle over long rows a pair is split over several CTAs: the second kernel costs about four
// tiles' time (4 x 280 x 4096: fp32, 18 tiles against 10, 23 us whole and 19 split; bf16, 10 against 6, 12.3
// and 13.7).  Rows are cut into stretches as far as the warps need them.  The shape alone decides, so the
// sums' order is the shape's.
Plan plan_of(int64_t batch, int64_t dim, int64_t seqlen, int io_dtype) {
    const int64_t V = io_dtype == SSM_BF16 ? 8 : 4, pairs = (dim + 1) / 2, slots = 148 * 2;   // two CTAs of eight warps an SM
    const int64_t tiles = (seqlen + V - 1 + 32 * V - 1) / (32 * V);
    if (batch <= 0 || seqlen <= 0) return {1, 1, 1, kWarps};
    auto plan = [&](int warps, int64_t ctas) {
        int64_t seg = (warps * ctas + batch - 1) / batch;
        if (seg > tiles) seg = tiles;
        Plan r{(tiles + seg - 1) / seg, 1, 1, warps};
        r.n_seg = (tiles + r.tiles_per_seg - 1) / r.tiles_per_seg;
        const int64_t most = (batch * r.n_seg + warps - 1) / warps;
        r.n_split = ctas < most ? ctas : most;
        return r;
    };
    auto walked = [&](const Plan& r) {
        const int64_t at_once = slots * kWarps / r.warps, rounds = (pairs * r.n_split + at_once - 1) / at_once;
        const int64_t warps = r.warps * r.n_split;
        return rounds * ((batch * r.n_seg + warps - 1) / warps) * (r.tiles_per_seg + 1);   // (a start costs about a tile)
    };
    const Plan eight = plan(kWarps, 1), four = plan(kWarps / 2, 1);
    const Plan one = walked(four) < walked(eight) ? four : eight;
    const Plan split = plan(kWarps, slots / pairs > 1 ? slots / pairs : 1);
    return walked(one) - walked(split) > 4 ? split : one;
}

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
int launch(const ConvBwd& p, int warps, bool aligned, cudaStream_t s) {
    const int64_t ctas = (p.dim + 1) / 2 * p.n_split;
    if (ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    const unsigned g = (unsigned)ctas;
    if (aligned && p.silu) conv1d_bwd_kernel<T, W, true, true><<<g, 32 * warps, 0, s>>>(p);
    else if (aligned) conv1d_bwd_kernel<T, W, true, false><<<g, 32 * warps, 0, s>>>(p);
    else if (p.silu) conv1d_bwd_kernel<T, W, false, true><<<g, 32 * warps, 0, s>>>(p);
    else conv1d_bwd_kernel<T, W, false, false><<<g, 32 * warps, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T>
int launch_t(const ConvBwd& p, int warps, int width, bool aligned, cudaStream_t s) {
    switch (width) {
        case 1: return launch<T, 1>(p, warps, aligned, s);
        case 2: return launch<T, 2>(p, warps, aligned, s);
        case 3: return launch<T, 3>(p, warps, aligned, s);
        case 4: return launch<T, 4>(p, warps, aligned, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

}  // namespace

extern "C" int ssm_causal_conv1d_bwd_workspace_size(int64_t batch, int64_t dim, int64_t seqlen, int32_t width,
                                                    int32_t io_dtype, size_t* bytes) {
    if (!bytes) return SSM_ERR_INVALID_ARG;
    const int rc = check_shape(batch, dim, seqlen, width, io_dtype);
    if (rc != SSM_OK) return rc;
    const Plan q = plan_of(batch, dim, seqlen, io_dtype);
    *bytes = q.n_split > 1 ? (size_t)(q.n_split * dim * (width + 1)) * 4 : 0;
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
    const bool tokens = batch > 0 && seqlen > 0;
    if (tokens && (!x || !dout || !dx || dx == x || dx == dout)) return SSM_ERR_INVALID_ARG;
    if (need > 0 && (!workspace || workspace_bytes < need)) return SSM_ERR_INVALID_ARG;
    const uintptr_t esz = io_dtype == SSM_BF16 ? 2 : 4;
    if (!all_aligned(esz, {x, dout, dx}) || !all_aligned(4, {w, bias, dw, dbias, workspace}))
        return SSM_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // without tokens every gradient is an empty sum: the kernel finds no stretch and writes zeros
    const Plan q = plan_of(batch, dim, seqlen, io_dtype);
    ConvBwd p{};
    p.x = x; p.dout = dout; p.w = w; p.bias = bias; p.dx = dx; p.dw = dw; p.dbias = dbias;
    p.part = static_cast<float*>(workspace);
    p.batch = tokens ? batch : 0; p.dim = dim; p.seqlen = seqlen;
    p.tiles_per_seg = q.tiles_per_seg; p.n_seg = q.n_seg; p.n_split = q.n_split;
    p.silu = silu ? 1 : 0;
    const bool aligned = seqlen * (int64_t)esz % 16 == 0 && all_aligned(16, {x, dout, dx});
    const int r = io_dtype == SSM_BF16 ? launch_t<__nv_bfloat16>(p, q.warps, width, aligned, s) : launch_t<float>(p, q.warps, width, aligned, s);
    if (r != SSM_OK || q.n_split == 1) return r;
    const int64_t n = dim * (width + 1);
    conv1d_bwd_sum_kernel<<<(unsigned)((n + 31) / 32), dim3(32, 8), 0, s>>>(p.part, q.n_split, dim, width, dw, dbias);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
