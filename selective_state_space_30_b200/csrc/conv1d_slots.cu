// The causal depthwise convolution with its history in a pool of slots: over prompts packed end
// to end, and for one new token of each row.  Declared in include/ssm_scan.h as
// ssm_causal_conv1d_packed_fwd and ssm_causal_conv1d_update; the convolution is
// ssm_causal_conv1d_fwd's (Mamba "architecture-details" page, "Model Configuration": d_conv).
//
//   v = bias[d] + sum_{k<W} w[d,k] x[d, t-W+1+k],   out = silu ? v / (1 + exp(-v)) : v
//
// A sequence's first W-1 tokens take their earlier inputs from its slot (or zero), and its last
// W-1 inputs replace the slot's.  HBM-bound: every input is read and every output written once.
//
// Measured on one B200, bf16, width 4: 32768 tokens in 32 prompts x 4096 channels 120 us (4.5 TB/s;
// a copy through the same loop, width 1 without silu, 95 us), of which the prompts' first tokens are
// 8 us; fp32, 2048 channels 121 us; 1013 tokens in 7 prompts x 1536 channels 5.8 us; one token of 4 rows x
// 1536 channels 2.7 us, of 248 rows x 4096 9.2 us (fp32 8.1), all in a graph.  Between the first of them
// and the HBM time (82 us) stand silu's two MUFU operations per output (60 us of that pipe) and the issue of
// the rest (110 instructions per 8 outputs).  With three CTAs an SM (80 registers) it took 142 us against
// 130 of four; inputs asked for ahead of the mask changed nothing there and made the small call 0.6 us longer.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pair.cuh"
#include "scan_kernel.cuh"   // silu1
#include "slots.h"
#include "ssm_scan.h"

namespace {

using ssm::aligned_to;
using ssm::all_aligned;
constexpr int kMaxWidth = 4;
constexpr int kThreads = 256;
constexpr int kMaxGridY = 65535;
constexpr int kTapRows = 256;     // rows whose taps a CTA keeps in shared memory

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V = 16 / sizeof(T) elements of a 16-byte piece
template <typename T> __device__ __forceinline__ void unpack(const uint4& q, float* v);
template <> __device__ __forceinline__ void unpack<float>(const uint4& q, float* v) {
    v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y); v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
}
template <> __device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float* v);
template <> __device__ __forceinline__ uint4 pack<float>(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
template <> __device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------- packed prompts

struct PackedConv {
    const void* x;
    const float *w, *bias;
    void* out;
    void* states;
    const int *cu, *slots;
    const unsigned char* has_state;
    int64_t dim, total, n_seq, n_slots, slot_stride;
    int64_t head_ctas;       // CTAs of the sequences' first tokens, ahead of the others
    unsigned head_tiles;     // channel tiles of those
    unsigned time_tiles;     // time tiles of the others
    int log_tx;              // 16-byte pieces of a row that a CTA covers, a power of two
    int rows_per_thread;
    int silu;
    int aligned;             // every row of x and out is 16-byte aligned
};

// The 16 bytes at p, where they lie inside [lo, hi); elements outside read as zero.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const unsigned char* p, const unsigned char* lo, const unsigned char* hi) {
    if (p >= lo && p + 16 <= hi) return __ldg(reinterpret_cast<const uint4*>(p));
    constexpr int V = 16 / sizeof(T);
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const unsigned char* q = p + e * (int)sizeof(T);
        v[e] = q >= lo && q < hi ? to_f<T>(*reinterpret_cast<const T*>(q)) : 0.f;
    }
    return pack<T>(v);
}

// Role 1, one thread per (sequence, channel): the outputs of the sequence's first W-1 tokens,
// which need the slot's history, and the slot's new history.  One thread reads the old history
// and writes the new one, so no other CTA's read can meet the write.
template <typename T, int W>
__device__ __forceinline__ void sequence_heads(const PackedConv& p, unsigned bid) {
    const int64_t seq = bid / p.head_tiles;
    const int64_t d = (int64_t)(bid % p.head_tiles) * kThreads + threadIdx.x;
    if (d >= p.dim) return;
    const ssm::TokenRange r = ssm::token_range(p.cu, seq, p.total);
    const int slot = p.slots ? __ldg(p.slots + seq) : (int)seq;
    const ssm::SlotKind kind = ssm::slot_kind(slot, p.n_slots);
    if (kind == ssm::kSlotPad) return;
    const int64_t len = r.hi - r.lo;
    T* orow = static_cast<T*>(p.out) + d * p.total + r.lo;
    if (kind == ssm::kSlotBad) {
        for (int64_t t = 0; t < len && t < W - 1; ++t) orow[t] = from_f<T>(__int_as_float(0x7FC00000));
        return;
    }
    const T* xrow = static_cast<const T*>(p.x) + d * p.total + r.lo;
    T* st = static_cast<T*>(p.states) + slot * p.slot_stride + d * (W - 1);
    const bool has = p.has_state && __ldg(p.has_state + seq) != 0;
    // the history, then the first tokens
    T v[2 * (W - 1)];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        v[k] = has ? st[k] : from_f<T>(0.f);
        v[W - 1 + k] = k < len ? xrow[k] : from_f<T>(0.f);
    }
    float w[W];
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = __ldg(p.w + d * W + k);
    const float b = p.bias ? __ldg(p.bias + d) : 0.f;
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        float o = b;
#pragma unroll
        for (int k = 0; k < W; ++k) o = fmaf(w[k], to_f<T>(v[t + k]), o);
        if (t < len) orow[t] = from_f<T>(p.silu ? ssm::silu1(o) : o);
    }
    // element k of the new history is input len - (W-1) + k, or an older one of the slot's
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        T keep;
        if (len >= W - 1) {
            keep = xrow[len - (W - 1) + k];
        } else {
            keep = v[k];
#pragma unroll
            for (int s = 1; s < W - 1; ++s)
                if (len == s) keep = v[s + k];
        }
        st[k] = keep;
    }
}

// One row's piece and what becomes of it: xw holds its four words behind the PW words before it;
// `mask`: the tokens to write, `nan`: those of them whose slot is bad.
template <int PW>
struct RowPiece {
    uint32_t xw[PW + 4];
    unsigned char* out;
    unsigned mask, nan;
};

template <typename T>
__device__ __forceinline__ void store_piece(unsigned char* out, unsigned mask, unsigned nan, float* o) {
    constexpr int V = 16 / sizeof(T);
    if (mask == 0u) return;
    if (nan != 0u) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if ((nan >> e) & 1u) o[e] = __int_as_float(0x7FC00000);
    }
    if (mask == (1u << V) - 1u) {
        *reinterpret_cast<uint4*>(out) = pack<T>(o);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if ((mask >> e) & 1u) reinterpret_cast<T*>(out)[e] = from_f<T>(o[e]);
    }
}

// The outputs of two rows' pieces.  The rows are the two halves of every f32x2 operation: a value
// then sits in one register pair for all taps, where pairs of neighbouring tokens would need a
// copy of it for every other tap (170 -> 163 us for 32768 tokens x 4096 channels in bf16; with the taps in shared
// memory and silu decided at compile time 142, with four CTAs an SM 130, with the taps of all rows
// there, which shortens the code, 123).
template <typename T, int W, int PW, bool SILU>
__device__ __forceinline__ void conv_pieces(const uint32_t (&x0)[PW + 4], const uint32_t (&x1)[PW + 4],
                                            const ssm::pair_t* w, ssm::pair_t bias, float* o0, float* o1) {
    constexpr int V = 16 / sizeof(T), ES = (int)sizeof(T), E = (PW + 4) * 4 / ES;
    ssm::pair_t xv[E];
#pragma unroll
    for (int k = 0; k < PW + 4; ++k) {
        if constexpr (sizeof(T) == 4) {
            xv[k] = ssm::pk(__uint_as_float(x0[k]), __uint_as_float(x1[k]));
        } else {
            xv[2 * k] = ssm::pk(__uint_as_float(x0[k] << 16), __uint_as_float(x1[k] << 16));
            xv[2 * k + 1] = ssm::pk(__uint_as_float(x0[k] & 0xFFFF0000u), __uint_as_float(x1[k] & 0xFFFF0000u));
        }
    }
    const ssm::pair_t* xh = xv + E - V - (W - 1);                 // xh[e + k] meets w[k] at token e
#pragma unroll
    for (int e = 0; e < V; ++e) {
        ssm::pair_t v = bias;
#pragma unroll
        for (int k = 0; k < W; ++k) v = ssm::pfma(w[k], xh[e + k], v);
        if (SILU) v = ssm::psilu(v);
        const float2 h = ssm::halves(v);
        o0[e] = h.x;
        o1[e] = h.y;
    }
}

// Role 2: every other token.  A CTA covers tx pieces of a row and walks rows; the 16-byte pieces
// follow each row's own alignment, so odd row lengths move whole pieces too.  Bit t of `live`
// says that token t0 + t has its W-1 earlier inputs in its own sequence; it is made once per CTA
// and serves every row.
template <typename T, int W, bool SILU>
__device__ __forceinline__ void sequence_bodies(const PackedConv& p, unsigned bid) {
    constexpr int V = 16 / sizeof(T), ES = (int)sizeof(T);
    constexpr int kWords = (kThreads * V + 2 * V + 31) / 32 + 1;
    __shared__ unsigned live[kWords], bad[kWords];
    __shared__ __align__(16) float2 tap_pairs[kTapRows / 2 * (W + 1)];
    const unsigned tile = bid % p.time_tiles, rt = bid / p.time_tiles;
    const int tx = 1 << p.log_tx, ty = kThreads >> p.log_tx;
    const int64_t span = (int64_t)tx * V;
    const int64_t t0 = tile * span - V;                 // token of bit 0: a piece may start up to V-1 tokens early
    const int bits = (int)span + V;
    for (int i = threadIdx.x; i < kWords; i += kThreads) live[i] = bad[i] = 0u;
    // The rows' taps and biases in shared memory, as pairs of the rows that are worked on together:
    // [pair][tap, then bias] of (row, row + ty), the last of an odd count twice.  (Loaded per row they
    // cost a third of the instructions.)
    const int per = kTapRows / 2 / ty;                            // pairs that a thread row may walk
    const int64_t d0 = (int64_t)rt * p.rows_per_thread * ty;
    for (int i = threadIdx.x; i < p.rows_per_thread * ty * (W + 1); i += kThreads) {
        const int row = i / (W + 1), k = i % (W + 1);
        const int r = row / ty, y = row % ty;                     // r-th row of thread row y
        const int64_t d = ssm::tap_channel(d0, row, ty, p.dim);
        if (d >= 0) {
            const float v = k < W ? __ldg(p.w + d * W + k) : p.bias ? __ldg(p.bias + d) : 0.f;
            float2* q = tap_pairs + (y * per + r / 2) * (W + 1) + k;
            (r & 1 ? q->y : q->x) = v;
        }
    }
    __syncthreads();
    // Sequences that meet [t0, t0 + bits).  Up to a few per thread are simply all looked at; with
    // more, the bounds rise, so a binary search finds the first.  Bounds out of order mark the wrong
    // tokens at most, each inside the buffer.
    int64_t a = 0;
    if (p.n_seq > 4 * kThreads) {
        int64_t b = p.n_seq;
        while (a < b) {
            const int64_t m = (a + b) / 2;
            if (__ldg(p.cu + m + 1) <= t0) a = m + 1;
            else b = m;
        }
    }
    bool met_bad = false;
    for (int64_t s = a + threadIdx.x; s < p.n_seq; s += kThreads) {
        const ssm::TokenRange r = ssm::token_range(p.cu, s, p.total);
        if (r.lo >= t0 + bits) {
            if (p.n_seq > 4 * kThreads) break;
            continue;
        }
        const ssm::SlotKind kind = ssm::slot_kind(p.slots ? __ldg(p.slots + s) : (int)s, p.n_slots);
        if (kind == ssm::kSlotPad) continue;
        met_bad = met_bad || kind == ssm::kSlotBad;
        int64_t lo = r.lo + (W - 1) - t0, hi = r.hi - t0;
        lo = lo < 0 ? 0 : lo;
        hi = hi > bits ? bits : hi;
        for (int64_t w = lo >> 5; w * 32 < hi; ++w) {
            const int f = lo > w * 32 ? (int)(lo - w * 32) : 0;
            const int e = hi < w * 32 + 32 ? (int)(hi - w * 32) : 32;
            if (f < e) {
                const unsigned m = (e == 32 ? 0xffffffffu : (1u << e) - 1u) & ~((1u << f) - 1u);
                atomicOr(live + w, m);
                if (kind == ssm::kSlotBad) atomicOr(bad + w, m);
            }
        }
    }
    const bool any_bad = __syncthreads_or(met_bad);
    const int px = threadIdx.x & (tx - 1), py = threadIdx.x >> p.log_tx, lane = threadIdx.x & 31;
    const unsigned char* lo = static_cast<const unsigned char*>(p.x);
    const unsigned char* hi = lo + p.dim * p.total * ES;
    const int64_t row_bytes = p.total * ES;
    constexpr unsigned sel = (1u << V) - 1u;
    // the W-1 inputs before a piece, as the 32-bit words that end it: the lane below holds them
    constexpr int PW = W == 1 ? 0 : sizeof(T) == 4 ? W - 1 : W / 2;
    const bool edge = px == 0 || lane == 0;
    const int64_t dr = (int64_t)rt * p.rows_per_thread * ty + py;
    const int64_t step = ty * row_bytes;
    const float2* taps = tap_pairs + py * per * (W + 1);
    if (p.aligned && tx >= 32) {
        // Every row starts on the 16-byte grid, so one mask serves all rows and a warp's pieces are
        // of one row.  Lanes behind the last token and rows behind the last one repeat the last
        // piece and write nothing; so do a row's first tokens, whose earlier inputs sequence_heads has.
        const int left = ((int)p.dim - (int)dr + ty - 1) >> (31 - __clz(ty));
        const int rows = left < p.rows_per_thread ? left : p.rows_per_thread;
        if (rows <= 0) return;
        int64_t t = tile * span + (int64_t)px * V;
        const int bit = px * V + V;
        const unsigned mask = __funnelshift_r(live[bit >> 5], live[(bit >> 5) + 1], bit & 31) & sel;
        const unsigned nan = any_bad ? __funnelshift_r(bad[bit >> 5], bad[(bit >> 5) + 1], bit & 31) & mask : 0u;
        const bool whole = __all_sync(0xffffffffu, mask == sel && nan == 0u);
        if (__all_sync(0xffffffffu, mask == 0u)) return;
        if (t > p.total - V) t = p.total - V;
        const bool past = t > 0;
        auto rows_of = [&](auto all_written) {
            const unsigned char* xp = lo + dr * row_bytes + t * ES;
            unsigned char* op = static_cast<unsigned char*>(p.out) + dr * row_bytes + t * ES;
            struct In {
                uint4 q;
                uint32_t b[PW > 0 ? PW : 1];                      // the words before (L1: the neighbour's)
            };
            auto load = [&](const unsigned char* q) {
                In in = {};
                in.q = __ldg(reinterpret_cast<const uint4*>(q));
                if (PW > 0 && past) {
                    if constexpr (PW == 2) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q) - 1);
                        in.b[0] = v.x; in.b[1 % PW] = v.y;
                    } else {
#pragma unroll
                        for (int k = 0; k < PW; ++k) in.b[k] = __ldg(reinterpret_cast<const uint32_t*>(q) + k - PW);
                    }
                }
                return in;
            };
            // two rows at a time, the next two already on their way
            In next[2] = {load(xp), load(xp + (rows > 1 ? step : 0))};
            for (int i0 = 0; i0 < rows; i0 += 2, taps += W + 1) {
                const In cur[2] = {next[0], next[1]};
                const bool two = i0 + 1 < rows;
                xp += 2 * step;
                if (i0 + 2 < rows) {
                    next[0] = load(xp);
                    next[1] = load(xp + (i0 + 3 < rows ? step : 0));
                }
                uint32_t xw[2][PW + 4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int k = 0; k < PW; ++k) xw[r][k] = cur[r].b[k];
                    xw[r][PW] = cur[r].q.x; xw[r][PW + 1] = cur[r].q.y; xw[r][PW + 2] = cur[r].q.z; xw[r][PW + 3] = cur[r].q.w;
                }
                ssm::pair_t w2[W + 1];
#pragma unroll
                for (int k = 0; k <= W; ++k) w2[k] = *reinterpret_cast<const ssm::pair_t*>(taps + k);
                float o0[V], o1[V];
                conv_pieces<T, W, PW, SILU>(xw[0], xw[1], w2, w2[W], o0, o1);
                if constexpr (decltype(all_written)::value) {
                    *reinterpret_cast<uint4*>(op) = pack<T>(o0);
                    if (two) *reinterpret_cast<uint4*>(op + step) = pack<T>(o1);
                } else {
                    store_piece<T>(op, mask, nan, o0);
                    store_piece<T>(op + step, two ? mask : 0u, nan, o1);
                }
                op += 2 * step;
            }
        };
        if (whole) rows_of(std::true_type{});
        else rows_of(std::false_type{});
        return;
    }
    unsigned char* const out0 = static_cast<unsigned char*>(p.out) + dr * row_bytes;
    const unsigned char* const x0 = lo + dr * row_bytes;
    // pieces follow out's 16-byte grid; where x's differs the inputs are read by elements.  Every
    // lane runs every row (shuffles); rows past the last read nothing.  Several rows' pieces are
    // loaded before the first is used.
    constexpr int U = 2;
    for (int i0 = 0; i0 < p.rows_per_thread; i0 += U) {
      uint4 piece[U];
#pragma unroll
      for (int r = 0; r < U; ++r) {
        const int i = i0 + r;
        const bool row_ok = i < p.rows_per_thread && dr + (int64_t)i * ty < p.dim;
        const unsigned char* orow = out0 + i * step;
        const int64_t t = tile * span + (int64_t)px * V - (int)((reinterpret_cast<uintptr_t>(orow) & 15u) / ES);
        const unsigned char* xp = x0 + i * step + t * ES;
        // neighbours need the piece even where this lane writes nothing
        if (!row_ok || t >= p.total) {
            piece[r] = make_uint4(0u, 0u, 0u, 0u);
        } else if ((reinterpret_cast<uintptr_t>(xp) & 15u) == 0) {
            piece[r] = load_piece<T>(xp, lo, hi);
        } else {
            float v[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const unsigned char* q = xp + e * ES;
                v[e] = q >= lo && q < hi ? to_f<T>(*reinterpret_cast<const T*>(q)) : 0.f;
            }
            piece[r] = pack<T>(v);
        }
      }
      RowPiece<PW> rp[2];
#pragma unroll
      for (int r = 0; r < U; ++r) {
        const int i = i0 + r;
        const int64_t d = dr + (int64_t)i * ty;
        const bool row_ok = i < p.rows_per_thread && d < p.dim;
        unsigned char* orow = out0 + i * step;
        const int m = (int)((reinterpret_cast<uintptr_t>(orow) & 15u) / ES);
        const int64_t t = tile * span + (int64_t)px * V - m;     // first token of the piece
        const int bit = px * V - m + V;
        RowPiece<PW>& q = rp[r & 1];
        q.mask = row_ok ? __funnelshift_r(live[bit >> 5], live[(bit >> 5) + 1], bit & 31) & sel : 0u;
        q.nan = any_bad ? __funnelshift_r(bad[bit >> 5], bad[(bit >> 5) + 1], bit & 31) & q.mask : 0u;
        q.out = orow + t * ES;
        const unsigned char* xp = x0 + i * step + t * ES;
        uint32_t(&xw)[PW + 4] = q.xw;
        xw[PW] = piece[r].x; xw[PW + 1] = piece[r].y; xw[PW + 2] = piece[r].z; xw[PW + 3] = piece[r].w;
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            xw[k] = __shfl_up_sync(0xffffffffu, xw[4 + k], 1);
            if (edge && q.mask != 0u) {
                const unsigned char* b = xp + (k - PW) * 4;
                if constexpr (sizeof(T) == 4) {
                    xw[k] = b >= lo ? *reinterpret_cast<const uint32_t*>(b) : 0u;
                } else {
                    const uint32_t b0 = b >= lo ? *reinterpret_cast<const unsigned short*>(b) : 0u;
                    const uint32_t b1 = b + 2 >= lo ? *reinterpret_cast<const unsigned short*>(b + 2) : 0u;
                    xw[k] = b0 | b1 << 16;
                }
            }
        }
        if ((r & 1) && (rp[0].mask | rp[1].mask) != 0u) {
            float o0[V], o1[V];
            ssm::pair_t w[W + 1];
#pragma unroll
            for (int k = 0; k <= W; ++k) w[k] = *reinterpret_cast<const ssm::pair_t*>(taps + (i >> 1) * (W + 1) + k);
            conv_pieces<T, W, PW, SILU>(rp[0].xw, rp[1].xw, w, w[W], o0, o1);
            store_piece<T>(rp[0].out, rp[0].mask, rp[0].nan, o0);
            store_piece<T>(rp[1].out, rp[1].mask, rp[1].nan, o1);
        }
      }
    }
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) conv1d_packed_kernel(const PackedConv p) {
    if constexpr (W > 1) {                              // width 1 keeps no history
        if (blockIdx.x < p.head_ctas) {
            sequence_heads<T, W>(p, blockIdx.x);
            return;
        }
    }
    sequence_bodies<T, W, SILU>(p, blockIdx.x - (unsigned)p.head_ctas);
}

template <typename T, int W>
int launch_packed(PackedConv p, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int64_t pieces = (p.total + V - 1 + V - 1) / V;   // of a row, its first one up to V-1 tokens early
    p.log_tx = 4;
    while (p.log_tx < 7 && 1 << p.log_tx < pieces) ++p.log_tx;
    const int tx = 1 << p.log_tx, ty = kThreads / tx;
    const int64_t tt = p.total > 0 ? (pieces + tx - 1) / tx : 0;
    // enough rows per CTA to carry the making of the mask, as long as 8 CTAs per SM remain; two at least,
    // which work together (1013 tokens x 1536 channels 6.2 us, with four 7.6)
    int rows = 2;
    while (rows * ty < kTapRows && rows < 64 && tt * ((p.dim + ty - 1) / ty) / (2 * rows) >= 148 * 8) rows *= 2;
    p.rows_per_thread = rows;
    const int64_t rtiles = (p.dim + (int64_t)ty * rows - 1) / ((int64_t)ty * rows);
    const int64_t head_tiles = (p.dim + kThreads - 1) / kThreads;
    p.head_ctas = W > 1 ? p.n_seq * head_tiles : 0;
    const int64_t ctas = p.head_ctas + tt * rtiles;
    if (ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    if (ctas == 0) return SSM_OK;
    p.head_tiles = (unsigned)head_tiles;
    p.time_tiles = (unsigned)(tt > 0 ? tt : 1);
    if (p.silu) conv1d_packed_kernel<T, W, true><<<(unsigned)ctas, kThreads, 0, s>>>(p);
    else conv1d_packed_kernel<T, W, false><<<(unsigned)ctas, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T>
int launch_packed_t(const PackedConv& p, int width, cudaStream_t s) {
    switch (width) {
        case 1: return launch_packed<T, 1>(p, s);
        case 2: return launch_packed<T, 2>(p, s);
        case 3: return launch_packed<T, 3>(p, s);
        case 4: return launch_packed<T, 4>(p, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

// -------------------------------------------------------------- single tokens

struct TokenConv {
    const void* x;
    const float *w, *bias;
    void* out;
    void* states;
    const int* slots;
    int64_t batch, dim, n_slots, slot_stride;
    int silu;
    int w_vec;
};

// C channels per thread, of one row: 16 bytes of x and out and W-1 times 16 bytes of the slot
// (C = V), or one channel (C = 1) where those are not 16-byte aligned.
template <typename T, int W, int C>
__global__ void __launch_bounds__(128) conv1d_update_kernel(const TokenConv p) {
    const int64_t d = ((int64_t)blockIdx.x * 128 + threadIdx.x) * C;
    if (d >= p.dim) return;
    // the taps and the bias of the thread's channels, ahead of the slot's chain of loads
    float w[C * W], bias[C];
    if (C * W % 4 == 0 && p.w_vec) {
#pragma unroll
        for (int k = 0; k < C * W; k += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(p.w + d * W + k));
            w[k] = q.x; w[(k + 1) % (C * W)] = q.y; w[(k + 2) % (C * W)] = q.z; w[(k + 3) % (C * W)] = q.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < C * W; ++k) w[k] = __ldg(p.w + d * W + k);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) bias[c] = p.bias ? __ldg(p.bias + d + c) : 0.f;
    for (int64_t b = blockIdx.y; b < p.batch; b += gridDim.y) {
        const int slot = p.slots ? __ldg(p.slots + b) : (int)b;
        const ssm::SlotKind kind = ssm::slot_kind(slot, p.n_slots);
        if (kind == ssm::kSlotPad) continue;
        float x[C], o[C], h[C * (W > 1 ? W - 1 : 1)];
        T* st = static_cast<T*>(p.states) + (kind == ssm::kSlotLive ? slot : 0) * p.slot_stride + d * (W - 1);
        const T* xr = static_cast<const T*>(p.x) + b * p.dim + d;
        T* orow = static_cast<T*>(p.out) + b * p.dim + d;
        if constexpr (C > 1) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(xr));
            unpack<T>(q, x);
        } else {
            x[0] = to_f<T>(*xr);
        }
        if (W > 1 && kind == ssm::kSlotLive) {
            if constexpr (C > 1) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) unpack<T>(reinterpret_cast<const uint4*>(st)[k], h + k * C);
            } else {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) h[k] = to_f<T>(st[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < C * (W - 1); ++k) h[k] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v = bias[c];
#pragma unroll
            for (int k = 0; k < W - 1; ++k) v = fmaf(w[c * W + k], h[c * (W - 1) + k], v);
            v = fmaf(w[c * W + W - 1], x[c], v);
            o[c] = p.silu ? ssm::silu1(v) : v;
            if (kind == ssm::kSlotBad) o[c] = __int_as_float(0x7FC00000);
        }
        // the oldest input leaves, this one enters
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) h[c * (W - 1) + k] = h[c * (W - 1) + k + 1];
            if (W > 1) h[c * (W - 1) + W - 2] = x[c];
        }
        if constexpr (C > 1) {
            *reinterpret_cast<uint4*>(orow) = pack<T>(o);
            if (kind == ssm::kSlotLive) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) reinterpret_cast<uint4*>(st)[k] = pack<T>(h + k * C);
            }
        } else {
            *orow = from_f<T>(o[0]);
            if (kind == ssm::kSlotLive) {
#pragma unroll
                for (int k = 0; k < W - 1; ++k) st[k] = from_f<T>(h[k]);
            }
        }
    }
}

template <typename T, int W>
int launch_update(const TokenConv& p, bool vec, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const int64_t per = vec ? V : 1;
    const int64_t bx = (p.dim / per + (p.dim % per ? 1 : 0) + 127) / 128;
    const int64_t by = p.batch < kMaxGridY ? p.batch : kMaxGridY;
    const dim3 g((unsigned)bx, (unsigned)by);
    if (vec) conv1d_update_kernel<T, W, V><<<g, 128, 0, s>>>(p);
    else conv1d_update_kernel<T, W, 1><<<g, 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T>
int launch_update_t(const TokenConv& p, int width, bool vec, cudaStream_t s) {
    switch (width) {
        case 1: return launch_update<T, 1>(p, vec, s);
        case 2: return launch_update<T, 2>(p, vec, s);
        case 3: return launch_update<T, 3>(p, vec, s);
        case 4: return launch_update<T, 4>(p, vec, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

}  // namespace

extern "C" int ssm_causal_conv1d_packed_fwd(int64_t dim, int64_t total, int64_t n_seq, int32_t width, int32_t io_dtype,
                                            const void* x, const float* w, const float* bias, int silu,
                                            const int32_t* cu_seqlens, const int32_t* slots, const uint8_t* has_state,
                                            void* states, int64_t n_slots, int64_t slot_stride, void* out,
                                            ssm_stream_t stream) {
    if (dim <= 0 || total < 0 || n_seq < 0 || n_slots < 0) return SSM_ERR_INVALID_ARG;
    if (dim > (1 << 24) || total > 0x7FFFFFFF || n_seq > 0x7FFFFFFF || n_slots > 0x7FFFFFFF) return SSM_ERR_INVALID_ARG;
    if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (width < 1 || width > kMaxWidth) return SSM_ERR_UNSUPPORTED;
    if (n_seq == 0) return SSM_OK;
    if (!w || !cu_seqlens || (width > 1 && !states)) return SSM_ERR_INVALID_ARG;
    if (total > 0 && (!x || !out || x == out)) return SSM_ERR_INVALID_ARG;
    if (width > 1 && slot_stride < dim * (width - 1)) return SSM_ERR_INVALID_ARG;
    const uintptr_t esz = io_dtype == SSM_BF16 ? 2 : 4;
    if (!all_aligned(esz, {x, out, states}) || !all_aligned(4, {w, bias, cu_seqlens, slots})) return SSM_ERR_INVALID_ARG;
    PackedConv p{};
    p.x = x; p.w = w; p.bias = bias; p.out = out; p.states = states;
    p.cu = cu_seqlens; p.slots = slots; p.has_state = has_state;
    p.dim = dim; p.total = total; p.n_seq = n_seq; p.n_slots = n_slots; p.slot_stride = slot_stride;
    p.silu = silu ? 1 : 0;
    p.aligned = total * (int64_t)esz % 16 == 0 && all_aligned(16, {x, out});
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return io_dtype == SSM_BF16 ? launch_packed_t<__nv_bfloat16>(p, width, s) : launch_packed_t<float>(p, width, s);
}

extern "C" int ssm_causal_conv1d_update(int64_t batch, int64_t dim, int32_t width, int32_t io_dtype, const void* x,
                                        const float* w, const float* bias, int silu, const int32_t* slots, void* states,
                                        int64_t n_slots, int64_t slot_stride, void* out, ssm_stream_t stream) {
    if (batch < 0 || dim <= 0 || n_slots < 0) return SSM_ERR_INVALID_ARG;
    if (dim > (1 << 24) || batch > 0x7FFFFFFF || n_slots > 0x7FFFFFFF) return SSM_ERR_INVALID_ARG;
    if (io_dtype != SSM_F32 && io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    if (width < 1 || width > kMaxWidth) return SSM_ERR_UNSUPPORTED;
    if (batch == 0) return SSM_OK;
    if (!x || !w || !out || (width > 1 && !states)) return SSM_ERR_INVALID_ARG;
    if (width > 1 && slot_stride < dim * (width - 1)) return SSM_ERR_INVALID_ARG;
    const int64_t esz = io_dtype == SSM_BF16 ? 2 : 4, V = 16 / esz;
    if (!all_aligned(esz, {x, out, states}) || !all_aligned(4, {w, bias, slots})) return SSM_ERR_INVALID_ARG;
    const bool vec = dim % V == 0 && all_aligned(16, {x, out, states}) && slot_stride % V == 0;
    TokenConv p{};
    p.x = x; p.w = w; p.bias = bias; p.out = out; p.states = states; p.slots = slots;
    p.batch = batch; p.dim = dim; p.n_slots = n_slots; p.slot_stride = slot_stride; p.silu = silu ? 1 : 0;
    p.w_vec = aligned_to(w, 16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return io_dtype == SSM_BF16 ? launch_update_t<__nv_bfloat16>(p, width, vec, s)
                                : launch_update_t<float>(p, width, vec, s);
}
