#pragma once
// The selective scan over prompts packed end to end, each continuing from its slot of a state
// pool (declared in include/ssm_scan.h as ssm_selective_scan_packed_fwd): the recurrence of the
// Mamba "architecture-details" page, section "How S6 Works", per sequence.
//
// Mathematics.  Per sequence, channel d and state n, over the sequence's own tokens t:
//   dt = softplus(delta + bias), h = exp(dt A) h + dt u B, y = sum_n C h + D u, out = y silu(z).
// A stretch of tokens maps the state by h -> P h + h_loc, with P = exp(A sum dt) and h_loc the
// end state from zero, so a sequence can be cut into chunks that run at the same time:
//   launch 1: the first chunk of each sequence in full; every middle chunk for (sum dt, h_loc) only
//   launch 2: every later chunk joins its predecessors' pairs and runs in full.
// Uncut sequences need launch 1 alone.  A middle chunk's exps are paid twice, so sequences are
// cut only where their count leaves SMs without work (choose_chunk).
//
// Bound: one ex2 per (t, channel, state), 16 per clock and SM, in the per-channel layout; the
// fp32 pipe (three operations per (t, channel, state)) in the per-head layout, whose decay is
// one ex2 per (t, channel).
//
// Layout.  A lane holds S states (4, from dstate 64 on 8) of CPL channels, N/S lanes a channel
// group: the B and C of a step, fp32 in shared memory, then serve CPL channels per load, and the
// sum over states crosses lanes only log2(N/S) times.  The tokens of a block (64 bytes of a row)
// are staged by 16-byte asynchronous copies one block ahead; rows whose starts are not 16-byte
// aligned are copied as the aligned pieces that hold them and read at their offset.  The warps of a
// CTA meet twice per block, around the conversion of B and C.
//
// Measured on one B200, bf16, dstate 16: 16384 tokens in 24 ragged prompts x 4096 channels 464 us
// in the mean of three draws (413 to 522 us for longest prompts of 1845 to 3954 tokens, whose chain of
// blocks is most of it), one prompt of 8191 tokens x 1536 channels 198 us in 24 chunks, of 8192 (rows on
// the 16-byte grid) 165.  MUFU two thirds busy while SMs have work.
// Uncut calls, on other draws: three CTAs an SM with more registers each 510 us and per-lane rows of y 492,
// against 538 of four CTAs that sum y by shuffles, as cut calls do (three CTAs there 213 against 200).
// Against it, from 492 and 200:
// eight states of two channels per lane (half the warps, longer chains) 721 and 260 us; blocks of 32
// bytes 636 and 226; eight warps a CTA 611 and 221; a quarter of the exponentials as polynomials on
// the fp32 pipe 4 to 9 % more (the issue slots they need are as scarce); outputs stored without their
// pass through shared memory 3 % more.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // ex2_approx, f32x2 operations, softplus, silu, window_reduce
#include "slots.h"
#include "ssm_scan.h"

namespace ssm {
namespace packed {

using ssm::add2;
using ssm::dup2;
using ssm::ex2_approx;
using ssm::fma2;
using ssm::kLog2e;
using ssm::mul2;

struct PackedParams {
    const void *u, *delta, *B, *C, *z;
    const float *A, *D, *bias;
    void* out;
    float* states;
    const int *cu, *slots;
    const unsigned char* has_state;
    float *ws_h, *ws_p;      // per chunk: (dim, dstate) states and, per channel, sum dt (or the product of decays)
    int64_t n_seq, total, n_slots, slot_stride;
    int64_t dim, nheads, ngroups, group_dim, head_dim;
    int64_t chunk;           // tokens of a chunk; 0: sequences are not cut
    int64_t n_chunks;        // chunks the workspace has room for
    unsigned tiles_per_group, n_tiles;
    int softplus, phase, state_vec;
    int grid16;              // every row starts on the 16-byte grid
    int stall;               // tensor cores: the block whose wait runs out (a test's), and the limit of waits
    uint64_t wait_ns;
};

template <typename T, int N, bool HEAD, bool ALIGNED, bool CUT = true>
struct PackedCfg {
    static constexpr bool kAligned = ALIGNED;
    static constexpr int ESZ = sizeof(T);
    static constexpr int V = 16 / ESZ;                  // elements per 16-byte piece
    static constexpr int RB = 64;                       // bytes of a row's block
    static constexpr int TB = RB / ESZ;                 // steps per block
    static constexpr int S = N <= 32 ? 4 : 8;           // states per lane
    static constexpr int TPC = N / S;                   // lanes per channel
    static constexpr int CPL = N == 128 ? 4 : 2;        // channels per lane
    static constexpr int LG = 32 / TPC;                 // lane groups of a warp
    static constexpr int CW = LG * CPL;                 // channels per warp
    static constexpr int W = N == 8 ? 2 : 4;            // warps
    static constexpr int CT = W * CW;                   // channels per tile
    static constexpr int NT = 32 * W;
    // CTAs per SM, at least.  Uncut calls end with the longest sequences' CTAs, which more registers
    // make faster; cut ones want as many chunks at a time as fit.
    static constexpr int CTAS = N > 32 ? 2 : CUT ? 4 : 3;
    static constexpr int WT = CPL * 4 >= TPC ? 4 : 8;   // steps per window
    static constexpr int PA = RB / 16;                  // 16-byte pieces of a row's block
    static constexpr int PIECES = ALIGNED ? PA : PA + 1;    // that hold it
    // bytes of a staged row.  Eight rows' pieces read at once have to lie in different banks:
    // aligned rows swap their pieces by bits of the row, the others are an odd number of pieces long
    static constexpr int PITCH = ALIGNED ? RB : RB + 16;
    __device__ static constexpr int piece_off(int row, int piece) {
        return row * PITCH + (ALIGNED ? piece ^ (row >> 1 & 3) : piece) * 16;
    }
    static constexpr int R_U = 0, R_Z = CT, R_DT = 2 * CT, R_B = 3 * CT, R_C = 3 * CT + N, ROWS = 3 * CT + 2 * N;
    static constexpr int STAGE = ROWS * PITCH;
    // steps of a prologue or epilogue item (one channel's)
    static constexpr int PS = CW * TB >= 256 ? 8 : 4;
    static constexpr int ITEMS = CW * TB / PS / 32;     // per lane
    static constexpr int OFF_BC = 2 * STAGE;            // fp32 [step][B of all states | C of all states]
    static constexpr int OFF_Q = OFF_BC + TB * 2 * N * 4;   // per warp: [step][channel] (dt or decay, dt u), then y
    // Uncut calls have the shared memory for a row of partial sums of y per lane and step, which the
    // epilogue adds; the others add them by shuffles, into q's place.  The rows run over q, which
    // ends where they end and whose steps are no longer: a step's row covers no later step of q.
    static constexpr bool YROWS = !CUT && N <= 32;
    static constexpr int Q_BYTES = TB * CW * 8;
    static constexpr int Q_WARP = YROWS ? TB * 32 * CPL * 4 : Q_BYTES;
    static_assert(!YROWS || (CPL == 2 && Q_WARP >= Q_BYTES), "q ends where the rows end");
    // where lane (lg, j) puts its sum for channel ch of step t (floats): a step's sums of a channel lie
    // side by side, and those of eight neighbouring channels in different banks
    __device__ static constexpr int y_off(int t, int lg, int ch, int j) {
        return t * 32 * CPL + ch * 32 + (lg ^ (ch * (LG / 2))) * TPC + j;
    }
    static constexpr int OFF_PAR = OFF_Q + W * Q_WARP;  // bias, D, and the head's A (log2 e folded in), per channel
    static constexpr int OFF_MISC = OFF_PAR + 3 * CT * 4;
    static constexpr int SMEM = OFF_MISC + 64;
    static_assert(CW * TB / PS % 32 == 0, "whole items per lane");
    static_assert(TB % WT == 0 && (CPL * WT) % 2 == 0, "whole windows");
};

__device__ __forceinline__ void cp16(unsigned dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// Elements off the 16-byte grid of the first of a row, for a row that starts at `p`.
template <typename T> __device__ __forceinline__ int skew(const void* p) {
    return (int)((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// CNT elements of a staged row, from element e on (aligned: a multiple of CNT).
template <class Cf, int CNT>
__device__ __forceinline__ void read_row(const unsigned char* stage, int row, int e, float (&v)[CNT]) {
    constexpr int V = Cf::V;
    if constexpr (Cf::ESZ == 4) {
        if constexpr (Cf::kAligned) {
#pragma unroll
            for (int i = 0; i < CNT; i += 4) {
                const float4 q = *reinterpret_cast<const float4*>(stage + Cf::piece_off(row, (e + i) / V));
                v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < CNT; ++i) v[i] = *reinterpret_cast<const float*>(stage + Cf::piece_off(row, 0) + (e + i) * 4);
        }
    } else {
        uint32_t w[CNT / 2];
        if constexpr (Cf::kAligned) {
            const unsigned char* p = stage + Cf::piece_off(row, e / V);
            if constexpr (CNT == 8) {
                const uint4 q = *reinterpret_cast<const uint4*>(p);
                w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
            } else {
                const uint2 q = *reinterpret_cast<const uint2*>(p + e % V * 2);
                w[0] = q.x; w[1] = q.y;
            }
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(stage + Cf::piece_off(row, 0) + ((e * 2) & ~3));
            const int sh = (e & 1) * 16;
            uint32_t lo = p[0];
#pragma unroll
            for (int i = 0; i < CNT / 2; ++i) {
                const uint32_t hi = p[i + 1];
                w[i] = __funnelshift_r(lo, hi, sh);
                lo = hi;
            }
        }
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

template <class Cf, int CNT>
__device__ __forceinline__ void write_row(unsigned char* stage, int row, int e, const float (&v)[CNT]) {
    constexpr int V = Cf::V;
    if constexpr (Cf::ESZ == 4) {
        if constexpr (Cf::kAligned) {
#pragma unroll
            for (int i = 0; i < CNT; i += 4)
                *reinterpret_cast<float4*>(stage + Cf::piece_off(row, (e + i) / V)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < CNT; ++i) *reinterpret_cast<float*>(stage + Cf::piece_off(row, 0) + (e + i) * 4) = v[i];
        }
    } else {
        uint32_t w[CNT / 2];
#pragma unroll
        for (int i = 0; i < CNT / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if constexpr (Cf::kAligned) {
            unsigned char* p = stage + Cf::piece_off(row, e / V);
            if constexpr (CNT == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(p + e % V * 2) = make_uint2(w[0], w[1]);
        } else {
            unsigned short* p = reinterpret_cast<unsigned short*>(stage + Cf::piece_off(row, 0)) + e;
#pragma unroll
            for (int i = 0; i < CNT; ++i) p[i] = (unsigned short)(w[i / 2] >> (16 * (i & 1)));
        }
    }
}

// Elements [a, b) of a 16-byte piece of V, in the largest aligned parts: up to the middle ever larger
// ones, then ever smaller.
template <int V, int ESZ>
__device__ __forceinline__ void store_part(unsigned char* dst, const unsigned char* src, int a, int b) {
    a = a < 0 ? 0 : a;
    b = b > V ? V : b;
    auto part = [&](auto word, int n) {
        using Word = decltype(word);
        *reinterpret_cast<Word*>(dst + a * ESZ) = *reinterpret_cast<const Word*>(src + a * ESZ);
        a += n;
    };
    if constexpr (ESZ == 2) {
        if ((a & 1) && a < b) part((unsigned short)0, 1);
        if ((a & 2) && a + 2 <= b) part(0u, 2);
        if (a + 4 <= b) part(uint2{}, 4);
        if (a + 2 <= b) part(0u, 2);
        if (a < b) part((unsigned short)0, 1);
    } else {
        if ((a & 1) && a < b) part(0u, 1);
        if (a + 2 <= b) part(uint2{}, 2);
        if (a < b) part(0u, 1);
    }
}

// What a CTA works on: one channel tile of one chunk of one sequence.
struct Task {
    int g, ci0, d0;          // group, first channel within it, first channel
    int nch;                 // channels of the tile
    int t0, t1;              // tokens
    int chunk_id;            // of the workspace
    int k;                   // chunk of its sequence
    int slot;
    bool last;
    bool has;                // starts from the slot's state
};

// One chunk (all of a sequence unless CUT).  LOCAL: only its decay and its end state from zero.
template <typename T, int N, bool HEAD, bool ALIGNED, bool LOCAL, bool CUT>
__device__ __forceinline__ void run_chunk(const PackedParams& p, const Task& tk, unsigned char* smem) {
    using Cf = PackedCfg<T, N, HEAD, ALIGNED, CUT>;
    constexpr int S = Cf::S, TPC = Cf::TPC, CPL = Cf::CPL, CW = Cf::CW, CT = Cf::CT, TB = Cf::TB, V = Cf::V;
    constexpr int ESZ = Cf::ESZ, NT = Cf::NT, WT = Cf::WT, PS = Cf::PS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lg = lane / TPC, j = lane % TPC;
    const int64_t L = p.total;
    const int head_dim = (int)p.head_dim;
    const int h_lo = HEAD ? tk.d0 / head_dim : tk.d0;                 // first delta row of the tile
    const int n_dt = HEAD ? (tk.d0 + tk.nch - 1) / head_dim - h_lo + 1 : tk.nch;
    float* bc = reinterpret_cast<float*>(smem + Cf::OFF_BC);
    float* yrows = reinterpret_cast<float*>(smem + Cf::OFF_Q + warp * Cf::Q_WARP);
    float2* q = reinterpret_cast<float2*>(smem + Cf::OFF_Q + (warp + 1) * Cf::Q_WARP - Cf::Q_BYTES);
    float* s_bias = reinterpret_cast<float*>(smem + Cf::OFF_PAR);
    float* s_D = s_bias + CT;
    float* s_a = s_D + CT;

    // the first step of block 0 sits on the 16-byte grid of an aligned row
    const int tb0 = tk.t0 & ~(V - 1);
    const int nblk = (tk.t1 - tb0 + TB - 1) / TB;

    const unsigned char* ub = static_cast<const unsigned char*>(p.u) + (int64_t)tk.d0 * L * ESZ;
    const unsigned char* zb = p.z ? static_cast<const unsigned char*>(p.z) + (int64_t)tk.d0 * L * ESZ : nullptr;
    const unsigned char* db = static_cast<const unsigned char*>(p.delta) + (int64_t)h_lo * L * ESZ;
    const unsigned char* Bb = static_cast<const unsigned char*>(p.B) + (int64_t)tk.g * N * L * ESZ;
    const unsigned char* Cb = static_cast<const unsigned char*>(p.C) + (int64_t)tk.g * N * L * ESZ;
    unsigned char* ob = static_cast<unsigned char*>(p.out) + (int64_t)tk.d0 * L * ESZ;

    // Copies of `rows` rows of a tensor (first row at `base`) into staged rows r0 .. of a stage.
    // A piece is copied if it holds a token of the chunk; others keep what the stage held, and
    // nothing computed from them is used.  `lo`, `hi`: the tensor's bytes; a piece that starts
    // before them (a base off the 16-byte grid) is copied by elements, one that ends behind them
    // is cut.
    auto stage_rows = [&](int stage, int r0, const unsigned char* base, int rows, int tb, const unsigned char* lo,
                          const unsigned char* hi) {
        unsigned char* sb = smem + stage * Cf::STAGE;
        if constexpr (ALIGNED) {
            const int g = tid % Cf::PA;
            const int ts = tb + g * V;
            if (ts < tk.t1 && ts + V > tk.t0) {
                const unsigned dst = ssm::smem_u32(sb);
                const unsigned char* src = base + (int64_t)ts * ESZ;
                for (int r = tid / Cf::PA; r < rows; r += NT / Cf::PA)
                    cp16(dst + Cf::piece_off(r0 + r, g), src + (int64_t)r * L * ESZ, 16);
            }
        } else {
            // eight lanes a row, those past its pieces idle; rows eight apart are alike on the grid
            static_assert(Cf::PIECES <= 8 && 8 * Cf::ESZ % 16 == 0, "a thread's rows have one skew");
            const int g = tid & 7, r1 = tid >> 3;
            if (g >= Cf::PIECES) return;
            const unsigned char* src = base + (int64_t)r1 * L * ESZ;
            const int ts = tb + g * V - skew<T>(src);
            if (ts >= tk.t1 || ts + V <= tk.t0) return;
            src += (int64_t)ts * ESZ;
            unsigned char* dst = sb + Cf::piece_off(r0 + r1, g);
            const int64_t step = (int64_t)(NT / 8) * L * ESZ;
            for (int r = r1; r < rows; r += NT / 8, src += step, dst += NT / 8 * Cf::PITCH) {
                if (src >= lo) {
                    const int64_t left = hi - src;
                    cp16(ssm::smem_u32(dst), src, left < 16 ? (int)left : 16);
                } else {
                    for (int e = 0; e < V; ++e)
                        if (src + e * ESZ >= lo && src + e * ESZ < hi)
                            *reinterpret_cast<T*>(dst + e * ESZ) = *reinterpret_cast<const T*>(src + e * ESZ);
                }
            }
        }
    };
    auto bytes_of = [&](int64_t rows) { return rows * L * ESZ; };
    auto issue = [&](int kb) {
        const int tb = tb0 + kb * TB;
        const int st = kb & 1;
        auto put = [&](int r0, const unsigned char* base, int rows, const void* t, int64_t t_rows) {
            const unsigned char* lo = static_cast<const unsigned char*>(t);
            stage_rows(st, r0, base, rows, tb, lo, lo + bytes_of(t_rows));
        };
        put(Cf::R_U, ub, tk.nch, p.u, p.dim);
        if (!LOCAL && zb) put(Cf::R_Z, zb, tk.nch, p.z, p.dim);
        put(Cf::R_DT, db, n_dt, p.delta, p.nheads);
        put(Cf::R_B, Bb, N, p.B, p.ngroups * N);
        if (!LOCAL) put(Cf::R_C, Cb, N, p.C, p.ngroups * N);
        cp_commit();
    };

    __syncthreads();
    if (nblk > 0) issue(0);
    for (int c = tid; c < CT; c += NT) {
        const int d = tk.d0 + (c < tk.nch ? c : 0);
        const int hd = HEAD ? d / head_dim : d;
        s_bias[c] = p.bias ? __ldg(p.bias + hd) : 0.f;
        s_D[c] = p.D ? __ldg(p.D + d) : 0.f;
        if constexpr (HEAD) s_a[c] = __ldg(p.A + hd) * kLog2e;
    }

    // this lane's channels and states
    float2 h[CPL][S / 2], a2[HEAD ? 1 : CPL][S / 2];
    float acc[CPL];
    bool ok[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int lc = warp * CW + lg * CPL + c;
        ok[c] = lc < tk.nch;
        const int64_t d = tk.d0 + (ok[c] ? lc : 0);
        acc[c] = HEAD ? 1.f : 0.f;
        if constexpr (!HEAD) {
            const float* ar = p.A + d * N + j * S;
#pragma unroll
            for (int s = 0; s < S / 2; ++s) a2[c][s] = make_float2(__ldg(ar + 2 * s) * kLog2e, __ldg(ar + 2 * s + 1) * kLog2e);
        }
        // the state that enters the chunk
        if (CUT && !LOCAL && tk.k > 0) {
            // join the chunks before: the first holds a state, the later ones (decay, state from zero)
            const int64_t c0 = tk.chunk_id - tk.k;
            const float* hr = p.ws_h + (c0 * p.dim + d) * N + j * S;
#pragma unroll
            for (int s = 0; s < S / 2; ++s) h[c][s] = __ldcg(reinterpret_cast<const float2*>(hr) + s);
            for (int i = 1; i < tk.k; ++i) {
                const float pr = __ldcg(p.ws_p + (c0 + i) * p.dim + d);
                const float* hi = p.ws_h + ((c0 + i) * p.dim + d) * N + j * S;
#pragma unroll
                for (int s = 0; s < S / 2; ++s) {
                    const float2 loc = __ldcg(reinterpret_cast<const float2*>(hi) + s);
                    float2 dec;
                    if constexpr (HEAD) {
                        dec = dup2(pr);
                    } else {
                        const float2 arg = mul2(dup2(pr), a2[c][s]);
                        dec = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
                    }
                    h[c][s] = fma2(dec, h[c][s], loc);
                }
            }
        } else if (!LOCAL && tk.has) {
            const float* hr = p.states + (int64_t)tk.slot * p.slot_stride + d * N + j * S;
            if (p.state_vec) {
#pragma unroll
                for (int s = 0; s < S / 2; s += 2) {
                    const float4 v = *reinterpret_cast<const float4*>(hr + 2 * s);
                    h[c][s] = make_float2(v.x, v.y);
                    h[c][s + 1] = make_float2(v.z, v.w);
                }
            } else {
#pragma unroll
                for (int s = 0; s < S / 2; ++s) h[c][s] = make_float2(hr[2 * s], hr[2 * s + 1]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < S / 2; ++s) h[c][s] = make_float2(0.f, 0.f);
        }
    }

    for (int kb = 0; kb < nblk; ++kb) {
        const int tb = tb0 + kb * TB;
        // the chunk's steps of the block: [lo, hi)
        const int lo = tk.t0 > tb ? tk.t0 - tb : 0;
        const int hi = tk.t1 - tb < TB ? tk.t1 - tb : TB;
        const bool whole = lo == 0 && hi == TB;
        unsigned char* sb = smem + (kb & 1) * Cf::STAGE;
        cp_wait_all();
        __syncthreads();   // the block is staged, and every warp is done with the block before
        if (kb + 1 < nblk) issue(kb + 1);

        // B and C to fp32, [step][state]; steps outside the chunk become zero
        constexpr int CV = ESZ == 2 ? 8 : 4;
        constexpr int BCR = LOCAL ? N : 2 * N;
        for (int i = tid; i < BCR * (TB / CV); i += NT) {
            const int r = i % BCR, e0 = i / BCR * CV;
            const unsigned char* src = r < N ? Bb : Cb;
            const int m = ALIGNED ? 0 : skew<T>(src + (int64_t)(r < N ? r : r - N) * L * ESZ);
            float v[CV];
            read_row<Cf, CV>(sb, Cf::R_B + r, m + e0, v);
#pragma unroll
            for (int e = 0; e < CV; ++e) bc[(e0 + e) * 2 * N + r] = whole || (e0 + e >= lo && e0 + e < hi) ? v[e] : 0.f;
        }
        // prologue: dt (or the decay) and dt u of the warp's channels
#pragma unroll
        for (int it = 0; it < Cf::ITEMS; ++it) {
            const int idx = lane + 32 * it, c = idx % CW, e0 = idx / CW * PS;
            const int lc = warp * CW + c;
            const int cl = lc < tk.nch ? lc : 0;
            const int dr = HEAD ? (tk.d0 + cl) / head_dim - h_lo : lc;
            float x[PS], uv[PS];
            const int mu = ALIGNED ? 0 : skew<T>(ub + (int64_t)lc * L * ESZ);
            const int md = ALIGNED ? 0 : skew<T>(db + (int64_t)dr * L * ESZ);
            read_row<Cf, PS>(sb, Cf::R_U + lc, mu + e0, uv);
            read_row<Cf, PS>(sb, Cf::R_DT + dr, md + e0, x);
            const float bias = s_bias[lc];
            const float ah = HEAD ? s_a[lc] : 0.f;
#pragma unroll
            for (int e = 0; e < PS; e += 2) {
                const float2 xb = add2(make_float2(x[e], x[e + 1]), dup2(bias));
                float2 dt = p.softplus ? ssm::softplus2(xb) : xb;
                float2 du = mul2(dt, make_float2(uv[e], uv[e + 1]));
                if (!whole) {
                    // steps outside the chunk: no decay, no input
                    if (!(e0 + e >= lo && e0 + e < hi)) { dt.x = 0.f; du.x = 0.f; }
                    if (!(e0 + e + 1 >= lo && e0 + e + 1 < hi)) { dt.y = 0.f; du.y = 0.f; }
                }
                if constexpr (HEAD) dt = make_float2(ex2_approx(dt.x * ah), ex2_approx(dt.y * ah));
                q[(e0 + e) * CW + c] = make_float2(dt.x, du.x);
                q[(e0 + e + 1) * CW + c] = make_float2(dt.y, du.y);
            }
        }
        __syncthreads();   // bc is complete; the warp's own q rows too

        // the recurrence (two windows at a time: the second one's loads pass under the first one's sums)
        const int w_end = (hi + WT - 1) / WT;
#pragma unroll 2
        for (int w = lo / WT; w < w_end; ++w) {
            float yw[CPL * WT];
#pragma unroll
            for (int tt = 0; tt < WT; ++tt) {
                const int t = w * WT + tt;
                float2 bb[S / 2], cc[S / 2];
                const float* br = bc + t * 2 * N + j * S;
#pragma unroll
                for (int s = 0; s < S / 2; s += 2) {
                    const float4 v = *reinterpret_cast<const float4*>(br + 2 * s);
                    bb[s] = make_float2(v.x, v.y);
                    bb[s + 1] = make_float2(v.z, v.w);
                    if constexpr (!LOCAL) {
                        const float4 x = *reinterpret_cast<const float4*>(br + N + 2 * s);
                        cc[s] = make_float2(x.x, x.y);
                        cc[s + 1] = make_float2(x.z, x.w);
                    }
                }
                const float4* qr = reinterpret_cast<const float4*>(q + t * CW + lg * CPL);
#pragma unroll
                for (int c2 = 0; c2 < CPL; c2 += 2) {
                    const float4 qq = qr[c2 / 2];
#pragma unroll
                    for (int ch = 0; ch < 2; ++ch) {
                        const int c = c2 + ch;
                        const float dv = ch ? qq.z : qq.x;
                        const float2 d2 = dup2(dv), du2 = dup2(ch ? qq.w : qq.y);
                        float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int s = 0; s < S / 2; ++s) {
                            float2 dA;
                            if constexpr (HEAD) {
                                dA = d2;
                            } else {
                                const float2 arg = mul2(d2, a2[c][s]);
                                dA = make_float2(ex2_approx(arg.x), ex2_approx(arg.y));
                            }
                            h[c][s] = fma2(dA, h[c][s], mul2(du2, bb[s]));
                            if constexpr (!LOCAL) y2 = fma2(cc[s], h[c][s], y2);
                        }
                        if constexpr (LOCAL) {
                            if constexpr (HEAD) acc[c] *= dv;
                            else acc[c] += dv;
                        } else {
                            yw[c * WT + tt] = y2.x + y2.y;
                        }
                    }
                }
            }
            if constexpr (!LOCAL && Cf::YROWS) {
                __syncwarp();                           // every lane has read the window's q
#pragma unroll
                for (int tt = 0; tt < WT; ++tt)
#pragma unroll
                    for (int c = 0; c < CPL; ++c) yrows[Cf::y_off(w * WT + tt, lg, c, j)] = yw[c * WT + tt];
            }
            if constexpr (!LOCAL && !Cf::YROWS) {
                // sum over the lanes of a channel; y takes the place of dt in q, which every lane
                // of the channel has read before the shuffles
                int off = 0;
                constexpr int NV = CPL * WT;
                if constexpr (TPC > 1) ssm::window_reduce<NV, TPC>(yw, j, off);
                constexpr int KEPT = NV >= TPC ? NV / TPC : 1;
                if (TPC <= NV || j % (TPC > NV ? TPC / NV : 1) == 0) {
#pragma unroll
                    for (int i = 0; i < KEPT; ++i) {
                        const int c = (off + i) / WT, tt = (off + i) % WT;
                        q[(w * WT + tt) * CW + lg * CPL + c].x = yw[i];
                    }
                }
            }
        }
        if constexpr (!LOCAL) {
            __syncwarp();
            // epilogue: (y + D u) silu(z), staged in the delta rows (every warp is past reading them)
#pragma unroll
            for (int it = 0; it < Cf::ITEMS; ++it) {
                const int idx = lane + 32 * it, c = idx % CW, e0 = idx / CW * PS;
                const int lc = warp * CW + c;
                const int64_t ro = (int64_t)lc * L * ESZ;
                float uv[PS], zv[PS], o[PS];
                read_row<Cf, PS>(sb, Cf::R_U + lc, (ALIGNED ? 0 : skew<T>(ub + ro)) + e0, uv);
                if (zb) read_row<Cf, PS>(sb, Cf::R_Z + lc, (ALIGNED ? 0 : skew<T>(zb + ro)) + e0, zv);
                const float2 D2 = dup2(s_D[lc]);
                auto y_of = [&](int t) {
                    if constexpr (Cf::YROWS) {
                        // the lanes' sums, in the order of the shuffles
                        const float* r = yrows + Cf::y_off(t, c / CPL, c % CPL, 0);
                        float part[TPC];
#pragma unroll
                        for (int k = 0; k < TPC; k += 2) {
                            const float2 f = *reinterpret_cast<const float2*>(r + k);
                            part[k] = f.x;
                            part[k + 1] = f.y;
                        }
#pragma unroll
                        for (int m = TPC / 2; m >= 1; m >>= 1)
#pragma unroll
                            for (int k = 0; k < m; ++k) part[k] += part[k + m];
                        return part[0];
                    } else {
                        return q[t * CW + c].x;
                    }
                };
#pragma unroll
                for (int e = 0; e < PS; e += 2) {
                    float2 y = fma2(D2, make_float2(uv[e], uv[e + 1]), make_float2(y_of(e0 + e), y_of(e0 + e + 1)));
                    if (zb) y = mul2(y, ssm::silu2(make_float2(zv[e], zv[e + 1])));
                    o[e] = y.x;
                    o[e + 1] = y.y;
                }
                write_row<Cf, PS>(sb, Cf::R_DT + lc, (ALIGNED ? 0 : skew<T>(ob + ro)) + e0, o);
            }
            __syncwarp();
            // to global memory, a row's pieces on neighbouring lanes
            for (int i = lane; i < CW * Cf::PIECES; i += 32) {
                const int r = i / Cf::PIECES, g = i % Cf::PIECES, lc = warp * CW + r;
                if (lc >= tk.nch) continue;
                unsigned char* row = ob + (int64_t)lc * L * ESZ;
                const int e0 = g * V - (ALIGNED ? 0 : skew<T>(row));     // first step of the piece
                const unsigned char* src = sb + Cf::piece_off(Cf::R_DT + lc, g);
                unsigned char* dst = row + (int64_t)(tb + e0) * ESZ;
                if (e0 >= lo && e0 + V <= hi) {
                    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
                } else {
                    store_part<V, ESZ>(dst, src, lo - e0, hi - e0);
                }
            }
        }
    }

    // the state that leaves the chunk
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        if (!ok[c]) continue;
        const int64_t d = tk.d0 + warp * CW + lg * CPL + c;
        if (!LOCAL && tk.last) {
            float* hr = p.states + (int64_t)tk.slot * p.slot_stride + d * N + j * S;
            if (p.state_vec) {
#pragma unroll
                for (int s = 0; s < S / 2; s += 2)
                    *reinterpret_cast<float4*>(hr + 2 * s) = make_float4(h[c][s].x, h[c][s].y, h[c][s + 1].x, h[c][s + 1].y);
            } else {
#pragma unroll
                for (int s = 0; s < S / 2; ++s) { hr[2 * s] = h[c][s].x; hr[2 * s + 1] = h[c][s].y; }
            }
        } else if (CUT && (LOCAL || tk.k == 0)) {
            float* hr = p.ws_h + ((int64_t)tk.chunk_id * p.dim + d) * N + j * S;
#pragma unroll
            for (int s = 0; s < S / 2; ++s) __stcg(reinterpret_cast<float2*>(hr) + s, h[c][s]);
            if (LOCAL && j == 0) __stcg(p.ws_p + (int64_t)tk.chunk_id * p.dim + d, acc[c]);
        }
    }
}

// Finds the x-th work item of the call; all threads of the CTA call it.  Returns false behind the
// last one.  Items go by sequence, the long ones first so that no long one starts last: sequences
// are ranked by the bucket of their length (two per octave) and within it by number.  Cut
// sequences have ceil(length / chunk) items each, at least one, and keep their own order, which
// their chunks' places in the workspace follow.  CUT: the call may cut, `cut`: it does.  The workspace
// and the grid have room for the chunks of sequences that share no token; where bounds run backwards and
// there would be more, every sequence is one item.
template <bool CUT>
__device__ __forceinline__ bool find_item(const PackedParams& p, int64_t x, int64_t* sh, int nt, int64_t& seq, int64_t& k,
                                          bool& cut) {
    // sh: [0] sequence, [1] item of it, [2 ..] warp sums, [34 ..] counts of the buckets
    constexpr int kBuckets = 64;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = nt / 32;
    cut = CUT;
    if (p.n_seq <= 32) {
        // few sequences, one per lane: every warp finds the item by itself, by exact length
        int64_t len = -1;
        if (lane < p.n_seq) {
            const TokenRange r = token_range(p.cu, lane, p.total);
            len = r.hi - r.lo;
        }
        int first = 0, n = 0;                           // the lane's sequence has items [first, first + n)
        if constexpr (CUT) {
            n = len > 0 ? (int)((len + p.chunk - 1) / p.chunk) : len == 0;
            int inc = n;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += v;
            }
            first = inc - n;
            cut = __shfl_sync(0xffffffffu, inc, 31) <= p.n_chunks;
        }
        if (!cut) {
            n = len >= 0;
            first = 0;
            const int l = (int)len;
            for (int i = 0; i < (int)p.n_seq; ++i) {
                const int v = __shfl_sync(0xffffffffu, l, i);
                first += v > l || (v == l && i < lane);
            }
        }
        const unsigned mine = __ballot_sync(0xffffffffu, n > 0 && x >= first && x < (int64_t)first + n);
        if (mine == 0u) return false;
        seq = __ffs(mine) - 1;
        k = x - __shfl_sync(0xffffffffu, first, (int)seq);
        return true;
    }
    unsigned* count = reinterpret_cast<unsigned*>(sh + 2 + 32);
    auto bucket = [&](int64_t len) {
        if (len <= 0) return kBuckets - 1;
        const int e = 31 - __clz((int)len);
        const int half = e > 0 ? (int)(len >> (e - 1)) & 1 : 0;
        return kBuckets - 2 - 2 * e - half;             // the longest come first
    };
    // the x-th of the items, of every sequence's chunks or of one bucket's sequences; returns how many were met
    auto search = [&](bool chunks, int want) {
        int64_t before = 0;
        if (tid == 0) sh[0] = -1;
        for (int64_t i0 = 0; i0 < p.n_seq; i0 += nt) {
            const int64_t i = i0 + tid;
            int64_t n = 0;
            if (i < p.n_seq) {
                const TokenRange r = token_range(p.cu, i, p.total);
                const int64_t len = r.hi - r.lo;
                n = chunks ? (len > 0 ? (len + p.chunk - 1) / p.chunk : 1) : bucket(len) == want;
            }
            int64_t inc = n;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, inc, m);
                if (lane >= m) inc += v;
            }
            __syncthreads();
            if (lane == 31) sh[2 + warp] = inc;
            __syncthreads();
            int64_t base = before, all = before;
            for (int w = 0; w < nw; ++w) {
                if (w < warp) base += sh[2 + w];
                all += sh[2 + w];
            }
            if (n > 0 && x >= base + inc - n && x < base + inc) {
                sh[0] = i;
                sh[1] = x - (base + inc - n);
            }
            before = all;
            if (!chunks && x < all) break;
        }
        __syncthreads();
        return before;
    };
    if constexpr (CUT) {
        cut = search(true, 0) <= p.n_chunks;
        if (!cut) __syncthreads();
    }
    if (!cut) {
        int want = 0;
        for (int i = tid; i < kBuckets; i += nt) count[i] = 0u;
        __syncthreads();
        for (int64_t i = tid; i < p.n_seq; i += nt) {
            const TokenRange r = token_range(p.cu, i, p.total);
            atomicAdd(count + bucket(r.hi - r.lo), 1u);
        }
        __syncthreads();
        while (want < kBuckets - 1 && x >= (int64_t)count[want]) x -= count[want++];
        search(false, want);
    }
    seq = sh[0];
    k = sh[1];
    return seq >= 0;
}

// What this launch does with the x-th item: fills in the task's tokens, slot and chunk (its channels
// are set), or, for a bad slot, writes the outputs' NaN.  All threads of the CTA call it.
enum Run { kRunNone, kRunFull, kRunLocal };
template <typename T, bool CUT>
__device__ __forceinline__ Run find_run(const PackedParams& p, int64_t x, int64_t* sh, int nt, Task& tk) {
    int64_t seq, k;
    bool cut;
    tk.chunk_id = (int)x;
    if (!find_item<CUT>(p, x, sh, nt, seq, k, cut)) return kRunNone;
    const TokenRange r = token_range(p.cu, seq, p.total);
    const int64_t t0 = r.lo + k * p.chunk;
    tk.k = (int)k;
    tk.t0 = (int)t0;
    tk.t1 = (int)(cut && r.hi - t0 > p.chunk ? t0 + p.chunk : r.hi);
    tk.last = tk.t1 == r.hi;
    tk.slot = p.slots ? __ldg(p.slots + seq) : (int)seq;
    tk.has = p.has_state && __ldg(p.has_state + seq) != 0;
    const SlotKind kind = slot_kind(tk.slot, p.n_slots);
    if (kind == kSlotPad) return kRunNone;
    if (kind == kSlotBad) {
        if (p.phase == (tk.k > 0 ? 2 : 1)) {
            const int64_t n = tk.t1 - tk.t0;
            for (int64_t i = threadIdx.x; i < n * tk.nch; i += nt)
                static_cast<T*>(p.out)[(tk.d0 + i / n) * p.total + tk.t0 + i % n] = T(__int_as_float(0x7FC00000));
        }
        return kRunNone;
    }
    // launch 1: first chunks in full, middle ones for their end state; launch 2: the later ones in full
    if (p.phase == 1) return tk.k == 0 ? kRunFull : tk.last ? kRunNone : kRunLocal;
    return tk.k > 0 ? kRunFull : kRunNone;
}

// CUT: sequences may be cut into chunks.
template <typename T, int N, bool HEAD, bool ALIGNED, bool CUT>
__global__ void __launch_bounds__(PackedCfg<T, N, HEAD, ALIGNED, CUT>::NT, PackedCfg<T, N, HEAD, ALIGNED, CUT>::CTAS)
scan_packed_kernel(const PackedParams p) {
    using Cf = PackedCfg<T, N, HEAD, ALIGNED, CUT>;
    extern __shared__ __align__(16) unsigned char packed_smem[];
    unsigned char* smem = packed_smem;
    const unsigned tile = blockIdx.x % p.n_tiles;
    Task tk;
    tk.g = (int)(tile / p.tiles_per_group);
    tk.ci0 = (int)(tile % p.tiles_per_group) * Cf::CT;
    tk.d0 = tk.g * (int)p.group_dim + tk.ci0;
    tk.nch = (int)p.group_dim - tk.ci0 < Cf::CT ? (int)p.group_dim - tk.ci0 : Cf::CT;
    const Run run = find_run<T, CUT>(p, blockIdx.x / p.n_tiles, reinterpret_cast<int64_t*>(smem), Cf::NT, tk);
    if (run == kRunFull) run_chunk<T, N, HEAD, ALIGNED, false, CUT>(p, tk, smem);
    if constexpr (CUT)
        if (run == kRunLocal) run_chunk<T, N, HEAD, ALIGNED, true, true>(p, tk, smem);
}

template <typename T, int N, bool HEAD, bool ALIGNED, bool CUT>
int launch(PackedParams& p, cudaStream_t s) {
    using Cf = PackedCfg<T, N, HEAD, ALIGNED, CUT>;
    p.tiles_per_group = (unsigned)((p.group_dim + Cf::CT - 1) / Cf::CT);
    const int64_t tiles = p.ngroups * p.tiles_per_group;
    const int64_t ctas = tiles * (CUT ? p.n_chunks : p.n_seq);
    if (tiles > 0x7FFFFFFF || ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    p.n_tiles = (unsigned)tiles;
    auto* k = scan_packed_kernel<T, N, HEAD, ALIGNED, CUT>;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM) != cudaSuccess) return SSM_ERR_CUDA;
    for (p.phase = 1; p.phase <= (CUT ? 2 : 1); ++p.phase) {
        k<<<(unsigned)ctas, Cf::NT, Cf::SMEM, s>>>(p);
        if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
    }
    return SSM_OK;
}

template <typename T, int N, bool HEAD, bool ALIGNED>
int launch(PackedParams& p, cudaStream_t s) {
    return p.chunk > 0 ? launch<T, N, HEAD, ALIGNED, true>(p, s) : launch<T, N, HEAD, ALIGNED, false>(p, s);
}

// One (dtype, dstate), in a translation unit of its own.
template <typename T, int N>
int launch_n(PackedParams& p, bool aligned, cudaStream_t s) {
    const bool head = p.nheads != p.dim;
    if (head) return aligned ? launch<T, N, true, true>(p, s) : launch<T, N, true, false>(p, s);
    return aligned ? launch<T, N, false, true>(p, s) : launch<T, N, false, false>(p, s);
}

}  // namespace packed
}  // namespace ssm
