// The scan over packed prompts on the tensor cores, for the per-head layout with head dim 64,
// dstate 128 and bf16 I/O: the chunked form ("Agent 229: SSM optimization patterns" page, section 2
// "Mamba-2 SSD" and section 9 "Chunked Computation") over sequences that start and end anywhere.
//
// One CTA runs one head through its tokens, Q = 128 at a time (a block).  With a_t = dt_t A log2 e,
// X, B, C the block's u, B, C rows, H (N x P) the state at its start, and s(i, j) the sum of a over
// the steps after j up to i:
//
//   S  = B^T X',  X'_j = 2^s(end, j) dt_j x_j       (N x P)     H <- 2^s(end, start) H + S
//   G  = C B^T,   M = G o [2^s(i, j) dt_j]_{j <= i}   (Q x Q)
//   Y  = M X + diag(2^s(i, start)) (C H)             (Q x P)     out = (Y + D x) silu(z)
//
// Steps outside the sequence have dt = 0 and their rows of B, C and X are zeroed in shared memory,
// so that no value there, NaN included, reaches a product.  A NaN or an infinity of the sequence's own u
// would reach the outputs of earlier steps through M's zeros: where the state turns out not to be finite,
// X is cleared of them and Y made again (elsewhere that costs a sum of 16 values in four of the warps).
//
// Precision.  B, C and X are bf16 and enter exactly.  X' is split into three bf16 terms (24 bits); the
// tensor core cuts its running sum of them, by 2^-22 of the magnitudes a step at the most.  Measured
// against 64 bits after 400 and 1000 steps, the state is off by 1.5e-7 to 1.9e-7 of its size (rms), the
// recurrence's in fp32 by 1.8e-7.  M and H are split into two terms (16 bits, 2^-17 of each product),
// far inside the rounding of the bf16 outputs.  Sums of a that are subtracted from one another
// lose their small differences, so every s(i, j) is added up from terms of its own: over stretches of
// 32 steps and groups of four, what is left of j's, the whole ones between, and the steps of i's; a
// step's own weight is its dt.  (The factors of a weight may leave fp32's range where it does not: with
// steps of either sign, a growth past 2^127 within a block overflows whatever decayed before it.)
//
// Order of a block.  The products run under the threads' work: G, then S and C H while M is made from
// G in tensor memory (M is Y's left operand there), Y while the state takes S and X' of the next
// block is made.  Three barriers a block.
//
// Bound: the threads' phases, chains of few instructions over 16 warps, one CTA per SM: a block takes
// 4.1 us, off the 16-byte grid 10.  (When it took 4.8, about 0.4 went into waiting for G, 1.2 into M, 1.4
// into the state and X', 1.3 into the outputs, half of that silu's two MUFU operations, and 0.3 into the
// copies' orders.)  Measured on one B200: 6 ragged prompts of 4096 tokens, 32 heads 62 us in the mean of
// three draws (the longest prompt 1468 to 1589 tokens; the scan kernel 340 to 380 for heads of 32 or of 128
// channels), one prompt of 8192 tokens, 16 heads 83 in chunks.  Steps, for other draws of the first of
// these: values in f32x2 pairs, log2 dt folded into the exponent and whole
// words of x, z and the outputs in the epilogue 120 us; M in tensor memory instead of shared memory, so
// that S need not have left its place, 104; the terms of X' and H side by side in one product each (a product
// of 64 columns takes as long to read its left operand as one of 192), the products asked for by a warp that
// M leaves idle and X' under Y 87; boxes of TMA instead of the threads' copies, and what seldom
// runs out of line 79; weights across stretches as products 78; the rule on cutting 74; epilogue rows in
// different banks, maps asked for early 73; weights across groups of four as products too, kernels of
// their own for cut and uncut calls 5 % less.
//
// Tiles arrive in the 128-byte swizzle that the tensor cores read, each as soon as its place is free: X a
// block ahead in a second buffer, B and C once G, S and C H are done, z once the outputs before it
// have left.  Rows off the 16-byte grid are shifted into place through registers.
//
// Every wait for the tensor cores or a copy is bounded; one that ran out ends the CTA's work with NaN in the
// rest of its outputs and is recorded in the device's status word.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "layout.h"            // encode_rows
#include "pair.cuh"
#include "scan_packed.cuh"
#include "ssd_packed.h"
#include "tcgen05_tmem.cuh"

namespace ssm {
namespace packed {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kQ = 128, kP = 64, kN = 128;
constexpr int kThreads = 512;
// warps with nothing of M to compute (steps 64 .. 95 and 96 .. 127 of rows 0 .. 31)
constexpr int kIssueWarp = 8, kCopyWarp = 9, kDecayWarp = 12;
constexpr uint32_t kTmemCols = 512;
// TMEM columns.  M's two terms lie where G was, 16 columns each for a stretch's 32 steps: each thread
// writes what it has read.  C H and S keep the products of H's and X' terms apart.
constexpr uint32_t kColG = 0, kColY = 128, kColCH = 192, kColS = 320;
constexpr int64_t kWaitUs = 500000;

// Kernel-side status of the device's calls since it was last read.
__device__ int g_status;
// Test hooks: the block, of even number, that waits for nothing instead of its products (-1: none), and the
// limit of a wait.
std::atomic<int> g_stall{-1};
std::atomic<int64_t> g_wait_us{kWaitUs};

// shared memory (bytes from a 1024-aligned base); a tile is two 64-step halves of rows of 128 bytes
constexpr int OFF_C = 0;                       // 128 states
constexpr int OFF_B = 32 * 1024;
constexpr int OFF_X = 64 * 1024;               // two buffers of 64 channels
constexpr int OFF_XW = 96 * 1024;              // X': [half][term]
constexpr int OFF_H = 144 * 1024;              // two terms of 128 x 64
constexpr int OFF_Z = 176 * 1024;              // z, then the outputs
constexpr int OFF_DEC = 192 * 1024;            // two blocks' Decay
constexpr int OFF_BAR = OFF_DEC + 2 * 4096;
constexpr int OFF_BAD = OFF_BAR + 256;         // what of X is not finite
constexpr int kSmem = OFF_BAD + 256 + 1024;   // and room to align the base

// A block's decay over its 128 steps, in stretches of 32 and groups of four: head, a, pre and the whole
// groups and stretches in log2 units, the others weights.
struct Decay {
    float head[kQ];       // from the stretch's start through the step
    float far[kQ];        // dt_j times the decay from behind j to the stretch's end: for later stretches
    float w[kQ];          // 2^s(end, j) dt_j
    float close[kQ];      // dt_j times the decay from behind j to its group's end: for later groups of the stretch
    float pre[kQ];        // from the group's start through the step
    float a[kQ], dt[kQ];  // the step's own
    float group[kQ / 4];  // whole groups
    float stretch[4];     // whole stretches
};
static_assert(sizeof(Decay) <= 4096, "fits its place");

// Four pairs of values as sums of K bf16 terms: `put(k, words)` takes term k's.
template <int K, class Put>
__device__ __forceinline__ void split8(pair_t (&v)[4], const Put& put) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 f = halves(v[q]);
            const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
            w[q] = *reinterpret_cast<const uint32_t*>(&t);
            if (k + 1 < K) v[q] = pfma(pk(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xFFFF0000u)), pk(-1.f), v[q]);
        }
        put(k, w);
    }
}
// Into K tiles `step` bytes apart, columns c0 .. c0 + 7 of row r.
template <int K>
__device__ __forceinline__ void store_split8(unsigned char* tile, int step, uint32_t r, uint32_t c0, pair_t (&v)[4]) {
    unsigned char* to = tile + tc::sw128_off(r, c0);
    split8<K>(v, [&](int k, const uint32_t (&w)[4]) {
        *reinterpret_cast<uint4*>(to + k * step) = make_uint4(w[0], w[1], w[2], w[3]);
    });
}

// The first step of a block whose u is not finite, per channel (kQ: none).
struct Bad {
    int first[kP];
};
static_assert(sizeof(Bad) <= 256, "fits its place");

// Notes what of a block's X is not finite and clears it; returns whether this thread met any.
__device__ __noinline__ bool clear_bad(Bad& bad, unsigned char* tile) {
    bool met = false;
    for (uint32_t i = threadIdx.x; i < kP * 16; i += kThreads) {
        const uint32_t p = i >> 4, s = (i & 15u) * 8u;
        unsigned short* v = reinterpret_cast<unsigned short*>(tile + (s >> 6) * 8192 + tc::sw128_off(p, s & 63u));
        for (uint32_t e = 0; e < 8; ++e)
            if ((v[e] & 0x7F80u) == 0x7F80u) {
                v[e] = 0;
                atomicMin(&bad.first[p], (int)(s + e));
                met = true;
            }
    }
    return met;
}

struct Block {
    int64_t tb;             // token of step 0
    int64_t t0, t1;         // the task's tokens
};

// The tensors as boxes of 64 steps, where their rows lie on the 16-byte grid.
struct SsdMaps {
    CUtensorMap u, z, B, C, out;
};

__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(tc::smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Stages ROWS rows (the first at `base`) of a block into a tile, from rows off the 16-byte grid; steps
// outside the task are zero.  [lo, hi): the tensor.  (Out of line, as is store_out: the block's loop is
// long, and what seldom runs in it costs instruction fetches: 5.40 -> 4.84 us a block.)
template <int ROWS>
__device__ __noinline__ void stage_tile(unsigned char* tile, const unsigned short* base, int64_t L, const Block& k,
                                        const unsigned short* lo, const unsigned short* hi) {
    // a thread's pieces: the same eight steps of every 32nd row, which the swizzle treats alike
    const int r0 = threadIdx.x >> 4, q = threadIdx.x & 15;
    unsigned char* dst = tile + (q >> 3) * (ROWS * 128) + tc::sw128_off(r0, (q & 7) * 8);
    const int64_t t = k.tb + 8 * q, step = 32 * L;
    const unsigned short* src = base + (int64_t)r0 * L + t;
    if (t >= k.t1 || t + 8 <= k.t0) {
#pragma unroll
        for (int i = 0; i < ROWS / 32; ++i) *reinterpret_cast<uint4*>(dst + i * 4096) = make_uint4(0u, 0u, 0u, 0u);
        return;
    }
    const bool whole = t >= k.t0 && t + 8 <= k.t1;
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i, src += step) {
        const uintptr_t m = reinterpret_cast<uintptr_t>(src) & 15u;
        const unsigned short* a = src - m / 2;
        uint32_t o[4] = {0u, 0u, 0u, 0u};
        if (whole && a >= lo && a + 16 <= hi) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(a)), y = __ldg(reinterpret_cast<const uint4*>(a) + 1);
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            // by whole words, then by half of one
            uint32_t s[6];
#pragma unroll
            for (int e = 0; e < 6; ++e) s[e] = (m & 8) ? w[e + 2] : w[e];
#pragma unroll
            for (int e = 0; e < 5; ++e) s[e] = (m & 4) ? s[e + 1] : s[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = __funnelshift_r(s[e], s[e + 1], (unsigned)(m & 2) * 8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (t + e >= k.t0 && t + e < k.t1) o[e / 2] |= (uint32_t)src[e] << (16 * (e & 1));
        }
        *reinterpret_cast<uint4*>(dst + i * 4096) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Zeroes the steps of a staged tile that lie outside the task.
template <int ROWS>
__device__ __forceinline__ void clear_outside(unsigned char* tile, const Block& k) {
    const int r0 = threadIdx.x >> 4, q = threadIdx.x & 15;
    const int64_t t = k.tb + 8 * q;
    if (t >= k.t0 && t + 8 <= k.t1) return;
    unsigned char* dst = tile + (q >> 3) * (ROWS * 128) + tc::sw128_off(r0, (q & 7) * 8);
    uint32_t keep[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        keep[e / 2] = (t + e >= k.t0 && t + e < k.t1 ? 0xFFFFu : 0u) | (t + e + 1 >= k.t0 && t + e + 1 < k.t1 ? 0xFFFF0000u : 0u);
#pragma unroll
    for (int i = 0; i < ROWS / 32; ++i) {
        uint4* w = reinterpret_cast<uint4*>(dst + i * 4096);
        const uint4 v = *w;
        *w = make_uint4(v.x & keep[0], v.y & keep[1], v.z & keep[2], v.w & keep[3]);
    }
}

// The outputs, staged in the z tile, to global memory: each thread the pieces that it staged.
__device__ __noinline__ void store_out(const unsigned char* tile, unsigned short* base, int64_t L, const Block& k, bool grid) {
    if (grid) {
#pragma unroll
        for (int i0 = 0; i0 < kP * 16; i0 += kThreads) {
            const int i = i0 + threadIdx.x, r = i >> 4, q = i & 15;
            const uint4 v = *reinterpret_cast<const uint4*>(tile + (q >> 3) * (kP * 128) + tc::sw128_off(r, (q & 7) * 8));
            const int64_t t = k.tb + 8 * q;
            unsigned short* dst = base + (int64_t)r * L + t;
            if (t >= k.t0 && t + 8 <= k.t1) {
                *reinterpret_cast<uint4*>(dst) = v;
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (t + e >= k.t0 && t + e < k.t1) dst[e] = (unsigned short)(w[e / 2] >> (16 * (e & 1)));
            }
        }
    } else {
        // off the grid: by elements, neighbouring steps on neighbouring lanes
        for (int i = threadIdx.x; i < kP * kQ; i += kThreads) {
            const int r = i >> 7, c = i & 127;
            const int64_t t = k.tb + c;
            if (t >= k.t0 && t < k.t1)
                base[(int64_t)r * L + t] =
                    *reinterpret_cast<const unsigned short*>(tile + (c >> 6) * (kP * 128) + tc::sw128_off(r, c & 63));
        }
    }
}

// A block's decay, by one warp: a group of four steps per lane, so eight lanes hold a stretch.
__device__ __forceinline__ void block_decay(const PackedParams& p, const unsigned short* delta, const Block& k, float Ah,
                                            float bias, int lane, Decay& o) {
    float dt[4], a[4], pre[4], run = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int64_t t = k.tb + 4 * lane + e;
        dt[e] = a[e] = 0.f;
        if (t >= k.t0 && t < k.t1) {
            const float x = __uint_as_float((uint32_t)__ldg(delta + t) << 16) + bias;
            dt[e] = p.softplus ? softplus1(x) : x;
            a[e] = dt[e] * Ah;
        }
        run += a[e];
        pre[e] = run;
    }
    // sums of the lanes before and behind within the stretch
    float before = run, behind = run;
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, before, s, 8), d = __shfl_down_sync(0xffffffffu, behind, s, 8);
        if ((lane & 7) >= s) before += u;
        if ((lane & 7) + s < 8) behind += d;
    }
    const float whole = __shfl_sync(0xffffffffu, before, 7, 8);
    float up = __shfl_up_sync(0xffffffffu, before, 1, 8), down = __shfl_down_sync(0xffffffffu, behind, 1, 8);
    if ((lane & 7) == 0) up = 0.f;
    if ((lane & 7) == 7) down = 0.f;
    float later = 0.f;                                   // the whole stretches behind this one
#pragma unroll
    for (int s = 3; s >= 1; --s) {
        const float v = __shfl_sync(0xffffffffu, whole, 8 * s);
        if (s > (lane >> 3)) later += v;
    }
    const float rest = ex2_approx(later);
    float suf = 0.f, head[4], far[4], w[4], close[4];
#pragma unroll
    for (int e = 3; e >= 0; --e) {
        head[e] = up + pre[e];
        far[e] = ex2_approx(suf + down) * dt[e];
        w[e] = far[e] * rest;
        close[e] = ex2_approx(suf) * dt[e];
        suf += a[e];
    }
    auto put = [&](float* to, const float (&v)[4]) {
        *reinterpret_cast<float4*>(to + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
    };
    put(o.head, head);
    put(o.far, far);
    put(o.w, w);
    put(o.close, close);
    put(o.pre, pre);
    put(o.a, a);
    put(o.dt, dt);
    o.group[lane] = run;
    if ((lane & 7) == 0) o.stretch[lane >> 3] = whole;
}

// Thread: TMEM lane and tile row `row`, and a quarter of that row's columns (32 of the 128 steps,
// 16 of the 64 channels).  LOCAL: only the end state from zero and the product of the decays.
template <bool LOCAL>
__device__ __forceinline__ void run_head(const PackedParams& p, const SsdMaps& maps, const Task& tk, unsigned char* smem) {
    uint64_t* mb_g = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t *mb_s = mb_g + 1, *mb_y = mb_g + 2, *mb_x = mb_g + 3, *mb_bc = mb_g + 4, *mb_z = mb_g + 5;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(mb_g + 6);
    int* status = reinterpret_cast<int*>(mb_g + 7);
    uint64_t* mb_fix = mb_g + 8;
    Decay* dec = reinterpret_cast<Decay*>(smem + OFF_DEC);
    Bad& bad = *reinterpret_cast<Bad*>(smem + OFF_BAD);
    static_assert(OFF_DEC % 16 == 0, "vector reads of the decay");
    unsigned char *sC = smem + OFF_C, *sB = smem + OFF_B, *sXw = smem + OFF_XW, *sH = smem + OFF_H, *sZ = smem + OFF_Z;

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int quarter = warp & 3, part = warp >> 2;
    const uint32_t row = (uint32_t)(32 * quarter + lane), j0 = (uint32_t)(32 * part), p0 = (uint32_t)(16 * part);
    const int64_t L = p.total, h = tk.d0 / kP, d_first = tk.d0, g_first = tk.g;
    const float Ah = __ldg(p.A + h) * kLog2e, bias = p.bias ? __ldg(p.bias + h) : 0.f;
    const unsigned short *u = static_cast<const unsigned short*>(p.u), *z = static_cast<const unsigned short*>(p.z),
                         *Bt = static_cast<const unsigned short*>(p.B), *Ct = static_cast<const unsigned short*>(p.C);
    unsigned short* out = static_cast<unsigned short*>(p.out) + (int64_t)tk.d0 * L;
    const unsigned short* delta = static_cast<const unsigned short*>(p.delta) + h * L;
    const bool gate = !LOCAL && z != nullptr, grid = p.grid16 != 0;
    const int64_t tb0 = grid ? tk.t0 & ~7 : tk.t0;
    const int nblk = (int)((tk.t1 - tb0 + kQ - 1) / kQ);
    auto block = [&](int c) { return Block{tb0 + (int64_t)c * kQ, tk.t0, tk.t1}; };
    // Copies of a block's tiles: boxes that one thread asks for on the 16-byte grid, else by all threads.
    auto inside = [&](int c) { return block(c).tb >= tk.t0 && block(c).tb + kQ <= tk.t1; };
    auto boxes = [&](unsigned char* tile, int half, const CUtensorMap* map, int c, int64_t row0, uint64_t* bar) {
        const int t = (int)block(c).tb;
        tma_2d(tile, map, t, (int)row0, bar);
        tma_2d(tile + half, map, t + 64, (int)row0, bar);
    };
    unsigned ph_x = 0u, ph_bc = 0u, ph_z = 0u;
    bool due_x = false, due_bc = false, due_z = false;   // boxes are on their way
    auto wait_box = [&](bool& due, uint64_t* bar, unsigned& phase) {
        if (!due) return true;
        if (!mbar_wait(bar, phase, p.wait_ns, status)) return false;
        phase ^= 1u;
        due = false;
        return true;
    };
    auto stage_x = [&](int c) {
        if (c >= nblk) return;
        unsigned char* tile = smem + OFF_X + (c & 1) * 16384;
        due_x = grid;
        if (!grid) {
            stage_tile<kP>(tile, u + d_first * L, L, block(c), u, u + p.dim * L);
        } else if (warp == kCopyWarp && tc::elect_one()) {
            mbar_arrive_tx(mb_x, 16384);
            boxes(tile, 8192, &maps.u, c, d_first, mb_x);
        }
    };
    auto stage_bc = [&](int c) {
        if (c >= nblk) return;
        due_bc = grid;
        if (!grid) {
            stage_tile<kN>(sB, Bt + g_first * kN * L, L, block(c), Bt, Bt + p.ngroups * kN * L);
            if (!LOCAL) stage_tile<kN>(sC, Ct + g_first * kN * L, L, block(c), Ct, Ct + p.ngroups * kN * L);
        } else if (warp == kCopyWarp && tc::elect_one()) {
            mbar_arrive_tx(mb_bc, LOCAL ? 32768u : 65536u);
            boxes(sB, 16384, &maps.B, c, g_first * kN, mb_bc);
            if (!LOCAL) boxes(sC, 16384, &maps.C, c, g_first * kN, mb_bc);
        }
    };
    auto stage_z = [&](int c) {
        // the outputs before are out of the tile
        if (grid && warp == kCopyWarp && tc::elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (!gate) return;
        due_z = grid;
        if (!grid) {
            stage_tile<kP>(sZ, z + d_first * L, L, block(c), z, z + p.dim * L);
        } else if (warp == kCopyWarp && tc::elect_one()) {
            mbar_arrive_tx(mb_z, 16384);
            boxes(sZ, 8192, &maps.z, c, d_first, mb_z);
        }
    };
    // Where boxes brought tokens of others: of X and B those have to be zero; of C and z they reach
    // outputs alone that are not written.
    auto wait_x = [&](int c) {
        const bool was = due_x, ok = wait_box(due_x, mb_x, ph_x);
        if (was && !inside(c)) clear_outside<kP>(smem + OFF_X + (c & 1) * 16384, block(c));
        return ok;
    };
    auto wait_bc = [&](int c) {
        const bool was = due_bc, ok = wait_box(due_bc, mb_bc, ph_bc);
        if (was && !inside(c)) clear_outside<kN>(sB, block(c));
        return ok;
    };

    tc::fence_async_smem();                             // (the item search wrote where boxes will)
    __syncthreads();
    if (!LOCAL && tid < kP) bad.first[tid] = kQ;
    if (tid == 0) {
        for (uint64_t* b = mb_g; b <= mb_z; ++b) mbar_init(b, 1);
        mbar_init(mb_fix, 1);
        *status = SSM_OK;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tc::alloc(tslot, kTmemCols);
    __syncthreads();
    stage_x(0);
    stage_bc(0);
    if (warp == kDecayWarp && nblk > 0) block_decay(p, delta, block(0), Ah, bias, lane, dec[0]);

    // the state: n = row, channels p0 .. p0 + 15
    float H[16], Dv[LOCAL ? 1 : 8];                     // the skip weights of the channels it writes
    const bool from_before = !LOCAL && tk.k > 0, from_slot = !LOCAL && tk.k == 0 && tk.has;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t d = d_first + p0 + k;
        H[k] = 0.f;
        if (from_slot) H[k] = p.states[(int64_t)tk.slot * p.slot_stride + d * kN + row];
        if (from_before) H[k] = __ldcg(p.ws_h + ((int64_t)(tk.chunk_id - tk.k) * p.dim + d) * kN + row);
        if constexpr (!LOCAL)
            if ((k & 4) == 0) Dv[k / 8 * 4 + (k & 3)] = p.D ? __ldg(p.D + d + 4 * (lane & 1)) : 0.f;
    }
    if (from_before) {
        // join the chunks before: the first holds a state, the later ones (decay, state from zero)
        for (int i = 1; i < tk.k; ++i) {
            const int64_t c = tk.chunk_id - tk.k + i;
            const float pr = __ldcg(p.ws_p + c * p.dim + d_first);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                H[k] = fmaf(pr, H[k], __ldcg(p.ws_h + (c * p.dim + d_first + p0 + k) * kN + row));
        }
    }
    const bool start_state = from_slot || from_before;
    auto store_state = [&]() {
#pragma unroll
        for (int k = 0; k < 16; k += 8) {
            pair_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = pk(H[k + 2 * e], H[k + 2 * e + 1]);
            store_split8<2>(sH, 16384, row, p0 + k, v);
        }
    };
    if (start_state) store_state();
    bool ok = wait_x(0);
    ok = wait_bc(0) && ok;
    tc::fence_async_smem();
    tc::fence_before();
    const bool staged = !__syncthreads_or(!ok);         // X, B, C, the decay and the state
    tc::fence_after();
    const uint32_t tbase = *tslot, trow = tbase + ((uint32_t)(32 * quarter) << 16);

    uint64_t* last_bar = nullptr;                       // the issuing thread's: its latest commit
    unsigned last_ph = 0;
    auto commit = [&](uint64_t* bar, unsigned ph) {
        tc::commit(bar);
        last_bar = bar;
        last_ph = ph;
    };
    // X' of a block, in three terms: two 8-step pieces of a channel per thread.
    auto make_xw = [&](int c) {
        const Decay& dc = dec[c & 1];
        const unsigned char* sX = smem + OFF_X + (c & 1) * 16384;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t e = (uint32_t)tid + (uint32_t)r * kThreads, pp = e >> 4, s8 = (e & 15u) * 8u;
            const uint4 raw = *reinterpret_cast<const uint4*>(sX + (s8 >> 6) * 8192 + tc::sw128_off(pp, s8 & 63u));
            const uint32_t w4[4] = {raw.x, raw.y, raw.z, raw.w};
            const ulonglong2* wj = reinterpret_cast<const ulonglong2*>(dc.w + s8);
            const ulonglong2 wa = wj[0], wb = wj[1];
            const pair_t w2[4] = {wa.x, wa.y, wb.x, wb.y};
            pair_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[k] = pmul(pk(__uint_as_float(w4[k] << 16), __uint_as_float(w4[k] & 0xFFFF0000u)), w2[k]);
            store_split8<3>(sXw + (s8 >> 6) * 24576, 8192, pp, s8 & 63u, v);
        }
    };
    // G, S and C H of a block, by one thread
    auto issue_products = [&](unsigned ph, bool with_state) {
        tc::fence_after();
        if constexpr (!LOCAL) {
            constexpr uint32_t id = tc::idesc_bf16(128, 128, true, true);
            const uint64_t a = tc::desc(sC, 16384, 1024, tc::kSwizzle128), b = tc::desc(sB, 16384, 1024, tc::kSwizzle128);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
                tc::mma_bf16(tbase + kColG, a + kk * (2048 >> 4), b + kk * (2048 >> 4), id, kk > 0 ? 1u : 0u);
            commit(mb_g, ph);
        }
        {
            constexpr uint32_t id = tc::idesc_bf16(128, 3 * kP, false, false);
            const uint64_t a = tc::desc(sB, 16, 1024, tc::kSwizzle128), b = tc::desc(sXw, 16, 1024, tc::kSwizzle128);
#pragma unroll
            for (int kk = 0; kk < kQ / 16; ++kk)
                tc::mma_bf16(tbase + kColS, a + (kk >> 2) * (16384 >> 4) + (kk & 3) * 2, b + (kk >> 2) * (24576 >> 4) + (kk & 3) * 2,
                             id, kk > 0 ? 1u : 0u);
        }
        if (!LOCAL && with_state) {
            constexpr uint32_t id = tc::idesc_bf16(128, 2 * kP, true, true);
            const uint64_t a = tc::desc(sC, 16384, 1024, tc::kSwizzle128), b = tc::desc(sH, 16384, 1024, tc::kSwizzle128);
#pragma unroll
            for (int kk = 0; kk < kN / 16; ++kk)
                tc::mma_bf16(tbase + kColCH, a + kk * (2048 >> 4), b + kk * (2048 >> 4), id, kk > 0 ? 1u : 0u);
        }
        commit(mb_s, ph);
    };
    // Y of a block, by one thread
    auto issue_y = [&](int c, uint64_t* bar, unsigned ph) {
        tc::fence_after();
        constexpr uint32_t id = tc::idesc_bf16(128, kP, false, false);
        const uint64_t b = tc::desc(smem + OFF_X + (c & 1) * 16384, 16, 1024, tc::kSwizzle128);
#pragma unroll
        for (int kk = 0; kk < kQ / 16; ++kk)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                tc::mma_bf16_ta(tbase + kColY, tbase + kColG + (kk >> 1) * 32 + s * 16 + (kk & 1) * 8,
                                b + (kk >> 2) * (8192 >> 4) + (kk & 3) * 2, id, kk > 0 || s > 0 ? 1u : 0u);
        commit(bar, ph);
    };
    unsigned ph_fix = 0u;
    if (nblk > 0) make_xw(0);
    tc::fence_async_smem();
    __syncthreads();
    if (staged) {
        stage_x(1);
        if (warp == kIssueWarp && nblk > 0 && tc::elect_one()) issue_products(0u, start_state);
        __syncwarp();
    }

    float total = 0.f;                                  // LOCAL: the sum of a over the task
    int done = 0;                                       // blocks whose outputs are written
    for (int c = 0; staged && c < nblk; ++c) {
        const unsigned ph = (unsigned)c & 1u;
        const Decay& dc = dec[c & 1];
        const unsigned char* sX = smem + OFF_X + (c & 1) * 16384;
        const bool with_state = c > 0 || start_state;
        if (warp == kDecayWarp && c + 1 < nblk) block_decay(p, delta, block(c + 1), Ah, bias, lane, dec[(c + 1) & 1]);
        bool found = false, spoiled = false;            // the block's u may hold, holds what is not finite
        ok = true;
        if constexpr (!LOCAL) {
            // ---- M, in two terms over G: row i = row, steps j0 .. (S and C H run)
            ok = mbar_wait(mb_g, ph, p.wait_ns, status);
            __syncwarp();
            tc::fence_after();
            uint32_t m0[16], m1[16];
            if (part > quarter) {                       // all steps behind the warp's rows
#pragma unroll
                for (int k = 0; k < 16; ++k) m0[k] = m1[k] = 0u;
            } else {
                uint32_t gv[32];
                tc::ld32(trow + kColG + j0, gv);
                const bool same = part == quarter;
                auto put = [&](int k, pair_t (&v)[4]) {
                    split8<2>(v, [&](int t, const uint32_t (&w)[4]) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) (t ? m1 : m0)[k / 2 + q] = w[q];
                    });
                };
                if (same) {
                    // of the stretch's own steps those up to the row's: over whole groups of four the weight is
                    // a product of the row's and the step's, in the row's own group it is made step by step
                    const int e = lane & 3, gi = lane >> 2;
                    const float4 a4 = *reinterpret_cast<const float4*>(dc.a + (row & ~3u));
                    const float4 d4 = *reinterpret_cast<const float4*>(dc.dt + (row & ~3u));
                    float s = e >= 3 ? a4.w : 0.f;
                    const float o2 = d4.z * ex2_approx(s);
                    s = e >= 2 ? s + a4.z : 0.f;
                    const float o1 = d4.y * ex2_approx(s);
                    s = e >= 1 ? s + a4.y : 0.f;
                    const pair_t own[2] = {pk(d4.x * ex2_approx(s), o1), pk(o2, d4.w)};
                    float run = dc.pre[row];            // from behind a group through the row
                    tc::wait_ld();
                    tc::after_wait(gv);
#pragma unroll
                    for (int k = 24; k >= 0; k -= 8) {
                        pair_t v[4];
#pragma unroll
                        for (int g = 1; g >= 0; --g) {
                            const int at = k / 4 + g;
                            const pair_t to = pk(ex2_approx(run));
                            const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(dc.close + j0 + 4 * at);
                            const float whole = dc.group[j0 / 4 + at];
                            run = at < gi ? run + whole : run;
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const int j = 4 * at + 2 * q;
                                const pair_t w = at == gi ? own[q] : pmul(to, q ? c2.y : c2.x);
                                const float2 f = halves(pmul(pk(__uint_as_float(gv[j]), __uint_as_float(gv[j + 1])), w));
                                v[2 * g + q] = pk(j <= lane ? f.x : 0.f, j + 1 <= lane ? f.y : 0.f);
                            }
                        }
                        put(k, v);
                    }
                } else {
                    // over whole stretches it is a product too
                    float ci = dc.head[row];
                    for (int s = part + 1; s < quarter; ++s) ci += dc.stretch[s];
                    const pair_t ci2 = pk(ex2_approx(ci));
                    const float* cj = dc.far + j0;
                    tc::wait_ld();
                    tc::after_wait(gv);
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        const ulonglong2 ca = *reinterpret_cast<const ulonglong2*>(cj + k);
                        const ulonglong2 cb = *reinterpret_cast<const ulonglong2*>(cj + k + 4);
                        const pair_t c2[4] = {ca.x, ca.y, cb.x, cb.y};
                        pair_t v[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            v[q] = pmul(pk(__uint_as_float(gv[k + 2 * q]), __uint_as_float(gv[k + 2 * q + 1])), pmul(ci2, c2[q]));
                        put(k, v);
                    }
                }
            }
            tc::st16(trow + kColG + j0, m0);
            tc::st16(trow + kColG + j0 + 16, m1);
            tc::wait_st();
        }
        ok = mbar_wait(c == p.stall ? mb_fix : mb_s, ph, p.wait_ns, status) && ok;
        tc::fence_after();
        ok = wait_x(c + 1) && ok;
        tc::fence_before();
        // (a wait that ran out is voted on before anything overwrites what the products may still read)
        if (__syncthreads_or(!ok)) break;
        if constexpr (!LOCAL) {
            if (warp == kIssueWarp && tc::elect_one()) issue_y(c, mb_y, ph);
            __syncwarp();
        }
        if constexpr (!LOCAL) stage_z(c);
        stage_bc(c + 1);
        __syncwarp();                                   // (one lane asked for the boxes)
        // ---- the state (Y runs)
        uint32_t cv[LOCAL ? 8 : 16];                    // C H
        {
            uint32_t s0[16], s1[16], s2[16];
            tc::ld16(trow + kColS + p0, s0);
            tc::ld16(trow + kColS + kP + p0, s1);
            tc::ld16(trow + kColS + 2 * kP + p0, s2);
            const float a = (dc.stretch[0] + dc.stretch[1]) + (dc.stretch[2] + dc.stretch[3]);
            const float d = ex2_approx(a);
            total += a;
            tc::wait_ld();
            tc::after_wait(s0);
            tc::after_wait(s1);
            tc::after_wait(s2);
#pragma unroll
            for (int k = 0; k < 16; ++k)
                H[k] = fmaf(d, H[k], __uint_as_float(s0[k]) + (__uint_as_float(s1[k]) + __uint_as_float(s2[k])));
            // what is not finite in X' is so in every row of the state then: one of them tells
            if (!LOCAL && quarter == 2) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < 16; ++k) sum += H[k];
                found = !(sum * 0.f == 0.f);
            }
            if constexpr (!LOCAL) {
                store_state();
                if (with_state) {
                    uint32_t c1[16];
                    tc::ld16(trow + kColCH + p0, cv);
                    tc::ld16(trow + kColCH + kP + p0, c1);
                    tc::wait_ld();
                    tc::after_wait(cv);
                    tc::after_wait(c1);
#pragma unroll
                    for (int k = 0; k < 16; ++k) cv[k] = __float_as_uint(__uint_as_float(cv[k]) + __uint_as_float(c1[k]));
                }
            }
        }
        // ---- X' of the next block
        if (c + 1 < nblk) make_xw(c + 1);
        if constexpr (!LOCAL) {
            ok = mbar_wait(mb_y, ph, p.wait_ns, status);
            tc::fence_after();
            ok = wait_box(due_z, mb_z, ph_z) && ok;
            if (__syncthreads_or(!ok || found)) {
                if (__syncthreads_or(!ok)) break;
                // M's zeros do not keep an infinity or a NaN in X from the outputs of earlier steps (0 * NaN):
                // X is cleared of it, Y made again, and the outputs from its step on are NaN
                const bool met = clear_bad(bad, smem + OFF_X + (c & 1) * 16384);
                tc::fence_async_smem();
                spoiled = __syncthreads_or(met);
                if (spoiled) {
                    if (warp == kIssueWarp && tc::elect_one()) issue_y(c, mb_fix, ph_fix);
                    __syncwarp();
                    ok = mbar_wait(mb_fix, ph_fix, p.wait_ns, status);
                    ph_fix ^= 1u;
                    if (__syncthreads_or(!ok)) break;
                    tc::fence_after();
                }
            }
            // ---- outputs of step row, channels p0 ..
            uint32_t yv[16];
            tc::ld16(trow + kColY + p0, yv);
            float e = dc.head[row];
            for (int s = 0; s < quarter; ++s) e += dc.stretch[s];
            e = ex2_approx(e);
            tc::wait_ld();
            tc::after_wait(yv);
            const unsigned char* xt = sX + (row >> 6) * 8192;
            unsigned char* zt = sZ + (row >> 6) * 8192;
            // neighbouring lanes trade a channel, so that each has two steps of one: whole words of
            // x, z and the outputs (channels four apart, whose rows the swizzle puts into different banks)
            const bool odd = lane & 1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = i / 4 * 8 + i % 4;
                float v0 = __uint_as_float(yv[k]), v1 = __uint_as_float(yv[k + 4]);
                if (with_state) {
                    v0 = fmaf(e, __uint_as_float(cv[k]), v0);
                    v1 = fmaf(e, __uint_as_float(cv[k + 4]), v1);
                }
                const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
                const uint32_t at = tc::sw128_off(p0 + k + (odd ? 4u : 0u), row & 62u);
                const uint32_t xw = *reinterpret_cast<const uint32_t*>(xt + at);
                pair_t v = pfma(pk(Dv[i]), pk(__uint_as_float(xw << 16), __uint_as_float(xw & 0xFFFF0000u)),
                                odd ? pk(got, v1) : pk(v0, got));
                uint32_t* zo = reinterpret_cast<uint32_t*>(zt + at);
                if (gate) {
                    const uint32_t zw = *zo;
                    v = pmul(v, psilu(pk(__uint_as_float(zw << 16), __uint_as_float(zw & 0xFFFF0000u))));
                }
                const float2 f = halves(v);
                const __nv_bfloat162 t = __floats2bfloat162_rn(f.x, f.y);
                *zo = *reinterpret_cast<const uint32_t*>(&t);
            }
            if (spoiled) {
                // from a channel's first step that is not finite on
                for (int i = 0; i < 8; ++i) {
                    const uint32_t ch = p0 + i / 4 * 8 + i % 4 + (odd ? 4u : 0u);
                    uint32_t* zo = reinterpret_cast<uint32_t*>(zt + tc::sw128_off(ch, row & 62u));
                    const int from = bad.first[ch], step = (int)(row & 126u);
                    if (step >= from) *zo = 0x7FC07FC0u;
                    else if (step + 1 >= from) *zo = (*zo & 0xFFFFu) | 0x7FC00000u;
                }
            }
        }
        ok = wait_bc(c + 1);
        tc::fence_async_smem();
        tc::fence_before();
        if (__syncthreads_or(!ok)) break;
        if constexpr (!LOCAL) {
            if (spoiled && tid < kP) bad.first[tid] = kQ;
            if (!grid || !inside(c)) {
                store_out(sZ, out, L, block(c), grid);
            } else if (warp == kCopyWarp && tc::elect_one()) {
                const int t = (int)block(c).tb;
                tma_store(&maps.out, t, (int)d_first, sZ);
                tma_store(&maps.out, t + 64, (int)d_first, sZ + 8192);
            }
        }
        stage_x(c + 2);
        if (warp == kIssueWarp && c + 1 < nblk && tc::elect_one()) issue_products(ph ^ 1u, true);
        __syncwarp();
        done = c + 1;
    }
    if (warp == kCopyWarp && tc::elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
    // a wait ran out: the products may still be under way, so wait (bounded) for the last batch
    // before TMEM and shared memory go; the outputs that are missing become NaN
    if (done < nblk) {
        if (tid == 0) atomicCAS(&g_status, SSM_OK, SSM_ERR_TIMEOUT);
        if (last_bar) mbar_wait(last_bar, last_ph, p.wait_ns, status);
        wait_box(due_x, mb_x, ph_x);
        wait_box(due_bc, mb_bc, ph_bc);
        wait_box(due_z, mb_z, ph_z);
        if constexpr (!LOCAL) {
            const int64_t a = tb0 + (int64_t)done * kQ > tk.t0 ? tb0 + (int64_t)done * kQ : tk.t0, n = tk.t1 - a;
            for (int64_t i = tid; i < n * kP; i += kThreads) out[i / n * L + a + i % n] = 0x7FC0;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) H[k] = __int_as_float(0x7FC00000);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t d = d_first + p0 + k;
        if (!LOCAL && tk.last) p.states[(int64_t)tk.slot * p.slot_stride + d * kN + row] = H[k];
        else if (LOCAL || tk.k == 0) __stcg(p.ws_h + ((int64_t)tk.chunk_id * p.dim + d) * kN + row, H[k]);
    }
    if (LOCAL && tid < kP) __stcg(p.ws_p + (int64_t)tk.chunk_id * p.dim + d_first + tid, ex2_approx(total));
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == 0) tc::dealloc(tbase, kTmemCols);
}

// CUT: sequences may be cut into chunks.
template <bool CUT>
__global__ void __launch_bounds__(kThreads, 1) ssd_packed_kernel(const PackedParams p, const __grid_constant__ SsdMaps maps) {
    extern __shared__ __align__(1024) unsigned char ssd_smem[];
    unsigned char* smem = ssd_smem + ((1024u - (smem_u32(ssd_smem) & 1023u)) & 1023u);
    if (threadIdx.x == 0 && p.grid16) {
        // the maps on their way while the CTA finds its task
        const CUtensorMap* m[5] = {&maps.u, &maps.B, &maps.C, p.z ? &maps.z : &maps.u, &maps.out};
#pragma unroll
        for (int i = 0; i < 5; ++i)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m[i])) : "memory");
    }
    const unsigned h = blockIdx.x % p.n_tiles;
    Task tk;
    tk.d0 = (int)h * kP;
    tk.g = tk.d0 / (int)p.group_dim;
    tk.ci0 = tk.d0 - tk.g * (int)p.group_dim;
    tk.nch = kP;
    const Run run = find_run<bf16, CUT>(p, blockIdx.x / p.n_tiles, reinterpret_cast<int64_t*>(smem), kThreads, tk);
    if (run == kRunFull) run_head<false>(p, maps, tk, smem);
    if constexpr (CUT)
        if (run == kRunLocal) run_head<true>(p, maps, tk, smem);
}

}  // namespace

bool ssd_packed_covers(const ssm_dims_t& d) {
    return d.io_dtype == SSM_BF16 && d.nheads != d.dim && d.dim / d.nheads == kP && d.dstate == kN && d.nheads % d.ngroups == 0;
}

int ssd_packed_launch(PackedParams& p, cudaStream_t s) {
    const int64_t ctas = p.nheads * (p.chunk > 0 ? p.n_chunks : p.n_seq);
    if (ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    p.n_tiles = (unsigned)p.nheads;
    SsdMaps maps{};
    if (p.grid16) {
        auto rows = [&](CUtensorMap* m, const void* t, int64_t n, uint32_t box) {
            return encode_rows(m, t, 2, (uint64_t)p.total, (uint64_t)n, box, CU_TENSOR_MAP_SWIZZLE_128B, 64);
        };
        const int64_t bc = p.ngroups * kN;
        if (!rows(&maps.u, p.u, p.dim, kP) || !rows(&maps.B, p.B, bc, kN) || !rows(&maps.C, p.C, bc, kN) ||
            !rows(&maps.out, p.out, p.dim, kP) || (p.z && !rows(&maps.z, p.z, p.dim, kP)))
            return SSM_ERR_CUDA;
    }
    p.wait_ns = (uint64_t)g_wait_us.load() * 1000u;
    p.stall = g_stall.load();
    auto* kernel = p.chunk > 0 ? ssd_packed_kernel<true> : ssd_packed_kernel<false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
        return SSM_ERR_CUDA;
    for (p.phase = 1; p.phase <= (p.chunk > 0 ? 2 : 1); ++p.phase) {
        kernel<<<(unsigned)ctas, kThreads, kSmem, s>>>(p, maps);
        if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
    }
    return SSM_OK;
}

}  // namespace packed
}  // namespace ssm

extern "C" int ssm_selective_scan_packed_device_status(ssm_stream_t stream) {
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int status = SSM_OK;
    const int clear = SSM_OK;
    if (cudaMemcpyFromSymbolAsync(&status, ssm::packed::g_status, sizeof status, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return SSM_ERR_CUDA;
    if (status != SSM_OK &&
        (cudaMemcpyToSymbolAsync(ssm::packed::g_status, &clear, sizeof clear, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
         cudaStreamSynchronize(s) != cudaSuccess))
        return SSM_ERR_CUDA;
    return status;
}

extern "C" int ssm_selective_scan_packed_test_hooks(int stall, int64_t wait_budget_us) {
    if (wait_budget_us < 0 || wait_budget_us > 10000000) return SSM_ERR_INVALID_ARG;
    ssm::packed::g_stall.store(stall ? 2 : -1);
    ssm::packed::g_wait_us.store(wait_budget_us ? wait_budget_us : ssm::packed::kWaitUs);
    return SSM_OK;
}
