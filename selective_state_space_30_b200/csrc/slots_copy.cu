// Copies, moves and clears of state slots (declared in include/ssm_scan.h as
// ssm_state_slots_copy): forking a sequence copies its slot to others, compacting a pool moves
// slots to the free ones in front, freeing clears.  The constant-size state of the Mamba
// "architecture-details" page ("Memory Efficiency") makes each a copy of fixed size.
//
//   for every layer:  new[dst[i]] = src[i] >= 0 ? old[src[i]] : 0        for all i at once
//
// Every source is read before any destination is written, so swaps and chains need no order: a
// CTA takes the same slice of bytes of every pair, stages all of them in shared memory, and
// writes them after a barrier; no other CTA touches that slice.  HBM-bound: 64 moves and 32 clears of
// 24 KB slots in 48 layers 36.0 us (5.2 TB/s of the 189 MB they cannot do without), a fork of one 96 KB
// slot into 8 in 24 layers 6.4 us in a graph; 96 KB staged per CTA instead of 32 takes 55 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "scan_kernel.cuh"   // smem_u32
#include "slots.h"         // all_aligned
#include "ssm_scan.h"

namespace {

constexpr int kThreads = 256;
// Bytes a CTA stages at most where its pairs' 16-byte pieces fit in as many: with 32 KB seven CTAs
// fit an SM, whose reads and writes overlap
constexpr int kStage = 32 * 1024;
constexpr int kMaxPairs = 4096;
constexpr int kStageMost = 32 * kMaxPairs;   // the shortest slice, and 16 bytes more where it is off the grid
constexpr int kMaxSlice = 4096;

struct CopyParams {
    unsigned char* pool;
    const int *src, *dst;
    int64_t n_slots, slot_bytes, slot_stride, layer_stride;
    int64_t slices;          // per slot
    int n_pairs, slice;      // slice: bytes, a multiple of 16
};

// A pair's staged slice: its 16-byte pieces, one more where the source is off the 16-byte grid.
__host__ __device__ constexpr int pitch_of(int slice) { return slice + 16; }

// 16 | every address and size
__global__ void __launch_bounds__(kThreads) slots_copy_kernel(const CopyParams p) {
    extern __shared__ __align__(16) unsigned char stage[];
    const int64_t layer = blockIdx.x / p.slices, c0 = blockIdx.x % p.slices * p.slice;
    unsigned char* base = p.pool + layer * p.layer_stride + c0;
    const int bytes = (int)(p.slot_bytes - c0 < p.slice ? p.slot_bytes - c0 : p.slice);
    const int n = bytes / 16, pitch = p.slice;
    // lanes side by side along a slice (a power of two of them), pairs across
    const int lanes = p.slice / 16, q = threadIdx.x & (lanes - 1);
    const int first = q < n ? threadIdx.x / lanes : p.n_pairs, step = kThreads / lanes;
    base += q * 16;
    uint4* mine = reinterpret_cast<uint4*>(stage) + q;
    auto read = [&](int pr) {
        const int s = __ldg(p.src + pr);
        uint4* to = mine + pr * (pitch / 16);
        if (s >= 0 && s < p.n_slots)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ssm::smem_u32(to)), "l"(base + s * p.slot_stride)
                         : "memory");
        else
            *to = make_uint4(0u, 0u, 0u, 0u);
        return s < p.n_slots;
    };
    auto write = [&](int pr, int d) {
        if (d >= 0 && d < p.n_slots) *reinterpret_cast<uint4*>(base + d * p.slot_stride) = *(mine + pr * (pitch / 16));
    };
    // the first pairs' destinations are read beside their sources, not behind the barrier
    constexpr int kKept = 4;
    int to[kKept];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int pr = first + k * step;
        to[k] = -1;
        if (pr < p.n_pairs) {
            const int d = __ldg(p.dst + pr);
            if (read(pr)) to[k] = d;
        }
    }
    for (int pr = first + kKept * step; pr < p.n_pairs; pr += step) read(pr);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kKept; ++k) write(first + k * step, to[k]);
    for (int pr = first + kKept * step; pr < p.n_pairs; pr += step)
        write(pr, __ldg(p.src + pr) < p.n_slots ? __ldg(p.dst + pr) : -1);
}

// Any alignment.  The source's 16-byte pieces are staged as they lie; the destination's pieces
// are put together at their offset, and the pieces that a slice's ends cut are written by bytes.
__global__ void __launch_bounds__(kThreads) slots_copy_bytes_kernel(const CopyParams p, const unsigned char* lo,
                                                                    const unsigned char* hi) {
    extern __shared__ __align__(16) unsigned char stage[];
    const int64_t layer = blockIdx.x / p.slices, c0 = blockIdx.x % p.slices * p.slice;
    unsigned char* base = p.pool + layer * p.layer_stride + c0;
    const int bytes = (int)(p.slot_bytes - c0 < p.slice ? p.slot_bytes - c0 : p.slice);
    const int pitch = pitch_of(p.slice), pieces = p.slice / 16 + 1;
    for (int i = threadIdx.x; i < p.n_pairs * pieces; i += kThreads) {
        const int pr = i / pieces, q = i % pieces;
        const int s = __ldg(p.src + pr);
        unsigned char* to = stage + pr * pitch + q * 16;
        if (s < 0 || s >= p.n_slots) {
            *reinterpret_cast<uint4*>(to) = make_uint4(0u, 0u, 0u, 0u);
            continue;
        }
        const unsigned char* from = base + s * p.slot_stride;
        const unsigned char* a = from - (reinterpret_cast<uintptr_t>(from) & 15u) + q * 16;
        if (a >= from + bytes) continue;
        if (a >= lo && a + 16 <= hi) {
            *reinterpret_cast<uint4*>(to) = __ldcg(reinterpret_cast<const uint4*>(a));
        } else {
            for (int e = 0; e < 16; ++e)
                if (a + e >= from && a + e < from + bytes) to[e] = a[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.n_pairs * pieces; i += kThreads) {
        const int pr = i / pieces, q = i % pieces;
        const int s = __ldg(p.src + pr), d = __ldg(p.dst + pr);
        if (d < 0 || d >= p.n_slots || s >= p.n_slots) continue;
        unsigned char* to = base + d * p.slot_stride;
        const int md = (int)(reinterpret_cast<uintptr_t>(to) & 15u);
        const int ms = s < 0 ? 0 : (int)(reinterpret_cast<uintptr_t>(base + s * p.slot_stride) & 15u);
        const int b0 = q * 16 - md;                      // first byte of the piece within the slice
        const int off = s < 0 ? 0 : b0 + ms;             // where it was staged
        const unsigned char* from = stage + pr * pitch;
        if (b0 >= 0 && b0 + 16 <= bytes) {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            if (s >= 0) {
                const uint32_t* f = reinterpret_cast<const uint32_t*>(from + (off & ~3));
                const int sh = (off & 3) * 8;
                uint32_t x = f[0];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t y = sh || e < 3 ? f[e + 1] : 0u;
                    w[e] = __funnelshift_r(x, y, sh);
                    x = y;
                }
            }
            *reinterpret_cast<uint4*>(to + b0) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int e = 0; e < 16; ++e)
                if (b0 + e >= 0 && b0 + e < bytes) to[b0 + e] = s < 0 ? 0 : from[off + e];
        }
    }
}

}  // namespace

extern "C" int ssm_state_slots_copy(void* pool, int64_t n_layers, int64_t n_slots, int64_t slot_bytes,
                                    int64_t slot_stride, int64_t layer_stride, const int32_t* src, const int32_t* dst,
                                    int64_t n_pairs, ssm_stream_t stream) {
    if (n_layers < 0 || n_slots < 0 || slot_bytes < 0 || n_pairs < 0) return SSM_ERR_INVALID_ARG;
    if (n_slots > 0x7FFFFFFF || slot_bytes > ((int64_t)1 << 40) || n_layers > (1 << 20)) return SSM_ERR_INVALID_ARG;
    if (n_pairs > kMaxPairs) return SSM_ERR_UNSUPPORTED;
    if (n_pairs == 0 || n_layers == 0 || slot_bytes == 0 || n_slots == 0) return SSM_OK;
    if (!pool || !src || !dst || !ssm::all_aligned(4, {src, dst})) return SSM_ERR_INVALID_ARG;
    // sizes whose products stay far inside 64 bits
    if (slot_stride < slot_bytes || slot_stride > ((int64_t)1 << 46) / n_slots) return SSM_ERR_INVALID_ARG;
    if (n_layers > 1 && (layer_stride < 0 || layer_stride > ((int64_t)1 << 46) / n_layers)) return SSM_ERR_INVALID_ARG;
    // a layer's slots in one piece after another layer's, or the layers of a slot next to each other
    const bool outer = layer_stride >= (n_slots - 1) * slot_stride + slot_bytes;
    const bool inner = layer_stride >= slot_bytes && slot_stride >= (n_layers - 1) * layer_stride + slot_bytes;
    if (n_layers > 1 && !outer && !inner) return SSM_ERR_INVALID_ARG;
    if (n_layers == 1) layer_stride = 0;
    const bool vec = ((reinterpret_cast<uintptr_t>(pool) | (uintptr_t)slot_bytes | (uintptr_t)slot_stride |
                       (uintptr_t)layer_stride) & 15u) == 0;
    CopyParams p{};
    p.pool = static_cast<unsigned char*>(pool);
    p.src = src; p.dst = dst;
    p.n_slots = n_slots; p.slot_bytes = slot_bytes; p.slot_stride = slot_stride; p.layer_stride = layer_stride;
    p.n_pairs = (int)n_pairs;
    // slices as long as the staging holds for all pairs, shorter where that leaves SMs idle
    const int extra = vec ? 0 : 16;
    int slice = kMaxSlice;
    while (slice > 16 && (slice + extra) * n_pairs > kStage) slice /= 2;
    static_assert((16 + 16) * kMaxPairs <= kStageMost && kStageMost <= 227 * 1024, "the shortest slices fit");
    while (slice > 512 && n_layers * ((slot_bytes + slice - 1) / slice) < 148 * 4) slice /= 2;
    p.slice = slice;
    p.slices = (slot_bytes + slice - 1) / slice;
    const int64_t ctas = n_layers * p.slices;
    if (ctas > 0x7FFFFFFF) return SSM_ERR_UNSUPPORTED;
    const int smem = (int)((slice + extra) * n_pairs);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (vec) {
        if (cudaFuncSetAttribute(slots_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMost) != cudaSuccess)
            return SSM_ERR_CUDA;
        slots_copy_kernel<<<(unsigned)ctas, kThreads, smem, s>>>(p);
    } else {
        if (cudaFuncSetAttribute(slots_copy_bytes_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageMost) !=
            cudaSuccess)
            return SSM_ERR_CUDA;
        const unsigned char* lo = p.pool;
        const unsigned char* hi = lo + (n_layers - 1) * layer_stride + (n_slots - 1) * slot_stride + slot_bytes;
        slots_copy_bytes_kernel<<<(unsigned)ctas, kThreads, smem, s>>>(p, lo, hi);
    }
    return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}
