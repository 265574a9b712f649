// C ABI of the scan over packed prompts (ssm_selective_scan_packed_fwd, include/ssm_scan.h): the
// checks of its arguments, the cutting of sequences into chunks, and the choice of the kernel.
// The kernel and its mathematics are in scan_packed.cuh; packed_n*.cu instantiate it.
#include "scan_packed.cuh"
#include "ssd_packed.h"

namespace ssm {
namespace packed {
#define SSM_PACKED_EXTERN(N)                                                           \
    extern template int launch_n<__nv_bfloat16, N>(PackedParams&, bool, cudaStream_t); \
    extern template int launch_n<float, N>(PackedParams&, bool, cudaStream_t);
SSM_PACKED_EXTERN(8)
SSM_PACKED_EXTERN(16)
SSM_PACKED_EXTERN(32)
SSM_PACKED_EXTERN(64)
SSM_PACKED_EXTERN(128)
}  // namespace packed
}  // namespace ssm

namespace {

using ssm::aligned_to;
using ssm::all_aligned;
using ssm::packed::launch_n;
using ssm::packed::PackedCfg;
using ssm::packed::PackedParams;

constexpr int64_t kNoChunk = 0;

// Channels of a tile, whatever the I/O type and alignment.
int tile_channels(int64_t N) {
    switch (N) {
        case 8: return PackedCfg<float, 8, false, true>::CT;
        case 16: return PackedCfg<float, 16, false, true>::CT;
        case 32: return PackedCfg<float, 32, false, true>::CT;
        case 64: return PackedCfg<float, 64, false, true>::CT;
        default: return PackedCfg<float, 128, false, true>::CT;
    }
}

// The tensor-core form, where it covers the shape and the sequences are 32 tokens or more in the
// mean: its blocks are 128 tokens long whatever a sequence fills of them (32 heads: 60 prompts of
// 10 tokens 175 us against the scan's 159, of 20 tokens 175 against 174, 40 of 32 tokens 120 against
// 124, of 51 tokens 122 against 192; 20 of 100 tokens and 8 heads 17 against 35).
bool on_tensor_cores(const ssm_dims_t& d) { return ssm::packed::ssd_packed_covers(d) && d.seqlen >= 32 * d.batch; }

// The tokens of a chunk, or kNoChunk: a function of the shape and the hint alone, so the same call
// gives the same bits.  `share` is what each CTA slot of the machine gets of the (token, tile)
// products.  Sequences are cut, into chunks of one share, where the longest is over four shares
// and so would still run when everything else is done: one prompt of 8191 tokens x 1536 channels
// takes 203 us cut at 352 tokens, 231 at 448, 292 at 672; 24 ragged prompts (16384 tokens x 4096
// channels, the longest under two shares) took 492 us uncut and 666 with every prompt cut at 1184 (what
// cutting its longest prompts alone takes has not been tried).  On the tensor cores a middle chunk's first
// pass costs less than half of its second, so three shares do: 4 prompts of
// 4096 tokens in all, 32 heads, the longest of 3000 (3.3 shares), 116 us uncut and 91 cut at 896; 6,
// the longest of 2241 (2.5 shares), 91 and 100, of 1508 (1.7) 65 and 99.
int64_t choose_chunk(const ssm_dims_t& d, int64_t max_seqlen) {
    const bool ssd = on_tensor_cores(d);
    const int64_t ct = tile_channels(d.dstate), gd = d.dim / d.ngroups;
    const int64_t tiles = ssd ? d.nheads : d.ngroups * ((gd + ct - 1) / ct);
    // without a hint the longest is taken for four times the mean
    const int64_t mean = d.batch > 0 ? (d.seqlen + d.batch - 1) / d.batch : 0;
    int64_t longest = max_seqlen > 0 ? max_seqlen : 4 * mean;
    if (longest > d.seqlen) longest = d.seqlen;
    const int64_t slots = 148 * (ssd ? 1 : d.dstate <= 32 ? 4 : 2);
    int64_t q = (d.seqlen * tiles + slots - 1) / slots;
    const int64_t least = d.seqlen / 64 > 128 ? d.seqlen / 64 : 128;
    if (q < least) q = least;
    const int64_t step = ssd ? 128 : 32;
    q = (q + step - 1) / step * step;
    return longest > (ssd ? 3 : 4) * q ? q : kNoChunk;
}

template <typename T>
int launch_t(PackedParams& p, int64_t N, bool aligned, cudaStream_t s) {
    switch (N) {
        case 8: return launch_n<T, 8>(p, aligned, s);
        case 16: return launch_n<T, 16>(p, aligned, s);
        case 32: return launch_n<T, 32>(p, aligned, s);
        case 64: return launch_n<T, 64>(p, aligned, s);
        case 128: return launch_n<T, 128>(p, aligned, s);
        default: return SSM_ERR_UNSUPPORTED;
    }
}

int check_dims(const ssm_dims_t* dims) {
    if (!dims) return SSM_ERR_INVALID_ARG;
    const ssm_dims_t& d = *dims;
    if (d.batch < 0 || d.dim <= 0 || d.seqlen < 0 || d.dstate <= 0 || d.nheads <= 0 || d.ngroups <= 0 || d.reserved != 0)
        return SSM_ERR_INVALID_ARG;
    if (d.dim % d.nheads || d.dim % d.ngroups) return SSM_ERR_INVALID_ARG;
    if (d.io_dtype != SSM_F32 && d.io_dtype != SSM_BF16) return SSM_ERR_INVALID_ARG;
    // cu_seqlens is 32-bit, and a block may reach past the last token; sizes whose products stay
    // far inside 64 bits
    if (d.seqlen > 0x7FFFFFFF - 1024 || d.batch > 0x7FFFFFFF || d.dim > (1 << 24)) return SSM_ERR_INVALID_ARG;
    const int64_t N = d.dstate;
    if (N != 8 && N != 16 && N != 32 && N != 64 && N != 128) return SSM_ERR_UNSUPPORTED;
    return SSM_OK;
}

struct Work {
    int64_t chunk, n_chunks;
    size_t h_bytes, bytes;
};

Work work_of(const ssm_dims_t& d, int64_t max_seqlen) {
    Work w{choose_chunk(d, max_seqlen), 0, 0, 0};
    if (w.chunk > 0) {
        w.n_chunks = d.batch + d.seqlen / w.chunk;
        w.h_bytes = ((size_t)w.n_chunks * d.dim * d.dstate * 4 + 255) / 256 * 256;
        w.bytes = w.h_bytes + (size_t)w.n_chunks * d.dim * 4;
    }
    return w;
}

}  // namespace

extern "C" int ssm_selective_scan_packed_workspace_size(const ssm_dims_t* dims, int64_t max_seqlen, size_t* bytes) {
    if (!bytes) return SSM_ERR_INVALID_ARG;
    const int rc = check_dims(dims);
    if (rc != SSM_OK) return rc;
    *bytes = work_of(*dims, max_seqlen).bytes;
    return SSM_OK;
}

extern "C" int ssm_selective_scan_packed_fwd(const ssm_dims_t* dims, const void* u, const void* delta, const float* A,
                                             const void* B, const void* C, const float* D, const void* z,
                                             const float* delta_bias, int softplus, const int32_t* cu_seqlens,
                                             const int32_t* slots, const uint8_t* has_state, float* states,
                                             int64_t n_slots, int64_t slot_stride, int64_t max_seqlen, void* out,
                                             void* workspace, size_t workspace_bytes, ssm_stream_t stream) {
    const int rc = check_dims(dims);
    if (rc != SSM_OK) return rc;
    const ssm_dims_t& d = *dims;
    if (n_slots < 0 || n_slots > 0x7FFFFFFF) return SSM_ERR_INVALID_ARG;
    if (d.batch == 0) return SSM_OK;
    if (!A || !cu_seqlens || !states) return SSM_ERR_INVALID_ARG;
    if (d.seqlen > 0 && (!u || !delta || !B || !C || !out)) return SSM_ERR_INVALID_ARG;
    if (slot_stride < d.dim * d.dstate) return SSM_ERR_INVALID_ARG;
    const size_t esz = d.io_dtype == SSM_BF16 ? 2 : 4;
    if (!all_aligned(esz, {u, delta, B, C, z, out}) || !all_aligned(4, {A, D, delta_bias, cu_seqlens, slots, states}))
        return SSM_ERR_INVALID_ARG;
    const Work w = work_of(d, max_seqlen);
    if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes || !aligned_to(workspace, 16))) return SSM_ERR_INVALID_ARG;
    PackedParams p{};
    p.u = u; p.delta = delta; p.B = B; p.C = C; p.z = z;
    p.A = A; p.D = D; p.bias = delta_bias; p.out = out; p.states = states;
    p.cu = cu_seqlens; p.slots = slots; p.has_state = has_state;
    p.ws_h = static_cast<float*>(workspace);
    p.ws_p = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + w.h_bytes);
    p.n_seq = d.batch; p.total = d.seqlen; p.n_slots = n_slots; p.slot_stride = slot_stride;
    p.dim = d.dim; p.nheads = d.nheads; p.ngroups = d.ngroups;
    p.group_dim = d.dim / d.ngroups; p.head_dim = d.dim / d.nheads;
    p.chunk = w.chunk; p.n_chunks = w.n_chunks;
    p.softplus = softplus ? 1 : 0;
    p.state_vec = aligned_to(states, 16) && slot_stride % 4 == 0;
    const bool aligned = d.seqlen * (int64_t)esz % 16 == 0 && all_aligned(16, {u, delta, B, C, z, out});
    p.grid16 = aligned;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (on_tensor_cores(d)) return ssm::packed::ssd_packed_launch(p, s);
    return d.io_dtype == SSM_BF16 ? launch_t<__nv_bfloat16>(p, d.dstate, aligned, s)
                                  : launch_t<float>(p, d.dstate, aligned, s);
}
