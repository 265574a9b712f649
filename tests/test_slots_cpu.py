"""Refusals of the slot and convolution-gradient operators, on the host before anything is launched, and the
fp64 forms that the GPU tests compare with."""
import ctypes

import numpy as np
import pytest

import oracle
import slots_plain as sp

A16 = 0x10000          # stand-in device addresses: 16-byte aligned,
OFF1 = 0x10001         # and off every element's alignment


@pytest.fixture(scope="module")
def ssm():
    import selective_state_space_30_b200 as m
    from selective_state_space_30_b200 import build
    build.build()
    m.load_library()
    return m


def _raises(ssm, status, fn, *args):
    assert fn(*args, check=False) == status, args


def test_conv_packed_refusals(ssm):
    ok = dict(dim=8, total=20, n_seq=2, width=4, io=ssm.SSM_BF16, x=A16, w=A16, bias=None, silu=True, cu=A16, slots=None,
              has=None, states=A16, n_slots=3, stride=24, out=2 * A16)

    def rc(**kw):
        a = dict(ok, **kw)
        return ssm.ssm_causal_conv1d_packed_fwd(*a.values(), check=False)

    inv, uns = ssm.SSM_ERR_INVALID_ARG, ssm.SSM_ERR_UNSUPPORTED
    for bad in (dict(dim=0), dict(total=-1), dict(n_seq=-1), dict(io=7), dict(x=None), dict(w=None), dict(cu=None),
                dict(states=None), dict(out=None), dict(out=A16), dict(n_slots=-1), dict(stride=23), dict(x=OFF1), dict(out=OFF1),
                dict(states=OFF1), dict(total=2 ** 31), dict(n_seq=2 ** 31), dict(n_slots=2 ** 31)):
        assert rc(**bad) == inv, bad
    assert rc(width=0) == uns and rc(width=5) == uns
    assert rc(n_seq=0, x=None, w=None, cu=None, states=None, out=None) == ssm.SSM_OK


def test_conv_update_refusals(ssm):
    ok = dict(batch=2, dim=8, width=4, io=ssm.SSM_F32, x=A16, w=A16, bias=None, silu=True, slots=None, states=A16, n_slots=3,
              stride=24, out=A16)

    def rc(**kw):
        return ssm.ssm_causal_conv1d_update(*dict(ok, **kw).values(), check=False)

    for bad in (dict(batch=-1), dict(dim=0), dict(io=2), dict(x=None), dict(w=None), dict(out=None), dict(states=None),
                dict(n_slots=-1), dict(stride=0), dict(x=0x10002), dict(states=0x10002)):
        assert rc(**bad) == ssm.SSM_ERR_INVALID_ARG, bad
    assert rc(width=5) == ssm.SSM_ERR_UNSUPPORTED
    assert rc(batch=0, x=None) == ssm.SSM_OK


def test_scan_packed_refusals(ssm):
    def dims(batch=2, dim=32, total=64, N=16, heads=0, groups=1, io=ssm.SSM_BF16):
        return ssm.make_dims(batch, dim, total, N, heads, groups, io)

    ok = dict(dims=dims(), u=A16, delta=A16, A=A16, B=A16, C=A16, D=None, z=None, bias=None, softplus=True, cu=A16, slots=None,
              has=None, states=A16, n_slots=4, stride=512, longest=0, out=A16, ws=None, nws=0)

    def rc(**kw):
        return ssm.ssm_selective_scan_packed_fwd(*dict(ok, **kw).values(), check=False)

    for bad in (dict(u=None), dict(delta=None), dict(A=None), dict(B=None), dict(C=None), dict(cu=None), dict(states=None),
                dict(out=None), dict(stride=511), dict(n_slots=-1), dict(u=OFF1), dict(z=OFF1), dict(out=OFF1),
                dict(dims=dims(heads=5)), dict(dims=dims(groups=3)), dict(dims=dims(batch=-1)), dict(dims=dims(io=4)),
                dict(dims=dims(total=2 ** 31))):
        assert rc(**bad) == ssm.SSM_ERR_INVALID_ARG, bad
    assert rc(dims=dims(N=24)) == ssm.SSM_ERR_UNSUPPORTED
    assert rc(dims=dims(batch=0), u=None, A=None, cu=None) == ssm.SSM_OK
    # a workspace where sequences are cut, and only there
    size = ssm.ssm_selective_scan_packed_workspace_size
    long = dims(batch=1, total=4096)
    need = size(long)
    assert need >= 4096 // 256 * 32 * 17 * 4
    assert size(long, 200) == 0 and size(dims()) == 0 and size(long, 4096) == need
    assert rc(dims=long) == ssm.SSM_ERR_INVALID_ARG
    assert rc(dims=long, ws=A16, nws=need - 1) == ssm.SSM_ERR_INVALID_ARG
    assert rc(dims=long, ws=A16 + 4, nws=need) == ssm.SSM_ERR_INVALID_ARG
    assert size(dims(N=24), check=False) == -ssm.SSM_ERR_UNSUPPORTED
    assert ssm.load_library().ssm_selective_scan_packed_workspace_size(ctypes.byref(long), 0, None) == ssm.SSM_ERR_INVALID_ARG


def test_state_update_slots_refusals(ssm):
    def dims(batch=2, dim=32, L=1, N=16, heads=0, groups=1, io=ssm.SSM_BF16):
        return ssm.make_dims(batch, dim, L, N, heads, groups, io)

    ok = dict(dims=dims(), states=A16, slots=None, n_slots=4, stride=512, u=A16, delta=A16, A=A16, B=A16, C=A16, D=None, z=None,
              bias=None, softplus=True, out=A16)

    def rc(**kw):
        return ssm.ssm_selective_state_update_slots(*dict(ok, **kw).values(), check=False)

    for bad in (dict(states=None), dict(u=None), dict(delta=None), dict(A=None), dict(B=None), dict(C=None), dict(out=None),
                dict(stride=508), dict(dims=dims(L=2)), dict(dims=dims(heads=5)), dict(n_slots=-1), dict(u=OFF1)):
        assert rc(**bad) == ssm.SSM_ERR_INVALID_ARG, bad
    for bad in (dict(dims=dims(N=24)), dict(states=A16 + 4), dict(stride=514), dict(B=A16 + 4), dict(C=A16 + 2),
                dict(A=A16 + 4)):
        assert rc(**bad) == ssm.SSM_ERR_UNSUPPORTED, bad
    assert rc(dims=dims(batch=0), u=None) == ssm.SSM_OK


def test_slots_copy_refusals(ssm):
    ok = dict(pool=A16, layers=2, n_slots=4, slot_bytes=64, slot_stride=64, layer_stride=256, src=A16, dst=A16, n=3)

    def rc(**kw):
        return ssm.ssm_state_slots_copy(*dict(ok, **kw).values(), check=False)

    for bad in (dict(pool=None), dict(src=None), dict(dst=None), dict(layers=-1), dict(n_slots=-1), dict(slot_bytes=-1),
                dict(n=-1), dict(slot_stride=63), dict(layer_stride=255), dict(layer_stride=-256),
                dict(layer_stride=64), dict(slot_stride=2 ** 45), dict(n_slots=2 ** 31)):
        assert rc(**bad) == ssm.SSM_ERR_INVALID_ARG, bad
    assert rc(n=4097) == ssm.SSM_ERR_UNSUPPORTED
    for empty in (dict(n=0), dict(layers=0), dict(slot_bytes=0), dict(n_slots=0)):
        assert rc(pool=None, **empty) == ssm.SSM_OK


def test_conv_bwd_refusals(ssm):
    size = ssm.ssm_causal_conv1d_bwd_workspace_size
    # a workspace where a channel's sums are split over CTAs: few channels and many rows
    need = size(40, 8, 30, 4, ssm.SSM_BF16)
    assert need >= 2 * 8 * 5 * 4 and size(40, 8, 0, 4, ssm.SSM_BF16) == 0 and size(8, 1536, 2048, 4, ssm.SSM_BF16) == 0
    ok = dict(batch=40, dim=8, L=30, width=4, io=ssm.SSM_BF16, x=A16, w=A16, bias=None, silu=True, dout=A16, dx=2 * A16, dw=A16,
              db=None, ws=A16, nws=need)

    def rc(**kw):
        return ssm.ssm_causal_conv1d_bwd(*dict(ok, **kw).values(), check=False)

    for bad in (dict(x=None), dict(w=None), dict(dout=None), dict(dx=None), dict(dx=A16), dict(x=2 * A16), dict(dw=None), dict(ws=None), dict(nws=need - 1),
                dict(batch=-1), dict(dim=0), dict(L=-1), dict(io=3), dict(x=OFF1), dict(dout=OFF1), dict(dx=OFF1)):
        assert rc(**bad) == ssm.SSM_ERR_INVALID_ARG, bad
    assert rc(width=5) == ssm.SSM_ERR_UNSUPPORTED and rc(width=0) == ssm.SSM_ERR_UNSUPPORTED
    lib = ssm.load_library()
    assert lib.ssm_causal_conv1d_bwd_workspace_size(1, 1, 1, 4, 0, None) == ssm.SSM_ERR_INVALID_ARG


def test_front_end_refusals(ssm):
    """What is no tensor, no CUDA tensor or of another rank is refused before the library is called."""
    import torch
    z, i32 = torch.zeros, torch.int32
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_packed(z(4, 8), z(4, 4), z(2, dtype=i32), z(1, 4, 3))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_update(z(2, 4), z(4, 4), z(2, 4, 3))
    with pytest.raises(ValueError, match="2 dimensions"):
        ssm.causal_conv1d_update(z(2, 4, 1), z(4, 4), z(2, 4, 3))
    with pytest.raises(TypeError, match="x must be a tensor"):
        ssm.causal_conv1d_update([1.0], z(4, 4), z(2, 4, 3))
    with pytest.raises(ValueError, match="x must be a tensor"):
        ssm.causal_conv1d_update(None, z(4, 4), z(2, 4, 3))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.selective_scan_packed(z(4, 8), z(4, 8), z(4, 16), z(1, 16, 8), z(1, 16, 8), z(2, dtype=i32), z(1, 4, 16))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.selective_state_update_slots(z(1, 4, 16), z(1, 4), z(1, 4), z(4, 16), z(1, 1, 16), z(1, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.state_slots_copy(z(2, 4), z(1, dtype=i32), z(1, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_bwd(z(1, 4, 8), z(4, 4), z(1, 4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_fn(z(1, 4, 8), z(4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_fwd(z(1, 4, 8), z(4, 4))


def test_front_ends_are_bound_to_the_loaded_library(ssm):
    """The compiled front ends take exactly the arguments that they document, and need the build."""
    from selective_state_space_30_b200 import _abi, _frontend
    front = _frontend.load()
    assert set(_frontend._ENTRIES) <= set(_abi.EXPORTS)
    with pytest.raises(TypeError, match="7 arguments wanted"):
        front.conv_update(1, 2)
    with pytest.raises(KeyError):
        front.bind({}, ssm.SsmError)


# ------------------------------------------------- the fp64 forms against the oracle

def test_plain_scan_is_the_oracles():
    """A packed scan is the batch oracle run per sequence, from the slot's state."""
    rng = np.random.default_rng(4)
    dim, N, G = 6, 8, 2
    lens = [5, 0, 9]
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    n = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    p = dict(u=n(dim, T), delta=n(dim, T), A=-np.abs(n(dim, N)), B=n(G, N, T), C=n(G, N, T), D=n(dim), z=n(dim, T),
             delta_bias=n(dim), softplus=True)
    pool = n(3, dim, N)
    slots, has = [2, 0, 1], [1, 1, 0]
    bounds = list(zip(cu[:-1].tolist(), cu[1:].tolist()))
    f = {k: v.astype(np.float64) if isinstance(v, np.ndarray) else v for k, v in p.items()}
    out, err, got_pool, _ = sp.scan_packed(f, bounds, slots, has, pool.astype(np.float64), np.zeros((dim, T)))
    import ssm_inputs as si
    for (lo, hi), s, h in zip(bounds, slots, has):
        if hi == lo:
            assert np.array_equal(got_pool[s], pool[s])
            continue
        d = si.Dims(1, dim, hi - lo, N, ngroups=G, dtype="f32")
        cut = {k: np.ascontiguousarray(p[k][..., lo:hi])[None] for k in ("u", "delta", "B", "C", "z")}
        o, last, _ = oracle.run_inputs(d, dict(p, **cut), h0=pool[s][None] if h else None)
        assert np.allclose(out[:, lo:hi], o[0], rtol=1e-12, atol=1e-13)
        assert np.allclose(got_pool[s], last[0], rtol=1e-12, atol=1e-13)
    assert np.all(err > 0) and err.max() < 1e-4


def test_plain_conv_is_the_oracles():
    rng = np.random.default_rng(5)
    x, w, b = rng.standard_normal((3, 20)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    x, w, b = (t.astype(np.float32) for t in (x, w, b))
    out, err, pool = sp.conv_packed(x.astype(np.float64), w.astype(np.float64), b.astype(np.float64), True, [(0, 20)], [0], [0],
                                    np.zeros((1, 3, 3)), np.zeros((3, 20)))
    assert np.allclose(out, oracle.causal_conv1d(x[None], w, b, silu=True)[0], rtol=1e-12, atol=1e-14)
    assert np.array_equal(pool[0], x[:, -3:])
    # two halves from the kept inputs
    o2, _, p2 = sp.conv_packed(x.astype(np.float64), w.astype(np.float64), b.astype(np.float64), True, [(0, 2)], [0], [0],
                               np.zeros((1, 3, 3)), np.zeros((3, 20)))
    o3, _, p3 = sp.conv_packed(x[:, 2:].astype(np.float64), w.astype(np.float64), b.astype(np.float64), True, [(0, 18)], [0], [1],
                               p2, np.zeros((3, 18)))
    assert np.allclose(np.concatenate([o2[:, :2], o3], 1), out, rtol=1e-13, atol=1e-15) and np.array_equal(p3, pool)


# ------------------------------------------------- index arithmetic of the kernels, compiled for the CPU

@pytest.fixture(scope="module")
def indexes(tmp_path_factory):
    """csrc/slots.h, whose functions read and compute indexes alone, as host code."""
    import os
    import subprocess
    from selective_state_space_30_b200 import build
    d = tmp_path_factory.mktemp("slots_h")
    src = d / "slots_h.cpp"
    src.write_text("""
#define __host__
#define __device__
#define __forceinline__ inline
template <typename T> T __ldg(const T* p) { return *p; }
#include "slots.h"
extern "C" long long tap_channel(long long d0, int row, int ty, long long dim) {
    return ssm::tap_channel(d0, row, ty, dim);
}
extern "C" void token_range(const int* cu, long long i, long long total, long long* out) {
    const ssm::TokenRange r = ssm::token_range(cu, i, total);
    out[0] = r.lo;
    out[1] = r.hi;
}
""")
    lib = d / "slots_h.so"
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-fPIC", "-shared", f"-I{build.CSRC}", str(src), "-o",
                    str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    so.tap_channel.restype = ctypes.c_longlong
    so.tap_channel.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_longlong]
    so.token_range.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.c_longlong, ctypes.c_longlong,
                               ctypes.POINTER(ctypes.c_longlong)]
    return so


def test_packed_conv_taps_stay_inside(indexes):
    """Every channel whose taps a CTA of the packed convolution reads exists, and every pair that it computes
    with has both: down to one channel, for every split of the threads into rows."""
    for ty in (2, 4, 8, 16):
        for rows in (2, 4, 16):
            for dim in (*range(1, 3 * ty + 2), 2 * rows * ty + 1, rows * ty, rows * ty - 1):
                for d0 in range(0, dim, rows * ty):
                    got = [indexes.tap_channel(d0, r, ty, dim) for r in range(rows * ty)]
                    assert all(-1 <= d < dim for d in got), (ty, rows, dim, d0)
                    for r in range(rows * ty):
                        if d0 + r < dim:
                            assert got[r] == d0 + r
                            if r // ty % 2 == 0:                       # its pair's second row
                                assert got[r + ty] == (d0 + r + ty if d0 + r + ty < dim else d0 + r), (ty, rows, dim, d0, r)


def test_token_ranges_are_clamped(indexes):
    big = 2 ** 31 - 1
    bounds = [0, 50, 20, big, -big - 1, 7, 64, 64]
    cu = (ctypes.c_int * len(bounds))(*bounds)
    out = (ctypes.c_longlong * 2)()
    for total in (0, 5, 64):
        for i in range(len(bounds) - 1):
            indexes.token_range(cu, i, total, out)
            lo = min(max(bounds[i], 0), total)
            assert (out[0], out[1]) == (lo, min(max(bounds[i + 1], lo), total))


def test_pointers_off_their_elements_are_refused(ssm):
    """Every array of the slot operators and of the convolution's gradients, the fp32 and int32 ones too: a
    pointer off its element's alignment must not reach a kernel."""
    inv = ssm.SSM_ERR_INVALID_ARG
    scan = ssm.make_dims(2, 32, 64, 16, 0, 1, ssm.SSM_BF16)
    step = ssm.make_dims(2, 32, 1, 16, 0, 1, ssm.SSM_BF16)
    need = ssm.ssm_causal_conv1d_bwd_workspace_size(40, 8, 30, 4, ssm.SSM_BF16)
    # (entry point, its arguments, its pointers' places)
    calls = [
        (ssm.ssm_causal_conv1d_packed_fwd, [8, 20, 2, 4, ssm.SSM_BF16, A16, A16, A16, True, A16, A16, A16, A16, 3, 24, 2 * A16],
         dict(x=5, w=6, bias=7, cu_seqlens=9, slots=10, states=12, out=15)),
        (ssm.ssm_causal_conv1d_update, [2, 8, 4, ssm.SSM_F32, A16, A16, A16, True, A16, A16, 3, 24, 2 * A16],
         dict(x=4, w=5, bias=6, slots=8, states=9, out=12)),
        (ssm.ssm_selective_scan_packed_fwd, [scan, A16, A16, A16, A16, A16, A16, A16, A16, True, A16, A16, A16, A16, 4, 512, 0,
                                             2 * A16, None, 0],
         dict(u=1, delta=2, A=3, B=4, C=5, D=6, z=7, delta_bias=8, cu_seqlens=10, slots=11, states=13, out=17)),
        (ssm.ssm_selective_state_update_slots, [step, A16, A16, 4, 512, A16, A16, A16, A16, A16, A16, A16, A16, True, 2 * A16],
         dict(states=1, slots=2, u=5, delta=6, A=7, B=8, C=9, D=10, z=11, delta_bias=12, out=14)),
        (ssm.ssm_state_slots_copy, [A16, 2, 4, 64, 64, 256, A16, A16, 3], dict(src=6, dst=7)),
        (ssm.ssm_causal_conv1d_bwd, [40, 8, 30, 4, ssm.SSM_BF16, A16, A16, A16, True, A16, 2 * A16, A16, A16, A16, need],
         dict(x=5, w=6, bias=7, dout=9, dx=10, dw=11, dbias=12, workspace=13)),
    ]
    for fn, args, at in calls:
        for name, i in at.items():
            off = args[:i] + [args[i] + 1] + args[i + 1:]
            assert fn(*off, check=False) == inv, (fn.__name__, name)
            if name not in ("x", "u", "delta", "B", "C", "z", "out", "dout", "dx"):    # four-byte elements
                off[i] = args[i] + 2
                if name != "states" or fn is not ssm.ssm_causal_conv1d_packed_fwd:     # (that one's are bf16)
                    assert fn(*off, check=False) == inv, (fn.__name__, name)


def test_packed_scan_hook_refusals(ssm):
    lib = ssm.load_library()
    for budget in (-1, 10 ** 7 + 1):
        assert lib.ssm_selective_scan_packed_test_hooks(0, budget) == ssm.SSM_ERR_INVALID_ARG
    assert ssm.ssm_selective_scan_packed_test_hooks(False) == ssm.SSM_OK


def test_front_end_refusals_with_a_stream(ssm):
    """The same refusals where a stream is given."""
    import torch
    z, i32 = torch.zeros, torch.int32
    for bad, error, word in ((z(2, 4), ValueError, "CUDA"), (None, ValueError, "x must be a tensor"), ([1.0], TypeError, "tensor")):
        with pytest.raises(error, match=word):
            ssm.causal_conv1d_update(bad, z(4, 4), z(2, 4, 3), stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.causal_conv1d_fwd(z(1, 4, 8), z(4, 4), stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.state_slots_copy(z(2, 4), z(1, dtype=i32), z(1, dtype=i32), stream=0)


def test_conv_bwd_cases_take_both_paths(ssm):
    """Which of the shapes that the GPU tests run split a channel's sums over CTAs (a workspace says so), so that a
    change of the rule does not leave one of the paths untested."""
    def split(batch, dim, seqlen, width, io):
        return ssm.ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, width, io) > 0

    assert split(1, 4, 20000, 4, ssm.SSM_F32) and split(40, 16, 130, 4, ssm.SSM_BF16) and split(1, 3, 40001, 3, ssm.SSM_BF16)
    assert not split(2, 24, 67, 4, ssm.SSM_BF16) and not split(1, 3, 5000, 4, ssm.SSM_F32)
    assert not split(1, 2, 8195, 4, ssm.SSM_BF16) and not split(2, 768, 1021, 3, ssm.SSM_F32)
