"""The causal convolution's gradients against the fp64 formulas and against differences (needs a B200).

Tolerances: the error bounds of tests/slots_plain.py (conv_bwd), plus half a step of dx's type.
"""
import numpy as np
import pytest
import torch

import slots_plain as sp
from test_slots_gpu import IO, f64, rnd, unaligned

pytestmark = pytest.mark.gpu

CASES = [
    # batch, dim, seqlen, width, dtype, silu, bias, shift
    (2, 40, 64, 4, "bf16", True, True, False),
    (2, 24, 67, 4, "bf16", True, True, False),       # rows off the 16-byte grid
    (3, 8, 96, 3, "f32", True, True, False),
    (1, 5, 1, 4, "bf16", True, True, False),         # shorter than the taps
    (2, 7, 2, 4, "f32", True, False, False),
    (2, 9, 33, 1, "f32", True, True, False),
    (2, 9, 515, 2, "bf16", False, True, True),
    (1, 3, 5000, 4, "f32", True, True, False),       # stretches
    (1, 2, 8195, 4, "bf16", True, True, True),
    (40, 16, 130, 4, "bf16", True, False, False),    # many partials
    (1, 4, 20000, 4, "f32", True, True, False),
    (1, 3, 40001, 3, "bf16", True, True, True),
    (2, 768, 301, 4, "f32", True, True, False),      # four warps a pair of channels
    (2, 601, 301, 4, "f32", True, True, True),       # and a last pair of one channel
    (3, 605, 900, 2, "bf16", True, False, False),
    (5, 601, 33, 4, "bf16", True, True, True),
    (3, 1400, 270, 3, "f32", False, True, False),
    (8, 1200, 300, 4, "bf16", True, True, False),    # eight, in several rounds
]


def _inputs(case, seed=5):
    batch, dim, L, width, dtype, silu, bias, shift = case
    gen = torch.Generator().manual_seed(seed)
    x, g = rnd(gen, batch, dim, L, dtype=dtype), rnd(gen, batch, dim, L, dtype=dtype)
    w, b = rnd(gen, dim, width, scale=0.5), rnd(gen, dim, scale=0.3) if bias else None
    if shift:
        x, g = unaligned(x), unaligned(g)
    return x, w, b, g, silu, dtype


@pytest.mark.parametrize("case", CASES, ids=str)
def test_conv_bwd(case):
    import selective_state_space_30_b200 as ssm
    x, w, b, g, silu, dtype = _inputs(case)
    ref, err = sp.conv_bwd(f64(x), f64(w), f64(b) if b is not None else np.zeros(w.shape[0]), f64(g), silu)
    got = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu)
    sp.check(f64(got["dx"]), ref[0], err[0], dtype, "dx")
    sp.check(f64(got["dw"]), ref[1], err[1], "f32", "dw")
    sp.check(f64(got["dbias"]), ref[2], err[2], "f32", "dbias")
    again = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu)
    assert all(torch.equal(got[k], again[k]) for k in got), "fixed-order sums repeat bit for bit"


def test_conv_bwd_plain_form_against_differences():
    """The fp64 formulas the test above uses, against central differences of the fp64 forward."""
    rng = np.random.default_rng(0)
    x, w, b = rng.standard_normal((2, 3, 6)), rng.standard_normal((3, 4)), rng.standard_normal(3)
    g = rng.standard_normal((2, 3, 6))

    def loss(x, w, b):
        xp = np.concatenate([np.zeros((2, 3, 3)), x], 2)
        return (sp.silu(sum(w[:, k, None] * xp[:, :, k:k + 6] for k in range(4)) + b[:, None]) * g).sum()

    ref, _ = sp.conv_bwd(x, w, b, g, True)
    for which, t in enumerate((x, w, b)):
        for i in np.ndindex(t.shape):
            args = [a.copy() for a in (x, w, b)]
            args[which][i] += 1e-5
            up = loss(*args)
            args[which][i] -= 2e-5
            assert abs((up - loss(*args)) / 2e-5 - ref[which][i]) < 1e-7


def test_conv_fn_gradients():
    """The autograd operation, its gradients the library's and, for a broadcast upstream gradient, the formula's."""
    import selective_state_space_30_b200 as ssm
    x, w, b, _, _, _ = _inputs((2, 12, 50, 4, "f32", True, True, False))
    x, w, b = (t.requires_grad_() for t in (x, w, b))
    out = ssm.causal_conv1d_fn(x, w, b)
    scale = torch.tensor(0.5, device="cuda")
    (out.sum() * scale).backward()                       # an expanded, stride-0 gradient
    ref, err = sp.conv_bwd(f64(x), f64(w), f64(b), np.full(x.shape, 0.5), True)
    for got, r, e, what in zip((x.grad, w.grad, b.grad), ref, err, ("dx", "dw", "dbias")):
        sp.check(f64(got), r, e, "f32", what)
    assert ssm.causal_conv1d_fn(x, w, None, False).requires_grad
    with pytest.raises(RuntimeError):                    # once differentiable
        gx, = torch.autograd.grad(ssm.causal_conv1d_fn(x, w, b).sum(), x, create_graph=True)
        gx.sum().backward()


def test_conv_bwd_in_a_graph():
    import selective_state_space_30_b200 as ssm
    x, w, b, g, silu, _ = _inputs(CASES[1])
    nbytes = ssm.ssm_causal_conv1d_bwd_workspace_size(*x.shape, w.shape[1], ssm.SSM_BF16)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    ssm.causal_conv1d_bwd(x, w, g, bias=b, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssm.causal_conv1d_bwd(x, w, g, bias=b, workspace=ws)
    x.copy_(rnd(torch.Generator().manual_seed(9), *x.shape, dtype="bf16"))
    graph.replay()
    want = ssm.causal_conv1d_bwd(x, w, g, bias=b)
    assert all(torch.equal(got[k], want[k]) for k in got)


def test_conv_feeds_the_scan_both_ways():
    """Convolution and scan as one differentiable path: the convolution's gradients take the scan's du."""
    import selective_state_space_30_b200 as ssm
    gen = torch.Generator().manual_seed(12)
    x, w, b = rnd(gen, 2, 32, 40).requires_grad_(), rnd(gen, 32, 4, scale=0.5).requires_grad_(), rnd(gen, 32).requires_grad_()
    delta, A = rnd(gen, 2, 32, 40, scale=0.5), -(torch.rand(32, 16, generator=gen) + 0.5).cuda()
    B, C = rnd(gen, 2, 1, 16, 40), rnd(gen, 2, 1, 16, 40)
    u = ssm.causal_conv1d_fn(x, w, b)
    u.retain_grad()
    out, _ = ssm.selective_scan_fn(u, delta, A, B, C)
    gen_g = rnd(gen, 2, 32, 40)
    out.backward(gen_g)
    want = ssm.causal_conv1d_bwd(x.detach(), w.detach(), u.grad, bias=b.detach())
    assert torch.equal(x.grad, want["dx"]) and torch.equal(w.grad, want["dw"]) and torch.equal(b.grad, want["dbias"])
    assert u.grad.any()


def test_conv_bwd_no_tokens():
    import selective_state_space_30_b200 as ssm
    for shape in ((0, 4, 9), (3, 4, 0)):
        x = torch.zeros(shape, dtype=IO["bf16"], device="cuda")
        g = ssm.causal_conv1d_bwd(x, torch.ones(4, 4, device="cuda"), x)
        assert g["dx"].shape == shape and not g["dw"].any() and not g["dbias"].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", [
    (2, 40, 64, 4, "bf16", False, True, False), (2, 24, 67, 4, "bf16", False, True, False),
    (3, 8, 96, 3, "f32", False, True, False), (1, 5, 1, 4, "bf16", False, True, False), (2, 7, 2, 4, "f32", False, False, False),
    (2, 9, 515, 2, "bf16", False, True, True), (1, 3, 5001, 4, "f32", False, True, False), (2, 9, 256, 4, "bf16", False, True, False),
    (2, 601, 257, 4, "f32", False, True, True), (1, 4, 20000, 4, "bf16", False, True, False)], ids=str)
def test_conv_bwd_last_input_not_finite(case, bad):
    """The last input of a row meets the last tap alone: the other taps' gradients stay finite."""
    import selective_state_space_30_b200 as ssm
    x, w, b, g, silu, dtype = _inputs(case)
    x[..., -1] = bad
    with np.errstate(invalid="ignore"):
        ref, err = sp.conv_bwd(f64(x), f64(w), f64(b) if b is not None else np.zeros(w.shape[0]), f64(g), silu)
    assert np.isfinite(ref[1][:, :-1]).all() and not np.isfinite(ref[1][:, -1]).any()
    got = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu)
    sp.check(f64(got["dx"]), ref[0], err[0], dtype, "dx")
    sp.check(f64(got["dw"])[:, :-1], ref[1][:, :-1], err[1][:, :-1], "f32", "dw")
    assert not np.isfinite(f64(got["dw"])[:, -1]).any()
    sp.check(f64(got["dbias"]), ref[2], err[2], "f32", "dbias")


@pytest.mark.parametrize("case", [(1, 4, 20000, 4, "f32", True, True, False), (40, 16, 130, 4, "bf16", True, True, False),
                                  (1, 3, 40001, 3, "bf16", False, True, True)], ids=str)
def test_conv_bwd_split_sums_in_a_graph(case):
    """A channel split over CTAs: the second kernel and the caller's workspace in a graph, which holds nothing
    from one replay to the next."""
    import selective_state_space_30_b200 as ssm
    x, w, b, g, silu, dtype = _inputs(case)
    nbytes = ssm.ssm_causal_conv1d_bwd_workspace_size(*x.shape, w.shape[1], ssm.SSM_BF16 if dtype == "bf16" else ssm.SSM_F32)
    assert nbytes > 0, "this case is here for the second kernel"
    ws = torch.empty(nbytes // 4, device="cuda")
    ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu, workspace=ws.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu, workspace=ws.view(torch.uint8))
    for seed in (9, 10):
        x.copy_(rnd(torch.Generator().manual_seed(seed), *x.shape, dtype=dtype))
        ws.fill_(float("nan"))
        graph.replay()
        ref, err = sp.conv_bwd(f64(x), f64(w), f64(b), f64(g), silu)
        for k, r, e, t in zip(("dx", "dw", "dbias"), ref, err, (dtype, "f32", "f32")):
            sp.check(f64(got[k]), r, e, t, k)
        want = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu)
        assert all(torch.equal(got[k], want[k]) for k in got)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [(2, 40, 64, 4, "bf16", True, True, False), (2, 24, 67, 3, "bf16", True, True, True),
                                  (1, 4, 5001, 4, "f32", True, False, False)], ids=str)
def test_conv_bwd_last_input_not_finite_with_silu(case, bad):
    """With silu the last token's own derivative is not finite then, and with it every tap; other rows stay."""
    import selective_state_space_30_b200 as ssm
    x, w, b, g, silu, dtype = _inputs(case)
    x[-1, 1, -1] = bad
    with np.errstate(invalid="ignore", over="ignore"):
        ref, err = sp.conv_bwd(f64(x), f64(w), f64(b) if b is not None else np.zeros(w.shape[0]), f64(g), silu)
    got = ssm.causal_conv1d_bwd(x, w, g, bias=b, silu=silu)
    rows = [r for r in range(x.shape[1]) if r != 1]
    assert not np.isfinite(ref[1][1]).any() and not np.isfinite(f64(got["dw"])[1]).any() and not torch.isfinite(got["dbias"][1])
    sp.check(f64(got["dw"])[rows], ref[1][rows], err[1][rows], "f32", "dw")
    sp.check(f64(got["dbias"])[rows], ref[2][rows], err[2][rows], "f32", "dbias")
    sp.check(f64(got["dx"])[:, rows], ref[0][:, rows], err[0][:, rows], dtype, "dx")
    # the row's own dx up to the tokens that reach the last one
    n = x.shape[2] - w.shape[1]
    sp.check(f64(got["dx"])[:, 1, :n], ref[0][:, 1, :n], err[0][:, 1, :n], dtype, "dx")
