"""The operators on packed prompts and state slots against their fp64 forms (needs a B200).

Tolerances are the running error bounds of tests/slots_plain.py.  Inputs are normals in the I/O type;
untouched places of outputs and pools hold a pattern that has to survive.
"""
import numpy as np
import pytest
import torch

import slots_plain as sp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    import selective_state_space_30_b200 as m
    return m


IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def rnd(gen, *shape, dtype="f32", scale=1.0):
    return (scale * torch.randn(*shape, generator=gen)).to(IO[dtype]).cuda()


def unaligned(t):
    """The same values one element off the allocation's alignment."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    v = buf[1:].view(t.shape)
    v.copy_(t)
    return v


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def packing(lens, head=0, tail=0):
    cu = np.concatenate([[0], np.cumsum(lens)]) + head
    return cu.astype(np.int64), int(cu[-1] + tail), list(zip(cu[:-1].tolist(), cu[1:].tolist()))


def gapped_pool(gen, n_slots, dim, last, dtype, gap):
    """A pool (n_slots, dim, last) whose slots lie `gap` elements apart, and the whole buffer."""
    buf = rnd(gen, n_slots, dim * last + gap, dtype=dtype)
    return buf[:, :dim * last].view(n_slots, dim, last) if gap == 0 else \
        torch.as_strided(buf, (n_slots, dim, last), (dim * last + gap, last, 1)), buf


# ------------------------------------------------------------------ the convolution

CONV = [
    # lens, dim, width, dtype, silu, bias, head, tail, gap, shift bases
    ([5, 1, 17, 0, 64, 3], 40, 4, "bf16", True, True, 0, 0, 0, False),     # 90 tokens: rows off the 16-byte grid
    ([8, 8, 16, 32], 16, 4, "bf16", True, True, 0, 0, 0, False),           # aligned rows
    ([1], 24, 4, "bf16", True, True, 0, 0, 0, False),
    ([1, 1, 1, 1, 2, 2, 3], 33, 4, "f32", True, False, 0, 5, 3, False),
    ([0, 0, 7, 0], 8, 3, "f32", False, True, 3, 6, 0, False),
    ([700, 3, 1300, 21], 70, 4, "bf16", True, True, 2, 7, 8, False),       # several time tiles
    ([2100], 9, 2, "f32", True, True, 0, 0, 0, True),
    ([40, 55], 12, 4, "bf16", True, True, 1, 0, 0, True),
    ([40, 56], 12, 1, "bf16", True, True, 0, 0, 0, False),                 # no history at all
    ([3, 4, 5] * 40, 300, 4, "bf16", True, True, 0, 0, 0, False),          # many short prompts
    ([1, 2, 0, 5] * 300, 3, 4, "bf16", True, True, 0, 0, 0, False),        # more than a CTA looks at one by one
    ([900, 1, 700], 1, 4, "f32", True, True, 0, 3, 0, False),              # one channel
    ([4096, 4096], 130, 4, "bf16", True, True, 0, 8, 0, False),            # aligned rows, whole pieces, an odd last pair
    ([2048, 2048], 67, 3, "f32", True, False, 0, 0, 0, False),
]


def _conv_case(case, seed=7):
    lens, dim, width, dtype, silu, bias, head, tail, gap, shift = case
    gen = torch.Generator().manual_seed(seed)
    cu, total, bounds = packing(lens, head, tail)
    n = len(lens)
    x = rnd(gen, dim, total, dtype=dtype)
    w = rnd(gen, dim, width, scale=0.5)
    b = rnd(gen, dim, scale=0.3) if bias else None
    pool, buf = gapped_pool(gen, n + 3, dim, width - 1, dtype, gap)
    out = rnd(gen, dim, total, dtype=dtype)
    if shift:
        x, out = unaligned(x), unaligned(out)
    rng = np.random.default_rng(seed)
    slots = rng.permutation(n + 3)[:n].tolist()
    has = rng.integers(0, 2, n).tolist()
    return x, w, b, pool, buf, out, cu, bounds, slots, has, silu, dtype


@pytest.mark.parametrize("case", CONV, ids=range(len(CONV)))
def test_conv_packed(ssm, case):
    x, w, b, pool, buf, out, cu, bounds, slots, has, silu, dtype = _conv_case(case)
    before = f64(buf)
    ref, err, ref_pool = sp.conv_packed(f64(x), f64(w), f64(b) if b is not None else np.zeros(w.shape[0]), silu, bounds,
                                        slots, has, f64(pool), f64(out))
    # tokens of no sequence are not read: NaN there changes nothing
    x[:, :bounds[0][0]] = float("nan")
    x[:, bounds[-1][1]:] = float("nan")
    got = ssm.causal_conv1d_packed(x, w, i32(cu), pool, slots=i32(slots), has_state=torch.tensor(has, dtype=torch.uint8).cuda(),
                                   bias=b, silu=silu, out=out)
    assert got is out
    sp.check(f64(got), ref, err, dtype, "out")
    assert np.array_equal(f64(pool), ref_pool), "the kept inputs are copies"
    after = f64(buf)
    gap = buf.shape[1] - pool.shape[1] * pool.shape[2]
    if gap:
        assert np.array_equal(after[:, -gap:], before[:, -gap:])


def test_conv_packed_padding_and_bad_slots(ssm):
    case = ([6, 9, 2, 30, 4], 20, 4, "bf16", True, True, 0, 3, 0, False)
    x, w, b, pool, buf, out, cu, bounds, slots, has, silu, dtype = _conv_case(case)
    has = [1] * 5
    slots[1], slots[3], slots[4] = -1, len(pool), 2 ** 31 - 1
    ref, err, ref_pool = sp.conv_packed(f64(x), f64(w), f64(b), silu, bounds, slots, has, f64(pool), f64(out))
    got = ssm.causal_conv1d_packed(x, w, i32(cu), pool, slots=i32(slots), has_state=torch.ones(5, dtype=torch.bool).cuda(),
                                   bias=b, silu=silu, out=out)
    sp.check(f64(got), ref, err, dtype, "out")
    assert np.array_equal(f64(pool), ref_pool)


def test_conv_packed_defaults(ssm):
    """No slots (slot i for i), no flags (from zero), an output of the call's own (zeros where no token is)."""
    gen = torch.Generator().manual_seed(3)
    x, w, pool = rnd(gen, 16, 40, dtype="bf16"), rnd(gen, 16, 4), rnd(gen, 2, 16, 3, dtype="bf16")
    bounds = [(0, 11), (11, 32)]
    ref, err, ref_pool = sp.conv_packed(f64(x), f64(w), np.zeros(16), True, bounds, [0, 1], [0, 0], f64(pool), np.zeros((16, 40)))
    got = ssm.causal_conv1d_packed(x, w, i32([0, 11, 32]), pool)
    sp.check(f64(got), ref, err, "bf16", "out")
    assert np.array_equal(f64(pool), ref_pool)


@pytest.mark.parametrize("dim,batch,width,dtype,gap", [
    (1536, 4, 4, "bf16", 0), (40, 7, 4, "bf16", 8), (33, 5, 4, "bf16", 0), (64, 3, 3, "f32", 4), (20, 9, 2, "f32", 1),
    (24, 3, 1, "bf16", 0), (5, 1, 4, "f32", 0), (200, 130, 4, "bf16", 5)])
@pytest.mark.parametrize("silu", [True, False])
def test_conv_update(ssm, dim, batch, width, dtype, gap, silu):
    gen = torch.Generator().manual_seed(11)
    x, w, b = rnd(gen, batch, dim, dtype=dtype), rnd(gen, dim, width, scale=0.5), rnd(gen, dim, scale=0.3)
    pool, buf = gapped_pool(gen, batch + 4, dim, width - 1, dtype, gap)
    out = rnd(gen, batch, dim, dtype=dtype)
    slots = np.random.default_rng(1).permutation(batch + 4)[:batch].tolist()
    if batch > 3:
        slots[1], slots[2] = -7, batch + 4
    xs, old, ref = f64(x), f64(pool), f64(out)
    err, ref_pool = np.zeros_like(ref), old.copy()
    for r, s in enumerate(slots):
        if 0 <= s < len(old):
            taps = np.concatenate([old[s], xs[r][:, None]], 1)
            ref[r], err[r] = sp.conv_token(taps, f64(w), f64(b), silu)
            ref_pool[s] = taps[:, 1:]
        elif s >= 0:
            ref[r] = np.nan
    before = f64(buf)
    got = ssm.causal_conv1d_update(x, w, pool, slots=i32(slots), bias=b, silu=silu, out=out)
    sp.check(f64(got), ref, err, dtype, "out")
    assert np.array_equal(f64(pool), ref_pool)
    if gap:
        assert np.array_equal(f64(buf)[:, -gap:], before[:, -gap:])


# ------------------------------------------------------------------------ the scan

def _scan_inputs(gen, rows, dim, heads, groups, N, dtype, prompts=True, z=True, D=True, bias=True, softplus=True):
    # `rows`: packed tokens (time last) or token rows (first)
    shape = (lambda *s: (*s, rows)) if prompts else (lambda *s: (rows, *s))
    p = dict(u=rnd(gen, *shape(dim), dtype=dtype), delta=rnd(gen, *shape(heads), dtype=dtype, scale=0.7),
             B=rnd(gen, *shape(groups, N), dtype=dtype), C=rnd(gen, *shape(groups, N), dtype=dtype),
             z=rnd(gen, *shape(dim), dtype=dtype) if z else None, D=rnd(gen, dim) if D else None,
             delta_bias=rnd(gen, heads, scale=0.5) - 2.0 if bias else None, softplus=softplus)
    if heads == dim:
        p["A"] = -(torch.rand(dim, N, generator=gen) * 8 + 0.1).cuda()
    else:
        p["A"] = -(torch.rand(heads, generator=gen) * 8 + 0.1).cuda()
    if not softplus:
        # dt itself: not negative
        p["delta"] = p["delta"].abs()
        p["delta_bias"] = p["delta_bias"].abs() if bias else None
    return p


def _plain(p):
    return {k: f64(v) if isinstance(v, torch.Tensor) else v for k, v in p.items()}


def _call(ssm, p, cu, states, out, **kw):
    return ssm.selective_scan_packed(p["u"], p["delta"], p["A"], p["B"], p["C"], cu, states, D=p["D"], z=p["z"],
                                     delta_bias=p["delta_bias"], softplus=p["softplus"], out=out, **kw)


def _chunk(ssm, p, n_seq, max_seqlen=0):
    """Whether the call cuts sequences: the workspace says so."""
    io = ssm.SSM_BF16 if p["u"].dtype == torch.bfloat16 else ssm.SSM_F32
    d = ssm.make_dims(n_seq, p["u"].shape[0], p["u"].shape[1], p["B"].shape[1], p["delta"].shape[0], p["B"].shape[0], io)
    return ssm.ssm_selective_scan_packed_workspace_size(d, max_seqlen)


def _tensor(dim, heads, N, dtype, total, n):
    """The calls that run on the tensor cores."""
    return dtype == "bf16" and heads < dim and dim // heads == 64 and N == 128 and total >= 32 * n


SCAN = [
    # lens, dim, heads, groups, N, dtype, head, tail, gap, shift, kw
    ([64, 32, 96], 64, 64, 1, 16, "bf16", 0, 0, 0, False, {}),                       # aligned rows
    ([5, 1, 17, 0, 44], 40, 40, 1, 16, "bf16", 0, 0, 0, False, {}),                  # 67 tokens
    ([1], 16, 16, 1, 16, "f32", 0, 0, 0, False, {}),
    ([33, 40, 7], 130, 130, 1, 16, "f32", 3, 5, 4, False, {}),                       # a ragged second tile
    ([21, 3], 24, 24, 2, 8, "bf16", 0, 0, 0, False, dict(z=False)),
    ([21, 30], 300, 300, 1, 8, "f32", 0, 1, 2, False, dict(D=False, bias=False)),
    ([50, 2, 30], 72, 72, 3, 32, "bf16", 0, 6, 0, True, {}),
    ([31, 64], 40, 40, 1, 64, "bf16", 1, 0, 0, False, dict(z=False, D=False)),
    ([19, 40], 36, 36, 2, 128, "f32", 0, 0, 0, False, {}),
    ([40, 24, 72], 128, 2, 1, 128, "bf16", 0, 0, 0, False, {}),                      # heads
    ([13, 50], 96, 6, 2, 128, "bf16", 0, 2, 0, False, {}),                           # heads and groups, 65 tokens
    # the tensor-core form: blocks of 128 steps
    ([150, 1, 0, 128, 121], 128, 2, 2, 128, "bf16", 0, 0, 0, False, {}),             # groups, aligned rows
    ([140, 260, 5], 64, 1, 1, 128, "bf16", 3, 4, 4, False, {}),                      # one head, rows off the grid
    ([130, 129, 31], 128, 2, 1, 128, "bf16", 0, 0, 3, True, dict(z=False)),          # shifted bases
    ([256, 40], 64, 1, 1, 128, "bf16", 8, 0, 0, False, dict(D=False, bias=False, softplus=False)),
    ([13, 50], 33, 11, 1, 64, "f32", 0, 0, 0, True, dict(z=False)),                  # heads of three channels
    ([20, 9, 3], 48, 3, 1, 16, "bf16", 0, 0, 0, False, {}),
    ([20, 9, 3], 64, 4, 1, 32, "f32", 0, 0, 0, False, dict(softplus=False)),
    ([25, 39], 64, 4, 2, 8, "bf16", 0, 0, 0, False, {}),
    ([20, 12], 32, 32, 1, 16, "bf16", 0, 0, 0, False, dict(softplus=False, bias=False)),
    ([2, 3, 1] * 30, 50, 50, 1, 16, "bf16", 0, 0, 0, False, {}),                     # many short prompts
    ([1, 0, 3] * 130, 4, 4, 1, 16, "f32", 0, 0, 0, False, {}),                       # more than a CTA's threads
    ([70, 1], 1, 1, 1, 8, "bf16", 0, 0, 0, False, {}),                               # one channel
    ([70, 9], 2, 1, 1, 16, "f32", 0, 0, 0, False, {}),                               # one head of two channels
]


@pytest.mark.parametrize("case", SCAN, ids=range(len(SCAN)))
def test_scan_packed(ssm, case):
    lens, dim, heads, groups, N, dtype, head, tail, gap, shift, kw = case
    gen = torch.Generator().manual_seed(21)
    cu, total, bounds = packing(lens, head, tail)
    n = len(lens)
    p = _scan_inputs(gen, total, dim, heads, groups, N, dtype, **kw)
    states, buf = gapped_pool(gen, n + 2, dim, N, "f32", gap)
    out = rnd(gen, dim, total, dtype=dtype)
    if shift:
        p = {k: unaligned(v) if k in ("u", "delta", "B", "C", "z") and v is not None else v for k, v in p.items()}
        out = unaligned(out)
    rng = np.random.default_rng(2)
    slots, has = rng.permutation(n + 2)[:n].tolist(), rng.integers(0, 2, n).tolist()
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, slots, has, f64(states), f64(out),
                                                  tensor=_tensor(dim, heads, N, dtype, total, n))
    for k in ("u", "delta", "B", "C", "z"):
        if p[k] is not None:
            p[k][..., :head] = float("nan")
            p[k][..., bounds[-1][1]:] = float("nan")
    before = f64(buf)
    flags = torch.tensor(has, dtype=torch.uint8).cuda()
    got = _call(ssm, p, i32(cu), states, out, slots=i32(slots), has_state=flags, max_seqlen=max(lens))
    sp.check(f64(got), ref, err, dtype, "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")
    if gap:
        assert np.array_equal(f64(buf)[:, -gap:], before[:, -gap:])


CUT = [
    # lens, dim, heads, groups, N, dtype, tail
    ([1500], 32, 32, 1, 16, "bf16", 4),
    ([1501], 48, 48, 1, 16, "f32", 0),
    ([300, 900, 1, 0, 129, 128, 640], 36, 36, 2, 16, "bf16", 0),      # cut and uncut sequences, whole chunks
    ([1203], 32, 2, 1, 128, "bf16", 1),
    ([700, 90], 24, 24, 1, 8, "f32", 0),
    ([40, 800], 20, 20, 1, 32, "bf16", 0),
    ([640, 333], 16, 16, 1, 64, "f32", 0),
    ([1200, 77], 64, 1, 1, 128, "bf16", 3),                           # tensor cores, aligned rows
    ([1111], 128, 2, 2, 128, "bf16", 0),                              # and off the grid
]


@pytest.mark.parametrize("case", CUT, ids=range(len(CUT)))
def test_scan_packed_cut_sequences(ssm, case):
    """Few long sequences: chunks that run at the same time and join their states."""
    lens, dim, heads, groups, N, dtype, tail = case
    gen = torch.Generator().manual_seed(22)
    cu, total, bounds = packing(lens, 0, tail)
    n = len(lens)
    p = _scan_inputs(gen, total, dim, heads, groups, N, dtype)
    assert _chunk(ssm, p, n, max(lens)) > 0, "this case is here for the cut path"
    states, out = rnd(gen, n, dim, N), rnd(gen, dim, total, dtype=dtype)
    has = [(i + 1) % 2 for i in range(n)]
    # chunks of at most 2 * 128 tokens at these sizes; the bound takes the longest, at every 32nd token's worth
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, list(range(n)), has, f64(states), f64(out), chunk=128,
                                                  tensor=_tensor(dim, heads, N, dtype, total, n))
    flags = torch.tensor(has, dtype=torch.bool).cuda()
    start = states.clone()
    got = _call(ssm, p, i32(cu), states, out, has_state=flags, max_seqlen=max(lens))
    sp.check(f64(got), ref, err, dtype, "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")
    # the same bits again
    again, out2 = start.clone(), out.clone()
    _call(ssm, p, i32(cu), again, out2, has_state=flags, max_seqlen=max(lens))
    assert torch.equal(again, states) and torch.equal(out2, out)


@pytest.mark.parametrize("z", [True, False])
@pytest.mark.parametrize("lens,head,tail,hint", [
    ([32], 0, 0, 0), ([40], 0, 0, 0), ([33, 31], 0, 0, 0), ([128], 0, 0, 0), ([127, 129], 0, 0, 0), ([300, 1, 211], 0, 0, 1),
    ([7, 260, 250], 5, 6, 1), ([1024], 0, 0, 0), ([900, 3], 1, 8, 0)])
def test_scan_packed_tensor_cores_on_the_grid(ssm, lens, head, tail, hint, z):
    """Rows on the 16-byte grid, whose blocks come and go as boxes: buffers shorter than a box, sequences that
    start and end inside one, neighbours and padding that hold NaN, cut sequences, no gate."""
    gen = torch.Generator().manual_seed(28)
    dim, N = 128, 128
    cu, total, bounds = packing(lens, head, tail)
    assert total % 8 == 0 and total >= 32 * len(lens)
    p = _scan_inputs(gen, total, dim, 2, 2, N, "bf16", z=z)
    states, out = rnd(gen, len(lens) + 1, dim, N), rnd(gen, dim, total, dtype="bf16")
    slots, has = [i + 1 for i in range(len(lens))], [i % 2 for i in range(len(lens))]
    if len(lens) > 2:
        slots[1] = -1
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, slots, has, f64(states), f64(out), chunk=128, tensor=True)
    skip = [(0, head), (bounds[-1][1], total)] + [b for b, s in zip(bounds, slots) if s < 0]
    for k in ("u", "delta", "B", "C", "z"):
        if p[k] is not None:
            for lo, hi in skip:
                p[k][..., lo:hi] = float("nan")
    got = _call(ssm, p, i32(cu), states, out, slots=i32(slots), has_state=torch.tensor(has, dtype=torch.uint8).cuda(),
                max_seqlen=hint)
    sp.check(f64(got), ref, err, "bf16", "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")


@pytest.mark.parametrize("total", [520, 523])
def test_scan_packed_tensor_cores_replayed_and_at_once(ssm, total):
    """One graph serves other lengths (bounds out of order among them), and calls on two streams at once, each
    with its own pool, give what they give alone; all bit for bit."""
    gen = torch.Generator().manual_seed(29)
    dim, N = 128, 128
    cu = i32([0, 300, 301, total])
    ps = [_scan_inputs(gen, total, dim, 2, 1, N, "bf16") for _ in range(2)]
    states, out = torch.zeros(3, dim, N, device="cuda"), torch.zeros(dim, total, device="cuda", dtype=torch.bfloat16)
    _call(ssm, ps[0], cu, states, out, max_seqlen=100)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(ssm, ps[0], cu, states, out, max_seqlen=100)
    for bounds in ([0, 300, 301, total], [0, 0, 0, 0], [5, 130, 258, 515], [0, total, total, total], [9, 5000, -3, 200]):
        want_s, want = torch.zeros_like(states), torch.zeros_like(out)
        _call(ssm, ps[0], i32(bounds), want_s, want, max_seqlen=100)
        states.zero_()
        out.zero_()
        cu.copy_(i32(bounds))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(states, want_s), bounds
        # out of order: [9, total) and [0, 200) are two sequences' tokens, and either's outputs may stay where both write
        once = slice(200, total) if min(bounds) < 0 else slice(0, total)
        assert torch.equal(out[:, once], want[:, once]), bounds
    cu.copy_(i32([0, 300, 301, total]))
    alone = []
    for p in ps:
        s = torch.zeros_like(states)
        alone.append((_call(ssm, p, cu, s, None), s))
    streams = [torch.cuda.Stream() for _ in ps]
    for _ in range(5):
        torch.cuda.synchronize()
        both = []
        for p, stream in zip(ps, streams):
            with torch.cuda.stream(stream):
                s = torch.zeros_like(states)
                both.append((_call(ssm, p, cu, s, None), s))
        torch.cuda.synchronize()
        for got, want in zip(both, alone):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dim,heads,N,head", [(32, 32, 16, 0), (64, 1, 128, 0), (128, 2, 128, 5)])
def test_scan_packed_steps_of_either_sign(ssm, dim, heads, N, head):
    """Without softplus a step is what delta and the bias add up to: negative ones let the state grow."""
    gen = torch.Generator().manual_seed(27)
    lens = [150, 40, 302]
    cu, total, bounds = packing(lens, head)
    p = _scan_inputs(gen, total, dim, heads, 1, N, "bf16", softplus=False)
    p["delta"] = rnd(gen, heads, total, dtype="bf16", scale=0.02)
    p["delta_bias"] = rnd(gen, heads, scale=0.005)
    states, out = rnd(gen, 3, dim, N), rnd(gen, dim, total, dtype="bf16")
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, [0, 1, 2], [1, 0, 1], f64(states), f64(out),
                                                  tensor=_tensor(dim, heads, N, "bf16", total, 3))
    got = _call(ssm, p, i32(cu), states, out, has_state=torch.tensor([1, 0, 1], dtype=torch.uint8).cuda(), max_seqlen=302)
    sp.check(f64(got), ref, err, "bf16", "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")


def test_scan_packed_hint_is_only_a_hint(ssm):
    """A max_seqlen that is too small, zero or too large: right results all the same."""
    gen = torch.Generator().manual_seed(23)
    lens = [700, 30]
    cu, total, bounds = packing(lens)
    p = _scan_inputs(gen, total, 24, 24, 1, 16, "f32")
    states = rnd(gen, 2, 24, 16)
    out = rnd(gen, 24, total)
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, [0, 1], [1, 1], f64(states), f64(out), chunk=128)
    flags = torch.ones(2, dtype=torch.uint8).cuda()
    for hint in (0, 1, 30, 700, 10 ** 9):
        s = states.clone()
        got = _call(ssm, p, i32(cu), s, None, has_state=flags, max_seqlen=hint)
        sp.check(f64(got), ref, err, "f32", "out")
        sp.check(f64(s), ref_pool, pool_err, "f32", "states")


@pytest.mark.parametrize("dim,heads,N", [(32, 32, 16), (64, 1, 128)])
@pytest.mark.parametrize("long", [False, True])
def test_scan_packed_padding_and_bad_slots(ssm, long, dim, heads, N):
    gen = torch.Generator().manual_seed(24)
    lens = [900, 20, 1000, 30, 7] if long else [9, 20, 4, 30, 7]
    cu, total, bounds = packing(lens, 0, 2)
    p = _scan_inputs(gen, total, dim, heads, 1, N, "bf16")
    assert (_chunk(ssm, p, 5, max(lens)) > 0) == long
    states, out = rnd(gen, 4, dim, N), rnd(gen, dim, total, dtype="bf16")
    slots, has = [4, 1, -1, 2 ** 31 - 1, 0], [1] * 5
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, slots, has, f64(states), f64(out), chunk=128 if long else 0,
                                                  tensor=_tensor(dim, heads, N, "bf16", total, 5))
    got = _call(ssm, p, i32(cu), states, out, slots=i32(slots), has_state=torch.ones(5, dtype=torch.uint8).cuda(),
                max_seqlen=max(lens))
    sp.check(f64(got), ref, err, "bf16", "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")


@pytest.mark.parametrize("dim,heads,N", [(16, 16, 16), (64, 1, 128)])
def test_scan_packed_neighbours_do_not_meet(ssm, dim, heads, N):
    """NaN and infinities in one sequence stay there, in aligned and unaligned rows, cut or not."""
    for lens in ([30, 34, 64], [30, 33, 20], [70, 66, 64], [70, 61, 90], [400, 301, 800]):
        gen = torch.Generator().manual_seed(25)
        cu, total, bounds = packing(lens)
        p = _scan_inputs(gen, total, dim, heads, 1, N, "bf16")
        states = rnd(gen, 3, dim, N)
        ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, [0, 1, 2], [0] * 3, f64(states), np.zeros((dim, total)),
                                                      chunk=128, tensor=_tensor(dim, heads, N, "bf16", total, 3))
        lo, hi = bounds[1]
        for k, bad in (("u", float("inf")), ("B", float("nan")), ("C", float("nan")), ("z", float("nan")), ("delta", 1e30)):
            p[k][..., lo:hi] = bad
        got = f64(_call(ssm, p, i32(cu), states, None))
        for i in (0, 2):
            a, b = bounds[i]
            sp.check(got[:, a:b], ref[:, a:b], err[:, a:b], "bf16", "out")
            sp.check(f64(states)[i], ref_pool[i], pool_err[i], "f32", "states")


@pytest.mark.parametrize("case", [
    # dim, heads, groups, N, batch, dtype, gap, kw
    (64, 64, 1, 16, 3, "bf16", 0, {}), (70, 70, 1, 16, 5, "f32", 4, {}), (48, 48, 2, 8, 4, "bf16", 8, dict(z=False)),
    (40, 40, 1, 32, 6, "f32", 0, dict(D=False, bias=False)), (24, 24, 3, 64, 2, "bf16", 0, {}),
    (36, 36, 1, 128, 5, "f32", 0, {}), (128, 2, 1, 128, 5, "bf16", 0, {}), (96, 6, 2, 64, 7, "bf16", 0, {}),
    (33, 11, 1, 16, 5, "f32", 12, dict(softplus=False)), (1536, 1536, 1, 16, 300, "bf16", 0, {}),
], ids=str)
def test_state_update_slots(ssm, case):
    dim, heads, groups, N, batch, dtype, gap, kw = case
    gen = torch.Generator().manual_seed(31)
    p = _scan_inputs(gen, batch, dim, heads, groups, N, dtype, prompts=False, **kw)
    states, buf = gapped_pool(gen, batch + 3, dim, N, "f32", gap)
    out = rnd(gen, batch, dim, dtype=dtype)
    slots = np.random.default_rng(3).permutation(batch + 3)[:batch].tolist()
    if batch > 3:
        slots[0], slots[2] = -1, batch + 3
    ref, err, ref_pool, pool_err = sp.scan_tokens(_plain(p), slots, f64(states), f64(out))
    before = f64(buf)
    got = ssm.selective_state_update_slots(states, p["u"], p["delta"], p["A"], p["B"], p["C"], slots=i32(slots), D=p["D"],
                                           z=p["z"], delta_bias=p["delta_bias"], softplus=p["softplus"], out=out)
    sp.check(f64(got), ref, err, dtype, "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")
    if gap:
        assert np.array_equal(f64(buf)[:, -gap:], before[:, -gap:])


# ----------------------------------------------------------------------- the slots

@pytest.mark.parametrize("shape,slot_dim,dtype,view", [
    ((6, 40), 0, torch.float32, None), ((6, 5, 33), 0, torch.bfloat16, None), ((3, 9, 7, 3), 1, torch.bfloat16, None),
    ((2, 70, 4096 + 24), 1, torch.float32, None), ((2, 9, 5000), 1, torch.uint8, None), ((8, 1), 0, torch.uint8, None),
    ((4, 9, 24, 16), 1, torch.float32, "gap"), ((9, 4, 50), 1, torch.bfloat16, "inner"),
    ((1, 9, 12289), 1, torch.bfloat16, "shift")], ids=str)
def test_slots_copy(ssm, shape, slot_dim, dtype, view):
    gen = torch.Generator().manual_seed(41)
    pool = torch.randint(0, 255, shape, generator=gen, dtype=torch.uint8).cuda().to(dtype)
    whole = pool
    if view == "gap":          # one of two tensors' worth per slot
        whole = torch.randn(*shape[:-1], 2 * shape[-1], generator=gen).cuda()
        whole = whole.view(shape[0], shape[1], 2, -1)
        pool = whole[:, :, 0].view(shape)
    elif view == "inner":      # the layers of a slot side by side
        whole = torch.randn(shape[1], shape[0], *shape[2:], generator=gen).cuda().to(dtype)
        pool = whole.transpose(0, 1)
        shape = tuple(pool.shape)
    elif view == "shift":
        pool = unaligned(pool)
        whole = pool
    n = shape[slot_dim]
    rng = np.random.default_rng(5)
    # a swap, a chain, a fork, a clear, a copy onto itself, and pairs that are skipped
    perm = rng.permutation(n).tolist()
    a = perm + [perm[0]] * 6
    pairs = [(a[0], a[1]), (a[1], a[0]), (-1, a[2])]
    if n > 6:
        pairs += [(a[0], a[3]), (a[3], a[4]), (a[4], a[5]), (a[6], a[6])]
    pairs += [(n, a[2]), (a[0], -1), (a[0], n), (2 ** 31 - 1, 0), (0, -2 ** 31)]
    before = pool.clone()
    ref = before.clone()
    idx = (slice(None),) * slot_dim
    for s, d in pairs:
        if s < n and 0 <= d < n:
            ref[idx + (d,)] = before[idx + (s,)] if s >= 0 else 0
    other = whole[:, :, 1].clone() if view == "gap" else None
    got = ssm.state_slots_copy(pool, i32([s for s, _ in pairs]), i32([d for _, d in pairs]), slot_dim=slot_dim)
    assert got is pool
    assert torch.equal(got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8))
    if other is not None:
        assert torch.equal(whole[:, :, 1], other)


@pytest.mark.parametrize("row,dtype", [(16, torch.float32), (7, torch.bfloat16)])
def test_slots_copy_permutes_a_large_pool(ssm, row, dtype):
    """As many pairs as a call takes, a random permutation: every source is read before it is written."""
    n = 4096
    pool = torch.randn(2, n, row, generator=torch.Generator().manual_seed(42)).to(dtype).cuda()
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(43))
    ref = pool[:, perm.cuda()].clone()
    ssm.state_slots_copy(pool, perm.int().cuda(), torch.arange(n, dtype=torch.int32).cuda(), slot_dim=1)
    assert torch.equal(pool, ref)


# ------------------------------------------------------------- together, as they are used

def test_prompts_then_tokens_then_a_fork(ssm):
    """Prompts in two halves, then tokens one by one, then a fork that goes on: the same as the whole
    sequence at once, within the bounds of both."""
    gen = torch.Generator().manual_seed(51)
    dim, N, width, lens = 48, 16, 4, [37, 20, 64]
    steps, half = 6, [19, 20, 1]
    n = len(lens)
    cu, total, bounds = packing([a + steps for a in lens])
    x = rnd(gen, dim, total)
    w, b = rnd(gen, dim, width, scale=0.5), rnd(gen, dim, scale=0.3)
    p = _scan_inputs(gen, total, dim, dim, 1, N, "f32")
    slots, pool_n = [4, 0, 2], 6
    conv_pool, states = rnd(gen, pool_n, dim, width - 1), rnd(gen, pool_n, dim, N)
    u_ref, u_err, _ = sp.conv_packed(f64(x), f64(w), f64(b), True, bounds, slots, [0] * n, f64(conv_pool), np.zeros((dim, total)))
    plain = _plain(p)
    plain["u"] = u_ref
    ref, err, ref_pool, pool_err = sp.scan_packed(plain, bounds, slots, [0] * n, f64(states), np.zeros((dim, total)))
    # what u's own error moves: the recurrence is linear in u
    mag = dict(plain, u=np.abs(u_err), B=np.abs(plain["B"]), C=np.abs(plain["C"]), D=np.abs(plain["D"]),
               z=np.full_like(plain["z"], 1e9))
    moved, _, moved_pool, _ = sp.scan_packed(mag, bounds, slots, [0] * n, np.zeros((pool_n, dim, N)), np.zeros((dim, total)))
    err = err + moved / 1e9 * np.maximum(np.abs(sp.silu(plain["z"])), 0.0) * 2
    pool_err = pool_err + 2 * np.abs(moved_pool)

    def cut(t, parts):
        return torch.cat([t[..., lo:hi] for lo, hi in parts], -1).contiguous()

    def prompts(parts, has):
        pcu, ptotal, pb = packing([hi - lo for lo, hi in parts])
        q = {k: cut(v, parts) if k in ("delta", "B", "C", "z") else v for k, v in p.items()}
        flags = torch.tensor([has] * n, dtype=torch.uint8).cuda()
        u = ssm.causal_conv1d_packed(cut(x, parts), w, i32(pcu), conv_pool, slots=i32(slots), has_state=flags, bias=b)
        o = ssm.selective_scan_packed(u, q["delta"], q["A"], q["B"], q["C"], i32(pcu), states, slots=i32(slots), has_state=flags,
                                      D=q["D"], z=q["z"], delta_bias=q["delta_bias"])
        for (lo, hi), (a, c) in zip(parts, pb):
            sp.check(f64(o)[:, a:c], ref[:, lo:hi], err[:, lo:hi], "f32", "prompt")

    prompts([(lo, lo + h) for (lo, _), h in zip(bounds, half)], 0)
    prompts([(lo + h, hi - steps) for (lo, hi), h in zip(bounds, half)], 1)

    def token(k, at, check=True):
        t = [hi - steps + k for _, hi in bounds] + [0]           # a padding row behind the live ones
        rows = at + [-1]
        u = ssm.causal_conv1d_update(x[:, t].t().contiguous(), w, conv_pool, slots=i32(rows), bias=b)
        o = ssm.selective_state_update_slots(states, u, p["delta"][:, t].t().contiguous(), p["A"],
                                             p["B"][:, :, t].permute(2, 0, 1).contiguous(),
                                             p["C"][:, :, t].permute(2, 0, 1).contiguous(), slots=i32(rows), D=p["D"],
                                             z=p["z"][:, t].t().contiguous(), delta_bias=p["delta_bias"])
        for r in range(n):
            sp.check(f64(o)[r], ref[:, t[r]], err[:, t[r]], "f32", f"token {k}")
        return o

    for k in range(steps - 2):
        token(k, slots)
    # fork every sequence into free slots; both go on alike, bit for bit
    forks = [1, 3, 5]
    for pool in (conv_pool, states):
        ssm.state_slots_copy(pool, i32(slots), i32(forks))
    first = [token(k, slots) for k in (steps - 2, steps - 1)]
    second = [token(k, forks) for k in (steps - 2, steps - 1)]
    assert all(torch.equal(f[:n], s[:n]) for f, s in zip(first, second))
    assert torch.equal(states[slots], states[forks]) and torch.equal(conv_pool[slots], conv_pool[forks])
    sp.check(f64(states)[slots], ref_pool[slots], pool_err[slots], "f32", "states")
    # free the first ones
    ssm.state_slots_copy(states, i32([-1] * n), i32(slots))
    assert not states[slots].any() and states[forks].any()


def test_graph_replay_reads_what_changed(ssm):
    """A decode step captured once and replayed with other slots, tokens and a shorter batch."""
    gen = torch.Generator().manual_seed(61)
    dim, N, width, batch = 64, 16, 4, 6
    w, b = rnd(gen, dim, width, scale=0.5), rnd(gen, dim, scale=0.3)
    p = _scan_inputs(gen, batch, dim, dim, 1, N, "bf16", prompts=False)
    conv_pool, states = rnd(gen, 9, dim, width - 1, dtype="bf16"), rnd(gen, 9, dim, N)
    x, slots = rnd(gen, batch, dim, dtype="bf16"), i32([0, 1, 2, 3, 4, 5])
    u, out = torch.zeros_like(x), torch.zeros_like(x)
    src, dst = i32([0]), i32([8])

    def step():
        ssm.causal_conv1d_update(x, w, conv_pool, slots=slots, bias=b, out=u)
        ssm.selective_state_update_slots(states, u, p["delta"], p["A"], p["B"], p["C"], slots=slots, D=p["D"], z=p["z"],
                                         delta_bias=p["delta_bias"], out=out)
        ssm.state_slots_copy(states, src, dst)

    saved = conv_pool.clone(), states.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new_slots, pair in (([5, 3, 7, -1, -1, -1], (3, 2)), ([8, 1, 0, 2, -1, 6], (1, 4))):
        conv_pool.copy_(saved[0])
        states.copy_(saved[1])
        slots.copy_(i32(new_slots))
        src.fill_(pair[0])
        dst.fill_(pair[1])
        x.copy_(rnd(gen, batch, dim, dtype="bf16"))
        u.zero_()
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), conv_pool.clone(), states.clone()
        conv_pool.copy_(saved[0])
        states.copy_(saved[1])
        u.zero_()
        out.fill_(3.0)
        step()
        assert all(torch.equal(a, c) for a, c in zip(got, (out, conv_pool, states)))
        assert torch.equal(out[[i for i, s in enumerate(new_slots) if s < 0]],
                           torch.full_like(out, 3.0)[:new_slots.count(-1)])


def test_packed_graph_with_other_lengths(ssm):
    """Prompts captured once, cut path included, and replayed with other lengths in the same buffer."""
    gen = torch.Generator().manual_seed(62)
    dim, N, total = 32, 16, 1200
    p = _scan_inputs(gen, total, dim, dim, 1, N, "bf16")
    w = rnd(gen, dim, 4)
    assert _chunk(ssm, p, 3) > 0
    cu = i32([0, 400, 800, 1200])
    conv_pool, states = rnd(gen, 3, dim, 3, dtype="bf16"), rnd(gen, 3, dim, N)
    u, out = torch.zeros_like(p["u"]), torch.zeros_like(p["u"])

    def run():
        ssm.causal_conv1d_packed(p["u"], w, cu, conv_pool, out=u)
        _call(ssm, dict(p, u=u), cu, states, out)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for bounds in ([0, 1, 1200, 1200], [5, 700, 703, 1100]):
        cu.copy_(i32(bounds))
        u.zero_(), out.zero_(), states.zero_(), conv_pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = u.clone(), out.clone(), states.clone(), conv_pool.clone()
        u.zero_(), out.zero_(), states.zero_(), conv_pool.zero_()
        run()
        assert all(torch.equal(a, c) for a, c in zip(got, (u, out, states, conv_pool)))
        assert out[:, bounds[0]:bounds[-1]].any() and not out[:, :bounds[0]].any() and not out[:, bounds[-1]:].any()


def test_on_another_stream(ssm):
    """Calls on a stream of their own, several at once, each with its own workspace."""
    gen = torch.Generator().manual_seed(63)
    p = _scan_inputs(gen, 1500, 32, 32, 1, 16, "bf16")
    cu = i32([0, 1500])
    want_s = torch.zeros(1, 32, 16).cuda()
    want = _call(ssm, p, cu, want_s, None)
    streams = [torch.cuda.Stream() for _ in range(3)]
    pools = [torch.zeros(1, 32, 16).cuda() for _ in streams]
    torch.cuda.synchronize()
    got = [_call(ssm, p, cu, s, None, stream=st) for s, st in zip(pools, streams)]
    got.append(_call(ssm, p, cu, torch.zeros(1, 32, 16).cuda(), None, stream=torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got) and all(torch.equal(s, want_s) for s in pools)


def test_offsets_past_32_bits(ssm):
    """A slot that starts more than 2^31 elements into its pool."""
    gen = torch.Generator().manual_seed(64)
    dim, N, stride = 16, 16, 2 ** 30 // 4
    buf = torch.empty(9 * stride + dim * N, device="cuda")
    states = torch.as_strided(buf, (10, dim, N), (stride, N, 1))
    small = torch.zeros(10, dim, N, device="cuda")
    states.zero_()
    p = _scan_inputs(gen, 40, dim, dim, 1, N, "bf16")
    q = _scan_inputs(gen, 2, dim, dim, 1, N, "bf16", prompts=False)
    for pool in (states, small):
        _call(ssm, p, i32([0, 21, 40]), pool, None, slots=i32([9, 8]))
        ssm.selective_state_update_slots(pool, q["u"], q["delta"], q["A"], q["B"], q["C"], slots=i32([9, 8]))
        ssm.state_slots_copy(pool, i32([9]), i32([0]))
        ssm.state_slots_copy(pool, i32([0, -1]), i32([8, 9]))
    assert torch.equal(states, small) and small[8].any()
    del buf, states
    x = rnd(gen, 2, 16, dtype="bf16")
    buf = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    far = torch.as_strided(buf, (2, 16, 3), (2 ** 31 + 64, 3, 1))
    near = torch.zeros(2, 16, 3, dtype=torch.bfloat16, device="cuda")
    far.zero_()
    w = rnd(gen, 16, 4)
    for pool in (far, near):
        ssm.causal_conv1d_update(x, w, pool)
        ssm.causal_conv1d_packed(x.t().contiguous(), w, i32([0, 1, 2]), pool, slots=i32([1, 0]),
                                 has_state=torch.ones(2, dtype=torch.uint8).cuda())
    assert torch.equal(far, near) and near[1].any()


def test_empty_calls(ssm):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    w = z(8, 4)
    pool, states = z(3, 8, 3) + 1, z(3, 8, 16) + 1
    # no sequences
    assert ssm.causal_conv1d_packed(z(8, 5), w, i32([0]), pool).shape == (8, 5)
    ssm.selective_scan_packed(z(8, 5), z(8, 5), z(8, 16), z(1, 16, 5), z(1, 16, 5), i32([0]), states)
    # no rows
    ssm.causal_conv1d_update(z(0, 8), w, pool)
    ssm.selective_state_update_slots(states, z(0, 8), z(0, 8), z(8, 16), z(0, 1, 16), z(0, 1, 16))
    ssm.state_slots_copy(states, i32([]), i32([]))
    torch.cuda.synchronize()
    assert (pool == 1).all() and (states == 1).all()
    # no tokens: a sequence that goes on keeps its state, a new one is zeros
    flags = torch.tensor([1, 0], dtype=torch.uint8).cuda()
    ssm.causal_conv1d_packed(z(8, 0), w, i32([0, 0, 0]), pool, has_state=flags)
    ssm.selective_scan_packed(z(8, 0), z(8, 0), z(8, 16), z(1, 16, 0), z(1, 16, 0), i32([0, 0, 0]), states, has_state=flags)
    torch.cuda.synchronize()
    for t in (pool, states):
        assert (t[0] == 1).all() and (t[1] == 0).all() and (t[2] == 1).all()


def test_bounds_out_of_order_stay_inside(ssm):
    """cu_seqlens that run backwards or past the buffer are clamped: other memory stays as it was."""
    gen = torch.Generator().manual_seed(65)
    dim, N, total = 24, 16, 64
    p = _scan_inputs(gen, total, dim, dim, 1, N, "bf16")
    guard = torch.full((3, dim, total), 7.0, dtype=torch.bfloat16, device="cuda")
    states, conv_pool = rnd(gen, 4, dim, N), rnd(gen, 4, dim, 3, dtype="bf16")
    w = rnd(gen, dim, 4)
    for cu in ([0, 50, 20, 10 ** 9], [-5, 3, -(2 ** 31), 40], [2 ** 31 - 1, 0, 64, 64]):
        _call(ssm, p, i32(cu), states, guard[1])
        ssm.causal_conv1d_packed(p["u"], w, i32(cu), conv_pool, out=guard[1])
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[2] == 7).all()


def test_overlapping_outputs_are_refused(ssm):
    gen = torch.Generator().manual_seed(5)
    x, w, pool, cu = rnd(gen, 8, 40), rnd(gen, 8, 4), rnd(gen, 2, 8, 3), i32([0, 15, 40])
    buf = torch.zeros(8 * 40 + 40, device="cuda")
    for out in (x, buf[40:].view(8, 40)):
        with pytest.raises(ValueError, match="out must not overlap x"):
            ssm.causal_conv1d_packed(x if out is x else buf[:320].view(8, 40), w, cu, pool, out=out)
    ssm.causal_conv1d_packed(buf[:160].view(4, 40), w[:4], cu, pool[:, :4].contiguous(), out=buf[160:320].view(4, 40))
    p = _scan_inputs(gen, 40, 8, 8, 1, 8, "f32")
    states = rnd(gen, 2, 8, 8)
    for k in ("u", "delta", "z", "B", "C"):
        with pytest.raises(ValueError, match=f"out must not overlap {k}"):
            _call(ssm, p, cu, states, p[k].view(8, 40))


def test_front_end_refusals(ssm):
    """Tensors of another shape, type, device or layout than an operator takes."""
    def t(*s, dt=torch.float32):
        return torch.zeros(*s, dtype=dt, device="cuda")

    bf = torch.bfloat16
    x, w, pool, cu = t(2, 8), t(8, 4), t(3, 8, 3), i32([0, 2])
    ok = dict(x=x, w=w, conv_states=pool)
    for bad, word in ((dict(x=t(2, 8).double()), "bfloat16 or float32"), (dict(x=t(8, 2).t()), "contiguous"),
                      (dict(w=t(7, 4)), "w must have shape"), (dict(w=t(8, 5)), "width of 1 to 4"),
                      (dict(w=t(8, 4, dt=bf)), "w must be"), (dict(w=t(4, 8).t()), "w must be contiguous"),
                      (dict(conv_states=t(3, 8, 2)), "conv_states must have shape"),
                      (dict(conv_states=t(3, 8, 3, dt=bf)), "conv_states must be"),
                      (dict(conv_states=t(3, 8, 6)[:, :, ::2]), "every slot"),
                      (dict(conv_states=torch.zeros(3, 8, 3)), "on the device"),
                      (dict(slots=t(2)), "slots must be"), (dict(slots=i32([0])), "slots must have shape"),
                      (dict(bias=t(7)), "bias must have shape"), (dict(out=t(2, 7)), "out must have shape"),
                      (dict(w=None), "w must be a tensor")):
        with pytest.raises(ValueError, match=word):
            ssm.causal_conv1d_update(**{**ok, **bad})
    with pytest.raises(ValueError, match="n_seq"):
        ssm.causal_conv1d_packed(t(8, 2), w, i32([]), pool)
    with pytest.raises(ValueError, match="cu_seqlens must be"):
        ssm.causal_conv1d_packed(t(8, 2), w, cu.long(), pool)
    with pytest.raises(ValueError, match="has_state must be"):
        ssm.causal_conv1d_packed(t(8, 2), w, cu, pool, has_state=i32([1]))
    good = dict(u=t(8, 2), delta=t(8, 2), A=t(8, 16), B=t(1, 16, 2), C=t(1, 16, 2), cu_seqlens=cu, states=t(3, 8, 16))
    for bad, word in ((dict(A=t(8)), "A must have shape"), (dict(A=None), "A must be a tensor"), (dict(C=t(1, 16, 3)), "C must"),
                      (dict(delta=t(8, 2, dt=bf)), "delta must be"), (dict(states=t(3, 8, 16, dt=bf)), "states must be"),
                      (dict(z=t(8, 3)), "z must"), (dict(workspace=torch.zeros(4, dtype=torch.uint8)), "workspace must")):
        with pytest.raises(ValueError, match=word):
            ssm.selective_scan_packed(**{**good, **bad})
    with pytest.raises(ssm.SsmError):                    # the library's own refusals: 24 states, heads that do not divide
        ssm.selective_scan_packed(**{**good, "A": t(8, 24), "B": t(1, 24, 2), "C": t(1, 24, 2), "states": t(3, 8, 24)})
    with pytest.raises(ssm.SsmError):
        ssm.selective_scan_packed(**{**good, "delta": t(3, 2), "A": t(3)})
    with pytest.raises(ssm.SsmError):                    # a workspace that is too small
        ssm.selective_scan_packed(**{**good, "u": t(8, 4096), "delta": t(8, 4096), "B": t(1, 16, 4096), "C": t(1, 16, 4096)},
                                  workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    step = dict(states=t(3, 8, 16), u=x, delta=t(2, 8), A=t(8, 16), B=t(2, 1, 16), C=t(2, 1, 16))
    for bad, word in ((dict(B=t(1, 1, 16)), "B must"), (dict(delta=t(2, 8, 1)), "dimensions"), (dict(D=t(7)), "D must")):
        with pytest.raises(ValueError, match=word):
            ssm.selective_state_update_slots(**{**step, **bad})
    with pytest.raises(ssm.SsmError):                    # slots off the 16-byte grid
        ssm.selective_state_update_slots(**{**step, "states": torch.as_strided(t(3 * 130), (3, 8, 16), (130, 16, 1))})
    for args, word in (((pool, i32([0]), i32([0, 1])), "dst must"), ((pool, t(1), i32([0])), "src must be"),
                       ((pool, i32([0]), i32([0]), 2), "slot_dim"), ((t(3, 8, 6)[:, :, ::2], i32([0]), i32([0])), "every slot")):
        with pytest.raises(ValueError, match=word):
            ssm.state_slots_copy(*args)
    with pytest.raises(ssm.SsmError):                    # layers that overlap
        ssm.state_slots_copy(torch.as_strided(t(100), (2, 3, 8), (4, 8, 1)), i32([0]), i32([1]), slot_dim=1)
    with pytest.raises(ssm.SsmError):                    # more pairs than a call takes
        ssm.state_slots_copy(pool, i32([-1] * 5000), i32([0] * 5000))
    with pytest.raises(ValueError, match="dout must"):
        ssm.causal_conv1d_bwd(t(1, 8, 4), w, t(1, 8, 5))


def test_overlapping_outputs_are_refused_everywhere(ssm):
    """Outputs on what a call reads: the batch convolution, the single-token calls, and the pools and weights of
    the packed ones.  The single-token calls may write over their own x, u or z, and give the same then."""
    gen = torch.Generator().manual_seed(6)
    w, b = rnd(gen, 8, 4), rnd(gen, 8)
    x = rnd(gen, 2, 8, 40)
    buf = torch.zeros(4 * 640, device="cuda")
    for a, out in ((x, x), (buf[:640].view(2, 8, 40), buf[1:641].view(2, 8, 40)), (buf[600:1240].view(2, 8, 40), buf[:640].view(2, 8, 40))):
        with pytest.raises(ValueError, match="out must not overlap x"):
            ssm.causal_conv1d_fwd(a, w, b, out=out)
    assert torch.equal(ssm.causal_conv1d_fwd(x, w, b, out=buf[:640].view(2, 8, 40)), ssm.causal_conv1d_fwd(x, w, b))
    # the packed convolution on its pool, its taps and its lengths
    px, cu = rnd(gen, 8, 40), i32([0, 15, 40])
    flat = torch.zeros(8 * 40 + 48, device="cuda")
    for out, kw, word in ((flat[:320].view(8, 40), dict(conv_states=flat[300:348].view(2, 8, 3)), "conv_states"),
                          (flat[:320].view(8, 40), dict(w=flat[316:348].view(8, 4)), "w"),
                          (flat[:320].view(8, 40), dict(conv_states=torch.as_strided(flat, (2, 8, 3), (300, 3, 1), 10)), "conv_states")):
        with pytest.raises(ValueError, match=f"out must not overlap {word}"):
            ssm.causal_conv1d_packed(**{**dict(x=px, w=w, cu_seqlens=cu, conv_states=rnd(gen, 2, 8, 3), out=out), **kw})
    p = _scan_inputs(gen, 40, 8, 8, 1, 8, "f32")
    with pytest.raises(ValueError, match="out must not overlap states"):
        _call(ssm, p, cu, flat[:128].view(2, 8, 8), flat[:320].view(8, 40))
    with pytest.raises(ValueError, match="out must not overlap A"):
        _call(ssm, dict(p, A=flat[304:368].view(8, 8)), cu, rnd(gen, 2, 8, 8), flat[:320].view(8, 40))
    # single tokens
    tx, pool = rnd(gen, 5, 8), rnd(gen, 5, 8, 3)
    t = torch.zeros(200, device="cuda")
    with pytest.raises(ValueError, match="out must not overlap x"):
        ssm.causal_conv1d_update(t[:40].view(5, 8), w, pool, out=t[8:48].view(5, 8))
    with pytest.raises(ValueError, match="out must not overlap conv_states"):
        ssm.causal_conv1d_update(tx, w, t[:120].view(5, 8, 3), out=t[100:140].view(5, 8))
    over, pools = tx.clone(), (pool.clone(), pool.clone())
    want = ssm.causal_conv1d_update(tx, w, pools[0], bias=b)
    assert torch.equal(ssm.causal_conv1d_update(over, w, pools[1], bias=b, out=over), want) and torch.equal(*pools)
    q = _scan_inputs(gen, 5, 8, 8, 1, 8, "f32", prompts=False)
    states = rnd(gen, 5, 8, 8)

    def step(st, out, **kw):
        a = {**q, **kw}
        return ssm.selective_state_update_slots(st, a["u"], a["delta"], a["A"], a["B"], a["C"], D=a["D"], z=a["z"],
                                                delta_bias=a["delta_bias"], out=out)

    for k in ("delta", "B", "C"):
        with pytest.raises(ValueError, match=f"out must not overlap {k}"):
            step(states, q[k].view(5, 8))
    for k in ("u", "z"):
        with pytest.raises(ValueError, match=f"out must not overlap {k}"):
            step(states, t[1:41].view(5, 8), **{k: t[:40].view(5, 8)})
    with pytest.raises(ValueError, match="out must not overlap states"):
        step(buf[:320].view(5, 8, 8), buf[280:320].view(5, 8))
    first = states.clone()
    want = step(first, None)
    for k in ("u", "z"):
        again, over = states.clone(), q[k].clone()
        assert torch.equal(step(again, over, **{k: over}), want) and torch.equal(again, first)


@pytest.mark.parametrize("dim,heads,N,T", [(32, 32, 16, 1200), (32, 32, 16, 1203), (64, 1, 128, 1200), (64, 1, 128, 1199)])
@pytest.mark.parametrize("many", [False, True])
def test_scan_packed_cut_with_shared_tokens(ssm, dim, heads, N, T, many):
    """Bounds that run backwards where sequences would be cut: each sequence still runs over its own clamped
    range, from its own slot to its own slot, however many chunks that would be."""
    gen = torch.Generator().manual_seed(32)
    p = _scan_inputs(gen, T, dim, heads, 1, N, "bf16")
    cu = [0, T, 0, T, 5, 10 ** 6, -7, 300]
    if many:                                             # more sequences than a warp's lanes
        cu = cu + [T] * 30
    n = len(cu) - 1
    hint = 0 if not many else T
    assert _chunk(ssm, p, n, hint) > 0, "this case is here for the cut path"
    bounds = [(min(max(a, 0), T), min(max(b, min(max(a, 0), T)), T)) for a, b in zip(cu, cu[1:])]
    states, out = rnd(gen, n + 1, dim, N), rnd(gen, dim, T, dtype="bf16")
    slots = np.random.default_rng(3).permutation(n + 1)[:n].tolist()
    has = [0] * n
    _, _, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, slots, has, f64(states), f64(out),
                                              tensor=_tensor(dim, heads, N, "bf16", T, n))
    _call(ssm, p, i32(cu), states, out, slots=i32(slots), has_state=torch.tensor(has, dtype=torch.uint8).cuda(), max_seqlen=hint)
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")
    # the first five tokens start every sequence that holds them
    alone = sp.scan_packed(_plain(p), [(0, T)], [0], [0], np.zeros((1, dim, N)), np.zeros((dim, T)),
                           tensor=_tensor(dim, heads, N, "bf16", T, n))
    sp.check(f64(out)[:, :5], alone[0][:, :5], alone[1][:, :5], "bf16", "out")


@pytest.mark.parametrize("dim,heads,head", [(64, 1, 0), (128, 2, 5)])
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("cut", [False, True])
def test_scan_packed_large_steps(ssm, dim, heads, head, softplus, cut):
    """Steps of a hundred and more among small ones: what decays to nothing leaves the others' weights as they
    are, however far the sums within a stretch run."""
    gen = torch.Generator().manual_seed(33)
    lens = [900, 40, 302] if cut else [150, 40, 302]
    cu, total, bounds = packing(lens, head)
    p = _scan_inputs(gen, total, dim, heads, 1, 128, "bf16", softplus=softplus)
    big = torch.rand(heads, total, generator=gen).cuda()
    steps = torch.where(big > 0.7, 400 * (big - 0.7) / 0.3, 0.05 + 0.1 * big)
    p["delta"] = (torch.where(steps > 20, steps, torch.log(torch.expm1(steps))) if softplus else steps).to(torch.bfloat16)
    p["delta_bias"] = None
    p["A"] = torch.tensor([-16.0, -0.7][:heads]).cuda()
    hint = 900 if cut else 302
    assert (_chunk(ssm, p, 3, hint) > 0) == cut
    states, out = rnd(gen, 3, dim, 128), rnd(gen, dim, total, dtype="bf16")
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, [0, 1, 2], [1, 0, 1], f64(states), f64(out),
                                                  chunk=128 if cut else 0, tensor=True, stretch_sums=False)
    got = _call(ssm, p, i32(cu), states, out, has_state=torch.tensor([1, 0, 1], dtype=torch.uint8).cuda(), max_seqlen=hint)
    sp.check(f64(got), ref, err, "bf16", "out")
    sp.check(f64(states), ref_pool, pool_err, "f32", "states")


@pytest.mark.parametrize("dim,heads,N", [(128, 2, 128), (32, 32, 16)])
@pytest.mark.parametrize("lens,head", [([300, 70, 260], 0), ([299, 70, 258], 3), ([1200, 40], 0), ([1201, 40], 1)])
def test_scan_packed_not_finite_inputs_stay_behind(ssm, dim, heads, N, lens, head):
    """NaN and infinities in u, delta, B, C and z spoil what the recurrence lets them spoil: no earlier token, no
    other channel, with C and z no later token either."""
    gen = torch.Generator().manual_seed(34)
    cu, total, bounds = packing(lens, head)
    n = len(lens)
    p = _scan_inputs(gen, total, dim, heads, 1, N, "bf16")
    cut = _chunk(ssm, p, n, max(lens)) > 0
    assert cut == (lens[0] > 1000)
    start = rnd(gen, n, dim, N)
    ref, err, ref_pool, pool_err = sp.scan_packed(_plain(p), bounds, list(range(n)), [1] * n, f64(start), np.zeros((dim, total)),
                                                  chunk=128 if cut else 0, tensor=_tensor(dim, heads, N, "bf16", total, n))
    flags = torch.ones(n, dtype=torch.uint8).cuda()
    nan, inf = float("nan"), float("inf")

    def run(q):
        states = start.clone()
        out = _call(ssm, q, i32(cu), states, None, has_state=flags, max_seqlen=max(lens))
        return f64(out), f64(states)

    # u: single channels, at the edges of blocks, stretches and groups, several in one block
    lo = bounds[0][0]
    places = [(3, lo, nan), (5, lo + 1, inf), (17, lo + 31, -inf), (18, lo + 32, nan), (30, lo + 127, nan), (31, lo + 128, inf),
              (8, lo + 200, nan), (8, lo + 203, nan), (9, bounds[0][1] - 1, nan), (11, bounds[1][0] + 37, -inf),
              (12, bounds[-1][0] + 5, nan), (12, bounds[-1][1] - 1, inf)]
    if dim > 32:
        places += [(64, lo + 64, nan), (127, lo + 255, inf), (100, bounds[1][1] - 1, nan)]
    q = dict(p, u=p["u"].clone())
    good, live = np.ones((dim, total), bool), np.ones((n, dim), bool)
    for c, t, v in places:
        q["u"][c, t] = v
        s = next(i for i, (a, b) in enumerate(bounds) if a <= t < b)
        good[c, t:bounds[s][1]] = False
        live[s, c] = False
    got, states = run(q)
    assert not np.isfinite(got[~good]).any() and not np.isfinite(states[~live]).any()
    sp.check(np.where(good, got, 0.0), np.where(good, ref, 0.0), err, "bf16", "out")
    sp.check(np.where(live[:, :, None], states, 0.0), np.where(live[:, :, None], ref_pool, 0.0), pool_err, "f32", "states")
    # one token of the others, everything behind it in its sequence (C, z: that token alone)
    for k, after in (("delta", True), ("B", True), ("C", False), ("z", False)):
        for s, at in ((0, 0), (0, 63), (0, 161), (1, 33), (n - 1, 5)):
            a, b = bounds[s]
            t = min(a + at, b - 1)
            q = dict(p, **{k: p[k].clone()})
            q[k][..., t] = nan
            got, states = run(q)
            good = np.ones((dim, total), bool)
            good[:, t:b if after else t + 1] = False
            assert not np.isfinite(got[~good]).any(), (k, t)
            sp.check(np.where(good, got, 0.0), np.where(good, ref, 0.0), err, "bf16", f"out, {k} at {t}")
            ok = np.ones(n, bool)
            ok[s] = not after
            sp.check(states[ok], ref_pool[ok], pool_err[ok], "f32", "states")
            assert ok[s] or not np.isfinite(states[s]).any()


@pytest.mark.parametrize("total,heads", [(472, 2), (473, 2), (4096, 16)])
def test_scan_packed_wait_that_runs_out_is_reported(ssm, total, heads):
    """With the hook on, the third block of a sequence gives up its wait: NaN from there on in its outputs and
    state, the status says so once, other sequences and the next call are as ever."""
    gen = torch.Generator().manual_seed(35)
    dim, N, short = 64 * heads, 128, 100
    p = _scan_inputs(gen, total, dim, heads, 1, N, "bf16")
    cu = i32([0, short, total])
    cut = _chunk(ssm, p, 2, total - short) > 0
    assert cut == (total > 1000)
    want_s = torch.zeros(2, dim, N, device="cuda")
    want = _call(ssm, p, cu, want_s, None, max_seqlen=total - short)
    assert ssm.ssm_selective_scan_packed_device_status() == ssm.SSM_OK
    ssm.ssm_selective_scan_packed_test_hooks(True, 20000)
    try:
        states = torch.zeros(2, dim, N, device="cuda")
        out = _call(ssm, p, cu, states, None, max_seqlen=total - short)
        assert ssm.ssm_selective_scan_packed_device_status() == ssm.SSM_ERR_TIMEOUT
    finally:
        ssm.ssm_selective_scan_packed_test_hooks(False)
    assert ssm.ssm_selective_scan_packed_device_status() == ssm.SSM_OK
    start = short - short % 8 if total % 8 == 0 else short     # where the sequence's first block lies
    assert torch.equal(out[:, :start + 256], want[:, :start + 256]) and torch.equal(states[0], want_s[0])
    assert torch.isnan(out[:, start + 256:]).all()
    assert torch.isnan(states[1]).all()
    again = torch.zeros(2, dim, N, device="cuda")
    assert torch.equal(_call(ssm, p, cu, again, None, max_seqlen=total - short), want) and torch.equal(again, want_s)
    assert ssm.ssm_selective_scan_packed_device_status() == ssm.SSM_OK


def test_inputs_freed_behind_a_call_on_another_stream(ssm):
    """The memory of a call's inputs is not handed out again while a stream that was given has yet to run it."""
    gen = torch.Generator().manual_seed(36)
    n, dim = 1024, 2056                                  # sizes of their own, so that a freed block would fit again
    w, pool, x = rnd(gen, dim, 4), torch.zeros(n, dim, 3, device="cuda"), rnd(gen, n, dim)
    want = ssm.causal_conv1d_update(x.clone(), w, pool.clone())
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        src, kept = x.clone(), pool.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)               # about 50 ms
        got = ssm.causal_conv1d_update(src, w, kept, stream=stream)
        del src
        again = torch.full((n, dim), 7.0, device="cuda")  # in src's place, if that were free
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del again, got, kept


def test_outputs_of_the_calls_own_are_written_whole(ssm):
    """Single tokens without slots have no padding: every row of an output that the call allocates is written, rows
    past the pool with NaN.  With slots the padding rows read as zero."""
    gen = torch.Generator().manual_seed(38)
    batch, dim, N = 70, 328, 16
    w, x = rnd(gen, dim, 4), rnd(gen, batch, dim)
    q = _scan_inputs(gen, batch, dim, dim, 1, N, "f32", prompts=False)

    def stale():
        held = torch.full((batch, dim), 3.0, device="cuda")
        del held                                          # the block that the call's output gets

    for n_slots in (batch, batch - 5):
        pool, states = rnd(gen, n_slots, dim, 3), rnd(gen, n_slots, dim, N)
        for slots in (None, [i if i % 3 else -1 for i in range(batch)]):
            idx = None if slots is None else i32(slots)
            pad = [] if slots is None else [i for i, s in enumerate(slots) if s < 0]
            rows = [i for i in range(batch) if i not in pad]
            def conv(st, out):
                return ssm.causal_conv1d_update(x, w, st, slots=idx, out=out)

            def scan(st, out):
                return ssm.selective_state_update_slots(st, q["u"], q["delta"], q["A"], q["B"], q["C"], slots=idx, D=q["D"],
                                                        z=q["z"], delta_bias=q["delta_bias"], out=out)

            for call, start in ((conv, pool), (scan, states)):
                want = call(start.clone(), torch.full((batch, dim), 5.0, device="cuda"))
                st = start.clone()
                stale()
                got = call(st, None)
                assert torch.equal(torch.nan_to_num(got[rows], 9.0), torch.nan_to_num(want[rows], 9.0))
                assert torch.isnan(got).any() == (n_slots < batch)
                assert not pad or not got[pad].any()


def test_given_stream_in_a_graph(ssm):
    """A call on a given stream that joins a capture."""
    gen = torch.Generator().manual_seed(37)
    w, pool, x = rnd(gen, 40, 4), torch.zeros(6, 40, 3, device="cuda"), rnd(gen, 6, 40)
    out = torch.zeros_like(x)
    want = ssm.causal_conv1d_update(x, w, pool.clone())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        ssm.causal_conv1d_update(x, w, pool, out=out, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del x, graph                                         # what the capture recorded is let go
    torch.cuda.synchronize()
    assert torch.full((6, 40), 2.0, device="cuda").sum() == 480
