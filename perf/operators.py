"""Measured cases of the operators that serve and train a Mamba layer around its scan.

Serving keeps every sequence's recurrent state in a slot of a pool: the last width - 1 inputs of
the causal convolution and the fp32 state of the selective scan.  Prompts arrive packed end to end
(time along the rows, cu_seqlens marking the bounds), continue from their slots and leave their
states there; then single tokens step the slots, and slots are forked, moved and freed.  Training
needs the convolution's gradients.

`run` computes each operator in its plain form (torch operations in fp32, rounded once at the end),
or, with `own` set, through the package's entry points.
"""
import math
import random

import torch

own = False

F32, BF16 = "f32", "bf16"


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float32


def _esize(case):
    return 2 if case["dtype"] == BF16 else 4


# ------------------------------------------------------------------ the cases

def _conv_prompts(dim, n_seq, total, tail, width, dtype, name=None):
    return _named(dict(op="conv_prompts", dim=dim, n_seq=n_seq, total=total, tail=tail, width=width, dtype=dtype), name)


def _conv_tokens(dim, batch, pad, width, dtype, name=None):
    return _named(dict(op="conv_tokens", dim=dim, batch=batch, pad=pad, width=width, dtype=dtype), name)


def _scan_prompts(dim, heads, groups, dstate, n_seq, total, tail, dtype, name=None):
    return _named(dict(op="scan_prompts", dim=dim, heads=heads, groups=groups, dstate=dstate, n_seq=n_seq, total=total,
                       tail=tail, dtype=dtype), name)


def _scan_tokens(dim, heads, groups, dstate, batch, pad, dtype, name=None):
    return _named(dict(op="scan_tokens", dim=dim, heads=heads, groups=groups, dstate=dstate, batch=batch, pad=pad,
                       dtype=dtype), name)


def _conv_bwd(batch, dim, seqlen, width, dtype, name=None):
    return _named(dict(op="conv_bwd", batch=batch, dim=dim, seqlen=seqlen, width=width, dtype=dtype), name)


def _slots_copy(layers, slots, row, pairs, freed, kind, dtype, name=None):
    return _named(dict(op="slots_copy", layers=layers, slots=slots, row=row, pairs=pairs, freed=freed, kind=kind,
                       dtype=dtype), name)


def _named(case, name):
    return dict(case, name=name) if name else case


def listed():
    return [
        # a few prompts of a chat turn through the layer of the 130M model: an odd packed length
        _conv_prompts(1536, 7, 1013, 0, 4, BF16, "conv-prompts-chat"),
        # a full prefill batch of the 1.4B model, its packed buffer longer than its prompts
        _conv_prompts(4096, 32, 32768, 24, 4, BF16, "conv-prompts-batch"),
        # the convolution of one decode step for a handful of users: launch latency
        _conv_tokens(1536, 4, 0, 4, BF16, "conv-tokens-few"),
        # ragged prompts of a prefill batch, 1.4B model
        _scan_prompts(4096, 4096, 1, 16, 24, 16384, 0, BF16, "scan-prompts-ragged"),
        # one long prompt alone, 130M model: few rows, an odd length
        _scan_prompts(1536, 1536, 1, 16, 1, 8191, 0, BF16, "scan-prompt-single"),
        # the per-head layout with 128 states, some prompts
        _scan_prompts(2048, 32, 1, 128, 6, 4096, 0, BF16, "scan-prompts-heads"),
        # one decode step for a handful of users, fp32
        _scan_tokens(1536, 1536, 1, 16, 4, 0, F32, "scan-tokens-few"),
        # one decode step of a full batch, padded to the size its graph was captured with
        _scan_tokens(4096, 4096, 1, 16, 248, 8, BF16, "scan-tokens-batch"),
        # training the 130M model's layer
        _conv_bwd(8, 1536, 2048, 4, BF16, "conv-bwd-130m"),
        # a small fp32 training run on an odd length
        _conv_bwd(2, 768, 1021, 3, F32, "conv-bwd-odd"),
        # a prompt forked into several continuations: scan states of every layer
        _slots_copy(24, 48, 1536 * 16, 8, 0, "fork", F32, "slots-fork"),
        # a pool compacted after sequences ended, the freed slots cleared: convolution states of every layer
        _slots_copy(48, 256, 4096 * 3, 64, 32, "move", BF16, "slots-compact"),
    ]


def _between(rng, lo, hi):
    """A whole number whose logarithm is spread evenly over the range."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("conv_prompts", "conv_tokens", "scan_prompts", "scan_prompts", "scan_tokens", "conv_bwd",
                     "slots_copy"))
    dtype = rng.choice((BF16, BF16, F32))
    if op == "conv_prompts":
        n_seq, dim = _between(rng, 1, 64), _between(rng, 24, 2048 if dtype == F32 else 4096)
        total = max(n_seq, _between(rng, 16, 32768))
        return _conv_prompts(dim, n_seq, total, rng.choice((0, 0, 5, 40)), rng.choice((2, 3, 4, 4)), dtype)
    if op == "conv_tokens":
        return _conv_tokens(_between(rng, 24, 5120), _between(rng, 1, 512), rng.choice((0, 0, 3, 17)),
                            rng.choice((2, 3, 4, 4)), dtype)
    if op == "conv_bwd":
        seqlen, dim = _between(rng, 3, 8192), _between(rng, 24, 2048)
        batch = max(1, min(_between(rng, 1, 32), 8 * 1536 * 2048 // ((2 if dtype == F32 else 1) * dim * seqlen)))
        return _conv_bwd(batch, dim, seqlen, rng.choice((2, 3, 4, 4)), dtype)
    if op == "slots_copy":
        kind = rng.choice(("fork", "move"))
        layers, pairs, freed = _between(rng, 1, 48), _between(rng, 1, 64), rng.choice((0, 0, 1, 9))
        row = 8 * _between(rng, 8, 4096) if rng.random() < 0.7 else 2 * _between(rng, 8, 8192) + 1
        slots = 2 * pairs + freed + _between(rng, 1, 64)
        return _slots_copy(layers, slots, row, pairs, freed, kind, dtype)
    heads_layout = rng.random() < 0.35
    if heads_layout:
        head_dim, dstate = rng.choice((16, 32, 64, 64, 128)), rng.choice((64, 128, 128))
        heads = _between(rng, 2, 2048 // head_dim)
        dim, groups = heads * head_dim, (2 if heads % 2 == 0 and rng.random() < 0.3 else 1)
    else:
        dstate = rng.choice((8, 16, 16, 16, 32))
        dim = 4 * _between(rng, 8, 1024)
        heads, groups = dim, rng.choice((1, 1, 1, 2))
    if op == "scan_tokens":
        # at most the states of the largest listed batch
        batch = max(1, min(_between(rng, 1, 512), 256 * 4096 * 16 // (dim * dstate)))
        return _scan_tokens(dim, heads, groups, dstate, batch, rng.choice((0, 0, 3, 8)), dtype)
    n_seq = _between(rng, 1, 64)
    most = max(64, min(16384, 4096 * 16384 * 16 // (dim * dstate * (2 if dtype == F32 else 1))))
    total = max(n_seq, _between(rng, 16, most))
    return _scan_prompts(dim, heads, groups, dstate, n_seq, total, rng.choice((0, 0, 3, 40)), dtype)


# ------------------------------------------------------------------ the inputs

def _lengths(rng, n, total):
    """n lengths of at least one token that add up to total, as ragged as requests are."""
    w = [math.exp(rng.gauss(0.0, 0.8)) for _ in range(n)]
    spare, s = total - n, sum(w)
    lens = [1 + int(spare * x / s) for x in w]
    lens[rng.randrange(n)] += total - sum(lens)
    return lens


def _packed(case, rng):
    lens = _lengths(rng, case["n_seq"], case["total"])
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    n_slots = case["n_seq"] + max(2, case["n_seq"] // 4)
    slots = rng.sample(range(n_slots), case["n_seq"])
    has = [1] * ((case["n_seq"] + 1) // 2) + [0] * (case["n_seq"] // 2)   # the first half or so continue from their slots
    rng.shuffle(has)
    return dict(lens=lens, n_slots=n_slots, max_seqlen=max(lens), used=cu[-1],
                cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                slots=torch.tensor(slots, dtype=torch.int32, device="cuda"),
                has=torch.tensor(has, dtype=torch.uint8, device="cuda"))


def _rows(case, rng):
    """Slots of a token batch; -1 marks the padding rows, which sit behind the live ones."""
    n, pad = case["batch"], case["pad"]
    n_slots = n + max(2, n // 4)
    slots = rng.sample(range(n_slots), n)
    return dict(n_slots=n_slots, slots=torch.tensor(slots + [-1] * pad, dtype=torch.int32, device="cuda"), rows=n + pad)


def _scan_weights(case, normal, uniform):
    D, H, N = case["dim"], case["heads"], case["dstate"]
    if H == D:
        A = -torch.arange(1, N + 1, dtype=torch.float32, device="cuda").repeat(D, 1)
    else:
        A = -(1.0 + 15.0 * uniform(H))
    dt = torch.exp(uniform(H) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    return dict(A=A.contiguous(), D=normal(D), delta_bias=dt + torch.log(-torch.expm1(-dt)))


def prepare(case, seed):
    rng = random.Random(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    io = _dtype(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op = case["op"]
    st = {"case": case}
    if op == "conv_prompts":
        D, W, T = case["dim"], case["width"], case["total"] + case["tail"]
        st.update(_packed(case, rng))
        st.update(x=normal(D, T, dtype=io), w=normal(D, W) / math.sqrt(W), bias=0.1 * normal(D),
                  pool=normal(st["n_slots"], D, W - 1, dtype=io), out=torch.zeros(D, T, dtype=io, device="cuda"))
    elif op == "conv_tokens":
        D, W = case["dim"], case["width"]
        st.update(_rows(case, rng))
        st.update(x=normal(st["rows"], D, dtype=io), w=normal(D, W) / math.sqrt(W), bias=0.1 * normal(D),
                  pool=normal(st["n_slots"], D, W - 1, dtype=io), out=torch.zeros(st["rows"], D, dtype=io, device="cuda"))
    elif op == "scan_prompts":
        D, H, G, N, T = case["dim"], case["heads"], case["groups"], case["dstate"], case["total"] + case["tail"]
        st.update(_packed(case, rng))
        st.update(_scan_weights(case, normal, uniform))
        st.update(u=normal(D, T, dtype=io), delta=(0.5 * normal(H, T)).to(io), B=normal(G, N, T, dtype=io),
                  C=normal(G, N, T, dtype=io), z=normal(D, T, dtype=io), pool=0.5 * normal(st["n_slots"], D, N),
                  out=torch.zeros(D, T, dtype=io, device="cuda"))
    elif op == "scan_tokens":
        D, H, G, N = case["dim"], case["heads"], case["groups"], case["dstate"]
        st.update(_rows(case, rng))
        st.update(_scan_weights(case, normal, uniform))
        R = st["rows"]
        st.update(u=normal(R, D, dtype=io), delta=(0.5 * normal(R, H)).to(io), B=normal(R, G, N, dtype=io),
                  C=normal(R, G, N, dtype=io), z=normal(R, D, dtype=io), pool=0.5 * normal(st["n_slots"], D, N),
                  out=torch.zeros(R, D, dtype=io, device="cuda"))
    elif op == "conv_bwd":
        Bt, D, L, W = case["batch"], case["dim"], case["seqlen"], case["width"]
        st.update(x=normal(Bt, D, L, dtype=io), dout=normal(Bt, D, L, dtype=io), w=normal(D, W) / math.sqrt(W),
                  bias=0.1 * normal(D))
    else:
        S, P, Fr = case["slots"], case["pairs"], case["freed"]
        ids = rng.sample(range(S), 2 * P + Fr)
        # a fork copies one slot to many, a move each of many to a place of its own
        src = [ids[0]] * P if case["kind"] == "fork" else ids[P:2 * P]
        st.update(pool=normal(case["layers"], S, case["row"], dtype=io), clears=Fr,
                  src=torch.tensor(src + [-1] * Fr, dtype=torch.int32, device="cuda"),
                  dst=torch.tensor((ids[1:P + 1] if case["kind"] == "fork" else ids[:P]) + ids[2 * P:],
                                   dtype=torch.int32, device="cuda"))
    return st


# ------------------------------------------------------------------ the plain forms

def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(x):
    # the linear part and the rest, which loses nothing on either side
    return torch.clamp(x, min=0.0) + torch.log1p(torch.exp(-torch.abs(x)))


def _token_places(st):
    """For every packed token its sequence and its place in it."""
    t = torch.arange(st["used"], device="cuda")
    seq = torch.searchsorted(st["cu"].long(), t, right=True) - 1
    return t, seq, t - st["cu"].long()[seq]


def _plain_conv_prompts(st):
    W, n = st["w"].shape[1], st["used"]
    slots, cu, pool = st["slots"].long(), st["cu"].long(), st["pool"]
    x = st["x"][:, :n].float()
    history = (pool[slots].float() * st["has"].float()[:, None, None]).permute(1, 0, 2)    # (dim, sequence, tap)
    t, seq, place = _token_places(st)
    v = st["bias"][:, None].expand(-1, n)
    for k in range(W):
        back = W - 1 - k
        before = history[:, seq, (place + k).clamp(max=max(W - 2, 0))] if back else 0.0
        v = v + st["w"][:, k, None] * torch.where(place >= back, x[:, (t - back).clamp(min=0)], before)
    st["out"][:, :n] = _silu(v).to(st["out"].dtype)
    # the last width - 1 inputs, from the history where the sequence is shorter
    end = cu[1:, None] - (W - 1) + torch.arange(W - 1, device="cuda")                      # (sequence, tap)
    own_input = end >= cu[:-1, None]
    old = (W - 1 + end - cu[:-1, None]).clamp(max=W - 2)
    kept = torch.where(own_input, x[:, end.clamp(min=0)], torch.gather(history, 2, old.expand(x.shape[0], -1, -1)))
    pool[slots] = kept.permute(1, 0, 2).to(pool.dtype)
    return [st["out"], pool]


def _plain_conv_tokens(st):
    n, pool = st["case"]["batch"], st["pool"]
    slots = st["slots"][:n].long()
    taps = torch.cat([pool[slots].float(), st["x"][:n].float()[:, :, None]], 2)
    st["out"][:n] = _silu((taps * st["w"]).sum(2) + st["bias"]).to(st["out"].dtype)
    pool[slots] = taps[:, :, 1:].to(pool.dtype)
    return [st["out"], pool]


def _per_channel(v, dim):
    """Rows of heads or groups repeated for each of their channels."""
    return v.repeat_interleave(dim // v.shape[0], 0, output_size=dim) if v.shape[0] != dim else v


def _plain_scan_prompts(st):
    n, D = st["used"], st["u"].shape[0]
    slots, cu, pool = st["slots"].long(), st["cu"].long(), st["pool"]
    u, z = st["u"][:, :n].float(), st["z"][:, :n].float()
    dt = _per_channel(_softplus(st["delta"][:, :n].float() + st["delta_bias"][:, None]), D)
    A = st["A"] if st["A"].dim() == 2 else _per_channel(st["A"], D)[:, None]
    Bm, Cm = (_per_channel(st[k][:, :, :n].float().transpose(1, 2), D) for k in ("B", "C"))     # (dim, time, state)
    a = torch.exp(dt[:, :, None] * A[:, None, :]).expand(-1, -1, pool.shape[2]).contiguous()
    h = (dt * u)[:, :, None] * Bm
    del Bm
    start = cu[:-1]
    h[:, start] += a[:, start] * (pool[slots] * st["has"].float()[:, None, None]).transpose(0, 1)
    a[:, start] = 0.0           # nothing passes from one sequence to the next
    shift = 1
    while shift < st["max_seqlen"]:     # (a, h) after (a', h') is (a a', a h' + h): doubled until it spans the longest prompt
        h[:, shift:] += a[:, shift:] * h[:, :-shift]
        a[:, shift:] = a[:, shift:] * a[:, :-shift]
        shift *= 2
    y = (h * Cm).sum(2) + st["D"][:, None] * u
    st["out"][:, :n] = (y * _silu(z)).to(st["out"].dtype)
    pool[slots] = h[:, cu[1:] - 1].transpose(0, 1)
    return [st["out"], pool]


def _plain_scan_tokens(st):
    n, D, pool = st["case"]["batch"], st["u"].shape[1], st["pool"]
    slots = st["slots"][:n].long()
    u, z = st["u"][:n].float(), st["z"][:n].float()
    dt = _per_channel(_softplus(st["delta"][:n].float() + st["delta_bias"]).t(), D).t()
    A = st["A"] if st["A"].dim() == 2 else _per_channel(st["A"], D)[:, None]
    Bm, Cm = (_per_channel(st[k][:n].float().transpose(0, 1), D).transpose(0, 1) for k in ("B", "C"))
    h = torch.exp(dt[:, :, None] * A) * pool[slots] + (dt * u)[:, :, None] * Bm
    y = (h * Cm).sum(2) + st["D"] * u
    st["out"][:n] = (y * _silu(z)).to(st["out"].dtype)
    pool[slots] = h
    return [st["out"], pool]


def _plain_conv_bwd(st):
    x, g, w = st["x"].float(), st["dout"].float(), st["w"]
    L, W = x.shape[2], w.shape[1]
    xp = torch.cat([x.new_zeros(x.shape[0], x.shape[1], W - 1), x], 2)
    v = st["bias"][:, None] + sum(w[:, k, None] * xp[:, :, k:k + L] for k in range(W))
    s = 1.0 / (1.0 + torch.exp(-v))
    dv = g * s * (1.0 + v * (1.0 - s))
    dvp = torch.cat([dv, x.new_zeros(x.shape[0], x.shape[1], W - 1)], 2)
    dx = sum(w[:, k, None] * dvp[:, :, W - 1 - k:W - 1 - k + L] for k in range(W))
    dw = torch.stack([(dv * xp[:, :, k:k + L]).sum((0, 2)) for k in range(W)], 1)
    return [dx.to(st["x"].dtype), dw, dv.sum((0, 2))]


def _plain_slots_copy(st):
    pool, src, dst = st["pool"], st["src"].long(), st["dst"].long()
    rows = pool[:, src.clamp(min=0)]
    pool[:, dst] = torch.where(src[:, None] >= 0, rows, torch.zeros_like(rows))
    return [pool]


def _own(st):
    import selective_state_space_30_b200 as ssm
    op = st["case"]["op"]
    if op == "conv_prompts":
        out = ssm.causal_conv1d_packed(st["x"], st["w"], st["cu"], st["pool"], slots=st["slots"], has_state=st["has"],
                                       bias=st["bias"], silu=True, out=st["out"])
        return [out, st["pool"]]
    if op == "conv_tokens":
        out = ssm.causal_conv1d_update(st["x"], st["w"], st["pool"], slots=st["slots"], bias=st["bias"], silu=True,
                                       out=st["out"])
        return [out, st["pool"]]
    if op == "scan_prompts":
        out = ssm.selective_scan_packed(st["u"], st["delta"], st["A"], st["B"], st["C"], st["cu"], st["pool"],
                                        slots=st["slots"], has_state=st["has"], D=st["D"], z=st["z"],
                                        delta_bias=st["delta_bias"], softplus=True, max_seqlen=st["max_seqlen"],
                                        out=st["out"])
        return [out, st["pool"]]
    if op == "scan_tokens":
        out = ssm.selective_state_update_slots(st["pool"], st["u"], st["delta"], st["A"], st["B"], st["C"],
                                               slots=st["slots"], D=st["D"], z=st["z"], delta_bias=st["delta_bias"],
                                               softplus=True, out=st["out"])
        return [out, st["pool"]]
    if op == "conv_bwd":
        g = ssm.causal_conv1d_bwd(st["x"], st["w"], st["dout"], bias=st["bias"], silu=True)
        return [g["dx"], g["dw"], g["dbias"]]
    return [ssm.state_slots_copy(st["pool"], st["src"], st["dst"], slot_dim=1)]


def run(state):
    if own:
        return _own(state)
    return globals()["_plain_" + state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    e, op = _esize(case), case["op"]
    if op == "conv_prompts":
        D, W, T, n = case["dim"], case["width"], case["total"], case["n_seq"]
        return {"bytes": 2 * D * T * e + D * (W + 1) * 4 + (n + (n + 1) // 2) * D * (W - 1) * e,
                "flops": D * T * (2 * W + 4)}
    if op == "conv_tokens":
        D, W, n = case["dim"], case["width"], case["batch"]
        return {"bytes": 2 * D * n * e + D * (W + 1) * 4 + 2 * n * D * (W - 1) * e, "flops": D * n * (2 * W + 4)}
    if op in ("scan_prompts", "scan_tokens"):
        D, H, G, N = case["dim"], case["heads"], case["groups"], case["dstate"]
        T = case["total"] if op == "scan_prompts" else case["batch"]
        states = case["n_seq"] + (case["n_seq"] + 1) // 2 if op == "scan_prompts" else 2 * T
        weights = (D * N if H == D else H) + D + H
        # an exp and its product for each decay, which a head's channels and states share
        decays = 2 * D * N if H == D else 2 * H
        return {"bytes": T * e * (3 * D + H + 2 * G * N) + 4 * weights + 4 * states * D * N,
                "flops": T * (5 * D * N + decays + 8 * D + 4 * H)}
    if op == "conv_bwd":
        M, D, W = case["batch"] * case["dim"] * case["seqlen"], case["dim"], case["width"]
        return {"bytes": 3 * M * e + 2 * D * (W + 1) * 4, "flops": M * (6 * W + 10)}
    # a fork reads its source once
    read = 1 if case["kind"] == "fork" else case["pairs"]
    return {"bytes": case["layers"] * case["row"] * e * (read + case["pairs"] + case["freed"]), "flops": 0}


# ------------------------------------------------------------------ the definitions, in 64 bits

def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _gate64(v):
    return v * torch.sigmoid(v)


def _bounds(st):
    cu = [0]
    for n in st["lens"]:
        cu.append(cu[-1] + n)
    return list(zip(cu[:-1], cu[1:], st["slots"].tolist(), st["has"].tolist()))


def _exact_conv_prompts(st):
    w, W = st["w"].double(), st["w"].shape[1]
    out, pool = st["out"].double(), st["pool"].double()
    for lo, hi, slot, has in _bounds(st):
        row = torch.cat([pool[slot] * has, st["x"][:, lo:hi].double()], 1)
        out[:, lo:hi] = _gate64((row.unfold(1, W, 1) * w[:, None]).sum(2) + st["bias"].double()[:, None])
        pool[slot] = row[:, row.shape[1] - (W - 1):]
    return [out, pool]


def _exact_conv_tokens(st):
    out, pool, w, W = st["out"].double(), st["pool"].double(), st["w"].double(), st["w"].shape[1]
    for r, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            old = pool[slot].clone()
            v = st["bias"].double() + w[:, W - 1] * st["x"][r].double() + torch.einsum("dk,dk->d", w[:, :W - 1], old)
            out[r] = _gate64(v)
            pool[slot, :, :W - 2] = old[:, 1:]
            pool[slot, :, W - 2] = st["x"][r].double()
    return [out, pool]


def _scan64(st):
    """Decay rates (dim, state or 1) and the maps from channels to heads and groups."""
    D, H, G = st["case"]["dim"], st["case"]["heads"], st["case"]["groups"]
    d = torch.arange(D, device="cuda")
    head, group = d // (D // H), d // (D // G)
    A = st["A"].double()
    return (A if A.dim() == 2 else A[head][:, None]), head, group


def _step64(st, A, head, group, h, u, delta, Bv, Cv, z):
    """One step of every given row; the rows come first."""
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    dt = torch.logaddexp(zero, delta.double() + st["delta_bias"].double())[:, head]
    u = u.double()
    h = h * torch.exp(dt[:, :, None] * A) + (dt * u)[:, :, None] * Bv.double()[:, group]
    y = torch.einsum("rdn,rdn->rd", h, Cv.double()[:, group]) + st["D"].double() * u
    return h, y * _gate64(z.double())


def _exact_scan_prompts(st):
    A, head, group = _scan64(st)
    longest = max(st["lens"])
    if longest * 400e-6 + longest * st["case"]["n_seq"] * A.shape[0] * st["pool"].shape[2] * 1.2e-10 > 18:
        return None
    out, pool = st["out"].double(), st["pool"].double()
    order = sorted(_bounds(st), key=lambda b: b[0] - b[1])      # the longest first, so that the live ones lead
    slots = torch.tensor([b[2] for b in order], device="cuda")
    first = torch.tensor([b[0] for b in order], device="cuda")
    h = pool[slots] * torch.tensor([float(b[3]) for b in order], device="cuda")[:, None, None]
    rows = {k: st[k].movedim(-1, 0) for k in ("u", "delta", "B", "C", "z")}
    live = len(order)
    for t in range(longest):
        while order[live - 1][1] - order[live - 1][0] <= t:
            live -= 1
        at = first[:live] + t
        h[:live], y = _step64(st, A, head, group, h[:live], *(rows[k][at] for k in ("u", "delta", "B", "C", "z")))
        out[:, at] = y.t()
    pool[slots] = h
    return [out, pool]


def _exact_scan_tokens(st):
    A, head, group = _scan64(st)
    out, pool = st["out"].double(), st["pool"].double()
    n = st["case"]["batch"]
    slots = st["slots"][:n].long()
    pool[slots], out[:n] = _step64(st, A, head, group, pool[slots], *(st[k][:n] for k in ("u", "delta", "B", "C", "z")))
    return [out, pool]


def _exact_conv_bwd(st):
    x, w, bias = (st[k].double().requires_grad_() for k in ("x", "w", "bias"))
    W = w.shape[1]
    row = torch.nn.functional.pad(x, (W - 1, 0))
    y = _gate64((row.unfold(2, W, 1) * w[:, None]).sum(3) + bias[:, None])
    return list(torch.autograd.grad(y, (x, w, bias), st["dout"].double()))


def _exact_slots_copy(st):
    before = st["pool"].double()
    after = before.clone()
    for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
        after[:, d] = before[:, s] if s >= 0 else 0.0
    return [after]
