"""Plain fp64 forms of the operators on packed prompts and state slots, with bounds on the error that
fp32 arithmetic may make in them.

Each form is a loop over the definition and returns the value with `err`, a bound on how far the kernel's
fp32 value may be from it, derived from the operations it takes (u = 2^-24, half an fp32 step):

  * a sum of n products, |terms| adding up to S:          (n + 1) u S
  * 2^x by ex2.approx: 2^-22 relative, and its argument v log2 e, two roundings: |v| 2^-23
  * 1/x by rcp.approx: 2^-23
  * silu(v) = v / (1 + e^-v), slope at most 1.1:          1.1 err(v) + (|v| + 4) 2^-23 |silu(v)|
  * softplus: the polynomial's 3.4e-7 of log1p(e) (tests/test_softplus_poly.py), e as 2^x above
  * a value stored in type t: eps(t) / 2 of it

The recurrence carries its bound along with the state: one step's decay is off by a relative
|dt A| (err(dt)/dt + 3 u) + 2^-22, its input by err(dt)/dt + 3 u, the sum by u.
"""
import numpy as np

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = 1e-37          # results below the smallest normal fp32 number may be zero


def silu(v):
    # without overflow on either side
    e = np.exp(-np.abs(v))
    return v * np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def silu_err(v, err_v):
    return 1.1 * err_v + (np.abs(v) + 4.0) * 2.0 ** -23 * np.abs(silu(v)) + TINY


def conv_token(taps, w, bias, use_silu):
    """taps (..., width), the newest last."""
    terms = taps * w
    v = terms.sum(-1) + bias
    err = (w.shape[-1] + 1) * U * (np.abs(terms).sum(-1) + np.abs(bias))
    return (silu(v), silu_err(v, err)) if use_silu else (v, err + TINY)


def conv_packed(x, w, bias, use_silu, bounds, slots, has, pool, out):
    """x (dim, total), pool (n_slots, dim, width - 1), out: what it held.  Returns out, err, pool."""
    W = w.shape[1]
    out, pool, before = out.copy(), pool.copy(), pool
    err = np.zeros_like(out)
    for i, (lo, hi) in enumerate(bounds):
        if slots[i] < 0:
            continue
        if slots[i] >= len(pool):
            out[:, lo:hi] = np.nan
            continue
        past = before[slots[i]] if has[i] else np.zeros_like(before[slots[i]])
        row = np.concatenate([past, x[:, lo:hi]], 1)
        for t in range(hi - lo):
            out[:, lo + t], err[:, lo + t] = conv_token(row[:, t:t + W], w, bias, use_silu)
        pool[slots[i]] = row[:, row.shape[1] - (W - 1):]
    return out, err, pool


def softplus(x):
    return np.logaddexp(0.0, x)


def step(h, err, u, delta, A, Bv, Cv, D, z, bias, sp):
    """One step of one row: h, err (dim, dstate); u, D, z (dim) or None; delta, bias (dim); Bv, Cv (dim, dstate)."""
    x = delta + bias
    dt = softplus(x) if sp else x
    rel = 3.4e-7 + 2.0 ** -22 + 2.0 ** -24 + (np.abs(delta) + np.abs(bias)) * 3 * U if sp else \
        np.where(x != 0, (np.abs(delta) + np.abs(bias)) * U / np.where(x != 0, np.abs(x), 1.0), 0.0)
    rel = rel[:, None]
    a = np.exp(dt[:, None] * A)
    inp = (dt * u)[:, None] * Bv
    da = np.abs(dt[:, None] * A) * (rel + 3 * U) + 2.0 ** -22
    new = a * h + inp
    # the fused sum rounds once
    err = a * (1 + da) * err + a * da * np.abs(h) + (rel + 3 * U) * np.abs(inp) + U * np.abs(new) + TINY
    skip = D * u if D is not None else np.zeros_like(u)
    terms = np.abs(Cv * new).sum(1) + np.abs(skip)
    y = (Cv * new).sum(1) + skip
    yerr = (np.abs(Cv) * err).sum(1) + (A.shape[-1] + 2 if A.shape[-1] > 1 else Cv.shape[-1] + 2) * U * terms
    if z is not None:
        g = silu(z)
        yerr = yerr * np.abs(g) + np.abs(y) * silu_err(z, 0.0) + 2 * U * np.abs(y * g)
        y = y * g
    return new, err, y, yerr + TINY


def spread(v, dim, axis=0):
    """Rows of heads or groups repeated for their channels."""
    return np.repeat(v, dim // v.shape[axis], axis) if v.shape[axis] != dim else v


def tensor_err(p, h0, A, delta, bias, lo, hi, dim, stretch_sums=True):
    """What the tensor-core form adds to the errors of the recurrence: for every token of a sequence a bound
    for y ahead of the gate, and one for the state behind it.  mag is the sum of the magnitudes that make up
    the state.

      * an MMA step adds 16 products and the accumulator, cut to the largest one's last bits: 2^-22 of the
        magnitudes.  The state takes 24 steps a block, y 32, G 8.
      * M and the state enter as two bf16 terms: 2^-18 of each product; X' as three: 2^-24 (in the steps')
      * the decay between two steps of a stretch is 2^(difference of two sums of at most 32 terms a): off by
        2 * 32 u max|sum|, relative.  Without `stretch_sums` it is held to what no sum's size enters: a decay
        that is not zero in fp32 is 2^-s, s < 127, whose sum of up to 14 roundings is off by 14 * 127 u ln 2 < 2^-13
    """
    mag, state, y = np.abs(h0), 24 * 2.0 ** -22, []
    a_abs = []
    for t in range(lo, hi):
        x = delta[:, t] + bias
        dt = softplus(x) if p["softplus"] else x
        a = np.abs(dt[:, None] * A) / np.log(2.0)
        a_abs.append(a.max())
        stretch = max(sum(a_abs[max(0, k - 31):k + 1]) for k in range(max(0, len(a_abs) - 32), len(a_abs)))
        mag = np.exp(dt[:, None] * A) * mag + np.abs((dt * p["u"][:, t])[:, None] * spread(p["B"][:, :, t], dim))
        y.append((2.0 ** -18 + 40 * 2.0 ** -22 + (64 * U * stretch if stretch_sums else 2.0 ** -13)) * (np.abs(spread(p["C"][:, :, t], dim)) * mag).sum(1))
    return y, state * mag


def scan_packed(p, bounds, slots, has, pool, out, chunk=0, tensor=False, stretch_sums=True):
    """p: u, delta, A, B, C, D, z, delta_bias, softplus.  `chunk`: tokens of a chunk where sequences are cut;
    the join's product of decays comes from a sum of up to `chunk` dt, whose rounding (chunk u, relative)
    moves exp(-x) by at most 0.37 chunk u, once per chunk.  `tensor`: the shape runs on the tensor cores."""
    dim = p["u"].shape[0]
    out, pool, before = out.copy(), pool.copy(), pool
    err_out, err_pool = np.zeros_like(out), np.zeros_like(pool)
    A = p["A"] if p["A"].ndim == 2 else spread(p["A"], dim)[:, None]
    delta = spread(p["delta"], dim)
    bias = spread(p["delta_bias"], dim) if p["delta_bias"] is not None else np.zeros(dim)
    for i, (lo, hi) in enumerate(bounds):
        if slots[i] < 0:
            continue
        if slots[i] >= len(pool):
            out[:, lo:hi] = np.nan
            continue
        h = before[slots[i]].copy() if has[i] else np.zeros(pool.shape[1:])
        err = np.zeros_like(h)
        for t in range(lo, hi):
            if chunk and t > lo and (t - lo) % chunk == 0:
                # the joined state: one more product and sum besides the decay's
                err = err + (0.37 * chunk + 8) * U * np.maximum(np.abs(h), top)
                top = np.abs(h)
            h, err, out[:, t], err_out[:, t] = step(
                h, err, p["u"][:, t], delta[:, t], A, spread(p["B"][:, :, t], dim), spread(p["C"][:, :, t], dim), p["D"],
                p["z"][:, t] if p["z"] is not None else None, bias, p["softplus"])
            top = np.maximum(top, np.abs(h)) if t > lo else np.abs(h)
        if tensor:
            more, state = tensor_err(p, before[slots[i]] if has[i] else np.zeros_like(h), A, delta, bias, lo, hi, dim,
                                     stretch_sums)
            for t, m in zip(range(lo, hi), more):
                err_out[:, t] += m * (np.abs(silu(p["z"][:, t])) if p["z"] is not None else 1.0)
            err = err + state
        pool[slots[i]], err_pool[slots[i]] = h, err
    return out, err_out, pool, err_pool


def scan_tokens(p, slots, pool, out):
    """Rows first: u (batch, dim), delta (batch, nheads), B and C (batch, ngroups, dstate)."""
    dim = p["u"].shape[1]
    out, pool, before = out.copy(), pool.copy(), pool
    err_out, err_pool = np.zeros_like(out), np.zeros_like(pool)
    A = p["A"] if p["A"].ndim == 2 else spread(p["A"], dim)[:, None]
    bias = spread(p["delta_bias"], dim) if p["delta_bias"] is not None else np.zeros(dim)
    for b, s in enumerate(slots):
        if s < 0:
            continue
        if s >= len(pool):
            out[b] = np.nan
            continue
        pool[s], err_pool[s], out[b], err_out[b] = step(
            before[s], 0.0, p["u"][b], spread(p["delta"][b], dim), A, spread(p["B"][b], dim), spread(p["C"][b], dim),
            p["D"], p["z"][b] if p["z"] is not None else None, bias, p["softplus"])
    return out, err_out, pool, err_pool


def conv_bwd(x, w, bias, dout, use_silu):
    """Gradients of the batch convolution and bounds on their errors: (dx, dw, dbias), (err...)."""
    Bt, D, L = x.shape
    W = w.shape[1]
    xp = np.concatenate([np.zeros((Bt, D, W - 1)), x], 2)
    terms = np.stack([w[:, k, None] * xp[:, :, k:k + L] for k in range(W)])
    v = terms.sum(0) + bias[:, None]
    verr = (W + 1) * U * (np.abs(terms).sum(0) + np.abs(bias)[:, None])
    if use_silu:
        e = np.exp(-np.abs(v))
        s = np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        c = np.where(v >= 0, e / (1.0 + e), 1.0 / (1.0 + e))          # 1 - s, no cancellation
        dv = dout * s * (1.0 + v * c)
        # s is off by (|v| + 3) 2^-23 relative times its slope's share c, plus 2^-23 of the reciprocal; 1 - s by as
        # much of s absolutely; silu'' is at most 1/2
        ds = (np.abs(v) * c + 3.0) * 2.0 ** -23
        dverr = np.abs(dout) * (0.5 * verr + s * (ds * np.abs(1.0 + v * c) + np.abs(v) * (s * ds + U) + U * (1 + np.abs(v))) +
                                2 * U * s * np.abs(1.0 + v * c))
    else:
        dv, dverr = dout.copy(), np.zeros_like(dout)
    pad = np.zeros((Bt, D, W - 1))
    dvp, dvep = np.concatenate([dv, pad], 2), np.concatenate([dverr, pad], 2)
    dx, dxerr, dxmag = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    for k in range(W):
        sl = slice(W - 1 - k, W - 1 - k + L)
        dx += w[:, k, None] * dvp[:, :, sl]
        dxmag += np.abs(w[:, k, None] * dvp[:, :, sl])
        dxerr += np.abs(w[:, k, None]) * dvep[:, :, sl]
    dxerr += W * U * dxmag
    dw = np.stack([(dv * xp[:, :, k:k + L]).sum((0, 2)) for k in range(W)], 1)
    n = Bt * L
    # additions that a value takes part in: a lane's tokens of its share of the batch (a quarter, rounded up; of a
    # row of t tiles of at most 256 tokens up to t + 2, eight tokens a lane each), its warp's lanes, eight warps,
    # and up to 296 partials by eight threads each
    depth = min(n, (Bt // 4 + 1) * (L // 32 + 32) + 5 + 8 + 37 + 8)
    dwerr = np.stack([(dverr * np.abs(xp[:, :, k:k + L])).sum((0, 2)) +
                      depth * U * np.abs(dv * xp[:, :, k:k + L]).sum((0, 2)) for k in range(W)], 1)
    db = dv.sum((0, 2))
    dberr = dverr.sum((0, 2)) + depth * U * np.abs(dv).sum((0, 2))
    return (dx, dw, db), (dxerr + TINY, dwerr + TINY, dberr + TINY)


def check(got, ref, err, dtype, what):
    """|got - ref| <= err + half a step of the stored type; NaN where and only where ref is."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places than expected"
    r = np.where(nan, 0.0, ref)
    bound = err + HALF[dtype] * (np.abs(r) + err)
    bad = (np.abs(np.where(nan, 0.0, got) - r) > bound) & ~nan
    if bad.any():
        k = tuple(int(i[0]) for i in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {k}: got {got[k]!r}, "
                             f"reference {ref[k]!r}, bound {bound[k]!r}")
