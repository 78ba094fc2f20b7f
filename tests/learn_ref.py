"""Plain float64 forms of the operators with which the router and the weights
learn, and the error bounds that their tests hold the kernels to.

Bounds: u = 2^-24 is half a unit in the last place of fp32, relative; a sum of
n terms in fp32, in whatever order, is off by at most n u sum|terms|; bf16
rounds by at most 2^-8 relative, E4M3 by 2^-4 (2^-10 below its normal range).
"""
import numpy as np
import torch

U = 2.0 ** -24
UB = 2.0 ** -8
FP8_MAX = 448.0
BLOCK = 256


def softmax64(logits, offset=None):
    z = logits.double() if offset is None else logits.double() + offset.double()
    e = torch.exp(z - z.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def softmax_steps(logits, offset=None):
    """Relative error of an fp32 softmax value, in units of u: l - max is off by
    up to |l - max| + |l| u (the offset's addition), which exp turns into a
    relative error; exp itself, the sum over E and the division add a few."""
    z = logits.double() if offset is None else logits.double() + offset.double()
    z = torch.where(torch.isfinite(z) & (z.abs() < 1e30), z, 0.0)
    reach = float(z.abs().max()) if z.numel() else 0.0
    return 6 * reach + logits.shape[1] + 16


def sequences(T, seq, mask):
    """Rows of each sequence that count."""
    on = np.ones(T, bool) if mask is None else mask.cpu().numpy().astype(bool)
    edge = [0, T] if seq is None else seq.tolist()
    return [torch.tensor([t for t in range(a, b) if on[t]], dtype=torch.long) for a, b in zip(edge, edge[1:])]


def balance(logits, idx, offset=None, mask=None, seq=None, weight=None):
    logits, idx = logits.cpu(), idx.cpu().long()
    T, E = logits.shape
    K = idx.shape[1]
    w = torch.full((E,), float(E), dtype=torch.float64) if weight is None else weight.cpu().double()
    out = []
    for rows in sequences(T, seq, mask):
        n = len(rows)
        c = torch.zeros(E, dtype=torch.float64)
        for i in idx[rows].reshape(-1).tolist():
            if 0 <= i < E:
                c[i] += 1
        if n == 0:
            z = torch.zeros(E, dtype=torch.float64)
            out.append((torch.zeros((), dtype=torch.float64), z, z, z))
            continue
        P = softmax64(logits[rows], None if offset is None else offset.cpu()).mean(0)
        f = w * c / (K * n)
        out.append(((f * P).sum(), c, P, f / n))
    return tuple(torch.stack([o[i] for o in out]) if out else torch.zeros(0) for i in range(4))


def route_backward(logits, idx=None, dgate=None, coef=None, dloss=None, offset=None, mask=None, seq=None):
    """(dlogits, the magnitude its error is relative to)."""
    logits = logits.cpu()
    T, E = logits.shape
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu().bool()
    a = torch.zeros(T, E, dtype=torch.float64)
    mag = torch.zeros(T, E, dtype=torch.float64)
    if dgate is not None:
        for t in range(T):
            for i, g in zip(idx[t].tolist(), dgate[t].double().tolist()):
                if 0 <= i < E:
                    a[t, i] += g
                    mag[t, i] += abs(g)
    live = on.clone() if dgate is not None else torch.zeros(T, dtype=torch.bool)
    if coef is not None:
        for s, rows in enumerate(sequences(T, seq, mask)):
            c = coef[s].cpu().double() * dloss[s].cpu().double()
            a[rows] += c
            mag[rows] += c.abs()
            live[rows] = True
    out, size = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    if live.any():
        p = softmax64(logits[live], None if offset is None else offset.cpu())
        al, ml = a[live], mag[live]
        out[live] = p * (al - (p * al).sum(1, keepdim=True))
        size[live] = p * (ml + (p * ml).sum(1, keepdim=True))
    return out, size


def combine_backward(dout, x, y, slot, gate):
    """(dgate, the sum of |terms| of each, dy; rows of dy no slot names are NaN)."""
    dout, x, y, slot, gate = (t.cpu() for t in (dout, x, y, slot, gate))
    T, K = slot.shape
    d = dout.double()
    dgate, mag = torch.zeros(T, K, dtype=torch.float64), torch.zeros(T, K, dtype=torch.float64)
    dy = torch.full(y.shape, float("nan"), dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            s = int(slot[t, k])
            row = (x[t] if s < 0 else y[s]).double()
            dgate[t, k], mag[t, k] = (d[t] * row).sum(), (d[t] * row).abs().sum()
            if s >= 0:
                dy[s] = gate[t, k].double() * d[t]
    return dgate, mag, dy


def adamw(p, g, m, v, n, lr, betas, eps, wd, gscale=1.0):
    """New (p, m, v) in float64 and the bounds of the fp32 step's errors.

    m: two products and a sum, 3 u of their magnitudes; v the same with g^2
    (all terms positive): 6 u v.  The step is m / (sqrt(v) + eps) times a
    constant: m's error divided by the denominator, plus the denominator's
    (half of v's 6 u, the root, product and sum: 8 u) and the constant's; the
    weight: 3 u |p|."""
    p, g, m, v = (t.double().cpu() for t in (p, g, m, v))
    b1, b2 = betas
    g = g * gscale
    m1 = b1 * m + (1 - b1) * g
    m_err = 4 * U * (abs(b1 * m) + abs((1 - b1) * g))
    v1 = b2 * v + (1 - b2) * g * g
    v_err = 6 * U * v1 + 1e-44
    den = (v1 / (1 - b2 ** n)).sqrt() + eps
    k = lr / (1 - b1 ** n)
    upd = k * m1 / den
    p1 = p * (1 - lr * wd) - upd
    p_err = 3 * U * (abs(p) + abs(upd)) + 16 * U * abs(upd) + k * m_err / den
    return (p1, m1, v1), (p_err, m_err + 1e-44, v_err)


def dequantise(codes, scales):
    """Values of E4M3 codes (any shape) with a scale per BLOCK elements, float64."""
    q = codes.reshape(-1).view(torch.float8_e4m3fn).double().cpu()
    s = scales.double().cpu().repeat_interleave(BLOCK)[: q.numel()]
    return (q * s).view(codes.shape)


def check_codes(codes, scales, want, err):
    """The codes are want's (float64, flat blocks; known to within err) nearest
    ones: each value is within half a step of it, plus err, the rounding of
    value * (448 / amax) (4 u), and the scale's own 3 u."""
    want, err = want.reshape(-1), err.reshape(-1)
    n = want.numel()
    for b in range(0, n, BLOCK):
        w, e = want[b:b + BLOCK], err[b:b + BLOCK]
        amax = max(float(w.abs().max()), 2.0 ** -100)
        s = float(scales[b // BLOCK])
        assert abs(s - amax / FP8_MAX) <= (4 * U * amax + float(e.max())) / FP8_MAX
        got = codes.reshape(-1)[b:b + BLOCK].view(torch.float8_e4m3fn).double().cpu()
        half = torch.clamp(got.abs() * 2.0 ** -4, min=2.0 ** -10)
        bound = half * s * (1 + 16 * U) + e + 8 * U * w.abs()
        bad = (got * s - w).abs() > bound
        yield b, bad, got, w
