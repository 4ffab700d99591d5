"""Gated linear recurrence in fp64 numpy, token by token: outputs, final states, gradients, paged decode.

    h[t] = a[t] h[t-1] + b[t], y = h;   log gate: a = e^g, b = x;  sigmoid gate: a = s(z), b = (1 - a) x
    D[t] = dy[t] + a[t+1] D[t+1] (+ d_final at the last token)

Besides the values, ``scan`` returns for every token the sum that a rounding of each step to u relative
accuracy can leave in it, in units of u: e[t] = a[t] e[t-1] + r[t] m[t], with m the same recurrence over
absolute values and r = 1 + |log a| (the argument's rounding grows with it)."""
import numpy as np

LOG_DECAY, SIGMOID = 0, 1


def gates(gate, kind):
    """(a, 1 - a) without cancellation."""
    g = np.asarray(gate, dtype=np.float64)
    if kind == LOG_DECAY:
        return np.exp(g), -np.expm1(g)
    e = np.exp(-np.abs(g))
    big, small = 1.0 / (1.0 + e), e / (1.0 + e)
    return np.where(g >= 0, big, small), np.where(g >= 0, small, big)


def _growth(a):
    with np.errstate(divide="ignore"):
        return 1.0 + np.minimum(np.abs(np.log(a)), 100.0)


def scan(x, gate, kind, cu, h0=None):
    """Returns dict: y [T, D], final [N, D], prev (h[t-1]) [T, D], err [T, D], err_prev, err_final."""
    x = np.asarray(x, dtype=np.float64)
    a, q = gates(gate, kind)
    b = x if kind == LOG_DECAY else q * x
    r = _growth(a)
    T, D = x.shape
    N = len(cu) - 1
    out = {k: np.zeros((T, D)) for k in ("y", "prev", "err", "err_prev")}
    out["final"], out["err_final"] = np.zeros((N, D)), np.zeros((N, D))
    for n in range(N):
        h = np.zeros(D) if h0 is None else np.asarray(h0[n], dtype=np.float64).copy()
        m, e = np.abs(h), np.zeros(D)
        for t in range(int(cu[n]), int(cu[n + 1])):
            out["prev"][t], out["err_prev"][t] = h, e
            h = a[t] * h + b[t]
            m = a[t] * m + np.abs(b[t])
            e = a[t] * e + r[t] * m
            out["y"][t], out["err"][t] = h, e
        out["final"][n], out["err_final"][n] = h, e
    return out


def grads(x, gate, kind, cu, dy, h0=None, d_final=None):
    """Returns dict: dx, dgate [T, D], dh0 [N, D] and their error sums err_dx, err_dgate, err_dh0."""
    x, dy = np.asarray(x, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    f = scan(x, gate, kind, cu, h0)
    a, q = gates(gate, kind)
    r = _growth(a)
    T, D = x.shape
    N = len(cu) - 1
    out = {k: np.zeros((T, D)) for k in ("dx", "dgate", "err_dx", "err_dgate")}
    out["dh0"], out["err_dh0"] = np.zeros((N, D)), np.zeros((N, D))
    for n in range(N):
        c = np.zeros(D) if d_final is None else np.asarray(d_final[n], dtype=np.float64).copy()
        m, e = np.abs(c), np.zeros(D)
        for t in range(int(cu[n + 1]) - 1, int(cu[n]) - 1, -1):
            Dt = dy[t] + c
            m = m + np.abs(dy[t])
            e = e + m
            if kind == LOG_DECAY:
                u, eu = a[t] * f["prev"][t], a[t] * (f["err_prev"][t] + r[t] * np.abs(f["prev"][t]))
                out["dx"][t], out["err_dx"][t] = Dt, e
            else:
                w = a[t] * q[t]
                u = w * (f["prev"][t] - x[t])
                eu = w * (f["err_prev"][t] + r[t] * (np.abs(f["prev"][t]) + np.abs(x[t])))
                out["dx"][t], out["err_dx"][t] = q[t] * Dt, q[t] * (e + np.abs(Dt))
            out["dgate"][t] = Dt * u
            out["err_dgate"][t] = np.abs(Dt) * eu + e * np.abs(u) + np.abs(Dt * u)
            c = a[t] * Dt
            e = a[t] * (e + r[t] * m)
            m = a[t] * m
        out["dh0"][n], out["err_dh0"][n] = c, e
    return out


def decode_paged(x, gate, kind, cu, pool, slots):
    """Returns (y [T, D], {slot: final state}, err [T, D], {slot: err}); rows of padded sequences are NaN."""
    x = np.asarray(x, dtype=np.float64)
    y, err, final, err_final = np.full(x.shape, np.nan), np.zeros(x.shape), {}, {}
    for n, s in enumerate(int(v) for v in slots):
        if s < 0:
            continue
        t0, t1 = int(cu[n]), int(cu[n + 1])
        f = scan(x[t0:t1], gate[t0:t1], kind, [0, t1 - t0], np.asarray(pool[s], dtype=np.float64)[None])
        y[t0:t1], err[t0:t1] = f["y"], f["err"]
        final[s], err_final[s] = f["final"][0], f["err_final"][0]
    return y, final, err, err_final
