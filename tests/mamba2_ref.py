"""Plain 64-bit forms of the Mamba-2 layer's convolution and single-token step
(numpy), each with a bound on how far fp32 arithmetic may be from it.

The bounds are running error analyses in units of U = 2^-24 (half a step of
fp32, relative).  A sum of n products, whatever its order, is off by at most
(n + 1) U of the sum of their magnitudes.  The hardware's exp2, log2 and
reciprocal are within one step (2 U): a sigmoid of a z that is off by e is off
by at most e/4 + (2 |z| + 6) U sigma, silu by 1.1 e + (2 |z| + 8) U |silu|, and
silu' (whose derivative is at most 1/2) by e/2 + (2 |z| + 10) (1 + |z|) U sigma."""
import numpy as np

U = 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -126


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def softplus(z):
    return np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))


def bounds_of(shape, cu):
    """(batch row, first token, token after the last, which sequence)."""
    if cu is None:
        return [(b, 0, shape[1], b) for b in range(shape[0])]
    return [(0, int(cu[k]), int(cu[k + 1]), k) for k in range(len(cu) - 1)]


def token_conv(x, w, b, silu=True, state=None, cu=None, dout=None, dstate=None):
    """({name: value}, {name: bound}): out and the state left, and with dout (or
    dstate) the gradients.  Arrays are (batch, L, D), or (tokens, D) with cu."""
    packed = cu is not None
    lift = lambda t: np.asarray(t, np.float64)[None] if packed else np.asarray(t, np.float64)  # noqa: E731
    x, w, (D, K) = lift(x), np.asarray(w, np.float64), np.shape(w)
    b = np.zeros(D) if b is None else np.asarray(b, np.float64)
    seqs = bounds_of(x.shape, cu)
    n = len(seqs)
    grad = dout is not None or dstate is not None
    val = dict(out=np.zeros_like(x), state=np.zeros((n, D, K)))
    bnd = dict(out=np.zeros_like(x), state=np.zeros((n, D, K)))
    if grad:
        dout = np.zeros_like(x) if dout is None else lift(dout)
        for d in (val, bnd):
            d.update(dx=np.zeros_like(x), dweight=np.zeros((D, K)), dbias=np.zeros(D), dstate_in=np.zeros((n, D, K)))
        mag_w, mag_b = np.zeros((D, K)), np.zeros(D)
    for r, lo, hi, k in seqs:
        L = hi - lo
        held = np.zeros((K, D)) if state is None else np.asarray(state, np.float64)[k].T
        row = np.concatenate((held, x[r, lo:hi]))
        val["state"][k] = row[L:].T
        taps = np.stack([row[1 + j:1 + j + L] for j in range(K)], -1)   # (L, D, K)
        pre = b + (taps * w).sum(-1)
        mag = np.abs(b) + np.abs(taps * w).sum(-1)
        ep = (K + 2) * U * mag
        s = sigmoid(pre)
        val["out"][r, lo:hi] = pre * s if silu else pre
        bnd["out"][r, lo:hi] = 1.1 * ep + (2 * np.abs(pre) + 8) * U * np.abs(pre * s) if silu else ep
        if not grad:
            continue
        d = dout[r, lo:hi]
        f = s * (1 + pre * (1 - s)) if silu else np.ones_like(pre)
        ef = ep / 2 + (2 * np.abs(pre) + 10) * (1 + np.abs(pre)) * U * s if silu else np.zeros_like(pre)
        e, ee = d * f, np.abs(d) * ef + U * np.abs(d * f)
        back, eback, mback = (np.zeros_like(row) for _ in range(3))
        for j in range(K):
            back[1 + j:1 + j + L] += e * w[:, j]
            eback[1 + j:1 + j + L] += ee * np.abs(w[:, j])
            mback[1 + j:1 + j + L] += np.abs(e * w[:, j])
        if dstate is not None:
            up = np.asarray(dstate, np.float64)[k].T
            back[L:] += up
            mback[L:] += np.abs(up)
        eback += (K + 2) * U * mback
        val["dx"][r, lo:hi], bnd["dx"][r, lo:hi] = back[K:], eback[K:]
        val["dstate_in"][k], bnd["dstate_in"][k] = back[:K].T, eback[:K].T
        val["dweight"] += (e[..., None] * taps).sum(0)
        val["dbias"] += e.sum(0)
        bnd["dweight"] += (ee[..., None] * np.abs(taps)).sum(0)
        bnd["dbias"] += ee.sum(0)
        mag_w += np.abs(e[..., None] * taps).sum(0)
        mag_b += np.abs(e).sum(0)
    if grad:
        # runs of up to 32 tokens in order, 16 runs in a tree, groups of 512 tokens in 4 strands
        terms = 32 + 8 + x.shape[0] * (x.shape[1] // 128 + 1) / 4 + 4
        bnd["dweight"] += terms * U * mag_w
        bnd["dbias"] += terms * U * mag_b
    if packed:
        for d in (val, bnd):
            for key in ("out", "dx"):
                if key in d:
                    d[key] = d[key][0]
    return val, bnd


def conv_step(state, x, w, b, silu=True, slots=None):
    """(out, its bound, the pool afterwards); rows of the batch one after the other."""
    state, x, w = np.array(state, np.float64), np.asarray(x, np.float64), np.asarray(w, np.float64)
    out, bnd = np.zeros_like(x), np.zeros_like(x)
    K = w.shape[1]
    for r in range(x.shape[0]):
        k = r if slots is None else int(slots[r])
        if not 0 <= k < state.shape[0]:
            continue
        state[k] = np.concatenate((state[k][:, 1:], x[r][:, None]), 1)
        pre = (state[k] * w).sum(-1) + (0 if b is None else b)
        ep = (K + 2) * U * (np.abs(state[k] * w).sum(-1) + (0 if b is None else np.abs(b)))
        s = sigmoid(pre)
        out[r] = pre * s if silu else pre
        bnd[r] = 1.1 * ep + (2 * np.abs(pre) + 8) * U * np.abs(pre * s) if silu else ep
    return out, bnd, state


def step_parts(dt, bias, A, softplus_on=True):
    """Step size, decay, and their relative errors, softplus being within 3 U of
    its value where its argument is exact."""
    pre = dt + (0 if bias is None else bias)
    delta = softplus(pre) if softplus_on else pre
    slope = sigmoid(pre) if softplus_on else np.ones_like(pre)
    with np.errstate(divide="ignore", invalid="ignore"):
        ed = np.where(delta != 0, slope * U * np.abs(pre) / np.abs(delta), 0) + (3 * U if softplus_on else 0)
    z = delta * A
    return delta, np.exp(z), ed, np.abs(z) * (ed + 3 * U) + 2 * U


def ssd_step(state, x, dt, A, B, C, D=None, z=None, bias=None, softplus_on=True, slots=None):
    """(out, its bound, the pool afterwards, its bound): (batch, H, P) inputs,
    (batch, G, N) B and C, one row after the other."""
    state, x, dt, A, B, C = (np.array(t, np.float64) for t in (state, x, dt, A, B, C))
    es = np.zeros_like(state)
    H, G, N = x.shape[1], B.shape[1], B.shape[2]
    B, C = np.repeat(B, H // G, 1), np.repeat(C, H // G, 1)
    out, bnd = np.zeros_like(x), np.zeros_like(x)
    for r in range(x.shape[0]):
        k = r if slots is None else int(slots[r])
        if not 0 <= k < state.shape[0]:
            continue
        delta, a, ed, ea = step_parts(dt[r], bias, A, softplus_on)
        col = lambda t: t[:, None, None]  # noqa: E731
        old = col(a) * state[k]
        new = col(delta) * x[r][..., None] * B[r][:, None]
        es[k] = col(a) * es[k] + np.abs(old) * (col(ea) + U) + np.abs(new) * (col(ed) + 3 * U)
        state[k] = old + new
        es[k] += U * np.abs(state[k]) + TINY
        y = (state[k] * C[r][:, None]).sum(-1)
        ey = (es[k] * np.abs(C[r][:, None])).sum(-1) + (N + 2) * U * np.abs(state[k] * C[r][:, None]).sum(-1)
        if D is not None:
            y = y + D[:, None] * x[r]
            ey = ey + 2 * U * (np.abs(D[:, None] * x[r]) + np.abs(y))
        if z is not None:
            g = z[r] * sigmoid(z[r])
            ey = ey * np.abs(g) + np.abs(y * g) * (2 * np.abs(z[r]) + 9) * U
            y = y * g
        out[r], bnd[r] = y, ey
    return out, bnd, state, es


CHUNK = 64   # tokens of the kernels' chunks, from each sequence's first on


def ssd_scan(x, dt, A, B, C, D=None, z=None, bias=None, softplus_on=True, h0=None, cu=None, dout=None, dlast=None, io="f32",
             sharp=False):
    """({name: value}, {name: bound}) of the Mamba-2 SSM over whole sequences and,
    with dout, of its gradients, token by token.  Arrays are (batch, L, H, P) and
    so on, or without the batch axis with cu.

    The bounds are multiples of the same sums taken over magnitudes (names that
    end in m).  With a the sums of A Delta in a chunk, at most a_max in size: a
    decay e^(a_t - a_s) is off by (20 a_max + 6) U (a prefix sum of 64 steps in six
    levels, its product with A log2 e, the difference, exp2); products of N, P
    and 64 terms, and a carry over the chunks with two roundings each, add
    (N + P + 64 + 4 chunks + 60) U: together e.  For bf16 IO an operand in two
    halves is off by 2^-16 of its size, two of them in a row by 2^-15; a rounded
    operand by 2^-8: the weighted scores (out, dx, dB, dC), the state in dx, and a
    gated dout in dx, dB and dC.  The flow through a step's decay is a difference
    of prefix sums over its chunk: 20 U of all that they sum.

    sharp: bounds that large steps elsewhere in a chunk leave as they are.  A term
    whose decay is e^-E is off by E (2 U + the steps' own relative error) of itself,
    whatever the other steps of the chunk: its exponent is rounded once, and again
    where a chunk ends (sums that carry E along end in x below).  The flow through a
    step is then a sum of terms which cross that step, and off by e of those alone."""
    packed = cu is not None
    lift = lambda t: None if t is None else (np.asarray(t, np.float64)[None] if packed else np.asarray(t, np.float64))  # noqa: E731
    x, dt, B, C, z, dout = (lift(t) for t in (x, dt, B, C, z, dout))
    A = np.asarray(A, np.float64)
    seqs = bounds_of(x.shape, cu)
    n, (H, P), (G, N) = len(seqs), x.shape[2:], B.shape[2:]
    each = H // G
    zero = lambda *s: np.zeros(s)  # noqa: E731
    names = dict(out=x.shape, last=(n, H, P, N))
    if dout is not None:
        names.update(dx=x.shape, ddt=dt.shape, dB=B.shape, dC=C.shape, dA=(H,), ddt_bias=(H,), dD=(H,), dh0=(n, H, P, N), dz=x.shape)
    val, bnd = ({k: zero(*s) for k, s in names.items()} for _ in range(2))
    half = 2.0 ** -8 if io == "bf16" else 0.0
    split = 2.0 ** -15 if io == "bf16" else 0.0
    Dh = np.zeros(H) if D is None else np.asarray(D, np.float64)
    col = lambda t: t[:, None]  # noqa: E731
    tokens = x.shape[0] * x.shape[1]
    for r, lo, hi, k in seqs:
        L = hi - lo
        h = zero(H, P, N) if h0 is None else np.asarray(h0, np.float64)[k]
        hm = np.abs(h)
        hx = np.zeros_like(h)
        delta, alpha, ed, _ = step_parts(dt[r, lo:hi], bias, A, softplus_on)
        amax = max((np.abs(A * delta[c:c + CHUNK].sum(0)).max() for c in range(0, L, CHUNK)), default=0)
        e = ((0 if sharp else 20 * amax) + 6 + N + P + 64 + 4 * (L // CHUNK + 1) + 60) * U + (ed.max() if L else 0)
        ex = 2 * U + ed.max() if sharp and L else 0.0
        rate = (np.abs(A * delta) if sharp else zero(L, H))[..., None, None]       # (L, H, 1, 1)
        Br, Cr = (np.repeat(t[r, lo:hi], each, 1)[:, :, None] for t in (B, C))      # (L, H, 1, N)
        xr = x[r, lo:hi][..., None]                                                # (L, H, P, 1)
        hs, hms, hxs, y, ym, yx = [h], [hm], [hx], zero(L, H, P), zero(L, H, P), zero(L, H, P)
        for t in range(L):
            add = delta[t][:, None, None] * xr[t] * Br[t]
            h = alpha[t][:, None, None] * h + add
            hx = alpha[t][:, None, None] * (hx + rate[t] * hm)
            hm = alpha[t][:, None, None] * hm + np.abs(add)
            hs.append(h)
            hms.append(hm)
            hxs.append(hx)
            yx[t] = (hx * np.abs(Cr[t])).sum(-1)
            y[t], ym[t] = (h * Cr[t]).sum(-1), (hm * np.abs(Cr[t])).sum(-1)
        val["last"][k], bnd["last"][k] = h, (e + split) * hm + ex * hx
        full = y + col(Dh) * x[r, lo:hi]
        efull = (e + split + half) * ym + ex * yx + 3 * U * (np.abs(col(Dh) * x[r, lo:hi]) + ym)
        s = None if z is None else sigmoid(z[r, lo:hi])
        gate = 1.0 if z is None else z[r, lo:hi] * s
        eg = 0.0 if z is None else (2 * np.abs(z[r, lo:hi]) + 9) * U
        val["out"][r, lo:hi] = full * gate
        bnd["out"][r, lo:hi] = efull * np.abs(gate) + np.abs(full * gate) * eg
        if dout is None:
            continue
        d = dout[r, lo:hi]
        if z is not None:
            f = s * (1 + z[r, lo:hi] * (1 - s))
            ef = (2 * np.abs(z[r, lo:hi]) + 11) * (1 + np.abs(z[r, lo:hi])) * U * s
            val["dz"][r, lo:hi] = d * full * f
            bnd["dz"][r, lo:hi] = np.abs(d) * (efull * np.abs(f) + np.abs(full) * ef) + 2 * U * np.abs(d * full * f)
        gated = half if z is not None else 0.0
        es = e + (np.max(eg) if np.size(eg) else 0) + (2 * split if z is not None else split)   # of sums that carry 16 bits
        dy = d * gate
        dh = zero(H, P, N) if dlast is None else np.asarray(dlast, np.float64)[k]
        dhm = np.abs(dh)
        dhx, flowx, toxx = np.zeros_like(dh), zero(L, H), zero(L, H)
        flow, flowm, tox, toxm, terms = (zero(L, H) for _ in range(5))
        ends = {}
        for t in range(L - 1, -1, -1):
            if t == L - 1 or (t + 1) % CHUNK == 0:
                ends[t // CHUNK] = (dhm * hms[t + 1]).sum((-1, -2))
            m = np.abs(dy[t])
            dC = (dy[t][..., None] * hs[t + 1]).sum(1)
            dCm = (m[..., None] * hms[t + 1]).sum(1)
            dh = dh + dy[t][..., None] * Cr[t]
            dhm = dhm + m[..., None] * np.abs(Cr[t])
            dCx = (m[..., None] * hxs[t + 1]).sum(1)
            to_x, to_xm, to_xx = (dh * Br[t]).sum(-1), (dhm * np.abs(Br[t])).sum(-1), (dhx * np.abs(Br[t])).sum(-1)
            dBx = col(delta[t]) * (dhx * np.abs(xr[t])).sum(1)
            dB = col(delta[t]) * (dh * xr[t]).sum(1)
            dBm = col(delta[t]) * (dhm * np.abs(xr[t])).sum(1)
            flow[t] = (dh * hs[t]).sum((-1, -2)) * alpha[t]
            flowm[t] = (dhm * hms[t]).sum((-1, -2)) * alpha[t]
            flowx[t] = (dhx * hms[t] + dhm * hxs[t] + rate[t] * dhm * hms[t]).sum((-1, -2)) * alpha[t]
            toxx[t] = (to_xx * np.abs(x[r, lo + t])).sum(-1)
            tox[t], toxm[t] = (to_x * x[r, lo + t]).sum(-1), (to_xm * np.abs(x[r, lo + t])).sum(-1)
            terms[t] = delta[t] * toxm[t] + (m * ym[t]).sum(-1)
            val["dx"][r, lo + t] = col(delta[t]) * to_x + col(Dh) * dy[t]
            bnd["dx"][r, lo + t] = (es + 2 * half + gated) * col(delta[t]) * to_xm + (gated + es) * np.abs(col(Dh) * dy[t]) + \
                ex * col(delta[t]) * to_xx
            for which, v, vm, vx in (("dB", dB, dBm, dBx), ("dC", dC, dCm, dCx)):
                val[which][r, lo + t] = v.reshape(G, each, N).sum(1)
                bnd[which][r, lo + t] = ((es + half + gated + each * U) * vm + ex * vx).reshape(G, each, N).sum(1)
            dhx = alpha[t][:, None, None] * (dhx + rate[t] * dhm)
            dh, dhm = alpha[t][:, None, None] * dh, alpha[t][:, None, None] * dhm
        total = np.stack([terms[c:c + CHUNK].sum(0) + ends[c // CHUNK] for c in range(0, L, CHUNK)]) if L else zero(0, H)
        eflow = es * flowm + (ex * flowx if sharp else 20 * U * np.repeat(total, CHUNK, 0)[:L])
        slope = sigmoid(dt[r, lo:hi] + (0 if bias is None else bias)) if softplus_on else np.ones((L, H))
        dd = tox + A * flow
        edd = es * toxm + ex * toxx + np.abs(A) * eflow + 3 * U * (toxm + np.abs(A) * flowm)
        val["ddt"][r, lo:hi] = dd * slope
        pre = np.abs(dt[r, lo:hi] + (0 if bias is None else bias))
        pre = np.where(slope > 0, pre, 0)   # no step at all: nothing to be off
        bnd["ddt"][r, lo:hi] = edd * slope + np.abs(dd) * slope * (2 * pre + 8) * U
        val["dh0"][k], bnd["dh0"][k] = dh, es * dhm + ex * dhx
        val["dA"] += (delta * flow).sum(0)
        bnd["dA"] += (delta * (eflow + (ed + U * (tokens / 64 + 70)) * flowm)).sum(0)
        val["ddt_bias"] += (dd * slope).sum(0)
        bnd["ddt_bias"] += (bnd["ddt"][r, lo:hi] + U * (tokens / 64 + 70) * np.abs(dd * slope)).sum(0)
        val["dD"] += (dy * x[r, lo:hi]).sum((0, 2))
        bnd["dD"] += ((es + U * (P + tokens / 64 + 70)) * np.abs(dy * x[r, lo:hi])).sum((0, 2))
    if packed:
        for q in (val, bnd):
            for key in ("out", "dx", "ddt", "dB", "dC", "dz"):
                if key in q:
                    q[key] = q[key][0]
    return val, bnd
