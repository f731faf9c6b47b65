"""Plain 64-bit forms of the gated recurrence and of the quantised state cache
(numpy, token by token and block by block), each with a bound on how far fp32
arithmetic may be from it.

The bounds are running error analyses, in units of U = 2^-24 (half a step of
fp32, relative): the hardware's exp2, log2, reciprocal and square root are
within one step (2 U).  sigma(z): the exponent's argument z log2(e) is off by
2 |z| U absolutely, so sigma by (2 |z| + 6) U relative; v = s sigma(z) with s
from a softplus good to 6 U: (2 |z| + 12) U; a = e^-v: (v (2 |z| + 14) + 2) U;
beta: the series and the square root add at most 12 U to half of v's error.
Every sum or product adds U of its result.
The hardware's exp2 gives 0 for what is below TINY = 2^-126, the least normal
fp32 number, so a decay a is also off by up to TINY absolutely, and a h by
TINY |h|.  A scan in tiles multiplies and adds
in another order, which at most doubles what the chain of steps collects."""
import numpy as np

U = 2.0 ** -24
TINY = 2.0 ** -126
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
BLOCK = 32


def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def _softplus(z):
    return np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))


def bounds_of(shape, cu):
    """(batch row, first token, token after the last, which sequence)."""
    if cu is None:
        return [(b, 0, shape[1], b) for b in range(shape[0])]
    return [(0, int(cu[k]), int(cu[k + 1]), k) for k in range(len(cu) - 1)]


def _token_parts(x, ga, gx, lam, c):
    s = c * _softplus(lam)
    sa, g = _sigmoid(ga), _sigmoid(gx)
    v = s * sa
    a = np.exp(-v)
    beta = np.sqrt(-np.expm1(-2 * v))
    za, zx = (np.where(np.isfinite(z), np.abs(z), 0) for z in (ga, gx))
    ea = (v * (2 * za + 14) + 2) * U                       # relative errors
    eb = (za + 24 + 2 * zx) * U
    return a, v, beta, sa, g, ea, eb


def gated_scan(x, ga, gx, lam, c=8.0, h0=None, cu=None, dout=None, dlast=None):
    """Forward, and with dout (or dlast) the gradients, in 64 bits.  Arrays are
    (batch, L, dim), or (tokens, dim) with cu.  Returns ({name: value},
    {name: bound}); rows of tokens in no sequence are zero."""
    packed = cu is not None
    x, ga, gx = (np.asarray(t, np.float64)[None] if packed else np.asarray(t, np.float64) for t in (x, ga, gx))
    lam = np.asarray(lam, np.float64)
    B, L, D = x.shape
    seqs = bounds_of(x.shape, cu)
    n = len(seqs) if packed else B
    h0v = np.zeros((n, D)) if h0 is None else np.asarray(h0, np.float64)
    a, v, beta, sa, g, ea, eb = _token_parts(x, ga, gx, lam, c)
    b = beta * g * x
    h, eh, prev, eprev = (np.zeros((B, L, D)) for _ in range(4))
    last, elast = h0v.copy(), np.zeros((n, D))
    for row, lo, hi, k in seqs:
        st, er = h0v[k].copy(), np.zeros(D)
        for t in range(lo, hi):
            prev[row, t], eprev[row, t] = st, er
            new = a[row, t] * st + b[row, t]
            er = a[row, t] * er + TINY * np.abs(st) + 2 * (np.abs(a[row, t] * st) * ea[row, t] + np.abs(b[row, t]) * eb[row, t]
                                                           + U * (np.abs(new) + np.abs(a[row, t] * st)))
            st = new
            h[row, t], eh[row, t] = st, er
        last[k], elast[k] = st, er
    val, bnd = dict(out=h, last=last), dict(out=eh, last=elast)
    if dout is not None:
        dout = np.asarray(dout, np.float64)[None] if packed else np.asarray(dout, np.float64)
        e, ee = np.zeros((B, L, D)), np.zeros((B, L, D))
        dh0, edh0 = np.zeros((n, D)), np.zeros((n, D))
        for row, lo, hi, k in seqs:
            carry = np.zeros(D) if dlast is None else np.asarray(dlast, np.float64)[k].copy()
            ec = np.zeros(D)
            for t in range(hi - 1, lo - 1, -1):
                e[row, t] = dout[row, t] + carry
                ee[row, t] = ec + 2 * U * (np.abs(e[row, t]) + np.abs(carry))
                carry = a[row, t] * e[row, t]
                ec = a[row, t] * ee[row, t] + TINY * np.abs(e[row, t]) + 2 * np.abs(carry) * (ea[row, t] + U)
            dh0[k], edh0[k] = carry, ec
        dx = e * beta * g
        edx = ee * beta * g + np.abs(dx) * (eb + 4 * U)
        q = np.where(beta > 0, a * a / np.where(beta > 0, beta, 1), 0)
        p1, p2 = g * x * q, a * prev
        dv = e * (p1 - p2)
        edv = ee * np.abs(p1 - p2) + np.abs(e) * (np.abs(p1) * (eb + 2 * ea + 8 * U) + np.abs(p2) * (ea + 4 * U)
                                                  + a * eprev)
        za = np.where(np.isfinite(ga), np.abs(ga), 0)
        zx = np.where(np.isfinite(gx), np.abs(gx), 0)
        # 1 - sigma from sigma's rounding: absolute error 2 U next to its own relative one
        dgx = dx * x * (1 - g)
        edgx = edx * np.abs(x) * (1 - g) + np.abs(dx * x) * ((2 * zx + 10) * g + 4) * U
        dga = dv * v * (1 - sa)
        edga = edv * v * (1 - sa) + np.abs(dv * v) * (((2 * za + 10) * sa + 4) + (2 * za + 16) * (1 - sa)) * U
        inside = np.zeros((B, L, 1))
        for row, lo, hi, k in seqs:
            inside[row, lo:hi] = 1
        sl = _sigmoid(lam)
        summed, esum = (dv * sa * inside).sum((0, 1)), (edv * sa * inside).sum((0, 1))
        size = (np.abs(dv) * sa * inside).sum((0, 1))
        count = max(1, int(inside.sum()))
        val.update(dx=dx * inside, dgate_a=dga * inside, dgate_x=dgx * inside, dlam=c * sl * summed, dh0=dh0)
        # a sum of `count` terms in any order: at most count U of the sum of magnitudes
        bnd.update(dx=edx, dgate_a=edga, dgate_x=edgx, dh0=edh0,
                   dlam=c * sl * (esum + size * (count + 2 * np.abs(lam) + 16) * U))
    if packed:
        for k in ("out", "dx", "dgate_a", "dgate_x"):
            if k in val:
                val[k], bnd[k] = val[k][0], bnd[k][0]
    return val, bnd


# -- the cache ------------------------------------------------------------------------------------------------------

MOST = {"int8": 127.0, "fp8": 448.0, "fp4": 6.0}


def scale_exponent(block, fmt):
    """Least e >= -127 with max |block| <= MOST 2^e, by trying."""
    amax = float(np.max(np.abs(block), initial=0.0))
    e = -127
    while amax > MOST[fmt] * 2.0 ** e:
        e += 1
    return e


def grid(fmt):
    """The values of a format's codes 0, 1, ... with the sign bit clear."""
    if fmt == "fp4":
        return np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    return np.array([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)][:127])


def encode(values, fmt):
    """Codes (uint8, one a value) and scale bytes of (..., n) float values."""
    values = np.asarray(values, np.float64)
    n = values.shape[-1]
    codes = np.zeros(values.shape, np.uint8)
    scales = np.zeros(values.shape[:-1] + (-(-n // BLOCK),), np.uint8)
    for idx in np.ndindex(scales.shape):
        sl = idx[:-1] + (slice(idx[-1] * BLOCK, min(n, (idx[-1] + 1) * BLOCK)),)
        block = values[sl]
        if not np.all(np.isfinite(block)):
            scales[idx] = 255
            continue
        e = scale_exponent(block, fmt)
        scales[idx] = e + 127
        w = block / 2.0 ** e
        if fmt == "int8":
            codes[sl] = np.rint(w).astype(np.int8).view(np.uint8)
        else:
            gr = grid(fmt)
            up = np.clip(np.searchsorted(gr, np.abs(w)), 1, len(gr) - 1)
            lo, hi = gr[up - 1], gr[up]
            mid = (lo + hi) / 2
            take = np.where(np.abs(w) > mid, up, np.where(np.abs(w) < mid, up - 1, np.where(up % 2 == 0, up, up - 1)))
            codes[sl] = take + np.where(np.signbit(w), 128 if fmt == "fp8" else 8, 0)
    return codes, scales


def decode(codes, scales, fmt):
    codes = np.asarray(codes)
    if fmt == "int8":
        q = codes.view(np.int8).astype(np.float64)
    else:
        sign = 128 if fmt == "fp8" else 8
        q = grid(fmt)[np.minimum(codes & (sign - 1), len(grid(fmt)) - 1)] * np.where(codes & sign, -1.0, 1.0)
    unit = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return q * np.repeat(unit, BLOCK, -1)[..., :codes.shape[-1]]


def pack4(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack4(held):
    return np.stack((held & 15, held >> 4), -1).reshape(held.shape[:-1] + (-1,))


def philox_bytes(seed, channel, row, n):
    """The byte for each of n states of a channel: Philox-4x32, 7 rounds, with
    Python's whole numbers."""
    out = []
    for block in range(-(-n // 16)):
        c = [channel, row, block, 0]
        k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(7):
            p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
            c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
            k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
        out += [(w >> (8 * j)) & 255 for w in c for j in range(4)]
    return np.array(out[:n])


def decode_step(state, x, dt, A, B, C, D=None, z=None, bias=None, softplus=True):
    """One selective-scan step in 64 bits on (rows, dim, N) states: (out, new
    state, bound on the state, bound on out)."""
    f = lambda t: np.asarray(t, np.float64)  # noqa: E731
    state, x, dt, A, B, C = (f(t) for t in (state, x, dt, A, B, C))
    dl = dt + (0 if bias is None else f(bias))
    zdl = np.abs(dl)
    if softplus:
        dl = _softplus(dl)
    cpg = x.shape[1] // (B.shape[1] if B.ndim == 3 else 1)
    Bf, Cf = (np.repeat(t, cpg, 1) if t.ndim == 3 else t[:, None] for t in (B, C))
    # Delta: 8 U relative and the bias' sum; the decay's argument Delta A by 4 U more
    edl = 8 + np.where(dl > 0, zdl / np.where(dl > 0, dl, 1), 0) * (0 if softplus else 1) + 2 * zdl * softplus
    arg = dl[..., None] * A
    new = np.exp(arg) * state + (dl * x)[..., None] * Bf
    eh = (np.abs(np.exp(arg) * state) * (np.abs(arg) * (edl[..., None] + 4) + 4)
          + np.abs((dl * x)[..., None] * Bf) * (edl[..., None] + 4) + np.abs(new)) * U
    y = (new * Cf).sum(-1) + (0 if D is None else f(D) * x)
    ey = (eh * np.abs(Cf)).sum(-1) + (np.abs(new * Cf).sum(-1) + (0 if D is None else np.abs(f(D) * x))) * (A.shape[1] + 2) * U
    if z is not None:
        gate = f(z) * _sigmoid(f(z))
        ey = ey * np.abs(gate) + np.abs(y * gate) * (2 * np.abs(f(z)) + 10) * U
        y = y * gate
    return y, new, eh, ey
