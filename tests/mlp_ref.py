"""Plain 64-bit forms of the operators between a gated MLP's GEMMs, and the
check of E4M3 codes against the real value that they stand for.

A quantised result is checked in two steps that hold for any summation order:
the scale must be the group's largest magnitude / 448 within the error of the
FP32 values (`err`, absolute, per element), and each code must be a nearest
E4M3 value of ref / scale: |code * scale - ref| is at most half the spacing of
E4M3 at that point times the scale, plus `err`."""
import numpy as np

GROUP = 128
U24 = 2.0 ** -24


def e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = -v if c & 128 else v
    t[0x7F] = t[0xFF] = np.nan
    return t


DECODE = e4m3_table()


def half_step(v):
    """Half the distance between neighbouring E4M3 values around |v|."""
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -6))
    return np.ldexp(1.0, e - 5)


def check_codes(codes, scales, ref, err, pow2=False, what=""):
    """codes uint8 [rows, cols] and scales [rows, cols/128] against ref in 64 bits."""
    rows, cols = ref.shape
    g = np.abs(ref).reshape(rows, cols // GROUP, GROUP)
    amax, eg = g.max(2), np.broadcast_to(err, ref.shape).reshape(g.shape).max(2)
    s = np.asarray(scales, np.float64)
    assert np.all(np.isfinite(s)) and np.all(s > 0), what
    if pow2:
        # the smallest power of two with amax <= 448 s, for some amax within the error
        assert np.all(np.frexp(s)[0] == 0.5), what
        live = amax > eg
        assert np.all((amax - eg <= 448 * s)[live]), what
        assert np.all((amax + eg > 224 * s)[live & (s > 2.0 ** -126)]), what
    else:
        # (a group that is zero up to the error may take scale 1 or a tiny one)
        off = np.abs(s * 448 - amax)
        bad = (off > eg + 4 * U24 * amax) & ~((amax <= eg) & (s == 1.0))
        assert not bad.any(), "%s: scale off by %g of %g" % (what, off[bad][0], amax[bad][0])
    sv = np.repeat(s, GROUP, 1)
    v = DECODE[codes]
    assert not np.isnan(v).any(), what
    t = ref / sv
    tol = half_step(np.maximum(np.abs(t), np.abs(v))) * (1 + 1e-6) + err / sv + 4 * U24 * np.abs(t)
    bad = np.abs(v - t) > tol
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d codes are not a nearest value; first at %s: code value %r, real value %r" %
                             (what, int(bad.sum()), i, v[i], t[i]))


def rms(h, eps):
    return 1.0 / np.sqrt((h * h).mean(1) + eps)


def norm_y(h, gamma, eps):
    return h * rms(h, eps)[:, None] * gamma


def norm_bwd(dy, h, rstd, gamma):
    """(dx, dgamma, bounds of the sums' terms for dx and dgamma)"""
    D = h.shape[1]
    r = rstd[:, None]
    a = dy * gamma
    dx = r * (a - h * r * r * (a * h).sum(1, keepdims=True) / D)
    tx = r * (np.abs(a) + np.abs(h) * r * r * np.abs(a * h).sum(1, keepdims=True) / D)
    terms = dy * h * r
    return dx, terms.sum(0), tx, np.abs(terms).sum(0)


def sigmoid(v):
    return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def gate(g, u):
    return g * sigmoid(g) * u


def gate_bwd(g, u, dh):
    sg = sigmoid(g)
    a = g * sg
    return dh * u * (sg + a * sigmoid(-g)), dh * a, a * u


def sigmoid_err(g):
    """Absolute error of an FP32 sigmoid made from an exponential good to 2 ulp
    plus |g| 2^-24 relative, an addition and a quotient good to 2 ulp."""
    sg = sigmoid(g)
    return sg * ((1 - sg) * (4 + np.abs(g)) * 2 * U24 + 6 * U24)
