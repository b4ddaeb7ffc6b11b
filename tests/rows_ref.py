"""Plain 64-bit references of the row operators (gated linear recurrence, norms around a block),
each with a bound on what 32-bit arithmetic may be off by.

The bounds are running error bounds: every 32-bit operation of the kernels is within a few units
of 2^-22 (the approximate exponential, reciprocal and root) or 2^-24 (the rest) of its operands'
magnitudes, so the errors follow the recurrence itself, on absolute values. EPS = 2^-22 times a count
of the operations in front of each term, doubled; an output in 16 bits adds half a unit in
its last place."""
import numpy as np

EPS = 2.0 ** -22
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 1e-36, "bf16": 1e-36, "f16": 2.0 ** -24}   # the spacing of a type's subnormals


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def rounded(ref, bound, kind):
    """The allowed distance of an output of a type from ref, given the 32-bit bound."""
    return bound * (1 + HALF_ULP[kind]) + HALF_ULP[kind] * np.abs(ref) + TINY[kind]


class Recurrence:
    """The recurrence over sequences `spans` (start, end) of rows; all arrays float64.

    h, hT and, after backward(), dx, dr, di, dlam, dh0; err[name] bounds each."""

    def __init__(self, x, r, i, lam, kappa, spans, h0=None):
        self.x, self.spans, self.kappa, self.lam = x, spans, kappa, lam
        rows, c = x.shape
        sp = np.maximum(lam, 0) + np.log1p(np.exp(-np.abs(lam)))
        self.rate = kappa * sp
        with np.errstate(divide="ignore", invalid="ignore"):
            slope = sigmoid(lam) / sp
        self.slope = np.where(lam < -30, 1.0, slope)
        self.sr, self.si = sigmoid(r), sigmoid(i)
        self.cr, self.ci = sigmoid(-r), sigmoid(-i)
        self.l = -self.rate * self.sr
        self.a = np.exp(self.l)
        self.s = np.sqrt(-np.expm1(2 * self.l))
        self.u = self.s * self.si * x
        # relative error of sigma: the exponential of a rounded argument, then about four
        # operations; that of l one more
        self.e_r = EPS * (8 + 2 * np.minimum(np.abs(r), 90.0))
        self.e_i = EPS * (8 + 2 * np.minimum(np.abs(i), 90.0))
        # a: one rounding of a number up to 1, and l's relative error times |l| a
        self.e_a = EPS * (1 + 4 * self.a) + (self.e_r + 4 * EPS) * np.abs(self.l) * self.a
        e_s = 0.5 * (self.e_r + 16 * EPS) + 4 * EPS
        self.e_u = e_s + self.e_i + 4 * EPS          # relative
        # a sigma below 2^-60 is not kept apart from 0: what that shifts the root by, absolute
        self.floor = np.sqrt(2 * np.minimum(self.rate, 1e30) * 2.0 ** -59) + 2.0 ** -40
        self.e_abs = self.floor * (self.si + 2.0 ** -59) * np.abs(x) + 2.0 ** -59 * self.s * np.abs(x)
        batch = len(spans)
        self.h0 = np.zeros((batch, c)) if h0 is None else h0
        self.h, self.before = np.zeros((rows, c)), np.zeros((rows, c))
        self.hT = self.h0.copy()
        self.big, self.err = np.zeros((rows, c)), {"h": np.zeros((rows, c)),
                                                   "hT": np.zeros((batch, c))}
        self.big_before, self.err_before = np.zeros((rows, c)), np.zeros((rows, c))
        for b, (p, q) in enumerate(spans):
            h, big, err = self.h0[b], np.abs(self.h0[b]), np.zeros(c)
            for t in range(p, q):
                self.before[t], self.big_before[t], self.err_before[t] = h, big, err
                h = self.a[t] * h + self.u[t]
                err = self.a[t] * err + self.e_a[t] * big + self.e_u[t] * np.abs(self.u[t]) + self.e_abs[t]
                big = self.a[t] * big + np.abs(self.u[t])
                err = err + 2 * EPS * big
                self.h[t], self.big[t], self.err["h"][t] = h, big, err
            self.hT[b], self.err["hT"][b] = h, err

    def backward(self, dh, dhT=None):
        rows, c = self.x.shape
        g, G, E = np.zeros((rows, c)), np.zeros((rows, c)), np.zeros((rows, c))
        self.dh0 = np.zeros_like(self.h0) if dhT is None else dhT.copy()
        self.err["dh0"] = np.zeros_like(self.h0)
        for b, (p, q) in enumerate(self.spans):
            carry = self.dh0[b]
            big, err = np.abs(carry), np.zeros(c)
            for t in range(q - 1, p - 1, -1):
                g[t] = dh[t] + carry
                G[t] = np.abs(dh[t]) + big
                E[t] = err + 2 * EPS * G[t]
                carry = self.a[t] * g[t]
                err = self.a[t] * E[t] + self.e_a[t] * G[t] + EPS * self.a[t] * G[t]
                big = self.a[t] * G[t]
            self.dh0[b], self.err["dh0"][b] = carry, err
        xa = np.abs(self.x)
        with np.errstate(divide="ignore", invalid="ignore"):
            ratio = np.where(self.s > 0, self.l / self.s, 0.0)
        self.dx = g * self.s * self.si
        self.err["dx"] = self.s * self.si * (E + G * (self.e_u + 4 * EPS)) + (G + E) * (
            self.floor + 2.0 ** -59)
        self.di = g * self.s * self.x * self.si * self.ci
        self.err["di"] = self.s * self.si * self.ci * xa * (E + G * (self.e_u + self.e_i + 8 * EPS)) \
            + (G + E) * xa * (self.floor * self.si * self.ci + 2.0 ** -59)
        first, second = self.l * self.a * self.before, self.si * self.x * self.a ** 2 * ratio
        d = g * (first - second)
        e1 = np.abs(self.l) * (self.a * self.err_before
                               + (self.e_a + self.a * (self.e_r + 8 * EPS)) * self.big_before)
        e2 = np.abs(second) * (1.5 * self.e_r + self.e_i + 24 * EPS) \
            + 2 * self.si * xa * self.a * np.abs(ratio) * self.e_a \
            + 2 * self.si * xa * self.floor + 2.0 ** -58 * (self.rate * self.big_before + xa)
        size = np.abs(self.l) * self.a * self.big_before + np.abs(second)
        e_d = E * size + G * (e1 + e2 + 4 * EPS * size)
        self.dr = d * self.cr
        self.err["dr"] = self.cr * (e_d + np.abs(d) * (self.e_r + 8 * EPS))
        self.dlam = d.sum(0) * self.slope
        self.err["dlam"] = self.slope * (e_d.sum(0)
                                         + G_sum(np.abs(d), rows)) + 8 * EPS * np.abs(self.dlam)
        return self


def G_sum(mag, rows):
    """Error of adding `rows` 32-bit terms one after another, in any order."""
    return (rows + 8) * 2.0 ** -24 * mag.sum(0)


def gate_ref(z, gate):
    s, c = sigmoid(z), sigmoid(-z)
    if gate == 0:
        return z * s, s * (1 + z * c)
    if gate == 1:
        return s, s * c
    return z, np.ones_like(z)


class Norms:
    """y, u and, after backward(), df, dz, dx, dw_post, dscale, dw_pre; err[name] bounds each.
    Absent parts are None."""

    def __init__(self, f, z=None, x=None, w_post=None, scale=None, w_pre=None, eps=1e-6, gate=0):
        width = f.shape[1]
        self.f, self.z, self.x, self.w_post, self.scale, self.w_pre = f, z, x, w_post, scale, w_pre
        self.gate, one = gate, np.ones(width)
        # a sum of width squares, in any order, to half its relative error
        self.e_sum = (width + 32) * 2.0 ** -25 + 4 * EPS
        self.q1 = 1 / np.sqrt((f * f).mean(1, keepdims=True) + eps)
        self.n = f * self.q1 if w_post is not None else f
        self.nw = self.n * (one if w_post is None else w_post)
        self.act, self.slope = (np.ones_like(f), np.zeros_like(f)) if z is None else gate_ref(z, gate)
        self.e_z = 0.0 if z is None else EPS * (8 + 2 * np.minimum(np.abs(z), 90.0))
        self.c = one if scale is None else scale
        self.t = self.nw * self.act
        base = np.zeros_like(f) if x is None else x
        self.y = base + self.c * self.t
        self.err = {"y": np.abs(self.c * self.t) * (self.e_sum + self.e_z + 8 * EPS)
                    + EPS * np.abs(base)}
        if w_pre is not None:
            self.q2 = 1 / np.sqrt((self.y ** 2).mean(1, keepdims=True) + eps)
            # relative error of 1/rms(y): the entries' errors in the root mean square, and the sum
            self.e_q2 = self.q2 * np.sqrt((self.err["y"] ** 2).mean(1, keepdims=True)) + self.e_sum
            self.u = self.y * self.q2 * w_pre
            self.err["u"] = np.abs(self.q2 * w_pre) * (
                self.err["y"] + np.abs(self.y) * (self.e_q2 + 4 * EPS))

    def backward(self, dy=None, du=None):
        f, c = self.f, self.c
        width, rows = f.shape[1], f.shape[0]
        d = np.zeros_like(f) if dy is None else dy.copy()
        e = EPS * np.abs(d)
        if du is not None:
            m = du * self.w_pre * self.q2
            dot, mag = (m * self.y).mean(1, keepdims=True), (np.abs(m * self.y)).mean(
                1, keepdims=True)
            back = self.y * self.q2 ** 2 * dot
            e_dot = mag * (2 * self.e_sum + 2 * self.e_q2 + 8 * EPS) \
                + (np.abs(m) * self.err["y"]).mean(1, keepdims=True)
            e = e + np.abs(m) * (self.e_q2 + 8 * EPS) + np.abs(self.y) * self.q2 ** 2 * e_dot \
                + mag * self.q2 ** 2 * (self.err["y"] + np.abs(self.y) * (3 * self.e_q2 + 8 * EPS)) \
                + 4 * EPS * (np.abs(d) + np.abs(m) + np.abs(back))
            d = d + m - back
            self.dw_pre = (du * self.y * self.q2).sum(0)
            mag = np.abs(du * self.y * self.q2)
            self.err["dw_pre"] = (np.abs(du) * self.q2 * (
                self.err["y"] + np.abs(self.y) * (self.e_q2 + 8 * EPS))).sum(0) + G_sum(mag, rows)
        self.dx, self.err["dx"] = d, e
        e_t = self.e_sum + self.e_z + 8 * EPS
        self.dscale = (d * self.t).sum(0)
        self.err["dscale"] = (e * np.abs(self.t) + np.abs(d * self.t) * e_t).sum(0) \
            + G_sum(np.abs(d * self.t), rows)
        d, e = d * c, np.abs(c) * (e + 2 * EPS * np.abs(d))
        self.dz = d * self.nw * self.slope
        size = sigmoid(0 if self.z is None else self.z) * (
            1 + np.abs(0 if self.z is None else self.z)) if self.gate == 0 else np.abs(self.slope)
        self.err["dz"] = np.abs(self.nw) * (e * np.abs(self.slope)
                                            + np.abs(d) * size * (e_t + self.e_z + 8 * EPS))
        d, e = d * self.act, np.abs(self.act) * (e + np.abs(d) * (self.e_z + 4 * EPS))
        if self.w_post is not None:
            self.dw_post = (d * self.n).sum(0)
            self.err["dw_post"] = (np.abs(self.n) * (e + np.abs(d) * e_t)).sum(0) \
                + G_sum(np.abs(d * self.n), rows)
            m, em = d * self.w_post, np.abs(self.w_post) * (e + 2 * EPS * np.abs(d))
            dot = (m * self.n).mean(1, keepdims=True)
            mag = np.abs(m * self.n).mean(1, keepdims=True)
            e_dot = (em * np.abs(self.n)).mean(1, keepdims=True) + mag * (3 * self.e_sum + 8 * EPS)
            self.df = self.q1 * (m - self.n * dot)
            e = self.q1 * (em + np.abs(self.n) * e_dot
                           + (np.abs(m) + np.abs(self.n) * mag) * (2 * self.e_sum + 8 * EPS))
        else:
            self.df = d
        self.err["df"] = e
        return self
