"""The gated linear recurrence in 64 bits, step by step, with bounds on how far
a correct fp32 evaluation may be from it.

The bounds follow the recurrence.  With M the largest |x| or |h0| that a state
has seen (h is a convex combination of those, and so is every partial state):

* sigmoid(v) from an ex2 and a reciprocal: v = g + bias and v log2(e) are each
  rounded, 2^-24 |v| apiece, which e^-v turns into a relative 2 |v| 2^-24; the
  constant, the two approximations (2 ulp each) and the sum add under 16 2^-24.
  So E(v) = (|v| + 8) 2^-23 relative covers sigmoid, and u with one more
  rounding.  Below the smallest normal number the reciprocal is flushed to
  zero (and e^-v above 2^128 is an infinity), which is 2^-126 absolute.
* a step h + u (x - h) rounds the difference, the sum and, where a segment's
  states are formed from its carry as b + P c, the product P and the sum again:
  at most 4 roundings of quantities up to 2 M, so 2^-21 M, beside what u's error
  moves: u E 2 M.  An error made earlier shrinks by (1 - u) like the state.

The backward's state gh has the same form with a, the same recurrence over
absolute values, in place of M.  A result in bf16 is off by another 2^-8 of its
value (half a step), in fp32 by 2^-24.
"""
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
R = 2.0 ** -21
FLUSH = 2.0 ** -126


def _lens(x, cu):
    if cu is None:
        return [(b * x.shape[1], x.shape[1]) for b in range(x.shape[0])]
    cu = [int(v) for v in cu]
    return [(cu[b], cu[b + 1] - cu[b]) for b in range(len(cu) - 1)]


def _flat(t, d):
    return t.detach().double().cpu().reshape(-1, d)


class Reference:
    """Forward values and bounds, on the CPU: out, h_final, before (the state
    before each row) and the error bounds e_h (row), e_out, e_final."""

    def __init__(self, x, g, z=None, rate=None, bias=None, h0=None, cu=None):
        d = x.shape[-1]
        self.d, self.dtype, self.seqs = d, x.dtype, _lens(x, cu)
        self.x, self.g = _flat(x, d), _flat(g, d)
        self.z = None if z is None else _flat(z, d)
        one = torch.ones(d, dtype=torch.float64)
        self.rate = one if rate is None else rate.detach().double().cpu()
        bias = 0 * one if bias is None else bias.detach().double().cpu()
        v = self.g + bias
        self.s = torch.sigmoid(v)
        self.d_s = self.s * (v.abs().clamp(max=1e30) + 8) * 2.0 ** -23 + FLUSH
        self.u = self.rate * self.s
        n = len(self.seqs)
        h0 = torch.zeros(n, d, dtype=torch.float64) if h0 is None else h0.detach().double().cpu()
        self.h_final, self.e_final = h0.clone(), torch.zeros_like(h0)
        self.before = torch.zeros_like(self.x)
        self.h, self.e_h, self.e_before = (torch.zeros_like(self.x) for _ in range(3))
        self.m = torch.zeros_like(self.x)
        for b, (r0, length) in enumerate(self.seqs):
            h, e, m = h0[b].clone(), torch.zeros(d, dtype=torch.float64), h0[b].abs()
            for r in range(r0, r0 + length):
                u, xr = self.u[r], self.x[r]
                self.before[r], self.e_before[r] = h, e
                m = torch.maximum(m, xr.abs())
                h = h + u * (xr - h)
                e = (1 - u) * e + self.rate * self.d_s[r] * 2 * m + R * m
                self.h[r], self.e_h[r], self.m[r] = h, e, m
            self.h_final[b], self.e_final[b] = h, e
        half = HALF_STEP[self.dtype]
        if self.z is None:
            self.out, self.e_out = self.h, self.e_h + half * self.h.abs()
        else:
            self.sz = torch.sigmoid(self.z)
            self.d_sz = self.sz * (self.z.abs().clamp(max=1e30) + 8) * 2.0 ** -23 + FLUSH
            gate = self.z * self.sz
            self.out = self.h * gate
            self.e_out = gate.abs() * self.e_h + self.h.abs() * self._e_gate() \
                + half * self.out.abs()

    def _e_gate(self):
        return self.z.abs() * (self.d_sz + self.sz * R)

    def gradients(self, dout, dh_final=None):
        """{name: (value, bound)}."""
        d, half = self.d, HALF_STEP[self.dtype]
        dout = _flat(dout, d)
        n = len(self.seqs)
        dh = torch.zeros(n, d, dtype=torch.float64) if dh_final is None \
            else dh_final.detach().double().cpu()
        gate = 1.0 if self.z is None else self.z * self.sz
        e_gate = 0.0 if self.z is None else self._e_gate()
        dy, e_dy = dout * gate, dout.abs() * e_gate
        gh, a, e = (torch.zeros_like(self.x) for _ in range(3))
        dh0, e_dh0 = dh.clone(), torch.zeros_like(dh)
        for b, (r0, length) in enumerate(self.seqs):
            c, ca, ce = dh[b], dh[b].abs(), torch.zeros(d, dtype=torch.float64)
            for r in range(r0 + length - 1, r0 - 1, -1):
                gh[r], a[r] = dy[r] + c, dy[r].abs() + ca
                e[r] = ce + e_dy[r] + R * a[r]
                c, ca = (1 - self.u[r]) * gh[r], (1 - self.u[r]) * a[r]
                ce = (1 - self.u[r]) * e[r] + (self.rate * self.d_s[r] + R) * a[r]
            dh0[b], e_dh0[b] = c, ce
        u, s, x = self.u, self.s, self.x
        d_u = self.rate * self.d_s
        dx = u * gh
        e_dx = u * (e + R * a) + d_u * a + half * dx.abs()
        diff = x - self.before
        du = gh * diff
        e_du = e * diff.abs() + a * (self.e_before + R * self.m)
        dg = du * u * (1 - s)
        e_dg = (1 - s) * (u * (e_du + R * du.abs()) + d_u * du.abs()) \
            + u * du.abs() * (self.d_s + s * R) + half * dg.abs()
        res = {"dx": (dx, e_dx), "dg": (dg, e_dg), "dz": (None, None), "dh0": (dh0, e_dh0)}
        if self.z is not None:
            slope = self.sz * (1 + self.z * (1 - self.sz))
            dz = dout * self.h * slope
            e_slope = (self.d_sz + self.sz * R) * (1 + self.z.abs())
            res["dz"] = (dz, dout.abs() * (slope.abs() * self.e_h + self.h.abs() * e_slope)
                         + half * dz.abs())
        # sums: the terms' own bounds, and one rounding (2^-24 of the sum so far, at
        # most the sum of absolute values) for each term
        count = 2.0 ** -24 * (x.shape[0] + 8)
        terms, e_terms = du * s, e_du * s + du.abs() * (self.d_s + s * R)
        res["drate"] = (terms.sum(0), e_terms.sum(0) + count * terms.abs().sum(0))
        raw = e_dg - half * dg.abs()  # dbias adds dg before it is rounded to the I/O type
        res["dbias"] = (dg.sum(0), raw.sum(0) + count * dg.abs().sum(0))
        return res


def assert_within(got, want, bound, what):
    got = got.detach().double().cpu().reshape(want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound - 1e-37
    worst = int(over.argmax()) if over.numel() else 0
    assert not over.numel() or over.reshape(-1)[worst] <= 0, (
        f"{what}: element {worst} is {got.reshape(-1)[worst]:.9g}, expected "
        f"{want.reshape(-1)[worst]:.9g} within {bound.reshape(-1)[worst]:.3g}")
