"""Pins of the 64-bit gated recurrence that the GPU tests compare with: the
closed form, the composition of segments, and its gradients against central
differences and against torch's own derivative of the written-out recurrence."""
import pytest
import torch

from tests.gated_ref import Reference


def _case(b, l, d, seed, gate=True, h0=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=r(b, l, d).float(), g=r(b, l, d).float(), z=r(b, l, d).float() if gate else None,
                rate=torch.rand(d, generator=g), bias=r(d).float(),
                h0=r(b, d).float() if h0 else None)


def test_constant_gate_is_geometric():
    x = torch.full((1, 40, 1), 2.0)
    g = torch.full((1, 40, 1), 0.25)
    ref = Reference(x, g, rate=torch.tensor([0.3]), h0=torch.tensor([[-1.0]]))
    u = float(torch.tensor(0.3).double()) * float(torch.sigmoid(torch.tensor(0.25).double()))
    t = torch.arange(1, 41, dtype=torch.float64)
    want = 2.0 + (-1.0 - 2.0) * (1 - u) ** t
    assert torch.allclose(ref.out[:, 0], want, rtol=1e-12, atol=1e-12)


def test_split_sequence_equals_whole():
    c = _case(1, 30, 5, 3)
    whole = Reference(**c)
    cut = lambda v, a, b: None if v is None else v[:, a:b]  # noqa: E731
    one = Reference(cut(c["x"], 0, 11), cut(c["g"], 0, 11), cut(c["z"], 0, 11), c["rate"],
                    c["bias"], c["h0"])
    two = Reference(cut(c["x"], 11, 30), cut(c["g"], 11, 30), cut(c["z"], 11, 30), c["rate"],
                    c["bias"], one.h_final)
    assert torch.allclose(torch.cat((one.out, two.out)), whole.out, rtol=1e-13, atol=1e-13)
    assert torch.allclose(two.h_final, whole.h_final, rtol=1e-13, atol=1e-13)


def test_packed_equals_sequences_alone():
    c = _case(1, 20, 3, 4)
    cu = [0, 7, 7, 8, 20]
    h0 = torch.randn(4, 3)
    flat = lambda v: v[0]  # noqa: E731
    packed = Reference(flat(c["x"]), flat(c["g"]), flat(c["z"]), c["rate"], c["bias"], h0, cu=cu)
    for b in range(4):
        sl = slice(cu[b], cu[b + 1])
        if cu[b] == cu[b + 1]:
            assert torch.equal(packed.h_final[b], h0[b].double())
            continue
        alone = Reference(c["x"][:, sl], c["g"][:, sl], c["z"][:, sl], c["rate"], c["bias"],
                          h0[b:b + 1])
        assert torch.equal(alone.out, packed.out[sl])


@pytest.mark.parametrize("gate", [True, False])
def test_gradients_against_differences_and_autograd(gate):
    c = _case(2, 6, 3, 8, gate=gate)
    g = torch.Generator().manual_seed(9)
    dout = torch.randn(2, 6, 3, generator=g)
    dh = torch.randn(2, 3, generator=g)
    got = {k: v[0] for k, v in Reference(**c).gradients(dout, dh).items()}

    def loss(**v):
        x, gg, z = (v[k].double() if v[k] is not None else None for k in ("x", "g", "z"))
        h, total = v["h0"].double(), 0.0
        for t in range(6):
            u = v["rate"].double() * torch.sigmoid(gg[:, t] + v["bias"].double())
            h = (1 - u) * h + u * x[:, t]
            out = h if z is None else h * z[:, t] * torch.sigmoid(z[:, t])
            total = total + (out * dout[:, t].double()).sum()
        return total + (h * dh.double()).sum()

    leaves = {k: (None if v is None else v.double().requires_grad_()) for k, v in c.items()}
    loss(**leaves).backward()
    for k, v in leaves.items():
        if v is None:
            assert got["dz"] is None
            continue
        assert torch.allclose(got["d" + k].reshape(v.shape), v.grad, rtol=1e-11, atol=1e-11), k
        # central differences at one element: the truncation is O(eps^2), the
        # cancellation 1e-16 / eps
        eps, at = 1e-5, tuple(0 for _ in v.shape)
        lo, hi = {**leaves}, {**leaves}
        for side, sign in ((lo, -1), (hi, 1)):
            side[k] = v.detach().clone()
            side[k][at] += sign * eps
        diff = (loss(**{q: (None if w is None else w.detach()) for q, w in hi.items()})
                - loss(**{q: (None if w is None else w.detach()) for q, w in lo.items()})) / (2 * eps)
        assert abs(float(diff) - float(v.grad[at])) < 1e-7
