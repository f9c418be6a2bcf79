"""The gated delta rule and its gradients over many chunks: every two-stage ring
is refilled several times, the barriers' phases return to where they began, and
the states and their gradients are carried far.  Each case is on its intended
side of the rule that picks whole heads or slices of 16 rows an SM.

Tolerances: those of the shorter calls.  A chunk's rounding enters the state
once and from then on decays with it (gates are negative, keys of length one),
so the relative error of a long chain is that of a few chunks.
"""
import pytest
import torch

from chunk_wise_weight_gb300 import build, ittt
import test_delta_gpu as seq
import test_delta_grad_gpu as grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    torch.manual_seed(0)
    build.build()
    return ittt.load()


def by_head(sequences, Hv, dv):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return dv > 32 and sequences * Hv * (dv // 16) > 2 * sms


def heads_for(sequences, dv):
    """The fewest value heads (a multiple of 2) with which the calls take whole heads."""
    Hv = 2
    while not by_head(sequences, Hv, dv):
        Hv += 2
    return Hv


def both(x, S0, dS1, do, cu=None):
    """Outputs (bf16 and fp32), states and gradients against the definition."""
    dk = x["q"].shape[-1]
    S1, dS0 = torch.empty_like(S0), torch.empty_like(S0)
    out = seq.call(x, state_in=S0, state_out=S1, cu_seqlens=cu)
    ref, rs = seq.reference(x, dk ** -0.5, S0, cu)
    seq.check_out(out, ref)
    seq.check_state(S1, rs)
    seq.check_out(seq.call(x, state_in=S0, out_dtype=torch.float32, cu_seqlens=cu), ref)
    got = grad.call(x, do, state_in=S0, grad_state_out=dS1, grad_state_in=dS0, cu_seqlens=cu)
    grad.check((*got, dS0), grad.reference(x, dk ** -0.5, S0, do, dS1, cu))
    again = grad.call(x, do, state_in=S0, grad_state_out=dS1, cu_seqlens=cu)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return S1, dS0


def inputs(B, S, T, Hk, Hv, dk, dv):
    x = seq.make(B, T, Hk, Hv, dk, dv, seed=T)
    return (x, 0.3 * torch.randn(S, Hv, dv, dk, device="cuda"), 0.1 * torch.randn(S, Hv, dv, dk, device="cuda"),
            torch.randn(B, T, Hv, dv, device="cuda").bfloat16())


@pytest.mark.parametrize("T,dk,dv", [(401, 64, 128), (401, 128, 64), (640, 128, 128)])
def test_whole_heads(cuda_device, T, dk, dv):
    Hv = heads_for(2, dv)
    both(*inputs(2, 2, T, Hv // 2, Hv, dk, dv))


@pytest.mark.parametrize("dk,dv", [(128, 112), (64, 128)])
def test_whole_heads_packed(cuda_device, dk, dv):
    cu = [0, 0, 50, 230, 550, 934, 934, 1300]  # 0, 1, 3, 5, 6, 0 and 6 chunks
    S = len(cu) - 1
    Hv = heads_for(S, dv)
    x, S0, dS1, do = inputs(1, S, cu[-1], Hv // 2, Hv, dk, dv)
    S1, dS0 = both(x, S0, dS1, do, cu)
    for s, (a, e) in enumerate(zip(cu, cu[1:])):
        if a == e:
            assert torch.equal(S1[s], S0[s]) and torch.equal(dS0[s], dS1[s])


@pytest.mark.parametrize("T,Hk,Hv,dk,dv", [(450, 1, 2, 128, 48), (390, 2, 4, 64, 128)])
def test_slices(cuda_device, T, Hk, Hv, dk, dv):
    assert not by_head(2, Hv, dv)
    both(*inputs(2, 2, T, Hk, Hv, dk, dv))


def test_slices_in_pairs_packed(cuda_device):
    """More slices than SMs, but not twice as many: two share a CTA."""
    cu = [0, 400, 400, 430, 810]
    sms, dv = torch.cuda.get_device_properties(0).multi_processor_count, 64
    Hv = sms // (4 * 4) // 2 * 2 + 2
    assert 4 * Hv * 4 > sms and not by_head(4, Hv, dv)
    x, S0, dS1, do = inputs(1, 4, cu[-1], Hv // 2, Hv, 128, dv)
    both(x, S0, dS1, do, cu)


# heads that forget within a token beside heads that keep thousands
DECAYS = (-1e-3, -0.1, -1.0, -3.0, -5.0, -8.0, -12.0, -16.0)


def check_gate_gradient(got, ref, g):
    """grad_g by token and head.  grad_g = e^g z, z the gradient at the factor e^g itself;
    every term of grad_g carries that factor, so its error is relative to e^g and to the
    size that z has in the head: products of 24-bit operands, sums of 128 terms whose
    magnitudes add up to some 11 times the sum (2^-24 * sqrt(128) * 11 = 2^-17), four such
    chained, taken at 2^-14."""
    a = torch.exp(g.double())
    z = torch.where(a > 0, ref / a, 0.0)
    size = (z ** 2).mean(dim=(0, 1), keepdim=True).sqrt()
    err = (got.double() - ref).abs()
    bound = 2.0 ** -14 * a * (z.abs() + size)
    # below fp32's normal numbers the decays themselves have fewer bits
    assert torch.all(err <= bound + 1e-35), float((err / (bound + 1e-35)).max())


@pytest.mark.parametrize("B,dk,dv", [(1, 128, 64), (2, 64, 128), (8, 128, 96), (8, 64, 144)])
def test_gate_gradient_of_every_token(cuda_device, B, dk, dv):
    T, Hv = 150, len(DECAYS)
    assert by_head(B, Hv, dv) == (B == 8)
    x, S0, dS1, do = inputs(B, B, T, Hv // 2, Hv, dk, dv)
    x["g"] = torch.tensor(DECAYS, device="cuda") * (0.8 + 0.4 * torch.rand(B, T, Hv, device="cuda"))
    x["g"][:, 70:75, :3] = -15.0         # strong tokens in heads that keep
    x["g"][:, 100, :6] = -60.0
    x["g"][:, 20, ::2] = -float("inf")   # resets
    x["g"][:, 64, 1::2] = -2000.0
    x["beta"][:, 30:33] = 0.0
    # the definition's exp has no gradient at -inf: a decay of e^-2000 is as much zero
    y = dict(x, g=torch.where(x["g"] < -1000, torch.full_like(x["g"], -2000.0), x["g"]))
    ref = grad.reference(y, dk ** -0.5, S0, do, dS1)
    dS0 = torch.empty_like(S0)
    got = grad.call(x, do, state_in=S0, grad_state_out=dS1, grad_state_in=dS0)
    grad.check((*got, dS0), ref)
    check_gate_gradient(got[3], ref[3], y["g"])
    assert torch.all(got[3][:, 20, ::2] == 0) and torch.all(got[3][:, 64, 1::2] == 0)
    # and the differences of the definition, each head's gates along one direction
    h, S64 = 1e-4, S0.double()
    way = torch.sign(torch.randn(Hv, device="cuda").double())
    args = [y[n].double() for n in ("q", "k", "v", "g", "beta")]
    spans = [(b, 0, T) for b in range(B)]

    def loss(shift):
        out, S1 = grad.forward64(*args[:3], args[3] + shift * way, args[4], dk ** -0.5, S64, spans)
        return (out * do.double()).sum((0, 1, 3)) + (S1 * dS1.double()).sum((0, 2, 3))

    slope = (loss(h) - loss(-h)) / (2 * h)  # heads do not meet: one slope each
    mine = (got[3].double() * way).sum((0, 1))
    size = got[3].double().abs().sum((0, 1))
    # the difference's own error: h^2 / 6 of the third derivative, and 1e-16 of the loss / h
    assert torch.all((slope - mine).abs() <= 2.0 ** -12 * size + 1e-8), (slope, mine)


def wrongly_rounded(got, ref):
    return float((got != ref.to(torch.bfloat16)).double().mean())


@pytest.mark.parametrize("B,dk,dv", [(1, 128, 64), (2, 64, 128), (20, 128, 96), (20, 64, 128)])
def test_bf16_results_are_rounded_once(cuda_device, B, dk, dv):
    """Every product has operands of 24 bits, so a bf16 result is the exact value's
    rounding but where that lies between two bf16 numbers by no more than the error.
    An error of 2^-21 of a head's typical value (24 bits, some sums) moves about
    2 * 2^-21 / 2^-8 of the elements of that size, and some eight times as many with
    the small ones: 2^-9 * 2^-2 = 2^-11.  (Operands of 16 bits move 32 times as many.)"""
    T, Hv = 300, 4
    assert by_head(B, Hv, dv) == (B == 20)
    x, S0, dS1, do = inputs(B, B, T, 2, Hv, dk, dv)
    assert wrongly_rounded(seq.call(x, state_in=S0), seq.reference(x, dk ** -0.5, S0)[0]) <= 2.0 ** -11
    got = grad.call(x, do, state_in=S0, grad_state_out=dS1)
    ref = grad.reference(x, dk ** -0.5, S0, do, dS1)
    for name, a, r in zip("qkv", got, ref):
        assert wrongly_rounded(a, r) <= 2.0 ** -11, name
