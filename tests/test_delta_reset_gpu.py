"""A reset (a gate of minus infinity) in every form of the gated delta rule: what
follows it equals, bit by bit, what follows it after any other past, and where the
reset is at the start of a chunk, or the call goes token by token, after a past that
is not finite too."""
import pytest
import torch

from chunk_wise_weight_gb300 import build, ittt
import test_delta_gpu as seq
import test_delta_grad_gpu as grad
from test_delta_deep_gpu import by_head

pytestmark = pytest.mark.gpu
INF = float("inf")
# token by token; slices; whole heads
FORMS = [(1, 16, 2, 128, 32, torch.bfloat16), (1, 40, 2, 64, 48, torch.float32), (2, 150, 2, 128, 48, torch.bfloat16),
         (20, 150, 4, 128, 96, torch.bfloat16), (20, 150, 4, 64, 128, torch.bfloat16)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    torch.manual_seed(0)
    build.build()
    return ittt.load()


def case(B, T, Hv, dk, dv, dtype, at):
    assert dtype != torch.bfloat16 or T <= 16 or by_head(B, Hv, dv) == (B == 20)
    x = seq.make(B, T, Hv // 2, Hv, dk, dv, dtype, seed=T)
    x["g"][:, at] = -INF
    return x, torch.randn(B, Hv, dv, dk, device="cuda")


def run(x, S0, **kw):
    S1 = torch.empty_like(S0)
    return seq.call(x, state_in=S0, state_out=S1, **kw), S1


@pytest.mark.parametrize("B,T,Hv,dk,dv,dtype", FORMS)
@pytest.mark.parametrize("where", [0.6, 0.1])
def test_nothing_finite_of_the_past_is_left(cuda_device, B, T, Hv, dk, dv, dtype, where):
    at = int(T * where)
    x, S0 = case(B, T, Hv, dk, dv, dtype, at)
    out, S1 = run(x, S0)
    past = {n: y.clone() for n, y in x.items()}
    for n in ("q", "k", "v"):
        past[n][:, :at] = torch.randn_like(past[n][:, :at])  # tokens of the reset's own chunk among them
    past["k"][:, :at] /= past["k"][:, :at].norm(dim=-1, keepdim=True)
    past["beta"][:, :at] = 0.5
    other, S2 = run(past, 3 * S0)
    assert not torch.equal(other[:, :at], out[:, :at])
    assert torch.equal(other[:, at:], out[:, at:]) and torch.equal(S2, S1)


@pytest.mark.parametrize("bad", [INF, float("nan")])
@pytest.mark.parametrize("B,T,Hv,dk,dv,dtype", FORMS)
def test_a_state_that_is_not_finite_is_cleared(cuda_device, B, T, Hv, dk, dv, dtype, bad):
    x, S0 = case(B, T, Hv, dk, dv, dtype, 0)
    S0.zero_()
    S0bad = torch.full_like(S0, bad)
    for kw in (dict(), dict(out_dtype=torch.float32)):
        out, S1 = run(x, S0, **kw)
        assert torch.isfinite(out).all()
        got, S2 = run(x, S0bad, **kw)
        assert torch.equal(got, out) and torch.equal(S2, S1)
    if dtype == torch.bfloat16:
        do, dS1 = torch.randn_like(x["v"]), torch.randn_like(S0)
        res = []
        for s in (S0, S0bad):
            dS0 = torch.empty_like(S0)
            res.append((*grad.call(x, do, state_in=s, grad_state_out=dS1, grad_state_in=dS0), dS0))
        assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(*res))
        assert torch.all(res[0][5] == 0)


@pytest.mark.parametrize("B,T,Hv,dk,dv,dtype", FORMS)
def test_a_past_that_is_not_finite_is_cleared(cuda_device, B, T, Hv, dk, dv, dtype):
    by_token = T <= 16 or dtype == torch.float32
    at = 7 if by_token else 64
    x, S0 = case(B, T, Hv, dk, dv, dtype, at)
    out, S1 = run(x, S0)
    x["v"][:, 3, 0] = INF
    x["v"][:, 4, -1] = float("nan")
    got, S2 = run(x, S0)
    assert not torch.isfinite(got[:, at - 1]).all()
    assert torch.equal(got[:, at:], out[:, at:]) and torch.equal(S2, S1)


def test_documents_that_start_with_a_reset(cuda_device):
    cu, H, dv, dk = [0, 70, 70, 83, 283], 2, 64, 128
    x = seq.make(1, cu[-1], 1, H, dk, dv)
    S0 = torch.full((len(cu) - 1, H, dv, dk), float("nan"), device="cuda")
    zero = torch.zeros_like(S0)
    for a, b in zip(cu, cu[1:]):
        if a < b:
            x["g"][:, a] = -INF
    (out, S1), (got, S2) = run(x, zero, cu_seqlens=cu), run(x, S0, cu_seqlens=cu)
    assert torch.equal(got, out) and torch.equal(S2[[0, 2, 3]], S1[[0, 2, 3]])
    assert torch.isnan(S2[1]).all()  # no token, no reset


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_step_into_rows_that_were_never_written(cuda_device, dtype):
    x = seq.make(3, 1, 2, 4, 64, 80, dtype)
    x["g"][0] = x["g"][2] = -INF
    pool = torch.full((5, 4, 80, 64), float("nan"), device="cuda")
    pool[4] = torch.randn(4, 80, 64, device="cuda")
    clean = torch.nan_to_num(pool)
    slots = torch.tensor([3, 4, 0], device="cuda")
    tok = [x[n][:, 0] for n in ("q", "k", "v", "g", "beta")]
    want, got = ittt.delta_step(*tok, clean, slots=slots), ittt.delta_step(*tok, pool, slots=slots)
    assert torch.isfinite(want).all() and torch.equal(got, want) and torch.equal(pool[slots], clean[slots])
    assert torch.isnan(pool[[1, 2]]).all()
