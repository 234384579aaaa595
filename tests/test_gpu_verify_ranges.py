"""wedlm_verify_drafts over the whole range of temperatures, against its definition in 64 bits."""
import pytest
import torch

from tests.verify_common import Case

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("V", [700, 40000])
def test_temperatures_from_end_to_end(dtype, probs, V):
    """Logits grow with the temperature, so that p stays what it is at 1: both ends of the
    range, their neighbours inside, and numbers between with every sort of significand."""
    f = torch.tensor([1e-30, 1e18], dtype=torch.float32)
    inside = torch.nextafter(f, torch.ones(2)).tolist()
    temps = f.tolist() + inside + [3.3e-30, 7.77e-25, 1.9999999e-20, 1e-10, 2.0 ** -40, 0.3333333,
                                   1.9999999, 123.456, 65504.0, 1e7, 3.0e12, 9.87e17]
    c = Case(len(temps), 3, V, dtype, probs, seed=V, temps=(1.0,))
    c.temp = torch.tensor(temps, device="cuda")
    c.logits = (c.logits.double() * c.temp.double()[:, None, None]).to(dtype)
    c.call()
    c.check()


@pytest.mark.parametrize("t", [1e-30, 1e18])
def test_temperatures_beyond_the_ends(t):
    from serving_wedlm_step_gb300 import binding as Bd
    c = Case(2, 2, 500, FP, False, seed=31, temps=(1.0,))
    c.temp[:] = t
    c.temp[1] = torch.nextafter(c.temp[1], torch.tensor(float("inf") if t > 1 else 0.0, device="cuda"))
    c.logits = (c.logits.double() * t).float()
    c.call()
    assert int(c.err) == Bd.DEV_NUMERIC
    assert int(c.acc[1]) == 0 and c.tok[1].tolist() == [-1] * 3 and torch.isnan(c.sp).tolist() == [False, True]


def test_scales_of_temperatures():
    """p of a token that is y = -120 .. -2 (in powers of two) from the only other one, at 8192
    temperatures: y is the logit times log2(e) / T, where quotient and product are off by half
    a step each and the constant by a fifth of one, 2.25 x 2^-24 |y| ln 2 of p; the exponentials
    are 2^-22 off, the sum and the quotient 2^-24.  With a scale a step further off some
    would be beyond that."""
    B, g = 8192, torch.Generator().manual_seed(32)
    lo, hi = torch.tensor([1e-30, 1e18]).double().log().tolist()
    t = torch.exp(lo + (hi - lo) * torch.rand(B, generator=g, dtype=torch.float64)).float().clamp(1e-30, 1e18)
    y = -2 - 118 * torch.rand(B, generator=g, dtype=torch.float64)
    z = (y * 0.6931471805599453 * t.double()).float()
    c = Case(B, 1, 2, FP, False, seed=33, temps=(1.0,), mask_id=-1)
    c.temp = t.cuda()
    c.logits = torch.stack([torch.zeros(B), z], 1)[:, None].repeat(1, 2, 1).cuda()
    c.x = torch.ones(B, 1, dtype=torch.int32, device="cuda")
    c.call()
    y = z.double() / t.double()
    want = 1 / (1 + (-y).exp())
    off = (c.dp[:, 0].cpu().double() / want - 1).abs()
    bound = 2.25 * 2.0 ** -24 * y.abs() + 2 * 2.0 ** -22 + 2 * 2.0 ** -24
    assert int(c.err) == 0 and (off <= bound).all(), (off / bound).max()
