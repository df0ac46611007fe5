"""GPU tests of qmv_sample at the ends of fp32's range. Definition and tolerances as in the operator's own tests."""
import pytest
import torch

from test_gpu_sample import run

pytestmark = pytest.mark.gpu


def rows(logits, u, temperature, top_p=None):
    M = len(u)
    full = lambda v: None if v is None else torch.full((M,), v, device="cuda")  # noqa: E731
    return dict(logits=torch.tensor([logits] * M, device="cuda"), u=torch.tensor(u, device="cuda"), temperature=full(temperature),
                top_k=None, top_p=full(top_p), min_p=None)


@pytest.mark.parametrize("temperature", [1e-40, 1e-45, 2.0 ** -127, 0.0, -1.0, float("nan")])
@pytest.mark.parametrize("top_p", [None, 0.9])
def test_temperatures_below_the_normal_range_take_the_first_token(temperature, top_p):
    args = rows([0.5, 2.0, 1e-45, 2.0, -1.0], [0.0, 0.3, 0.7, 0.99999], temperature, top_p)
    token, prob = run(args)
    assert token.tolist() == [1] * 4 and prob.tolist() == [1.0] * 4


def test_the_least_temperature():
    """2^-126: logits that are equal share, one that is 2^-126 less weighs 1 / e, any other 0."""
    args = rows([0.0, 2.0 ** -126, 2.0 ** -126, 1e-30 * 0, -1e-30], [0.0, 0.05, 0.2, 0.6, 0.8, 0.99], 2.0 ** -126)
    token, prob = run(args)
    e = 2.718281828459045
    whole = 2 + 2 / e                               # logits 0 and 3 weigh 1 / e each
    assert token.tolist() == [0, 0, 1, 2, 2, 3]
    want = torch.tensor([{0: 1 / e, 1: 1, 2: 1, 3: 1 / e}[t] / whole for t in token.tolist()], device="cuda")
    assert bool(((prob - want).abs() <= 2.0 ** -22 * want).all())


def test_logits_further_apart_than_the_range_reaches():
    args = rows([3e38, -3e38, 3e38 - 1e37, -float("inf")], [0.0, 0.5, 0.53, 0.9, 0.9999], 1e38)
    token, prob = run(args)
    w = 0.9048374180359595                          # e^-0.1, but for the rounding of 3e38 - 1e37 and 1e37 / 1e38
    assert token.tolist() == [0, 0, 2, 2, 2]
    assert abs(float(prob[0]) - 1 / (1 + w)) < 1e-6
