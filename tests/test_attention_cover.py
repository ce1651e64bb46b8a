"""The planted values do what they are for, on the CPU: one token left out or counted twice moves the 64-bit form's
output beyond the tolerances of the GPU tests that use them."""
import pytest
import torch

from tests import attention_ref as ref
from tests.attention_cover import cover


@pytest.mark.parametrize("n,K,D,step,every,tol", [
    (20000, 1, 128, 64, False, 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15), (40000, 1, 64, 64, False, 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15),
    (5000, 8, 128, 64, True, 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15), (9000, 2, 64, 128, False, 2.0 ** -7 + 2.0 ** -15),
    (2500, 2, 64, 128, True, 2.0 ** -7 + 2.0 ** -15)])
def test_one_token_shows(n, K, D, step, every, tol):
    g = torch.Generator().manual_seed(n)
    k = torch.randn(n, K, D, generator=g)
    v = torch.zeros(n, K * D)
    most = cover(v, [0, n], K, D, step, every)
    assert most <= 24
    v = v.view(n, K, D)
    q = torch.randn(1, K, D, generator=g)
    want, size = ref.attend(q, k, v, D ** -0.5)
    for t in [0, 1, step - 1, step, n // 2 // step * step, n - n % step - 1, n - 1]:
        if not bool((v[t] != 0).any()):
            continue
        keep = torch.arange(n) != t
        for kk, vv in ((k[keep], v[keep]), (torch.cat([k, k[t:t + 1]]), torch.cat([v, v[t:t + 1]]))):
            got, _ = ref.attend(q, kk, vv, D ** -0.5)
            off = (got - want).abs() > tol * size + 1e-30
            assert bool(off.any()), t
