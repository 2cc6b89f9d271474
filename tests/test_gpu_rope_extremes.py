"""rope_cache's norm where squares, their mean or eps leave fp32's normal range,
against the fp64 oracle.  Bounds: attention_util (the norm's own, 2^-18, and one
rounding to bf16; below bf16's normal range its step, 2^-133)."""
import numpy as np
import pytest
import torch

import oracle
import synth
from attention_util import rope_bound, values, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def check(got, x, w, eps, what):
    eps = float(np.float32(eps))
    want = oracle.rope_heads(values(x), norm=values(w), eps=eps)
    bound = rope_bound(values(x), None, None, values(w), eps, False)
    within(got, want, bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133, what)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [1.5e-45, 1e-40, 1e-38, 1e-30, 1e-24, 1e-12, 1e-6, 1.0, 1e20, 1e36, 3e38, 3.4028234e38])
def test_any_eps_and_size(q4, D, eps):
    """Heads of sizes 2^-133 to 2^126, one size to a token, and heads whose
    values differ in size, under any eps that a call may have."""
    T, Hq = 132, 3
    g = synth.make_gen(("extremes", D, eps))
    size = torch.tensor([2.0 ** (-133 + 2 * t) for t in range(T - 2)] + [1.0, 1.0], dtype=torch.float64)
    x = torch.randn(T, Hq + 1, D, generator=g, dtype=torch.float64).clamp(-1.9, 1.9) * size[:, None, None]
    x[T - 2] *= 2.0 ** torch.randint(-120, -20, (Hq + 1, D), generator=g).double()
    x[T - 1] *= 2.0 ** torch.randint(30, 126, (Hq + 1, D), generator=g).double()
    x = x.to(torch.bfloat16).cuda()
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    q, k = x[:, :Hq], x[:, Hq:]
    qo, ko = q4.rope_cache(q, k, q_norm=w[0], k_norm=w[1], eps=eps)
    check(qo, q, w[0], eps, "q")
    check(ko, k, w[1], eps, "k")
