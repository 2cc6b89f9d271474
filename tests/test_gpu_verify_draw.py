"""The draw of verify_full at the boundaries of its running sums, where the last
bits of the kernel's fp64 arithmetic decide.

Every probability is within about 5e-15 of its value (an exponential 1.3e-16,
its argument 1.1e-16 |log2 p| with |log2 p| below 20 where nearly all of a row's
mass lies, at most about 30 roundings of 1.1e-16 in a row's sum), a difference
p - q within 1e-14 of p, and with R the mass of max(p - q, 0) a boundary of the
draw within 1e-14 / R of its place in [0, 1)."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q4():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bit_weight_only_q4g128_amd as m
    return m


def raised(V, values, seed=0):
    """Logits and the draft's: the same but for the largest, a bf16 step up, so
    that max(p - q, 0) is a multiple of p everywhere else and 0 there.  values:
    the spread of normal logits, or the values that parts of the row have, one
    after the other (so that errors which go by the value do not average out)."""
    if isinstance(values, tuple):
        z = torch.tensor(values).repeat_interleave(-(-V // len(values)))[:V].to(torch.bfloat16)
        z[V // 3] = 2.0
    else:
        z = (torch.randn(V, generator=synth.make_gen(("raised", V, seed))) * values).to(torch.bfloat16)
    at = int(z.float().argmax())
    y = z.clone()
    y[at] = (z[at].float() * (1 + 2.0 ** -7)).to(torch.bfloat16)
    assert float(y[at]) > float(z[at]) > 0
    return z, y, at


def near_boundaries(z, y, at, T, count):
    """Uniforms (fp32 values) next to boundaries of that draw, not nearer than
    twice 1e-14 / R, and the tokens they give; in 80-bit arithmetic."""
    ld = np.longdouble
    zz, yy = z.double().numpy().astype(ld) / ld(np.float32(T)), y.double().numpy().astype(ld) / ld(np.float32(T))
    e, f = np.exp(zz - zz.max()), np.exp(yy - yy.max())
    p, q = e / e.sum(), f / f.sum()
    R = float(np.maximum(p - q, 0).sum())
    e[at] = 0
    V, c = len(e), np.cumsum(e)
    c = c / c[-1]
    u = c[:-1].astype(np.float32)
    near = np.abs(u.astype(ld) - c[:-1]).astype(np.float64)
    far = 2e-14 / R
    bounds = c[:-1][np.arange(V - 1) != at]         # (at itself has no mass: its boundary is the one before it)

    def alone(i):       # no boundary as near as that
        j = int(np.searchsorted(bounds, ld(u[i])))
        return all(abs(v - ld(u[i])) >= far for v in bounds[max(j - 1, 0):j + 1])

    order = []
    for i in np.argsort(near):
        if near[i] >= far and 0.0 < u[i] < 1.0 and alone(i):
            order.append(int(i))
            if len(order) == count:
                break
    tokens = [int(np.argmax(c > ld(u[i]))) for i in order]
    return u[order], tokens, far, near[order]


@pytest.mark.parametrize("values", [2.5, (1.5, 1.0), (1.25, 0.5, 1.75), (0.75, 1.125, 0.0, 1.0)])
@pytest.mark.parametrize("V,T", [(4099, 0.8), (16384, 1.0), (16385, 0.8), (40003, 0.5)])
def test_residual_draw_next_to_a_boundary(q4, V, T, values):
    z, y, at = raised(V, values)
    us, tokens, far, near = near_boundaries(z, y, at, T, 96)
    B = len(us)
    print(f"V={V} T={T} {values}: {B} uniforms {near.min():.2g} to {near.max():.2g} from a boundary, allowed from {far:.2g}", flush=True)
    assert B >= 32
    u = torch.stack([torch.full((B,), 1 - 2.0 ** -24), torch.from_numpy(us)], 1).contiguous()
    logits = gpu(z).expand(B, 2, V).contiguous()
    draft_logits = gpu(y).expand(B, 1, V).contiguous()
    draft = torch.full((B, 1), at, dtype=torch.int32, device="cuda")
    token, count, _ = q4.verify_full(logits, draft, gpu(u), draft_logits=draft_logits, temperature=T)
    assert int(count.sum()) == 0                # (q > p and the largest u: refused)
    assert token[:, 0].tolist() == tokens


def test_draw_next_to_a_masked_region(q4):
    """Rows of equal logits whose masses before and behind a masked region are
    equal, and a uniform of one half: the running sums over the empty region lie
    within an fp64 rounding of the place that is sought.  The token is one of the
    region's neighbours, and never -1 or a masked one."""
    V, B = 16384, 400
    rng = np.random.default_rng(0)
    logits = np.full((B, 2, V), -np.inf, np.float32)
    allowed = []
    for b in range(B):
        a, gap = int(rng.integers(2, 5)), int(rng.integers(1, 3))       # parts of 2048: before the region, the region
        before = [2048 * c + rng.permutation(2048)[:rng.integers(1, 700)] for c in range(a)]
        left = np.sort(np.concatenate(before))
        right = 2048 * (a + gap) + np.sort(rng.permutation(V - 2048 * (a + gap))[:len(left)])
        logits[b, 0, left] = logits[b, 0, right] = 1.0
        allowed.append((int(left[-1]), int(right[0])))
    logits[:, 1] = 0.0
    token, count, _ = q4.verify_full(gpu(torch.from_numpy(logits).to(torch.bfloat16)), torch.zeros(B, 1, dtype=torch.int32, device="cuda"),
                                     torch.full((B, 2), 0.5, device="cuda"), n_draft=torch.zeros(B, dtype=torch.int32, device="cuda"))
    assert int(count.sum()) == 0
    wrong = [(b, t, allowed[b]) for b, t in enumerate(token[:, 0].tolist()) if t not in allowed[b]]
    assert not wrong, f"{len(wrong)} of {B}: {wrong[:5]}"
