"""The binding of the 8-bit product and of the verification, without a GPU."""
import pytest
import torch

q4 = pytest.importorskip("bit_weight_only_q4g128_amd")


def product(M=20, N=1030, K=2048):
    G = K // 128
    c = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    return c(M, K), torch.ones(M, G), c(N, K), torch.ones(-(-N // 128), G)


def test_size_query_makes_no_outputs(monkeypatch):
    """The question for a workspace's size allocates nothing (outputs may be
    larger than what is left)."""
    x, xs, w, ws = product()
    out = torch.zeros(20, 1030, dtype=torch.bfloat16)
    resid = torch.zeros(20, 1030, dtype=torch.bfloat16)
    monkeypatch.setattr(q4, "_check", lambda *a: None)      # (host tensors stand for the GPU's)

    def made(*a, **k):
        raise AssertionError("a tensor was made")

    for name in ("new_empty", "new_zeros"):
        monkeypatch.setattr(torch.Tensor, name, made)
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, made)
    given = q4.fp8b128_workspace_bytes([(x, xs, w, ws, resid, out)])
    assert given > 65536
    assert q4.fp8b128_workspace_bytes([(x, xs, w, ws, resid, None)]) == given
    group = [(x, xs, w, ws, None, None)] * 8
    assert q4.fp8b128_workspace_bytes(group) >= 0
    with pytest.raises(q4.Q4GemvError) as e:
        q4.fp8b128_workspace_bytes([(x, xs, w, ws, None, out), (x, xs, w, ws, None, out)])
    assert e.value.status == -4


@pytest.mark.parametrize("workspace", [1 << 20, b"\0" * 256, "none", [0]])
def test_workspace_that_is_no_tensor(monkeypatch, workspace):
    """Refused as any other argument of a wrong type is."""
    monkeypatch.setattr(q4, "_check", lambda *a: None)      # (host tensors stand for the GPU's)
    lg, d, u = torch.zeros(1, 2, 8, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 2)
    for call in (lambda: q4.fp8b128_gemm(*product(4, 256, 256), workspace=workspace),
                 lambda: q4.verify_topk(lg, d, u, top_k=2, workspace=workspace), lambda: q4.verify_full(lg, d, u, workspace=workspace)):
        with pytest.raises(TypeError, match="workspace"):
            call()
