"""The attention calls' binding, without a GPU: host tensors stand for the GPU's,
and nothing is launched."""
import pytest
import torch

q4 = pytest.importorskip("bit_weight_only_q4g128_amd")


@pytest.fixture
def launched(monkeypatch):
    """Calls that would have gone to the library."""
    calls = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(q4, "_enqueue", lambda index, fn, *args: calls.append(args))
    return calls


def parts(T, Hq=4, Hk=2, D=64):
    base = torch.zeros(T, Hq + 2 * Hk, D, dtype=torch.bfloat16)
    return base, base[:, :Hq], base[:, Hq:Hq + Hk], base[:, Hq + Hk:]


@pytest.mark.parametrize("interleaved", [False, True])
def test_outputs_at_an_inputs_address(launched, interleaved):
    """In place is the input itself.  Another tensor that begins where the input
    does, whose tokens do not lie as the input's, would be filled at the
    input's places: refused."""
    T = 5
    base, q, k, v = parts(T)
    flat = base.view(-1)
    q_out = flat[:q.numel()].view(q.shape)
    k_at = k.storage_offset()
    k_out = flat[k_at:k_at + k.numel()].view(k.shape)
    assert q_out.data_ptr() == q.data_ptr() and k_out.data_ptr() == k.data_ptr()
    for kw in (dict(q_out=q_out), dict(k_out=k_out)):
        with pytest.raises(ValueError, match="in place"):
            q4.rope_cache(q, k, interleaved=interleaved, **kw)
    assert not launched
    # the input itself, another view of the same rows, and of one token
    assert q4.rope_cache(q, k, q_out=q, k_out=k)[0] is q
    c = q.contiguous()
    again = c.view(c.shape)
    assert q4.rope_cache(c, k, q_out=again)[0] is again
    base, q, k, v = parts(1)
    one = base.view(-1)[:q.numel()].view(q.shape)
    assert q4.rope_cache(q, k, q_out=one)[0] is one
    assert len(launched) == 3


@pytest.mark.parametrize("scale", [2.0 ** 127 * (1 + 2.0 ** -23), 2.4e38, 3e38, 3.4028234e38])
def test_scale_past_its_limit(scale):
    """scale * log2 e is an fp32 number."""
    from test_abi_attention import ESHAPE, decode, prefill
    assert decode(scale=scale) == ESHAPE
    assert decode(scale=scale, ks=(1 << 40) * 23, vs=(1 << 40) * 24) == ESHAPE
    assert prefill(scale=scale) == ESHAPE
