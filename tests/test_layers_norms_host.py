"""Host-side checks of the norm layers and of attention with changed scores (no GPU work)."""
import pytest
import torch


def test_norm_layers_refuse_what_the_library_cannot_read():
    from sample_grad_norms_amd.layers import LayerNorm, RMSNorm
    with pytest.raises(ValueError, match="GPU tensor"):
        LayerNorm(8)(torch.zeros(2, 8))
    with pytest.raises(ValueError, match="GPU tensor"):
        RMSNorm(8)(torch.zeros(2, 8))
    m, r = LayerNorm(8, eps=1e-3, dtype=torch.bfloat16), RMSNorm(16)
    assert m.weight.dtype == m.bias.dtype == torch.bfloat16 and bool((m.weight == 1).all()) and bool((m.bias == 0).all())
    assert r.bias is None and r.rms and not m.rms and m.eps == 1e-3 and LayerNorm(8, bias=False).bias is None
    assert set(dict(r.named_parameters())) == {"weight"}


def test_calls_refuse_cpu_tensors():
    import sample_grad_norms_amd as dp
    x, w = torch.zeros(2, 3, 8), torch.ones(8)
    with pytest.raises(ValueError, match="GPU tensor"):
        dp.layernorm_forward(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        dp.layernorm_backward(x, x, w, None, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="GPU tensor"):
        dp.layernorm_norm(x, x)
    with pytest.raises(TypeError):
        dp.layernorm_forward(None, w)


def test_attention_refuses_slopes_that_want_a_gradient():
    from sample_grad_norms_amd.layers import attention
    q = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="detach"):
        attention(q, q, q, slopes=torch.zeros(4, requires_grad=True))
    with pytest.raises(ValueError, match="GPU tensor"):
        attention(q, q, q, cap=3.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_off_a_boundary_are_copied(dtype):
    from sample_grad_norms_amd.layers import _aligned
    buf = torch.arange(4096, dtype=torch.float32).to(dtype)
    for t in (buf[1:97].view(4, 24), buf[:96].view(24, 4).t(), buf[0].expand(3, 8)):
        r = _aligned(t)
        assert r.is_contiguous() and r.data_ptr() % 16 == 0 and r.data_ptr() != t.data_ptr() and torch.equal(r, t)
    t = buf[:96].view(4, 24)
    assert _aligned(t) is t
