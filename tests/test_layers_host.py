"""Host-side checks of the layers and of the step wrapper's embedding tables (no GPU work)."""
import pytest
import torch
from torch import nn

from workloads import llama_block as lb


class _Tied(nn.Module):
    def __init__(self, kind):
        super().__init__()
        from sample_grad_norms_amd.layers import Embedding
        self.emb = Embedding(16, 8)
        if kind == "linear":
            self.other = nn.Linear(8, 16, bias=False)
        elif kind == "embedding":
            self.other = nn.Embedding(16, 8)
        else:
            self.other = Embedding(16, 8)
        self.other.weight = self.emb.weight


@pytest.mark.parametrize("kind", ["linear", "embedding"])
def test_refuses_a_table_shared_with_another_kind_of_module(kind):
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    with pytest.raises(ValueError, match="shared with modules that are not"):
        RandomizedClipping(_Tied(kind), C=1.0, noise_multiplier=1.0)


def test_covers_tables_and_refuses_plain_embeddings():
    from sample_grad_norms_amd.dpsgd_rc import RandomizedClipping
    rc = RandomizedClipping(_Tied("table"), C=1.0, noise_multiplier=1.0)
    assert len(rc.params) == 1 and len(rc.tables) == 2
    with pytest.raises(ValueError, match="unclipped"):
        RandomizedClipping(nn.Sequential(nn.Embedding(4, 8), nn.Linear(8, 8, bias=False)), C=1.0, noise_multiplier=1.0)
    model = lb.build(1, layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16, vocab_in=20)
    rc = RandomizedClipping(model, C=1.0, noise_multiplier=1.0)
    assert rc.params[-1] is model.embed.weight and len(rc.params) == 9
    model.embed.weight.requires_grad_(False)
    assert len(RandomizedClipping(model, C=1.0, noise_multiplier=1.0).params) == 8


def test_the_stack_keeps_its_weights():
    """A table added to the stack leaves the linear weights of a seed as they were."""
    a = lb.build(5, layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16)
    b = lb.build(5, layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16, vocab_in=20)
    other = dict(b.named_parameters())
    assert all(torch.equal(p, other[n]) for n, p in a.named_parameters())
    with pytest.raises(ValueError, match="ops"):
        lb.LlamaStack(layers=1, dim=32, heads=2, kv_heads=1, hidden=64, vocab=16, ops="other")


def test_layers_refuse_cpu_tensors_and_wrong_shapes():
    from sample_grad_norms_amd.layers import Embedding, attention
    with pytest.raises(ValueError, match="GPU tensor"):
        Embedding(4, 8)(torch.zeros(2, dtype=torch.int64))
    q = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        attention(q, q, q)
    with pytest.raises(ValueError, match="no cu_seqlens"):
        attention(q, q, q, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="shapes"):
        attention(q, q[:1], q)
    with pytest.raises(ValueError, match="must be"):
        attention(q[0, 0], q[0, 0], q[0, 0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_the_library_cannot_read_are_copied(dtype):
    """Views off a 16-byte boundary, rows whose strides are, a lone row of any stride, and
    tokens too far apart; what can be read stays where it is."""
    from sample_grad_norms_amd.layers import _rows
    buf = torch.arange(4096, dtype=torch.float32).to(dtype)
    views = [buf[1:1 + 96].view(4, 3, 8), buf.as_strided((1, 2, 8), (9, 8, 1)), buf.as_strided((5, 1, 8), (16, 3, 1)),
             buf.as_strided((4, 2, 8), (24, 8, 1), 4 if dtype == torch.bfloat16 else 2), buf[:96].view(8, 4, 3).transpose(0, 2)[:, :, :8],
             buf[0].expand(2, 2, 8), torch.empty((1 << 22) + 8, dtype=dtype).as_strided((2, 1, 8), (1 << 22, 8, 1))]
    for t in views:
        r = _rows(t)
        assert r.is_contiguous() and r.data_ptr() % 16 == 0 and r.data_ptr() != t.data_ptr()
        assert all(s % (16 // r.element_size()) == 0 for s in r.stride()[:2]) and r.stride(2) == 1
        if t.numel() < 1000:
            assert torch.equal(r, t)
    for t in (buf[:96].view(4, 3, 8), buf[:192].view(4, 3, 16)[:, :, 8:], buf[:96].view(3, 4, 8).transpose(0, 1), buf[:8].expand(4, 3, 8)):
        assert _rows(t) is t
