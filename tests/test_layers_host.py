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
