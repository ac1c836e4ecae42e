"""The generation example refuses prompts that it cannot process before anything reaches the GPU (none needed here)."""
import pytest
import torch

from bit_delta_tenant_gb300.decode_step import Shape, Tenants


@pytest.fixture
def tenants():
    """Two sequences' bookkeeping without the model: what is refused touches nothing else, a prompt of one token nothing more."""
    t = object.__new__(Tenants)
    t.shape, t.m, t.max_tokens = Shape(layers=0, vocab=100), 2, 8
    t.tokens, t.positions = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    t.page_table, t.variants = torch.zeros((2, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    t.embedding = None
    return t


@pytest.mark.parametrize("prompt", [[], [1] * 9, [100], [5, -1, 7], [3, 100, 4], [[1, 2], [3, 4]]])
def test_prompts(tenants, prompt):
    for given in (prompt, torch.tensor(prompt, dtype=torch.int64)):
        with pytest.raises(ValueError):
            tenants.prefill(0, given)
    assert tenants.tokens.tolist() == [0, 0]


@pytest.mark.parametrize("i", [-1, 2])
def test_sequences(tenants, i):
    with pytest.raises(ValueError):
        tenants.prefill(i, [1])


def test_one_token(tenants):
    tenants.prefill(1, [99])
    assert tenants.tokens.tolist() == [0, 99] and tenants.positions.tolist() == [0, 0]
