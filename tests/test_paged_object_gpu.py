"""api.PagedLatentCache beyond the plain step: full caches, rows written without
append, batches in which some sequences rest."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
D = 576


def _cache(*args, **kw):
    from sparse_attention_04_b200 import api
    return api.PagedLatentCache(*args, **kw)


def _rows(g, *shape):
    return torch.randn(*shape, D, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("slots,P,n", [(40, 16, 24), (40, 16, 20), (1, 64, 32), (1, 64, 63), (33, 32, 32)])
def test_a_full_cache_is_cut_to_any_length(cuda_device, slots, P, n):
    """Slots come in whole pages; a cut of all of them moves min(n, L - n) rows
    when the last ones are the heaviest."""
    c = _cache(1, slots, H=16, page_size=P)
    L = c.slots
    c.kv_pages.copy_(torch.arange(L, device=cuda_device).view(c.kv_pages.shape[0], P, 1).expand_as(c.kv_pages))
    c.lens.fill_(L)
    c.acc.copy_(torch.arange(L, device=cuda_device)[None])
    c.evict(n)
    assert int(c.status.item()) == 0
    assert int(c.lens.item()) == n and int(c.n_moves.item()) == min(n, L - n)
    assert sorted(c.kv_pages.view(-1, D)[:n, 0].tolist()) == list(range(L - n, L))


def test_a_given_limit_of_moves_is_kept_and_reported(cuda_device):
    c = _cache(1, 64, H=16, page_size=64, max_moves=3)
    c.lens.fill_(64)
    c.acc.copy_(torch.arange(64, device=cuda_device)[None])
    c.evict(32)
    assert int(c.status.item()) == 7 and int(c.lens.item()) == 64
    c.status.zero_()
    c.evict(61)
    assert int(c.status.item()) == 0 and int(c.lens.item()) == 61
