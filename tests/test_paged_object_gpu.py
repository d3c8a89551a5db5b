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


def test_filled_rows_have_positions(cuda_device):
    """After fill, an eviction knows which tokens are the newest; appended tokens
    go on behind them, and a second fill starts afresh."""
    g = torch.Generator(device=cuda_device).manual_seed(1)
    c = _cache(2, 64, H=16, page_size=16)
    for lens in ([50, 7], torch.tensor([64, 1], device=cuda_device)):
        c.kv_pages.copy_(torch.randn(c.kv_pages.shape, generator=g, device=cuda_device))
        c.fill(lens)
        n = torch.as_tensor(lens).tolist()
        assert c.lens.tolist() == n and c.end_pos.tolist() == n and not c.acc.any()
        c.acc[0, :30] = 1.0  # the newest tokens weigh nothing
        c.evict(20, 8)
        assert c.lens.tolist() == [min(20, k) for k in n] and int(c.status.item()) == 0
        assert set(range(n[0] - 8, n[0])) <= set(c.pos[0, :20].tolist())
        assert c.pos[1, :n[1]].tolist() == list(range(n[1]))
        c.append(_rows(g, 2, 1))
        assert c.pos[0, 20].item() == n[0] and c.pos[1, n[1]].item() == n[1]


@pytest.mark.parametrize("graph", [False, True])
def test_sequences_that_rest_keep_what_they_have(cuda_device, graph):
    """A padded batch: an empty sequence stays empty, a finished one is not
    written, the others grow."""
    g = torch.Generator(device=cuda_device).manual_seed(2)
    c = _cache(4, 64, H=16, page_size=16, out_dtype=torch.float32)
    c.kv_pages.fill_(float("nan"))
    for b, n in ((1, 5), (3, 17)):  # prompts of different lengths, one by one
        c.append(_rows(g, 4, n), active=torch.arange(4, device=cuda_device) == b)
    assert c.lens.tolist() == [0, 5, 0, 17]
    active = torch.tensor([False, True, True, False], device=cuda_device)
    x = _rows(g, 4, 1)
    run = lambda: c.append(x, active=active)
    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        cg = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(cg, stream=s):
            run()
        run = cg.replay
    for step in range(20):
        before, pos, acc = c.kv_pages.clone(), c.pos.clone(), c.acc.clone()
        x.copy_(_rows(g, 4, 1))
        c.acc.add_(1)
        run()
        torch.cuda.synchronize()
        assert c.lens.tolist() == [0, 6 + step, 1 + step, 17] and c.end_pos.tolist() == c.lens.tolist()
        acc += 1
        for b in (1, 2):
            s = int(c.lens[b]) - 1
            before.view(4, 64, D)[b, s], pos[b, s], acc[b, s] = x[b, 0], s, 0
        assert torch.equal(c.kv_pages.view(torch.int16), before.view(torch.int16))
        assert torch.equal(c.pos, pos) and torch.equal(c.acc, acc)
    out = c.attend(_rows(g, 4, 1, 16), SCALE)
    torch.cuda.synchronize()
    assert torch.all(out[0] == 0) and torch.all(c.lse[0] == float("-inf"))
    assert torch.isfinite(out).all() and int(c.status.item()) == 0


@pytest.mark.parametrize("T,H", [(4, 16), (7, 16), (3, 16), (2, 128), (40, 3), (5, 33)])
def test_prompt_chunks_and_single_tokens_through_one_object(cuda_device, T, H):
    """Calls with fewer tokens than the object was made for give the bits of an
    object made for that many."""
    g = torch.Generator(device=cuda_device).manual_seed(T + H)
    c = _cache(3, 3000, T=T, H=H, page_size=32)
    c.append(_rows(g, 3, 2900), active=torch.tensor([True, False, True], device=cuda_device))
    c.append(_rows(g, 3, T))
    for t in sorted({T, 1, 2, T - 1} - {0}, reverse=True):
        q = _rows(g, 3, t, H)
        one = _cache(3, 3000, T=t, H=H, page_size=32)
        for name in ("kv_pages", "lens", "end_pos", "acc", "pos"):
            getattr(one, name).copy_(getattr(c, name))
        assert one.workspace.numel() <= c.workspace.numel()
        out, want = c.attend(q, SCALE), one.attend(q, SCALE)
        assert out.shape == want.shape and torch.equal(out, want)
        assert torch.equal(c.collect(q, SCALE, 0.5), one.collect(q, SCALE, 0.5))
    assert int(c.status.item()) == 0
    from sparse_attention_04_b200 import _lib
    for bad in (_rows(g, 3, T + 1, H), _rows(g, 3, 0, H), _rows(g, 2, T, H), _rows(g, 3, T)):
        with pytest.raises(_lib.DSAError):
            c.attend(bad, SCALE)
        with pytest.raises(_lib.DSAError):
            c.collect(bad, SCALE)
