"""More of the paged operators on the GPU: what their answers must not depend on,
sizes at the limits of the interface, bad pages in every part of a call."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
U = 2.0 ** -24
D, DV = 576, 512


def _lib():
    from sparse_attention_04_b200 import _lib as L
    return L


def _attend(q, kv, table, lens, out_dtype=torch.float32, scale=SCALE):
    L, (B, T, H, _) = _lib(), q.shape
    out = torch.full((B, T, H, DV), float("nan"), dtype=out_dtype, device=q.device)
    lse = torch.full((B, T, H), float("nan"), device=q.device)
    ws = torch.full((max(16, L.paged_mla_workspace_size(B, T, H)),), 0xff, dtype=torch.uint8, device=q.device)
    st = torch.zeros(1, dtype=torch.int32, device=q.device)
    L.paged_mla(q, kv, table, lens, scale, out, lse=lse, workspace=ws, status=st)
    torch.cuda.synchronize()
    return out, lse, int(st.item())


@pytest.mark.parametrize("H,T", [(128, 1), (40, 3), (16, 1), (16, 2), (1, 1)])
@pytest.mark.parametrize("lens", [[2048], [20000, 300, 64, 5000], [9000] * 5])
def test_fp32_output_keeps_fp32_sums(cuda_device, H, T, lens):
    """A query of zeros weighs every slot alike: P = 1, and the sums of whole
    numbers below 2^24 are exact in fp32 whatever their order, so that only the
    reciprocal and the product with it round (u each; one more for the
    reciprocal's own error).  Partial sums kept in fewer bits would show."""
    g = torch.Generator(device=cuda_device).manual_seed(H)
    per = [-(-n // 64) for n in lens]
    kv = torch.randint(129, 256, (sum(per), 64, D), generator=g, device=cuda_device).to(torch.bfloat16)
    table = torch.zeros(len(lens), max(per), dtype=torch.int32, device=cuda_device)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = torch.arange(at, at + k, device=cuda_device)
        at += k
    q = torch.zeros(len(lens), T, H, D, dtype=torch.bfloat16, device=cuda_device)
    out, lse, st = _attend(q, kv, table, torch.tensor(lens, dtype=torch.int32, device=cuda_device))
    assert st == 0
    for b, n_all in enumerate(lens):
        rows = kv[table[b, :per[b]].long()].view(-1, D)[:n_all, :DV].double()
        for t in range(T):
            n = n_all - T + t + 1
            assert n * 255 < 1 << 24
            ref = rows[:n].mean(0).expand(H, DV)
            err = (out[b, t].double() - ref).abs()
            assert torch.all(err <= 3 * U * ref), (b, t, float((err / ref).max() / U))
            assert torch.all((lse[b, t].double() - math.log(n)).abs() <= 8 * U * math.log(n))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [128, 40, 16])
def test_rows_whose_weights_all_vanish_do_not_depend_on_the_split(cuda_device, H, out_dtype):
    """Every score is -inf: lse = -inf, and out = sum 0 * v, NaN in the columns
    that hold infinities and 0 in the others, whether a row is split or not."""
    g = torch.Generator(device=cuda_device).manual_seed(3)
    kv = torch.randn(16, 64, D, generator=g, device=cuda_device).to(torch.bfloat16)
    kv[..., 5] = float("-inf")
    for B in (1, 3, 400):  # one row over the whole card, ..., whole rows
        table = torch.arange(16, dtype=torch.int32, device=cuda_device).expand(B, 16).contiguous()
        lens = torch.full((B,), 1000, dtype=torch.int32, device=cuda_device)
        q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device=cuda_device)
        q[..., 5] = 1.0
        out, lse, st = _attend(q, kv, table, lens, out_dtype)
        assert st == 0 and torch.all(lse == float("-inf"))
        assert torch.isnan(out[..., 5]).all(), B
        out[..., 5] = 0
        assert torch.all(out == 0), B


@pytest.mark.parametrize("H", [16, 128])
def test_two_sequences_of_a_billion_slots(cuda_device, H):
    """Page lists that name the same pages again and again: a worker's part takes
    longer than one wait may.  Zero scores: out is the mean of rows of ones,
    lse = log n.  An accumulator takes a chunk's sum at a time, 2^18 of them here,
    each addition off by 2u: 2^-5."""
    free, _ = torch.cuda.mem_get_info()
    n, P = (1 << 30) + 64 * 1000, 64
    if free < 8 * n // P * 4:
        pytest.skip("needs room for the page lists")
    table = (torch.arange(n // P, dtype=torch.int32, device=cuda_device) % 1024).expand(2, -1).contiguous()
    kv = torch.ones(1024, P, D, dtype=torch.bfloat16, device=cuda_device)
    lens = torch.full((2,), n, dtype=torch.int32, device=cuda_device)
    q = torch.zeros(2, 1, H, D, dtype=torch.bfloat16, device=cuda_device)
    out, lse, st = _attend(q, kv, table, lens)
    assert st == 0
    assert torch.all((out - 1).abs() <= 2.0 ** -5)
    assert torch.all((lse - math.log(n)).abs() <= 2.0 ** -5)


def test_a_batch_of_16_million_mostly_empty_sequences(cuda_device):
    """The largest batch: a worker writes 113 K empty rows before it comes to a
    chunk that its other warps have long been waiting for."""
    L, B = _lib(), 1 << 24
    free, _ = torch.cuda.mem_get_info()
    if free < B * 2 * (D + DV) + (4 << 30):
        pytest.skip("needs 41 GB")
    kv = torch.ones(16, 64, D, dtype=torch.bfloat16, device=cuda_device)
    table = torch.arange(16, dtype=torch.int32, device=cuda_device).expand(B, 16)[:, :11].contiguous()
    lens = torch.zeros(B, dtype=torch.int32, device=cuda_device)
    lens[-1], lens[1000] = 700, 1
    q = torch.zeros(B, 1, 1, D, dtype=torch.bfloat16, device=cuda_device)
    out = torch.full((B, 1, 1, DV), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    ws = torch.empty(L.paged_mla_workspace_size(B, 1, 1), dtype=torch.uint8, device=cuda_device)
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    L.paged_mla(q, kv, table, lens, SCALE, out, workspace=ws, status=st)
    assert int(st.item()) == 0
    assert torch.all(out[-1] == 1) and torch.all(out[1000] == 1)
    out[-1], out[1000] = 0, 0
    assert not out.view(torch.int32).any()


@pytest.mark.parametrize("H,T", [(128, 1), (20, 5)])
@pytest.mark.parametrize("lens", [[100], [60000, 7000], [3000, 40, 0, 700]])
def test_a_wait_that_runs_out_in_mid_stream_then_the_next_call_is_right(cuda_device, H, T, lens):
    """The test hook holds back the first product with the values: messages
    between the CTAs are under way when the waits run out."""
    L, B = _lib(), len(lens)
    g = torch.Generator(device=cuda_device).manual_seed(4)
    per = max(-(-n // 64) for n in lens)
    kv = torch.randn(B * per, 64, D, generator=g, device=cuda_device).to(torch.bfloat16)
    table = torch.arange(B * per, dtype=torch.int32, device=cuda_device).view(B, per)
    q = torch.randn(B, T, H, D, generator=g, device=cuda_device).to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    want = _attend(q, kv, table, n)
    assert want[2] == 0
    L.debug_stall_attention(3, 2_000_000, at_product=True)
    try:
        assert [_attend(q, kv, table, n)[2] for _ in range(3)] == [5, 5, 5]
    finally:
        L.debug_stall_attention(0, 0)
    for _ in range(2):
        out, lse, st = _attend(q, kv, table, n)
        assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("P,H,T", [(64, 100, 3), (16, 128, 2), (48, 7, 1), (128, 128, 1), (32, 16, 20)])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_beside_bad_pages_by_definition(cuda_device, P, H, T, in_place):
    """Slots on bad pages get decay * acc and count in nothing else, over every
    query tile of a sequence (up to three here)."""
    from test_paged_gpu import Cache, _attend as attend, _factor, _q

    class Holed(Cache):
        """Rows by the page lists as they were."""

        def rows(self, b, slots):
            return getattr(self, "good", self.table)[b].long()[slots // self.P] * self.P + slots % self.P

    lens = [700, 3 * P, 0, P, 5000, T]
    c = Holed(cuda_device, lens, P, seed=P + T)
    c.good = c.table.clone()
    bad = {0: [1, (700 - 1) // P], 1: [0, 1, 2], 3: [0], 4: [0, 7, 8, 4999 // P]}
    for b, pages in bad.items():
        for i in pages:
            c.table[b, i] = (-1, c.kv.shape[0], -(1 << 31), (1 << 31) - 1)[i % 4]

    def skip(b):
        s = torch.zeros(lens[b], dtype=torch.bool, device=c.dev)
        for i in bad.get(b, []):
            s[P * i:P * i + P] = True
        return s

    q = _q(c, len(lens), T, H)
    _, lse, st = attend(c, q)
    assert st == 6
    acc = torch.rand(len(lens), 5008, generator=c.g, device=c.dev)
    before = acc.clone()
    out = acc if in_place else torch.full_like(acc, -7.0)
    status = torch.zeros(1, dtype=torch.int32, device=c.dev)
    _lib().paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=None if in_place else out, decay=0.75,
                         status=status)
    assert int(status.item()) == 6
    for b, n_all in enumerate(lens):
        k, ref = c.of(b), before[b, :n_all].double() * 0.75
        tol = 4 * U * ref.abs()
        for t in range(T):
            n = max(0, n_all - T + t + 1)
            rows = ~torch.isinf(lse[b, t])  # the others saw nothing
            if n == 0 or not bool(rows.any()):
                assert n == 0 or bool(skip(b)[:n].all())
                continue
            qq, L = q[b, t].double()[rows], lse[b, t].double()[rows]
            x = SCALE * (qq @ k[:n].T)
            w = (x - L[:, None]).exp() * (~skip(b)[:n])
            # a logit as in the attention's tests, its exponent, and the sum over the rows
            f = _factor(SCALE, k[:n], qq, x) + 8 * U * L.abs()[:, None] + H * T * 2 * U
            ref[:n] += w.sum(0)
            tol[:n] += (w * f).sum(0) * 1.01
        err = (out[b, :n_all].double() - ref).abs()
        assert torch.all(err <= tol + 4 * U * ref.abs() + 1e-30), (b, float((err / (tol + 1e-30)).max()))
        assert torch.equal(out[b, :n_all][skip(b)], before[b, :n_all][skip(b)] * 0.75), b
        assert torch.equal(out[b, n_all:], before[b, n_all:] if in_place else torch.full_like(before[b, n_all:], -7.0)), b


@pytest.mark.parametrize("ld,budget,recent", [(512, 100, 10), (70000, 30001, 500), (6 << 20, 3000001, 1000)])
def test_plan_into_the_lengths_themselves_up_to_the_largest(cuda_device, ld, budget, recent):
    """new_lens is lens; the largest row has almost no keys on chip."""
    L = _lib()
    g = torch.Generator(device=cuda_device).manual_seed(ld)
    B = 2
    acc = torch.randint(0, max(4, ld // 3), (B, ld), generator=g, device=cuda_device).float()  # with ties
    pos = torch.stack([torch.randperm(ld, generator=g, device=cuda_device) for _ in range(B)]).to(torch.int32)
    old = [ld, ld - 77]
    lens = torch.tensor(old, dtype=torch.int32, device=cuda_device)
    end = torch.full((B,), ld, dtype=torch.int32, device=cuda_device)
    n_moves = torch.empty_like(lens)
    dst = torch.empty(B, budget, dtype=torch.int32, device=cuda_device)
    src, st = torch.empty_like(dst), torch.zeros(1, dtype=torch.int32, device=cuda_device)
    L.evict_plan(acc, pos, lens, end, budget, recent, lens, n_moves, dst, src, status=st)
    assert int(st.item()) == 0 and lens.tolist() == [budget] * B
    for b, n in enumerate(old):
        order = acc[b, :n].argsort(descending=True, stable=True)
        kept_always = pos[b, :n] >= ld - recent
        order = order[kept_always[order].int().argsort(descending=True, stable=True)]
        keep = torch.zeros(n, dtype=torch.bool, device=cuda_device)
        keep[order[:budget]] = True
        holes, tail = (~keep[:budget]).nonzero()[:, 0], budget + keep[budget:].nonzero()[:, 0]
        m = int(n_moves[b])
        assert m == len(holes) == len(tail)
        assert torch.equal(dst[b, :m].long(), holes) and torch.equal(src[b, :m].long(), tail)
        assert torch.all(dst[b, m:] == -1) and torch.all(src[b, m:] == -1)


def test_two_overlapping_calls_that_share_a_workspace_stay_inside_their_arrays(cuda_device):
    """A mistake of the caller: results are wrong, but nothing is read or written
    outside, and the calls are right again one after the other."""
    L = _lib()
    g = torch.Generator(device=cuda_device).manual_seed(5)
    jobs = []
    kv = torch.randn(400, 64, D, generator=g, device=cuda_device).to(torch.bfloat16)
    sizes = [([3000, 20, 0, 9000], 128, 1), ([25000], 16, 1), ([700] * 30, 40, 3)]
    ws = torch.zeros(max(L.paged_mla_workspace_size(len(n), T, H) for n, H, T in sizes), dtype=torch.uint8, device=cuda_device)
    for n, H, T in sizes:
        B = len(n)
        table = torch.randint(0, 400, (B, 400), generator=g, device=cuda_device, dtype=torch.int32)
        q = torch.randn(B, T, H, D, generator=g, device=cuda_device).to(torch.bfloat16)
        lens = torch.tensor(n, dtype=torch.int32, device=cuda_device)
        want = _attend(q, kv, table, lens)
        # guard rows before and behind out and lse
        out = torch.full((3, B, T, H, DV), 7.0, device=cuda_device)
        lse = torch.full((3, B, T, H), 7.0, device=cuda_device)
        st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
        run = lambda q=q, table=table, lens=lens, out=out, lse=lse, st=st: L.paged_mla(
            q, kv, table, lens, SCALE, out[1], lse=lse[1], workspace=ws, status=st)
        s, cg = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(cg, stream=s):
            for _ in range(10):
                run()
        jobs.append((s, cg, run, want, out, lse, st))
    for _ in range(50):
        for s, cg, *_rest in jobs:
            with torch.cuda.stream(s):
                cg.replay()
    torch.cuda.synchronize()
    for _, _, run, want, out, lse, st in jobs:
        assert int(st.item()) in (0, 3)
        st.zero_()
        for t in (out, lse):
            assert torch.all(t[0] == 7) and torch.all(t[2] == 7)
        run()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and torch.equal(out[1], want[0]) and torch.equal(lse[1], want[1])


@pytest.mark.parametrize("H,T", [(128, 1), (100, 3)])
def test_weights_wait_runs_out_then_the_next_call_is_right(cuda_device, H, T):
    """The test hook on the accumulated weights: a launch that gives up reports it."""
    from test_paged_gpu import Cache, _attend as attend, _check_weights, _q
    L = _lib()
    c = Cache(cuda_device, [9000, 40, 0, 700], 64, seed=40)
    q = _q(c, 4, T, H)
    _, lse, st = attend(c, q)
    assert st == 0
    acc = torch.rand(4, 9000, generator=c.g, device=c.dev)
    L.debug_stall_attention(2, 2_000_000)
    try:
        for _ in range(2):
            out, status = torch.zeros_like(acc), torch.zeros(1, dtype=torch.int32, device=c.dev)
            L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=out, status=status)
            assert int(status.item()) == 5
    finally:
        L.debug_stall_attention(0, 0)
    _, st = _check_weights(c, q, lse, acc, 0.5)
    assert st == 0


@pytest.mark.parametrize("lens,T", [([100], 1), ([148 * 64], 1), ([2 * 148 * 64], 2), ([3 * 148 * 64], 1), ([60000, 7000, 0], 2),
                                    ([3000, 40, 0, 700] * 40, 1)])
def test_few_rows_give_up_together_in_mid_stream(cuda_device, lens, T):
    """The same for tiles of few rows, whose eight consumer warps meet in every
    chunk: scores that rise from chunk to chunk make them wait for the product
    that never comes in each of the places where they can."""
    L, B, H = _lib(), len(lens), 16
    g = torch.Generator(device=cuda_device).manual_seed(6)
    per = max(-(-n // 64) for n in lens)
    kv = torch.randn(per, 64, D, generator=g, device=cuda_device)
    kv[..., 0] = torch.arange(per, device=cuda_device)[:, None]
    kv = kv.to(torch.bfloat16)
    table = torch.arange(per, dtype=torch.int32, device=cuda_device).expand(B, per).contiguous()
    q = torch.randn(B, T, H, D, generator=g, device=cuda_device)
    q[..., 0] = 160.0  # 11 and more per chunk after scaling: the maximum rises by more than 2^8
    q = q.to(torch.bfloat16)
    n = torch.tensor(lens, dtype=torch.int32, device=cuda_device)
    want = _attend(q, kv, table, n)
    assert want[2] == 0
    L.debug_stall_attention(20, 1_000_000, at_product=True)
    try:
        assert [_attend(q, kv, table, n)[2] for _ in range(20)] == [5] * 20
    finally:
        L.debug_stall_attention(0, 0)
    out, lse, st = _attend(q, kv, table, n)
    assert st == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])
