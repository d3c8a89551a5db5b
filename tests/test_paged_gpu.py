"""The paged latent cache on the GPU, each operator against its definition in
64 bits: append, attention over the whole cache, accumulated weights, eviction
plan and row moves, alone and in a run as a server uses them.

Tolerances.  u = 2^-24 (fp32) and e = 2^-8 (bf16) are half a step, relative.
A logit is a sum of 576 exact products: its fp32 error is at most
  d = scale * 576 * 2u * sum_i |q_i k_i|
(2u: the tensor core may truncate), and the exponent adds 4u * |x| + 2^-22 for
scaling, subtraction and ex2.  A weight p is then off by the factor
exp(2 (d + 4u|x| + 2^-22)) - 1 against another row's sum.  In the output every p
is rounded once to bf16 (e), sums in fp32 add n * 2u at most, a row that several
clusters share has its partials in fp16 (half a step 2^-11 of the value, or of
2^-14 times the largest of 32 columns where that is more), and a bf16 output is
rounded once more (e)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
U, E = 2.0 ** -24, 2.0 ** -8
D, DV = 576, 512
NAN = float("nan")


def _lib():
    from sparse_attention_04_b200 import _lib as L
    return L


class Cache:
    """Pages in shuffled order; everything no sequence holds is NaN, and the
    page lists end in numbers that would fault if they were followed."""

    def __init__(self, dev, lens, P, seed=0, cap=None, spare=2):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.dev, self.P, self.lens_py, self.g = dev, P, list(lens), g
        per = [-(-max(L, c) // P) for L, c in zip(lens, cap or lens)]
        n = sum(per) + spare
        order = torch.randperm(n, generator=g, device=dev).tolist()
        width = max(max(per), 1)
        table = [[(1 << 30) + 7] * width for _ in lens]
        at = 0
        for b, k in enumerate(per):
            table[b][:k] = order[at:at + k]
            at += k
        self.table = torch.tensor(table, dtype=torch.int32, device=dev)
        self.kv = torch.full((n, P, D), NAN, dtype=torch.bfloat16, device=dev)
        self.lens = torch.tensor(self.lens_py, dtype=torch.int32, device=dev)
        for b, L in enumerate(self.lens_py):
            if L:
                self.flat[self.rows(b, torch.arange(L, device=dev))] = torch.randn(
                    L, D, generator=g, device=dev).to(torch.bfloat16)

    @property
    def flat(self):
        return self.kv.view(-1, D)

    def rows(self, b, slots):
        return self.table[b].long()[slots // self.P] * self.P + slots % self.P

    def of(self, b, n=None):
        n = self.lens_py[b] if n is None else n
        return self.flat[self.rows(b, torch.arange(n, device=self.dev))].double()


def _status(dev):
    return torch.zeros(1, dtype=torch.int32, device=dev)


def _q(c, B, T, H, mul=1.0):
    return (torch.randn(B, T, H, D, generator=c.g, device=c.dev) * mul).to(torch.bfloat16)


def _attend(c, q, out_dtype=torch.bfloat16, scale=SCALE, ws_fill=0xff, lens=None):
    L = _lib()
    B, T, H, _ = q.shape
    out = torch.full((B, T, H, DV), NAN, dtype=out_dtype, device=c.dev)
    lse = torch.full((B, T, H), NAN, device=c.dev)
    ws = torch.full((max(16, L.paged_mla_workspace_size(B, T, H)),), ws_fill, dtype=torch.uint8, device=c.dev)
    st = _status(c.dev)
    L.paged_mla(q, c.kv, c.table, c.lens if lens is None else lens, scale, out, lse=lse, workspace=ws, status=st)
    torch.cuda.synchronize()
    return out, lse, int(st.item())


def _factor(scale, k, q, x):
    """exp(2 (d + 4u|x| + 2^-22)) - 1, by query row [H, 1]."""
    d = abs(scale) * D * 2 * U * (q.abs() @ k.abs().T).amax(1, keepdim=True)
    return (2 * (d + 4 * U * x.abs().amax(1, keepdim=True) + 2.0 ** -22)).exp() - 1


def _check_attention(c, q, out, lse, scale=SCALE, skip=None):
    """Every row of out and lse against softmax(scale q k) v in 64 bits; skip(b)
    gives the slots of sequence b that do not count."""
    B, T, H, _ = q.shape
    for b in range(B):
        k_all = c.of(b)
        for t in range(T):
            n = c.lens_py[b] - T + t + 1
            ok = torch.ones(max(n, 0), dtype=torch.bool, device=c.dev)
            if skip is not None and n > 0:
                ok &= ~skip(b)[:n]
            if n <= 0 or not bool(ok.any()):
                assert torch.all(out[b, t] == 0), (b, t)
                assert torch.all(lse[b, t] == float("-inf")), (b, t)
                continue
            k, qq = k_all[:n][ok], q[b, t].double()
            x = scale * (qq @ k.T)
            p = x.softmax(1)
            ref, spread = p @ k[:, :DV], p @ k[:, :DV].abs()
            f = _factor(scale, k, qq, x)
            top = spread.view(H, -1, 32).amax(2, keepdim=True).expand(-1, -1, 32).reshape(H, -1)
            tol = ((f + E + n * 2 * U) * spread + 2.0 ** -11 * torch.maximum(spread, 2.0 ** -14 * top)) * 1.01
            if out.dtype == torch.bfloat16:
                tol = tol + E * (ref.abs() + tol)
            err = (out[b, t].double() - ref).abs()
            assert torch.all(err <= tol), (b, t, n, float((err / (tol + 1e-300)).max()))
            ref_lse = x.logsumexp(1)
            tol_lse = (f[:, 0] + n * 2 * U) * 1.01 + 4 * U * (ref_lse.abs() + 30)
            err = (lse[b, t].double() - ref_lse).abs()
            assert torch.all(err <= tol_lse), (b, t, n, float((err / tol_lse).max()))


# ---------------------------------------------------------------- attention

LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 1000]


@pytest.mark.parametrize("P", [16, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("H", [1, 16, 27, 32, 33, 100, 128])
def test_attention_at_every_edge_of_pages_and_tiles(cuda_device, P, H):
    c = Cache(cuda_device, LENS, P, seed=P + H)
    q = _q(c, len(LENS), 1, H)
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)


@pytest.mark.parametrize("H", [1, 6, 7, 16, 64, 128])
@pytest.mark.parametrize("T", [2, 5])
def test_attention_of_several_new_tokens_is_causal(cuda_device, T, H):
    lens = [0, 1, T - 1, T, T + 1, 64, 66, 130, 777]
    c = Cache(cuda_device, lens, 32, seed=T)
    q = _q(c, len(lens), T, H)
    # the newest token's row is NaN: only the last query row may see it
    for b, L in enumerate(lens):
        if L > 1:
            c.flat[c.rows(b, torch.tensor([L - 1], device=c.dev))] = NAN
    out, lse, st = _attend(c, q)
    assert st == 0
    for b, L in enumerate(lens):
        if L > 1:
            assert torch.isnan(out[b, T - 1]).all() and torch.isnan(lse[b, T - 1]).all(), b
    # the rows before it, as if the newest token were not there yet
    short = [max(0, L - 1) if L > 1 else L for L in lens]
    c.lens_py = short
    for b, L in enumerate(lens):
        sub = slice(0, T - 1) if L > 1 else slice(0, T)
        one = Cache.__new__(Cache)
        one.__dict__.update(c.__dict__)
        one.lens_py, one.table = [short[b]], c.table[b:b + 1]
        _check_attention(one, q[b:b + 1, sub], out[b:b + 1, sub], lse[b:b + 1, sub])


@pytest.mark.parametrize("lens,H,T", [([40000], 128, 1), ([33000, 5, 0, 70001, 12345], 128, 1), ([9999] * 3, 128, 2),
                                      ([50021, 3, 800], 16, 1), ([20000] * 9, 40, 3), ([40000], 8, 3),
                                      ([33000, 5, 0, 70001, 12345], 16, 2), ([9999] * 150, 32, 1)])
def test_attention_of_long_rows_split_and_joined(cuda_device, lens, H, T):
    c = Cache(cuda_device, lens, 64, seed=len(lens))
    q = _q(c, len(lens), T, H)
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)
    again = _attend(c, q, ws_fill=0x7f)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("H", [128, 20, 5])
def test_attention_of_many_short_rows(cuda_device, H):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 400, (300,), generator=g).tolist()
    c = Cache(cuda_device, lens, 16, seed=1)
    q = _q(c, len(lens), 1, H)
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)


@pytest.mark.parametrize("H", [128, 9])
def test_attention_in_fp32_and_with_other_scales(cuda_device, H):
    lens = [1, 100, 3001]
    c = Cache(cuda_device, lens, 64, seed=5)
    for scale, mul in ((SCALE, 1.0), (-SCALE, 1.0), (0.0, 1.0), (1.0, 1.0), (SCALE, 30.0)):
        q = _q(c, 3, 1, H, mul)
        out, lse, st = _attend(c, q, torch.float32, scale)
        assert st == 0
        _check_attention(c, q, out, lse, scale)


@pytest.mark.parametrize("H", [128, 12, 32])
def test_attention_follows_a_rising_maximum(cuda_device, H):
    """Keys in order of growing logits: the running maximum moves in every tile."""
    c = Cache(cuda_device, [2000], 64, seed=6)
    q = _q(c, 1, 1, H)
    direction = q[0, 0].double().mean(0)
    k = torch.randn(2000, D, generator=c.g, device=c.dev, dtype=torch.float64) * 0.1
    k += torch.linspace(-60, 60, 2000, device=c.dev)[:, None] * direction / direction.norm()
    c.flat[c.rows(0, torch.arange(2000, device=c.dev))] = k.to(torch.bfloat16)
    for sign in (1.0, -1.0):
        qq = (q * sign).contiguous()
        out, lse, st = _attend(c, qq, torch.float32, 1.0)
        assert st == 0
        _check_attention(c, qq, out, lse, 1.0)


@pytest.mark.parametrize("H", [128, 16])
def test_attention_beyond_32_bit_offsets(cuda_device, H):
    """A pool of 4.6 G elements, the sequence on its last pages."""
    P, n = 64, 125000
    c = Cache(cuda_device, [1500], P, seed=7)
    kv = torch.empty((n, P, D), dtype=torch.bfloat16, device=c.dev)
    pages = c.table.shape[1]
    table = torch.arange(n - pages, n, dtype=torch.int32, device=c.dev)[None].contiguous()
    kv[table[0].long()] = c.kv[c.table[0].long()]
    c.kv, c.table = kv, table
    q = _q(c, 1, 1, H)
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)
    acc = torch.zeros(1, 1500, device=c.dev)
    _check_weights(c, q, lse, acc, 1.0)


@pytest.mark.parametrize("H", [128, 16])
def test_attention_takes_a_bad_page_as_masked(cuda_device, H):
    lens = [300, 300, 64, 5000]
    c = Cache(cuda_device, lens, 64, seed=8)
    bad = {0: [1], 2: [0], 3: [0, 40, 78]}
    for b, pages in bad.items():
        for i in pages:
            c.table[b, i] = -1 if i % 2 else c.kv.shape[0]

    def skip(b):
        s = torch.zeros(lens[b], dtype=torch.bool, device=c.dev)
        for i in bad.get(b, []):
            s[64 * i:64 * i + 64] = True
        return s

    q = _q(c, 4, 1, H)
    out, lse, st = _attend(c, q)
    assert st == 6  # DSA_ERR_BAD_INDEX
    c.table.clamp_(0, c.kv.shape[0] - 1)  # for the reference: any page, its slots are skipped
    for b in range(4):
        for i in bad.get(b, []):
            c.kv[c.table[b, i].long()] = torch.nan_to_num(c.kv[c.table[b, i].long()])
    _check_attention(c, q, out, lse, skip=skip)


def test_attention_takes_a_bad_length_as_empty(cuda_device):
    c = Cache(cuda_device, [100, 100, 100], 16, seed=9)
    q = _q(c, 3, 1, 16)
    lens = torch.tensor([100, -3, 7 * 16 + 1], dtype=torch.int32, device=c.dev)
    out, lse, st = _attend(c, q, lens=lens)
    assert st == 7  # DSA_ERR_BAD_OFFSETS
    c.lens_py = [100, 0, 0]
    _check_attention(c, q, out, lse)


def test_attention_without_lse_and_status_on_a_side_stream(cuda_device):
    L = _lib()
    c = Cache(cuda_device, [700, 30], 32, seed=10)
    q = _q(c, 2, 1, 128)
    ref, lse, _ = _attend(c, q)
    out = torch.empty_like(ref)
    ws = torch.empty(max(16, L.paged_mla_workspace_size(2, 1, 128)), dtype=torch.uint8, device=c.dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    L.paged_mla(q, c.kv, c.table, c.lens, SCALE, out, workspace=ws, stream=s)
    with torch.cuda.stream(s):
        out2 = torch.empty_like(ref)
        L.paged_mla(q, c.kv, c.table, c.lens, SCALE, out2, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(out2, ref)


def test_attention_of_a_wider_page_table(cuda_device):
    """A page table cut out of a wider one, and a capacity far above the lengths."""
    c = Cache(cuda_device, [400, 1000], 64, seed=11, cap=[400, 1000])
    wide = torch.full((2, 4000), -5, dtype=torch.int32, device=c.dev)
    wide[:, 7:7 + c.table.shape[1]] = c.table
    q = _q(c, 2, 1, 128)
    ref, lse, _ = _attend(c, q)
    c.table = wide[:, 7:3000]
    out, lse2, st = _attend(c, q)
    assert st == 0 and torch.equal(out, ref) and torch.equal(lse, lse2)


@pytest.mark.parametrize("T,H,lens", [(300, 128, [300, 900]), (1000, 2, [1000, 1010, 3]), (129, 1, [400, 129]),
                                      (10, 13, [2000, 9, 64]), (65, 64, [65, 500])])
def test_attention_of_many_new_tokens(cuda_device, T, H, lens):
    """Prompts: several tiles of tokens per sequence, the last one partly filled,
    tokens before the sequence's first slot."""
    c = Cache(cuda_device, lens, 16, seed=T)
    q = _q(c, len(lens), T, H)
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)
    _, st = _check_weights(c, q, lse, torch.rand(len(lens), 2000, generator=c.g, device=c.dev), 0.5)
    assert st == 0


def test_attention_with_nothing_but_padding_and_with_more_sequences_than_clusters(cuda_device):
    c = Cache(cuda_device, [0] * 5, 16, seed=60)
    q = _q(c, 5, 1, 128)
    out, lse, st = _attend(c, q)
    assert st == 0 and torch.all(out == 0) and torch.all(lse == float("-inf"))
    lens = [0, 1] * 1000 + [4000]
    c = Cache(cuda_device, lens, 16, seed=61)
    q = _q(c, len(lens), 1, 16)
    out, lse, st = _attend(c, q)
    assert st == 0
    some = [0, 1, 2, 999, 1000, 1999, 2000]
    one = Cache.__new__(Cache)
    for b in some:
        one.__dict__.update(c.__dict__)
        one.lens_py, one.table = [lens[b]], c.table[b:b + 1]
        _check_attention(one, q[b:b + 1], out[b:b + 1], lse[b:b + 1])
    # every sequence of one slot returns that slot's row, rounded
    ones = torch.arange(1, 2000, 2, device=c.dev)
    rows = c.flat[c.table[ones, 0].long() * 16][:, None, None, :DV]
    assert torch.equal(out[ones], rows.expand(-1, 1, 16, -1))


@pytest.mark.parametrize("H,T", [(128, 1), (16, 4), (16, 2), (3, 1)])
def test_attention_over_infinities_and_huge_values(cuda_device, H, T):
    """Values near the type's largest in the cache, infinities in slots behind the
    end; nothing overflows on the way (partials are scaled)."""
    c = Cache(cuda_device, [9000, 100], 64, seed=62)
    c.kv.copy_(torch.where(c.kv.isnan(), torch.full_like(c.kv, float("inf")), c.kv))
    for b, n in enumerate(c.lens_py):
        rows = c.rows(b, torch.arange(n, device=c.dev))
        c.flat[rows, :256] *= 2.0 ** 100
        c.flat[rows, 256:512] *= 2.0 ** -100
        c.flat[rows, 300:304] *= 2.0 ** 12  # beside much smaller columns
    q = _q(c, 2, T, H)
    q[..., :512] = 0  # the logits come from the last 64 columns
    out, lse, st = _attend(c, q, torch.float32)
    assert st == 0
    _check_attention(c, q, out, lse)


# ---------------------------------------------------------------- weights

def _check_weights(c, q, lse, acc, decay, skip=None, in_place=False):
    L = _lib()
    B, T, H, _ = q.shape
    st = _status(c.dev)
    before = acc.clone()
    out = acc if in_place else torch.full_like(acc, -7.0)
    L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=None if in_place else out, decay=decay, status=st)
    torch.cuda.synchronize()
    for b in range(B):
        n_all = c.lens_py[b]
        k = c.of(b)
        ref = before[b, :n_all].double() * decay
        tol = 4 * U * ref.abs()
        for t in range(T):
            n = n_all - T + t + 1
            if n <= 0:
                continue
            x = SCALE * (q[b, t].double() @ k[:n].T)
            w = (x - lse[b, t].double()[:, None]).exp()
            f = _factor(SCALE, k[:n], q[b, t].double(), x) + 8 * U * lse[b, t].double().abs()[:, None] + H * T * 2 * U
            if skip is not None:
                w[:, skip(b)[:n]] = 0
            ref[:n] += w.sum(0)
            tol[:n] += (w * f).sum(0) * 1.01
        err = (out[b, :n_all].double() - ref).abs()
        assert torch.all(err <= tol + 4 * U * ref.abs() + 1e-30), (b, float((err / (tol + 1e-30)).max()))
        behind = before[b, n_all:] if in_place else torch.full_like(before[b, n_all:], -7.0)
        assert torch.equal(out[b, n_all:], behind), b
    return out, int(st.item())


@pytest.mark.parametrize("P,H,T", [(16, 128, 1), (48, 16, 1), (64, 128, 2), (64, 1, 1), (128, 100, 1), (80, 64, 2),
                                   (32, 40, 5), (256, 127, 3)])
def test_weights_at_every_edge(cuda_device, P, H, T):
    c = Cache(cuda_device, LENS, P, seed=P + H + T)
    q = _q(c, len(LENS), T, H)
    _, lse, st = _attend(c, q)
    assert st == 0
    acc = torch.rand(len(LENS), 1004, generator=c.g, device=c.dev)
    out, st = _check_weights(c, q, lse, acc, 0.75)
    assert st == 0
    again, _ = _check_weights(c, q, lse, acc, 0.75)
    assert torch.equal(out, again)
    _, st = _check_weights(c, q, lse, acc, 1.0, in_place=True)
    assert st == 0


def test_weights_of_long_rows_sum_to_the_number_of_query_heads(cuda_device):
    lens = [50000, 3, 20001]
    c = Cache(cuda_device, lens, 64, seed=12)
    q = _q(c, 3, 1, 128)
    _, lse, _ = _attend(c, q)
    L = _lib()
    out = torch.zeros(3, 50000, device=c.dev)
    L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, None, acc_out=out)
    # each head's weights sum to 1, up to the factor in a weight and in lse
    assert torch.all((out.double().sum(1) - 128).abs() <= 128 * 4e-3)
    _check_weights(c, q, lse, out, 0.0)


def test_weights_on_a_bad_page_only_decay(cuda_device):
    c = Cache(cuda_device, [200, 130], 64, seed=13)
    q = _q(c, 2, 1, 32)
    _, lse, _ = _attend(c, q)
    keep = c.table.clone()
    c.table[0, 1] = -1
    L, acc = _lib(), torch.rand(2, 200, generator=c.g, device=c.dev)
    out, st = torch.empty_like(acc), _status(c.dev)
    L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=out, decay=0.5, status=st)
    assert int(st.item()) == 6
    c.table = keep
    good = torch.empty_like(acc)
    L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=good, decay=0.5)
    assert torch.equal(out[0, 64:128], acc[0, 64:128] * 0.5)
    assert torch.equal(out[0, :64], good[0, :64]) and torch.equal(out[0, 128:], good[0, 128:])
    assert torch.equal(out[1, :130], good[1, :130])


@pytest.mark.parametrize("B", [31, 128, 129, 330])
def test_weights_of_many_sequences(cuda_device, B):
    """Few and many sequences find their parts in two ways; a bad length among
    them is reported and empty."""
    g = torch.Generator().manual_seed(B)
    lens = (torch.randint(0, 500, (B,), generator=g) * (torch.rand(B, generator=g) < 0.8)).tolist()
    c = Cache(cuda_device, lens, 32, seed=B)
    q = _q(c, B, 1, 8)
    out, lse, st = _attend(c, q)
    assert st == 0
    acc = torch.rand(B, 512, generator=c.g, device=c.dev)
    _, st = _check_weights(c, q, lse, acc, 0.5)
    assert st == 0
    c.lens[B // 2], c.lens_py[B // 2] = -4, 0
    _, st = _check_weights(c, q, lse, acc, 0.5)
    assert st == 7


def test_weights_of_an_empty_row_add_nothing(cuda_device):
    """lse = -inf: the row saw nothing."""
    c = Cache(cuda_device, [64], 64, seed=14)
    q = _q(c, 1, 1, 4)
    lse = torch.full((1, 1, 4), float("-inf"), device=c.dev)
    acc = torch.rand(1, 64, generator=c.g, device=c.dev)
    out = torch.empty_like(acc)
    _lib().paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, acc, acc_out=out)
    assert torch.equal(out, acc)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("P", [16, 48])
def test_append_writes_exactly_the_last_slots(cuda_device, T, P):
    L = _lib()
    lens = [T, T + 1, 0, 100, 47 + T, max(0, T - 1)]
    c = Cache(cuda_device, lens, P, seed=T + P)
    B = len(lens)
    new = _q(c, B, T, 1)[:, :, 0].contiguous()
    acc = torch.rand(B, 148, generator=c.g, device=c.dev)
    pos = torch.randint(0, 99, (B, 148), generator=c.g, device=c.dev, dtype=torch.int32)
    end = torch.randint(1000, 2000, (B,), generator=c.g, device=c.dev, dtype=torch.int32)
    want, acc_w, pos_w = c.kv.clone(), acc.clone(), pos.clone()
    for b, n in enumerate(lens):
        if n >= T:
            s = torch.arange(n - T, n, device=c.dev)
            want.view(-1, D)[c.rows(b, s)] = new[b]
            acc_w[b, n - T:n] = 0
            pos_w[b, n - T:n] = torch.arange(T, device=c.dev, dtype=torch.int32) + int(end[b]) - T
    st = _status(c.dev)
    L.paged_append(new, c.kv, c.table, c.lens, acc=acc, pos=pos, end_pos=end, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == (7 if 0 < T - 1 else 0)  # the last sequence is shorter than T
    assert torch.equal(c.kv.view(torch.int16), want.view(torch.int16))
    assert torch.equal(acc, acc_w) and torch.equal(pos, pos_w)


def test_append_without_slot_arrays_and_with_a_bad_page(cuda_device):
    L = _lib()
    c = Cache(cuda_device, [64, 65], 64, seed=15)
    c.table[1, 1] = -2
    new = _q(c, 2, 2, 1)[:, :, 0].contiguous()
    want = c.kv.clone()
    want.view(-1, D)[c.rows(0, torch.tensor([62, 63], device=c.dev))] = new[0]
    want.view(-1, D)[c.rows(1, torch.tensor([63], device=c.dev))] = new[1, :1]
    st = _status(c.dev)
    L.paged_append(new, c.kv, c.table, c.lens, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 6
    assert torch.equal(c.kv.view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------- plan and moves

def _plan_ref(acc, pos, lens, end, budget, recent):
    """(kept slots, [(dst, src)]) per sequence, from the definition."""
    res = []
    for b, n_all in enumerate(lens):
        n = min(n_all, budget)
        a, p = acc[b, :n_all].double().cpu().tolist(), None if pos is None else pos[b].tolist()
        prot = [recent > 0 and p[s] >= end[b] - recent for s in range(n_all)]
        val = [(float("-inf"), 0) if x != x else (x, 1) for x in a]  # NaN below -inf
        order = sorted(range(n_all), key=lambda s: (not prot[s], -val[s][0], -val[s][1], s))
        kept = set(order[:n])
        holes = [s for s in range(n) if s not in kept]
        tail = [s for s in range(n, n_all) if s in kept]
        res.append((kept, list(zip(holes, tail))))
    return res


def _run_plan(acc, pos, lens, end, budget, recent, width=None):
    L, dev, B = _lib(), acc.device, acc.shape[0]
    width = width or max(1, min(budget, max(0, max(lens) - budget)))
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    new, n = t([-9] * B), t([-9] * B)
    dst = torch.full((B, width), -9, dtype=torch.int32, device=dev)
    src = torch.full((B, width), -9, dtype=torch.int32, device=dev)
    st = _status(dev)
    L.evict_plan(acc, pos, t(lens), t(end) if end is not None else None, budget, recent, new, n, dst, src, status=st)
    torch.cuda.synchronize()
    return new.tolist(), n.tolist(), dst.tolist(), src.tolist(), int(st.item())


def _check_plan(acc, pos, lens, end, budget, recent, width=None):
    new, n, dst, src, st = _run_plan(acc, pos, lens, end, budget, recent, width)
    assert st == 0
    for b, (kept, moves) in enumerate(_plan_ref(acc, pos, lens, end, budget, recent)):
        assert new[b] == min(lens[b], budget) and n[b] == len(moves), b
        got = list(zip(dst[b], src[b]))
        assert got[:len(moves)] == moves, b
        assert all(g == (-1, -1) for g in got[len(moves):]), b


@pytest.mark.parametrize("ld,budget,recent", [(64, 1, 0), (64, 31, 31), (1024, 500, 100), (1024, 1023, 1), (8192, 4096, 0),
                                              (8196, 100, 7), (20000, 9999, 512), (70000, 33333, 33333)])
def test_plan_keeps_the_heaviest_and_the_newest(cuda_device, ld, budget, recent):
    g = torch.Generator(device=cuda_device).manual_seed(ld + budget)
    lens = [ld, 0, 1, min(ld, budget), min(ld, budget + 1), ld - 3, ld // 2]
    B = len(lens)
    acc = torch.randn(B, ld, generator=g, device=cuda_device).mul_(3).exp_()
    pos = torch.stack([torch.randperm(ld, generator=g, device=cuda_device) for _ in range(B)]).to(torch.int32)
    _check_plan(acc, pos, lens, [ld] * B, budget, recent, width=min(budget, ld))


@pytest.mark.parametrize("ld", [256, 12000])
def test_plan_of_ties_and_special_values(cuda_device, ld):
    g = torch.Generator(device=cuda_device).manual_seed(ld)
    vals = torch.tensor([0.0, -0.0, 1.0, 1.0, float("inf"), float("-inf"), NAN, -1.0, 1e-45, 3e38], device=cuda_device)
    acc = vals[torch.randint(0, 10, (5, ld), generator=g, device=cuda_device)]
    acc[1] = 0.5          # all alike
    acc[2] = 0.0
    acc[2, ::2] = -0.0
    acc[3] = NAN
    pos = torch.arange(ld, dtype=torch.int32, device=cuda_device).repeat(5, 1)
    for budget, recent in ((ld // 3, 0), (ld // 3, ld // 4), (ld - 1, 5), (1, 1)):
        _check_plan(acc, pos, [ld, ld, ld - 1, ld, ld], [ld] * 5, budget, recent)
    _check_plan(acc, None, [ld] * 5, None, ld // 2, 0)


@pytest.mark.parametrize("ld", [8, 1000, 20000, 400000])
def test_plan_with_more_protected_slots_than_the_budget(cuda_device, ld):
    """Positions that repeat, or an end_pos that lags: the protected slots
    compete by weight, NaN last, then by slot; the others stay out."""
    g = torch.Generator(device=cuda_device).manual_seed(ld)
    vals = torch.tensor([0.0, -0.0, 2.5, -1.0, float("inf"), float("-inf"), NAN, 3e38], device=cuda_device)
    acc = torch.randn(4, ld, generator=g, device=cuda_device).exp_()
    acc[1] = vals[torch.randint(0, 8, (ld,), generator=g, device=cuda_device)]
    acc[2] = NAN
    pos = torch.randint(0, 10, (4, ld), generator=g, device=cuda_device, dtype=torch.int32)
    pos[3] = 9  # every slot
    for budget, recent in ((max(2, ld // 8), 2), (ld // 2, min(6, ld // 2)), (1, 1)):
        _check_plan(acc, pos, [ld, ld, ld, ld - 1], [10] * 4, budget, recent)


def test_plan_of_a_sequence_beyond_shared_memory(cuda_device):
    ld = 500000  # more keys than eight CTAs hold on chip
    g = torch.Generator(device=cuda_device).manual_seed(1)
    acc = torch.rand(1, ld, generator=g, device=cuda_device)
    _check_plan(acc, None, [ld - 1], None, 300000, 0)


def test_plan_refuses_what_does_not_fit(cuda_device):
    acc = torch.rand(3, 64, device=cuda_device)
    new, n, dst, src, st = _run_plan(acc, None, [65, -1, 64], None, 32, 0, width=32)
    assert st == 7 and new[:2] == [65, -1] and n[:2] == [0, 0] and set(dst[0] + dst[1] + src[0] + src[1]) == {-1}
    assert new[2] == 32
    acc = torch.arange(64, device=cuda_device, dtype=torch.float32).repeat(3, 1)  # the last 32 stay: 32 moves
    new, n, dst, src, st = _run_plan(acc, None, [64, 20, 33], None, 32, 0, width=31)
    assert st == 7 and new == [64, 20, 32] and n == [0, 0, 1] and set(dst[0]) == {-1}


@pytest.mark.parametrize("P", [16, 48])
def test_moves_carry_rows_weights_and_positions(cuda_device, P):
    L = _lib()
    lens = [500, 0, 301, 1000]
    c = Cache(cuda_device, lens, P, seed=20)
    g, B, ld = c.g, 4, 1000
    acc = torch.rand(B, ld, generator=g, device=c.dev)
    pos = torch.randint(0, 9999, (B, ld), generator=g, device=c.dev, dtype=torch.int32)
    budget = 300
    moves = [m for _, m in _plan_ref(acc, pos, lens, [0] * B, budget, 0)]
    width = max(map(len, moves)) + 3
    dst = torch.full((B, width), 1 << 30, dtype=torch.int32, device=c.dev)  # behind n_moves: never looked at
    src = torch.full((B, width), 1 << 30, dtype=torch.int32, device=c.dev)
    want, acc_w, pos_w = c.kv.clone(), acc.clone(), pos.clone()
    for b, m in enumerate(moves):
        if m:
            d, s = (torch.tensor(v, device=c.dev) for v in zip(*m))
            dst[b, :len(m)], src[b, :len(m)] = d.int(), s.int()
            want.view(-1, D)[c.rows(b, d)] = c.flat[c.rows(b, s)]
            acc_w[b, d], pos_w[b, d] = acc[b, s], pos[b, s]
    n = torch.tensor([len(m) for m in moves], dtype=torch.int32, device=c.dev)
    st = _status(c.dev)
    L.paged_move(c.kv, c.table, n, dst, src, acc=acc, pos=pos, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(c.kv.view(torch.int16), want.view(torch.int16))
    assert torch.equal(acc, acc_w) and torch.equal(pos, pos_w)


def test_moves_leave_bad_slots_and_pages_out(cuda_device):
    L = _lib()
    c = Cache(cuda_device, [128, 128], 64, seed=21)
    t = lambda v: torch.tensor(v, dtype=torch.int32, device=c.dev)
    want = c.kv.clone()
    want.view(-1, D)[c.rows(0, torch.tensor([3], device=c.dev))] = c.flat[c.rows(0, torch.tensor([100], device=c.dev))]
    st = _status(c.dev)
    L.paged_move(c.kv, c.table, t([4, 9]), t([[-1, 3, 5, 128], [0, 1, 2, 3]]), t([[90, 100, 1 << 20, 2], [0, 0, 0, 0]]), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) in (6, 7)
    assert torch.equal(c.kv.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("B", [3, 255, 256, 257, 700])
def test_moves_of_many_sequences_with_lists_of_every_length(cuda_device, B):
    """The lists of a group of sequences are dealt out together: none, one, many
    moves per sequence, one of them long, two with a number of moves that does
    not fit."""
    L = _lib()
    P, cap, ld_moves, ld = 16, 64, 32, 64
    c = Cache(cuda_device, [cap] * B, P, seed=B)
    g = torch.Generator().manual_seed(B)
    n = torch.randint(0, 4, (B,), generator=g)
    n[torch.randint(0, B, (B // 3,), generator=g)] = 0
    n[B // 2], n[B - 1] = ld_moves, 1
    dst = torch.full((B, ld_moves), -9, dtype=torch.int32)
    src = torch.full((B, ld_moves), -9, dtype=torch.int32)
    acc = torch.rand(B, ld, generator=g).to(c.dev)
    pos = torch.randint(0, 99999, (B, ld), generator=g, dtype=torch.int32).to(c.dev)
    want_kv, want_acc, want_pos = c.kv.clone(), acc.clone(), pos.clone()
    bad = {0: ld_moves + 1, 1: -1}
    for b in range(B):
        k = int(n[b])
        dst[b, :k] = torch.randperm(32, generator=g)[:k]
        src[b, :k] = 32 + torch.randperm(32, generator=g)[:k]
        if b in bad:
            n[b] = bad[b]
        elif k:
            d, s = dst[b, :k].long().to(c.dev), src[b, :k].long().to(c.dev)
            want_kv.view(-1, D)[c.rows(b, d)] = c.flat[c.rows(b, s)]
            want_acc[b, d], want_pos[b, d] = acc[b, s], pos[b, s]
    st = _status(c.dev)
    L.paged_move(c.kv, c.table, n.int().to(c.dev), dst.to(c.dev), src.to(c.dev), acc=acc, pos=pos, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 7
    assert torch.equal(c.kv.view(torch.int16), want_kv.view(torch.int16))
    assert torch.equal(acc, want_acc) and torch.equal(pos, want_pos)


# ---------------------------------------------------------------- as a server runs them

@pytest.mark.parametrize("graph", [False, True])
def test_decode_with_eviction_step_by_step(cuda_device, graph):
    """Append, attend, collect weights; over budget, plan and move.  Beside it
    the same in 64 bits on lists of rows; the plan's choice is taken from the
    device's own weights (a tie in 64 bits need not be one in 32)."""
    L, dev = _lib(), cuda_device
    B, H, P, budget, recent, ld = 3, 128, 16, 96, 8, 112
    c = Cache(dev, [90, 40, 0], P, seed=30, cap=[ld] * 3)
    lens, end = c.lens, c.lens.clone()
    acc, pos = torch.zeros(B, ld, device=dev), torch.zeros(B, ld, dtype=torch.int32, device=dev)
    pos[:] = torch.arange(ld, device=dev, dtype=torch.int32)
    caches = [c.of(b) for b in range(B)]  # rows by slot
    weights = [torch.zeros(n, dtype=torch.float64, device=dev) for n in c.lens_py]
    places = [list(range(n)) for n in c.lens_py]
    new = torch.zeros(B, 1, D, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device=dev)
    out, lse = torch.empty(B, 1, H, DV, device=dev), torch.empty(B, 1, H, device=dev)
    ws = torch.empty(max(16, L.paged_mla_workspace_size(B, 1, H)), dtype=torch.uint8, device=dev)
    st = _status(dev)
    new_lens, n_moves = torch.empty_like(lens), torch.empty_like(lens)
    dst, src = (torch.empty(B, 8, dtype=torch.int32, device=dev) for _ in range(2))

    def step():
        lens.add_(1)
        end.add_(1)
        L.paged_append(new, c.kv, c.table, lens, acc=acc, pos=pos, end_pos=end, status=st)
        L.paged_mla(q, c.kv, c.table, lens, SCALE, out, lse=lse, workspace=ws, status=st)
        L.paged_weights(q, c.kv, c.table, lens, lse, SCALE, acc, decay=0.9, status=st)
        L.evict_plan(acc, pos, lens, end, budget, recent, new_lens, n_moves, dst, src, status=st)
        L.paged_move(c.kv, c.table, n_moves, dst, src, acc=acc, pos=pos, status=st)
        lens.copy_(new_lens)

    run = step
    if graph:
        state = [t.clone() for t in (lens, end, acc, pos, c.kv)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for t, v in zip((lens, end, acc, pos, c.kv), state):
            t.copy_(v)
        run = g.replay
    for i in range(25):
        new.copy_(torch.randn(B, 1, D, generator=c.g, device=dev))
        q.copy_(torch.randn(B, 1, H, D, generator=c.g, device=dev))
        run()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        for b in range(B):
            caches[b] = torch.cat([caches[b], new[b].double()])
            places[b].append(int(end[b]) - 1)
            n = caches[b].shape[0]
            k, qq = caches[b], q[b, 0].double()
            x = SCALE * (qq @ k.T)
            p = x.softmax(1)
            f = _factor(SCALE, k, qq, x)
            tol = (f + E + n * 2 * U) * (p @ k[:, :DV].abs()) * 1.01
            assert torch.all((out[b, 0].double() - p @ k[:, :DV]).abs() <= tol), (i, b)
            weights[b] = torch.cat([weights[b], torch.zeros(1, dtype=torch.float64, device=dev)]) * 0.9 + p.sum(0)
            if n > budget:
                assert int(new_lens[b]) == budget and n == budget + 1
                if int(n_moves[b]):
                    assert int(n_moves[b]) == 1
                    d = int(dst[b, 0])
                    assert int(src[b, 0]) == budget
                else:
                    d = budget  # the newest slot itself went
                assert places[b][d] < int(end[b]) - recent
                lightest = min(w for w, pl in zip(weights[b].tolist(), places[b]) if pl < int(end[b]) - recent)
                # both sides' weights carry the factor of one step ten times over at most (decay 0.9)
                assert float(weights[b][d]) <= lightest * (1 + 20 * float(f.max())), (i, b)
                if d < budget:
                    caches[b][d], weights[b][d], places[b][d] = caches[b][budget], weights[b][budget], places[b][budget]
                caches[b], weights[b], places[b] = caches[b][:budget], weights[b][:budget], places[b][:budget]
            m = caches[b].shape[0]
            assert int(lens[b]) == m
            c.lens_py[b] = m
            assert torch.equal(c.of(b), caches[b]), (i, b)
            assert pos[b, :m].tolist() == places[b], (i, b)


def test_cache_object_runs_the_same_calls(cuda_device):
    """api.PagedLatentCache against the calls it is made of, over a prompt and
    steps with eviction; the padded (empty) case is a cache that was never filled."""
    from sparse_attention_04_b200 import api
    L, dev, B, H = _lib(), cuda_device, 2, 16
    g = torch.Generator(device=dev).manual_seed(5)
    one = api.PagedLatentCache(B, 40, T=2, H=H, page_size=16, out_dtype=torch.float32)
    assert torch.all(one.attend(torch.ones(B, 2, H, D, dtype=torch.bfloat16, device=dev), SCALE) == 0)
    kv, lens, end = one.kv_pages.clone().zero_(), torch.zeros_like(one.lens), torch.zeros_like(one.lens)
    one.kv_pages.zero_()
    acc, pos = torch.zeros_like(one.acc), torch.zeros_like(one.pos)
    ws = torch.empty(L.paged_mla_workspace_size(B, 2, H), dtype=torch.uint8, device=dev)
    out, lse = torch.empty(B, 2, H, DV, device=dev), torch.empty(B, 2, H, device=dev)
    t = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=dev)
    new, n, dst, src = t(B), t(B), t(B, 20), t(B, 20)
    for step in range(25):
        x = torch.randn(B, 2, D, generator=g, device=dev).to(torch.bfloat16)
        q = torch.randn(B, 2, H, D, generator=g, device=dev).to(torch.bfloat16)
        got = one.append(x).attend(q, SCALE).clone()
        one.collect(q, SCALE, 0.9)
        one.evict(36, 4)
        lens += 2
        end += 2
        L.paged_append(x, kv, one.page_table, lens, acc=acc, pos=pos, end_pos=end)
        L.paged_mla(q, kv, one.page_table, lens, SCALE, out, lse=lse, workspace=ws)
        L.paged_weights(q, kv, one.page_table, lens, lse, SCALE, acc, decay=0.9)
        L.evict_plan(acc, pos, lens, end, 36, 4, new, n, dst, src)
        L.paged_move(kv, one.page_table, n, dst, src, acc=acc, pos=pos)
        lens.copy_(new)
        assert torch.equal(got, out) and torch.equal(one.acc, acc) and torch.equal(one.pos, pos), step
        assert torch.equal(one.lens, lens) and torch.equal(one.kv_pages, kv), step
    assert lens.tolist() == [36, 36] and int(one.status.item()) == 0


def test_cache_object_appended_to_beyond_its_slots(cuda_device):
    """40 slots in pages of 16 are 48; a sequence that grows past them is empty
    for every call, and the other one goes on."""
    from sparse_attention_04_b200 import api
    dev, H = cuda_device, 16
    c = api.PagedLatentCache(2, 40, H=H, page_size=16, out_dtype=torch.float32)
    assert c.slots == 48
    c.kv_pages.fill_(NAN)  # what was never written may hold anything
    c.lens[0] = 30
    c.kv_pages[:2] = 1.0
    g = torch.Generator(device=dev).manual_seed(6)
    for step in range(20):
        x = torch.randn(2, 1, D, generator=g, device=dev).to(torch.bfloat16)
        q = torch.randn(2, 1, H, D, generator=g, device=dev).to(torch.bfloat16)
        out = c.append(x).attend(q, SCALE)
        acc = c.collect(q, SCALE)
        torch.cuda.synchronize()
        full = 31 + step > 48
        assert int(c.status.item()) == (7 if full else 0), step
        assert torch.isfinite(out).all() and torch.isfinite(acc).all()
        assert bool((out[0] == 0).all()) == full and not (out[1] == 0).all()
    c.evict(24)
    assert c.lens.tolist() == [50, 20]


@pytest.mark.parametrize("H", [128, 16])
def test_attention_wait_runs_out_then_next_call_is_correct(cuda_device, H):
    """The timeout path (test hook): a bounded wait that never comes true ends the
    launch with DSA_ERR_TIMEOUT, and the launch after it is right."""
    L = _lib()
    c = Cache(cuda_device, [3000, 40, 0, 700], 64, seed=40)
    q = _q(c, 4, 1, H)
    L.debug_stall_attention(1, 5_000_000)
    try:
        _, _, st = _attend(c, q)
    finally:
        L.debug_stall_attention(0, 0)
    assert st == 5
    out, lse, st = _attend(c, q)
    assert st == 0
    _check_attention(c, q, out, lse)


@pytest.mark.parametrize("H", [64, 16])
def test_two_streams_and_two_graphs_with_a_workspace_each(cuda_device, H):
    """Calls that overlap: the results are those of the calls alone."""
    L = _lib()
    cs = [Cache(cuda_device, lens, 32, seed=50 + i) for i, lens in enumerate(([5000, 300], [77, 9000]))]
    qs = [_q(c, 2, 1, H) for c in cs]
    want = [_attend(c, q)[:2] for c, q in zip(cs, qs)]
    n = L.paged_mla_workspace_size(2, 1, H)
    got, graphs, streams = [], [], [torch.cuda.Stream() for _ in cs]
    for c, q, s in zip(cs, qs, streams):
        out, lse, ws = torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty(n, dtype=torch.uint8, device=c.dev)
        acc = torch.zeros(2, 9000, device=c.dev)
        got.append((out, lse, acc, ws))
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                L.paged_mla(q, c.kv, c.table, c.lens, SCALE, out, lse=lse, workspace=ws)
                L.paged_weights(q, c.kv, c.table, c.lens, lse, SCALE, None, acc_out=acc)
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, (out, lse, acc, _), w in zip(cs, got, want):
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
        alone = torch.zeros_like(acc)
        L.paged_weights(qs[cs.index(c)], c.kv, c.table, c.lens, lse, SCALE, None, acc_out=alone)
        assert torch.equal(acc, alone)


def test_first_call_of_a_process_may_be_captured():
    """Kernel attributes are set on the first call; that call may be inside a capture."""
    import subprocess
    import sys
    code = """
import torch
from sparse_attention_04_b200 import _lib as L
dev = torch.device("cuda:0")
kv = torch.randn(4, 64, 576, device=dev).to(torch.bfloat16)
table = torch.arange(4, dtype=torch.int32, device=dev).view(1, 4)
lens = torch.tensor([200], dtype=torch.int32, device=dev)
q = torch.randn(1, 1, 128, 576, device=dev).to(torch.bfloat16)
out, lse = torch.zeros(1, 1, 128, 512, device=dev), torch.zeros(1, 1, 128, device=dev)
acc = torch.zeros(1, 256, device=dev)
i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
new, n, dst, src = i(1), i(1), i(1, 128), i(1, 128)
ws = torch.empty(L.paged_mla_workspace_size(1, 1, 128), dtype=torch.uint8, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    L.paged_mla(q, kv, table, lens, 0.07, out, lse=lse, workspace=ws)
    L.paged_weights(q, kv, table, lens, lse, 0.07, acc)
    L.evict_plan(acc, None, lens, None, 100, 0, new, n, dst, src)
    L.paged_move(kv, table, n, dst, src, acc=acc)
g.replay()
torch.cuda.synchronize()
assert int(new) == 100 and abs(float(acc[0, :200].sum())) > 100 and float(out.abs().sum()) > 0
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
