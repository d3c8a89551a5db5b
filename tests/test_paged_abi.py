"""CPU checks of the paged-cache calls: every bad argument is refused on the
host before anything is launched, by the C entry points and by the binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from sparse_attention_04_b200 import build
    build.build()
    from sparse_attention_04_b200 import _lib
    return _lib


P = lambda x: ctypes.c_void_p(x)
A = 4096  # an aligned fake device address: the calls below must fail before any use


def _refused(f, base, changes):
    for where, value, code in changes:
        args = list(base)
        args[where] = value
        assert f(*args) == code, (where, value)


def test_append_refusals(L):
    #       kv_new lens   table  ld max B  T  page n_pages kv  acc   pos   end   ld_slots st stream
    base = [P(A), P(A), P(A), 8, 8, 2, 1, 64, 100, P(A), P(A), P(A), P(A), 512, None, None]
    _refused(L.lib.dsa_paged_append, base, [
        (0, None, 1), (1, None, 1), (2, None, 1), (9, None, 1), (0, P(A + 8), 1), (9, P(A + 2), 1), (2, P(A + 2), 1),
        (3, 7, 1), (4, 0, 1), (5, 0, 1), (6, 0, 1), (5, 1 << 25, 2), (7, 0, 1), (7, 24, 1), (7, -16, 1), (8, 0, 1),
        (8, 1 << 31, 1), (12, None, 1), (13, 0, 1), (13, 510, 1), (10, P(A + 4), 1), (11, P(A + 4), 1), (13, 1 << 31, 1),
        (1, P(A + 2), 1), (12, P(A + 1), 1), (14, P(A + 2), 1)])


def test_attention_refusals(L):
    #       q     kv    table  ld max lens  B  T  H   page n_pages scale out  dt lse  ws    bytes    st    stream
    base = [P(A), P(A), P(A), 8, 8, P(A), 2, 1, 128, 64, 100, 0.07, P(A), 0, None, P(A), 1 << 40, None, None]
    _refused(L.lib.dsa_paged_mla, base, [
        (0, None, 1), (1, None, 1), (2, None, 1), (5, None, 1), (12, None, 1), (0, P(A + 2), 1), (1, P(A + 8), 1),
        (12, P(A + 4), 1), (3, 7, 1), (6, 0, 1), (7, -1, 1), (8, 0, 1), (8, 129, 2), (6, (1 << 24) + 1, 2), (9, 8, 1),
        (9, 65, 1), (10, 0, 1), (10, 1 << 30, 1), (11, float("nan"), 1), (13, 1, 1), (13, 7, 1), (5, P(A + 2), 1), (14, P(A + 2), 1), (17, P(A + 3), 1)])
    need = L.paged_mla_workspace_size(2, 1, 128)
    if need:
        _refused(L.lib.dsa_paged_mla, base, [(15, None, 3), (15, P(A + 8), 3), (16, need - 1, 3)])
    assert L.paged_mla_workspace_size(0, 1, 128) == 0 and L.paged_mla_workspace_size(1, 1, 129) == 0


def test_weights_refusals(L):
    #       q     kv    table  ld max lens  lse  B  T  H   page n_pages scale decay acc  out   ld   st    stream
    base = [P(A), P(A), P(A), 8, 8, P(A), P(A), 2, 1, 128, 64, 100, 0.07, 1.0, None, P(A), 512, None, None]
    _refused(L.lib.dsa_paged_weights, base, [
        (0, None, 1), (1, None, 1), (2, None, 1), (5, None, 1), (6, None, 1), (15, None, 1), (0, P(A + 2), 1),
        (14, P(A + 4), 1), (15, P(A + 4), 1), (16, 0, 1), (16, 511, 1), (7, 0, 1), (8, 0, 1), (9, 0, 1), (9, 129, 2),
        (10, 40, 1), (11, 0, 1), (12, float("nan"), 1), (13, float("nan"), 1), (5, P(A + 1), 1), (6, P(A + 2), 1),
        (17, P(A + 2), 1)])


def test_plan_refusals(L):
    #       acc   pos   lens  end  B  ld  budget recent new  n     dst   src   ldm st    stream
    base = [P(A), P(A), P(A), P(A), 2, 512, 100, 10, P(A), P(A), P(A), P(A), 50, None, None]
    _refused(L.lib.dsa_evict_plan, base, [
        (0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (8, None, 1), (9, None, 1), (10, None, 1), (11, None, 1),
        (0, P(A + 4), 1), (1, P(A + 8), 1), (4, 0, 1), (5, 0, 1), (5, 510, 1), (5, (6 << 20) + 4, 2), (6, 0, 1), (7, -1, 1),
        (7, 101, 1), (12, 0, 1), (2, P(A + 2), 1), (3, P(A + 2), 1), (8, P(A + 1), 1), (9, P(A + 2), 1), (10, P(A + 2), 1),
        (11, P(A + 3), 1), (13, P(A + 2), 1)])


def test_move_refusals(L):
    #       kv    table ld max page n_pages n     dst   src   ldm B  acc  pos   ld   st    stream
    base = [P(A), P(A), 8, 8, 64, 100, P(A), P(A), P(A), 50, 2, P(A), P(A), 512, None, None]
    _refused(L.lib.dsa_paged_move, base, [
        (0, None, 1), (1, None, 1), (6, None, 1), (7, None, 1), (8, None, 1), (2, 7, 1), (3, 0, 1), (4, 50, 1), (5, 0, 1),
        (9, 0, 1), (10, 0, 1), (11, P(A + 4), 1), (12, P(A + 4), 1), (13, 0, 1), (13, 6, 1), (0, P(A + 4), 1), (6, P(A + 2), 1), (7, P(A + 2), 1),
        (8, P(A + 1), 1), (14, P(A + 2), 1)])


def test_binding_refuses_tensors_that_do_not_fit(L):
    """Shapes, types and places are checked before the library sees a pointer;
    CPU tensors are refused like any other wrong place."""
    kv = torch.zeros(4, 16, 576, dtype=torch.bfloat16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    lens = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 1, 8, 576, dtype=torch.bfloat16)
    out = torch.zeros(2, 1, 8, 512)
    acc = torch.zeros(2, 32)
    moves = torch.zeros(2, 4, dtype=torch.int32)
    for call in (lambda: L.paged_append(q[:, :, 0], kv, table, lens),
                 lambda: L.paged_mla(q, kv, table, lens, 1.0, out),
                 lambda: L.paged_mla(q, kv.float(), table, lens, 1.0, out),
                 lambda: L.paged_mla(q, kv[:, :, :512], table, lens, 1.0, out),
                 lambda: L.paged_weights(q, kv, table, lens, out[..., 0], 1.0, acc),
                 lambda: L.evict_plan(acc, None, lens, None, 4, 0, lens, lens, moves, moves),
                 lambda: L.evict_plan(acc, None, lens, None, 4, 0, lens, lens, moves[:1], moves[:1]),
                 lambda: L.paged_move(kv, table, lens, moves, moves)):
        with pytest.raises(L.DSAError):
            call()


def test_binding_checks_each_argument_against_the_others(L):
    dev = -1  # what get_device() says of CPU tensors
    t = torch.zeros(3, 5)
    assert L._arg(None, torch.float32, (3, 5), "x", dev) is None
    assert L._arg(t, torch.float32, (3, 5), "x", dev) == t.data_ptr()
    for bad, shape in ((t.double(), (3, 5)), (t, (3, 4)), (t.t(), (5, 3)), (t[:, :4], (3, 4))):
        with pytest.raises(L.DSAError):
            L._arg(bad, torch.float32, shape, "x", dev)
    assert L._arg(t[:, :4], torch.float32, (3, 4), "x", dev, rows=True) == t.data_ptr()
    assert L._row_pitch(t[:, :4]) == 5
    for bad, shape in ((t.t(), (5, 3)), (t[:1].expand(3, 5), (3, 5))):
        with pytest.raises(L.DSAError):
            L._arg(bad, torch.float32, shape, "x", dev, rows=True)
    with pytest.raises(L.DSAError):
        L._arg(t, torch.float32, (3, 5), "x", 0)
