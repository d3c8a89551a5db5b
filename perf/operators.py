"""Cases of the paged latent cache: the append of new tokens, the attention over
the whole cache, the accumulated attention weight per slot, the eviction plan
and the row moves that carry it out.

A sequence b owns the first lens[b] slots of its page list; slot s is row
page_table[b, s // P] * P + s % P of the page pool [n_pages, P, 576] (512 latent
|| 64 rope, bf16).  Its T newest tokens sit in its last T slots, and query row t
sees the slots s <= lens[b] - T + t.
"""
import math
import random

import numpy as np
import torch

own = False

D, DV = 576, 512
SCALE = 192 ** -0.5


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of four sequences: four rows, only latency counts
        dict(name="append_step", op="append", B=4, T=1, P=64, lo=100, hi=5000, lens_seed=1),
        # eight 4096-token prompts enter the cache at once
        dict(name="append_prompts", op="append", B=8, T=4096, P=64, lo=4096, hi=8192, lens_seed=2),
        # one short conversation, all 128 heads: the smallest attention call
        dict(name="attn_short", op="attn", B=1, T=1, H=128, P=64, lo=2048, hi=2048, lens_seed=3),
        # one 32K conversation, all 128 heads: one row split over the card
        dict(name="attn_32k", op="attn", B=1, T=1, H=128, P=64, lo=32768, hi=32768, lens_seed=4),
        # a tensor-parallel rank's 16 heads, two tokens a step, small pages, odd lengths
        dict(name="attn_h16", op="attn", B=24, T=2, H=16, P=16, lo=37, hi=30011, lens_seed=5),
        # the batched decode of 32 sequences between 8K and 128K
        dict(name="attn_batched", op="attn", B=32, T=1, H=128, P=64, lo=8192, hi=131072, lens_seed=6),
        # the weights of one token over a 32K cache
        dict(name="weights_32k", op="weights", B=1, T=1, H=128, P=64, lo=32768, hi=32768, decay=1.0, lens_seed=7),
        # a batch with odd lengths and a page size that is no power of two, decayed weights
        dict(name="weights_batched", op="weights", B=16, T=1, H=128, P=48, lo=1001, hi=65003, decay=0.98, lens_seed=8),
        # a full cache after every step: one token too many in each of eight sequences
        dict(name="plan_step", op="plan", B=8, lo=4097, hi=4097, budget=4096, recent=256, lens_seed=9),
        # long prompts cut to half a cache, ragged
        dict(name="plan_half", op="plan", B=32, lo=65536, hi=131072, budget=65536, recent=1024, lens_seed=10),
        # the moves after a step over budget by a few tokens
        dict(name="move_step", op="move", B=8, P=64, lo=4100, hi=4112, budget=4096, lens_seed=11),
        # the moves after long prompts were cut to half
        dict(name="move_half", op="move", B=8, P=64, lo=65536, hi=131072, budget=49152, lens_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "weights", "plan", "move"])
    P = rng.choice([16, 32, 48, 64, 80, 128, 256])
    seed = rng.randrange(1 << 20)
    if op == "append":
        B, T = _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
        T = max(1, min(T, 32768 // B))
        return dict(op=op, B=B, T=T, P=P, lo=T, hi=T + _log_int(rng, 1, 4096), lens_seed=seed)
    if op in ("attn", "weights"):
        B = _log_int(rng, 1, 48)
        hi = _log_int(rng, 1, 131072 if B == 1 else min(131072, (1 << 20) // B))
        H = rng.choice([1, 8, 16, 32, 64, 128, rng.randint(2, 127)])
        T = rng.choice([1, 1, 1, 2, 3]) if hi < 40000 else 1
        c = dict(op=op, B=B, T=T, H=H, P=P, lo=_log_int(rng, 1, hi), hi=hi, lens_seed=seed)
        if op == "weights":
            c["decay"] = rng.choice([1.0, 0.98, 0.5])
        return c
    if op == "plan":
        B = _log_int(rng, 1, 48)
        hi = _log_int(rng, 2, min(131072, (1 << 21) // B))
        budget = _log_int(rng, 1, hi)
        return dict(op=op, B=B, lo=_log_int(rng, 1, hi), hi=hi, budget=budget, recent=rng.randint(0, budget), lens_seed=seed)
    B = _log_int(rng, 1, 32)
    hi = _log_int(rng, 2, min(131072, (1 << 19) // B))
    return dict(op=op, B=B, P=P, lo=_log_int(rng, 1, hi), hi=hi, budget=_log_int(rng, 1, hi), lens_seed=seed)


def _lens(case):
    """The sequences' lengths: the case's own, whatever the seed of the values."""
    r = random.Random("%d %d %d %d" % (case["B"], case["lo"], case["hi"], case["lens_seed"]))
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _n_moves(case):
    """Moves per sequence: what evicting slots uniformly leaves to move, on average."""
    n = case["budget"]
    return [0 if L <= n else min(n, L - n, int(round((L - n) * (n / L)))) for L in _lens(case)]


def _max_moves(case):
    return max(1, min(case["budget"], max(0, case["hi"] - case["budget"])))


def _pitch(n):
    return -(-n // 4) * 4


# ---------------------------------------------------------------- inputs

def _pool(g, dev, lens, P, spare=3):
    """A pool of filled pages in shuffled order, and the sequences' page lists."""
    per = [-(-L // P) for L in lens]
    n = sum(per) + spare
    order = torch.randperm(n, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    table = torch.full((len(lens), max(max(per), 1)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(per):
        table[b, :k] = order[at:at + k]
        at += k
    return torch.empty((n, P, D), dtype=torch.bfloat16, device=dev).normal_(generator=g), table


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, B, lens_py = case["op"], case["B"], _lens(case)
    lens = torch.tensor(lens_py, dtype=torch.int32, device=dev)
    st = dict(case=case, lens=lens, lens_max=max(lens_py), status=torch.zeros(1, dtype=torch.int32, device=dev))
    if op in ("append", "attn", "weights", "move"):
        st["kv"], st["table"] = _pool(g, dev, lens_py, case["P"])
    if op in ("append", "plan", "move", "weights"):
        ld = _pitch(case["hi"])
        # summed attention weights: a few slots hold most, many hold next to nothing, fresh ones zero
        acc = torch.randn((B, ld), generator=g, device=dev).mul_(2).exp_()
        st["acc"] = torch.where(torch.rand((B, ld), generator=g, device=dev) < 0.1, torch.zeros_like(acc), acc)
    if op in ("append", "plan", "move"):
        # the slots' positions after earlier evictions: distinct, in no order, some tokens gone
        st["end_pos"] = lens + 1000
        keys = torch.rand((B, ld), generator=g, device=dev)
        keys = torch.where(torch.arange(ld, device=dev) < lens[:, None], keys, 2.0)
        pos = keys.argsort(1).argsort(1).to(torch.int32)
        st["pos"] = torch.where(pos >= (lens // 2)[:, None], pos + 1000, pos)
    if op == "append":
        st["new"] = torch.randn((B, case["T"], D), generator=g, device=dev).to(torch.bfloat16)
    if op in ("attn", "weights"):
        st["q"] = torch.randn((B, case["T"], case["H"], D), generator=g, device=dev).to(torch.bfloat16)
    if op == "attn":
        st["out"] = torch.empty((B, case["T"], case["H"], DV), dtype=torch.bfloat16, device=dev)
        st["lse"] = torch.empty((B, case["T"], case["H"]), dtype=torch.float32, device=dev)
    if op == "weights":
        # the attention call before left the rows' log-sum-exp
        k, limit = _rows(st), _limits(st)
        s = torch.matmul(st["q"].flatten(1, 2), k.transpose(1, 2)).float() * SCALE
        s.masked_fill_(torch.arange(s.shape[2], device=dev) >= limit[:, :, None], float("-inf"))
        st["lse"] = torch.logsumexp(s, 2).view(B, case["T"], case["H"]).contiguous()
        st["acc_out"] = st["acc"].clone()
    if op == "plan":
        m = _max_moves(case)
        st["new_lens"], st["n_moves"] = torch.empty_like(lens), torch.empty_like(lens)
        st["dst"] = torch.empty((B, m), dtype=torch.int32, device=dev)
        st["src"] = torch.empty((B, m), dtype=torch.int32, device=dev)
    if op == "move":
        m, n = _max_moves(case), case["budget"]
        st["n_moves"] = torch.tensor(_n_moves(case), dtype=torch.int32, device=dev)
        st["dst"] = torch.full((B, m), -1, dtype=torch.int32, device=dev)
        st["src"] = torch.full((B, m), -1, dtype=torch.int32, device=dev)
        for b, (L, k) in enumerate(zip(lens_py, _n_moves(case))):
            if k:
                st["dst"][b, :k] = torch.randperm(n, generator=g, device=dev)[:k].sort().values
                st["src"][b, :k] = n + torch.randperm(L - n, generator=g, device=dev)[:k].sort().values
    return st


# ---------------------------------------------------------------- plain forms

def _row_of(table, P, slots):
    """Pool rows of slots [B, n]; slots past the page list give some row of the pool."""
    page = table.gather(1, (slots // P).clamp_(0, table.shape[1] - 1).long()).long()
    return page.clamp_min_(0) * P + slots % P


def _rows(st):
    """The cache rows [B, lens_max, 576], zero behind each sequence's last."""
    slots = torch.arange(st["lens_max"], device=st["lens"].device).expand(len(st["lens"]), -1)
    rows = st["kv"].view(-1, D)[_row_of(st["table"], st["kv"].shape[1], slots)]
    return rows.masked_fill_((slots >= st["lens"][:, None])[:, :, None], 0)


def _limits(st):
    """Slots that query row (t, h) sees: [B, T * H]."""
    T, H = st["case"]["T"], st["case"]["H"]
    t = torch.arange(T * H, device=st["lens"].device) // H
    return (st["lens"][:, None] - T + t + 1).clamp_min(0)


def _logits(st, k):
    s = torch.matmul(st["q"].flatten(1, 2).float(), k.transpose(1, 2)).mul_(SCALE)
    return s.masked_fill_(torch.arange(s.shape[2], device=s.device) >= _limits(st)[:, :, None], float("-inf"))


def _attn(st):
    k = _rows(st).float()
    s = _logits(st, k)
    m = s.amax(2, keepdim=True)
    p = (s - torch.where(m == float("-inf"), torch.zeros_like(m), m)).exp_()
    l = p.sum(2, keepdim=True)
    o = torch.matmul(p, k[:, :, :DV]) / torch.where(l > 0, l, torch.ones_like(l))
    st["out"].copy_(o.view_as(st["out"]))
    st["lse"].copy_((m + l.log()).view_as(st["lse"]))
    return dict(out=st["out"], lse=st["lse"])


def _weights(st):
    s = _logits(st, _rows(st).float())
    w = (s - st["lse"].flatten(1, 2)[:, :, None]).exp_().masked_fill_(s == float("-inf"), 0)
    n = w.shape[2]
    held = torch.arange(n, device=w.device) < st["lens"][:, None]
    new = st["acc"][:, :n] * st["case"]["decay"] + w.sum(1)
    st["acc_out"][:, :n] = torch.where(held, new, st["acc_out"][:, :n])
    return st["acc_out"]


def _append(st):
    T = st["case"]["T"]
    slots = st["lens"][:, None] - T + torch.arange(T, device=st["lens"].device)
    st["kv"].view(-1, D)[_row_of(st["table"], st["kv"].shape[1], slots).flatten()] = st["new"].view(-1, D)
    st["acc"].scatter_(1, slots.long(), 0.0)
    st["pos"].scatter_(1, slots.long(), (slots + (st["end_pos"] - st["lens"])[:, None]).int())
    return dict(kv=st["kv"], acc=st["acc"], pos=st["pos"])


def _plan(st):
    c, acc, lens = st["case"], st["acc"], st["lens"][:, None]
    slot = torch.arange(acc.shape[1], device=acc.device).expand_as(acc)
    held = slot < lens
    kept_always = st["pos"] >= st["end_pos"][:, None] - c["recent"]
    # stable sorts, the least important key first: slot, weight, protection, presence
    order = torch.where(held, acc, float("-inf")).argsort(dim=1, descending=True, stable=True)
    rank_by = torch.where(held, 1 + kept_always.int(), 0).gather(1, order)
    order = order.gather(1, rank_by.argsort(dim=1, descending=True, stable=True))
    rank = torch.empty_like(order).scatter_(1, order, slot)
    n = lens.clamp_max(c["budget"])
    keep = held & (rank < n)
    hole, survivor = (slot < n) & ~keep, (slot >= n) & keep
    for mark, out in ((hole, st["dst"]), (survivor, st["src"])):
        at = torch.where(mark, mark.int().cumsum(1) - 1, out.shape[1])
        wide = torch.full((out.shape[0], out.shape[1] + 1), -1, dtype=torch.int32, device=out.device)
        out.copy_(wide.scatter_(1, at, slot.int())[:, :-1])
    st["new_lens"].copy_(n[:, 0])
    st["n_moves"].copy_(hole.sum(1))
    return dict(new_lens=st["new_lens"], n_moves=st["n_moves"], dst=st["dst"], src=st["src"])


def _move(st):
    P, flat = st["kv"].shape[1], st["kv"].view(-1, D)
    live = torch.arange(st["dst"].shape[1], device=flat.device) < st["n_moves"][:, None]
    b, i = live.nonzero(as_tuple=True)
    dst, src = st["dst"][b, i].long(), st["src"][b, i].long()
    flat[st["table"][b, dst // P].long() * P + dst % P] = flat[st["table"][b, src // P].long() * P + src % P]
    st["acc"][b, dst] = st["acc"][b, src]
    st["pos"][b, dst] = st["pos"][b, src]
    return dict(kv=st["kv"], acc=st["acc"], pos=st["pos"])


# ---------------------------------------------------------------- one pass

def run(state):
    op, c = state["case"]["op"], state["case"]
    if not own:
        return dict(append=_append, attn=_attn, weights=_weights, plan=_plan, move=_move)[op](state)
    from sparse_attention_04_b200 import _lib
    s = state
    if op == "append":
        _lib.paged_append(s["new"], s["kv"], s["table"], s["lens"], acc=s["acc"], pos=s["pos"], end_pos=s["end_pos"],
                          status=s["status"])
        return dict(kv=s["kv"], acc=s["acc"], pos=s["pos"])
    if op == "attn":
        if "workspace" not in s:
            n = _lib.paged_mla_workspace_size(c["B"], c["T"], c["H"])
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=s["q"].device)
        _lib.paged_mla(s["q"], s["kv"], s["table"], s["lens"], SCALE, s["out"], lse=s["lse"], workspace=s["workspace"],
                       status=s["status"])
        return dict(out=s["out"], lse=s["lse"])
    if op == "weights":
        _lib.paged_weights(s["q"], s["kv"], s["table"], s["lens"], s["lse"], SCALE, s["acc"], acc_out=s["acc_out"],
                           decay=c["decay"], status=s["status"])
        return s["acc_out"]
    if op == "plan":
        _lib.evict_plan(s["acc"], s["pos"], s["lens"], s["end_pos"], c["budget"], c["recent"], s["new_lens"], s["n_moves"],
                        s["dst"], s["src"], status=s["status"])
        return dict(new_lens=s["new_lens"], n_moves=s["n_moves"], dst=s["dst"], src=s["src"])
    _lib.paged_move(s["kv"], s["table"], s["n_moves"], s["dst"], s["src"], acc=s["acc"], pos=s["pos"], status=s["status"])
    return dict(kv=s["kv"], acc=s["acc"], pos=s["pos"])


def work(case):
    op, B, lens = case["op"], case["B"], _lens(case)
    if op == "append":
        n = B * case["T"]
        return dict(bytes=n * (2 * 2 * D + 8) + 12 * B, flops=0)
    if op == "plan":
        return dict(bytes=8 * sum(lens) + 8 * B * _max_moves(case) + 16 * B, flops=0)
    if op == "move":
        return dict(bytes=sum(_n_moves(case)) * (2 * 2 * D + 16 + 8) + 4 * B, flops=0)
    T, H = case["T"], case["H"]
    seen = sum(max(0, L - T + t + 1) for L in lens for t in range(T))
    table = 4 * sum(-(-L // case["P"]) for L in lens) + 4 * B
    if op == "attn":
        return dict(bytes=2 * D * sum(lens) + table + B * T * H * (2 * D + 2 * DV + 4), flops=2 * H * (D + DV) * seen)
    return dict(bytes=(2 * D + 8) * sum(lens) + table + B * T * H * (2 * D + 4), flops=2 * H * D * seen)


# ---------------------------------------------------------------- by definition, in 64 bits

def _cache_of(st, b):
    """Sequence b's cache rows in 64 bits."""
    L, P = int(st["lens"][b]), st["kv"].shape[1]
    pages = st["table"][b, :-(-L // P)].long()
    return st["kv"][pages].reshape(-1, D)[:L].double()


def exact(case, seed):
    st = prepare(case, seed)
    op, B = case["op"], case["B"]
    lens = [int(x) for x in st["lens"]]
    if op == "append":
        kv, acc, pos, T, P = st["kv"].double(), st["acc"].double(), st["pos"], case["T"], case["P"]
        for b, L in enumerate(lens):
            s = torch.arange(L - T, L, device=kv.device)
            kv[st["table"][b].long()[s // P], s % P] = st["new"][b].double()
            acc[b, L - T:L] = 0
            pos[b, L - T:L] = (s + int(st["end_pos"][b]) - L).int()
        return dict(kv=kv, acc=acc, pos=pos)
    if op == "move":
        kv, acc, pos, P = st["kv"].double(), st["acc"].double(), st["pos"], case["P"]
        for b in range(B):
            n = int(st["n_moves"][b])
            d, s, pages = st["dst"][b, :n].long(), st["src"][b, :n].long(), st["table"][b].long()
            kv[pages[d // P], d % P] = kv[pages[s // P], s % P]
            acc[b, d], pos[b, d] = acc[b, s], pos[b, s]
        return dict(kv=kv, acc=acc, pos=pos)
    if op == "plan":
        acc, pos = st["acc"].cpu().numpy(), st["pos"].cpu().numpy()
        m = _max_moves(case)
        new_lens, n_moves = np.zeros(B, np.int32), np.zeros(B, np.int32)
        dst, src = np.full((B, m), -1, np.int32), np.full((B, m), -1, np.int32)
        for b, L in enumerate(lens):
            n = min(L, case["budget"])
            protected = pos[b, :L] >= int(st["end_pos"][b]) - case["recent"]
            best = np.lexsort((np.arange(L), -acc[b, :L].astype(np.float64), ~protected))[:n]
            kept = np.zeros(L, bool)
            kept[best] = True
            holes, tail = np.nonzero(~kept[:n])[0], n + np.nonzero(kept[n:])[0]
            new_lens[b], n_moves[b] = n, len(holes)
            dst[b, :len(holes)], src[b, :len(tail)] = holes, tail
        return dict(new_lens=new_lens, n_moves=n_moves, dst=dst, src=src)
    T, H = case["T"], case["H"]
    if op == "attn":
        out = torch.zeros((B, T, H, DV), dtype=torch.float64, device=st["q"].device)
        lse = torch.full((B, T, H), float("-inf"), dtype=torch.float64, device=st["q"].device)
        for b, L in enumerate(lens):
            k = _cache_of(st, b)
            for t in range(T):
                n = L - T + t + 1
                if n > 0:
                    x = SCALE * (st["q"][b, t].double() @ k[:n].T)
                    lse[b, t] = x.logsumexp(1)
                    out[b, t] = x.softmax(1) @ k[:n, :DV]
        return dict(out=out, lse=lse)
    new = st["acc_out"].double()
    for b, L in enumerate(lens):
        k = _cache_of(st, b)
        total = st["acc"][b, :L].double() * case["decay"]
        for t in range(T):
            n = L - T + t + 1
            if n > 0:
                x = SCALE * (st["q"][b, t].double() @ k[:n].T) - st["lse"][b, t].double()[:, None]
                total[:n] += x.exp().sum(0)
        new[b, :L] = total
    return new
