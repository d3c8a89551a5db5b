"""Convenience layer over the C ABI for torch users.

Allocates outputs and workspaces as torch CUDA tensors (PyTorch is used for
device memory and streams only) and calls the library through `_lib`.  Every
step of the path runs in the library's kernels.
"""
from __future__ import annotations

import dataclasses
import math
from typing import Optional

import torch

from . import _lib
from .inputs import D_QK, D_V, Inputs


@dataclasses.dataclass
class StepResult:
    out: torch.Tensor           # [B,T,H,512]
    lse: torch.Tensor           # [B,T,H] fp32
    scores: torch.Tensor        # [B*T, ld] fp32 (a view of the workspace for decode)
    indices: torch.Tensor       # [B*T, k] int32
    status: torch.Tensor        # int32 [1], device
    ld: int


def _out_dtype(wl):
    return torch.float32 if wl.out_dtype == "f32" else torch.bfloat16


class DecodeStep:
    """Buffers for repeated dsa_decode_step calls on one workload shape."""

    def __init__(self, B: int, max_end_pos: int, k: int, H: int, out_dtype=torch.bfloat16, device="cuda"):
        self.B, self.max_end_pos, self.k, self.H = B, max_end_pos, k, H
        nbytes = _lib.decode_step_workspace_size(B, max_end_pos, k, H)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        so, ld, io, _ = _lib.decode_step_workspace_layout(B, max_end_pos, k, H)
        self.ld = ld
        self.scores = self.workspace[so:so + B * ld * 4].view(torch.float32).view(B, ld)
        self.indices = self.workspace[io:io + B * k * 4].view(torch.int32).view(B, k)
        self.out = torch.empty((B, 1, H, D_V), dtype=out_dtype, device=device)
        self.lse = torch.empty((B, 1, H), dtype=torch.float32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def __call__(self, q_idx, w, k_idx, k_scale, q, kv, offsets, kv_rows, scale, stream=None):
        _lib.decode_step(q_idx, w, k_idx, k_scale, q, kv, offsets, self.B, self.max_end_pos, kv_rows,
                         self.k, self.H, scale, self.out, lse=self.lse, workspace=self.workspace,
                         status=self.status, stream=stream)
        return self.out


class HostDecodeStep:
    """A decode step fed from pinned host memory whose output goes back to
    pinned host memory: the form a server uses when the new token's
    projections arrive from the host.

    The caller fills the pinned views host_q_idx [B,1,64,128] bf16, host_w
    [B,1,64] fp32, host_k_new [B,1,128] bf16, host_kv_new [B,1,576] bf16 and
    host_q [B,1,H,576] bf16, calls the object with the resident caches, and
    reads host_out [B,1,H,512] once the stream has been synchronised (and only
    then refills the inputs).  One call issues on the current stream

        copy kernel (q_I, w, k_new, kv_new) -> dsa_cache_append
        -> [dsa_quantize_queries for e4m3 keys] -> dsa_indexer_scores
        -> dsa_topk -> dsa_sparse_mla -> copy kernel (out)

    How q, the largest input, crosses PCIe depends on its size (measured on
    B200, microseconds per host-fed step):
      - up to Q_WITH_INPUTS_MAX bytes (one 128-head row): in the same copy
        kernel as the small inputs, so that the whole dsa_decode_step follows
        with q complete and the attention loads its query tile before the
        selection ends (decode 32K: 36.3 against 37.5 with the side stream);
      - up to Q_KERNEL_COPY_MAX bytes: on a side stream, by a copy kernel
        launched once the indexer has finished, so it crosses PCIe while the
        selection runs on a few SMs; the attention waits for it.  Started with
        the step, its CTAs took registers that the indexer's CTAs needed and
        held them back (fp8 B=4: 78.8 against 71.4; in the first copy 78.1);
      - above that: by the copy engine on the side stream from the start of
        the step, so that a long transfer overlaps the indexer too and holds
        no SM.
    When every end_pos <= k the attention-only form of dsa_decode_step runs
    once q is in.  Each call starts after everything issued before it on the
    stream."""

    Q_WITH_INPUTS_MAX = 1 << 18
    Q_KERNEL_COPY_MAX = 1 << 20

    def __init__(self, B: int, max_end_pos: int, k: int, H: int, idx_dtype: str = "bf16",
                 out_dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        self.step = DecodeStep(B, max_end_pos, k, H, out_dtype, dev)
        self.B, self.max_end_pos, self.k, self.H = B, max_end_pos, k, H
        self.fp8 = idx_dtype == "e4m3"
        # one pinned staging buffer for the small inputs (and q, when it is
        # small enough to travel with them), 256-byte aligned sections
        q_bytes = B * H * 576 * 2
        self.q_with_inputs = q_bytes <= self.Q_WITH_INPUTS_MAX
        spec = [(torch.bfloat16, (B, 1, 64, 128)), (torch.float32, (B, 1, 64)),
                (torch.bfloat16, (B, 1, 128)), (torch.bfloat16, (B, 1, 576))]
        if self.q_with_inputs:
            spec.append((torch.bfloat16, (B, 1, H, 576)))
        sizes = [math.prod(shape) * torch.empty((), dtype=dt).element_size() for dt, shape in spec]
        offs, tot = [], 0
        for sz in sizes:
            offs.append(tot)
            tot += -(-sz // 256) * 256
        self.host_small = torch.zeros(tot, dtype=torch.uint8, pin_memory=True)
        self._small = torch.empty(tot, dtype=torch.uint8, device=dev)

        def views(buf):
            return [buf[o:o + n].view(dt).view(*shape) for o, n, (dt, shape) in zip(offs, sizes, spec)]

        hv, dv = views(self.host_small), views(self._small)
        self.host_q_idx, self.host_w, self.host_k_new, self.host_kv_new = hv[:4]
        self._q_idx, self._w, self._k_new, self._kv_new = dv[:4]
        if self.q_with_inputs:
            self.host_q, self._q = hv[4], dv[4]
        else:
            self.host_q = torch.zeros((B, 1, H, 576), dtype=torch.bfloat16, pin_memory=True)
            self._q = torch.empty((B, 1, H, 576), dtype=torch.bfloat16, device=dev)
        self.host_out = torch.zeros(tuple(self.step.out.shape), dtype=out_dtype, pin_memory=True)
        if self.fp8:
            self._q8 = torch.empty((B, 1, 64, 128), dtype=torch.uint8, device=dev)
            self._w8 = torch.empty((B, 1, 64), dtype=torch.float32, device=dev)
        m_off = _lib.decode_step_workspace_layout(B, max_end_pos, k, H)[3]
        self._ws_mla = self.step.workspace[m_off:]
        self._side = torch.cuda.Stream(dev)
        self.h2d_bytes = tot + (0 if self.q_with_inputs else self.host_q.numel() * 2)
        self.d2h_bytes = self.host_out.numel() * self.host_out.element_size()

    def _copy_q(self, cur):
        """q's transfer on the side stream, after everything issued so far on `cur`."""
        self._side.wait_stream(cur)
        with torch.cuda.stream(self._side):
            if self.host_q.numel() * 2 <= self.Q_KERNEL_COPY_MAX:
                _lib.copy_host_to_device(self._q, self.host_q)
            else:
                self._q.copy_(self.host_q, non_blocking=True)

    def __call__(self, k_idx, k_scale, kv, offsets, kv_rows, scale):
        st, B = self.step, self.B
        cur = torch.cuda.current_stream()
        q_by_kernel = self.host_q.numel() * 2 <= self.Q_KERNEL_COPY_MAX
        short = self.max_end_pos <= self.k
        if not self.q_with_inputs and (short or not q_by_kernel):
            self._copy_q(cur)
        _lib.copy_host_to_device(self._small, self.host_small)
        _lib.cache_append(self._k_new, self._kv_new, offsets, B, 1, k_idx, k_scale, kv, kv_rows, status=st.status)
        q_idx, w = self._q_idx, self._w
        if self.fp8:
            _lib.quantize_queries(q_idx, w, B, self._q8, self._w8)
            q_idx, w = self._q8, self._w8
        if self.q_with_inputs:
            # q is complete before the step's first kernel: the fused step
            st(q_idx, w, k_idx, k_scale, self._q, kv, offsets, kv_rows, scale)
        elif short:
            cur.wait_stream(self._side)
            st(q_idx, w, k_idx, k_scale, self._q, kv, offsets, kv_rows, scale)
        else:
            _lib.indexer_scores(q_idx, w, k_idx, k_scale, offsets, B, 1, kv_rows, st.scores, st.ld,
                                status=st.status)
            if q_by_kernel:
                self._copy_q(cur)  # crosses PCIe beside the selection
            _lib.topk(st.scores, st.ld, offsets, B, 1, self.k, st.indices, status=st.status)
            cur.wait_stream(self._side)
            _lib.sparse_mla(self._q, kv, offsets, st.indices, B, 1, self.H, self.k, scale, kv_rows, st.out,
                            lse=st.lse, workspace=self._ws_mla, status=st.status)
        _lib.copy_device_to_host(self.host_out, st.out)
        return self.host_out


class PagedLatentCache:
    """A paged latent cache of B sequences and what a decode step does with it:

        out = cache.append(kv_new).attend(q, scale)    # attention over all of it
        cache.collect(q, scale, decay)                 # attention weight per slot
        cache.evict(budget, recent)                    # keep the heaviest and newest

    Lengths, positions and the eviction plan stay on the device, so that the
    whole step can be captured in one CUDA graph.  T: most tokens of a sequence
    that attend to the cache in one call (a prompt's, say; single tokens go
    through the same object).  Every sequence has page lists for `slots` slots,
    rounded up to whole pages; a scheduler that hands pages out writes its own
    numbers into page_table.  Append the prompt, or write its rows into kv_pages
    and call fill.  A sequence appended to beyond its slots is reported in status
    and counts as empty until lens is set again.  max_moves: rows an eviction may
    move per sequence, enough for every cut unless given; a sequence that needs
    more is reported in status and not cut.

    kv_pages [pages, page_size, 576] bf16, page_table [B, pages per sequence],
    lens and end_pos [B], acc and pos [B, slots] (see include/dsa.h)."""

    def __init__(self, B: int, slots: int, T: int = 1, H: int = 128, page_size: int = 64, max_moves: Optional[int] = None,
                 out_dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        pages = -(-slots // page_size)
        self.B, self.T, self.H, self.slots = B, T, H, pages * page_size
        self.kv_pages = torch.empty((B * pages, page_size, D_QK), dtype=torch.bfloat16, device=dev)
        self.page_table = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.end_pos = torch.zeros(B, dtype=torch.int32, device=dev)
        self.acc = torch.zeros((B, self.slots), dtype=torch.float32, device=dev)
        self.pos = torch.zeros((B, self.slots), dtype=torch.int32, device=dev)
        self.out = torch.empty((B, T, H, D_V), dtype=out_dtype, device=dev)
        self.lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
        with torch.cuda.device(self.lens.device):  # fewer tokens may need more: their tiles go to another kernel
            nbytes = max(_lib.paged_mla_workspace_size(B, t, H) for t in range(1, max(1, min(T, 128 // max(H, 1))) + 1))
        self.workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=dev)
        # a cut of L slots to n moves min(n, L - n) rows at most
        moves = max(1, max_moves if max_moves is not None else self.slots // 2)
        self.new_lens, self.n_moves = torch.zeros_like(self.lens), torch.zeros_like(self.lens)
        self.move_dst = torch.empty((B, moves), dtype=torch.int32, device=dev)
        self.move_src = torch.empty((B, moves), dtype=torch.int32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def fill(self, lens):
        """The first lens[b] slots of every sequence hold its tokens 0 .. lens[b] - 1
        (rows written into kv_pages directly): sets lens, end_pos, pos and acc,
        whatever they held before."""
        self.lens.copy_(torch.as_tensor(lens))
        self.end_pos.copy_(self.lens)
        self.pos.copy_(torch.arange(self.slots, dtype=torch.int32, device=self.pos.device).expand_as(self.pos))
        self.acc.zero_()
        return self

    def append(self, kv_new, active=None):
        """The newest tokens' rows [B,T,576], any T, of every sequence, or of those
        where active [B] (bool) holds: the others keep what they have, and an
        empty one stays empty.  Prompts of different lengths go in one by one."""
        T, lens = kv_new.shape[1], self.lens
        if active is None:
            self.lens.add_(T)
            self.end_pos.add_(T)
        else:
            self.lens.add_(active, alpha=T)
            self.end_pos.add_(active, alpha=T)
            lens = self.lens * active  # an empty sequence is not written
        _lib.paged_append(kv_new, self.kv_pages, self.page_table, lens, acc=self.acc, pos=self.pos, end_pos=self.end_pos,
                          status=self.status)
        return self

    def _rows(self, q):
        """out and lse of a call with q's number of tokens: the first elements of self.out and self.lse."""
        t = q.shape[1] if q.dim() == 4 else 0
        if t == self.T:
            return self.out, self.lse
        if not 0 < t < self.T:
            raise _lib.DSAError(1, f"PagedLatentCache: q must be [B, T, H, 576] with 1 to {self.T} tokens")
        n = self.B * t * self.H
        return (self.out.view(-1, D_V)[:n].view(self.B, t, self.H, D_V), self.lse.view(-1)[:n].view(self.B, t, self.H))

    def attend(self, q, scale):
        """Attention of q [B,t,H,576], t <= T, over each whole cache: out [B,t,H,512]; lse beside it."""
        out, lse = self._rows(q)
        _lib.paged_mla(q, self.kv_pages, self.page_table, self.lens, scale, out, lse=lse, workspace=self.workspace,
                       status=self.status)
        return out

    def collect(self, q, scale, decay=1.0):
        """Adds the weight that the slots got from the last attend's q to acc."""
        _lib.paged_weights(q, self.kv_pages, self.page_table, self.lens, self._rows(q)[1], scale, self.acc, decay=decay,
                           status=self.status)
        return self.acc

    def evict(self, budget, recent=0):
        """Cuts every sequence to `budget` slots; the `recent` newest tokens stay."""
        _lib.evict_plan(self.acc, self.pos, self.lens, self.end_pos, budget, recent, self.new_lens, self.n_moves,
                        self.move_dst, self.move_src, status=self.status)
        _lib.paged_move(self.kv_pages, self.page_table, self.n_moves, self.move_dst, self.move_src, acc=self.acc,
                        pos=self.pos, status=self.status)
        self.lens.copy_(self.new_lens)
        return self.lens


def decode_step(inp: Inputs, step: Optional[DecodeStep] = None) -> StepResult:
    """Runs the fused decode step (T must be 1) on device-resident inputs."""
    wl = inp.wl
    assert wl.T == 1
    if step is None:
        step = DecodeStep(wl.B, max(inp.end_pos), wl.topk, wl.H, _out_dtype(wl), inp.q.device)
    step(inp.q_idx, inp.w, inp.k_idx, inp.k_scale, inp.q, inp.kv, inp.offsets, inp.rows, wl.scale)
    return StepResult(step.out, step.lse, step.scores, step.indices, step.status, step.ld)


def staged(inp: Inputs) -> StepResult:
    """Runs the three stages as separate calls (any T, e.g. causal prefill)."""
    wl = inp.wl
    dev = inp.q.device
    B, T, H, k = wl.B, wl.T, wl.H, wl.topk
    n = B * T
    ld = (max(inp.end_pos) + 3) // 4 * 4
    scores = torch.empty((n, ld), dtype=torch.float32, device=dev)
    indices = torch.empty((n, k), dtype=torch.int32, device=dev)
    out = torch.empty((B, T, H, D_V), dtype=_out_dtype(wl), device=dev)
    lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ws_bytes = _lib.sparse_mla_workspace_size(B, T, H, k)
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    _lib.indexer_scores(inp.q_idx, inp.w, inp.k_idx, inp.k_scale, inp.offsets, B, T, inp.rows, scores, ld,
                        status=status)
    _lib.topk(scores, ld, inp.offsets, B, T, k, indices, status=status)
    _lib.sparse_mla(inp.q, inp.kv, inp.offsets, indices, B, T, H, k, wl.scale, inp.rows, out, lse=lse,
                    workspace=ws, status=status)
    return StepResult(out, lse, scores, indices, status, ld)
