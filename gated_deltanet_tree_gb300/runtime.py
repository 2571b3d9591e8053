"""Buffer ownership around the C ABI: factor banks, workspace, schedules.

PyTorch provides device memory and streams; every computation is a call into
libgdn_tree.so through the ctypes binding.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import numpy as np
import torch

from . import _native as N


def make_dims(Hk: int, Hv: int, dk: int, dv: int, K: int, conv_mode: int = 1, act: int = 1,
              in_dtype: int = N.GDN_DTYPE_BF16, q_scale: float = 1.0, l2_eps: float = 1e-6) -> N.gdn_dims:
    return N.gdn_dims(Hk=Hk, Hv=Hv, dk=dk, dv=dv, K=K, conv_mode=conv_mode, act=act, in_dtype=in_dtype,
                      q_scale=q_scale, l2_eps=l2_eps)


def channels(d: N.gdn_dims) -> int:
    return 2 * d.Hk * d.dk + d.Hv * d.dv


class DeviceSchedule:
    """A packed batch schedule resident on the device."""

    def __init__(self, parents: Sequence[np.ndarray], n_max: int, device, nb_cap: Optional[int] = None,
                 words_out: Optional[torch.Tensor] = None, stream=None, per_node: bool = False):
        B = len(parents)
        P = np.full((B, n_max), -1, dtype=np.int32)
        n = np.zeros(B, dtype=np.int32)
        for b, p in enumerate(parents):
            P[b, :len(p)] = p
            n[b] = len(p)
        pack = N.gdn_pack_schedules_per_node if per_node else N.gdn_pack_schedules
        words, nb, depth = pack(P, n, with_depth=True)
        self.parents, self.n, self.nb_max = P, n, nb if nb_cap is None else max(nb, nb_cap)
        self.depth_max = depth
        if words_out is None:
            self.words = torch.from_numpy(words).to(device)
        else:
            words_out.copy_(torch.from_numpy(words), non_blocking=False)
            self.words = words_out
        self.host_words = words
        self.struct = N.gdn_batch_schedule(B=B, n_max=n_max, nb_max=self.nb_max, depth_max=depth,
                                           words=self.words.data_ptr())


class TreeVerifier:
    """Factor banks, pending-path record, error words and workspace for one batch shape."""

    def __init__(self, dims: N.gdn_dims, B: int, layers: int, n_max: int, device="cuda"):
        self.dims, self.B, self.layers, self.n_max = dims, B, layers, n_max
        self.device = torch.device(device)
        f32 = dict(dtype=torch.float32, device=self.device)
        C = channels(dims)
        rows = B * layers * n_max
        self.bank_k = [torch.zeros(rows * dims.Hk * dims.dk, **f32) for _ in range(2)]
        self.bank_u = [torch.zeros(rows * dims.Hv * dims.dv, **f32) for _ in range(2)]
        self.bank_a = [torch.zeros(rows * dims.Hv, **f32) for _ in range(2)]
        self.bank_x = [torch.zeros(rows * C, **f32) if dims.conv_mode == 1 else None for _ in range(2)]
        i32 = dict(dtype=torch.int32, device=self.device)
        self.pend_path = torch.zeros(B * n_max, **i32)
        self.pend_len = torch.zeros(B, **i32)
        self.err = torch.zeros(4, **i32)
        self.ws_bytes = N.gdn_workspace_bytes(dims, B, layers, n_max)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
        self.banks = N.gdn_banks()
        for i in range(2):
            self.banks.k[i] = self.bank_k[i].data_ptr()
            self.banks.u[i] = self.bank_u[i].data_ptr()
            self.banks.a[i] = self.bank_a[i].data_ptr()
            self.banks.x[i] = self.bank_x[i].data_ptr() if self.bank_x[i] is not None else None
        self.banks.pend_path = self.pend_path.data_ptr()
        self.banks.pend_len = self.pend_len.data_ptr()
        self.banks.err = self.err.data_ptr()
        N.gdn_banks_init(self.banks, B, layers, n_max)

    # bank views ---------------------------------------------------------------
    def bank_view(self, field: str, i: int) -> torch.Tensor:
        d, sh = self.dims, (self.B, self.layers, self.n_max)
        if field == "k":
            return self.bank_k[i].view(*sh, d.Hk, d.dk)
        if field == "u":
            return self.bank_u[i].view(*sh, d.Hv, d.dv)
        if field == "a":
            return self.bank_a[i].view(*sh, d.Hv)
        if field == "x":
            return self.bank_x[i].view(*sh, channels(d))
        raise KeyError(field)

    # calls ---------------------------------------------------------------------
    def schedule(self, parents: Sequence[np.ndarray], nb_cap: Optional[int] = None,
                 per_node: bool = False) -> DeviceSchedule:
        return DeviceSchedule(parents, self.n_max, self.device, nb_cap, per_node=per_node)

    def verify(self, sched: DeviceSchedule, x_raw, conv_w, beta, log_g, state, conv_state, out_o, boundary,
               stream=None, boundary_scratch: bool = False, chain_walk: bool = False, ut_simt: bool = False,
               tc_per_head: bool = False, chains: bool = False):
        flags = (N.GDN_VERIFY_BOUNDARY_SCRATCH if boundary_scratch else 0) | \
                (N.GDN_VERIFY_CHAIN_WALK if chain_walk else 0) | \
                (N.GDN_VERIFY_UT_SIMT if ut_simt else 0) | \
                (N.GDN_VERIFY_TC_PER_HEAD if tc_per_head else 0) | \
                (N.GDN_VERIFY_CHAINS if chains else 0)
        N.gdn_tree_verify(self.dims, self.layers, sched.struct, x_raw, conv_w, beta, log_g, state, conv_state,
                          out_o, boundary, self.banks, self.workspace, self.ws_bytes, flags, stream)

    def commit(self, sched: DeviceSchedule, path: torch.Tensor, length: torch.Tensor, compact: bool = False,
               stream=None):
        N.gdn_commit_fold(self.dims, self.layers, sched.struct, path, length,
                          N.GDN_COMMIT_COMPACT if compact else 0, self.banks, stream)

    def finish(self, state, conv_state, stream=None):
        N.gdn_finish(self.dims, self.B, self.layers, state, conv_state, self.banks, stream)

    def check_error(self, stream=None):
        N.gdn_check_error(self.banks, stream)


def paths_tensor(paths: Sequence[Sequence[int]], n_max: int, device) -> tuple:
    """Host paths -> (path [B, n_max] int32, len [B] int32) device tensors."""
    B = len(paths)
    P = np.zeros((B, n_max), dtype=np.int32)
    L = np.zeros(B, dtype=np.int32)
    for b, p in enumerate(paths):
        P[b, :len(p)] = p
        L[b] = len(p)
    return torch.from_numpy(P).to(device), torch.from_numpy(L).to(device)


_DTYPES = {torch.float32: N.GDN_DTYPE_F32, torch.bfloat16: N.GDN_DTYPE_BF16}


def _dtype_code(dtype: torch.dtype, what: str) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"{what} is {dtype}: fp32 and bf16 are supported")
    return code


def make_attn_dims(Hq: int, Hkv: int, D: int, dtype: torch.dtype = torch.bfloat16,
                   scale: Optional[float] = None) -> N.gdn_attn_dims:
    """Shapes of one full-attention layer; scale defaults to 1 / sqrt(D)."""
    return N.gdn_attn_dims(Hq=Hq, Hkv=Hkv, D=D, dtype=_dtype_code(dtype, "dtype"),
                           scale=D ** -0.5 if scale is None else scale, q_row=0, kv_row=0)


def _row_stride(t: torch.Tensor, name: str, shape: tuple) -> int:
    """Elements from one node's row of t [B, layers, n, heads, D] to the next; rows of a fused projection (a slice of
    wider rows) are taken as they lie."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the call needs {shape}")
    B, L, n, H, D = shape
    if t.is_contiguous():
        return H * D
    row = t.stride(2) if n > 1 else (t.stride(1) if L > 1 else t.stride(0) if B > 1 else H * D)
    want = (L * n * row, n * row, row, D, 1)
    for size, got, need in zip(shape, t.stride(), want):
        if size > 1 and got != need:
            raise ValueError(f"{name} has strides {t.stride()}: rows need one stride, heads and channels contiguous")
    return _stride_in_range(row, H * D, name)


def _stride_in_range(row: int, least: int, name: str) -> int:
    """A row stride as the calls take it: 0 would stand for contiguous rows there, and 32 bits hold it."""
    if not least <= row < 1 << 31:
        raise ValueError(f"{name} has rows {row} elements apart: rows of {least} elements may neither overlap nor repeat "
                         f"(a broadcast), nor lie 2^31 elements apart; make it contiguous")
    return row


def _finish_fills(device: torch.device):
    """Waits for what the current stream has filled on a device, so that a first call on any stream finds it filled."""
    if device.type == "cuda":
        torch.cuda.current_stream(device).synchronize()


class KV4Cache:
    """The paged 4-bit key/value cache of a stack of full-attention layers: the pool, page table and lengths the
    caller gives (or empty() makes) and the counters and workspace of the calls on them.

    A call may go to any stream, or into a CUDA graph.  The calls on one cache share its counters and workspace, so they
    must follow one another: order those on different streams by events."""

    def __init__(self, dims: N.gdn_attn_dims, pool: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor):
        if pool.dim() != 4 or pool.dtype != torch.uint8 or tuple(pool.shape[2:]) != (dims.Hkv, 72 * dims.D):
            raise ValueError(f"pool is [layers, n_pages, Hkv, 72 D] uint8, got {tuple(pool.shape)} {pool.dtype}")
        for t, name, nd in ((page_table, "page_table", 2), (seq_len, "seq_len", 1)):
            if t.dtype != torch.int32 or t.dim() != nd:
                raise ValueError(f"{name} is int32 with {nd} dimensions, got {tuple(t.shape)} {t.dtype}")
        if page_table.shape[0] != seq_len.shape[0]:
            raise ValueError("page_table and seq_len disagree on the number of requests")
        for t in (pool, page_table, seq_len):
            if not t.is_contiguous() or t.device != pool.device:
                raise ValueError("pool, page_table and seq_len are contiguous tensors of one device")
        self.dims = N.gdn_attn_dims.from_buffer_copy(dims)
        self.dims.q_row = self.dims.kv_row = 0                 # contiguous rows; a call with others makes its own copy
        self.pool, self.page_table, self.seq_len = pool, page_table, seq_len
        self.device = pool.device
        self.B, self.layers, self.pages_max = seq_len.shape[0], pool.shape[0], page_table.shape[1]
        self.ticket = torch.zeros(self.B, dtype=torch.int32, device=self.device)
        self.err = torch.zeros(4, dtype=torch.int32, device=self.device)
        # Made for the largest call, once: a workspace that grew with the calls would be filled on another stream than the
        # kernel's, and freed under kernels in flight and captured graphs.  Its size is bounded by the CTAs of a launch
        self.workspace = torch.zeros(max(256, *(N.gdn_kv4_workspace_bytes(self.dims, self.B, self.layers, n, 0)
                                                for n in range(1, N.GDN_MAX_NODES + 1))),
                                     dtype=torch.uint8, device=self.device)
        self.struct = N.gdn_kv4_cache(pool=pool.data_ptr(), page_table=page_table.data_ptr(),
                                      seq_len=seq_len.data_ptr(), ticket=self.ticket.data_ptr(),
                                      err=self.err.data_ptr(), B=self.B, layers=self.layers,
                                      pages_max=self.pages_max, n_pages=pool.shape[1])
        # what every call passes, once (a call's own time on the host is what a small one costs)
        self._type = torch.bfloat16 if dims.dtype == N.GDN_DTYPE_BF16 else torch.float32
        self._index = pool.get_device()
        self._refs = (ctypes.byref(self.dims), ctypes.byref(self.struct))
        self._heads = (dims.Hq, dims.Hkv, dims.D)
        _finish_fills(self.device)

    @classmethod
    def empty(cls, dims: N.gdn_attn_dims, B: int, layers: int, pages_max: int, device="cuda") -> "KV4Cache":
        """A cache of pages_max pages (of 64 tokens) a request, each request's pages consecutive, all lengths 0."""
        pool = torch.zeros(layers, B * pages_max, dims.Hkv, 72 * dims.D, dtype=torch.uint8, device=device)
        table = torch.arange(B * pages_max, dtype=torch.int32, device=device).view(B, pages_max)
        return cls(dims, pool, table, torch.zeros(B, dtype=torch.int32, device=device))

    def _check_type(self, t: torch.Tensor, name: str):
        if t.dtype is not self._type or t.get_device() != self._index:
            _dtype_code(t.dtype, name)
            raise ValueError(f"{name} is {t.dtype} on {t.device}: not the cache's type or device")

    def _check_i32(self, t: torch.Tensor, name: str, shape: tuple):
        if t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} is a contiguous int32 tensor {shape} on {self.device}, got {tuple(t.shape)} "
                             f"{t.dtype} on {t.device}")

    def _rows(self, k: torch.Tensor, v: torch.Tensor) -> tuple:
        """Rows a request and their stride."""
        if k.dim() != 5:
            raise ValueError(f"k_new is [B, layers, n, Hkv, D], got {tuple(k.shape)}")
        n = k.shape[2]
        _, Hkv, D = self._heads
        want = (self.B, self.layers, n, Hkv, D)
        self._check_type(k, "k_new")
        self._check_type(v, "v_new")
        row = _row_stride(k, "k_new", want)
        if row != _row_stride(v, "v_new", want):
            raise ValueError("k_new and v_new have different row strides")
        return n, row

    def _dims(self, q_row: int, kv_row: int):
        """The cache's shapes with a call's row strides.  They are never written to the cache's own: a refused call would
        leave them behind, and calls from two threads would take each other's."""
        Hq, Hkv, D = self._heads
        if q_row == Hq * D and kv_row == Hkv * D:
            return self._refs[0]
        d = N.gdn_attn_dims.from_buffer_copy(self.dims)
        d.q_row, d.kv_row = q_row, kv_row
        return ctypes.byref(d)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, count: torch.Tensor,
               path: Optional[torch.Tensor] = None, stream=None):
        """Quantise rows k_new, v_new [B, layers, n, Hkv, D] into the cache: the first count[b], or the rows path[b]
        names, and advance the lengths (on the device)."""
        n, row = self._rows(k_new, v_new)
        self._check_i32(count, "count", (self.B,))
        if path is not None:
            self._check_i32(path, "path", (self.B, n))
        Hq, _, D = self._heads
        N._check(N.lib().gdn_kv4_append(self._dims(Hq * D, row), self.layers, n, k_new.data_ptr(), v_new.data_ptr(),
                                        None if path is None else path.data_ptr(), count.data_ptr(), self._refs[1],
                                        N._stream_of(stream, self._index)))

    def read(self, start: Optional[torch.Tensor], n: int, dtype: torch.dtype = torch.float32, stream=None):
        """Values of tokens start[b] .. start[b] + n - 1 (None: from 0) -> k, v [B, layers, n, Hkv, D]; zeros past a
        request's length.  With a stream given they are complete on that one."""
        if start is not None:
            self._check_i32(start, "start", (self.B,))
        code = _dtype_code(dtype, "dtype")
        shape = (self.B, self.layers, n, *self._heads[1:])
        if stream is None or self.device.type != "cuda":
            k = torch.empty(shape, dtype=dtype, device=self.device)     # (two views of one tensor take twice the host time)
            v = torch.empty(shape, dtype=dtype, device=self.device)
        else:
            # memory of the stream that writes it: a block of the current stream's may still be in use there
            writer = torch.cuda.ExternalStream(N._stream(stream), device=self.device)
            with torch.cuda.stream(writer):
                k = torch.empty(shape, dtype=dtype, device=self.device)
                v = torch.empty(shape, dtype=dtype, device=self.device)
            for t in (k, v):                                            # the current stream will read them
                t.record_stream(torch.cuda.current_stream(self.device))
        dims, cache = self._refs
        N._check(N.lib().gdn_kv4_read(dims, self.layers, n, None if start is None else start.data_ptr(), code,
                                      k.data_ptr(), v.data_ptr(), cache, N._stream_of(stream, self._index)))
        return k, v

    def attention(self, q: torch.Tensor, k_new: Optional[torch.Tensor], v_new: Optional[torch.Tensor],
                  out: torch.Tensor, sched: Optional[DeviceSchedule] = None, max_len: int = 0, stream=None):
        """Nodes q [B, layers, n_max, Hq, D] attend to the cached tokens and (with k_new, v_new) to their ancestors'
        and their own rows; sched None: one node a request.  max_len bounds the lengths where the host knows it."""
        n = 1 if sched is None else sched.struct.n_max
        Hq, Hkv, D = self._heads
        self._check_type(q, "q")
        self._check_type(out, "out")
        q_row = _row_stride(q, "q", (self.B, self.layers, n, Hq, D))
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out is contiguous with the shape of q")
        if (k_new is None) != (v_new is None):
            raise ValueError("k_new and v_new: both or neither")
        kv_row = Hkv * D
        if k_new is not None:
            n_new, kv_row = self._rows(k_new, v_new)
            if n_new != n:
                raise ValueError("k_new and q have different node counts")
        cache = self._refs[1]
        N._check(N.lib().gdn_kv4_attention(self._dims(q_row, kv_row), self.layers, None if sched is None else ctypes.byref(sched.struct),
                                           q.data_ptr(), None if k_new is None else k_new.data_ptr(),
                                           None if v_new is None else v_new.data_ptr(), out.data_ptr(), cache, max_len,
                                           self.workspace.data_ptr(), self.workspace.numel(),
                                           N._stream_of(stream, self._index)))

    def check_error(self, stream=None):
        """Waits for the stream and raises what the calls reported; every call can be made again after it."""
        try:
            N.gdn_check_error_words(self.err, stream)
        except N.GdnError as e:
            if e.status == N.GDN_ERR_TIMEOUT:       # CTAs that left early have not counted themselves
                self.workspace.zero_()
                _finish_fills(self.device)
            raise


class TreeAcceptor:
    """Outputs, error words and workspace of the acceptance of drafted tokens for one batch shape."""

    def __init__(self, B: int, n_max: int, V: int, device="cuda"):
        self.B, self.n_max, self.V = B, n_max, V
        self.device = torch.device(device)
        i32 = dict(dtype=torch.int32, device=self.device)
        self.path = torch.full((B, n_max), -1, **i32)
        self.len = torch.zeros(B, **i32)
        self.next = torch.zeros(B, **i32)
        self.err = torch.zeros(4, **i32)
        self.ws_bytes = N.gdn_accept_workspace_bytes(B, n_max, V)
        self.workspace = torch.zeros(max(self.ws_bytes, 256), dtype=torch.uint8, device=self.device)
        self._index = self.path.get_device()
        self._out = (self.path.data_ptr(), self.len.data_ptr(), self.next.data_ptr(), self.err.data_ptr(),
                     self.workspace.data_ptr(), self.workspace.numel())
        _finish_fills(self.device)

    def _rows(self, t: torch.Tensor, name: str) -> int:
        want = (self.B, self.n_max, self.V)
        if t.shape != want or t.get_device() != self._index:
            raise ValueError(f"{name} is {want} on {self.device}, got {tuple(t.shape)} on {t.device}")
        if t.is_contiguous():
            return self.V
        row = t.stride(1) if self.n_max > 1 else t.stride(0) if self.B > 1 else self.V
        if (self.V > 1 and t.stride(2) != 1) or (self.B > 1 and t.stride(0) != self.n_max * row):
            raise ValueError(f"{name} has strides {t.stride()}: rows need one stride and contiguous values")
        return _stride_in_range(row, self.V, name)

    def _small(self, t: Optional[torch.Tensor], name: str, shape: tuple, dtype: torch.dtype) -> int:
        if t is None:
            raise ValueError(f"{name} is needed where a temperature is given")
        if t.shape != shape or t.dtype is not dtype or not t.is_contiguous() or t.get_device() != self._index:
            raise ValueError(f"{name} is a contiguous {dtype} tensor {shape} on {self.device}, got {tuple(t.shape)} "
                             f"{t.dtype} on {t.device}")
        return t.data_ptr()

    def accept(self, sched: DeviceSchedule, logits: torch.Tensor, tokens: torch.Tensor,
               uniform: Optional[torch.Tensor] = None, gumbel: Optional[torch.Tensor] = None,
               temperature: Optional[torch.Tensor] = None, draft_probs: Optional[torch.Tensor] = None, stream=None):
        """Walk every request's tree -> (path [B, n_max] padded with -1, len [B], next [B]), this object's buffers;
        path and len go into TreeVerifier.commit and KV4Cache.append as they are.  temperature None: greedy."""
        row = self._rows(logits, "logits")
        tok = self._small(tokens, "tokens", (self.B, self.n_max), torch.int32)
        if sched.struct.B != self.B or sched.struct.n_max != self.n_max:
            raise ValueError("the schedule's batch is not this object's")
        u = g = t = dp = None
        if temperature is not None:
            t = self._small(temperature, "temperature", (self.B,), torch.float32)
            u = self._small(uniform, "uniform", (self.B, self.n_max), torch.float32)
            g = self._small(gumbel, "gumbel", (self.B, self.V), torch.float32)
        draft = N.GDN_DTYPE_F32
        if draft_probs is not None:
            draft = _dtype_code(draft_probs.dtype, "draft_probs")
            if self._rows(draft_probs, "draft_probs") != row:
                raise ValueError("draft_probs and logits have different row strides")
            dp = draft_probs.data_ptr()
        N._check(N.lib().gdn_tree_accept(ctypes.byref(sched.struct), self.V, row, _dtype_code(logits.dtype, "logits"),
                                         logits.data_ptr(), tok, dp, draft, u, g, t, *self._out,
                                         N._stream_of(stream, self._index)))
        return self.path, self.len, self.next

    def check_error(self, stream=None):
        N.gdn_check_error_words(self.err, stream)
