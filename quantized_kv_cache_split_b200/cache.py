"""A paged, block-quantized KV cache on one GPU, driven through libkvq.

PyTorch supplies device memory and the stream; every computation (quantizing
appended K/V, split-KV decode attention with sparse V, the log-sum-exp merge)
is a libkvq call.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np
import torch

from . import _binding as kb


class QuantizedKVCache:
    """K and V planes of one attention layer.

    Layout (per plane pair): codes uint8 [num_pages, num_kv_heads, page_size, row_bytes],
    scales fp16 [num_pages, num_kv_heads, page_size, scale_count].  A contiguous
    cache is page_size = capacity with one page per sequence.
    """

    def __init__(self, fmt: str, head_dim: int, num_kv_heads: int, page_size: int, num_pages: int,
                 device="cuda", codebook: Optional[torch.Tensor] = None,
                 signs: Optional[torch.Tensor] = None):
        self.fmt = fmt
        self.head_dim = head_dim
        self.num_kv_heads = num_kv_heads
        self.page_size = page_size
        self.num_pages = num_pages
        self.device = torch.device(device)
        row = kb.kvq_code_row_bytes(fmt, head_dim)
        nsc = kb.kvq_scale_row_count(fmt, head_dim)
        if row == 0 or nsc == 0:
            raise kb.KvqError("QuantizedKVCache", kb.KVQ_ERR_UNSUPPORTED)
        shape = (num_pages, num_kv_heads, page_size)
        self.k_codes = torch.zeros(shape + (row,), dtype=torch.uint8, device=self.device)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_scales = torch.zeros(shape + (nsc,), dtype=torch.float16, device=self.device)
        self.v_scales = torch.zeros_like(self.k_scales)
        self.codebook = None
        self.signs = None
        if fmt == "lut4":
            if codebook is None:
                cb = kb.kvq_lloyd_max_codebook(16, 1.0 / math.sqrt(head_dim))
                codebook = torch.from_numpy(cb.view(np.int16).copy())
            self.codebook = codebook.to(self.device).contiguous()
            if signs is None:
                raise ValueError("lut4 needs the rotation signs")
            self.signs = signs.to(device=self.device, dtype=torch.int8).contiguous()
        self.desc = kb.make_desc(fmt, head_dim, num_kv_heads, page_size, num_pages,
                                 self.codebook, self.signs)
        self._ws = None
        self._index = _cuda_index(self.device)
        self._ws_rows = {}       # prompt and prefix attention: a workspace per stream
        self._rows_bytes = {}    # workspace bytes of recent request shapes
        self._flags = torch.zeros(256, dtype=torch.uint8, device=self.device)  # their flag word
        _settle(self.device)

    # ---------------------------------------------------------------- writes
    def write(self, k: torch.Tensor, v: torch.Tensor, slots: Optional[torch.Tensor] = None,
              stream=None):
        """Quantize fp16 K/V [n_tokens, num_kv_heads, head_dim] into physical ``slots``."""
        n = k.shape[0]
        kb.kvq_quantize_kv(self.desc, k, v, n, slots, self.k_codes, self.k_scales, self.v_codes,
                           self.v_scales, stream)

    # ---------------------------------------------------------------- decode
    def workspace(self, batch: int, num_q_heads: int, max_seq_len: int, split_tokens: int,
                  options: int = 0):
        L = kb.kvq_resolve_split(self.desc, batch, num_q_heads, max_seq_len, split_tokens, options)
        nbytes = kb.kvq_workspace_size(batch, num_q_heads, self.head_dim, max_seq_len, L)
        if self._ws is None or self._ws.numel() < nbytes:
            self._ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            kb.kvq_workspace_init(self._ws, self._ws.numel())  # once; any later shape reuses it
        return self._ws, nbytes, L

    def attention(self, q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                  page_table: Optional[torch.Tensor] = None, max_pages: int = 1,
                  tau: float = 1e-6, sm_scale: Optional[float] = None, split_tokens: int = 0,
                  out: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None,
                  max_scope: str = "split", fused: bool = True, v_fetch: str = "auto",
                  stream=None) -> torch.Tensor:
        """Decode attention of q [batch, num_q_heads, head_dim] (fp16) -> fp32 output.

        ``fused``: merge the split partials inside the decode kernel (one launch);
        otherwise kvq_combine merges them in a second launch.  ``max_scope``: the running
        maximum the skip test uses: "split" (each split's own), "cluster" (shared by the
        splits of a thread-block cluster) or "sequence" (over all splits of the
        sequence and KV head).  ``v_fetch``: how V rows reach the SM when tau > 0:
        "kept" (only the kept rows, after the skip test), "with_k" (every V tile with its
        K tile; skipped rows are left out of the contraction only) or "auto" (with_k);
        the result is the same.  ``stream``: as for prompt_attention.  Make one call of a shape
        before capturing it: the workspace is cleared when it is made."""
        other = _elsewhere(stream, self._index)
        if other is not None:
            return _run_on(other, self._index, out, self.attention, q, seq_lens, max_seq_len, page_table, max_pages, tau,
                           sm_scale, split_tokens, out, stats, max_scope, fused, v_fetch)
        scopes = {"split": 0, "cluster": kb.KVQ_OPT_SHARED_MAX, "sequence": kb.KVQ_OPT_GLOBAL_MAX}
        fetches = {"auto": 0, "kept": kb.KVQ_OPT_V_KEPT_ONLY, "with_k": kb.KVQ_OPT_V_WITH_K}
        if max_scope not in scopes:
            raise ValueError(f"max_scope must be one of {sorted(scopes)}, not {max_scope!r}")
        if v_fetch not in fetches:
            raise ValueError(f"v_fetch must be one of {sorted(fetches)}, not {v_fetch!r}")
        B, Hq, D = q.shape
        if sm_scale is None:
            sm_scale = 1.0 / math.sqrt(D)
        opts = scopes[max_scope]
        ws, nbytes, L = self.workspace(B, Hq, max_seq_len, split_tokens, opts)
        opts |= fetches[v_fetch]
        if out is None:
            out = torch.empty((B, Hq, D), dtype=torch.float32, device=self.device)
        kb.kvq_decode_attn(self.desc, q, B, Hq, self.k_codes, self.k_scales, self.v_codes,
                           self.v_scales, page_table, max_pages, seq_lens, max_seq_len, sm_scale,
                           tau, L, ws, nbytes, stats, out if fused else None, opts, stream)
        if not fused:
            kb.kvq_combine(self.desc, ws, B, Hq, max_seq_len, L, seq_lens, out, opts, stream)
        return out

    # ---------------------------------------------------------------- prompts, shared prefixes
    def _rows_call(self, kind, size_fn, args, q, out, out_dtype, sm_scale):
        """Checks of q and out, the workspace, the output, the scale and the stream of a call on
        torch's current stream."""
        D = self.head_dim
        if q.dim() != 3 or q.shape[2] != D:
            raise ValueError(f"q must be [tokens, heads, {D}], not {tuple(q.shape)}")
        _want("q", q, torch.float16, self._index)
        if out is None:
            out = torch.empty_like(q) if out_dtype is torch.float16 else torch.empty_like(q, dtype=out_dtype)
        elif out.shape != q.shape:
            raise ValueError(f"out must have q's shape {tuple(q.shape)}, not {tuple(out.shape)}")
        out_type = _OUT_TYPES.get(out.dtype)
        if out_type is None:
            raise ValueError(f"the output is float32 or float16, not {out.dtype}")
        _want("out", out, out.dtype, self._index)
        stream = _raw_stream(self._index)
        key = (kind,) + args
        nbytes = self._rows_bytes.get(key)
        if nbytes is None:
            if len(self._rows_bytes) >= 64:
                self._rows_bytes.clear()
            nbytes = self._rows_bytes[key] = size_fn(self.desc, *args)
        if torch._C._cuda_isCurrentStreamCapturing():
            # the graph's own memory: no other graph and no later call uses it
            ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        else:
            ws = self._ws_rows.get(stream)
            if ws is None or ws.numel() < nbytes:
                # an outgrown one goes back to its stream's memory; a quarter more than it, so that
                # slowly growing requests do not ask for another each time
                size = max(nbytes, 256, 0 if ws is None else ws.numel() * 5 // 4)
                self._ws_rows[stream] = ws = None
                ws = self._ws_rows[stream] = torch.empty(size, dtype=torch.uint8, device=self.device)
        return ws, out, out_type, 1.0 / math.sqrt(D) if sm_scale is None else sm_scale, stream

    def prompt_attention(self, q: torch.Tensor, token_offsets: torch.Tensor, seq_lens: torch.Tensor,
                         max_seq_len: int, page_table: Optional[torch.Tensor] = None,
                         max_pages: int = 1, causal: bool = True, sm_scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                         stream=None) -> torch.Tensor:
        """Attention of each request's new tokens over its positions in the cache.

        ``q`` [n_tokens, num_q_heads, head_dim] (fp16): the new tokens of all requests,
        packed; request b's are rows ``token_offsets[b]`` .. ``token_offsets[b + 1] - 1``
        and the last ones of its ``seq_lens[b]`` positions (write their K and V first).
        ``causal``: a token sees the positions up to its own.  Rows outside every request are
        padding and keep what ``out`` holds there.  Lengths, offsets and the table are int32
        tensors on the cache's GPU.

        ``max_seq_len`` bounds the lengths, and how the work is cut follows it: pass the nearest
        bound that the host knows (a quarter of it used costs up to three times the time).

        ``stream`` (a torch stream or a handle): launch there instead of on the current stream.
        The inputs must be ready for it and stay alive until the call has run; a new output
        belongs to that stream's memory, so wait for the stream before using it elsewhere.

        The workspace is kept per stream, and a captured call has one of its own in its graph's
        memory: calls on different streams and replays of different graphs may overlap."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.prompt_attention(q, token_offsets, seq_lens, max_seq_len, page_table, max_pages, causal,
                                             sm_scale, out, out_dtype, stream)
        other = _elsewhere(stream, self._index)
        if other is not None:
            return _run_on(other, self._index, out, self.prompt_attention, q, token_offsets, seq_lens, max_seq_len,
                           page_table, max_pages, causal, sm_scale, out, out_dtype)
        B = seq_lens.numel()
        _want("seq_lens", seq_lens, torch.int32, self._index)
        _want("token_offsets", token_offsets, torch.int32, self._index, B + 1)
        if page_table is not None:
            _want("page_table", page_table, torch.int32, self._index, B * max_pages)
        n, Hq = q.shape[0], q.shape[1]
        ws, out, out_type, sm_scale, stream = self._rows_call("prompt", kb.kvq_prompt_workspace_size, (n, Hq, B, max_seq_len),
                                                          q, out, out_dtype, sm_scale)
        kb.kvq_prompt_attn(self.desc, q, n, Hq, self.k_codes, self.k_scales, self.v_codes, self.v_scales, page_table,
                           max_pages, seq_lens, max_seq_len, token_offsets, B, causal, sm_scale, ws, ws.numel(), out,
                           out_type, stream, flags=self._flags)
        return out

    def prefix_attention(self, q: torch.Tensor, prefix_table: Optional[torch.Tensor],
                         prefix_lens: torch.Tensor, max_prefix_len: int, seq_lens: torch.Tensor,
                         max_seq_len: int, page_table: Optional[torch.Tensor] = None,
                         max_pages: int = 1, group_offsets: Optional[torch.Tensor] = None,
                         max_prefix_pages: Optional[int] = None, sm_scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, out_dtype=torch.float32,
                         stream=None) -> torch.Tensor:
        """Decode attention of q [batch, num_q_heads, head_dim] (fp16) for requests that share
        prefixes: group g (requests ``group_offsets[g]`` .. ``group_offsets[g + 1] - 1``; None:
        one group of all) attends to the ``prefix_lens[g]`` positions of row g of
        ``prefix_table`` and each request to its own ``seq_lens[b]`` positions as well.  The
        prefix is read once per group, not once per request.  Lengths, offsets and tables are
        int32 tensors on the cache's GPU.  ``stream`` and the workspace: as for prompt_attention."""
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self._index):
                return self.prefix_attention(q, prefix_table, prefix_lens, max_prefix_len, seq_lens, max_seq_len,
                                             page_table, max_pages, group_offsets, max_prefix_pages, sm_scale, out,
                                             out_dtype, stream)
        other = _elsewhere(stream, self._index)
        if other is not None:
            return _run_on(other, self._index, out, self.prefix_attention, q, prefix_table, prefix_lens, max_prefix_len,
                           seq_lens, max_seq_len, page_table, max_pages, group_offsets, max_prefix_pages, sm_scale, out,
                           out_dtype)
        B, ng = q.shape[0], prefix_lens.numel()
        if max_prefix_pages is None:
            if prefix_table is None:
                raise ValueError("max_prefix_pages is needed without a prefix_table")
            max_prefix_pages = prefix_table.shape[-1]
        _want("prefix_lens", prefix_lens, torch.int32, self._index)
        _want("seq_lens", seq_lens, torch.int32, self._index, B)
        if prefix_table is not None:
            _want("prefix_table", prefix_table, torch.int32, self._index, ng * max_prefix_pages)
        if group_offsets is not None:
            _want("group_offsets", group_offsets, torch.int32, self._index, ng + 1)
        if page_table is not None:
            _want("page_table", page_table, torch.int32, self._index, B * max_pages)
        Hq = q.shape[1]
        ws, out, out_type, sm_scale, stream = self._rows_call(
            "prefix", kb.kvq_prefix_workspace_size, (B, Hq, ng, max_prefix_len, max_seq_len), q, out, out_dtype, sm_scale)
        kb.kvq_prefix_attn(self.desc, q, B, Hq, self.k_codes, self.k_scales, self.v_codes, self.v_scales, prefix_table,
                           max_prefix_pages, prefix_lens, max_prefix_len, group_offsets, ng, page_table, max_pages,
                           seq_lens, max_seq_len, sm_scale, ws, ws.numel(), out, out_type, stream,
                           flags=self._flags)
        return out

    def device_flags(self) -> int:
        """KVQ_FLAG_* bits of the calls so far, replays of captured ones among them."""
        torch.cuda.synchronize(self._index)  # their streams
        flags = kb.kvq_read_device_flags(self._flags)
        return flags if self._ws is None else flags | kb.kvq_read_device_flags(self._ws)


def _want(name: str, t: torch.Tensor, dtype: torch.dtype, index: int, numel: Optional[int] = None) -> None:
    """The kernels read plain contiguous memory of the cache's GPU: refuse anything else."""
    if t.dtype is not dtype or not t.is_contiguous() or t.get_device() != index or (
            numel is not None and t.numel() != numel):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{index}"
                         + (f" of {numel} elements" if numel is not None else "")
                         + f", not {t.dtype} {tuple(t.shape)} on {t.device}"
                         + ("" if t.is_contiguous() else " (not contiguous)"))


def _cuda_index(device: torch.device) -> int:
    """The GPU of a device ("cuda" is the current one); -1 without one."""
    if device.type != "cuda":
        return -1
    return torch.cuda.current_device() if device.index is None else device.index


def _settle(device: torch.device) -> None:
    """Wait until buffers just made hold their first values: their first use may be on any stream."""
    if device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(device).synchronize()


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _elsewhere(stream, index: int):
    """The torch stream of a call's ``stream`` argument when that is not the current one, else None."""
    if stream is None:
        return None
    raw = kb._stream(stream)
    if raw == 1:  # the legacy default stream's other name
        raw = 0
    if raw == _raw_stream(index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(raw, device=index) if raw else torch.cuda.default_stream(index)


def _run_on(other, index: int, out, method, *args):
    """method(*args) with ``other`` as the current stream, so that what it allocates is that
    stream's memory: torch reuses a freed block in the order of the stream that it belongs to, and
    of no other.  The current stream is expected to use a new output later on."""
    here = torch.cuda.current_stream(index)
    with torch.cuda.stream(other):
        res = method(*args)
    if out is None:
        res.record_stream(here)
    return res


_OUT_TYPES = {torch.float32: kb.KVQ_OUT_F32, torch.float16: kb.KVQ_OUT_F16}


class PagePlanner:
    """The page bookkeeping of serving steps on the GPU (kvq_plan_step).

    Owns the buffers a step writes: ``seq_lens`` [batch], ``token_offsets`` [batch + 1],
    ``slots`` and ``positions`` [max_tokens], ``free_count`` [1].  The page table and the stack
    of free pages are the caller's and are updated in place; pass ``planner.seq_lens`` and
    ``planner.free_count`` back in for the next step to keep the whole state on the GPU."""

    def __init__(self, batch: int, page_size: int, num_pages: int, max_pages: int, max_tokens: int,
                 device="cuda"):
        self.batch, self.page_size, self.num_pages = batch, page_size, num_pages
        self.max_pages, self.max_tokens = max_pages, max_tokens
        self.device = torch.device(device)
        self._index = _cuda_index(self.device)
        ints = lambda n: torch.zeros(n, dtype=torch.int32, device=self.device)  # noqa: E731
        self.seq_lens, self.token_offsets, self.free_count = ints(batch), ints(batch + 1), ints(1)
        self.slots, self.positions = ints(max_tokens).fill_(-1), ints(max_tokens)
        self._ws = torch.zeros(256, dtype=torch.uint8, device=self.device)
        _settle(self.device)

    def step(self, new_lens: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
             free_pages: torch.Tensor, free_count: torch.Tensor, stream=None) -> None:
        """Plan one step: ``new_lens[b]`` tokens to append per request, -1 where it ends.  All
        are int32 tensors on the planner's GPU: ``page_table`` [batch, max_pages],
        ``free_pages`` [num_pages]."""
        i = self._index
        if torch.cuda.current_device() != i:
            with torch.cuda.device(i):
                return self.step(new_lens, page_table, seq_lens, free_pages, free_count, stream)
        _want("new_lens", new_lens, torch.int32, i, self.batch)
        _want("page_table", page_table, torch.int32, i, self.batch * self.max_pages)
        _want("seq_lens", seq_lens, torch.int32, i, self.batch)
        _want("free_pages", free_pages, torch.int32, i)
        if free_pages.numel() < self.num_pages:
            raise ValueError(f"free_pages must hold num_pages = {self.num_pages} entries, not {free_pages.numel()}")
        _want("free_count", free_count, torch.int32, i, 1)
        kb.kvq_plan_step(self.batch, self.page_size, self.num_pages, self.max_pages, self.max_tokens,
                         seq_lens, new_lens, free_pages, free_count, page_table, self.seq_lens,
                         self.free_count, self.token_offsets, self.slots, self.positions, self._ws,
                         256, _raw_stream(i) if stream is None else stream)

    def device_flags(self) -> int:
        """KVQ_FLAG_* bits of the steps so far (a flagged step changed nothing)."""
        torch.cuda.synchronize(self._index)  # the steps' streams
        return kb.kvq_read_device_flags(self._ws)
