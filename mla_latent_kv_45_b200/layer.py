"""An MLA layer through the C-ABI calls: one decode step, or a chunk of a prompt.

The order is the pages' per-token inference flow ("解耦 RoPE（MLA 下）" §五):
append the new token's [c ; k_R] row, build the absorbed query, attend over
the whole cache (the new row included), then up-project.  Device tensors only;
every step runs in the CUDA library.

A prompt takes many tokens of several sequences at once and attends in the
expanded form ("解耦 RoPE（MLA 下）" §七 ``forward_naive``), where the weights are
plain matrix products of torch around the library's calls.
"""

from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L


class DecodeLayer:
    """Weights of one layer (device tensors, ``[out, in]`` layout) plus a workspace."""

    def __init__(self, dims: L.Dims, weights: dict, batch: int, num_splits: int = 0,
                 device="cuda"):
        self.dims = dims
        self.w = weights
        self.batch = batch
        self.num_splits = num_splits
        self.d_model = weights["W_DKV"].shape[1]
        self.d_q = weights["W_DQ"].shape[0] if weights.get("W_DQ") is not None else 0
        nbytes = L.mla_workspace_size(dims, batch, self.d_model, self.d_q, num_splits)
        if nbytes == 0:
            raise ValueError("unsupported dims for the workspace")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        L.mla_workspace_init(self.ws)
        # the cache append runs on a second stream, beside the query absorption
        # (the two only meet at the attention), with a workspace of its own
        self.ws_append = torch.empty(nbytes, dtype=torch.uint8, device=device)
        L.mla_workspace_init(self.ws_append)
        self.side = torch.cuda.Stream(device=device)
        H, dt = dims.n_heads, dims.torch_dtype
        self.q_lat = torch.empty(batch, H, dims.d_c + dims.d_rope, dtype=dt, device=device)
        self.z = torch.empty(batch, H, dims.d_c, dtype=dt, device=device)
        self.lse = torch.empty(batch, H, dtype=torch.float32, device=device)
        d_out = self.d_model if weights.get("W_O") is not None else H * dims.d_v
        self.out = torch.empty(batch, d_out, dtype=dt, device=device)

    def step(self, cache: L.PagedCache, h: torch.Tensor, positions: torch.Tensor,
             stream=None, events=None) -> torch.Tensor:
        """Appends h's rows at ``positions`` and returns the layer output.

        ``cache.seq_lens`` must already count the new rows (positions + 1).
        The append runs on a side stream concurrently with the query absorption;
        the attention waits for both.  ``events`` (7 CUDA events, optional) are
        recorded around each call: append [0, 1] on the side stream, absorb
        [2, 3], attention [4, 5] and un-absorption [5, 6] on the main stream.
        """
        w, d = self.w, self.dims
        main = stream if stream is not None else torch.cuda.current_stream()
        side = self.side
        side.wait_stream(main)
        if events:
            events[0].record(side)
        L.mla_cache_append(d, cache, h, w["W_DKV"], w["W_KR"], w["gamma"], positions,
                           self.ws_append, side)
        if events:
            events[1].record(side)
            events[2].record(main)
        L.mla_absorb_q(d, h, w.get("W_DQ"), w["W_UQ"], w["W_QR"], w["W_UK"], positions,
                       self.q_lat, self.ws, main)
        if events:
            events[3].record(main)
        main.wait_stream(side)
        if events:
            events[4].record(main)
        L.mla_decode_attn(d, cache, self.q_lat, self.z, self.lse, self.num_splits, self.ws, main)
        if events:
            events[5].record(main)
        L.mla_unabsorb_out(d, self.z, w["W_UV"], w.get("W_O"), self.out, self.ws, main)
        if events:
            events[6].record(main)
        return self.out

    def capture(self, cache: L.PagedCache, h: torch.Tensor, positions: torch.Tensor
                ) -> "StepGraph":
        """The decode step over these buffers, captured once as a CUDA graph.

        The graph reads ``h``, ``positions``, ``cache.seq_lens`` and the cache
        in place and writes ``self.out`` (and the cache row): copy each step's
        inputs into those buffers and call ``replay()``.  One eager step runs
        first so that every one-time set-up (per-device kernel attributes)
        happens outside the capture.
        """
        self.step(cache, h, positions)
        torch.cuda.synchronize()
        return StepGraph(lambda s: self.step(cache, h, positions, s), self.out)

    def device_error(self) -> int:
        """Synchronises; returns the first nonzero device status of both workspaces."""
        st = L.mla_get_device_error(self.ws_append, self.side)
        st2 = L.mla_get_device_error(self.ws)
        return st if st != 0 else st2


class PromptLayer:
    """A chunk of new tokens of several sequences through one layer.

    Weights as for ``DecodeLayer``; buffers for ``tokens`` new tokens of ``batch``
    sequences that have ``rows`` cached rows in all once the chunk is appended.
    Prompts may come in one chunk or in several: a chunk attends over everything its
    sequences have in the cache.  The same cache then serves ``DecodeLayer``.  The weights
    are laid out when the layer is made (W_DKV and W_KR are copied, the others are views): make
    another after changing them.  Nothing is recorded for a backward pass.
    """

    @torch.inference_mode(False)      # buffers that later steps may write in either mode
    @torch.no_grad()
    def __init__(self, dims: L.Dims, weights: dict, batch: int, tokens: int, rows: int,
                 device="cuda"):
        if min(batch, tokens, rows) < 1:
            raise ValueError(f"no buffers for {batch} sequences, {tokens} tokens, {rows} rows")
        nbytes = L.mla_prompt_workspace_size(dims, batch, tokens)
        if nbytes == 0:
            raise ValueError("unsupported dims for the workspace")
        self.dims, self.batch, self.tokens, self.n_rows = dims, batch, tokens, rows
        w, dt, H = weights, dims.torch_dtype, dims.n_heads
        # [out, in] weights as the right-hand sides of the products; the two
        # projections of the cache row become one
        self.w_row = torch.cat([w["W_DKV"], w["W_KR"]]).T
        self.w_dq = None if w.get("W_DQ") is None else w["W_DQ"].T
        self.w_uq, self.w_qr = w["W_UQ"].T, w["W_QR"].T
        self.w_uk, self.w_uv = w["W_UK"].T, w["W_UV"].T
        self.w_o = None if w.get("W_O") is None else w["W_O"].T
        self.gamma = w["gamma"]
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        with torch.cuda.device(self.ws.device):     # (the current stream is the layer's device's)
            L.mla_workspace_init(self.ws)
        new = lambda *s: torch.empty(*s, dtype=dt, device=device)  # noqa: E731
        # the projections of the cache row stay in fp32 until they are normalised and
        # rotated, as in the decode step
        self.x = torch.empty(tokens, dims.d_c + dims.d_rope, dtype=torch.float32, device=device)
        self.c_q = None if self.w_dq is None else new(tokens, self.w_dq.shape[1])
        self.q_nope, self.q_rope = new(tokens, H, dims.d_nope), new(tokens, H, dims.d_rope)
        self.rows = new(rows, dims.d_c + dims.d_rope)
        self.k_nope, self.v = new(rows, H, dims.d_nope), new(rows, H, dims.d_v)
        self.o = new(tokens, H, dims.d_v)
        self.lse = torch.empty(tokens, H, dtype=torch.float32, device=device)
        self.out = (self.o.view(tokens, -1) if self.w_o is None
                    else new(tokens, self.w_o.shape[1]))

    @torch.no_grad()
    def step(self, cache: L.PagedCache, h: torch.Tensor, cu_tokens: torch.Tensor,
             ctx_lens: Optional[torch.Tensor], cu_rows: torch.Tensor, stream=None) -> torch.Tensor:
        """The layer output of the tokens ``h`` ``[tokens, d_model]``.

        Sequence b's new tokens are rows ``cu_tokens[b] .. cu_tokens[b+1]`` of h and
        follow the ``ctx_lens[b]`` rows (None: no rows) that it has in the cache;
        ``cu_rows`` are the offsets of all its rows, cu_rows[b+1] - cu_rows[b] =
        ctx_lens[b] + cu_tokens[b+1] - cu_tokens[b] (int32 device tensors, all read
        on the device).  cache.seq_lens is not read.  Output rows of tokens that no sequence
        has mean nothing.  The result is the layer's buffer; the inputs have to stay as they are
        until ``stream`` (None: the current one) has come past the step.
        """
        if h.shape[0] != self.tokens:     # (the products would resize their outputs)
            raise ValueError(f"h has {h.shape[0]} tokens, the buffers are for {self.tokens}")
        s = stream if stream is not None else torch.cuda.current_stream(self.ws.device)
        d = self.dims
        with torch.cuda.stream(s):
            torch.mm(h, self.w_row, out_dtype=torch.float32, out=self.x)
            c_q = h if self.c_q is None else torch.mm(h, self.w_dq, out=self.c_q)
            torch.mm(c_q, self.w_uq, out=self.q_nope.view(self.tokens, -1))
            torch.mm(c_q, self.w_qr, out=self.q_rope.view(self.tokens, -1))
            L.mla_prompt_append(d, cache, self.x, self.gamma, cu_tokens, ctx_lens, self.q_rope,
                                self.q_rope, self.ws, s)
            L.mla_cache_gather(d, cache, cu_rows, None, self.rows, self.ws, s)
            c = self.rows[:, :d.d_c]
            torch.mm(c, self.w_uk, out=self.k_nope.view(self.n_rows, -1))
            torch.mm(c, self.w_uv, out=self.v.view(self.n_rows, -1))
            L.mla_prompt_attn(d, self.q_nope, self.q_rope, self.k_nope, self.rows[:, d.d_c:],
                              self.v, cu_tokens, cu_rows, self.o, self.lse, self.ws, s)
            if self.w_o is not None:
                torch.mm(self.o.view(self.tokens, -1), self.w_o, out=self.out)
        return self.out

    def capture(self, cache: L.PagedCache, h: torch.Tensor, cu_tokens: torch.Tensor,
                ctx_lens: Optional[torch.Tensor], cu_rows: torch.Tensor) -> "StepGraph":
        """The chunk over these buffers as a CUDA graph; lengths are read at replay."""
        with torch.cuda.device(self.ws.device):
            self.step(cache, h, cu_tokens, ctx_lens, cu_rows)
            torch.cuda.synchronize()
            return StepGraph(lambda s: self.step(cache, h, cu_tokens, ctx_lens, cu_rows, s),
                             self.out)

    def device_error(self) -> int:
        """Waits for the layer's device (a step or a replay may be on any stream of it); returns
        the device status of the workspace."""
        with torch.cuda.device(self.ws.device):
            torch.cuda.synchronize()
            return L.mla_get_device_error(self.ws)


class StepGraph:
    """A CUDA graph of one call sequence issued by ``fn(stream)``; ``replay``
    launches the same kernels on the current stream with no per-kernel host
    work."""

    def __init__(self, fn, out: torch.Tensor):
        self.out = out
        self.graph = torch.cuda.CUDAGraph()
        main = torch.cuda.current_stream()
        cap = torch.cuda.Stream(device=main.device)
        cap.wait_stream(main)
        with torch.cuda.stream(cap):
            with torch.cuda.graph(self.graph, stream=cap):
                fn(cap)
        main.wait_stream(cap)

    def replay(self) -> torch.Tensor:
        self.graph.replay()
        return self.out
