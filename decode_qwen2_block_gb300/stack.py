"""A stack of decoder blocks driven through the C ABI.

Runs one phase over every layer in order (layer l's output is layer l+1's
input), with the BLK_FLAG_CHAIN promise set so that each layer's first
kernel overlaps the previous layer's last kernel, and can capture a decode
step into a CUDA graph (one graph per cache length, since cache_len is a
by-value argument).  All work is the library's kernels; torch only supplies
device memory, streams and graphs.
"""
from __future__ import annotations

import ctypes

import torch

from . import (BLK_ERR_CACHE_OVERFLOW, BLK_ERR_PAGE, BLK_ERR_SHAPE, BLK_OK, BlkError, Block,
               BlkQWeights, BlkWeights, blk_decode_batch_stack,
               blk_decode_batch_stack_workspace_bytes, blk_decode_stack, blk_decode_stack_q,
               blk_prefill_stack, blk_prefill_stack_workspace_bytes, blk_step_paged_stack)


class LayerStack:
    def __init__(self, shape, layer_weights, max_ctx: int, max_T: int, caches=None,
                 chain: bool = True, device="cuda"):
        """layer_weights: list of dicts of fp16 CUDA tensors (one per layer).
        caches: optional list of (k_cache, v_cache) per layer; allocated
        (zero-filled) when None."""
        self.shape = shape
        self.n_layers = len(layer_weights)
        self.block = Block(shape, max_ctx, chain=chain)
        self.wdev = layer_weights
        self.w = [Block.weights(wd) for wd in layer_weights]
        H, Hkv, D = shape.hidden, shape.n_kv_heads, shape.head_dim
        if caches is None:
            caches = [(torch.zeros((Hkv, max_ctx, D), dtype=torch.float16, device=device),
                       torch.zeros((Hkv, max_ctx, D), dtype=torch.float16, device=device))
                      for _ in range(self.n_layers)]
        self.caches = caches
        # one workspace for every call: the one-layer calls, decode, and the
        # prefill stack (which also keeps its activation buffers in it)
        nbytes = max(self.block.workspace_bytes(max_T),
                     blk_prefill_stack_workspace_bytes(self.block.handle, max_T))
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.max_T = max_T
        # ping-pong activations between layers
        self.bufs = [torch.empty((max_T, H), dtype=torch.float16, device=device) for _ in range(2)]
        self.graphs = {}
        n = self.n_layers
        self._w_arr = (BlkWeights * n)(*self.w)
        self._kc_arr = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc, _ in caches])
        self._vc_arr = (ctypes.c_void_p * n)(*[vc.data_ptr() for _, vc in caches])

    def decode_step(self, x, pos, cache_len: int, out=None, stream=None):
        """One token through every layer in one library call (blk_decode_stack).
        Returns the last layer's output."""
        out = self.bufs[0][:1] if out is None else out
        s = torch.cuda.current_stream() if stream is None else stream
        rc = blk_decode_stack(self.block.handle, self._w_arr, self.n_layers, self._kc_arr,
                              self._vc_arr, x.data_ptr(), pos.data_ptr(), cache_len,
                              out.data_ptr(), None, None, self.ws.data_ptr(),
                              self.ws.numel(), s.cuda_stream)
        if rc != BLK_OK:
            raise BlkError(rc, "blk_decode_stack")
        return out

    def prefill_step(self, x, pos, cache_len: int, out=None, stream=None):
        """T new tokens through every layer in one library call
        (blk_prefill_stack; prefill when cache_len is 0, else prefill_kv).
        Returns the last layer's output."""
        T = x.shape[0]
        out = self.bufs[0][:T] if out is None else out
        s = torch.cuda.current_stream() if stream is None else stream
        rc = blk_prefill_stack(self.block.handle, self._w_arr, self.n_layers, self._kc_arr,
                               self._vc_arr, x.data_ptr(), pos.data_ptr(), T, cache_len,
                               out.data_ptr(), self.ws.data_ptr(), self.ws.numel(), s.cuda_stream)
        if rc != BLK_OK:
            raise BlkError(rc, "blk_prefill_stack")
        return out

    def run(self, phase: str, x, pos, cache_len: int, layer_outputs=None, stream=None):
        """Runs `phase` over all layers; returns the last layer's output (a
        view of an internal buffer).  layer_outputs, if given, is a list that
        receives a copy of each layer's input (for layer-local checks); the
        layers then run as one call each."""
        T = x.shape[0]
        if phase == "decode" and layer_outputs is None:
            return self.decode_step(x, pos, cache_len, stream=stream)
        if layer_outputs is None:
            return self.prefill_step(x, pos, 0 if phase == "prefill" else cache_len,
                                     stream=stream)
        cur = x
        for l in range(self.n_layers):
            out = self.bufs[l % 2][:T]
            if layer_outputs is not None:
                layer_outputs.append(cur.clone())
            kc, vc = self.caches[l]
            if phase == "decode":
                self.block.decode(self.w[l], cur, pos, cache_len, kc, vc, out, self.ws,
                                  stream=stream)
            elif phase == "prefill":
                self.block.prefill(self.w[l], cur, pos, kc, vc, out, self.ws, stream=stream)
            else:
                self.block.prefill_kv(self.w[l], cur, pos, cache_len, kc, vc, out, self.ws,
                                      stream=stream)
            cur = out
        return cur

    def capture(self, phase: str, x, pos, cache_len: int, key=None):
        """Captures one pass over all layers into a CUDA graph.  x and pos must
        stay alive and at the same address for every replay."""
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                out = self.run(phase, x, pos, cache_len, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        self.graphs[key if key is not None else (phase, cache_len)] = (g, out)
        return g, out


class BatchStack:
    """B sequences, one new token each, through a stack of decoder blocks in
    one library call per step (blk_decode_batch_stack)."""

    def __init__(self, shape, layer_weights, max_ctx: int, max_B: int, caches=None,
                 device="cuda"):
        """layer_weights: list of dicts of fp16 CUDA tensors (one per layer).
        caches: optional list of (k_cache, v_cache) per layer, each
        [max_B, Hkv, max_ctx, D]; allocated (zero-filled) when None.  A step
        with B <= max_B sequences uses the first B of every cache."""
        self.shape = shape
        self.n_layers = len(layer_weights)
        self.block = Block(shape, max_ctx, chain=True)
        self.wdev = layer_weights
        self.w = [Block.weights(wd) for wd in layer_weights]
        Hkv, D = shape.n_kv_heads, shape.head_dim
        if caches is None:
            caches = [(torch.zeros((max_B, Hkv, max_ctx, D), dtype=torch.float16, device=device),
                       torch.zeros((max_B, Hkv, max_ctx, D), dtype=torch.float16, device=device))
                      for _ in range(self.n_layers)]
        self.caches = caches
        self.max_B = max_B
        nbytes = blk_decode_batch_stack_workspace_bytes(self.block.handle, max_B)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        n = self.n_layers
        self._w_arr = (BlkWeights * n)(*self.w)
        self._kc_arr = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc, _ in caches])
        self._vc_arr = (ctypes.c_void_p * n)(*[vc.data_ptr() for _, vc in caches])

    def step(self, x, pos, cache_lens, max_cache_len: int, out, stream=None):
        """x, out: fp16 [B, hidden]; pos, cache_lens: int64 [B] on the device;
        max_cache_len bounds the cache lengths.  Returns out."""
        B = x.shape[0]
        if B > self.max_B:
            raise BlkError(BLK_ERR_SHAPE, "BatchStack.step: B > max_B")
        s = torch.cuda.current_stream() if stream is None else stream
        rc = blk_decode_batch_stack(self.block.handle, self._w_arr, self.n_layers, self._kc_arr,
                                    self._vc_arr, x.data_ptr(), pos.data_ptr(),
                                    cache_lens.data_ptr(), B, max_cache_len, out.data_ptr(),
                                    self.ws.data_ptr(), self.ws.numel(), s.cuda_stream)
        if rc != BLK_OK:
            raise BlkError(rc, "blk_decode_batch_stack")
        return out


class PagedStack:
    """Up to max_seqs sequences through a stack of decoder blocks over a paged
    K/V cache: any number of new tokens per sequence and step (a prompt or a
    chunk of it, drafts, one token), one library call for the step's plan
    (blk_page_plan) and one for all layers (blk_step_paged_stack).

    A sequence takes pages as it grows and gives them back with ``free``.
    ``prefill_prefix`` computes a prefix that every sequence then begins with:
    its pages are held once, and a step reads its keys once for the whole batch
    where that pays.  The host knows the lengths it asked for, so no step waits
    for the GPU.  Steps follow one another whatever streams they are given."""

    def __init__(self, shape, layer_weights, max_ctx: int, n_pages: int, page_size: int,
                 max_seqs: int, max_rows: int, device="cuda"):
        self.shape = shape
        self.n_layers = len(layer_weights)
        self.block = Block(shape, max_ctx, chain=True)
        self.wdev = layer_weights
        self.max_ctx, self.page, self.n_pages = max_ctx, page_size, n_pages
        self.max_seqs, self.max_rows, self.device = max_seqs, max_rows, device
        pool = (n_pages, shape.n_kv_heads, page_size, shape.head_dim)
        self._last = torch.cuda.current_stream()  # the buffers' stream, then the last step's
        self.pools = [(torch.zeros(pool, dtype=torch.float16, device=device),
                       torch.zeros(pool, dtype=torch.float16, device=device))
                      for _ in range(self.n_layers)]
        self.max_blocks = -(-max_ctx // page_size)
        self.table = torch.full((max_seqs, self.max_blocks), -1, dtype=torch.int32, device=device)
        self.prefix = None                       # int32 pages of the shared prefix
        self.prefix_ids: list[int] = []
        self.lens = [0] * max_seqs               # slots of every sequence
        self.pages: list[list[int]] = [[] for _ in range(max_seqs)]   # its own pages
        self.free_ids = list(range(n_pages))
        nbytes = self.block.step_paged_workspace_bytes(max_rows, max_seqs)
        if nbytes == 0:
            raise BlkError(BLK_ERR_SHAPE, "PagedStack: max_rows or max_seqs")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        # with the streams that each is made on or recorded for
        self._held = [(t, [self._last]) for t in (*sum(self.pools, ()), self.table, self.ws)]
        n = self.n_layers
        self._w_arr = (BlkWeights * n)(*[Block.weights(w) for w in layer_weights])
        self._k_arr = (ctypes.c_void_p * n)(*[k.data_ptr() for k, _ in self.pools])
        self._v_arr = (ctypes.c_void_p * n)(*[v.data_ptr() for _, v in self.pools])

    def _ints(self, values, dtype):
        return torch.tensor(values, dtype=dtype).to(self.device, non_blocking=True)

    def _follow(self, stream):
        """The step's stream, behind the last step's.  All that a step makes or writes of the
        runner's own is on it: the current stream may be another one that nothing orders."""
        s = torch.cuda.current_stream() if stream is None else stream
        if s != self._last:
            s.wait_stream(self._last)
            self._last = s
        return s

    def _hold(self, s):
        """The runner's buffers, on a stream other than the one each was made on: their
        memory is not given away under a step that still runs there."""
        for t, streams in self._held:
            if s not in streams:
                t.record_stream(s)
                streams.append(s)

    def _run(self, table, lens, news, x, out, prefix, stream):
        """Plans and runs one step of the sequences of `table`; returns (out, how many of
        free_ids it took)."""
        n, B = x.shape[0], len(lens)
        need = [-(-(have + more) // self.page) - -(-have // self.page)
                for have, more in zip(lens, news)]
        if max(have + more for have, more in zip(lens, news)) > self.max_ctx:
            raise BlkError(BLK_ERR_CACHE_OVERFLOW, "PagedStack.step")
        if sum(need) > len(self.free_ids):
            raise BlkError(BLK_ERR_PAGE, "PagedStack.step: no pages left")
        if n != sum(news) or n > self.max_rows or min(news) < 0:
            raise BlkError(BLK_ERR_SHAPE, "PagedStack.step: rows")
        s = self._follow(stream)
        self._hold(s)
        with torch.cuda.stream(s):
            i64 = torch.int64
            lens_d, news_d = self._ints(lens, i64), self._ints(news, i64)
            free_d = self._ints(self.free_ids[:sum(need)], torch.int32)
            ints = torch.empty(2 * n + B + 2, dtype=i64, device=self.device)
            slots, pos, used, start = ints.split((n, n, 1, B + 1))
            out = torch.empty_like(x) if out is None else out
            self.block.page_plan(self.page, lens_d, news_d, free_d, table, start, slots, pos, used,
                                 stream=s)
            batch = self.block.paged_batch(
                start, lens_d, table, n, self.page, self.n_pages, max(news),
                max(have + more for have, more in zip(lens, news)), prefix_pages=prefix)
            self.block._paged_rows(batch, x, pos, slots, out)
            rc = blk_step_paged_stack(self.block.handle, self._w_arr, self.n_layers, batch,
                                      self._k_arr, self._v_arr, x.data_ptr(), pos.data_ptr(),
                                      slots.data_ptr(), out.data_ptr(), self.ws.data_ptr(),
                                      self.ws.numel(), s.cuda_stream)
        if rc != BLK_OK:
            raise BlkError(rc, "blk_step_paged_stack")
        return out, need

    def prefill_prefix(self, x, stream=None):
        """Computes the shared prefix from its rows x (fp16 [P, hidden], P a multiple of
        the page size) before any sequence has tokens; returns the last layer's rows."""
        if any(self.lens) or self.prefix is not None or x.shape[0] % self.page:
            raise BlkError(BLK_ERR_SHAPE, "PagedStack.prefill_prefix")
        s = self._follow(stream)
        with torch.cuda.stream(s):
            table = torch.full((1, self.max_blocks), -1, dtype=torch.int32, device=self.device)
            out, need = self._run(table, [0], [x.shape[0]], x, None, None, s)
            self.prefix = table[0, :need[0]].clone()
            self._held.append((self.prefix, [s]))
            self.table[:, :need[0]] = self.prefix
        self.prefix_ids = self.free_ids[:need[0]]
        del self.free_ids[:need[0]]
        self.lens = [x.shape[0]] * self.max_seqs
        return out

    def step(self, x, new_lens, out=None, stream=None):
        """new_lens: new tokens of sequences 0, 1, ... (a list, at most max_seqs of them,
        zeros allowed); x: fp16 [sum(new_lens), hidden], their rows back to back.
        Returns the last layer's rows."""
        B = len(new_lens)
        if not 0 < B <= self.max_seqs or sum(new_lens) < 1:
            raise BlkError(BLK_ERR_SHAPE, "PagedStack.step: new_lens")
        out, need = self._run(self.table[:B], self.lens[:B], list(new_lens), x, out, self.prefix,
                              stream)
        for b, k in enumerate(need):
            self.pages[b] += self.free_ids[:k]
            del self.free_ids[:k]
            self.lens[b] += new_lens[b]
        return out

    def free(self, b: int):
        """Gives sequence b's own pages back; it begins anew behind the prefix."""
        self.free_ids += self.pages[b]
        self.pages[b] = []
        self.lens[b] = len(self.prefix_ids) * self.page


class QuantDecodeStack:
    """Decode through a stack of blocks with weight-only quantized projections
    (blk_decode_stack_q), one library call per step."""

    def __init__(self, shape, qweights, max_ctx: int, caches=None, chain: bool = True,
                 device="cuda"):
        """qweights: list of BlkQWeights (one per layer; the tensors they
        point to must stay alive).  caches: optional list of (k_cache,
        v_cache) per layer, [Hkv, max_ctx, D]; zero-filled when None."""
        self.shape = shape
        self.n_layers = len(qweights)
        self.block = Block(shape, max_ctx, chain=chain)
        Hkv, D = shape.n_kv_heads, shape.head_dim
        if caches is None:
            caches = [(torch.zeros((Hkv, max_ctx, D), dtype=torch.float16, device=device),
                       torch.zeros((Hkv, max_ctx, D), dtype=torch.float16, device=device))
                      for _ in range(self.n_layers)]
        self.caches = caches
        self.ws = torch.empty(self.block.qworkspace_bytes(1), dtype=torch.uint8, device=device)
        self.out = torch.empty((1, shape.hidden), dtype=torch.float16, device=device)
        n = self.n_layers
        self._w_arr = (BlkQWeights * n)(*qweights)
        self._kc_arr = (ctypes.c_void_p * n)(*[kc.data_ptr() for kc, _ in caches])
        self._vc_arr = (ctypes.c_void_p * n)(*[vc.data_ptr() for _, vc in caches])

    def decode_step(self, x, pos, cache_len: int, out=None, stream=None):
        out = self.out if out is None else out
        s = torch.cuda.current_stream() if stream is None else stream
        rc = blk_decode_stack_q(self.block.handle, self._w_arr, self.n_layers, self._kc_arr,
                                self._vc_arr, x.data_ptr(), pos.data_ptr(), cache_len,
                                out.data_ptr(), None, None, self.ws.data_ptr(), self.ws.numel(),
                                s.cuda_stream)
        if rc != BLK_OK:
            raise BlkError(rc, "blk_decode_stack_q")
        return out

    def capture(self, x, pos, cache_len: int):
        """One decode step captured into a CUDA graph (x, pos stay alive)."""
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                out = self.decode_step(x, pos, cache_len, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        return g, out
