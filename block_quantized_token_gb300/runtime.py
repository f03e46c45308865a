"""Thin Python owners of er_model / er_kv handles, with torch as the device allocator.

Weights arrive as host arrays in GGUF layout (uint8 block bytes, float32 gains,
float16 embedding) keyed by GGUF tensor name; they are staged on the device,
handed to er_model_create (which repacks them into model-owned memory) and
released.  All compute happens in liber.so.
"""

from __future__ import annotations

import ctypes
from typing import Callable, Mapping

import numpy as np
import torch

from . import er

_LAYER_FIELDS = (("attn_norm", "attn_norm"), ("wq", "attn_q"), ("wk", "attn_k"), ("wv", "attn_v"),
                 ("wo", "attn_output"), ("ffn_norm", "ffn_norm"), ("w_gate", "ffn_gate"), ("w_up", "ffn_up"),
                 ("w_down", "ffn_down"))


KV_TYPES = {"f16": er.DTYPES["f16"], "q8_0": er.DTYPES["q8_0"]}  # er_kv_create_typed storage codes


def make_config(shape, max_batch: int = 1) -> er.er_config:
    """er_config from any object with the ModelShape fields."""
    return er.er_config(dim=shape.dim, n_layers=shape.n_layers, n_heads=shape.n_heads, n_kv_heads=shape.n_kv_heads,
                        head_dim=shape.head_dim, ffn_dim=shape.ffn_dim, vocab=shape.vocab,
                        rope_base=float(shape.rope_base), rms_eps=float(shape.rms_eps),
                        w_type=er.DTYPES[shape.w_type], tied=1 if shape.tied else 0, max_batch=max_batch)


def _to_device(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class DecodeModel:
    """Owns an er_model built from host tensors (name -> array or a callable name -> array)."""

    def __init__(self, shape, tensors: Mapping[str, np.ndarray] | Callable[[str], np.ndarray],
                 max_batch: int = 1, device: str = "cuda"):
        get = tensors if callable(tensors) else tensors.__getitem__
        self.shape = shape
        self.device = torch.device(device)
        keep = []

        def dev(name):
            t = _to_device(get(name), self.device)
            keep.append(t)
            return t.data_ptr()

        layers = (er.er_layer_weights * shape.n_layers)()
        for l in range(shape.n_layers):
            for field, leaf in _LAYER_FIELDS:
                setattr(layers[l], field, dev(f"blk.{l}.{leaf}.weight"))
        w = er.er_weights(tok_embd=dev("token_embd.weight"), output_norm=dev("output_norm.weight"),
                          output=None if shape.tied else dev("output.weight"),
                          layers=ctypes.cast(layers, ctypes.POINTER(er.er_layer_weights)))
        self.cfg = make_config(shape, max_batch)
        stream = torch.cuda.current_stream(self.device).cuda_stream
        self.handle = er.er_model_create(self.cfg, w, stream)
        del keep

    @property
    def device_bytes(self) -> int:
        return er.er_model_device_bytes(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            er.er_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


class DecodeState:
    """Owns an er_kv (KV cache + scratch of `batch` sequences) of a DecodeModel."""

    def __init__(self, model: DecodeModel, batch: int, capacity: int, kv_type: str = "f16"):
        """kv_type "f16" (fp16 rows) or "q8_0" (packed Q8_0 blocks, quantised as rows are written)."""
        self.model, self.batch, self.capacity = model, batch, capacity
        if kv_type not in KV_TYPES:
            raise ValueError(f"kv_type must be one of {sorted(KV_TYPES)}")
        self.kv_type = kv_type
        self.handle = er.er_kv_create_typed(model.handle, batch, capacity, KV_TYPES[kv_type])

    def write_rows(self, seq: int, layer: int, k_rows: np.ndarray | torch.Tensor, v_rows, start: int = 0,
                   stream: int | None = None) -> None:
        """Copy token-major fp16 rows [n, n_kv_heads*head_dim] into cache rows start..start+n-1."""
        dev = self.model.device
        k = k_rows if isinstance(k_rows, torch.Tensor) else _to_device(np.asarray(k_rows, np.float16), dev)
        v = v_rows if isinstance(v_rows, torch.Tensor) else _to_device(np.asarray(v_rows, np.float16), dev)
        k, v = k.contiguous(), v.contiguous()
        st = torch.cuda.current_stream(dev).cuda_stream if stream is None else stream
        er.er_kv_write(self.handle, seq, layer, start, k.shape[0], k.data_ptr(), v.data_ptr(), st)
        torch.cuda.current_stream(dev).synchronize()

    def read_rows(self, seq: int, layer: int, start: int, n: int) -> tuple[torch.Tensor, torch.Tensor]:
        s = self.model.shape
        k = torch.empty((n, s.n_kv_heads * s.head_dim), dtype=torch.float16, device=self.model.device)
        v = torch.empty_like(k)
        st = torch.cuda.current_stream(self.model.device).cuda_stream
        er.er_kv_read(self.handle, seq, layer, start, n, k.data_ptr(), v.data_ptr(), st)
        torch.cuda.current_stream(self.model.device).synchronize()
        return k, v

    def read_blocks(self, seq: int, layer: int, start: int, n: int) -> tuple[np.ndarray, np.ndarray]:
        """Q8_0 cache rows start..start+n-1 as GGUF blocks: (d fp16, q int8) per side, shaped
        [n, n_kv_heads*head_dim/32] and [n, n_kv_heads*head_dim]."""
        s = self.model.shape
        nb = s.n_kv_heads * s.head_dim // 32
        k = torch.empty((n, nb, 34), dtype=torch.uint8, device=self.model.device)
        v = torch.empty_like(k)
        st = torch.cuda.current_stream(self.model.device).cuda_stream
        er.er_kv_read_blocks(self.handle, seq, layer, start, n, k.data_ptr(), v.data_ptr(), st)
        torch.cuda.current_stream(self.model.device).synchronize()
        out = []
        for t in (k, v):
            a = t.cpu().numpy()
            d = np.ascontiguousarray(a[:, :, :2]).view(np.float16).reshape(n, nb)
            q = np.ascontiguousarray(a[:, :, 2:]).view(np.int8).reshape(n, nb * 32)
            out += [d, q]
        return tuple(out)

    def prefill(self, seq: int, tokens: torch.Tensor, start: int, logits: torch.Tensor | None = None,
                stream: int | None = None) -> None:
        """Run the decoder over device int32 `tokens` of sequence `seq` at positions start.., writing the cache."""
        st = torch.cuda.current_stream(self.model.device).cuda_stream if stream is None else stream
        er.er_prefill(self.handle, seq, tokens.data_ptr() if tokens.numel() else None, int(tokens.numel()), start,
                      None if logits is None else logits.data_ptr(), st)

    def step(self, tokens: torch.Tensor, positions: torch.Tensor, logits: torch.Tensor | None,
             argmax: torch.Tensor | None, graph: bool = True, stream: int | None = None) -> None:
        st = torch.cuda.current_stream(self.model.device).cuda_stream if stream is None else stream
        fn = er.er_decode_step if graph else er.er_decode_step_eager
        fn(tokens.data_ptr(), positions.data_ptr(), self.handle, None if logits is None else logits.data_ptr(),
           None if argmax is None else argmax.data_ptr(), st)

    def set_schedule(self, schedule: int) -> None:
        er.er_kv_set_schedule(self.handle, schedule)

    def set_wide_gemv(self, variant: int) -> None:
        er.er_kv_set_wide_gemv(self.handle, variant)

    @property
    def schedule(self) -> int:
        return er.er_kv_get_schedule(self.handle)

    def device_error(self) -> tuple[int, int, int]:
        return er.er_get_device_error(self.handle)

    def close(self) -> None:
        if getattr(self, "handle", None):
            er.er_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()


_ROW_TYPES = {torch.float32: er.ER_F32, torch.float16: er.ER_F16, torch.bfloat16: er.ER_BF16}
_ROPE_STYLES = {"pairs": er.ER_ROPE_PAIRS, "halves": er.ER_ROPE_HALVES}


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def rope_table(head_dim: int, base: float, n_positions: int, device: str = "cuda") -> torch.Tensor:
    """(cos, sin) of p * base^(-2 i / head_dim), fp32 [n_positions, head_dim / 2, 2], made on the device."""
    out = torch.empty((n_positions, head_dim // 2, 2), dtype=torch.float32, device=device)
    with torch.cuda.device(out.device):  # (a default stream's handle is the same on every device)
        er.er_rope_table(head_dim, base, n_positions, out.data_ptr(), torch.cuda.current_stream(out.device).cuda_stream)
    return out


class PagedCache:
    """Owns an er_pages handle and, unless given, its pool: a paged 4-bit K/V cache (er_pages_* in er_pages.h).

    Row tensors are [tokens, heads, head_dim] with dense heads and any stride between tokens; int tensors are dense
    int32; all on the cache's device, which need not be the current one.
    """

    def __init__(self, n_layers: int, n_pages: int, page_rows: int, n_kv_heads: int, head_dim: int,
                 pool: torch.Tensor | None = None, device: str = "cuda"):
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        self.cfg = er.er_pages_config(n_layers, n_pages, page_rows, n_kv_heads, head_dim, er.ER_Q4_0)
        need = er.er_pages_pool_bytes(self.cfg)
        if not need:
            er.er_pages_create(self.cfg, None)  # raises with the reason
        if pool is None:
            pool = torch.empty(need, dtype=torch.uint8, device=device)
        if not pool.is_cuda or not pool.is_contiguous() or pool.numel() * pool.element_size() != need:
            raise ValueError(f"pool must be a dense CUDA tensor of {need} bytes")
        self.pool, self.device, self._index = pool, pool.device, pool.get_device()
        with torch.cuda.device(self.device):
            self.handle = er.er_pages_create(self.cfg, pool.data_ptr())

    # The checks below stand before calls that take the GPU 6 us, so they ask each tensor as little as they can (a
    # device's index and a raw stream cost a tenth of the device and stream objects).
    def _there(self, fn: Callable, *args):
        """A refused fn(handle, ...) once more with the cache's device current, if it was not: the library asks for that before
        it does anything, so calls need not ask first (0.45 us each)."""
        if torch._C._cuda_getDevice() == self._index:
            raise  # the refusal being handled
        with torch.cuda.device(self._index):
            return fn(self.handle, *args)

    def _stream(self, stream: int | None) -> int:
        return torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream

    def _ints(self, n: int, *tensors: torch.Tensor) -> None:
        for t in tensors:
            if t.dtype is not torch.int32 or t.get_device() != self._index or t.numel() < n or not t.is_contiguous():
                raise ValueError(f"a dense int32 tensor of {n} values on {self.device} is needed")

    def _rows(self, x: torch.Tensor, n: int, heads: int | None, dtype: torch.dtype | None) -> int:
        """Checks row tensors [n, heads, head_dim]; returns the stride between tokens."""
        shape = x.shape
        if len(shape) != 3 or shape[2] != self.head_dim or (heads is not None and shape[1] != heads):
            raise ValueError(f"rows must be [tokens, heads, {self.head_dim}]")
        s0, s1, s2 = x.stride()
        if shape[0] < n or x.get_device() != self._index or (dtype is not None and x.dtype is not dtype) or s2 != 1 or \
                (s1 != self.head_dim and shape[1] > 1):
            raise ValueError(f"rows must be {n} dense heads' rows of one type on {self.device}")
        if dtype is None and x.dtype not in _ROW_TYPES:
            raise ValueError("rows must be float32, float16 or bfloat16")
        return s0 if shape[0] > 1 else shape[1] * self.head_dim

    def _table(self, tables: torch.Tensor, n_seqs: int) -> int:
        self._ints(0, tables)
        if tables.dim() != 2 or tables.shape[0] < n_seqs:
            raise ValueError("tables must be [sequences, pages]")
        return tables.shape[1]

    def plan(self, lens: torch.Tensor, new: torch.Tensor, tables: torch.Tensor, free: torch.Tensor,
             free_count: torch.Tensor, lens_out: torch.Tensor, free_count_out: torch.Tensor, q_start: torch.Tensor,
             positions: torch.Tensor, slots: torch.Tensor, seqs: torch.Tensor, stream: int | None = None) -> None:
        """Pages, positions and slots of a step in which request b brings new[b] tokens (er_pages_plan)."""
        n, rows = lens.numel(), slots.numel()
        self._ints(n, lens, new, lens_out)
        self._ints(rows, positions, slots, seqs)
        self._ints(n + 1, q_start)
        self._ints(1, free_count, free_count_out)
        self._ints(self.cfg.n_pages, free)
        a = er.er_pages_plan_args(n, rows, self._table(tables, n), lens.data_ptr(), new.data_ptr(), free.data_ptr(),
                                  free_count.data_ptr(), tables.data_ptr(), lens_out.data_ptr(),
                                  free_count_out.data_ptr(), q_start.data_ptr(), positions.data_ptr(), slots.data_ptr(),
                                  seqs.data_ptr())
        st = self._stream(stream)
        try:
            er.er_pages_plan(self.handle, a, st)
        except er.ErError:
            self._there(er.er_pages_plan, a, st)

    def release(self, done: torch.Tensor, lens: torch.Tensor, tables: torch.Tensor, free: torch.Tensor,
                free_count: torch.Tensor, stream: int | None = None) -> None:
        """Gives the pages of the requests with done[b] != 0 back to the free list (er_pages_release)."""
        n = lens.numel()
        self._ints(n, done, lens)
        self._ints(1, free_count)
        self._ints(self.cfg.n_pages, free)
        a = (n, done.data_ptr(), lens.data_ptr(), tables.data_ptr(), self._table(tables, n), free.data_ptr(),
             free_count.data_ptr(), self._stream(stream))
        try:
            er.er_pages_release(self.handle, *a)
        except er.ErError:
            self._there(er.er_pages_release, *a)

    def append(self, layer: int, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
               positions: torch.Tensor | None, slots: torch.Tensor, q_out: torch.Tensor | None = None,
               q_gain: torch.Tensor | None = None, k_gain: torch.Tensor | None = None, eps: float = 1e-5,
               rope: torch.Tensor | None = None, rope_style: str = "pairs", stream: int | None = None) -> None:
        """Norms and rotates q and k, writes q_out and puts k and v into their slots (er_pages_append)."""
        n, hd = k.shape[0], self.head_dim
        ks, vs = self._rows(k, n, self.n_kv_heads, None), self._rows(v, n, self.n_kv_heads, k.dtype)
        if (q is None) != (q_out is None):
            raise ValueError("q and q_out go together")
        qs = os_ = heads = 0
        if q is not None:
            heads = q.shape[1]
            qs, os_ = self._rows(q, n, heads, k.dtype), self._rows(q_out, n, heads, k.dtype)
        self._ints(n, slots)
        for g in (q_gain, k_gain):
            if g is not None and (g.dtype is not torch.float32 or g.numel() != hd or not g.is_contiguous() or
                                  g.get_device() != self._index):
                raise ValueError(f"a gain must be {hd} float32 values")
        if rope is not None:
            if rope.dtype is not torch.float32 or not rope.is_contiguous() or rope.get_device() != self._index or \
                    rope.dim() != 3 or rope.shape[1] != hd // 2 or rope.shape[2] != 2:
                raise ValueError(f"the rope table must be float32 [positions, {hd // 2}, 2]")
            if positions is None:
                raise ValueError("a rope table needs positions")
            self._ints(n, positions)
        if rope_style not in _ROPE_STYLES:
            raise ValueError(f"rope_style must be one of {sorted(_ROPE_STYLES)}")
        a = er.er_pages_append_args(n, heads, _ROW_TYPES[k.dtype], _ROPE_STYLES[rope_style],
                                    0 if rope is None else rope.shape[0], _ptr(q), k.data_ptr(), v.data_ptr(), _ptr(q_out),
                                    qs, ks, vs, os_, _ptr(q_gain), _ptr(k_gain), _ptr(rope),
                                    None if rope is None else positions.data_ptr(), slots.data_ptr(), eps)
        st = self._stream(stream)
        try:
            er.er_pages_append(self.handle, layer, a, st)
        except er.ErError:
            self._there(er.er_pages_append, layer, a, st)

    def read(self, layer: int, slots: torch.Tensor, k_out: torch.Tensor | None, v_out: torch.Tensor | None,
             stream: int | None = None) -> None:
        """Values of the rows at `slots` into dense k_out / v_out [n, n_kv_heads, head_dim] (er_pages_read)."""
        n = slots.numel()
        self._ints(n, slots)
        dtype = None
        for t in (k_out, v_out):
            if t is not None:
                if not t.is_contiguous():
                    raise ValueError("k_out and v_out must be dense")
                self._rows(t, n, self.n_kv_heads, dtype)
                dtype = t.dtype
        if dtype is None:
            return
        a = (layer, n, slots.data_ptr(), _ROW_TYPES[dtype], _ptr(k_out), _ptr(v_out), self._stream(stream))
        try:
            er.er_pages_read(self.handle, *a)
        except er.ErError:
            self._there(er.er_pages_read, *a)

    def attention(self, layer: int, q: torch.Tensor, out: torch.Tensor, q_start: torch.Tensor, lens: torch.Tensor,
                  tables: torch.Tensor, scale: float = 0.0, window: int = 0, lse: torch.Tensor | None = None,
                  stream: int | None = None) -> None:
        """Attention of rows q_start[b] .. q_start[b + 1] - 1 of q over sequence b's lens[b] cached rows
        (er_pages_attention)."""
        n, heads, seqs = q.shape[0], q.shape[1], lens.numel()
        qs, os_ = self._rows(q, n, heads, None), self._rows(out, n, heads, q.dtype)
        self._ints(seqs, lens)
        self._ints(seqs + 1, q_start)
        if lse is not None and (lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != self._index or
                                lse.numel() < n * heads):
            raise ValueError("lse must be dense float32 [tokens, heads]")
        a = er.er_pages_attention_args(seqs, n, heads, _ROW_TYPES[q.dtype], self._table(tables, seqs), window,
                                       q.data_ptr(), out.data_ptr(), _ptr(lse), qs, os_,
                                       q_start.data_ptr(), lens.data_ptr(), tables.data_ptr(), scale)
        st = self._stream(stream)
        try:
            er.er_pages_attention(self.handle, layer, a, st)
        except er.ErError:
            self._there(er.er_pages_attention, layer, a, st)

    def error(self) -> tuple[int, int]:
        """(status, flags) of the calls so far; synchronises (er_pages_error)."""
        try:
            return er.er_pages_error(self.handle)
        except er.ErError:
            return self._there(er.er_pages_error)

    def close(self) -> None:
        if getattr(self, "handle", None):
            er.er_pages_destroy(self.handle)
            self.handle = None

    def __del__(self):
        self.close()
