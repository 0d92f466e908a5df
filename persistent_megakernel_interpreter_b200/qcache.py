"""The 8-bit KV cache (``mk_qcache`` in mk.h): buffers, and the calls that work on them.

Keys and values are int8 codes with one fp32 scale per block of 32 tokens of one head; the
tokens of a row's open block stay bf16 until it is full. ``QCache(cfg, max_batch, max_seq)``
allocates the buffers, ``QCache.from_tensors`` takes a caller's. ``append`` stores new tokens
(a decoded one, a prompt, or a whole bf16 cache), ``attention`` attends to them with one query
token per row, ``reorder`` lets rows follow other rows (beams, forks, compaction), and
``Megakernel.decode_step_qcache`` runs a whole decode step on the cache.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .config import ModelConfig

BLOCK = _lib.QCACHE_BLOCK


class QCache:
    def __init__(self, cfg: ModelConfig, max_batch: int = 1, max_seq: int = 256, device: int | None = None):
        device = torch.cuda.current_device() if device is None else device
        shape = (cfg.n_layers, max_batch, cfg.n_kv_heads, max_seq, cfg.head_dim)
        blocks = (max_seq + BLOCK - 1) // BLOCK

        def zeros(*size, dtype):
            return torch.zeros(size, dtype=dtype, device=torch.device("cuda", device))

        self._adopt(zeros(*shape, dtype=torch.int8), zeros(*shape, dtype=torch.int8),
                    zeros(*shape[:3], blocks, dtype=torch.float32), zeros(*shape[:3], blocks, dtype=torch.float32),
                    zeros(*shape[:3], BLOCK, shape[4], dtype=torch.bfloat16),
                    zeros(*shape[:3], BLOCK, shape[4], dtype=torch.bfloat16))

    @classmethod
    def from_tensors(cls, k_codes, v_codes, k_scale, v_scale, k_tail, v_tail) -> "QCache":
        """A cache over the caller's buffers: codes int8 [layers][rows][heads][max_seq][dim], scales
        fp32 [layers][rows][heads][ceil(max_seq / 32)], tails bf16 [layers][rows][heads][32][dim]."""
        c = cls.__new__(cls)
        c._adopt(k_codes, v_codes, k_scale, v_scale, k_tail, v_tail)
        return c

    def _adopt(self, k_codes, v_codes, k_scale, v_scale, k_tail, v_tail) -> None:
        n_layers, max_batch, n_heads, max_seq, dim = k_codes.shape
        outer = (n_layers, max_batch, n_heads)
        for t, dt, tail in ((k_codes, torch.int8, (max_seq, dim)), (v_codes, torch.int8, (max_seq, dim)),
                            (k_scale, torch.float32, ((max_seq + BLOCK - 1) // BLOCK,)),
                            (v_scale, torch.float32, ((max_seq + BLOCK - 1) // BLOCK,)),
                            (k_tail, torch.bfloat16, (BLOCK, dim)), (v_tail, torch.bfloat16, (BLOCK, dim))):
            assert t.is_cuda and t.dtype == dt and t.is_contiguous() and tuple(t.shape) == outer + tail
            assert t.device == k_codes.device
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.k_tail, self.v_tail = k_tail, v_tail
        self.n_layers, self.max_batch, self.n_kv_heads, self.max_seq, self.head_dim = tuple(k_codes.shape)
        self.device, self._device = k_codes.device, k_codes.get_device()
        self._c = _lib.MkQcache(n_layers, max_batch, n_heads, max_seq, dim, 0, k_codes.data_ptr(),
                                v_codes.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), k_tail.data_ptr(),
                                v_tail.data_ptr())
        self._ref, self._address = ctypes.byref(self._c), ctypes.addressof(self._c)

    def append(self, k, v, positions, counts=None, first_layer: int = 0, stream=None) -> None:
        """Stores ``k`` and ``v`` (bf16 [layers][rows][heads][tokens][dim], any strides with the dims
        contiguous) from slot ``positions[row]`` on: ``counts[row]`` tokens of each row (all of them
        where ``counts`` is None), in layers ``first_layer`` on."""
        _lib.check(_lib.call().qcache_append(self._address, self._device, k, v, positions, counts, first_layer, stream),
                   "mk_qcache_append")

    def reorder(self, parents, lengths, starts=None, stream=None) -> None:
        """Row r takes over row parents[r]'s slots starts[r] .. lengths[parents[r]] - 1, all rows at once."""
        _lib.check(_lib.call().qcache_reorder(self._address, self._device, parents, lengths, starts, stream),
                   "mk_qcache_reorder")

    def attention_workspace(self, rows: int, n_heads: int, max_ctx: int):
        """A workspace for ``attention`` calls of this size, or None where they need none. Calls that
        may overlap on the GPU need one each."""
        n = _lib.call().qcache_attention_workspace(self._address, rows, n_heads, max_ctx)
        return torch.empty(n, dtype=torch.uint8, device=self.device) if n else None

    def attention(self, layer: int, q, positions, out, max_ctx: int | None = None, workspace=None, stream=None,
                  lengths=None) -> None:
        """out[row][head] = attention of q[row][head] (fp32 [rows][n_heads][dim]) over slots
        0 .. positions[row] of ``layer``; a negative position gives zeros. ``max_ctx``: at most the first
        max_ctx slots of a row are read (max_seq where None). ``lengths`` (int32 [rows]): the tokens that
        each row holds. Where it is None a position has to be the row's last token, another one of its
        open block, or the last of a closed block. Without a ``workspace`` one is allocated for the call."""
        max_ctx = self.max_seq if max_ctx is None else max_ctx
        if workspace is None:
            rows, n_heads = q.shape[:2]
            if stream is None:
                workspace = self.attention_workspace(rows, n_heads, max_ctx)
            else:
                with torch.cuda.stream(stream):  # its memory is given back in the order of that stream
                    workspace = self.attention_workspace(rows, n_heads, max_ctx)
        _lib.check(_lib.call().qcache_attention(self._address, self._device, layer, q, positions, out, max_ctx, workspace,
                                                stream, lengths), "mk_qcache_attention")
