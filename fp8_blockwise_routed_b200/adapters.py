"""Low-rank adapters of many requests beside a projection they share.

A batch groups its tokens by adapter once (LoraBatch); every projection of
the model that carries adapters (LoraAdapters) then uses the same grouping.
RoutedMoE and RoutedMoEMX take both in ``forward`` and add the adapters'
rows to the layer's; next to another projection (the shared expert's, say)
``LoraAdapters.forward`` adds to that projection's FP32 rows in place.

Every step runs in libfp8moe's kernels (moe_permute, moe_lora,
moe_lora_backward).
"""
from __future__ import annotations

import torch

from . import (_capturing, _device_of, _empty, _refuse, moe_lora, moe_lora_backward,
               moe_lora_backward_workspace_bytes, moe_permute, moe_route_workspace_bytes)


class LoraBatch:
    """The tokens of a batch grouped by adapter: ``assign`` takes one adapter
    id per token (int32, -1: none) for up to ``max_tokens`` tokens."""

    def __init__(self, n_adapters: int, max_tokens: int, device="cuda"):
        self.n, self.max_tokens, self.T = int(n_adapters), int(max_tokens), 0
        i32 = torch.int32
        self.offsets = torch.zeros((self.n + 1,), dtype=i32, device=device)
        self._sorted = torch.empty((max(self.max_tokens, 1),), dtype=i32, device=device)
        self.ws = torch.empty((moe_route_workspace_bytes(self.max_tokens, self.n, 1),), dtype=torch.uint8,
                              device=device)

    @property
    def sorted(self) -> torch.Tensor:
        return self._sorted[: self.T]

    def assign(self, adapter_ids: torch.Tensor, stream=None) -> "LoraBatch":
        T = adapter_ids.shape[0]
        assert T <= self.max_tokens and adapter_ids.shape == (T,) and adapter_ids.dtype == torch.int32
        assert adapter_ids.is_contiguous() and adapter_ids.device == self.offsets.device
        self.T = T
        with _device_of(adapter_ids):
            moe_permute(adapter_ids.view(T, 1), self.n, self.offsets, self._sorted, self.ws, stream)
        return self


class LoraAdapters:
    """Resident adapters of one projection: lora_a [n, rank, K] and lora_b
    [n, rank, N] BF16 (rank-major: lora_b is the transpose of an output
    projection's [N, rank]), scales [n] FP32 or None, and the buffer of the
    shrunk rows for up to ``max_tokens`` tokens.  A backward call uses the
    rows of the forward call before it (zeros if there was none), and is
    refused for a batch of another size than that call's; once forward is
    captured into a graph, whose replays are not seen here, that is the
    caller's to keep."""

    def __init__(self, lora_a, lora_b, scales, max_tokens: int):
        self.a, self.b, self.scales = lora_a, lora_b, scales
        self.n, self.rank, self.K = lora_a.shape
        self.N = lora_b.shape[2]
        self.max_tokens = int(max_tokens)
        self.v = torch.zeros((self.max_tokens, self.rank), dtype=torch.float32, device=lora_a.device)
        self._grad = self._ws = None
        self._last = None       # tokens of the last forward call
        self._captured = False

    def forward(self, batch: LoraBatch, x, base, out, out_bf16=None, stream=None):
        """out = base + the adapters' rows, for the tokens that have one;
        base may be out (added in place) or None (0)."""
        T = x.shape[0]
        assert T == batch.T and T <= self.max_tokens and batch.n == self.n
        moe_lora(x, self.a, self.b, self.scales, batch.offsets, batch.sorted, base, self.v[:T], out, out_bf16, stream)
        self._last = T
        if _capturing(x):
            self._captured = True
        return out

    def backward(self, batch: LoraBatch, x, dout, dx_base=None, dx=None, stream=None, d_a=None, d_b=None):
        """(d_a, d_b) FP32 for dout [T, N] BF16; dx, if given, receives
        dx_base plus the adapters' part for the tokens that have one.  d_a,
        d_b: where to write the gradients; without them they go to buffers of
        this object, which the next call overwrites (add them up before it)."""
        T = x.shape[0]
        assert T == batch.T and T <= self.max_tokens and batch.n == self.n
        if self._last not in (None, T) and not self._captured:
            _refuse("LoraAdapters.backward", f"the last forward call was of {self._last} tokens, not {T}")
        dev = self.a.device
        if self._ws is None:
            self._ws = _empty((moe_lora_backward_workspace_bytes(self.max_tokens, self.rank),), torch.uint8, dev,
                              stream)
        if (d_a is None or d_b is None) and self._grad is None:
            self._grad = (_empty(self.a.shape, torch.float32, dev, stream),
                          _empty(self.b.shape, torch.float32, dev, stream))
        d_a = self._grad[0] if d_a is None else d_a
        d_b = self._grad[1] if d_b is None else d_b
        moe_lora_backward(x, self.a, self.b, self.scales, batch.offsets, batch.sorted, self.v[:T], dout, dx_base, dx,
                          d_a, d_b, self._ws, stream)
        return d_a, d_b
