"""Mixture-of-experts operators on compressed weights: the routing of tokens to experts and
the weighted sum of the experts' rows back to the tokens."""

from __future__ import annotations

from typing import TYPE_CHECKING, NamedTuple

from . import _binding as B
from .layer import _raw_stream, check_tensor

if TYPE_CHECKING:
    import torch


def _cuda_device(device) -> torch.device:
    import torch

    device = torch.device(device)
    return torch.device("cuda", torch.cuda.current_device()) if device.type == "cuda" and device.index is None else device


class VQRouting(NamedTuple):
    """What ``VQRouter.forward`` returns for T tokens (int32, weights float32).

    ``ids`` and ``weights`` [T, k]: a token's experts, best first, and their weights;
    ``offsets`` [E + 1]: the rows of expert e are offsets[e] .. offsets[e + 1] - 1 of the
    expert-ordered rows; ``rows`` [T * k]: the token of each such row; ``slots`` [T, k]: the
    row of each (token, choice).  Masked places have id -1, weight 0 and slot -1."""

    ids: torch.Tensor
    weights: torch.Tensor
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


class VQRouter:
    """Top-k routing of up to `max_tokens` tokens over E experts (vq_router_forward).

    `renorm`: the k weights of a token add up to 1; otherwise they are softmax
    probabilities over all E experts."""

    def __init__(self, E, k, max_tokens, renorm=False, device="cuda"):
        import torch

        self.E, self.k, self.max_tokens, self.renorm = E, k, max_tokens, bool(renorm)
        self.handle = None
        self.device = _cuda_device(device)
        with torch.cuda.device(self.device):
            self.handle = B.vq_router_create(E, k, max_tokens, renorm)

    def forward(self, logits, out: VQRouting | None = None, stream=None) -> VQRouting:
        """logits [T, E], float16, bfloat16 or float32, contiguous; -inf and NaN mask an expert.
        `out`: the tensors of an earlier result of the same T, written again."""
        import torch

        T, E, k, dev = logits.shape[0], self.E, self.k, self.device
        dtype = {torch.float16: B.VQ_F16, torch.bfloat16: B.VQ_BF16, torch.float32: B.VQ_F32}.get(logits.dtype)
        if dtype is None:
            raise ValueError(f"logits must be float16, bfloat16 or float32: got {logits.dtype}")
        check_tensor(logits, "logits", (T, E), logits.dtype, dev)
        if out is None:
            i32 = torch.int32
            out = VQRouting(torch.empty((T, k), dtype=i32, device=dev), torch.empty((T, k), device=dev, dtype=torch.float32),
                            torch.empty(E + 1, dtype=i32, device=dev), torch.empty(T * k, dtype=i32, device=dev),
                            torch.empty((T, k), dtype=i32, device=dev))
        else:
            for name, shape, dt in (("ids", (T, k), torch.int32), ("weights", (T, k), torch.float32),
                                    ("offsets", (E + 1,), torch.int32), ("rows", (T * k,), torch.int32),
                                    ("slots", (T, k), torch.int32)):
                check_tensor(getattr(out, name), name, shape, dt, dev)
        B.vq_router_forward(self.handle, logits, dtype, *out, T, _raw_stream(stream, dev.index))
        return out

    __call__ = forward

    def close(self):
        if getattr(self, "handle", None):
            B.vq_router_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def combine(y, weights, slots, residual=None, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] + residual[t] (vq_experts_combine).

    y [rows, N] (float16 or bfloat16, N a multiple of 8), weights float32 and slots int32
    [T, k] as a ``VQRouting`` has them; a slot outside y's rows adds nothing.  `residual`
    [T, N] may be `out`.  The current device must be the tensors'."""
    import torch

    if y.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError(f"y must be float16 or bfloat16: got {y.dtype}")
    dev, (n, N), (T, k) = y.device, y.shape, slots.shape
    if dev.type != "cuda" or dev.index != torch.cuda.current_device():
        raise ValueError(f"y must be on the current CUDA device: got {dev}")
    check_tensor(y, "y", (n, N), y.dtype, dev)
    check_tensor(slots, "slots", (T, k), torch.int32, dev)
    check_tensor(weights, "weights", (T, k), torch.float32, dev)
    if residual is not None:
        check_tensor(residual, "residual", (T, N), y.dtype, dev)
    if out is None:
        out = torch.empty((T, N), dtype=y.dtype, device=dev)
    else:
        check_tensor(out, "out", (T, N), y.dtype, dev)
    B.vq_experts_combine(y, n, weights, slots, residual, out, T, k, N,
                         B.VQ_BF16 if y.dtype == torch.bfloat16 else B.VQ_F16, _raw_stream(stream, dev.index))
    return out
