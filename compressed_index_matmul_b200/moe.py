"""Mixture-of-experts operators on compressed weights: the products grouped by expert, the
routing of tokens to experts and the weighted sum of the experts' rows back to the tokens."""

from __future__ import annotations

from typing import TYPE_CHECKING, NamedTuple

from . import _binding as B
from .layer import _new, _raw_stream, check_tensor

if TYPE_CHECKING:
    import torch


def _cuda_device(device) -> torch.device:
    import torch

    device = torch.device(device)
    return torch.device("cuda", torch.cuda.current_device()) if device.type == "cuda" and device.index is None else device


def _on_device(a, device):
    """A plane, codebook or scale array on the device, its bits as they are."""
    import numpy as np
    import torch

    if isinstance(a, np.ndarray):
        a = np.ascontiguousarray(a)
        a = torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a)
    return a.to(device).contiguous()


class VQExperts:
    """E compressed weight matrices of one shape, multiplied group by group (vq_experts_forward).

    ``arrays``: numpy arrays or torch tensors named as in ``VQLinear`` (lo, hi4, s2, idx16, idx8,
    cb1, cb2, cbr, cb8, scales, mult), each with a leading dimension E in include/vqlinear.h's
    storage format; the codebooks' is 1 (or left out) with `shared_codebooks`.  Index planes are
    8-bit or 16-bit integers, codebooks and scales float16 or its bits in 16-bit integers.  For the
    residual ladder cbr is [n16 - 1, E or 1, 65536, 8] and idx16 [E, n16 * N * K / 8].
    `glu`: rows [0, N/2) of every matrix are a gate, the others its up projection, and the output
    has N/2 columns, act(gate) * up.  `act` is a VQ_ACT_*, `bias` [E, N] or None.
    A call takes at most `max_rows` rows, all experts together.  `gather`: calls may pass `rows`,
    for which the handle keeps a buffer of max_rows x K elements."""

    def __init__(self, E, N, K, fmt, scale_group, act_dtype, max_rows, arrays: dict, act=B.VQ_ACT_NONE, glu=False,
                 bias=None, shared_codebooks=False, gather=True, device="cuda"):
        import numpy as np
        import torch

        self.handle = None
        self.E, self.N, self.K, self.fmt, self.scale_group, self.act_dtype = E, N, K, fmt, scale_group, act_dtype
        self.max_rows, self.act, self.glu, self.shared = max_rows, act, bool(glu), bool(shared_codebooks)
        self.n_out = N // 2 if glu else N
        self.device = dev = _cuda_device(device)
        names = ("lo", "hi4", "s2", "idx16", "idx8", "cb1", "cb2", "cbr", "cb8", "scales")
        t = self.t = {k: _on_device(arrays[k], dev) for k in names if arrays.get(k) is not None}
        n, sets = N * (K // 8), 1 if shared_codebooks else E
        ladder, k16 = fmt == B.VQ_FMT_VQ16_RVQ, fmt in (B.VQ_FMT_VQ16, B.VQ_FMT_VQ16_RVQ)
        self.n16 = t["idx16"].numel() // (E * n) if ladder and "idx16" in t else 0
        self.n8 = int(ladder and "idx8" in t)
        self.mult = tuple(float(m) for m in np.asarray(arrays["mult"], dtype=np.float32)) if ladder else ()
        byte, index16 = (torch.uint8, torch.int8), (torch.int16, torch.uint16)
        half = (torch.float16, *index16)  # or its bits
        want = {"scales": (E * N * (1 if scale_group == K else K // 64), half),
                "cb1": (sets * (65536 if k16 else 4096) * 8, half)}
        if k16:
            want["idx16"] = (E * n * max(1, self.n16), index16)
        else:
            want |= {"lo": (E * n, byte), "hi4": (E * n // 2, byte)}
        if fmt == B.VQ_FMT_RVQ12_4:
            want |= {"s2": (E * n // 2, byte), "cb2": (sets * 16 * 8, half)}
        if ladder and self.n16 > 1:
            want["cbr"] = ((self.n16 - 1) * sets * 65536 * 8, half)
        if self.n8:
            want |= {"idx8": (E * n, byte), "cb8": (sets * 256 * 8, half)}
        for name, (count, types) in want.items():
            if name not in t or t[name].numel() != count or t[name].dtype not in types:
                got = f"{t[name].numel()} of {t[name].dtype}" if name in t else "none"
                raise ValueError(f"{name} must have {count} entries of one of {list(types)} for E={E}, N={N}, K={K}: got {got}")
        if ladder and len(self.mult) != self.n16 + self.n8 - 1:
            raise ValueError(f"mult must have {self.n16 + self.n8 - 1} entries, one per residual stage: got {len(self.mult)}")
        self.bias = None
        if bias is not None:
            self.bias = bias.to(dev)
            check_tensor(self.bias, "bias", (E, N), self.torch_dtype, dev)
        cbr = tuple(t["cbr"].data_ptr() + i * sets * 65536 * 16 for i in range(self.n16 - 1)) if "cbr" in want else ()
        self.planes = B.make_planes(t.get("lo"), t.get("hi4"), t.get("s2"), t.get("idx16"), t.get("idx8"))
        self.codebooks = B.make_codebooks(t["cb1"], t.get("cb2"), cbr, t.get("cb8"))
        with torch.cuda.device(dev):
            self.handle = B.vq_experts_create(E, N, K, fmt, scale_group, act_dtype, max_rows, act, glu, shared_codebooks,
                                              self.n16, self.n8, self.mult, gather)

    @property
    def torch_dtype(self):
        import torch

        return torch.bfloat16 if self.act_dtype == B.VQ_BF16 else torch.float16

    def forward(self, x, offsets, rows=None, y=None, stream=None):
        """y[r] = act(x[rows[r]] . W_e^T + bias[e]) for offsets[e] <= r < offsets[e + 1].

        x [x_rows, K]; offsets int32 [E + 1] and rows int32 [T] on the device, as ``VQRouter``
        gives them; without `rows` row r reads x[r].  A `rows` value outside x reads as zeros.
        Returns y [T, N] (glu: [T, N/2]); rows of y outside offsets[0] .. offsets[E] are not
        written."""
        import torch

        dt, dev = self.torch_dtype, self.device
        n = x.shape[0]
        check_tensor(x, "x", (n, self.K), dt, dev)
        check_tensor(offsets, "offsets", (self.E + 1,), torch.int32, dev)
        T = n
        if rows is not None:
            T = rows.shape[0]
            check_tensor(rows, "rows", (T,), torch.int32, dev)
        if y is None:
            y = _new((T, self.n_out), dt, dev, stream)
        else:
            check_tensor(y, "y", (T, self.n_out), dt, dev)
        if T > 0:
            B.vq_experts_forward(self.handle, x, n, rows, offsets, self.planes, self.codebooks, self.t["scales"], self.bias,
                                 y, T, _raw_stream(stream, dev.index))
        return y

    __call__ = forward

    def set_path(self, path: int):
        """VQ_PATH_GEMV, VQ_PATH_TC or VQ_PATH_AUTO (vq_experts_set_path)."""
        B.vq_experts_set_path(self.handle, path)

    def plan(self, T: int) -> dict:
        return B.vq_experts_plan(self.handle, T)

    def close(self):
        if getattr(self, "handle", None):
            B.vq_experts_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


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
            out = VQRouting(_new((T, k), i32, dev, stream), _new((T, k), torch.float32, dev, stream),
                            _new(E + 1, i32, dev, stream), _new(T * k, i32, dev, stream), _new((T, k), i32, dev, stream))
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
        out = _new((T, N), y.dtype, dev, stream)
    else:
        check_tensor(out, "out", (T, N), y.dtype, dev)
    B.vq_experts_combine(y, n, weights, slots, residual, out, T, k, N,
                         B.VQ_BF16 if y.dtype == torch.bfloat16 else B.VQ_F16, _raw_stream(stream, dev.index))
    return out
