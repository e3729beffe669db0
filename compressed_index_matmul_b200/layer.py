"""VQLinear: one compressed layer resident on the GPU plus its library handle."""

from __future__ import annotations

import numpy as np

from . import _binding as B


def _dev(a: np.ndarray, device):
    import torch

    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)  # same bits; int16 is torch's portable 16-bit container
    return torch.from_numpy(a).to(device)


def _raw_stream(stream, index):
    """The raw handle of `stream`, or of the current stream of device `index`."""
    if stream is None:
        import torch

        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _new(shape, dtype, device, stream=None):
    """An uninitialised tensor for work on `stream` (None: the device's current stream), taken from
    that stream's memory: a block freed on another one may still be in use there."""
    import torch

    raw = None if stream is None else _raw_stream(stream, device.index)
    if raw is None or raw == _raw_stream(None, device.index):
        return torch.empty(shape, dtype=dtype, device=device)
    # ExternalStream takes 0, the default stream's handle, for none given and gives a pool stream's memory
    of = torch.cuda.default_stream(device) if raw == 0 else torch.cuda.ExternalStream(raw, device=device)
    with torch.cuda.stream(of):
        return torch.empty(shape, dtype=dtype, device=device)


def check_tensor(t, name, shape, dtype, device):
    """Raise ValueError unless `t` is a contiguous tensor of this shape, type and device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}: got "
                         f"{t.dtype} {list(t.shape)} on {t.device}, strides {list(t.stride())}")


class VQLinear:
    """Holds the planes, codebooks and scales of one layer in device memory.

    ``arrays`` is a dict with numpy arrays named as in include/vqlinear.h
    (lo, hi4, s2, idx16, idx8, cb1, cb2, cbr, cb8, scales; fp16 as uint16 bits) and the
    layer shape (N, K, fmt, scale_group).  For the residual ladder (VQ_FMT_VQ16_RVQ)
    idx16 holds one plane per 16-bit stage, cbr is [n16 - 1, 65536, 8] and ``mult``
    the float32 multipliers of the residual stages; the stage counts follow from the
    arrays.  An optional ``corr`` dict (row_ptr int32 [N+1], col int32, val fp16 bits)
    is the sparse correction sidecar; the handle is then created with corr = 1 and
    every forward passes it.  ``forward(x)`` calls vq_linear_forward.
    """

    def __init__(self, N, K, fmt, scale_group, act_dtype, max_M, arrays: dict, device="cuda", rht=0):
        import torch

        self.N, self.K, self.fmt, self.scale_group, self.act_dtype, self.max_M = N, K, fmt, scale_group, act_dtype, max_M
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.t = {k: _dev(v, self.device) for k, v in arrays.items() if v is not None and k in
                  ("lo", "hi4", "s2", "idx16", "idx8", "cb1", "cb2", "cbr", "cb8", "scales")}
        self.n16, self.n8, self.mult = 0, 0, ()
        cbr = ()
        if fmt == B.VQ_FMT_VQ16_RVQ:
            ng = N * (K // 8)
            self.n16 = int(np.asarray(arrays["idx16"]).size // ng)
            self.n8 = 1 if arrays.get("idx8") is not None else 0
            self.mult = tuple(float(m) for m in np.asarray(arrays["mult"], dtype=np.float32))
            if "cbr" in self.t:
                stride = 65536 * 8 * 2
                cbr = tuple(self.t["cbr"].data_ptr() + i * stride for i in range(self.n16 - 1))
        self.corr = 0
        if arrays.get("corr") is not None:
            c = arrays["corr"]
            self.corr = 1
            self.t["corr_rows"] = _dev(np.asarray(c["row_ptr"], np.int32), self.device)
            if len(c["col"]):
                self.t["corr_cols"] = _dev(np.asarray(c["col"], np.int32), self.device)
                self.t["corr_vals"] = _dev(np.asarray(c["val"], np.uint16), self.device)
        self.planes = B.make_planes(self.t.get("lo"), self.t.get("hi4"), self.t.get("s2"), self.t.get("idx16"),
                                    self.t.get("idx8"), self.t.get("corr_rows"), self.t.get("corr_cols"),
                                    self.t.get("corr_vals"))
        self.codebooks = B.make_codebooks(self.t["cb1"], self.t.get("cb2"), cbr, self.t.get("cb8"))
        with torch.cuda.device(self.device):
            self.handle = B.vq_linear_create(N, K, fmt, scale_group, act_dtype, max_M, rht, self.n16, self.n8,
                                             self.mult, self.corr)

    @property
    def torch_dtype(self):
        import torch

        return torch.bfloat16 if self.act_dtype == B.VQ_BF16 else torch.float16

    def forward(self, x, y=None, stream=None):
        M = x.shape[0]
        if y is None:
            y = _new((M, self.N), self.torch_dtype, self.device, stream)
        B.vq_linear_forward(self.handle, x, self.planes, self.codebooks, self.t["scales"], y, M, self.N, self.K,
                            stream)
        return y

    __call__ = forward

    def forward_rotated(self, x, signs, y=None, stream=None):
        """y = rotate(x) . W^T (vq_linear_forward_rotated); `signs` is an int8 tensor of +-1 [K]."""
        M = x.shape[0]
        if y is None:
            y = _new((M, self.N), self.torch_dtype, self.device, stream)
        B.vq_linear_forward_rotated(self.handle, x, signs, self.planes, self.codebooks, self.t["scales"], y, M, self.N,
                                    self.K, stream)
        return y

    def forward_fused(self, x, act=B.VQ_ACT_NONE, bias=None, mul=None, residual=None, signs=None, y=None, stream=None):
        """y = act(x . W^T + bias) * mul + residual in one forward (vq_linear_forward_epilogue).

        x [M, K], bias [N], mul and residual [M, N] are contiguous tensors of the layer's
        type on its device, each of the last three may be None; mul and residual may be `y`
        itself (``forward_fused(x, residual=h, y=h)`` adds to h in place).  `act` is a VQ_ACT_*.
        With `signs` (int8 [K]) x is rotated first, as by ``forward_rotated``."""
        import torch

        dt, dev, M, N = self.torch_dtype, self.device, x.shape[0], self.N
        check_tensor(x, "x", (M, self.K), dt, dev)
        if bias is not None:
            check_tensor(bias, "bias", (N,), dt, dev)
        if mul is not None:
            check_tensor(mul, "mul", (M, N), dt, dev)
        if residual is not None:
            check_tensor(residual, "residual", (M, N), dt, dev)
        if signs is not None:
            check_tensor(signs, "signs", (self.K,), torch.int8, dev)
        if y is None:
            y = _new((M, N), dt, dev, stream)
        else:
            check_tensor(y, "y", (M, N), dt, dev)
        if M > 0:
            B.vq_linear_forward_epilogue(self.handle, x, self.planes, self.codebooks, self.t["scales"],
                                         B.make_epilogue(act, bias, mul, residual), y, M, N, self.K, signs,
                                         _raw_stream(stream, dev.index))
        return y

    def set_path(self, path: int):
        B.vq_linear_set_path(self.handle, path)

    def set_sm_budget(self, sms: int):
        """Run the batch-1 table kernel on at most `sms` SMs (0: all of them)."""
        B.vq_linear_set_sm_budget(self.handle, sms)

    def launches(self, M: int) -> int:
        return B.vq_linear_launches(self.handle, M)

    def plan(self, M: int) -> dict:
        """How a forward of M tokens runs (path, launches, ctas, splits)."""
        return B.vq_linear_plan(self.handle, M)

    def close(self):
        if getattr(self, "handle", None):
            B.vq_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
