"""The dense product y = act(x W^T + b) + r and its gradients (moe_linear,
moe_linear_backward): a descriptor and an object that holds the weights.
"""

from __future__ import annotations

import contextlib

import torch

from . import _abi as abi
from .layer import _DT, _TORCH_DT

_ACT = {"none": abi.MOE_ACT_NONE, "relu": abi.MOE_ACT_RELU, "silu": abi.MOE_ACT_SILU, "gelu": abi.MOE_ACT_GELU}


def make_linear_desc(M: int, N: int, K: int, dtype="bf16", act: str = "none", out_f32: bool = False,
                     grad_f32: bool = False, ld_x: int = 0, ld_w: int = 0, ld_y: int = 0, ld_r: int = 0, ld_z: int = 0,
                     ld_dx: int = 0) -> abi.MoELinearDesc:
    """Row strides ld_* in elements; 0: the rows are contiguous."""
    return abi.MoELinearDesc(M=M, N=N, K=K, dtype=_DT[dtype], act=_ACT[act], out_f32=int(bool(out_f32)),
                             grad_f32=int(bool(grad_f32)), ld_x=ld_x, ld_w=ld_w, ld_y=ld_y, ld_r=ld_r, ld_z=ld_z,
                             ld_dx=ld_dx)


_HERE = contextlib.nullcontext()


class Linear:
    """A dense product with device-resident weights w [N, K] and bias [N] (fp32, or None).

    forward(x [M, K]) and backward(x, dy [M, N]) take any M; the descriptor gives the other sizes, the types
    and the row stride of w.  The row strides of the other tensors are read from the tensors.  Nothing is kept
    from one call to the next: workspace and outputs come from torch's allocator on the call's stream.
    """

    def __init__(self, desc: abi.MoELinearDesc, w: torch.Tensor, bias: torch.Tensor | None = None):
        self.desc = desc
        self.dtype = _TORCH_DT.get(desc.dtype)
        self.out_dtype = torch.float32 if desc.out_f32 else self.dtype
        self.grad_dtype = torch.float32 if desc.grad_f32 else self.dtype
        self.w, self.bias = w, bias                  # keeps the tensors alive
        self._check("w", w, desc.N, desc.K, self.dtype)
        if w.stride(0) != (desc.ld_w or desc.K) and desc.N > 1:
            raise ValueError(f"w: expected a row stride of {desc.ld_w or desc.K}, got {w.stride(0)}")
        if bias is not None and (tuple(bias.shape) != (desc.N,) or bias.dtype != torch.float32):
            raise ValueError(f"bias: expected a [{desc.N}] torch.float32 tensor, got {list(bias.shape)} {bias.dtype}")

    def _check(self, name, t, rows, cols, dtype) -> None:
        if t is None:
            return
        if t.shape != (rows, cols) or t.dtype != dtype:
            raise ValueError(f"{name}: expected a [{rows}, {cols}] {dtype} tensor, got {list(t.shape)} {t.dtype}")
        s0, s1 = t.stride()
        if cols > 1 and s1 != 1 or rows > 1 and s0 < cols:
            raise ValueError(f"{name}: expected contiguous rows that do not overlap, got strides {(s0, s1)}")
        if t.device != self.w.device:
            raise ValueError(f"{name}: on {t.device}, the weights are on {self.w.device}")

    def _call_desc(self, x, y=None, residual=None, z=None, dx=None) -> abi.MoELinearDesc:
        d = self.desc
        M = x.shape[0]

        def ld(t):          # (one row has no stride)
            return t.stride(0) if t is not None and M > 1 else 0

        return abi.MoELinearDesc(M, d.N, d.K, d.dtype, d.act, d.out_f32, d.grad_f32, ld(x), d.ld_w, ld(y), ld(residual),
                                 ld(z), ld(dx))

    def _on(self, stream):
        """(context, stream) of a call: where it allocates and launches.  The weights' device need not be current."""
        if not self.w.is_cuda:
            raise ValueError("libmoe takes CUDA tensors")
        if stream is None:
            if self.w.get_device() == torch.cuda.current_device():
                return _HERE, None
            return torch.cuda.device(self.w.device), None
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.w.device)
        if stream.device != self.w.device:
            raise ValueError(f"stream: on {stream.device}, the weights are on {self.w.device}")
        return torch.cuda.stream(stream), stream

    def forward(self, x: torch.Tensor, residual=None, y=None, z=None, stream=None) -> torch.Tensor:
        """y = act(x w^T + bias) + residual; the pre-activation is written to z where one is given."""
        d = self.desc
        M = x.shape[0] if x.dim() == 2 else -1
        self._check("x", x, M, d.K, self.dtype)
        self._check("residual", residual, M, d.N, self.out_dtype)
        self._check("y", y, M, d.N, self.out_dtype)
        self._check("z", z, M, d.N, self.dtype)
        ctx, stream = self._on(stream)
        with ctx:
            if y is None:
                y = torch.empty((M, d.N), dtype=self.out_dtype, device=x.device)
            cd = self._call_desc(x, y, residual, z)
            need = abi.moe_linear_workspace_size(cd)
            ws = torch.empty((need,), dtype=torch.uint8, device=x.device) if need > 0 else None
            abi.moe_linear(cd, x, self.w, self.bias, residual, y, z, ws, stream)
        return y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, z=None, dx=None, dw=None, db=None, need_dx: bool = True,
                 need_dw: bool = True, need_db: bool | None = None, stream=None):
        """(dx, dw, db); one that is not needed is None (db by default: only with a bias).  z: as forward wrote it."""
        d = self.desc
        M = x.shape[0] if x.dim() == 2 else -1
        self._check("x", x, M, d.K, self.dtype)
        self._check("dy", dy, M, d.N, self.out_dtype)
        self._check("z", z, M, d.N, self.dtype)
        self._check("dx", dx, M, d.K, self.dtype)
        self._check("dw", dw, d.N, d.K, self.grad_dtype)
        if z is None and d.act != abi.MOE_ACT_NONE:
            raise ValueError("z: the gradient of an activation needs the pre-activation")
        if db is not None and (tuple(db.shape) != (d.N,) or db.dtype != torch.float32):
            raise ValueError(f"db: expected a [{d.N}] torch.float32 tensor, got {list(db.shape)} {db.dtype}")
        ctx, stream = self._on(stream)
        with ctx:
            if dx is None and need_dx:
                dx = torch.empty((M, d.K), dtype=self.dtype, device=x.device)
            if dw is None and need_dw:
                dw = torch.empty((d.N, d.K), dtype=self.grad_dtype, device=x.device)
            if db is None and (self.bias is not None if need_db is None else need_db):
                db = torch.empty((d.N,), dtype=torch.float32, device=x.device)
            if dx is None and dw is None and db is None:
                return None, None, None
            cd = self._call_desc(x, dy, None, z, dx)
            need = abi.moe_linear_backward_workspace_size(cd)
            ws = torch.empty((need,), dtype=torch.uint8, device=x.device) if need > 0 else None
            abi.moe_linear_backward(cd, x, self.w, z, dy, dx, dw, db, ws, stream)
        return dx, dw, db

    __call__ = forward
