"""Marshalling between torch tensors and the C ABI.

PyTorch only provides device memory and streams here; the calls go straight to
libdspark.so through :mod:`._abi`.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np
import torch

from . import _abi

_DT = {"f32": _abi.DSPARK_F32, "bf16": _abi.DSPARK_BF16}


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# (the current stream's handle without a Stream object, which takes longer than a launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, here: Optional[int] = None) -> int:
    """The stream's handle; None: the current one (of the current GPU, `here` where it is known)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if here is None else here)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def to_device(a, device="cuda") -> torch.Tensor:
    """numpy -> device tensor; uint16 arrays are bf16 bit patterns."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(a).to(device)


def make_config(B, L_in, H, V, r, top_k, sample_from_anchor, conf_min, dtype,
                topk_markov=True, skip_truncated=False) -> _abi.dspark_config:
    return _abi.dspark_config(B=B, L_in=L_in, H=H, V=V, r=r, top_k=top_k,
                              sample_from_anchor=int(bool(sample_from_anchor)),
                              topk_markov=int(bool(topk_markov)), conf_min=float(conf_min),
                              dtype=_DT[dtype] if isinstance(dtype, str) else int(dtype),
                              skip_truncated=int(bool(skip_truncated)))


@dataclasses.dataclass
class Head:
    """Device copies of a drafter head and the matching dspark_head struct."""
    lm_head: torch.Tensor
    markov_w1: Optional[torch.Tensor]      # None: no Markov term (dspark_head_loss, r = 0)
    markov_w2: Optional[torch.Tensor]
    lm_bias: Optional[torch.Tensor] = None
    d2t: Optional[torch.Tensor] = None
    w_conf: Optional[torch.Tensor] = None
    b_conf: float = 0.0
    prepared: Optional[torch.Tensor] = None

    @property
    def V_head(self) -> int:
        return int(self.lm_head.shape[0])

    def struct(self) -> _abi.dspark_head:
        return _abi.dspark_head(lm_head=_ptr(self.lm_head), lm_bias=_ptr(self.lm_bias),
                                d2t=_ptr(self.d2t), V_head=self.V_head,
                                markov_w1=_ptr(self.markov_w1),
                                markov_w2=_ptr(self.markov_w2), w_conf=_ptr(self.w_conf),
                                b_conf=float(self.b_conf), prepared=_ptr(self.prepared))

    def prepare(self, cfg, stream=None) -> "Head":
        """Fill ``prepared`` with dspark_prepare_head (enables the pruned chain)."""
        bare = dataclasses.replace(self, prepared=None)
        n = _abi.dspark_prepare_head_size(cfg, bare.struct())
        if n == 0:
            _abi.check(_abi.DSPARK_ERR_UNSUPPORTED)
        buf = torch.empty(n, dtype=torch.uint8, device=self.lm_head.device)
        _abi.check(_abi.dspark_prepare_head(cfg, bare.struct(), buf.data_ptr(), n,
                                            _stream(stream)))
        self.prepared = buf
        return self


def head_to_device(h: dict, form: str = "full", device="cuda") -> Head:
    """Upload a head dict of ``workloads.make_head``.

    form "full": lm_head / markov_w2 over the whole vocabulary (+ lm_bias if any);
    form "d2t": the compact head of the emittable rows plus the d2t table (the
    reduced-vocabulary form of llama.cpp PR #26275); the gather is done here on the host.
    """
    w_conf = None if h.get("w_conf") is None else to_device(h["w_conf"], device)
    if form == "full":
        return Head(to_device(h["lm_head"], device), to_device(h["markov_w1"], device),
                    to_device(h["markov_w2"], device),
                    None if h.get("lm_bias") is None else to_device(h["lm_bias"], device),
                    None, w_conf, h.get("b_conf", 0.0))
    if form == "d2t":
        rows = h["emit_rows"]
        return Head(to_device(h["lm_head"][rows], device), to_device(h["markov_w1"], device),
                    to_device(np.ascontiguousarray(h["markov_w2"][:, rows]), device),
                    to_device(h["lm_bias"][rows], device),
                    to_device(rows.astype(np.int32), device), w_conf, h.get("b_conf", 0.0))
    raise ValueError(form)


@dataclasses.dataclass
class Outputs:
    draft: torch.Tensor
    n_draft: torch.Tensor
    topk_ids: Optional[torch.Tensor] = None
    topk_vals: Optional[torch.Tensor] = None
    conf: Optional[torch.Tensor] = None
    logits: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, B, N, k, V_head, device="cuda", topk=True, conf=True, logits=False):
        i32 = dict(dtype=torch.int32, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        return cls(torch.empty(B, N, **i32), torch.empty(B, **i32),
                   torch.empty(B, N, k, **i32) if topk else None,
                   torch.empty(B, N, k, **f32) if topk else None,
                   torch.empty(B, N, **f32) if conf else None,
                   torch.empty(B, N, V_head, **f32) if logits else None)

    def struct(self) -> _abi.dspark_outputs:
        return _abi.dspark_outputs(draft=_ptr(self.draft), n_draft=_ptr(self.n_draft),
                                   topk_ids=_ptr(self.topk_ids), topk_vals=_ptr(self.topk_vals),
                                   conf=_ptr(self.conf), logits=_ptr(self.logits))

    def numpy(self) -> dict:
        return {k: (None if v is None else v.cpu().numpy())
                for k, v in dataclasses.asdict(self).items()}


def workspace_for(cfg, head: Head, device="cuda") -> torch.Tensor:
    n = _abi.dspark_propose_workspace_size(cfg, head.struct())
    if n == 0:
        _abi.check(_abi.DSPARK_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def propose(cfg, head: Head, hidden: torch.Tensor, anchors: torch.Tensor, out: Outputs,
            workspace: torch.Tensor, stream=None, conf_hidden: Optional[torch.Tensor] = None
            ) -> None:
    """dspark_propose on torch tensors; raises DSparkError on a non-OK status."""
    _abi.check(_abi.dspark_propose(cfg, head.struct(), hidden.data_ptr(), anchors.data_ptr(),
                                   out.struct(), workspace.data_ptr(), workspace.numel(),
                                   _stream(stream), _ptr(conf_hidden)))


def verify(draft, n_draft, target, accepted, bonus, emitted=None, stream=None) -> None:
    """dspark_verify on torch tensors; raises DSparkError on a non-OK status."""
    B, N = draft.shape
    _abi.check(_abi.dspark_verify(B, N, draft.data_ptr(), n_draft.data_ptr(),
                                  target.data_ptr(), accepted.data_ptr(), bonus.data_ptr(),
                                  _ptr(emitted), _stream(stream)))


def tree_verify(topk_ids, n_draft, target, accepted, bonus, emitted=None, path=None,
                stream=None) -> None:
    """dspark_tree_verify on torch tensors; raises DSparkError on a non-OK status."""
    B, N, k = topk_ids.shape
    _abi.check(_abi.dspark_tree_verify(B, N, k, topk_ids.data_ptr(), n_draft.data_ptr(),
                                       target.data_ptr(), accepted.data_ptr(),
                                       bonus.data_ptr(), _ptr(emitted), _ptr(path),
                                       _stream(stream)))


def device_status(workspace: torch.Tensor, stream=None) -> int:
    return _abi.dspark_device_status(workspace.data_ptr(), _stream(stream))


def pass_stats(workspace: torch.Tensor, stream=None) -> dict:
    return _abi.dspark_pass_stats(workspace.data_ptr(), _stream(stream))


# ------------------------------------------------------------------ training the head
_TORCH_DT = {_abi.DSPARK_F32: torch.float32, _abi.DSPARK_BF16: torch.bfloat16}
_REDUCTION = {"sum": _abi.DSPARK_LOSS_SUM, "mean": _abi.DSPARK_LOSS_MEAN}


def _checked(name: str, t: Optional[torch.Tensor], shape, dtype) -> Optional[int]:
    """The address of a dense tensor of the given shape and type (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _here() -> int:
    """The current GPU, -2 where there is none.  (torch.cuda.current_device takes twice as long.)"""
    try:
        return torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        return -2


def _on_this_gpu(names, *tensors) -> int:
    """Refuses tensors (None: absent) that are not on the current GPU: the kernels would take their
    addresses all the same.  Returns the GPU."""
    here = _here()
    for t in tensors:
        if t is not None and t.get_device() != here:         # (-1: not on a GPU)
            name = [n for n, u in zip(names, tensors) if u is t][0]
            raise ValueError(f"{name}: need a tensor on the current GPU, got one on {t.device}")
    return here


def _room(workspace: torch.Tensor):
    """A workspace's address and bytes."""
    if not workspace.is_contiguous():
        raise ValueError("workspace: need a contiguous tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def make_loss_config(T, H, V, r, dtype, reduction="mean", loss_scale=1.0,
                     vocab_pieces=0) -> _abi.dspark_loss_config:
    return _abi.dspark_loss_config(T=T, H=H, V=V, r=r,
                                   dtype=_DT[dtype] if isinstance(dtype, str) else int(dtype),
                                   reduction=_REDUCTION[reduction],
                                   vocab_pieces=int(vocab_pieces),
                                   loss_scale=float(loss_scale))


@dataclasses.dataclass
class LossOutputs:
    loss: torch.Tensor
    total: torch.Tensor
    n_rows: Optional[torch.Tensor] = None
    d_hidden: Optional[torch.Tensor] = None
    d_lm_head: Optional[torch.Tensor] = None
    d_markov_w1: Optional[torch.Tensor] = None
    d_markov_w2: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, cfg, head: Head, d_hidden=True, d_lm_head=True, d_markov=True,
                 device="cuda"):
        e = dict(dtype=_TORCH_DT[cfg.dtype], device=device)
        f32 = dict(dtype=torch.float32, device=device)
        markov = d_markov and cfg.r > 0
        return cls(torch.empty(cfg.T, **f32), torch.empty(1, **f32),
                   torch.empty(1, dtype=torch.int32, device=device),
                   torch.empty(cfg.T, cfg.H, **e) if d_hidden else None,
                   torch.empty(head.V_head, cfg.H, **e) if d_lm_head else None,
                   torch.empty(cfg.V, cfg.r, **e) if markov else None,
                   torch.empty(cfg.r, head.V_head, **e) if markov else None)

    def struct(self) -> _abi.dspark_loss_outputs:
        return _abi.dspark_loss_outputs(
            loss=_ptr(self.loss), total=_ptr(self.total), n_rows=_ptr(self.n_rows),
            d_hidden=_ptr(self.d_hidden), d_lm_head=_ptr(self.d_lm_head),
            d_markov_w1=_ptr(self.d_markov_w1), d_markov_w2=_ptr(self.d_markov_w2))


def loss_workspace_for(cfg, head: Head, out: LossOutputs, device="cuda") -> torch.Tensor:
    n = _abi.dspark_head_loss_workspace_size(cfg, head.struct(), out.struct())
    if n == 0:
        _abi.check(_abi.DSPARK_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def head_loss(cfg, head: Head, hidden, prev, labels, out: LossOutputs, workspace,
              weights=None, stream=None) -> None:
    """dspark_head_loss on torch tensors; raises DSparkError on a non-OK status."""
    e, f32, i32 = _TORCH_DT.get(cfg.dtype), torch.float32, torch.int32
    V, r, vh = cfg.V, cfg.r, head.V_head
    tensors = (
        ("lm_head", head.lm_head, (vh, cfg.H), e), ("lm_bias", head.lm_bias, (vh,), f32),
        ("d2t", head.d2t, (vh,), i32), ("markov_w1", head.markov_w1, (V, r), e),
        ("markov_w2", head.markov_w2, (r, vh), e), ("loss", out.loss, (cfg.T,), f32),
        ("total", out.total, (1,), f32), ("n_rows", out.n_rows, (1,), i32),
        ("d_hidden", out.d_hidden, (cfg.T, cfg.H), e),
        ("d_lm_head", out.d_lm_head, (vh, cfg.H), e),
        ("d_markov_w1", out.d_markov_w1, (V, r), e),
        ("d_markov_w2", out.d_markov_w2, (r, vh), e))
    for t in tensors:
        _checked(*t)
    prev = prev if r > 0 else None
    args = (_checked("hidden", hidden, (cfg.T, cfg.H), e), _checked("prev", prev, (cfg.T,), i32),
            _checked("labels", labels, (cfg.T,), i32), _checked("weights", weights, (cfg.T,), f32))
    here = _on_this_gpu(
        [t[0] for t in tensors] + ["hidden", "prev", "labels", "weights", "workspace"],
        *[t[1] for t in tensors], hidden, prev, labels, weights, workspace)
    _abi.check(_abi.dspark_head_loss(cfg, head.struct(), *args, out.struct(), *_room(workspace),
                                     _stream(stream, here)))


def make_norm_config(T, H, dtype, eps=1e-6, residual_scale=1.0, weight_offset=0.0,
                     gate_span=1) -> _abi.dspark_norm_config:
    return _abi.dspark_norm_config(T=T, H=H,
                                   dtype=_DT[dtype] if isinstance(dtype, str) else int(dtype),
                                   gate_span=int(gate_span), eps=float(eps),
                                   residual_scale=float(residual_scale),
                                   weight_offset=float(weight_offset))


@dataclasses.dataclass
class NormGrads:
    d_x: torch.Tensor
    d_y: Optional[torch.Tensor]
    d_gate: Optional[torch.Tensor]
    d_w_post: Optional[torch.Tensor]
    d_w_pre: torch.Tensor

    @classmethod
    def allocate(cls, cfg, gate=True, w_post=True, y=True, device="cuda"):
        e = dict(dtype=_TORCH_DT[cfg.dtype], device=device)
        rows = (cfg.T + cfg.gate_span - 1) // cfg.gate_span
        return cls(torch.empty(cfg.T, cfg.H, **e),
                   torch.empty(cfg.T, cfg.H, **e) if y else None,
                   torch.empty(rows, cfg.H, **e) if gate else None,
                   torch.empty(cfg.H, **e) if w_post else None, torch.empty(cfg.H, **e))


def norm_workspace_for(cfg, device="cuda") -> torch.Tensor:
    n = _abi.dspark_block_norm_workspace_size(cfg)
    if n == 0:
        _abi.check(_abi.DSPARK_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def _norm_shapes(cfg):
    rows = (cfg.T + cfg.gate_span - 1) // cfg.gate_span if cfg.gate_span > 0 else 0
    return (cfg.T, cfg.H), (rows, cfg.H), (cfg.H,), _TORCH_DT.get(cfg.dtype)


def block_norm(cfg, x, y, w_pre, h, x_out=None, gate=None, w_post=None, stream=None) -> None:
    """dspark_block_norm on torch tensors; raises DSparkError on a non-OK status."""
    row, gat, vec, e = _norm_shapes(cfg)
    args = (_checked("x", x, row, e), _checked("y", y, row, e), _checked("gate", gate, gat, e),
            _checked("w_post", w_post, vec, e), _checked("w_pre", w_pre, vec, e),
            _checked("x_out", x_out, row, e), _checked("h", h, row, e))
    here = _on_this_gpu(("x", "y", "gate", "w_post", "w_pre", "x_out", "h"),
                        x, y, gate, w_post, w_pre, x_out, h)
    _abi.check(_abi.dspark_block_norm(cfg, *args, _stream(stream, here)))


def block_norm_backward(cfg, x, y, w_pre, d_h, out: NormGrads, workspace, d_x_out=None,
                        gate=None, w_post=None, stream=None) -> None:
    """dspark_block_norm_backward on torch tensors; raises DSparkError on a non-OK status."""
    row, gat, vec, e = _norm_shapes(cfg)
    args = (_checked("x", x, row, e), _checked("y", y, row, e), _checked("gate", gate, gat, e),
            _checked("w_post", w_post, vec, e), _checked("w_pre", w_pre, vec, e),
            _checked("d_h", d_h, row, e), _checked("d_x_out", d_x_out, row, e),
            _checked("d_x", out.d_x, row, e), _checked("d_y", out.d_y, row, e),
            _checked("d_gate", out.d_gate, gat, e), _checked("d_w_post", out.d_w_post, vec, e),
            _checked("d_w_pre", out.d_w_pre, vec, e))
    here = _on_this_gpu(
        ("x", "y", "gate", "w_post", "w_pre", "d_h", "d_x_out", "d_x", "d_y", "d_gate", "d_w_post",
         "d_w_pre", "workspace"), x, y, gate, w_post, w_pre, d_h, d_x_out, out.d_x, out.d_y,
        out.d_gate, out.d_w_post, out.d_w_pre, workspace)
    _abi.check(_abi.dspark_block_norm_backward(cfg, *args, *_room(workspace), _stream(stream, here)))


class GradList:
    """The gradients of one clip_grads call and where their clipped values go (``outs``;
    None: in place).  Holds the tensors, so that the addresses stay valid."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("outs must have one tensor for each gradient")
        dt = {v: k for k, v in _TORCH_DT.items()}
        self.array = (_abi.dspark_grad * len(self.grads))()
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.dtype not in dt:
                raise ValueError(f"gradient {i}: float32 or bfloat16, not {g.dtype}")
            _checked(f"gradient {i}", g, g.shape, g.dtype)
            _checked(f"outs[{i}]", o, g.shape, g.dtype)
            _on_this_gpu((f"gradient {i}", f"outs[{i}]"), g, o)
            self.array[i] = _abi.dspark_grad(in_=g.data_ptr(), out=o.data_ptr(), n=g.numel(),
                                             dtype=dt[g.dtype])

    def __len__(self):
        return len(self.grads)


def clip_workspace_for(grads: GradList, device="cuda") -> torch.Tensor:
    n = _abi.dspark_clip_grads_workspace_size(len(grads), grads.array)
    if n == 0:
        _abi.check(_abi.DSPARK_ERR_INVALID_ARG)
    return torch.empty(n, dtype=torch.uint8, device=device)


def clip_grads(grads: GradList, max_norm, norm, workspace, stream=None) -> None:
    """dspark_clip_grads on torch tensors; raises DSparkError on a non-OK status."""
    at = _checked("norm", norm, (1,), torch.float32)
    here = _on_this_gpu(("norm", "workspace"), norm, workspace)
    _abi.check(_abi.dspark_clip_grads(len(grads), grads.array, float(max_norm), at,
                                      *_room(workspace), _stream(stream, here)))
