"""Sequencing of the four library calls for one layer (or a batch of experts).

Allocation of outputs and workspaces goes through torch; every computation is
one of the library's entry points.
"""
from __future__ import annotations

import contextlib
from typing import Dict, Optional, Sequence

import numpy as np
import torch

from . import (BF16, E4M3, F16, F32, GptqError, GptqParams, OP_ABS, OP_AWQ_SEARCH, OP_DISTILL, OP_FORWARD,
               OP_FP8_MATMUL, OP_HESSIAN, OP_LOGPROBS, OP_LORA, OP_POLICY, OP_PREPARE, OP_QUANTIZE, OP_W4A16, OP_W4A16_LORA, ENOTPD, _check, dtype_code,
               gptq_abs_accumulate, gptq_awq_apply, gptq_awq_search, gptq_hessian_accumulate, gptq_layer_forward,
               gptq_lora_grad_workspace_size,
               gptq_pack_bits, gptq_pack_int4, gptq_pack_int4_permuted, gptq_prepare_hinv, gptq_quantize_layer,
               gptq_w4a16_matmul, gptq_workspace_size, lib)


def to_device(arr: np.ndarray, dtype: str, device="cuda") -> torch.Tensor:
    """Host array in storage form ('f32', 'f16', or 'bf16' as uint16 bits) -> device tensor."""
    if dtype == "bf16":
        return torch.from_numpy(np.ascontiguousarray(arr).view(np.int16)).to(device).view(torch.bfloat16)
    return torch.from_numpy(np.ascontiguousarray(arr)).to(device)


def _on(stream, device: torch.device):
    """Context in which what torch allocates on the device belongs to the call's stream."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream)


def _ws(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class HessianState:
    """The running accumulator (S, D, N) of one layer or of a batch of experts,
    all in device memory (N: int64 rows used per entry)."""

    def __init__(self, d_in: int, batch: int = 1, device="cuda", track_abs: bool = False):
        self.d_in, self.batch, self.device = int(d_in), int(batch), device
        self.S = torch.zeros(batch, d_in, d_in, dtype=torch.float32, device=device)
        self.D = torch.zeros(batch, d_in, dtype=torch.float64, device=device)
        # per-channel sum of |x| (activation-aware scaling), when asked for
        self.A = torch.zeros(batch, d_in, dtype=torch.float64, device=device) if track_abs else None
        self.n = torch.zeros(batch, dtype=torch.int64, device=device)
        self._ws = None

    def workspace(self, n_rows: int) -> torch.Tensor:
        need = gptq_workspace_size(OP_HESSIAN, None, 1, self.d_in, n_rows, self.batch)
        if self._ws is None or self._ws.numel() < need:
            self._ws = _ws(need, self.device)
        return self._ws

    def zero(self) -> None:
        self.S.zero_()
        self.D.zero_()
        if self.A is not None:
            self.A.zero_()
        self.n.zero_()

    def add(self, X: torch.Tensor, row_idx: Optional[torch.Tensor] = None,
            row_ptr: Optional[Sequence[int]] = None, stream=None) -> None:
        n_rows = X.shape[0]
        rows_for_ws = n_rows if row_idx is None else int(np.max(np.diff(np.asarray(row_ptr))))
        ws = self.workspace(rows_for_ws)
        nb = self.batch if row_idx is not None else 1
        if self.A is not None:
            need = gptq_workspace_size(OP_ABS, None, 1, self.d_in, rows_for_ws, nb)
            if ws.numel() < need:
                ws = self._ws = _ws(need, self.device)
            gptq_abs_accumulate(self.A, X, dtype_code(X.dtype), n_rows, self.d_in, X.stride(0), row_idx, row_ptr,
                                nb, ws, ws.numel(), stream)
        gptq_hessian_accumulate(self.S, self.D, self.n, X, self.d_in, n_rows, X.stride(0), dtype_code(X.dtype),
                                row_idx, row_ptr, nb, ws, ws.numel(), stream)


class Prepared:
    def __init__(self, U, perm, info):
        self.U, self.perm, self.info = U, perm, info


def prepare(state: HessianState, params: GptqParams, ws: Optional[torch.Tensor] = None, stream=None,
            check: bool = True) -> Prepared:
    d, b, dev = state.d_in, state.batch, state.device
    U = torch.empty(b, d, d, dtype=torch.float32, device=dev)
    perm = torch.empty(b, d, dtype=torch.int32, device=dev) if params.act_order else None
    info = torch.empty(b, dtype=torch.int32, device=dev)
    need = gptq_workspace_size(OP_PREPARE, None, 1, d, 0, b)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    gptq_prepare_hinv(state.S, state.D, state.n, d, b, params, U, perm, info, ws, ws.numel(), stream)
    out = Prepared(U, perm, info)
    if check:
        bad = info.cpu().numpy()
        if np.any(bad != 0):
            raise GptqError(ENOTPD, f"gptq_prepare_hinv (info={bad.tolist()})")
    return out


def quantize(W: torch.Tensor, prep: Prepared, params: GptqParams, want_q: bool = False,
             ws: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """W: (batch, d_out, d_in) or (d_out, d_in) tensor of fp32/fp16/bf16."""
    if W.dim() == 2:
        W = W.unsqueeze(0)
    b, d_out, d_in = W.shape
    dev = W.device
    ng = d_in // params.group_size
    codes = torch.empty(b, d_out, d_in, dtype=torch.uint8, device=dev)
    scales = torch.empty(b, d_out, ng, dtype=torch.int16, device=dev)
    zeros = torch.empty(b, d_out, ng, dtype=torch.uint8, device=dev)
    g_idx = torch.empty(b, d_in, dtype=torch.int32, device=dev)
    Q = torch.empty(b, d_out, d_in, dtype=torch.float32, device=dev) if want_q else None
    need = gptq_workspace_size(OP_QUANTIZE, params, d_out, d_in, 0, b)
    if ws is None or ws.numel() < need:
        ws = _ws(need, dev)
    gptq_quantize_layer(W, dtype_code(W.dtype), d_out, d_in, W.stride(1), b, prep.U, prep.perm, params, codes,
                        scales, zeros, g_idx, Q, ws, ws.numel(), stream)
    return dict(codes=codes, scales=scales, zeros=zeros, g_idx=g_idx, Q=Q)


def pack(codes: torch.Tensor, bits: int, stream=None) -> torch.Tensor:
    """Pack the last dimension of a uint8 code tensor (4-bit nibbles or a dense bit stream)."""
    shape = codes.shape
    rows = int(np.prod(shape[:-1]))
    cols = shape[-1]
    out = torch.empty(*shape[:-1], cols * bits // 8, dtype=torch.uint8, device=codes.device)
    if bits == 4:
        gptq_pack_int4(codes, rows, cols, out, stream)
    else:
        gptq_pack_bits(codes, rows, cols, bits, out, stream)
    return out


def pack_int4_permuted(codes: torch.Tensor, perm: torch.Tensor, stream=None) -> torch.Tensor:
    """4-bit packing of a (rows, cols) code matrix with its columns taken in the order perm."""
    rows, cols = codes.shape
    out = torch.empty(rows, cols // 2, dtype=torch.uint8, device=codes.device)
    gptq_pack_int4_permuted(codes, rows, cols, perm, out, stream)
    return out


def w4a16_matmul(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                 group_size: int, perm: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = X Q^T (fp32) from the packed 4-bit weights; X is (M, d_in) fp16 or bf16."""
    M, d_in = X.shape
    d_out = qweight.shape[0]
    if Y is None:
        Y = torch.empty(M, d_out, dtype=torch.float32, device=X.device)
    need = gptq_workspace_size(OP_W4A16, None, d_out, d_in, M, 1)
    if ws is None or ws.numel() < need:
        ws = _ws(need, X.device)
    gptq_w4a16_matmul(X, dtype_code(X.dtype), M, d_in, X.stride(0), qweight, scales, zeros, perm, d_out,
                      group_size, Y, Y.stride(0), ws, ws.numel(), stream)
    return Y


def awq_search(W: torch.Tensor, state: HessianState, Xs: torch.Tensor, params: GptqParams,
               alphas: Sequence[float], entry: int = 0, stream=None) -> Dict[str, object]:
    """Candidate errors, the chosen index and its per-channel scales for one
    layer W (d_out, d_in), from the state's |x| sums and a token sample Xs."""
    d_out, d_in = W.shape
    dev = W.device
    err = torch.empty(len(alphas), dtype=torch.float64, device=dev)
    s = torch.empty(d_in, dtype=torch.float32, device=dev)
    best = torch.empty(1, dtype=torch.int32, device=dev)
    need = gptq_workspace_size(OP_AWQ_SEARCH, None, d_out, d_in, Xs.shape[0], len(alphas))
    ws = _ws(need, dev)
    gptq_awq_search(W, dtype_code(W.dtype), d_out, d_in, W.stride(0), state.A[entry], state.n[entry:entry + 1], Xs,
                    dtype_code(Xs.dtype), Xs.shape[0], Xs.stride(0), params, alphas, err, s, best, ws, ws.numel(),
                    stream)
    return dict(err=err, s=s, best=best)


def awq_apply(W: torch.Tensor, state: HessianState, s: torch.Tensor, entry: int = 0, stream=None) -> torch.Tensor:
    """Scale the state's Hessian in place and return W' = fp32(W s)."""
    d_out, d_in = W.shape
    Wp = torch.empty(d_out, d_in, dtype=torch.float32, device=W.device)
    gptq_awq_apply(state.S[entry], state.D[entry], d_in, s, W, dtype_code(W.dtype), d_out, W.stride(0), Wp, stream)
    return Wp


def layer_forward(X: torch.Tensor, Q: torch.Tensor, act: int, Y: Optional[torch.Tensor] = None,
                  ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = round(act(X Q^T)) in X's format; Q (d_out, d_in) fp32 dequantized weights."""
    n, d_in = X.shape
    d_out = Q.shape[0]
    if Y is None:
        Y = torch.empty(n, d_out, dtype=X.dtype, device=X.device)
    need = gptq_workspace_size(OP_FORWARD, None, d_out, d_in, n, 1)
    if ws is None or ws.numel() < need:
        ws = _ws(need, X.device)
    gptq_layer_forward(X, dtype_code(X.dtype), n, d_in, X.stride(0), Q, d_out, Q.stride(0), act, Y, Y.stride(0),
                       ws, ws.numel(), stream)
    return Y


# ---------------------------------------------------------------- answers: scoring, distillation, adapters
# The calls below are made once per token when a model is served, so they check
# their arguments with few and cheap questions and hand plain addresses to the
# library.
_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream_of(stream, device: int) -> int:
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(function, name: str, device: int, *args) -> None:
    """function(*args) with the tensors' GPU as the current one, which the library launches on."""
    if _current_device() == device:
        _check(function(*args), name)
    else:
        with torch.cuda.device(device):
            _check(function(*args), name)


def _rows(t: torch.Tensor, what: str):
    """(rows, columns, row stride, device index) of a 2-d GPU tensor with contiguous, disjoint rows."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{what}: a GPU tensor is needed")
    if t.dim() != 2:
        raise ValueError(f"{what}: a 2-d tensor is needed")
    n, w = t.shape
    ld, one = t.stride()
    if one != 1 and w > 1 or ld < w and n > 1:
        raise ValueError(f"{what}: contiguous, disjoint rows are needed")
    return n, w, ld if ld > w else w, device


def _dense(t: torch.Tensor, dtype, shape, what: str, device: int) -> int:
    """Address of a contiguous tensor of this type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {device} is needed")
    return t.data_ptr()


def _workspace(ws: torch.Tensor, device: int):
    if not ws.is_contiguous() or ws.get_device() != device:
        raise ValueError(f"ws: a contiguous tensor on GPU {device} is needed")
    return ws.data_ptr(), ws.numel() * ws.element_size()


class Buffers(dict):
    """Output tensors of a call, by name, that were checked when they were made: `key` says for which sizes,
    `addresses` where they are.  Setting an entry makes them ordinary, to be checked in every call."""

    def __init__(self, key, tensors: Dict[str, torch.Tensor]):
        super().__init__(tensors)
        self.key, self.addresses = key, [t.data_ptr() for t in tensors.values()]

    def _changed(self, *args, **kwargs):
        raise TypeError("use out[name] = tensor")

    def __setitem__(self, name, value):
        self.key = None
        super().__setitem__(name, value)

    __delitem__ = pop = popitem = clear = update = setdefault = __ior__ = _changed


def _logprobs_out(n: int, k: int, dev, written: bool) -> Buffers:
    """written: every call fills in logprob; otherwise it starts as 0, what a row that is not scored has."""
    out = {"logprob": (torch.empty if written else torch.zeros)(n, dtype=torch.float32, device=dev)}
    out.update((name, torch.empty(n, dtype=torch.float32, device=dev)) for name in ("lse", "entropy"))
    out["top_logprob"] = torch.empty(n, k, dtype=torch.float32, device=dev)
    out["top_id"] = torch.empty(n, k, dtype=torch.int32, device=dev)
    return Buffers(("logprobs", n, k, dev.index), out)


def token_logprobs_buffers(logits: torch.Tensor, k: int = 0):
    """(out, ws) of token_logprobs calls with these sizes, to be kept from call to call."""
    n, v = logits.shape
    return (_logprobs_out(n, k, logits.device, False),
            _ws(gptq_workspace_size(OP_LOGPROBS, None, 1, v, n, max(k, 1)), logits.device))


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, k: int = 0, temperature: float = 1.0,
                   out: Optional[Dict[str, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> Dict[str, torch.Tensor]:
    """Log probability of targets[i] (int32; outside the vocabulary: not scored, 0), log-sum-exp, entropy and the k
    best alternatives (log probabilities and ids, ties to the lower id) of every row of logits at a temperature.
    Without targets the logprob entry is 0 in a new result (and new buffers), and not written in a given one."""
    n, v, ld, device = _rows(logits, "logits")
    target = _dense(targets, torch.int32, (n,), "targets", device) if targets is not None else None
    if out is None:
        with _on(stream, logits.device):
            out = _logprobs_out(n, k, logits.device, target is not None)
    if type(out) is Buffers and out.key == ("logprobs", n, k, device):
        lp, lse, ent, top_lp, top_id = out.addresses
    else:
        lp, lse, ent = (_dense(out[name], torch.float32, (n,), name, device) for name in ("logprob", "lse", "entropy"))
        top_lp = _dense(out["top_logprob"], torch.float32, (n, k), "top_logprob", device)
        top_id = _dense(out["top_id"], torch.int32, (n, k), "top_id", device)
    if ws is None:
        with _on(stream, logits.device):
            ws = _ws(gptq_workspace_size(OP_LOGPROBS, None, 1, v, n, max(k, 1)), logits.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_token_logprobs, "gptq_token_logprobs", device, logits.data_ptr(), _DTYPE.get(logits.dtype, -1), n, v,
          ld, target, temperature, k, lp if target is not None else None, lse, ent, top_lp, top_id, at, nbytes,
          _stream_of(stream, device))
    return out


def _distill_out(n: int, v: int, dtype, dev, want_grad: bool) -> Buffers:
    out = {"loss": torch.empty(n, dtype=torch.float32, device=dev)}
    if want_grad:
        out["grad"] = torch.empty(n, v, dtype=dtype, device=dev)
    return Buffers(("distill", n, v if want_grad else 0, dtype, dev.index), out)


def distill_topk_buffers(logits: torch.Tensor, k: int, want_grad: bool = True):
    """(out, ws) of distill_topk calls with these sizes, to be kept from call to call."""
    n, v = logits.shape
    return (_distill_out(n, v, logits.dtype, logits.device, want_grad),
            _ws(gptq_workspace_size(OP_DISTILL, None, 1, v, n, k), logits.device))


def distill_topk(logits: torch.Tensor, top_id: torch.Tensor, top_logprob: torch.Tensor, temperature: float = 1.0,
                 tail: bool = True, weight: Optional[torch.Tensor] = None, want_grad: bool = True,
                 out: Optional[Dict[str, torch.Tensor]] = None, ws: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
    """Loss of every row of the student's logits against the teacher's top list (int32 ids, fp32 log probabilities
    at the same temperature) and, with want_grad, the gradient of sum(weight * loss) in the logits' type.  out may
    hold the logits themselves as "grad": the gradient then replaces them."""
    n, v, ld, device = _rows(logits, "logits")
    dtype = logits.dtype
    k = top_id.shape[-1]
    ids = _dense(top_id, torch.int32, (n, k), "top_id", device)
    lps = _dense(top_logprob, torch.float32, (n, k), "top_logprob", device)
    weights = _dense(weight, torch.float32, (n,), "weight", device) if weight is not None else None
    if out is None:
        with _on(stream, logits.device):
            out = _distill_out(n, v, dtype, logits.device, want_grad)
    ld_g, grad = v, None
    if type(out) is Buffers and out.key == ("distill", n, v if want_grad else 0, dtype, device):
        loss = out.addresses[0]
        if want_grad:
            grad = out.addresses[1]
    else:
        loss = _dense(out["loss"], torch.float32, (n,), "loss", device)
        if want_grad:
            g = out["grad"]
            gn, gv, ld_g, g_device = _rows(g, "grad")
            if g.dtype is not dtype or (gn, gv, g_device) != (n, v, device):
                raise ValueError("grad: the logits' type, shape and device are needed")
            grad = g.data_ptr()
    if ws is None:
        with _on(stream, logits.device):
            ws = _ws(gptq_workspace_size(OP_DISTILL, None, 1, v, n, k), logits.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_distill_topk, "gptq_distill_topk", device, logits.data_ptr(), _DTYPE.get(dtype, -1), n, v, ld, ids,
          lps, k, temperature, bool(tail), weights, loss, grad, ld_g, at, nbytes, _stream_of(stream, device))
    return out


_POLICY = ("loss", "logprob", "ratio", "kl")


def _policy_out(n: int, v: int, dtype, dev, want_grad: bool) -> Buffers:
    out = {name: torch.empty(n, dtype=torch.float32, device=dev) for name in _POLICY}
    if want_grad:
        out["grad"] = torch.empty(n, v, dtype=dtype, device=dev)
    return Buffers(("policy", n, v if want_grad else 0, dtype, dev.index), out)


def policy_loss_buffers(logits: torch.Tensor, want_grad: bool = True):
    """(out, ws) of policy_loss calls with these sizes, to be kept from call to call."""
    n, v = logits.shape
    return (_policy_out(n, v, logits.dtype, logits.device, want_grad),
            _ws(gptq_workspace_size(OP_POLICY, None, 1, v, n, 1), logits.device))


def policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logprob: torch.Tensor, advantage: torch.Tensor,
                ref_logprob: Optional[torch.Tensor] = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, temperature: float = 1.0, weight: Optional[torch.Tensor] = None,
                want_grad: bool = True, out: Optional[Dict[str, torch.Tensor]] = None,
                ws: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Clipped policy loss of every row (answered tokens int32, outside the vocabulary: not scored; fp32 log
    probabilities of the behaviour and the reference at the same temperature, as token_logprobs gives them) with its
    log probability, ratio and KL term, and with want_grad the gradient of sum(weight * loss) in the logits' type.
    out may hold the logits themselves as "grad": the gradient then replaces them."""
    n, v, ld, device = _rows(logits, "logits")
    dtype = logits.dtype
    target = _dense(targets, torch.int32, (n,), "targets", device)
    old = _dense(old_logprob, torch.float32, (n,), "old_logprob", device)
    adv = _dense(advantage, torch.float32, (n,), "advantage", device)
    ref = _dense(ref_logprob, torch.float32, (n,), "ref_logprob", device) if ref_logprob is not None else None
    weights = _dense(weight, torch.float32, (n,), "weight", device) if weight is not None else None
    if out is None:
        with _on(stream, logits.device):
            out = _policy_out(n, v, dtype, logits.device, want_grad)
    ld_g, grad = v, None
    if type(out) is Buffers and out.key == ("policy", n, v if want_grad else 0, dtype, device):
        values = out.addresses[:4]
        if want_grad:
            grad = out.addresses[4]
    else:
        values = [_dense(out[name], torch.float32, (n,), name, device) for name in _POLICY]
        if want_grad:
            grad, ld_g = _out_rows(out["grad"], dtype, n, v, "grad", device)
    if ws is None:
        with _on(stream, logits.device):
            ws = _ws(gptq_workspace_size(OP_POLICY, None, 1, v, n, 1), logits.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_policy_loss, "gptq_policy_loss", device, logits.data_ptr(), _DTYPE.get(dtype, -1), n, v, ld, target,
          old, adv, ref, clip_low, clip_high, kl_coef, temperature, weights, *values, grad, ld_g, at, nbytes,
          _stream_of(stream, device))
    return out


def _adapters(A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor, scale, dtype, M: int, d_in: int, device: int):
    """(adapters, rank, d_out, address of A, B, adapter, scale)."""
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A, B: (adapters, rank, d_in) and (adapters, d_out, rank) are needed")
    n, r, _ = A.shape
    d_out = B.shape[1]
    return (n, r, d_out, _dense(A, dtype, (n, r, d_in), "A", device), _dense(B, dtype, (n, d_out, r), "B", device),
            _dense(adapter, torch.int32, (M,), "adapter", device),
            _dense(scale, torch.float32, (n,), "scale", device) if scale is not None else None)


def _out_rows(t: torch.Tensor, dtype, M: int, d_out: int, what: str, device: int):
    """(address, row stride) of an (M, d_out) tensor."""
    m, w, ld, on = _rows(t, what)
    if t.dtype is not dtype or (m, w, on) != (M, d_out, device):
        raise ValueError(f"{what}: a {dtype} tensor of shape {(M, d_out)} on GPU {device} is needed")
    return t.data_ptr(), ld


def lora_buffers(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, y_dtype=torch.float32):
    """(Y, ws) of lora_add calls with these sizes, to be kept from call to call."""
    M, d_in = X.shape
    d_out, r = B.shape[1], B.shape[2]
    return (torch.empty(M, d_out, dtype=y_dtype, device=X.device),
            _ws(gptq_workspace_size(OP_LORA, None, d_out, d_in, M, r), X.device))


def lora_add(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor,
             scale: Optional[torch.Tensor] = None, base: Optional[torch.Tensor] = None,
             Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[m] = base[m] + scale[a] (X[m] A_a^T) B_a^T, a = adapter[m] (int32; outside the adapters: none).  A is
    (n, rank, d_in), B (n, d_out, rank) in X's type; Y fp32 or X's type, base in Y's type; Y may be base itself."""
    M, d_in, ld_x, device = _rows(X, "X")
    dtype = X.dtype
    n, r, d_out, pa, pb, pad, ps = _adapters(A, B, adapter, scale, dtype, M, d_in, device)
    if Y is None:
        with _on(stream, X.device):
            Y = torch.empty(M, d_out, dtype=base.dtype if base is not None else torch.float32, device=X.device)
    py, ld_y = _out_rows(Y, Y.dtype, M, d_out, "Y", device)
    p0, ld_b = _out_rows(base, Y.dtype, M, d_out, "base", device) if base is not None else (None, d_out)
    if ws is None:
        with _on(stream, X.device):
            ws = _ws(gptq_workspace_size(OP_LORA, None, d_out, d_in, M, r), X.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_lora_add, "gptq_lora_add", device, X.data_ptr(), _DTYPE.get(dtype, -1), M, d_in, ld_x, pa, pb, n, r,
          ps, pad, p0, ld_b, py, _DTYPE.get(Y.dtype, -1), d_out, ld_y, at, nbytes, _stream_of(stream, device))
    return Y


def w4a16_lora_buffers(X: torch.Tensor, A: torch.Tensor, B: torch.Tensor):
    """(Y, ws) of w4a16_lora_matmul calls with these sizes, to be kept from call to call."""
    M, d_in = X.shape
    d_out, r = B.shape[1], B.shape[2]
    return (torch.empty(M, d_out, dtype=torch.float32, device=X.device),
            _ws(gptq_workspace_size(OP_W4A16_LORA, None, d_out, d_in, max(M, 1), r), X.device))


def w4a16_lora_matmul(X: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      group_size: int, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor,
                      scale: Optional[torch.Tensor] = None, perm: Optional[torch.Tensor] = None,
                      Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """w4a16_matmul (up to 64 tokens, or none) plus every token's adapter, as lora_add adds it."""
    M, d_in, ld_x, device = _rows(X, "X")
    dtype = X.dtype
    n, r, d_out, pa, pb, pad, ps = _adapters(A, B, adapter, scale, dtype, M, d_in, device)
    ng = d_in // group_size if group_size > 0 else 0
    pq = _dense(qweight, torch.uint8, (d_out, d_in // 2), "qweight", device)
    if scales.dtype is not torch.int16 and scales.dtype is not torch.float16:
        raise ValueError("scales: fp16, or their bits as int16, are needed")
    psc = _dense(scales, scales.dtype, (d_out, ng), "scales", device)
    pz = _dense(zeros, torch.uint8, (d_out, ng), "zeros", device)
    pp = _dense(perm, torch.int32, (d_in,), "perm", device) if perm is not None else None
    if Y is None:
        with _on(stream, X.device):
            Y = torch.empty(M, d_out, dtype=torch.float32, device=X.device)
    py, ld_y = _out_rows(Y, torch.float32, M, d_out, "Y", device)
    if M == 0:
        return Y
    if ws is None:
        with _on(stream, X.device):
            ws = _ws(gptq_workspace_size(OP_W4A16_LORA, None, d_out, d_in, M, r), X.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_w4a16_lora_matmul, "gptq_w4a16_lora_matmul", device, X.data_ptr(), _DTYPE.get(dtype, -1), M, d_in,
          ld_x, pq, psc, pz, pp, d_out, group_size, pa, pb, n, r, ps, pad, py, ld_y, at, nbytes,
          _stream_of(stream, device))
    return Y


# ---------------------------------------------------------------- 8-bit numbers with block scales
_CODES, _BYTES = torch.float8_e4m3fn, torch.float8_e8m0fnu
F8_BLOCK = 128


def _blocks(n: int) -> int:
    return -(-n // F8_BLOCK)


def _fp8_out(rows: int, cols: int, dev, tiles: bool) -> Buffers:
    nb, rt = _blocks(cols), _blocks(rows)
    out = {"codes": torch.empty(rows, nb * F8_BLOCK, dtype=_CODES, device=dev),
           "scales": torch.empty(rt if tiles else rows, nb, dtype=_BYTES, device=dev)}
    if tiles:
        out["codes_t"] = torch.empty(cols, rt * F8_BLOCK, dtype=_CODES, device=dev)
        out["scales_t"] = torch.empty(nb, rt, dtype=_BYTES, device=dev)
    return Buffers(("fp8", rows, cols, tiles, dev.index), out)


def fp8_quantize_buffers(X: torch.Tensor, tiles: bool = False) -> Buffers:
    """out of fp8_quantize calls with these sizes, to be kept from call to call."""
    return _fp8_out(X.shape[0], X.shape[1], X.device, tiles)


def _codes(t: torch.Tensor, rows: int, cols: int, what: str, device: int):
    """(address, row stride) of a (rows, cols) tensor of codes on 16-byte rows."""
    n, w, ld, on = _rows(t, what)
    if t.dtype is not _CODES or (n, w, on) != (rows, cols, device) or ld % 16 or t.data_ptr() % 16:
        raise ValueError(f"{what}: a {_CODES} tensor of shape {(rows, cols)} with 16-byte aligned rows on GPU {device} "
                         "is needed")
    return t.data_ptr(), ld


def fp8_quantize(X: torch.Tensor, tiles: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
    """e4m3 codes of X's rows, padded with zeros to whole blocks of 128, and a power-of-two scale (E8M0) for each
    block: 128 elements of a row, or with `tiles` (weights) 128 x 128 of them, then with the transpose as
    "codes_t" and "scales_t" (left out of a given `out` without them)."""
    rows, cols, ld_x, device = _rows(X, "X")
    if out is None:
        with _on(stream, X.device):
            out = _fp8_out(rows, cols, X.device, tiles)
    nb, rt = _blocks(cols), _blocks(rows)
    ld_c, ld_ct, codes_t, scales_t = nb * F8_BLOCK, rt * F8_BLOCK, None, None
    if type(out) is Buffers and out.key == ("fp8", rows, cols, tiles, device):
        codes, scales = out.addresses[:2]
        if tiles:
            codes_t, scales_t = out.addresses[2:]
    else:
        codes, ld_c = _codes(out["codes"], rows, nb * F8_BLOCK, "codes", device)
        scales = _dense(out["scales"], _BYTES, (rt if tiles else rows, nb), "scales", device)
        if tiles and "codes_t" in out:
            codes_t, ld_ct = _codes(out["codes_t"], cols, rt * F8_BLOCK, "codes_t", device)
            scales_t = _dense(out["scales_t"], _BYTES, (nb, rt), "scales_t", device)
    _call(lib.gptq_fp8_quantize, "gptq_fp8_quantize", device, X.data_ptr(), _DTYPE.get(X.dtype, -1), rows, cols, ld_x,
          F8_BLOCK if tiles else 1, codes, ld_c, scales, codes_t, ld_ct, scales_t, _stream_of(stream, device))
    return out


def fp8_matmul_buffers(X: torch.Tensor, W: torch.Tensor, y_dtype=torch.float32):
    """(Y, ws) of fp8_matmul calls with these sizes, to be kept from call to call."""
    return (torch.empty(X.shape[0], W.shape[0], dtype=y_dtype, device=X.device),
            _ws(gptq_workspace_size(OP_FP8_MATMUL, None, W.shape[0], X.shape[1], X.shape[0], 1), X.device))


def fp8_matmul(X: torch.Tensor, W: torch.Tensor, w_scales: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
               Y: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, y_dtype=torch.float32,
               stream=None) -> torch.Tensor:
    """Y = X W^T.  W: codes (d_out, d_in padded to whole blocks) with the scales of 128 x 128 tiles.  X: codes with
    x_scales (M, blocks), or fp32, fp16 or bf16 values (M, d_in) that the call quantizes as fp8_quantize does.  Y has
    the type y_dtype unless it is given.  The input's gradient: the same call with the transposed weights."""
    M, d_in, ld_x, device = _rows(X, "X")
    d_out, nb = W.shape[0], _blocks(d_in)
    pw, ld_w = _codes(W, d_out, nb * F8_BLOCK, "W", device)
    psw = _dense(w_scales, _BYTES, (_blocks(d_out), nb), "w_scales", device)
    px, psx, kind = X.data_ptr(), None, _DTYPE.get(X.dtype, -1)
    if X.dtype is _CODES:
        px, ld_x = _codes(X, M, d_in, "X", device)
        if x_scales is None:
            raise ValueError("x_scales: codes need their scales")
        psx, kind = _dense(x_scales, _BYTES, (M, nb), "x_scales", device), E4M3
    elif x_scales is not None:
        raise ValueError("x_scales: only codes have scales")
    if Y is None:
        with _on(stream, X.device):
            Y = torch.empty(M, d_out, dtype=y_dtype, device=X.device)
    py, ld_y = _out_rows(Y, Y.dtype, M, d_out, "Y", device)
    if ws is None:
        with _on(stream, X.device):
            ws = _ws(gptq_workspace_size(OP_FP8_MATMUL, None, d_out, d_in, M, 1), X.device)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_fp8_matmul, "gptq_fp8_matmul", device, px, kind, psx, M, d_in, ld_x, pw, ld_w, psw, d_out, py,
          _DTYPE.get(Y.dtype, -1), ld_y, at, nbytes, _stream_of(stream, device))
    return Y


def _grad_out(A: torch.Tensor, B: torch.Tensor, M: int, dx_dtype) -> Buffers:
    n, r, d_in = A.shape
    out = {"dA": torch.empty(A.shape, dtype=torch.float32, device=A.device),
           "dB": torch.empty(B.shape, dtype=torch.float32, device=A.device)}
    if dx_dtype is not None:
        out["dX"] = torch.empty(M, d_in, dtype=dx_dtype, device=A.device)
    return Buffers(("lora_grad", n, r, d_in, B.shape[1], M if dx_dtype is not None else -1, dx_dtype, A.device.index), out)


def _grad_ws(M: int, A: torch.Tensor, B: torch.Tensor) -> torch.Tensor:
    return _ws(gptq_lora_grad_workspace_size(M, A.shape[2], B.shape[1], A.shape[1], A.shape[0]), A.device)


def lora_grad_buffers(X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor, dx_dtype=None):
    """(out, ws) of lora_grad calls with these sizes, to be kept from call to call; dX of dx_dtype unless it is None."""
    return _grad_out(A, B, X.shape[0], dx_dtype), _grad_ws(X.shape[0], A, B)


def lora_grad(X: torch.Tensor, dY: torch.Tensor, A: torch.Tensor, B: torch.Tensor, adapter: torch.Tensor,
              scale: Optional[torch.Tensor] = None, x_scales: Optional[torch.Tensor] = None,
              base: Optional[torch.Tensor] = None, want_dx: bool = False, out: Optional[Dict[str, torch.Tensor]] = None,
              ws: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients dA, dB (fp32) of lora_add's factors from the gradient dY of its result (A's type or fp32) and, with
    want_dx, a base or an out that has "dX", dX = base + scale[a] (dY B_a) A_a (base's type, else A's).  X: A's type,
    or codes of fp8_quantize with x_scales (an 8-bit checkpoint).  base may be dX itself."""
    dtype = A.dtype
    M, wide, ld_x, device = _rows(X, "X")
    d_in = A.shape[-1]
    n, r, d_out, pa, pb, pad, ps = _adapters(A, B, adapter, scale, dtype, M, d_in, device)
    px, psx, kind = X.data_ptr(), None, _DTYPE.get(X.dtype, -1)
    if X.dtype is _CODES:
        px, ld_x = _codes(X, M, _blocks(d_in) * F8_BLOCK, "X", device)
        if x_scales is None:
            raise ValueError("x_scales: codes need their scales")
        psx, kind = _dense(x_scales, _BYTES, (M, _blocks(d_in)), "x_scales", device), E4M3
    elif wide != d_in or x_scales is not None:
        raise ValueError("X: d_in columns are needed, and only codes have scales")
    py, ld_dy = _out_rows(dY, dY.dtype, M, d_out, "dY", device)
    if out is None:
        dx = base.dtype if base is not None else dtype if want_dx else None
        with _on(stream, X.device):
            out = _grad_out(A, B, M, dx)
    pdx, ld_dx, dx = None, d_in, torch.float32
    has_dx = "dX" in out
    if has_dx:
        dx = out["dX"].dtype
    elif want_dx:
        raise ValueError("want_dx: out has no dX")
    if type(out) is Buffers and out.key == ("lora_grad", n, r, d_in, d_out, M if has_dx else -1, dx if has_dx else None,
                                            device):
        pda, pdb = out.addresses[:2]
        if has_dx:
            pdx = out.addresses[2]
    else:
        pda = _dense(out["dA"], torch.float32, (n, r, d_in), "dA", device)
        pdb = _dense(out["dB"], torch.float32, (n, d_out, r), "dB", device)
        if has_dx:
            pdx, ld_dx = _out_rows(out["dX"], dx, M, d_in, "dX", device)
    if base is not None and not has_dx:
        raise ValueError("base: out has no dX to add it to")
    p0, ld_b = _out_rows(base, dx, M, d_in, "base", device) if base is not None else (None, d_in)
    if ws is None:
        with _on(stream, X.device):
            ws = _grad_ws(M, A, B)
    at, nbytes = _workspace(ws, device)
    _call(lib.gptq_lora_grad, "gptq_lora_grad", device, px, kind, psx, M, d_in, ld_x, py, _DTYPE.get(dY.dtype, -1),
          d_out, ld_dy, pa, pb, _DTYPE.get(dtype, -1), n, r, ps, pad, pda, pdb, p0, ld_b, pdx, _DTYPE.get(dx, -1), ld_dx,
          at, nbytes, _stream_of(stream, device))
    return out


def calibrate_block(chunks: Sequence[torch.Tensor], W1: torch.Tensor, W2: torch.Tensor, params: GptqParams,
                    act: int, stream=None) -> Dict[str, object]:
    """Sequential calibration of y = act(x W1^T) W2^T: layer 1 on the chunks,
    layer 2 on the rounded activations of the quantized layer 1, produced
    chunk by chunk with layer_forward."""
    d_in, h = W1.shape[1], W1.shape[0]
    st1 = HessianState(d_in, 1, W1.device)
    for X in chunks:
        st1.add(X, stream=stream)
    p1 = prepare(st1, params, stream=stream)
    r1 = quantize(W1, p1, params, want_q=True, stream=stream)
    del st1
    Q1 = r1["Q"][0]
    st2 = HessianState(h, 1, W1.device)
    n_max = max(X.shape[0] for X in chunks)
    ws = _ws(gptq_workspace_size(OP_FORWARD, None, h, d_in, n_max, 1), W1.device)
    for X in chunks:
        st2.add(layer_forward(X, Q1, act, ws=ws, stream=stream), stream=stream)
    del ws
    p2 = prepare(st2, params, stream=stream)
    r2 = quantize(W2, p2, params, want_q=True, stream=stream)
    return dict(layer1=r1, layer2=r2, prep1=p1, prep2=p2, state2=st2)
