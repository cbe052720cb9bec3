"""Python binding of the C ABI: same names, torch tensors in, pointers out.

Argument marshalling only: every step of the optimizer runs in the CUDA
library.  Tensors must already live on the current CUDA device; streams are
torch streams (default: the current stream).

The C ABI takes plain pointer arrays and cannot see their lengths or the
tensors behind them, so the binding checks what it marshals: list lengths
against the groups, and each tensor's device, dtype, contiguity and element
count against the layout the library will read and write.  Raw integer
pointers are passed through unchecked.
"""
from __future__ import annotations

import ctypes
import math
from ctypes import c_double, c_float, c_int64, c_void_p
from typing import List, Optional, Sequence, Tuple

import torch

from . import _native as N
from ._native import AdamWGroup, MuonGroup, check

GroupSpec = Tuple[int, int, int, int, int, float]  # rows, cols, count, first, grad_dtype, lr_scale


def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptrs(tensors) -> ctypes.Array:
    arr = (c_void_p * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        arr[i] = t if isinstance(t, int) else t.data_ptr()
    return arr


def _group_fields(s) -> Tuple[int, int, int, int, int]:
    if isinstance(s, MuonGroup):
        return s.rows, s.cols, s.count, s.first, s.grad_dtype
    r, c, n, first, dt, _ = s
    return int(r), int(c), int(n), int(first), int(dt)


def _torch_dtype(code: int):
    return torch.bfloat16 if code == N.MUON_BF16 else torch.float32


def _check_tensor(t, what: str, numel: int, dtype) -> None:
    if isinstance(t, int):
        return
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous() and t.numel() == numel):
        raise ValueError(f"{what}: expected a contiguous CUDA {dtype} tensor of {numel} elements, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}"
                         + ("" if t.is_contiguous() else ", not contiguous"))


def _check_group_lists(groups: Sequence, lists) -> None:
    """lists: (name, tensors, dtype) with dtype None meaning the group's grad dtype."""
    for s in groups:
        r, c, n, first, dt = _group_fields(s)
        if n <= 0 or first < 0:
            continue   # the library rejects the group itself
        for name, seq, dtype in lists:
            if len(seq) < first + n:
                raise ValueError(f"{name}: {len(seq)} entries, the groups index up to {first + n - 1}")
            want = _torch_dtype(dt) if dtype is None else dtype
            for j in range(first, first + n):
                _check_tensor(seq[j], f"{name}[{j}]", r * c, want)


def _check_step_args(groups, params, grads, momentum) -> None:
    _check_group_lists(groups, (("params", params, torch.float32), ("grads", grads, None),
                                ("momentum", momentum, torch.float32)))


def make_groups(specs: Sequence) -> ctypes.Array:
    arr = (MuonGroup * max(len(specs), 1))()
    for i, s in enumerate(specs):
        if isinstance(s, MuonGroup):
            arr[i] = s
        else:
            r, c, n, first, dt, ls = s
            arr[i] = MuonGroup(int(r), int(c), int(n), int(first), int(dt), float(ls))
    return arr


def _coeff_array(coeffs, ns_steps: int):
    if ns_steps == 0:
        return None
    flat: List[float] = []
    if len(coeffs) == 3 and not hasattr(coeffs[0], "__len__"):
        flat = [float(x) for x in coeffs] * ns_steps
    else:
        for row in list(coeffs)[:ns_steps]:
            vals = [float(x) for x in row]
            if len(vals) != 3:
                raise ValueError("coeffs: every row is one (a, b, c) triple")
            flat.extend(vals)
    if len(flat) != 3 * ns_steps:
        raise ValueError(f"coeffs: {len(flat) // 3} rows of (a, b, c) for ns_steps = {ns_steps}")
    arr = (c_float * len(flat))(*flat)
    return arr


def muon_workspace_size(groups: Sequence, flags: int = 0) -> int:
    g = make_groups(groups)
    return int(N.lib().muon_workspace_size(g, len(groups), flags))


def muon_workspace_min_size(groups: Sequence, flags: int = 0) -> int:
    g = make_groups(groups)
    return int(N.lib().muon_workspace_min_size(g, len(groups), flags))


def muon_step(params, grads, momentum, groups: Sequence, lr: float, beta: float, wd: float,
              ns_steps: int, coeffs, flags: int, workspace, workspace_bytes: Optional[int] = None,
              stream=None) -> None:
    """One Muon step; see include/muon_b200.h.  params/grads/momentum are lists
    of tensors (or raw pointers) in pointer-array order."""
    _check_step_args(groups, params, grads, momentum)
    g = make_groups(groups)
    ca = _coeff_array(coeffs, ns_steps)
    wsb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    ws = workspace if isinstance(workspace, int) else workspace.data_ptr()
    st = N.lib().muon_step(_ptrs(params), _ptrs(grads), _ptrs(momentum), g, len(groups),
                           float(lr), float(beta), float(wd), int(ns_steps), ca, int(flags),
                           c_void_p(ws), wsb, c_void_p(_stream_handle(stream)))
    check(st, "muon_step")


def muon_step_replicated(params, grads, momentum, groups: Sequence, lr: float, beta: float, wd: float,
                         ns_steps: int, coeffs, flags: int, workspace, replicas: Sequence[Sequence],
                         workspace_bytes: Optional[int] = None, stream=None) -> None:
    """muon_step that also writes each updated matrix into every replica list
    (replicas[r][i] is copy r of params[i]; tensors or raw device pointers,
    possibly in peer GPUs' memory)."""
    _check_step_args(groups, params, grads, momentum)
    for r, rep in enumerate(replicas):
        _check_group_lists(groups, ((f"replicas[{r}]", rep, torch.float32),))
    g = make_groups(groups)
    ca = _coeff_array(coeffs, ns_steps)
    wsb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    ws = workspace if isinstance(workspace, int) else workspace.data_ptr()
    rows = [_ptrs(rep) for rep in replicas]
    table = (ctypes.POINTER(c_void_p) * max(len(rows), 1))(
        *[ctypes.cast(r, ctypes.POINTER(c_void_p)) for r in rows])
    st = N.lib().muon_step_replicated(_ptrs(params), _ptrs(grads), _ptrs(momentum), g, len(groups),
                                      float(lr), float(beta), float(wd), int(ns_steps), ca, int(flags),
                                      c_void_p(ws), wsb, table, len(rows), c_void_p(_stream_handle(stream)))
    check(st, "muon_step_replicated")


def muon_reduce_mean(dst: Sequence, sources: Sequence[Sequence], stream=None) -> None:
    """dst[i] <- mean over r of sources[r][i] (fp32 or bf16 tensors of one
    dtype; sources may live in peer GPUs' memory)."""
    if not dst:
        return
    if dst[0].dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("muon_reduce_mean: tensors must be fp32 or bf16")
    dt = N.MUON_BF16 if dst[0].dtype == torch.bfloat16 else N.MUON_F32
    for r, src in enumerate(sources):
        if len(src) != len(dst):
            raise ValueError(f"muon_reduce_mean: sources[{r}] has {len(src)} tensors, dst {len(dst)}")
    for i, t in enumerate(dst):
        _check_tensor(t, f"dst[{i}]", t.numel(), dst[0].dtype)
        for r, src in enumerate(sources):
            _check_tensor(src[i], f"sources[{r}][{i}]", t.numel(), dst[0].dtype)
    numel = (c_int64 * len(dst))(*[t.numel() for t in dst])
    rows = [_ptrs(src) for src in sources]
    table = (ctypes.POINTER(c_void_p) * max(len(rows), 1))(
        *[ctypes.cast(r, ctypes.POINTER(c_void_p)) for r in rows])
    st = N.lib().muon_reduce_mean(_ptrs(dst), table, len(rows), numel, len(dst), dt,
                                  c_void_p(_stream_handle(stream)))
    check(st, "muon_reduce_mean")


def muon_step_scheduled(params, grads, momentum, groups: Sequence, lr: float, beta: float, wd: float,
                        ns_steps: int, coeffs, flags: int, workspace, schedule_state,
                        workspace_bytes: Optional[int] = None, stream=None) -> None:
    """muon_step with the learning rate multiplied by the device schedule
    state's lr_mult (schedule_state: a 16-byte device tensor, see
    new_schedule_state)."""
    _check_step_args(groups, params, grads, momentum)
    g = make_groups(groups)
    ca = _coeff_array(coeffs, ns_steps)
    wsb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    ws = workspace if isinstance(workspace, int) else workspace.data_ptr()
    st = N.lib().muon_step_scheduled(_ptrs(params), _ptrs(grads), _ptrs(momentum), g, len(groups),
                                     float(lr), float(beta), float(wd), int(ns_steps), ca, int(flags),
                                     c_void_p(ws), wsb, c_void_p(schedule_state.data_ptr()),
                                     c_void_p(_stream_handle(stream)))
    check(st, "muon_step_scheduled")


def new_schedule_state(device, lr_mult: float = 1.0, step: int = 0):
    """A device-resident schedule state {float lr_mult; float reserved; int64 step}."""
    import struct
    raw = struct.pack("<ffq", float(lr_mult), 0.0, int(step))
    return torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(device)


def read_schedule_state(state):
    import struct
    lr_mult, _, step = struct.unpack("<ffq", bytes(state.cpu().numpy().tobytes()))
    return lr_mult, step


def muon_schedule_advance(schedule_state, total_steps: int, warmup_frac: float = 0.1,
                          warmdown_frac: float = 0.2, final_frac: float = 0.1, stream=None) -> None:
    st = N.lib().muon_schedule_advance(c_void_p(schedule_state.data_ptr()), int(total_steps),
                                       float(warmup_frac), float(warmdown_frac), float(final_frac),
                                       c_void_p(_stream_handle(stream)))
    check(st, "muon_schedule_advance")


def muon_schedule_advance_cosine(schedule_state, total_steps: int, warmup_steps: int,
                                 final_frac: float = 0.1, stream=None) -> None:
    st = N.lib().muon_schedule_advance_cosine(c_void_p(schedule_state.data_ptr()), int(total_steps),
                                              int(warmup_steps), float(final_frac),
                                              c_void_p(_stream_handle(stream)))
    check(st, "muon_schedule_advance_cosine")


def muon_orthogonalize(inputs, outputs, groups: Sequence, ns_steps: int, coeffs, flags: int,
                       workspace, workspace_bytes: Optional[int] = None, stream=None) -> None:
    _check_group_lists(groups, (("inputs", inputs, None), ("outputs", outputs, torch.float32)))
    g = make_groups(groups)
    ca = _coeff_array(coeffs, ns_steps)
    wsb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    ws = workspace if isinstance(workspace, int) else workspace.data_ptr()
    st = N.lib().muon_orthogonalize(_ptrs(inputs), _ptrs(outputs), g, len(groups), int(ns_steps), ca,
                                    int(flags), c_void_p(ws), wsb, c_void_p(_stream_handle(stream)))
    check(st, "muon_orthogonalize")


class AdamWSpec:
    """One AdamW group: lists of tensors plus hyperparameters."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, lr, beta1, beta2, eps, wd,
                 grad_dtype: Optional[int] = None):
        self.params, self.grads, self.exp_avg, self.exp_avg_sq = params, grads, exp_avg, exp_avg_sq
        self.lr, self.beta1, self.beta2, self.eps, self.wd = lr, beta1, beta2, eps, wd
        if grad_dtype is None:
            grad_dtype = N.MUON_BF16 if (grads and grads[0].dtype == torch.bfloat16) else N.MUON_F32
        self.grad_dtype = grad_dtype


def _adamw_groups(groups: Sequence[AdamWSpec]):
    n = len(groups)
    arr = (AdamWGroup * max(n, 1))()
    keep = []
    for i, g in enumerate(groups):
        n_t = len(g.params)
        for name in ("grads", "exp_avg", "exp_avg_sq"):
            if len(getattr(g, name)) != n_t:
                raise ValueError(f"AdamW group {i}: {len(getattr(g, name))} {name} for {n_t} params")
        for k, t in enumerate(g.params):
            ne = t.numel()
            _check_tensor(t, f"AdamW group {i} params[{k}]", ne, torch.float32)
            _check_tensor(g.grads[k], f"AdamW group {i} grads[{k}]", ne, _torch_dtype(int(g.grad_dtype)))
            _check_tensor(g.exp_avg[k], f"AdamW group {i} exp_avg[{k}]", ne, torch.float32)
            _check_tensor(g.exp_avg_sq[k], f"AdamW group {i} exp_avg_sq[{k}]", ne, torch.float32)
        p, gr, m, v = _ptrs(g.params), _ptrs(g.grads), _ptrs(g.exp_avg), _ptrs(g.exp_avg_sq)
        numel = (c_int64 * max(len(g.params), 1))(*[t.numel() for t in g.params])
        keep.extend([p, gr, m, v, numel])
        arr[i] = AdamWGroup(ctypes.cast(p, ctypes.POINTER(c_void_p)),
                            ctypes.cast(gr, ctypes.POINTER(c_void_p)),
                            ctypes.cast(m, ctypes.POINTER(c_void_p)),
                            ctypes.cast(v, ctypes.POINTER(c_void_p)),
                            numel, len(g.params), int(g.grad_dtype), float(g.lr), float(g.beta1),
                            float(g.beta2), float(g.eps), float(g.wd))
    return arr, keep


class AdamWArgs:
    """AdamW groups (AdamWSpecs) checked and laid out for the library, for an
    adamw_step that follows."""

    def __init__(self, groups: Sequence[AdamWSpec]):
        self.groups, self._keep = _adamw_groups(groups)
        self._tensors = list(groups)   # the pointers' owners
        self.count = len(groups)


def adamw_step(groups, step: int, stream=None) -> None:
    """One AdamW step of the groups (AdamWSpecs, or AdamWArgs)."""
    a = groups if isinstance(groups, AdamWArgs) else AdamWArgs(groups)
    st = N.lib().adamw_step(a.groups, a.count, int(step), c_void_p(_stream_handle(stream)))
    check(st, "adamw_step")


def adamw_step_scheduled(groups: Sequence[AdamWSpec], schedule_state, stream=None) -> None:
    """adamw_step with lr * lr_mult and t = step read from the device schedule state."""
    arr, keep = _adamw_groups(groups)
    st = N.lib().adamw_step_scheduled(arr, len(groups), c_void_p(schedule_state.data_ptr()),
                                      c_void_p(_stream_handle(stream)))
    check(st, "adamw_step_scheduled")


# ------------------------------------------- operators that make the gradients
# These run many times a step, some for a few microseconds, so their checks are
# kept short: one device index per tensor, no device switch where the tensors'
# device is the current one, shapes walked only where a tensor is strided.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_DTYPE = {torch.float32: N.MUON_F32, torch.bfloat16: N.MUON_BF16}


def _device_of(fn: str, names: str, *tensors) -> int:
    """The one CUDA device of the tensors (names: theirs, in order); None is skipped."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            bad = names.split()[next(i for i, x in enumerate(tensors)
                                     if x is not None and (x.get_device() < 0 or x.get_device() != dev))]
            where = [f"{n} on {x.device}" for n, x in zip(names.split(), tensors) if x is not None]
            if any(x is not None and x.get_device() < 0 for x in tensors):
                raise ValueError(f"{fn}: {bad} is not a CUDA tensor, or the others are not ({', '.join(where)})")
            raise ValueError(f"{fn}: {bad} is on another device ({', '.join(where)})")
    return dev


def _launch(fn: str, dev: int, stream, call, *args) -> None:
    """call(*args, stream) with the tensors' device current, on `stream` or
    that device's current stream."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"{fn}: stream of {stream.device}, tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    if _current_device() == dev:
        st = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = call(*args, handle)
    if st != N.MUON_OK:
        check(st, fn)


def _dtype_code(fn: str, name: str, t) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{fn}: {name} must be fp32 or bf16, got {t.dtype}")
    return code


def _rows(fn: str, name: str, t, cols: Optional[int] = None, rows: Optional[int] = None):
    """(rows, columns, pitch) of an activation tensor [..., columns]: rows of
    adjacent elements a constant pitch apart."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{fn}: {name} has no dimension")
    c = shape[-1]
    r = shape[0] if len(shape) == 2 else math.prod(shape[:-1])
    if (cols is not None and c != cols) or (rows is not None and r != rows):
        raise ValueError(f"{fn}: {name} {tuple(shape)} is not {'*' if rows is None else rows} rows of "
                         f"{'*' if cols is None else cols}")
    if t.is_contiguous():
        return r, c, c
    if c > 1 and t.stride(-1) != 1:
        raise ValueError(f"{fn}: the elements of a row of {name} are not adjacent")
    pitch, span = None, 1   # leading dimensions, innermost first, must step evenly through the rows
    for size, stride in list(zip(shape[:-1], t.stride()[:-1]))[::-1]:
        if size == 1:
            continue
        if pitch is None:
            pitch = stride
        elif stride != pitch * span:
            raise ValueError(f"{fn}: the rows of {name} are not a constant pitch apart")
        span *= size
    if pitch is None or r == 0:
        pitch = c
    if pitch < c:
        raise ValueError(f"{fn}: the rows of {name} overlap")
    return r, c, pitch


def _dense(fn: str, name: str, t, numel: int, last: int, dtype=None) -> None:
    """A contiguous tensor of numel elements, rows of `last`."""
    if t.numel() != numel or t.shape[-1:] != (last,) or not t.is_contiguous() or \
            (dtype is not None and t.dtype is not dtype):
        raise ValueError(f"{fn}: {name} must be contiguous{'' if dtype is None else f' {dtype}'}, {numel} elements in "
                         f"rows of {last}, got {t.dtype} {tuple(t.shape)}")


def _row_values(fn: str, name: str, t, rows: int) -> None:
    if t.numel() != rows or t.dtype is not torch.float32 or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be contiguous fp32, one value for each of {rows} rows, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _ids(fn: str, ids):
    d = ids.dtype
    if (d is not torch.int64 and d is not torch.int32) or not ids.is_contiguous():
        raise ValueError(f"{fn}: ids must be a contiguous int32 or int64 tensor")
    return (64 if d is torch.int64 else 32), ids.numel()


def _table(fn: str, name: str, t):
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous [vocab, dim] tensor, got {tuple(t.shape)}")
    return t.shape


def _workspace(fn: str, ws) -> int:
    if not ws.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous")
    return ws.numel() * ws.element_size()


def muon_embedding_forward(table, ids, out, scale: float = 1.0, stream=None) -> None:
    """out[t] <- scale * table[ids[t]]; zeros where ids[t] is outside
    [0, vocab).  table: fp32 or bf16 [vocab, dim]; ids: int32 or int64, any
    shape; out: fp32 or bf16 [*ids.shape, dim] (rows may be strided)."""
    fn = "muon_embedding_forward"
    dev = _device_of(fn, "table ids out", table, ids, out)
    vocab, dim = _table(fn, "table", table)
    bits, n = _ids(fn, ids)
    _, _, pitch = _rows(fn, "out", out, dim, n)
    _launch(fn, dev, stream, N.lib().muon_embedding_forward, table.data_ptr(), _dtype_code(fn, "table", table), vocab,
            dim, ids.data_ptr(), bits, n, scale, out.data_ptr(), _dtype_code(fn, "out", out), pitch)


def muon_embedding_grad_workspace_size(vocab: int, dim: int, n: int) -> int:
    return int(N.lib().muon_embedding_grad_workspace_size(int(vocab), int(dim), int(n)))


def muon_embedding_grad(dout, ids, grad, workspace, scale: float = 1.0, accumulate: bool = False,
                        stream=None) -> None:
    """grad[v] <- (grad[v] +) scale * sum of dout[t] over t with ids[t] = v.
    dout: fp32 or bf16 [*ids.shape, dim]; grad: fp32 or bf16 [vocab, dim]."""
    fn = "muon_embedding_grad"
    dev = _device_of(fn, "dout ids grad workspace", dout, ids, grad, workspace)
    vocab, dim = _table(fn, "grad", grad)
    bits, n = _ids(fn, ids)
    _, _, pitch = _rows(fn, "dout", dout, dim, n)
    _launch(fn, dev, stream, N.lib().muon_embedding_grad, dout.data_ptr(), _dtype_code(fn, "dout", dout), pitch,
            ids.data_ptr(), bits, n, vocab, dim, scale, grad.data_ptr(), _dtype_code(fn, "grad", grad),
            1 if accumulate else 0, workspace.data_ptr(), _workspace(fn, workspace))


def muon_layer_norm_forward(x, gain, bias, y, mean, rstd, eps: float = 1e-5, stream=None) -> None:
    """y <- (x - mean) * rstd * gain + bias over the last dimension; mean and
    rstd (fp32, one per row) are written for the backward pass.  x, y: fp32 or
    bf16; gain, bias: fp32 [cols] (bias may be None)."""
    fn = "muon_layer_norm_forward"
    dev = _device_of(fn, "x gain bias y mean rstd", x, gain, bias, y, mean, rstd)
    rows, cols, xp = _rows(fn, "x", x)
    _, _, yp = _rows(fn, "y", y, cols, rows)
    _dense(fn, "gain", gain, cols, cols, torch.float32)
    if bias is not None:
        _dense(fn, "bias", bias, cols, cols, torch.float32)
    _row_values(fn, "mean", mean, rows)
    _row_values(fn, "rstd", rstd, rows)
    _launch(fn, dev, stream, N.lib().muon_layer_norm_forward, x.data_ptr(), _dtype_code(fn, "x", x), xp, rows, cols,
            gain.data_ptr(), None if bias is None else bias.data_ptr(), eps, y.data_ptr(), _dtype_code(fn, "y", y), yp,
            mean.data_ptr(), rstd.data_ptr())


def muon_layer_norm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(N.lib().muon_layer_norm_backward_workspace_size(int(rows), int(cols)))


def muon_layer_norm_backward(dy, x, gain, mean, rstd, dx, dgain, dbias, workspace, accumulate: bool = False,
                             stream=None) -> None:
    """The gradients of muon_layer_norm_forward: dx (the type of x and dy),
    and dgain and dbias (fp32 or bf16 [cols]; dbias may be None), overwritten
    or added to."""
    fn = "muon_layer_norm_backward"
    dev = _device_of(fn, "dy x gain mean rstd dx dgain dbias workspace", dy, x, gain, mean, rstd, dx, dgain, dbias, workspace)
    rows, cols, xp = _rows(fn, "x", x)
    _, _, dyp = _rows(fn, "dy", dy, cols, rows)
    _, _, dxp = _rows(fn, "dx", dx, cols, rows)
    if not (dy.dtype is x.dtype and dx.dtype is x.dtype):
        raise ValueError(f"{fn}: dy, x and dx must have one type, got {dy.dtype}, {x.dtype}, {dx.dtype}")
    _dense(fn, "gain", gain, cols, cols, torch.float32)
    _row_values(fn, "mean", mean, rows)
    _row_values(fn, "rstd", rstd, rows)
    _dense(fn, "dgain", dgain, cols, cols)
    if dbias is not None:
        _dense(fn, "dbias", dbias, cols, cols, dgain.dtype)
    _launch(fn, dev, stream, N.lib().muon_layer_norm_backward, dy.data_ptr(), dyp, x.data_ptr(),
            _dtype_code(fn, "x", x), xp, rows, cols, gain.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(),
            dxp, dgain.data_ptr(), None if dbias is None else dbias.data_ptr(), _dtype_code(fn, "dgain", dgain),
            1 if accumulate else 0, workspace.data_ptr(), _workspace(fn, workspace))


CHECKPOINT_BLOCK = 128   # features that share one exponent of a checkpoint


class Checkpoint:
    """Activations [rows, cols] kept in 8 bits: codes, uint8 [rows, pitch]
    (8-bit floats, 4 exponent and 3 mantissa bits; pitch a multiple of 16, at
    least cols), and exponents, uint8 [rows, ceil(cols / 128)]."""

    def __init__(self, codes, exponents, cols: int):
        cols = int(cols)
        nb = (cols + CHECKPOINT_BLOCK - 1) // CHECKPOINT_BLOCK
        if codes.dim() != 2 or codes.dtype != torch.uint8 or not codes.is_contiguous() or codes.shape[1] < cols \
                or codes.shape[1] % 16 != 0 or cols < 1:
            raise ValueError("Checkpoint: codes must be contiguous uint8 [rows, pitch], pitch a multiple of 16 and "
                             f"at least cols = {cols}, got {codes.dtype} {tuple(codes.shape)}")
        _dense("Checkpoint", "exponents", exponents, codes.shape[0] * nb, nb, torch.uint8)
        self.codes, self.exponents, self.cols = codes, exponents, cols

    @property
    def rows(self) -> int:
        return self.codes.shape[0]


def new_checkpoint(rows: int, cols: int, device) -> Checkpoint:
    """An uninitialised checkpoint for muon_checkpoint_pack to fill."""
    pitch = (int(cols) + 15) // 16 * 16
    nb = (int(cols) + CHECKPOINT_BLOCK - 1) // CHECKPOINT_BLOCK
    return Checkpoint(torch.empty(int(rows), pitch, dtype=torch.uint8, device=device),
                      torch.empty(int(rows), nb, dtype=torch.uint8, device=device), cols)


def muon_checkpoint_pack(x, ckpt: Checkpoint, stream=None) -> None:
    """Fill ckpt from x, fp32 or bf16 [..., cols] (rows may be strided)."""
    fn = "muon_checkpoint_pack"
    codes, exps = ckpt.codes, ckpt.exponents
    dev = _device_of(fn, "x codes exponents", x, codes, exps)
    rows, cols, pitch = _rows(fn, "x", x, ckpt.cols, codes.shape[0])
    _launch(fn, dev, stream, N.lib().muon_checkpoint_pack, x.data_ptr(), _dtype_code(fn, "x", x), pitch, rows, cols,
            codes.data_ptr(), codes.shape[1], exps.data_ptr())


def muon_checkpoint_unpack(ckpt: Checkpoint, out, stream=None) -> None:
    """out <- the values the checkpoint stands for (fp32 or bf16, both exact)."""
    fn = "muon_checkpoint_unpack"
    codes, exps = ckpt.codes, ckpt.exponents
    dev = _device_of(fn, "codes exponents out", codes, exps, out)
    rows, cols, pitch = _rows(fn, "out", out, ckpt.cols, codes.shape[0])
    _launch(fn, dev, stream, N.lib().muon_checkpoint_unpack, codes.data_ptr(), codes.shape[1], exps.data_ptr(), rows,
            cols, out.data_ptr(), _dtype_code(fn, "out", out), pitch)


def muon_checkpoint_weight_grad_workspace_size(rows: int, n: int, k: int, dy_dtype, dy_aligned: bool = True) -> int:
    """dy_dtype: torch.float32 or torch.bfloat16.  dy_aligned=False also counts
    the copy of a bf16 dy whose pointer or row pitch is not a multiple of 16
    bytes."""
    code = {torch.float32: N.MUON_F32, torch.bfloat16: N.MUON_BF16}.get(dy_dtype, -1)
    return int(N.lib().muon_checkpoint_weight_grad_workspace_size(int(rows), int(n), int(k), code,
                                                                   1 if dy_aligned else 0))


def muon_checkpoint_weight_grad(dy, ckpt: Checkpoint, grad, workspace, accumulate: bool = False,
                                stream=None) -> None:
    """grad [n, k] <- (grad +) dy^T x: the gradient of W [n, k] in y = x W^T from
    dy (fp32 or bf16 [..., n]) and the checkpoint of x [rows, k]."""
    fn = "muon_checkpoint_weight_grad"
    codes, exps = ckpt.codes, ckpt.exponents
    dev = _device_of(fn, "dy codes exponents grad workspace", dy, codes, exps, grad, workspace)
    rows, n, pitch = _rows(fn, "dy", dy, None, codes.shape[0])
    _dense(fn, "grad", grad, n * ckpt.cols, ckpt.cols)
    _launch(fn, dev, stream, N.lib().muon_checkpoint_weight_grad, dy.data_ptr(), _dtype_code(fn, "dy", dy), pitch, rows,
            n, codes.data_ptr(), codes.shape[1], exps.data_ptr(), ckpt.cols, grad.data_ptr(),
            _dtype_code(fn, "grad", grad), 1 if accumulate else 0, workspace.data_ptr(), _workspace(fn, workspace))


class LinearGrad:
    """The gradient of a hidden matrix W [n, k] (y = x W^T) by its factors: dy
    [..., n] and the checkpoint of x.  MuonAdamW.step takes it in a gradient's
    place and forms the gradient itself."""

    def __init__(self, dy, checkpoint: Checkpoint):
        self.dy, self.checkpoint = dy, checkpoint

    def workspace_size(self, grad) -> int:
        dy = self.dy
        es = dy.element_size()
        aligned = dy.data_ptr() % 16 == 0 and all(st * es % 16 == 0 for st in dy.stride()[:-1])
        return muon_checkpoint_weight_grad_workspace_size(self.checkpoint.rows, grad.shape[0], grad.shape[1], dy.dtype,
                                                          aligned)

    def write(self, grad, workspace, accumulate: bool = False, stream=None) -> None:
        muon_checkpoint_weight_grad(self.dy, self.checkpoint, grad, workspace, accumulate=accumulate, stream=stream)


class EmbeddingGrad:
    """The gradient of an embedding table by its factors: dout [..., dim], the
    token ids and the lookup's scale.  MuonAdamW.step takes it in a gradient's
    place and forms the gradient itself."""

    def __init__(self, dout, ids, scale: float = 1.0):
        self.dout, self.ids, self.scale = dout, ids, scale

    def workspace_size(self, grad) -> int:
        return muon_embedding_grad_workspace_size(grad.shape[0], grad.shape[1], self.ids.numel())

    def write(self, grad, workspace, accumulate: bool = False, stream=None) -> None:
        muon_embedding_grad(self.dout, self.ids, grad, workspace, scale=self.scale, accumulate=accumulate,
                            stream=stream)


def muon_query_status(workspace, stream=None) -> int:
    ws = workspace if isinstance(workspace, int) else workspace.data_ptr()
    return int(N.lib().muon_query_status(c_void_p(ws), c_void_p(_stream_handle(stream))))


def adamw_query_status(stream=None) -> int:
    """MUON_ERR_TIMEOUT if a bounded wait in an AdamW kernel on this device ran
    out since the last call (the record is then cleared), else MUON_OK."""
    return int(N.lib().adamw_query_status(c_void_p(_stream_handle(stream))))


# --------------------------------------------------------------- profiler
def muon_profiler_enable(on: bool) -> bool:
    return bool(N.lib().muon_profiler_enable(1 if on else 0))


def muon_profiler_reset() -> None:
    N.lib().muon_profiler_reset()


def muon_profiler_read() -> dict:
    """{kernel kind: (device ms summed, launches)} since the last reset."""
    L = N.lib()
    k = L.muon_kernel_kind_count()
    ms = (c_double * k)()
    cnt = (c_int64 * k)()
    L.muon_profiler_read(ms, cnt, k)
    return {L.muon_kernel_kind_name(i).decode(): (ms[i], int(cnt[i])) for i in range(k)}
