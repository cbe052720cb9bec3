"""MuonAdamW: the hybrid optimizer over two disjoint parameter sets.

Hidden 2-D weight matrices go to Muon; embeddings, the LM head, norm gains
and biases go to AdamW ("Chapter 4: The MuonAdamW Optimizer", Parameter
Dispatch; "3.9 Optimizers", Wiring the hybrid recipe).  The caller decides
the split.  This class only owns the state tensors (momentum, exp_avg,
exp_avg_sq, the step count), groups matrices by shape, and calls the C ABI;
all arithmetic runs in the CUDA library.
"""
from __future__ import annotations

import contextlib
from typing import Dict, List, Optional, Sequence

import torch

from . import _native as N
from . import api

DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)


class MuonAdamW:
    def __init__(self, muon_params: Sequence[torch.Tensor], adamw_groups: Sequence[Dict] = (),
                 lr: float = 0.02, momentum: float = 0.95, weight_decay: float = 0.01,
                 ns_steps: int = 5, coeffs=DEFAULT_COEFFS, nesterov: bool = True,
                 cautious: bool = True, lr_scale_fn=None, fp32_debug: bool = False,
                 fused_update: bool = True, normuon: bool = False, row_equilibrate: bool = False,
                 workspace_bytes: Optional[int] = None):
        """muon_params: fp32 2-D CUDA tensors.  adamw_groups: dicts with keys
        params, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.  lr_scale_fn:
        optional (rows, cols) -> float learning-rate multiplier per shape.
        normuon: row-normalise the orthogonalised update (NorMuon).
        row_equilibrate: row-equilibrate the momentum-smoothed matrix before
        the orthogonalisation (MuonEq)."""
        self.lr, self.beta, self.wd = lr, momentum, weight_decay
        self.ns_steps, self.coeffs = ns_steps, coeffs
        self.flags = ((N.MUON_NESTEROV if nesterov else 0) | (N.MUON_CAUTIOUS_WD if cautious else 0)
                      | (N.MUON_FP32_DEBUG if fp32_debug else 0)
                      | (0 if fused_update else N.MUON_UNFUSED_UPDATE)
                      | (N.MUON_NORMUON if normuon else 0)
                      | (N.MUON_ROW_EQUILIBRATE if row_equilibrate else 0))
        # shape groups: matrices with equal (rows, cols) are contiguous in the pointer arrays
        muon_params = list(muon_params)
        order: Dict[tuple, List[int]] = {}
        for k, p in enumerate(muon_params):
            if p.dim() != 2 or p.dtype != torch.float32 or not p.is_cuda or not p.is_contiguous():
                raise ValueError("Muon parameters must be contiguous fp32 2-D CUDA tensors")
            order.setdefault(tuple(p.shape), []).append(k)
        self.muon_params: List[torch.Tensor] = []
        self._order: List[int] = []   # internal position -> position in muon_params as given
        self._shapes = []
        for (r, c), ks in order.items():
            self._shapes.append((r, c, len(ks), len(self.muon_params),
                                 float(lr_scale_fn(r, c)) if lr_scale_fn else 1.0))
            self.muon_params.extend(muon_params[k] for k in ks)
            self._order.extend(ks)
        self.momentum = [torch.zeros_like(p) for p in self.muon_params]
        self.adamw_groups = []
        for g in adamw_groups:
            ps = list(g["params"])
            self.adamw_groups.append(dict(
                params=ps, lr=g.get("lr", 3e-4), betas=g.get("betas", (0.9, 0.95)),
                eps=g.get("eps", 1e-8), weight_decay=g.get("weight_decay", 0.0),
                exp_avg=[torch.zeros_like(p) for p in ps],
                exp_avg_sq=[torch.zeros_like(p) for p in ps]))
        self.step_count = 0
        ws_need = api.muon_workspace_size(self._groups([torch.float32] * len(self._shapes)), self.flags) \
            if self.muon_params else 0
        nbytes = ws_need if workspace_bytes is None else max(int(workspace_bytes), 0)
        dev = self.muon_params[0].device if self.muon_params else torch.device("cuda")
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        self.workspace[:256].zero_()   # its status word, before the first step writes it
        self._factor_workspace: Optional[torch.Tensor] = None   # grown by the gradients formed here
        self._captured_workspaces: List[torch.Tensor] = []        # those that a captured step writes when replayed
        self._factor_status = torch.zeros(1, dtype=torch.int32, device=dev)   # their status words together

    def _groups(self, grad_dtypes):
        """Group descriptors, one gradient dtype per shape group."""
        return [(r, c, n, first, N.MUON_BF16 if dt == torch.bfloat16 else N.MUON_F32, ls)
                for (r, c, n, first, ls), dt in zip(self._shapes, grad_dtypes)]

    def _grad_dtypes(self, grads):
        """The gradient dtype of each shape group (fp32 or bf16, uniform within a group)."""
        out = []
        for (r, c, n, first, _) in self._shapes:
            dts = {grads[k].dtype for k in range(first, first + n)}
            if len(dts) != 1 or not dts <= {torch.float32, torch.bfloat16}:
                raise ValueError(f"the grads of the {r}x{c} Muon matrices must all be fp32 or all bf16")
            out.append(dts.pop())
        return out

    @staticmethod
    def _factors(param: torch.Tensor, grad):
        """The factors a gradient is given by, one per micro-batch; None for a tensor."""
        if isinstance(grad, torch.Tensor):
            return None
        parts = list(grad) if isinstance(grad, (list, tuple)) else [grad]
        if not parts or not all(isinstance(f, (api.LinearGrad, api.EmbeddingGrad)) for f in parts):
            raise ValueError("a gradient is a tensor, a LinearGrad or EmbeddingGrad, or a list of these")
        if param.dim() != 2:
            raise ValueError(f"a gradient given by its factors is a matrix, its parameter is {tuple(param.shape)}")
        return parts

    def _reserve(self, need: int, device) -> None:
        """A factor workspace of at least `need` bytes, allocated on the current stream."""
        ws = self._factor_workspace
        if ws is None or ws.numel() < need:
            if ws is not None and ws.is_cuda:   # steps before this one may still be using it, on any stream
                ws.record_stream(torch.cuda.current_stream(ws.device))
            ws = self._factor_workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
        if torch.cuda.is_current_stream_capturing() and not any(w is ws for w in self._captured_workspaces):
            self._captured_workspaces.append(ws)

    def _formed(self, param: torch.Tensor, grad, stream, first: int = 0):
        """The gradient tensor of one parameter: `grad` itself, or, where it is
        given by its factors (api.LinearGrad, api.EmbeddingGrad, or a list of
        them, one per micro-batch), their sum, formed in param.grad (allocated
        in param.grad_dtype, else fp32, where there is none).

        first: factors formed before these in the same step.  Every call has its
        status word at the start of its workspace and clears it, so factor i of
        a step takes the workspace from 256 i on: its word, and below it those
        of the factors before, which no later one touches."""
        parts = MuonAdamW._factors(param, grad)
        if parts is None:
            return grad
        fresh = param.grad is None
        try:
            # allocated on the stream that writes them, so that memory freed on
            # another stream is not reused while it is still read there
            with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                if fresh:
                    param.grad = torch.empty_like(param, dtype=getattr(param, "grad_dtype", None) or torch.float32,
                                                  requires_grad=False)
                MuonAdamW._reserve(self, max(256 * (first + k) + f.workspace_size(param) for k, f in enumerate(parts)),
                                   param.device)
            for k, f in enumerate(parts):
                f.write(param.grad, self._factor_workspace[256 * (first + k):], accumulate=k > 0, stream=stream)
        except Exception:
            if fresh:   # not a gradient: not all of it has been written
                param.grad = None
            raise
        return param.grad

    def _form_all(self, params: Sequence[torch.Tensor], grads: Sequence, stream) -> List[torch.Tensor]:
        """The gradient tensors of all parameters; the status words of what is
        formed here go into _factor_status."""
        if all(isinstance(x, torch.Tensor) for x in grads):
            return list(grads)
        parts = [self._factors(p, x) or [] for p, x in zip(params, grads)]
        sizes = [f.workspace_size(p) for p, fs in zip(params, parts) for f in fs]
        on_stream = lambda: torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()
        with on_stream():   # the whole step's, so that no word is lost to a larger workspace halfway
            self._reserve(max(256 * i + n for i, n in enumerate(sizes)), self._factor_status.device)
        out, first = [], 0
        for p, x, fs in zip(params, grads, parts):
            out.append(self._formed(p, x, stream, first))
            first += len(fs)
        with on_stream():
            words = self._factor_workspace[:256 * first].view(torch.int32).view(first, 64)[:, 0]
            self._factor_status.bitwise_or_(words.amax())
        return out

    def query_status(self, stream=None) -> int:
        """MUON_ERR_TIMEOUT where a bounded wait on the device ran out: in the
        last Muon step, or, since the last call (the record is then cleared), in
        an AdamW step on this device or in a gradient that a step formed from
        its factors; else MUON_OK.  Synchronises `stream` (default: the current
        one), which must be the steps' or ordered after it."""
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            formed = N.MUON_ERR_TIMEOUT if int(self._factor_status.item()) != 0 else N.MUON_OK
            if formed != N.MUON_OK:
                self._factor_status.zero_()
        return next((st for st in (formed, api.muon_query_status(self.workspace, stream),
                                   api.adamw_query_status(stream)) if st != N.MUON_OK), N.MUON_OK)

    @torch.no_grad()
    def step(self, stream=None, replicas: Optional[Sequence[Sequence[torch.Tensor]]] = None,
             muon_grads: Optional[Sequence[torch.Tensor]] = None,
             adamw_grads: Optional[Sequence[Sequence[torch.Tensor]]] = None) -> None:
        """One MuonAdamW step.  replicas: optional copies of the Muon
        parameters (replicas[r][k] is copy r of the k-th tensor given at
        construction, e.g. another data-parallel rank's replica in peer
        memory); each receives the updated values (muon_step_replicated).
        muon_grads / adamw_grads: the gradients to use instead of each
        parameter's .grad (muon_grads[k] for the k-th Muon tensor given at
        construction, adamw_grads[g][j] for tensor j of AdamW group g).  A
        gradient may be given by its factors (api.LinearGrad for a hidden
        matrix whose input was kept as an 8-bit checkpoint, api.EmbeddingGrad
        for an embedding table, or a list of them, one per micro-batch): the
        step then forms it in the parameter's .grad, from nothing.  A gradient
        that is refused, in either list, is refused before any parameter or
        state has changed (gradients formed by then stay in their .grad).  Waits
        on the device are bounded; query_status says whether one ran out."""
        def given(params, of_call, wrong_length: str, missing: str) -> List:
            """What stands for each parameter's gradient, lengths and types checked."""
            if of_call is None:
                of_call = [p.grad for p in params]
            if len(of_call) != len(params):
                raise ValueError(wrong_length)
            for p, x in zip(params, of_call):
                if x is None:
                    raise ValueError(missing)
                if not isinstance(x, torch.Tensor):
                    self._factors(p, x)
            return list(of_call)

        grads: List = []
        if self.muon_params:
            if muon_grads is not None and len(muon_grads) == len(self._order):
                muon_grads = [muon_grads[k] for k in self._order]
            grads = given(self.muon_params, muon_grads, "muon_grads must hold one gradient per Muon parameter",
                          "every Muon parameter needs a .grad")
        if adamw_grads is not None and len(adamw_grads) != len(self.adamw_groups):
            raise ValueError("adamw_grads must hold one list per AdamW group")
        grads_a = [given(g["params"], None if adamw_grads is None else adamw_grads[gi],
                         f"adamw_grads[{gi}] must hold one gradient per parameter of its group",
                         "every AdamW parameter needs a .grad") for gi, g in enumerate(self.adamw_groups)]
        formed = self._form_all(self.muon_params + [p for g in self.adamw_groups for p in g["params"]],
                                grads + [x for xs in grads_a for x in xs], stream)
        grads, at = formed[:len(grads)], len(grads)
        for gi, xs in enumerate(grads_a):
            grads_a[gi], at = formed[at:at + len(xs)], at + len(xs)
        gd = self._grad_dtypes(grads)
        adamw = api.AdamWArgs([
            api.AdamWSpec(g["params"], xs, g["exp_avg"], g["exp_avg_sq"], g["lr"], g["betas"][0], g["betas"][1],
                          g["eps"], g["weight_decay"]) for g, xs in zip(self.adamw_groups, grads_a)])
        if self.muon_params:
            if replicas:
                reps = [[rep[k] for k in self._order] for rep in replicas]
                api.muon_step_replicated(self.muon_params, grads, self.momentum, self._groups(gd), self.lr,
                                         self.beta, self.wd, self.ns_steps, self.coeffs, self.flags,
                                         self.workspace, reps, stream=stream)
            else:
                api.muon_step(self.muon_params, grads, self.momentum, self._groups(gd), self.lr,
                              self.beta, self.wd, self.ns_steps, self.coeffs, self.flags,
                              self.workspace, stream=stream)
        self.step_count += 1
        if self.adamw_groups:
            api.adamw_step(adamw, self.step_count, stream=stream)

    def state_dict(self) -> dict:
        """Step count and optimizer state; "momentum" follows the order in
        which the Muon parameters were given, not the internal grouping."""
        mom: List[Optional[torch.Tensor]] = [None] * len(self.momentum)
        for k, pos in enumerate(self._order):
            mom[pos] = self.momentum[k].clone()
        return {"step": self.step_count,
                "momentum": mom,
                "exp_avg": [[t.clone() for t in g["exp_avg"]] for g in self.adamw_groups],
                "exp_avg_sq": [[t.clone() for t in g["exp_avg_sq"]] for g in self.adamw_groups]}

    def load_state_dict(self, sd: dict) -> None:
        """Restore a state_dict of an optimizer over parameters of the same
        shapes, given in the same order; nothing is changed if it does not fit."""
        def fits(dst: List[torch.Tensor], src, what: str) -> None:
            if len(src) != len(dst) or any(tuple(a.shape) != tuple(b.shape) for a, b in zip(dst, src)):
                raise ValueError(f"state_dict: {what} does not match this optimizer's parameters")
        mom_internal = [sd["momentum"][pos] for pos in self._order] \
            if len(sd["momentum"]) == len(self.momentum) else sd["momentum"]
        fits(self.momentum, mom_internal, "momentum")
        if len(sd["exp_avg"]) != len(self.adamw_groups) or len(sd["exp_avg_sq"]) != len(self.adamw_groups):
            raise ValueError("state_dict: AdamW group count does not match")
        for g, ea, es in zip(self.adamw_groups, sd["exp_avg"], sd["exp_avg_sq"]):
            fits(g["exp_avg"], ea, "exp_avg")
            fits(g["exp_avg_sq"], es, "exp_avg_sq")
        self.step_count = int(sd["step"])
        for dst, src in zip(self.momentum, mom_internal):
            dst.copy_(src)
        for g, ea, es in zip(self.adamw_groups, sd["exp_avg"], sd["exp_avg_sq"]):
            for dst, src in zip(g["exp_avg"], ea):
                dst.copy_(src)
            for dst, src in zip(g["exp_avg_sq"], es):
                dst.copy_(src)
