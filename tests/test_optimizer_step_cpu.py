"""MuonAdamW.step on the host: what it checks before anything changes.  The
library's calls are recorded, not made."""
import pytest
import torch

from muon_polar_orthogonalized_b200 import api
from muon_polar_orthogonalized_b200.optimizer import MuonAdamW


class Factor(api.LinearGrad):
    """Writes ones, or fails."""

    def __init__(self, fails=False):
        self.fails = fails

    def workspace_size(self, grad):
        return 256

    def write(self, grad, workspace, accumulate=False, stream=None):
        if self.fails:
            raise ValueError("a factor of another shape")
        grad.fill_(1.0)


@pytest.fixture
def opt(monkeypatch):
    """An optimizer over CPU tensors (its constructor wants CUDA ones)."""
    o = MuonAdamW.__new__(MuonAdamW)
    o.lr, o.beta, o.wd, o.ns_steps, o.coeffs, o.flags = 0.02, 0.95, 0.01, 5, (1.0, 1.0, 1.0), 0
    o.muon_params = [torch.zeros(4, 6), torch.zeros(4, 6)]
    o._order, o._shapes = [1, 0], [(4, 6, 2, 0, 1.0)]
    o.momentum = [torch.zeros(4, 6) for _ in range(2)]
    ps = [torch.zeros(8, 4), torch.zeros(4)]
    o.adamw_groups = [dict(params=ps, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0,
                           exp_avg=[torch.zeros_like(p) for p in ps], exp_avg_sq=[torch.zeros_like(p) for p in ps])]
    o.step_count = 0
    o.workspace = torch.zeros(256, dtype=torch.uint8)
    o._factor_workspace, o._captured_workspaces = None, []
    o.launched = []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    for name in ("muon_step", "muon_step_replicated"):
        monkeypatch.setattr(api, name, lambda *a, **k: o.launched.append("muon"))
    return o


MG = lambda: [torch.ones(4, 6), torch.ones(4, 6)]
AG = lambda: [torch.ones(8, 4), torch.ones(4)]


@pytest.mark.parametrize("match,grads", [
    ("one gradient per Muon", lambda: dict(muon_grads=MG()[:1], adamw_grads=[AG()])),
    ("Muon parameter needs", lambda: dict(adamw_grads=[AG()])),
    ("Muon parameter needs", lambda: dict(muon_grads=[MG()[0], None], adamw_grads=[AG()])),
    ("gradient is a tensor", lambda: dict(muon_grads=[MG()[0], "ones"], adamw_grads=[AG()])),
    ("must all be fp32", lambda: dict(muon_grads=[MG()[0], MG()[0].bfloat16()], adamw_grads=[AG()])),
    ("one list per AdamW group", lambda: dict(muon_grads=MG(), adamw_grads=[])),
    ("one gradient per parameter", lambda: dict(muon_grads=MG(), adamw_grads=[AG()[:1]])),
    ("AdamW parameter needs", lambda: dict(muon_grads=MG())),
    ("AdamW parameter needs", lambda: dict(muon_grads=MG(), adamw_grads=[[AG()[0], None]])),
    ("gradient is a tensor", lambda: dict(muon_grads=MG(), adamw_grads=[[AG()[0], []]])),
    ("gradient is a tensor", lambda: dict(muon_grads=MG(), adamw_grads=[["ones", AG()[1]]])),
    ("is a matrix", lambda: dict(muon_grads=MG(), adamw_grads=[[AG()[0], Factor()]])),
    ("another shape", lambda: dict(muon_grads=MG(), adamw_grads=[[Factor(fails=True), AG()[1]]])),
    ("another shape", lambda: dict(muon_grads=[Factor(), Factor(fails=True)], adamw_grads=[AG()])),
    ("expected a contiguous", lambda: dict(muon_grads=MG(), adamw_grads=[[AG()[0].bfloat16(), AG()[1]]])),
])
def test_a_refused_gradient_changes_nothing(opt, match, grads):
    with pytest.raises(ValueError, match=match):
        opt.step(**grads())
    assert opt.launched == [] and opt.step_count == 0


def test_a_gradient_that_was_not_formed_is_not_left_behind(opt):
    p = opt.adamw_groups[0]["params"][0]
    with pytest.raises(ValueError, match="another shape"):
        opt.step(muon_grads=MG(), adamw_grads=[[[Factor(), Factor(fails=True)], AG()[1]]])
    assert p.grad is None
    kept = p.grad = torch.full_like(p, 3.0)
    with pytest.raises(ValueError, match="another shape"):
        opt.step(muon_grads=MG(), adamw_grads=[[Factor(fails=True), AG()[1]]])
    assert p.grad is kept
