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
    o._factor_status = torch.zeros(1, dtype=torch.int32)
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


class Reporting(Factor):
    """A factor whose call clears its status word, fills its scratch, and reports."""

    def __init__(self, word, need):
        self.fails, self.word, self.need = False, word, need

    def workspace_size(self, grad):
        return self.need

    def write(self, grad, workspace, accumulate=False, stream=None):
        assert workspace.data_ptr() % 4 == 0 and workspace.numel() >= self.need
        workspace[:self.need] = 0x5A
        workspace[:4].view(torch.int32)[0] = self.word
        grad.fill_(1.0)


def test_a_factor_that_reports_is_not_forgotten(opt, monkeypatch):
    """The word of any factor of a step reaches query_status, whatever the later
    factors and steps write, and once."""
    from muon_polar_orthogonalized_b200 import _native as N
    muon, adamw = [N.MUON_OK], [N.MUON_OK]
    monkeypatch.setattr(api, "muon_query_status", lambda ws, stream=None: muon[0])
    monkeypatch.setattr(api, "adamw_query_status", lambda stream=None: adamw[0])
    opt.adamw_groups = []
    assert opt.query_status() == N.MUON_OK
    for k in range(4):
        words = [Reporting(1 if i == k else 0, need) for i, need in enumerate((300, 5000, 256, 100000 >> k))]
        opt.step(muon_grads=[words[:3], words[3]])
        opt.step(muon_grads=[Reporting(0, 700), [Reporting(0, 256), Reporting(0, 256)]])
        opt.step(muon_grads=MG())
        assert opt.query_status() == N.MUON_ERR_TIMEOUT
        assert opt.query_status() == N.MUON_OK
    opt.step(muon_grads=[Reporting(0, 300), Reporting(0, 9000)])
    assert opt.query_status() == N.MUON_OK
    muon[0] = N.MUON_ERR_TIMEOUT
    assert opt.query_status() == N.MUON_ERR_TIMEOUT
    muon[0], adamw[0] = N.MUON_OK, N.MUON_ERR_TIMEOUT
    assert opt.query_status() == N.MUON_ERR_TIMEOUT
    assert len(opt.launched) == 13
