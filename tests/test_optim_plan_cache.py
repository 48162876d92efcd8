"""Which plans MuonWithAuxAdam keeps from step to step.  On the CPU, with a
context that only counts."""

import pytest

torch = pytest.importorskip("torch")


class Plan:
    def __init__(self, live):
        self.live = live
        live.add(self)

    def step(self, *args, **kw):
        pass

    def run(self, max_norm):
        return torch.ones(2)

    def bind_grads(self, grads):
        pass

    def forget_grads(self):
        pass


class Counter:
    def __init__(self):
        import weakref
        self.built, self.live = 0, weakref.WeakSet()

    def adamw_plan(self, *lists):
        self.built += 1
        return Plan(self.live)

    def grad_norm_plan(self, grads):
        return self.adamw_plan()


@pytest.fixture
def make(monkeypatch):
    from matrix_aware_optimizer_step_b200 import optim
    monkeypatch.setattr(torch.nn.Parameter, "is_cuda", True, raising=False)
    monkeypatch.setattr(optim, "MuonContext", lambda device: Counter())
    monkeypatch.setattr(optim, "default_adamw_plan_hparams", lambda **kw: None)

    def build(groups):
        return optim.MuonWithAuxAdam([dict(params=ps, use_muon=False, state_bits=8, max_grad_norm=1.0)
                                      for ps in groups], device=0, check_every=0)

    return build


def params(n):
    ps = [torch.nn.Parameter(torch.zeros(4)) for _ in range(n)]
    for p in ps:
        p.grad = torch.zeros(4)
    return ps


def test_many_groups_build_their_plans_once(make):
    """A rate for each tensor is a group for each tensor."""
    opt = make([[p] for p in params(100)])
    for _ in range(4):
        opt.step()
    assert opt.ctx.built == 200


def test_alternating_sets_of_gradients_build_their_plans_once(make):
    ps = params(3)
    opt = make([ps])
    kept = ps[2].grad
    for t in range(12):
        ps[2].grad = kept if t % 2 else None
        opt.step()
    # two norms, and steps over {0, 1}, {0, 1} with 2 apart in its step count
    assert opt.ctx.built <= 2 + 3


def test_plans_that_are_not_used_any_more_go(make):
    """Sets of parameters that never come again do not gather."""
    ps = params(40)
    opt = make([ps])
    grads = [p.grad for p in ps]
    most = 0
    for t in range(200):
        for i, p in enumerate(ps):
            p.grad = grads[i] if (t * 2654435761 + i * 40503) >> 7 & 1 else None
        opt.step()
        most = max(most, len(opt.ctx.live))
    for p, g in zip(ps, grads):
        p.grad = g
    for _ in range(40):
        opt.step()
    assert len(opt.ctx.live) <= 1 + len({opt.state[p]["step"] for p in ps})
    assert most < 17 * 41
