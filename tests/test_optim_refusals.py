"""A step that MuonWithAuxAdam refuses has changed nothing: no parameter, no
step count.  On the CPU, with a context that writes down what it is asked."""

import math

import pytest

torch = pytest.importorskip("torch")


class Plan:
    def __init__(self, calls):
        self.calls = calls
        self.fail = False

    def step(self, step, hp, grad_scale=None, seed=None):
        if hp is None:
            raise ValueError("refused by the library")
        self.calls.append((step, seed))

    def run(self, max_norm):
        return torch.ones(2)

    def bind_grads(self, grads):
        pass

    def forget_grads(self):
        pass


class Recorder:
    def __init__(self):
        self.calls = []

    def adamw_plan(self, *lists):
        return Plan(self.calls)

    def grad_norm_plan(self, grads):
        return Plan(self.calls)


@pytest.fixture
def opt(monkeypatch):
    """Two AdamW groups that take plans, two parameters each."""
    from matrix_aware_optimizer_step_b200 import optim
    monkeypatch.setattr(torch.nn.Parameter, "is_cuda", True, raising=False)
    monkeypatch.setattr(optim, "MuonContext", lambda device: Recorder())
    monkeypatch.setattr(optim, "default_adamw_plan_hparams", lambda lr, **kw: None if lr is None else kw)
    ps = [torch.nn.Parameter(torch.zeros(4)) for _ in range(4)]
    for p in ps:
        p.grad = torch.zeros(4)
    return optim.MuonWithAuxAdam([dict(params=ps[:2], use_muon=False, state_bits=8, seed=1),
                                  dict(params=ps[2:], use_muon=False, state_bits=8, max_grad_norm=1.0)],
                                 device=0, check_every=0)


def steps(opt):
    return [opt.state[p].get("step", 0) for g in opt.param_groups for p in g["params"]]


@pytest.mark.parametrize("key,bad", [("seed", -1), ("seed", 1 << 32), ("seed", 1.5), ("seed", "1"),
                                     ("max_grad_norm", -1.0), ("max_grad_norm", math.nan), ("state_bits", 4)])
@pytest.mark.parametrize("group", [0, 1])
def test_a_value_changed_to_something_invalid_is_found_before_anything_moves(opt, key, bad, group):
    opt.step()
    assert steps(opt) == [1] * 4 and len(opt.ctx.calls) == 2
    good = opt.param_groups[group][key]
    opt.param_groups[group][key] = bad
    with pytest.raises(ValueError):
        opt.step()
    assert steps(opt) == [1] * 4 and len(opt.ctx.calls) == 2
    opt.param_groups[group][key] = good
    opt.step()
    assert steps(opt) == [2] * 4 and [c[0] for c in opt.ctx.calls] == [1, 1, 2, 2]


@pytest.mark.parametrize("key,bad", [("seed", 1.5), ("seed", "1"), ("max_grad_norm", "1")])
def test_the_constructor_refuses_what_a_step_would(opt, key, bad):
    with pytest.raises(ValueError):
        type(opt)([dict(params=[torch.nn.Parameter(torch.zeros(4))], use_muon=False, **{key: bad})], device=0)


def test_a_seed_of_another_integer_type(opt):
    import numpy as np
    opt.param_groups[0]["seed"] = np.int64(7)
    opt.step()
    assert (1, 7) in opt.ctx.calls and type(opt.ctx.calls[0][1]) is int


def test_a_group_without_the_keys_steps(opt):
    for k in ("seed", "max_grad_norm"):
        del opt.param_groups[0][k]
    opt.step()
    assert steps(opt) == [1] * 4


def test_a_call_that_the_library_refuses_is_not_counted(opt):
    opt.step()
    good = opt.param_groups[1]["lr"]
    opt.param_groups[1]["lr"] = None
    with pytest.raises(ValueError):
        opt.step()
    assert steps(opt) == [2, 2, 1, 1]
    opt.param_groups[1]["lr"] = good
    opt.step()
    assert steps(opt) == [3, 3, 2, 2] and opt.ctx.calls[-1][0] == 2
