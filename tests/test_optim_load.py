"""MuonWithAuxAdam.load_state_dict: torch's hooks around it see and change
what it loads, each tensor is taken once and in its own type, and a load that
cannot be done leaves the optimizer as it was.  On the CPU: the library is
not called."""

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def make(monkeypatch):
    """Optimizers over CPU parameters, with no context behind them."""
    from matrix_aware_optimizer_step_b200 import optim
    monkeypatch.setattr(torch.nn.Parameter, "is_cuda", True, raising=False)
    monkeypatch.setattr(optim, "MuonContext", lambda device: None)

    def build(params, **over):
        return optim.MuonWithAuxAdam([dict(dict(params=params, use_muon=False), **over)], device=0)

    return build


def params(n, dtype=torch.float32):
    return [torch.nn.Parameter(torch.zeros(300, dtype=dtype)) for _ in range(n)]


def eight_bit(opt, p, value):
    opt.state[p].update(step=value, exp_avg=torch.full((300,), value, dtype=torch.int8),
                        exp_avg_sq=torch.full((300,), value, dtype=torch.uint8),
                        exp_avg_scale=torch.full((2,), value / 7, dtype=torch.float32),
                        exp_avg_sq_scale=torch.full((2,), value / 9, dtype=torch.float32))


def test_a_pre_hook_reorders_the_checkpoint(make):
    """The saved order is b, a; a hook puts it back by name."""
    a, b = params(2)
    one = make([("b", b), ("a", a)], state_bits=8)
    eight_bit(one, a, 1)
    eight_bit(one, b, 2)
    saved = one.state_dict()
    c, d = params(2)
    two = make([("a", c), ("b", d)], state_bits=8)

    def by_name(opt, sd):
        names, own = sd["param_groups"][0]["param_names"], opt.param_groups[0]["param_names"]
        state = {i: sd["state"][sd["param_groups"][0]["params"][names.index(x)]] for i, x in enumerate(own)}
        group = dict(sd["param_groups"][0], params=list(range(len(own))), param_names=list(own))
        return dict(sd, state=state, param_groups=[group])

    two.register_load_state_dict_pre_hook(by_name)
    two.load_state_dict(saved)
    assert (two.state[c]["step"], two.state[d]["step"]) == (1, 2)
    assert int(two.state[c]["exp_avg"][0]) == 1 and int(two.state[d]["exp_avg_sq"][0]) == 2


def test_a_pre_hook_replaces_tensors_and_may_return_nothing(make):
    a, = params(1)
    one = make([a], state_bits=8)
    eight_bit(one, a, 3)
    c, = params(1)
    two = make([c], state_bits=8)
    seen = []
    two.register_load_state_dict_pre_hook(lambda opt, sd: seen.append(sorted(sd["state"][0])))

    def doubled(opt, sd):
        st = dict(sd["state"][0], exp_avg_scale=sd["state"][0]["exp_avg_scale"] * 2)
        return dict(sd, state={0: st})

    two.register_load_state_dict_pre_hook(doubled)
    two.load_state_dict(one.state_dict())
    assert seen == [["exp_avg", "exp_avg_scale", "exp_avg_sq", "exp_avg_sq_scale", "step"]]
    assert torch.equal(two.state[c]["exp_avg_scale"], 2 * one.state[a]["exp_avg_scale"])
    two.load_state_dict(one.state_dict())           # the hooks are still there, and there are no others
    assert len(seen) == 2 and torch.equal(two.state[c]["exp_avg_scale"], 2 * one.state[a]["exp_avg_scale"])


def test_a_post_hook_sees_and_changes_the_loaded_state(make):
    a, = params(1, torch.bfloat16)
    one = make([a], state_bits=8)
    eight_bit(one, a, 5)
    c, = params(1, torch.bfloat16)
    two = make([c], state_bits=8)
    seen = []

    def post(opt):
        st = opt.state[c]
        seen.append((st["step"], st["exp_avg"].dtype, st["exp_avg_scale"].dtype))
        st["step"] = 40
        st["exp_avg"] = torch.full((300,), 9, dtype=torch.int8)

    two.register_load_state_dict_post_hook(post)
    two.load_state_dict(one.state_dict())
    assert seen == [(5, torch.int8, torch.float32)]
    assert two.state[c]["step"] == 40 and int(two.state[c]["exp_avg"][0]) == 9


def test_types_copies_and_state_of_no_parameter(make):
    """Codes keep their type and floating state becomes fp32, in copies; what
    belongs to no parameter is kept; plans of the old state are dropped."""
    a, b = params(2, torch.bfloat16)
    one = make([a, b])
    eight_bit(one, a, 3)
    one.state[b].update(step=torch.tensor(6.0), exp_avg=torch.full((300,), 1 / 3, dtype=torch.float64))
    saved = one.state_dict()
    saved["state"]["elsewhere"] = {"kept": 1}
    c, d = params(2, torch.bfloat16)
    two = make([c, d])
    two._plans["stale"] = object()
    two.load_state_dict(saved)
    assert two.state[c]["exp_avg"].dtype == torch.int8 and two.state[c]["exp_avg_sq"].dtype == torch.uint8
    assert torch.equal(two.state[c]["exp_avg_scale"], one.state[a]["exp_avg_scale"])
    assert two.state[d]["step"] == 6 and isinstance(two.state[d]["step"], int)
    assert two.state[d]["exp_avg"].dtype == torch.float32 and float(two.state[d]["exp_avg"][0]) == float(
        torch.tensor(1 / 3, dtype=torch.float32))
    assert two.state[c]["exp_avg"].data_ptr() != one.state[a]["exp_avg"].data_ptr()
    assert two.state["elsewhere"] == {"kept": 1} and not two._plans


def test_tensors_never_take_the_parameters_type(make, monkeypatch):
    """No code passes through a floating type on its way in: the largest new
    tensor of a load is as large as the saved one."""
    a, = params(1)
    one = make([a], state_bits=8)
    eight_bit(one, a, 3)
    c, = params(1)
    two = make([c], state_bits=8)
    made = []
    to = torch.Tensor.to

    def spy(self, *args, **kw):
        r = to(self, *args, **kw)
        made.append((self.dtype, r.dtype))
        return r

    monkeypatch.setattr(torch.Tensor, "to", spy)
    two.load_state_dict(one.state_dict())
    assert made and not [x for x in made if x[0] in (torch.int8, torch.uint8) and x[1] != x[0]]


def test_tensors_inside_other_values_are_taken_the_same_way(make):
    """As the base class does: what a caller keeps beside the moments, in
    dictionaries and lists, moves and is cast like them."""
    a, = params(1)
    one = make([a])
    kept = dict(ema=torch.ones(3, dtype=torch.float64), more=[torch.ones(2, dtype=torch.int8), (5, "text")])
    one.state[a].update(step=1, mine=kept)
    c, = params(1, torch.bfloat16)
    two = make([c])
    two.load_state_dict(one.state_dict())
    mine = two.state[c]["mine"]
    assert mine["ema"].dtype == torch.float32 and mine["more"][0].dtype == torch.int8
    assert type(mine["more"]) is list and mine["more"][1] == (5, "text")
    assert mine["more"][0].data_ptr() != kept["more"][0].data_ptr()


def test_a_load_that_fails_changes_nothing(make):
    a, b = params(2)
    one = make([a, b], state_bits=8)
    eight_bit(one, a, 3)
    c, = params(1)
    two = make([c])
    eight_bit(two, c, 8)
    kept = two._plans["kept"] = object()
    for bad in (one.state_dict(), {"state": {}, "param_groups": []}):
        with pytest.raises(ValueError):
            two.load_state_dict(bad)
    assert two.state[c]["step"] == 8 and int(two.state[c]["exp_avg"][0]) == 8 and two._plans["kept"] is kept
    seen = []
    two.register_load_state_dict_post_hook(lambda opt: seen.append(len(opt.state)))
    good = make(params(1)).state_dict()             # nothing left over of the failed loads
    two.load_state_dict(good)
    assert seen == [0] and not two.state.get(c)
