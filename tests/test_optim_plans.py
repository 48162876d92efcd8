"""MuonWithAuxAdam's AdamW groups with 8-bit moments, bf16 parameters,
clipping and stochastic rounding."""

import copy
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")


def test_refuses_bad_group_values_without_gpu():
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    p = torch.nn.Parameter(torch.zeros(4))
    for bad in (dict(state_bits=4), dict(max_grad_norm=-1.0), dict(max_grad_norm=math.nan), dict(seed=-1),
                dict(seed=1 << 32)):
        with pytest.raises(ValueError):
            MuonWithAuxAdam([dict(params=[p], use_muon=False, **bad)])


gpu = pytest.mark.gpu
SHAPES = [(300, 40), (257,), (3, 5, 7)]


def params(dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.nn.Parameter((torch.randn(s, generator=gen, device="cuda") * 0.02).to(dtype)) for s in SHAPES]


def grad(ps, t, dtype=None):
    gen = torch.Generator(device="cuda").manual_seed(100 + t)
    for p in ps:
        p.grad = (torch.randn(p.shape, generator=gen, device="cuda") * 1e-2).to(dtype or p.dtype)


@gpu
@pytest.mark.parametrize("dtype,bits,seed,clip", [(torch.float32, 8, None, None), (torch.bfloat16, 8, 5, 0.1),
                                                  (torch.bfloat16, 32, 5, None), (torch.float32, 32, None, 0.1)])
def test_steps_equal_direct_plan_calls(dtype, bits, seed, clip):
    """Gradients that move from step to step, a parameter without one in one
    step: bit for bit what plan calls give."""
    import matrix_aware_optimizer_step_b200 as mx
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    from matrix_aware_optimizer_step_b200.plans import state8_zeros
    a, b = params(dtype), params(dtype)
    opt = MuonWithAuxAdam([dict(params=a, use_muon=False, lr=1e-3, betas=(0.9, 0.99), state_bits=bits, seed=seed,
                                max_grad_norm=clip)])
    st = [state8_zeros(p) if bits == 8 else dict(exp_avg=torch.zeros_like(p, dtype=torch.float32),
                                                 exp_avg_sq=torch.zeros_like(p, dtype=torch.float32)) for p in b]
    steps = [0, 0, 0]
    hp = mx.default_adamw_plan_hparams(lr=1e-3, beta1=0.9, beta2=0.99)
    with mx.MuonContext(0) as ctx:
        for t in range(1, 6):
            grad(a, t)
            grad(b, t)
            if t == 2:
                a[1].grad = b[1].grad = None
            opt.step()
            live = [i for i in range(3) if b[i].grad is not None]
            f = None
            if clip is not None:
                f = ctx.grad_norm_plan([b[i].grad.view(-1) for i in live]).run(clip)[1:].clone()
            by = {}
            for i in live:
                steps[i] += 1
                by.setdefault(steps[i], []).append(i)
            for step, ix in by.items():
                q = [[b[i].detach().view(-1) for i in ix], [b[i].grad.view(-1) for i in ix]]
                q += [[st[i][k].view(-1) for i in ix] for k in st[0]]
                ctx.adamw_plan(*q).step(step, hp, grad_scale=f, seed=seed)
        torch.cuda.synchronize()
    for x, y, s in zip(a, b, st):
        assert torch.equal(x, y)
        for k, v in s.items():
            assert opt.state[x][k].dtype == v.dtype and torch.equal(opt.state[x][k], v)


@gpu
def test_nonfinite_gradient_skips_the_clipped_group():
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    a = params()
    opt = MuonWithAuxAdam([dict(params=a, use_muon=False, state_bits=8, max_grad_norm=1.0)])
    grad(a, 1)
    opt.step()
    before = [p.detach().clone() for p in a], copy.deepcopy([opt.state[p] for p in a])
    grad(a, 2)
    a[2].grad[1, 2, 3] = math.nan
    opt.step()
    torch.cuda.synchronize()
    for p, q, s in zip(a, *before):
        assert torch.equal(p, q)
        assert all(torch.equal(opt.state[p][k], v) for k, v in s.items() if k != "step")
    grad(a, 3)
    opt.step()
    torch.cuda.synchronize()
    assert not any(torch.equal(p, q) for p, q in zip(a, before[0]))


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [8, 32])
def test_checkpoint_resumes_bit_for_bit(dtype, bits):
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam

    def make(ps):
        return MuonWithAuxAdam([dict(params=ps, use_muon=False, state_bits=bits, seed=3, max_grad_norm=1.0)])

    a, b = params(dtype), params(dtype)
    one, two = make(a), make(b)
    for t in range(1, 7):
        grad(a, t)
        one.step()
    for t in range(1, 4):
        grad(b, t)
        two.step()
    saved = copy.deepcopy(two.state_dict())
    c = [torch.nn.Parameter(p.detach().clone()) for p in b]
    three = make(c)
    three.load_state_dict(saved)
    for t in range(4, 7):
        grad(c, t)
        three.step()
    torch.cuda.synchronize()
    for x, y in zip(a, c):
        assert torch.equal(x, y)
        for k, v in one.state[x].items():
            w = three.state[y][k]
            assert (w == v) if not isinstance(v, torch.Tensor) else (w.dtype == v.dtype and torch.equal(w, v)), k


@gpu
def test_changing_state_bits_converts_the_moments():
    """32 -> 8 -> 32 bits: moments within half a code of what they were (1/c +
    1/(4 c^2) of the value, c at least 1 code, plus the smallest code)."""
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    a = params()
    opt = MuonWithAuxAdam([dict(params=a, use_muon=False, lr=0.0, weight_decay=0.0, max_grad_norm=1e9,
                                betas=(0.9, 0.95))])
    grad(a, 1)
    opt.step()
    m0 = [opt.state[p]["exp_avg"].clone() for p in a]
    v0 = [opt.state[p]["exp_avg_sq"].clone() for p in a]
    opt._moments(a, 8)
    assert all(opt.state[p]["exp_avg"].dtype == torch.int8 and "exp_avg_scale" in opt.state[p] for p in a)
    opt._moments(a, 32)
    torch.cuda.synchronize()
    for p, m, v in zip(a, m0, v0):
        st = opt.state[p]
        assert "exp_avg_scale" not in st and st["exp_avg"].dtype == torch.float32 and st["exp_avg"].shape == p.shape
        # one code's step in the value: (2 c + 1) s, half of it and a rounding; c = 127 sqrt(|m| / max)
        for x, y, levels, second in ((st["exp_avg"], m, 127.0, False), (st["exp_avg_sq"], v, 256.0, True)):
            x, y = x.double().flatten().cpu().numpy(), y.double().flatten().cpu().numpy()
            if second:
                x, y = np.sqrt(x), np.sqrt(y)
            for at in range(0, y.size, 256):
                xb, yb = np.abs(x[at:at + 256]), np.abs(y[at:at + 256])
                big = yb.max()
                code = lambda z: levels * np.sqrt(z / big)   # noqa: E731
                low = 1.0 if second else 0.0
                assert np.all(np.abs(code(xb) - np.maximum(code(yb), low)) <= 0.5 + 1e-3)
    # and through step(): the group's key alone
    opt.param_groups[0]["state_bits"] = 8
    grad(a, 2)
    opt.step()
    opt.param_groups[0].update(state_bits=32, max_grad_norm=None)
    grad(a, 3)
    opt.step()
    torch.cuda.synchronize()
    assert all(opt.state[p]["exp_avg"].dtype == torch.float32 and opt.state[p]["step"] == 3 for p in a)


@gpu
def test_a_model_in_bf16_trains_with_8_bit_moments():
    """Runs for some steps beside a Muon group and stays finite."""
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(64, 256), torch.nn.GELU(), torch.nn.Linear(256, 8)).cuda()
    emb = torch.nn.Parameter(torch.randn(50, 64, device="cuda", dtype=torch.bfloat16) * 0.1)
    opt = MuonWithAuxAdam([dict(params=[model[0].weight], use_muon=True),
                           dict(params=[model[0].bias, model[2].weight, model[2].bias, emb], use_muon=False, lr=1e-3,
                                betas=(0.9, 0.999), state_bits=8, seed=1, max_grad_norm=1.0)], check_every=5)
    ids = torch.randint(0, 50, (128,), device="cuda")
    for _ in range(10):
        opt.zero_grad(set_to_none=True)
        loss = model(emb[ids].float()).square().mean()
        loss.backward()
        opt.step()
    assert all(bool(torch.isfinite(p).all()) for p in list(model.parameters()) + [emb])


@gpu
def test_groups_and_checkpoints_from_before_the_new_keys():
    """A group added with the old keys only, and a checkpoint whose state is
    of another floating type, step as ever."""
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    a, b = params(), params(seed=1)
    opt = MuonWithAuxAdam([dict(params=a, use_muon=False)])
    opt.add_param_group(dict(params=b, use_muon=False, lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.0))
    grad(a + b, 1)
    opt.step()
    sd = copy.deepcopy(opt.state_dict())
    for g in sd["param_groups"]:
        for k in ("state_bits", "max_grad_norm", "seed"):
            g.pop(k, None)
    for st in sd["state"].values():
        st["exp_avg"] = st["exp_avg"].double()
    opt.load_state_dict(sd)
    grad(a + b, 2)
    opt.step()
    torch.cuda.synchronize()
    assert all(opt.state[p]["exp_avg"].dtype == torch.float32 for p in a + b)


@gpu
def test_plans_do_not_keep_gradients_alive():
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    p = torch.nn.Parameter(torch.zeros(1 << 20, device="cuda"))
    opt = MuonWithAuxAdam([dict(params=[p], use_muon=False, state_bits=8, max_grad_norm=1.0)])
    for t in range(3):
        p.grad = torch.randn_like(p)
        opt.step()
        opt.zero_grad(set_to_none=True)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    p.grad = torch.randn_like(p)
    assert torch.cuda.memory_allocated() - held == 4 << 20
    opt.step()
    opt.zero_grad(set_to_none=True)
    assert torch.cuda.memory_allocated() == held


@gpu
def test_refuses_state_bits_changed_to_a_form_that_is_not_there():
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    ps = params()
    opt = MuonWithAuxAdam([dict(params=ps, use_muon=False)])
    before = [p.detach().clone() for p in ps]
    grad(ps, 1)
    opt.param_groups[0]["state_bits"] = 16
    with pytest.raises(ValueError):
        opt.step()
    assert all(torch.equal(p, q) for p, q in zip(ps, before))
    opt.param_groups[0]["state_bits"] = 8
    opt.step()
    assert not torch.equal(ps[0], before[0])
