"""A change of state_bits that cannot be carried out leaves the moments as
they were."""

import pytest

torch = pytest.importorskip("torch")


class Broken:
    """A context whose conversions fail at a chosen place."""

    def __init__(self, where):
        self.where = where

    def at(self, place):
        if place == self.where:
            raise RuntimeError(place)

    def state8_plan(self, values, codes, scales):
        self.at("create")
        return self

    def pack(self):
        self.at("run")

    unpack = pack

    def close(self):
        pass

    def check_device(self):
        self.at("check")


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("where", ["create", "run", "check"])
def test_a_failed_conversion_keeps_the_moments(monkeypatch, where, bits):
    from matrix_aware_optimizer_step_b200 import optim
    from matrix_aware_optimizer_step_b200.plans import state8_zeros
    monkeypatch.setattr(torch.nn.Parameter, "is_cuda", True, raising=False)
    monkeypatch.setattr(optim, "MuonContext", lambda device: Broken(where))
    p, q = (torch.nn.Parameter(torch.zeros(300)) for _ in range(2))
    opt = optim.MuonWithAuxAdam([dict(params=[p, q], use_muon=False)], device=0)
    held = {}
    for x in (p, q):
        st = opt.state[x]
        st.update(state8_zeros(x) if bits == 32 else dict(exp_avg=torch.ones(300), exp_avg_sq=torch.ones(300)), step=4)
        held[x] = dict(st)
    with pytest.raises(RuntimeError, match=where):
        opt._moments([p, q], bits)
    for x in (p, q):
        assert list(opt.state[x]) == list(held[x]) and all(opt.state[x][k] is v for k, v in held[x].items())


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_a_conversion_that_the_device_skipped_raises_and_keeps_the_moments(bits):
    """With a device-side failure unreported, kernels write nothing: the
    moments stay what they were, step() says so, and the next one converts."""
    import matrix_aware_optimizer_step_b200 as mx
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    p = torch.nn.Parameter(torch.randn(1000, device="cuda") * 0.02)
    opt = MuonWithAuxAdam([dict(params=[p], use_muon=False, state_bits=40 - bits, max_grad_norm=1.0)])
    p.grad = torch.randn_like(p) * 1e-2
    opt.step()
    torch.cuda.synchronize()
    before, kept = p.detach().clone(), {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in opt.state[p].items()}
    opt.param_groups[0]["state_bits"] = bits
    opt.ctx.selftest_wait()
    with pytest.raises(mx.MuonError):
        opt.step()
    assert torch.equal(p, before) and list(opt.state[p]) == list(kept)
    for k, v in kept.items():
        assert torch.equal(opt.state[p][k], v) if isinstance(v, torch.Tensor) else opt.state[p][k] == v
    opt.step()
    torch.cuda.synchronize()
    assert opt.state[p]["step"] == kept["step"] + 1 and not torch.equal(p, before)
    assert ("exp_avg_scale" in opt.state[p]) == (bits == 8)


@pytest.mark.gpu
@pytest.mark.parametrize("first,moment_bytes", [(32, 8.0), (8, 2.0 + 8 / 256)])
def test_a_conversion_frees_the_old_moments(first, moment_bytes):
    """32 to 8 bits gives back 8 B a parameter for 2 B and a scale for each
    256, and back again: no plan holds what was there before."""
    from matrix_aware_optimizer_step_b200.optim import MuonWithAuxAdam
    n = 1 << 20
    p = torch.nn.Parameter(torch.zeros(n, device="cuda"))
    q = torch.nn.Parameter(torch.zeros(n, device="cuda"))
    opt = MuonWithAuxAdam([dict(params=[p, q], use_muon=False, state_bits=first, max_grad_norm=1.0)])
    p.grad, q.grad = torch.ones_like(p), torch.ones_like(q)
    for both in (True, False, True):               # plans over both and over one
        q.grad = torch.ones_like(q) if both else None
        opt.step()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    opt.param_groups[0]["state_bits"] = 40 - first
    opt.step()
    torch.cuda.synchronize()
    other = 10.0 + 8 / 256 - moment_bytes
    change = torch.cuda.memory_allocated() - held
    assert abs(change - 2 * n * (other - moment_bytes)) <= 4096
