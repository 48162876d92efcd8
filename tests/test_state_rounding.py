"""Stochastic rounding of bf16 parameters in AdamW plans, element by element.

With zero gradients and moments the update is zero and the new parameter is
p * decay rounded once to fp32 (decay = 1 - lr wd formed in 64 bits, rounded
once): known exactly, so the stored bf16 value is too, from the hashed 16 bits
that state8_ref restates."""

import numpy as np
import pytest

import oracle
import state8_ref as ref

torch = pytest.importorskip("torch")
U = 2.0 ** -24
F = np.float32
gpu = pytest.mark.gpu
# whole blocks, ragged ends, less than a block, and one list place each
SIZES = [4096, 1, 257, 100, 20011]


def test_the_reference_rounds_up_with_the_dropped_bits_probability():
    """Truncation, rounding to nearest and the other half of the hash word all
    give other values than round_bf16 with its 16 bits."""
    p = (np.random.default_rng(1).standard_normal(20000) * 0.02).astype(F)
    h, hp = ref.hashed(p.size, 3, 2, 1)
    right = ref.round_bf16(p, hp)
    cut = (p.view(np.uint32) & np.uint32(0xFFFF0000)).view(F)
    for other in (cut, ref.round_bf16(p), ref.round_bf16(p, h), ref.round_bf16(p, np.roll(hp, 1))):
        assert np.mean(other != right) > 0.2
    away = np.abs(right) >= np.abs(p)
    low = (p.view(np.uint32) & np.uint32(0xFFFF)).astype(np.float64) / 65536
    assert abs(away.mean() - low.mean()) < 5 * 0.5 / np.sqrt(p.size)


def plan_of(ctx, ps, gs, s8):
    from matrix_aware_optimizer_step_b200.plans import state8_zeros
    z = [state8_zeros(p) if s8 else dict(exp_avg=torch.zeros_like(p, dtype=torch.float32),
                                         exp_avg_sq=torch.zeros_like(p, dtype=torch.float32)) for p in ps]
    names = ["exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if s8 else [])
    return ctx.adamw_plan(ps, gs, *[[s[k] for s in z] for k in names])


@pytest.fixture(scope="module")
def ctx():
    import matrix_aware_optimizer_step_b200 as mx
    with mx.MuonContext(0) as c:
        yield c


@gpu
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("gbf16", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_bits_of_stochastically_rounded_parameters(ctx, s8, gbf16, shift):
    """Bit for bit over three steps, at every size and both alignments."""
    import matrix_aware_optimizer_step_b200 as mx
    rng = np.random.default_rng(5)
    hp = mx.default_adamw_plan_hparams(lr=0.1, weight_decay=0.7)
    decay = F(1.0 - 0.1 * 0.7)
    now = [ref.round_bf16((rng.standard_normal(n) * 0.02).astype(F)) for n in SIZES]
    ps = []
    for p in now:
        buf = torch.zeros(p.size + shift, dtype=torch.bfloat16, device="cuda")
        buf[shift:].copy_(torch.from_numpy(p))
        ps.append(buf[shift:])
    gs = [torch.zeros(n, dtype=torch.bfloat16 if gbf16 else torch.float32, device="cuda") for n in SIZES]
    plan = plan_of(ctx, ps, gs, s8)
    for t, seed in ((1, 9), (2, 9), (3, 2 ** 32 - 1)):
        plan.step(t, hp, seed=seed)
        torch.cuda.synchronize()
        for i, p in enumerate(ps):
            h16 = ref.hashed(p.numel(), seed, t, i)[1]
            now[i] = ref.round_bf16(now[i] * decay, h16)
            assert np.array_equal(p.float().cpu().numpy(), now[i]), (i, t)


@gpu
@pytest.mark.parametrize("s8", [False, True])
def test_stochastic_rounding_is_unbiased_and_the_update_goes_through_it(ctx, s8):
    """A step with gradients: the stored value is round_bf16 of the exact one
    wherever fp32 arithmetic cannot decide, and the mean error over all
    elements is zero within five standard errors.

    The new parameter in fp32 is off by at most E = 4 U |p| + 16 U |update| (the roundings on its way, a parameter's
    four and the update's sixteen).  An element whose dropped bits, plus its 16 hashed ones, come within E of a
    carry may go either way; any other is decided.  The share of the first kind is at most about
    E / (bf16 step) = 20 U / 2^-8 = 3e-4 of |p|'s own steps, times two for either side."""
    import matrix_aware_optimizer_step_b200 as mx
    rng = np.random.default_rng(6)
    n, lr, wd = 1 << 20, 1e-3, 0.01
    p0 = ref.round_bf16((rng.uniform(0.5, 1.0, n) * 0.02 * np.sign(rng.standard_normal(n))).astype(F))
    g = (rng.standard_normal(n) * 1e-3).astype(F)
    p = torch.from_numpy(p0).cuda().bfloat16()
    plan_of(ctx, [p], [torch.from_numpy(g).cuda()], s8).step(1, mx.default_adamw_plan_hparams(lr=lr, weight_decay=wd),
                                                             seed=77)
    torch.cuda.synchronize()
    got = p.float().cpu().numpy().astype(np.float64)
    z = np.zeros(n)
    exact, _, _ = oracle.adamw_step(p0, g.astype(np.float64), z, z, 1,
                                    dict(lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=wd))
    e = 4 * U * np.abs(p0.astype(np.float64)) + 16 * U * np.abs(exact - p0 * (1 - lr * wd))
    h16 = ref.hashed(n, 77, 1, 0)[1]
    # between the fp32 values either side: both ends rounded with the same bits
    lo = ref.round_bf16(np.nextafter((exact - e).astype(F), F(-np.inf)), h16)
    hi = ref.round_bf16(np.nextafter((exact + e).astype(F), F(np.inf)), h16)
    assert np.all((got >= lo) & (got <= hi))
    decided = lo == hi
    assert np.array_equal(got[decided], lo[decided]) and decided.mean() > 0.998
    # in units of the bf16 step at |exact|; an error below one step has a standard deviation of at most 1/2
    step = 2.0 ** (np.floor(np.log2(np.abs(exact))) - 7)
    err = (got - exact) / step
    assert np.abs(err).max() < 1.01 and abs(err.mean()) < 5 * 0.5 / np.sqrt(n) + 2.0 ** -16


@gpu
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("n", [4096, 300])
def test_bad_parameters_keep_what_they_are_when_rounded_stochastically(ctx, s8, n):
    """NaN stays NaN and infinities their sign, whole blocks and tails; their
    neighbours round as ever."""
    import matrix_aware_optimizer_step_b200 as mx
    p0 = ref.round_bf16((np.random.default_rng(7).standard_normal(n) * 0.02).astype(F))
    bad = {3: np.nan, 100: np.inf, 101: -np.inf, n - 1: np.nan}
    p = torch.from_numpy(p0).cuda().bfloat16()
    for i, x in bad.items():
        p[i] = x
    # a NaN whose bits a carry would turn into a number
    p.view(torch.int16)[200] = 0x7FFF
    bad[200] = np.nan
    plan_of(ctx, [p], [torch.zeros(n, device="cuda")], s8).step(
        1, mx.default_adamw_plan_hparams(lr=0.1, weight_decay=0.7), seed=3)
    torch.cuda.synchronize()
    got = p.float().cpu().numpy()
    for i, x in bad.items():
        assert np.isnan(got[i]) if np.isnan(x) else got[i] == x, (i, got[i])
    ok = np.setdiff1d(np.arange(n), list(bad))
    want = ref.round_bf16(p0 * F(1.0 - 0.1 * 0.7), ref.hashed(n, 3, 1, 0)[1])
    assert np.array_equal(got[ok], want[ok])
