"""AdamW plans (fp32 and 8-bit moments), the gradient norm and the moment
conversion.

Stored codes and scales are compared bit for bit with a NumPy float32
restatement of the documented arithmetic (state8_ref); values are compared
with the float64 oracle under bounds that count roundings: u = 2^-24 for each
fp32 operation, half a step for a stored code or bf16 value.
"""

import ctypes
import math
import os

import numpy as np
import pytest

import oracle
import state8_ref as ref

torch = pytest.importorskip("torch")
U = 2.0 ** -24
BF = 2.0 ** -8          # half a step of bf16, relative
SIZES = [1, 7, 255, 256, 257, 511, 1000, 4096, 4097, 12301]


# ---------------------------------------------------------------------------
# CPU: the definition, the ABI without a device
# ---------------------------------------------------------------------------

def test_code_rounding_of_the_reference():
    """Nearest rounding moves a real-valued code by at most 1/2, so a value by
    at most (1/c + 1/(4 c^2)) of itself; the largest element is exact to
    rounding; zero blocks stay zero; a second moment is never zero where its
    block holds anything."""
    rng = np.random.default_rng(0)
    m = (rng.standard_normal(3000) * np.exp(rng.standard_normal(3000))).astype(np.float32)
    m[512:768] = 0
    c, s = ref.encode_m(m)
    d = ref.decode_m(c, s).astype(np.float64)
    nz = c != 0
    k = np.abs(c[nz].astype(np.float64))
    assert np.all(np.abs(d[nz] - m[nz]) <= np.abs(d[nz]) * (1 / k + 1 / (4 * k * k) + 1e-5))
    assert np.all(d[512:768] == 0) and s[2] == 0
    v = (m.astype(np.float64) ** 2).astype(np.float32)
    cv, sv = ref.encode_v(v)
    dv = ref.decode_v(cv, sv)
    assert np.all(dv[v > 0] > 0) and np.all(dv[512:768] == 0)
    oc, os_, _ = oracle.state8_encode(m)
    assert np.mean(oc != c) < 1e-3 and np.allclose(os_, s, rtol=2 * U, atol=0)
    ov, _, _ = oracle.state8_encode(v, True)
    assert np.mean(ov != cv) < 1e-3


def test_stochastic_codes_are_unbiased():
    """The mean of floor(y + u) over hashed u is y: within 5 standard errors
    (at most 0.5 / sqrt(n)), plus half a step of the 16-bit numbers, and the
    fp32 rounding of y + u below 256 (2^-17)."""
    n = 200000
    h, hp = ref.hashed(n, seed=7, step=3, tensor=2)
    for y in (0.3, 5.01, 100.5, 200.999):
        for bits in (h, ref.swap(h), hp):
            mean = np.floor(np.float32(y) + ref.unit(bits)).astype(np.float64).mean()
            assert abs(mean - np.float32(y)) < 5 * 0.5 / math.sqrt(n) + 2.0 ** -17 + 2.0 ** -17
    # other steps, tensors and seeds give other numbers
    for other in (dict(seed=7, step=4, tensor=2), dict(seed=7, step=3, tensor=3), dict(seed=8, step=3, tensor=2)):
        assert np.mean(ref.hashed(n, **other)[0] == h) < 1e-3


def test_struct_layouts_match_the_header(tmp_path):
    import shutil
    import subprocess
    from matrix_aware_optimizer_step_b200 import binding as b
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    pairs = {"muon_plan_tensor": b.PlanTensor, "muon_adamw_plan_hparams": b.AdamwPlanHparams,
             "muon_grad_tensor": b.GradTensor, "muon_state8_tensor": b.State8Tensor}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "muon.h"', "int main(void) {"]
    for cname, cls in pairs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'  printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-I", inc, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    got = {(out[i], out[i + 1]): int(out[i + 2]) for i in range(0, len(out), 3)}
    for cname, cls in pairs.items():
        assert got[(cname, "size")] == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert got[(cname, f)] == getattr(cls, f).offset, (cname, f)


def test_entry_points_refuse_null_without_a_device():
    from matrix_aware_optimizer_step_b200 import build
    build.build()
    import matrix_aware_optimizer_step_b200 as m
    lib = m.load_library()
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    hp = m.default_adamw_plan_hparams()
    assert (hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay) == (3e-4, 0.9, 0.95, 1e-8, 0.01)
    with pytest.raises(TypeError):
        m.default_adamw_plan_hparams(beta3=0.5)
    bad = m.binding.MUON_ERR_INVALID_ARG
    assert lib.muon_adamw_plan_create(None, None, 0, 32, ctypes.byref(h)) == bad and not h.value
    assert lib.muon_grad_norm_plan_create(None, None, 0, ctypes.byref(h)) == bad
    assert lib.muon_state8_plan_create(None, None, 0, ctypes.byref(h)) == bad
    assert lib.muon_adamw_plan_step(None, ctypes.byref(hp), 1, None, None, None, 0, 0, None) == bad
    assert lib.muon_grad_norm_run(None, 1.0, None, None) == bad
    assert lib.muon_grad_norm_out_bytes(None, ctypes.byref(n)) == bad
    assert lib.muon_plan_bind_grads(None, None, 0) == bad
    assert lib.muon_state8_pack(None, None) == bad and lib.muon_state8_unpack(None, None) == bad
    lib.muon_plan_destroy(None)


def test_state8_zeros_and_scales():
    from matrix_aware_optimizer_step_b200 import plans
    assert [plans.state8_scales(n) for n in (0, 1, 256, 257)] == [0, 1, 1, 2]
    z = plans.state8_zeros(torch.zeros(3, 100))
    assert z["exp_avg"].dtype == torch.int8 and z["exp_avg_sq"].dtype == torch.uint8
    assert z["exp_avg"].shape == (3, 100) and z["exp_avg_scale"].numel() == 2
    assert np.all(ref.decode_v(z["exp_avg_sq"].numpy().ravel(), z["exp_avg_sq_scale"].numpy()) == 0)


# ---------------------------------------------------------------------------
# GPU
# ---------------------------------------------------------------------------

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from matrix_aware_optimizer_step_b200 import build
    build.build()
    import matrix_aware_optimizer_step_b200 as m
    return m


@pytest.fixture(scope="module")
def ctx(mx):
    with mx.MuonContext(0) as c:
        yield c


def grads_np(rng, n, bf16):
    g = rng.standard_normal(n) * np.exp(rng.standard_normal(n)) * 1e-3
    g[rng.random(n) < 0.2] = 0
    g = g.astype(np.float32)
    return ref.round_bf16(g) if bf16 else g


def place(x, dtype, shift):
    """x as a contiguous CUDA slice that starts `shift` elements into its
    allocation, between two guards of 64 elements that nothing may write."""
    buf = torch.full((shift + 64 + x.size + 64,), 7, dtype=dtype, device="cuda")
    t = buf[shift + 64:shift + 64 + x.size]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return t, buf


class Tensors:
    """A list of tensors on the GPU and the NumPy state they should have."""

    def __init__(self, sizes, seed, pbf16=False, gbf16=True, s8=False, copy=False, shift=0, zero=False):
        self.rng = np.random.default_rng(seed)
        self.gbf16, self.pbf16, self.s8, self.copy, self.sizes = gbf16, pbf16, s8, copy, sizes
        pd, gd = (torch.bfloat16 if pbf16 else torch.float32), (torch.bfloat16 if gbf16 else torch.float32)
        self.p, self.m, self.v, self.ms, self.vs = [], [], [], [], []
        self.bufs, self.tp, self.tg, self.tm, self.tv, self.tms, self.tvs, self.tc = [], [], [], [], [], [], [], []
        for n in sizes:
            p = (self.rng.standard_normal(n) * 0.02).astype(np.float32)
            p = ref.round_bf16(p) if pbf16 else p
            m0 = np.zeros(n, np.float32) if zero else (self.rng.standard_normal(n) * 3e-4).astype(np.float32)
            v0 = np.zeros(n, np.float32) if zero else (self.rng.standard_normal(n) ** 2 * 1e-6).astype(np.float32)
            if s8:
                c, s = ref.encode_m(m0)
                d, t = ref.encode_v(v0)
                m0, v0 = ref.decode_m(c, s), ref.decode_v(d, t)
                for lst, x, dt in ((self.tm, c, torch.int8), (self.tv, d, torch.uint8), (self.tms, s, torch.float32),
                                   (self.tvs, t, torch.float32)):
                    self.add(lst, x, dt, shift)
                self.ms.append(s); self.vs.append(t)
            else:
                self.add(self.tm, m0, torch.float32, shift)
                self.add(self.tv, v0, torch.float32, shift)
            self.p.append(p); self.m.append(m0); self.v.append(v0)
            self.add(self.tp, p, pd, shift)
            self.add(self.tg, np.zeros(n, np.float32), gd, shift)
            if copy:
                self.add(self.tc, np.zeros(n, np.float32), torch.bfloat16, shift)

    def add(self, lst, x, dtype, shift):
        t, buf = place(x, dtype, shift)
        lst.append(t)
        self.bufs.append((buf, t.numel(), shift + 64))

    def guards_intact(self):
        for buf, n, at in self.bufs:
            assert bool((buf[:at] == 7).all()) and bool((buf[at + n:] == 7).all())

    def new_grads(self):
        gs = [grads_np(self.rng, n, self.gbf16) for n in self.sizes]
        for t, g in zip(self.tg, gs):
            t.copy_(torch.from_numpy(g))
        return gs

    def plan(self, ctx):
        return ctx.adamw_plan(self.tp, self.tg, self.tm, self.tv, self.tms if self.s8 else None,
                              self.tvs if self.s8 else None, self.tc if self.copy else None)


def f32(t):
    return t.detach().float().cpu().numpy()


def check_step(T, gs, t, beta1, beta2, lr, eps, wd, scale=None, seed=None):
    """Advance T's NumPy state by one step and compare the GPU's with it."""
    for i, g in enumerate(gs):
        n = g.size
        m32, v32 = ref.moments(T.m[i], T.v[i], g, beta1, beta2, scale)
        hp = dict(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=wd)
        g64 = g.astype(np.float64) * (1.0 if scale is None else float(np.float32(scale)))
        p1, m1, v1 = oracle.adamw_step(T.p[i], g64, T.m[i], T.v[i], t, hp)
        # moments: two products and a sum (and the clipped gradient's, twice in v); beta and 1 - beta rounded to fp32
        mb = 5 * U * (beta1 * np.abs(T.m[i].astype(np.float64)) + (1 - beta1) * np.abs(g64))
        vb = 8 * U * v1
        h16 = None
        if seed is not None:
            hc, hpar = ref.hashed(n, seed, t, i)
            h16 = hpar if T.pbf16 else None
        # parameter: at most 12 roundings on the way of the update (moments, root, quotient, corrections), 4 on the
        # parameter's own way; the moments' own bound moves m through the quotient
        upd = (p1 - T.p[i].astype(np.float64) * (1 - lr * wd))
        denom = np.sqrt(v1 / (1 - beta2 ** t)) + eps
        pb = 4 * U * np.abs(T.p[i].astype(np.float64)) + 16 * U * np.abs(upd) + lr / (1 - beta1 ** t) * mb / denom
        got = f32(T.tp[i]).astype(np.float64)
        if T.pbf16:
            # nearest: half a step; stochastic: less than a whole one (and the fp32 error may pass a boundary)
            pb = pb * 2 + (2 * BF if seed is not None else BF) * np.maximum(np.abs(p1), np.abs(got)) + 1e-38
        assert np.all(np.abs(got - p1) <= pb + 1e-30), (i, n, t)
        if T.copy:
            assert np.array_equal(f32(T.tc[i]), ref.round_bf16(f32(T.tp[i])))
        if T.s8:
            um = uv = np.float32(0.5)
            if seed is not None:
                uv, um = ref.unit(hc), ref.unit(ref.swap(hc))
            c, s = ref.encode_m(m32, um)
            d, q = ref.encode_v(v32, uv)
            for name, want, t_ in (("m", c, T.tm[i]), ("v", d, T.tv[i]), ("m_scale", s, T.tms[i]),
                                   ("v_scale", q, T.tvs[i])):
                have = t_.cpu().numpy()
                assert np.array_equal(have, want), (name, n, t, np.flatnonzero(have != want)[:5])
            T.m[i], T.v[i] = ref.decode_m(c, s), ref.decode_v(d, q)
            if seed is None:
                # what is stored against the oracle's moments: half a code, and the code's own fp32 error
                _, _, y = oracle.state8_encode(m1)
                assert np.all(np.abs(np.abs(c.astype(np.float64)) - y) <= 0.5 + 127 * 8 * U + np.where(
                    np.abs(m1) > 0, 64 * mb / np.maximum(np.abs(m1), 1e-300) * y, 0))
        else:
            assert np.all(np.abs(f32(T.tm[i]) - m1) <= mb)
            assert np.all(np.abs(f32(T.tv[i]) - v1) <= vb)
            T.m[i], T.v[i] = f32(T.tm[i]), f32(T.tv[i])
        T.p[i] = f32(T.tp[i])


@gpu
@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("gbf16", [True, False])
@pytest.mark.parametrize("pbf16,copy,seed", [(False, False, None), (False, True, None), (True, False, None),
                                             (True, False, 99)])
def test_adamw32_steps(ctx, mx, pbf16, copy, seed, gbf16, shift):
    T = Tensors(SIZES, 1, pbf16, gbf16, False, copy, shift)
    plan = T.plan(ctx)
    hp = mx.default_adamw_plan_hparams(beta2=0.999)
    for t in (1, 2, 700):
        gs = T.new_grads()
        plan.step(t, hp, seed=seed)
        torch.cuda.synchronize()
        check_step(T, gs, t, 0.9, 0.999, 3e-4, 1e-8, 0.01, None, seed)
    T.guards_intact()


@gpu
@pytest.mark.parametrize("shift", [0, 1, 4])
@pytest.mark.parametrize("gbf16", [True, False])
@pytest.mark.parametrize("pbf16,copy,seed", [(False, False, None), (False, True, 5), (True, False, None),
                                             (True, False, 2 ** 32 - 1)])
def test_adamw8_steps(ctx, mx, pbf16, copy, seed, gbf16, shift):
    """Codes and scales bit for bit over several steps, from zero state."""
    T = Tensors(SIZES, 2, pbf16, gbf16, True, copy, shift, zero=True)
    plan = T.plan(ctx)
    hp = mx.default_adamw_plan_hparams(lr=1e-3, beta1=0.8, beta2=0.99, weight_decay=0.1, eps=1e-6)
    scale = torch.tensor([0.37], device="cuda")
    for t in (1, 2, 3, 10):
        gs = T.new_grads()
        plan.step(t, hp, grad_scale=scale if t != 2 else None, seed=seed)
        torch.cuda.synchronize()
        check_step(T, gs, t, 0.8, 0.99, 1e-3, 1e-6, 0.1, 0.37 if t != 2 else None, seed)
    T.guards_intact()


@gpu
def test_adamw8_many_values_bit_for_bit(ctx, mx):
    """Two million elements of a wide spread: any code that approximate
    arithmetic would round across a boundary shows."""
    T = Tensors([2_000_003], 3, False, False, True)
    plan = T.plan(ctx)
    for t, seed in ((5, None), (6, 11)):
        gs = T.new_grads()
        plan.step(t, mx.default_adamw_plan_hparams(beta2=0.999), seed=seed)
        torch.cuda.synchronize()
        check_step(T, gs, t, 0.9, 0.999, 3e-4, 1e-8, 0.01, None, seed)


@gpu
@pytest.mark.parametrize("s8", [False, True])
def test_more_tensors_than_one_launch_and_mixed_types(ctx, mx, s8):
    """1100 tensors (three launches of one kind), then a list of every type:
    each tensor as it would be alone."""
    rng = np.random.default_rng(4)
    T = Tensors([int(x) for x in rng.integers(1, 700, 1100)], 5, False, True, s8)
    T.plan(ctx)
    plan, gs = T.plan(ctx), T.new_grads()
    plan.step(3, seed=1 if s8 else None)
    torch.cuda.synchronize()
    check_step(T, gs, 3, 0.9, 0.95, 3e-4, 1e-8, 0.01, None, 1 if s8 else None)
    T.guards_intact()
    Ts = [Tensors([300, 0, 5000], 6 + k, p, g, s8) for k, (p, g) in enumerate([(0, 0), (0, 1), (1, 0), (1, 1)])]
    both = [x for pair in zip(*[list(zip(t.tp, t.tg, t.tm, t.tv, t.tms or t.tm, t.tvs or t.tv)) for t in Ts])
            for x in pair]
    gs = [t.new_grads() for t in Ts]
    lists = list(zip(*both))
    plan = ctx.adamw_plan(*lists[:4], *(lists[4:] if s8 else ()))
    plan.step(2)
    torch.cuda.synchronize()
    for t, g in zip(Ts, gs):
        nonempty = [i for i, n in enumerate(t.sizes) if n]
        for name in ("p", "m", "v", "ms", "vs", "tp", "tm", "tv", "tms", "tvs", "sizes"):
            lst = getattr(t, name)
            if lst:
                setattr(t, name, [lst[i] for i in nonempty])
        check_step(t, [g[i] for i in nonempty], 2, 0.9, 0.95, 3e-4, 1e-8, 0.01)


@gpu
def test_blocks_with_no_or_bad_moments(ctx, mx):
    """Zero gradients on zero state leave zeros; a block below 2^-100 is
    stored as zero; NaN and infinity spoil their own block of 256 only."""
    n = 256 * 6
    g = np.full(n, 1e-3, np.float32)
    g[:256] = 0
    g[256:512] = 1e-33          # m = 1e-34 < 2^-100; v underflows to 0
    g[512 + 5] = np.nan
    g[768 + 7] = np.inf
    T = Tensors([n], 7, False, False, True, zero=True)
    T.tg[0].copy_(torch.from_numpy(g))
    p0 = T.p[0].copy()
    T.plan(ctx).step(1)
    torch.cuda.synchronize()
    c, s = T.tm[0].cpu().numpy(), T.tms[0].cpu().numpy()
    d, q = T.tv[0].cpu().numpy(), T.tvs[0].cpu().numpy()
    m32, v32 = ref.moments(T.m[0], T.v[0], g, 0.9, 0.95)
    with np.errstate(invalid="ignore"):
        ec, es = ref.encode_m(m32)
        ed, eq = ref.encode_v(v32)
    assert np.array_equal(c, ec) and np.array_equal(d, ed)
    assert np.array_equal(s, es, equal_nan=True) and np.array_equal(q, eq, equal_nan=True)
    assert s[0] == 0 and s[1] == 0 and q[0] == 0 and np.isnan(s[2]) and np.isnan(s[3]) and np.isnan(q[3])
    p = f32(T.tp[0])
    assert np.isnan(p[517]) and np.isfinite(np.delete(p, [517, 775])).all()
    assert np.allclose(p[:256], p0[:256] * (1 - 3e-4 * 0.01), rtol=2 * U, atol=0)


@gpu
def test_nonfinite_factor_device_step_and_rate_leave_everything(ctx, mx):
    """A factor or rate that is not finite, or a device step below 1, writes
    nothing."""
    T = Tensors([1000, 5000], 8, True, True, True)
    plan = T.plan(ctx)
    T.new_grads()
    state = T.tp + T.tm + T.tv + T.tms + T.tvs
    before = [t.clone() for t in state]
    dev = dict(device="cuda")
    for kw in (dict(grad_scale=torch.tensor([math.nan], **dev)), dict(grad_scale=torch.tensor([math.inf], **dev)),
               dict(lr=torch.tensor([math.nan], **dev))):
        plan.step(1, **kw)
    plan.step(torch.tensor([0], **dev))
    plan.step(torch.tensor([-3], **dev), seed=3)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state, before))
    plan.step(1)
    torch.cuda.synchronize()
    assert not any(torch.equal(a, b) for a, b in zip(state, before))


@gpu
@pytest.mark.parametrize("s8", [False, True])
def test_device_step_and_rate_match_host_ones_and_capture(ctx, mx, s8):
    """A captured step with the count and rate on the device, replayed, gives
    what eager calls give: codes bit for bit, parameters within the rounding
    of the two corrections (formed in 64 bits on either side)."""
    A = Tensors([700, 9000], 9, not s8, True, s8)
    B = Tensors([700, 9000], 9, not s8, True, s8)
    for a, b in zip(A.tg, B.tg):
        x = torch.randn(a.numel(), device="cuda") * 1e-3
        a.copy_(x); b.copy_(x)
    pa, pb = A.plan(ctx), B.plan(ctx)
    na, nb = ctx.grad_norm_plan(A.tg), ctx.grad_norm_plan(B.tg)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    hp = mx.default_adamw_plan_hparams(beta2=0.999)
    out = nb.new_output()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.add_(1)
        f = nb.run(0.01, out=out)
        pb.step(step, hp, lr=lr, grad_scale=f[1:], seed=17)
    assert int(step) == 0
    for t in range(1, 6):
        rate = 1e-3 / t
        lr.fill_(rate)
        graph.replay()
        hq = mx.default_adamw_plan_hparams(beta2=0.999, lr=float(np.float32(rate)))
        pa.step(t, hq, grad_scale=na.run(0.01)[1:], seed=17)
        for a in A.tg + B.tg:      # both move on to new gradients between replays
            a.mul_(-0.7)
    torch.cuda.synchronize()
    for x, y in zip(A.tm + A.tv + A.tms + A.tvs, B.tm + B.tv + B.tms + B.tvs):
        assert torch.equal(x, y)
    for x, y in zip(A.tp, B.tp):
        assert np.all(np.abs(f32(x) - f32(y)) <= (2 * BF if not s8 else 20 * U) * np.abs(f32(x)) + 1e-9)
    del graph


@gpu
def test_rebinding_gradients(ctx, mx):
    T = Tensors([300, 2000], 10, False, True, True)
    plan, norm = T.plan(ctx), ctx.grad_norm_plan(T.tg)
    gs = T.new_grads()
    fresh = [t.clone() for t in T.tg]
    for t in T.tg:
        t.fill_(math.nan)
    plan.bind_grads(fresh)
    norm.bind_grads(fresh)
    r = norm.run()
    plan.step(1)
    torch.cuda.synchronize()
    check_step(T, gs, 1, 0.9, 0.95, 3e-4, 1e-8, 0.01)
    assert abs(float(r[0]) - oracle.grad_norm(gs)[0]) <= 4 * U * float(r[0])
    for bad in (fresh[:1], [fresh[0].float(), fresh[1]], [fresh[1], fresh[0]], [fresh[0].cpu(), fresh[1]]):
        with pytest.raises((ValueError, TypeError)):
            plan.bind_grads(bad)
    with pytest.raises(mx.MuonError):
        plan.bind_grads([T.tm[0].view(torch.uint8).new_zeros(600).view(torch.bfloat16), T.tp[1].view(torch.bfloat16)[:2000]])


@gpu
def test_plan_refusals(ctx, mx):
    def f(n, dt=torch.float32):
        return torch.zeros(n, dtype=dt, device="cuda")
    p, g, m, v, c = f(512), f(512), f(512), f(512), f(512, torch.bfloat16)
    m8, v8, s = f(512, torch.int8), f(512, torch.uint8), f(2)
    s2 = f(2)
    ok = ctx.adamw_plan([p], [g], [m], [v])
    for args, kw in [(([p], [g], [m], [v], [s]), {}),                           # one list of scales
                     (([p], [g], [m8], [v8]), {}),                              # 8-bit moments without scales
                     (([p], [g], [m], [v], [s], [s2]), {}),                     # fp32 moments with scales
                     (([p], [g], [v8], [m8], [s], [s2]), {}),                   # types swapped
                     (([p], [g], [m8], [v8], [f(1)], [s2]), {}),                # too few scales
                     (([p], [g[:511]], [m], [v]), {}),
                     (([p, p], [g], [m], [v]), {}),
                     (([p.half()], [g], [m], [v]), {}),
                     (([p.cpu()], [g], [m], [v]), {}),
                     (([f((512, 2))[:, 0]], [g], [m], [v]), {}),
                     (([c], [g], [m], [v]), dict(param_copies=[f(512, torch.bfloat16)])),
                     (([p], [g], [m], [v]), dict(param_copies=[p]))]:
        with pytest.raises((ValueError, TypeError)):
            ctx.adamw_plan(*args, **kw)
    big = f(1024)
    for args in [([p, p], [g, g], [m, f(512)], [v, f(512)]),                    # the same parameter twice
                 ([p], [g], [m], [m]),                                          # both moments in one tensor
                 ([p], [p], [m], [v]),                                          # gradient is the parameter
                 ([big[:512], big[511:1023]], [g, g], [m, f(512)], [v, f(512)])]:
        with pytest.raises(mx.MuonError) as e:
            ctx.adamw_plan(*args)
        assert e.value.status == mx.binding.MUON_ERR_INVALID_ARG
    for kw in (dict(step=0), dict(step=-1), dict(step=1, hp=mx.default_adamw_plan_hparams(beta1=1.0)),
               dict(step=1, hp=mx.default_adamw_plan_hparams(beta2=-0.1)),
               dict(step=1, hp=mx.default_adamw_plan_hparams(eps=0.0)),
               dict(step=1, hp=mx.default_adamw_plan_hparams(eps=1e-60)),
               dict(step=1, hp=mx.default_adamw_plan_hparams(lr=math.nan)),
               dict(step=1, hp=mx.default_adamw_plan_hparams(weight_decay=math.inf))):
        with pytest.raises(mx.MuonError):
            ok.step(**kw)
    for kw in (dict(seed=-1), dict(seed=2 ** 32), dict(grad_scale=torch.ones(1)), dict(grad_scale=0.5),
               dict(lr=f(1, torch.float64)), dict(grad_scale=f(0))):
        with pytest.raises((ValueError, TypeError)):
            ok.step(1, **kw)
    with pytest.raises((ValueError, TypeError)):
        ok.step(f(1, torch.int32))
    n = ctx.grad_norm_plan([g])
    for bad in (-1.0, math.nan):
        with pytest.raises(mx.MuonError):
            n.run(bad)
    with pytest.raises(ValueError):
        n.run(1.0, out=f(2))
    with pytest.raises(TypeError):
        ctx.grad_norm_plan([g.double()])
    with pytest.raises(mx.MuonError):
        ctx.state8_plan([f(512)], [m8], [m8.view(torch.float32)[:2]])            # scales inside the codes
    with pytest.raises(ValueError):
        ctx.state8_plan([f(512)], [f(511, torch.int8)], [s])
    with pytest.raises(TypeError):
        ctx.state8_plan([f(512)], [f(512, torch.int16)], [s])
    torch.cuda.synchronize()
    assert all(int(torch.count_nonzero(t)) == 0 for t in (p, m, v, m8, v8, s))
    # closed plans and contexts
    ok.close()
    with pytest.raises(mx.MuonError):
        ok.step(1)
    other = mx.MuonContext(0)
    q = other.adamw_plan([p], [g], [m], [v])
    other.close()
    with pytest.raises(mx.MuonError):
        q.step(1)
    with pytest.raises(ValueError):
        other.adamw_plan([p], [g], [m], [v])
    q.close()
    # empty lists
    e = ctx.adamw_plan([], [], [], [])
    e.step(1)
    ctx.state8_plan([], [], []).pack()
    r = ctx.grad_norm_plan([]).run(1.0)
    assert r.tolist() == [0.0, 1.0]


@gpu
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("shift", [0, 1])
def test_grad_norm(ctx, mx, bf16, shift):
    rng = np.random.default_rng(11)
    for sizes in ([1], [768], SIZES, [0, 3, 0], [8191, 8193, 1_000_003], [int(x) for x in rng.integers(1, 300, 1000)]):
        gs = [grads_np(rng, n, bf16) for n in sizes]
        ts = [place(g, torch.bfloat16 if bf16 else torch.float32, shift)[0] for g in gs]
        plan = ctx.grad_norm_plan(ts)
        for max_norm in (math.inf, 1e-3, 0.0):
            want, factor = oracle.grad_norm(gs, max_norm)
            r = plan.run(max_norm).double().tolist()
            # squares of 8 elements in fp32 (at most 8 roundings, halved by the root), the result rounded once
            assert abs(r[0] - want) <= 5 * U * want
            assert abs(r[1] - factor) <= 7 * U * factor
        first = plan.run().clone()
        for _ in range(3):
            assert torch.equal(plan.run(), first)


@gpu
def test_grad_norm_range_and_bad_values(ctx, mx):
    """Squares that leave fp32's range, either way, do not lose the norm; NaN
    and infinity leave no factor."""
    for mag in (1e-30, 1e-22, 1e-13, 1e17, 1e19, 1e30):
        g = np.full(3000, mag, np.float32)
        g[::3] = 0
        g[7] = -2 * mag
        r = ctx.grad_norm_plan([torch.from_numpy(g).cuda()]).run(1.0).double().tolist()
        want, factor = oracle.grad_norm([g], 1.0)
        assert abs(r[0] - want) <= 5 * U * want and abs(r[1] - factor) <= 7 * U * factor
    for bad in (math.nan, math.inf, -math.inf):
        for at in (0, 1234, 2999):
            t = torch.ones(3000, device="cuda")
            t[at] = bad
            r = ctx.grad_norm_plan([t, torch.ones(5, device="cuda").bfloat16()]).run(1.0).tolist()
            assert not math.isfinite(r[0]) and math.isnan(r[1])
    t = torch.full((3000,), 3e38, device="cuda")              # finite gradients, a norm beyond fp32
    r = ctx.grad_norm_plan([t]).run(1.0).tolist()
    assert r[0] == math.inf and math.isnan(r[1])


@gpu
def test_norm_runs_side_by_side_have_their_own_outputs(ctx, mx):
    g = torch.randn(5_000_000, device="cuda")
    plan = ctx.grad_norm_plan([g])
    want = plan.run(1.0).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [plan.new_output() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                r = plan.run(1.0, out=o)
            assert r.data_ptr() == o.data_ptr()
    torch.cuda.synchronize()
    assert all(torch.equal(o[:2], want) for o in outs)


@gpu
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_state8_conversion(ctx, mx, bf16, shift):
    rng = np.random.default_rng(12)
    vals, codes, scales, raw, bufs = [], [], [], [], []
    for second in (False, True):
        for n in SIZES:
            x = (rng.standard_normal(n) * np.exp(2 * rng.standard_normal(n)) * 1e-3).astype(np.float32)
            if n > 600:
                x[:256] = 0
                x[300] = 0
            x = np.abs(x) if second else x
            x = ref.round_bf16(x) if bf16 else x
            raw.append((second, x))
            for lst, arr, dt in ((vals, x, torch.bfloat16 if bf16 else torch.float32),
                                 (codes, np.full(n, 55), torch.uint8 if second else torch.int8),
                                 (scales, np.full(-(-n // 256), 3.0, np.float32), torch.float32)):
                t, b = place(arr, dt, shift)
                lst.append(t)
                bufs.append((b, n if lst is not scales else -(-n // 256), shift + 64))
    plan = ctx.state8_plan(vals, codes, scales)
    plan.pack()
    torch.cuda.synchronize()
    for (second, x), c, s in zip(raw, codes, scales):
        ec, es = (ref.encode_v if second else ref.encode_m)(x)
        assert np.array_equal(c.cpu().numpy(), ec) and np.array_equal(s.cpu().numpy(), es)
    plan.unpack()
    torch.cuda.synchronize()
    for (second, x), t, c, s in zip(raw, vals, codes, scales):
        want = (ref.decode_v if second else ref.decode_m)(c.cpu().numpy(), s.cpu().numpy())
        assert np.array_equal(f32(t), ref.round_bf16(want) if bf16 else want)
    for b, n, at in bufs:
        assert bool((b[:at] == 7).all()) and bool((b[at + n:] == 7).all())


@gpu
def test_state8_bad_values_spoil_their_block_only(ctx, mx):
    m = torch.ones(1024, device="cuda")
    v = torch.ones(1024, device="cuda")
    m[3], m[300], v[600], v[900] = math.nan, math.inf, -1.0, math.inf
    cm, cv = torch.zeros(1024, dtype=torch.int8, device="cuda"), torch.zeros(1024, dtype=torch.uint8, device="cuda")
    sm, sv = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    om, ov = torch.empty_like(m), torch.empty_like(v)
    ctx.state8_plan([m, v], [cm, cv], [sm, sv]).pack()
    ctx.state8_plan([om, ov], [cm, cv], [sm, sv]).unpack()
    torch.cuda.synchronize()
    assert om.view(4, 256).isnan().all(1).tolist() == [True, True, False, False]
    assert ov.view(4, 256).isnan().all(1).tolist() == [False, False, True, True]
    assert torch.allclose(om[512:], torch.ones(512, device="cuda"), rtol=4 * U)


@gpu
def test_run_of_all_operators_as_a_loop_uses_them(ctx, mx):
    """A 32-bit checkpoint taken into 8 bits, clipped steps on a side stream,
    one step with a NaN gradient that is skipped, and the state read back."""
    from matrix_aware_optimizer_step_b200.plans import state8_zeros
    rng = np.random.default_rng(13)
    sizes = [5000, 768, 33]
    p0 = [(rng.standard_normal(n) * 0.02).astype(np.float32) for n in sizes]
    m0 = [(rng.standard_normal(n) * 1e-3).astype(np.float32) for n in sizes]
    v0 = [(rng.standard_normal(n) ** 2 * 1e-6).astype(np.float32) for n in sizes]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        P = [torch.from_numpy(x.copy()).cuda() for x in p0]
        G = [torch.zeros_like(x) for x in P]
        C = [x.bfloat16() for x in P]
        Z = [state8_zeros(x) for x in P]
        M = [torch.from_numpy(x).cuda() for x in m0]
        V = [torch.from_numpy(x).cuda() for x in v0]
        codes = [z["exp_avg"] for z in Z] + [z["exp_avg_sq"] for z in Z]
        scales = [z["exp_avg_scale"] for z in Z] + [z["exp_avg_sq_scale"] for z in Z]
        conv = ctx.state8_plan(M + V, codes, scales)
        conv.pack()
        plan = ctx.adamw_plan(P, G, codes[:3], codes[3:], scales[:3], scales[3:], C)
        norm = ctx.grad_norm_plan(G)
        p = [x.copy() for x in p0]
        cm, cv = [ref.encode_m(x) for x in m0], [ref.encode_v(x) for x in v0]
        for t in range(1, 7):
            gs = [grads_np(rng, n, False) for n in sizes]
            if t == 4:
                gs[1][5] = np.nan
            for a, b in zip(G, gs):
                a.copy_(torch.from_numpy(b))
            f = norm.run(1e-2)
            plan.step(t, grad_scale=f[1:], seed=123)
            if t == 4:
                continue
            factor = np.float32(float(f[1]))
            assert abs(float(factor) - oracle.grad_norm(gs, 1e-2)[1]) <= 8 * U
            for i, g in enumerate(gs):
                m, v = ref.moments(ref.decode_m(*cm[i]), ref.decode_v(*cv[i]), g, 0.9, 0.95, factor)
                p[i] = oracle.adamw_step(p[i], g.astype(np.float64) * float(factor), ref.decode_m(*cm[i]),
                                         ref.decode_v(*cv[i]), t)[0]
                h, _ = ref.hashed(g.size, 123, t, i)
                cm[i], cv[i] = ref.encode_m(m, ref.unit(ref.swap(h))), ref.encode_v(v, ref.unit(h))
        conv.unpack()
    side.synchronize()
    for i in range(3):
        assert np.array_equal(codes[i].cpu().numpy(), cm[i][0]) and np.array_equal(codes[3 + i].cpu().numpy(), cv[i][0])
        assert np.array_equal(f32(M[i]), ref.decode_m(*cm[i])) and np.array_equal(f32(V[i]), ref.decode_v(*cv[i]))
        # five steps of at most 20 roundings on updates below 5 * lr / (1 - 0.9), and 4 on the parameter
        assert np.all(np.abs(f32(P[i]) - p[i]) <= 5 * (4 * U * np.abs(p[i]) + 20 * U * 5 * 3e-3))
        assert np.array_equal(f32(C[i]), ref.round_bf16(f32(P[i])))


@gpu
def test_flagged_context_writes_nothing(ctx, mx):
    """After a device-side wait gave up, plan calls leave every tensor as it
    is until check_device reports it; the norm, which changes no state, runs."""
    T = Tensors([1000], 14, False, True, True)
    plan, norm = T.plan(ctx), ctx.grad_norm_plan(T.tg)
    gs = T.new_grads()
    out = torch.full((1000,), 3.0, device="cuda")
    conv = ctx.state8_plan([out], [T.tm[0]], [T.tms[0]])
    before = T.tp[0].clone()
    ctx.selftest_wait()
    plan.step(1)
    conv.unpack()
    r = norm.run()
    torch.cuda.synchronize()
    assert torch.equal(T.tp[0], before) and bool((out == 3).all()) and float(r[0]) > 0
    with pytest.raises(mx.MuonError):
        ctx.check_device()
    plan.step(1)
    torch.cuda.synchronize()
    check_step(T, gs, 1, 0.9, 0.95, 3e-4, 1e-8, 0.01)


@gpu
def test_one_tensor_past_2_to_31_elements(ctx, mx):
    """Offsets beyond 32 bits: 2^31 + 1000 elements, the last blocks checked
    bit for bit and the guard behind them."""
    n = (1 << 31) + 1000
    gen = torch.Generator(device="cuda").manual_seed(3)
    buf = torch.full((n + 64,), 7, dtype=torch.bfloat16, device="cuda")
    p = buf[:n]
    p.fill_(0.5)
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    k = -(-n // 256)
    ms, vs = torch.zeros(k, device="cuda"), torch.zeros(k, device="cuda")
    first = (n - 3000) // 256 * 256
    tail = (torch.randn(n - first, generator=gen, device="cuda") * 1e-3).bfloat16()
    g[first:] = tail
    plan, norm = ctx.adamw_plan([p], [g], [m], [v], [ms], [vs]), ctx.grad_norm_plan([g])
    r = norm.run()
    plan.step(1, seed=21)
    torch.cuda.synchronize()
    x = f32(tail)
    assert abs(float(r[0]) - oracle.grad_norm([x])[0]) <= 5 * U * float(r[0])
    z = np.zeros(x.size, np.float32)
    m32, v32 = ref.moments(z, z, x, 0.9, 0.95)
    h, hp = ref.hashed(x.size, 21, 1, 0, first=first)
    c, s = ref.encode_m(m32, ref.unit(ref.swap(h)))
    d, q = ref.encode_v(v32, ref.unit(h))
    assert np.array_equal(m[first:].cpu().numpy(), c) and np.array_equal(v[first:].cpu().numpy(), d)
    assert np.array_equal(ms[first // 256:].cpu().numpy(), s) and np.array_equal(vs[first // 256:].cpu().numpy(), q)
    assert int(torch.count_nonzero(m[:first])) == 0 and bool((buf[n:] == 7).all())
    values = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    ctx.state8_plan([values], [m], [ms]).unpack()
    torch.cuda.synchronize()
    assert np.array_equal(f32(values[first:]), ref.round_bf16(ref.decode_m(c, s)))


@gpu
@pytest.mark.parametrize("mag", [1e-9, 1e-12, 1e-14, 1e-17, 1e-20, 1e12])
@pytest.mark.parametrize("eps", [1e-8, 1e-20])
def test_adamw8_over_the_range_of_gradients(ctx, mx, mag, eps):
    """Blocks either side of the range that the fast path takes, subnormal
    second moments among them, and an eps that its flushes would reach: codes
    bit for bit, parameters within their bound."""
    T = Tensors([4099], 30, False, False, True, zero=True)
    plan, rng = T.plan(ctx), np.random.default_rng(31)
    hp = mx.default_adamw_plan_hparams(eps=eps)
    for t in (1, 2):
        g = (rng.standard_normal(4099) * np.exp(3 * rng.standard_normal(4099)) * mag).astype(np.float32)
        T.tg[0].copy_(torch.from_numpy(g))
        plan.step(t, hp)
        torch.cuda.synchronize()
        m32, v32 = ref.moments(T.m[0], T.v[0], g, 0.9, 0.95)
        (c, s), (d, q) = ref.encode_m(m32), ref.encode_v(v32)
        assert np.array_equal(T.tm[0].cpu().numpy(), c) and np.array_equal(T.tv[0].cpu().numpy(), d)
        assert np.array_equal(T.tms[0].cpu().numpy(), s) and np.array_equal(T.tvs[0].cpu().numpy(), q)
        # the parameter from the fp32 moments (a subnormal v has few bits: its root is taken as it is)
        r = np.sqrt(v32.astype(np.float64))
        upd = 3e-4 / (1 - 0.9 ** t) * m32.astype(np.float64) / (r / math.sqrt(1 - 0.95 ** t) + eps)
        p1 = T.p[0].astype(np.float64) * (1 - 3e-4 * 0.01) - upd
        assert np.all(np.abs(f32(T.tp[0]) - p1) <= 4 * U * np.abs(T.p[0]) + 16 * U * np.abs(upd) + 1e-30)
        T.m[0], T.v[0], T.p[0] = ref.decode_m(c, s), ref.decode_v(d, q), f32(T.tp[0])


@gpu
def test_two_graphs_of_one_plan_and_a_plan_freed_during_capture(ctx, mx):
    T = Tensors([5000], 32, False, True, True)
    R = Tensors([5000], 32, False, True, True)
    plan, direct = T.plan(ctx), R.plan(ctx)
    doomed = ctx.state8_plan([torch.zeros(300, device="cuda")], [torch.zeros(300, dtype=torch.int8, device="cuda")],
                             [torch.zeros(2, device="cuda")])
    gs = [T.new_grads()[0] for _ in range(2)]
    bufs = [torch.from_numpy(g).cuda().bfloat16() for g in gs]
    graphs = []
    for t, b in enumerate(bufs, 1):
        plan.bind_grads([b])
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            plan.step(t, seed=4)
            if t == 1:
                doomed.close()
        graphs.append(graph)
    plan.bind_grads(T.tg)          # captured calls keep their gradients
    for t, b in enumerate(bufs, 1):
        graphs[t - 1].replay()
        direct.bind_grads([b])
        direct.step(t, seed=4)
    torch.cuda.synchronize()
    for x, y in zip(T.tp + T.tm + T.tv + T.tms + T.tvs, R.tp + R.tm + R.tv + R.tms + R.tvs):
        assert torch.equal(x, y)
    del graphs


@gpu
def test_first_norm_on_another_stream(ctx):
    for k in range(20):
        g = torch.full((1000 * (k + 1),), 2.0, device="cuda")
        torch.cuda.synchronize()
        plan = ctx.grad_norm_plan([g])
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            r = plan.run(1.0)
        side.synchronize()
        assert abs(float(r[0]) - 2 * math.sqrt(g.numel())) <= 5 * U * float(r[0])


@gpu
def test_one_tensor_past_2_to_33_elements_hashes_its_high_word(ctx, mx):
    """2^33 + 600 elements: pair numbers beyond 32 bits, the last blocks'
    stochastic codes bit for bit."""
    n = (1 << 33) + 600
    if torch.cuda.mem_get_info()[0] < 7 * n:
        pytest.skip("needs 60 GB of device memory")
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.int8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(-(-n // 256), device="cuda"), torch.zeros(-(-n // 256), device="cuda")
    first = (1 << 33) - 512
    x = grads_np(np.random.default_rng(33), n - first, True)
    g[first:] = torch.from_numpy(x).cuda().bfloat16()
    ctx.adamw_plan([p], [g], [m], [v], [ms], [vs]).step(1, seed=77)
    torch.cuda.synchronize()
    z = np.zeros(x.size, np.float32)
    m32, v32 = ref.moments(z, z, x, 0.9, 0.95)
    h, _ = ref.hashed(x.size, 77, 1, 0, first=first)
    c, s = ref.encode_m(m32, ref.unit(ref.swap(h)))
    d, q = ref.encode_v(v32, ref.unit(h))
    assert np.array_equal(m[first:].cpu().numpy(), c) and np.array_equal(v[first:].cpu().numpy(), d)
    assert np.array_equal(ms[first // 256:].cpu().numpy(), s) and np.array_equal(vs[first // 256:].cpu().numpy(), q)
    del p, g, m, v
    torch.cuda.empty_cache()


@gpu
def test_first_calls_of_a_process_inside_a_capture():
    """Nothing is left to load or set up when a plan's first call is captured
    (a new process: this one has loaded the kernels)."""
    import subprocess
    import sys
    code = """
import torch
from matrix_aware_optimizer_step_b200 import MuonContext
from matrix_aware_optimizer_step_b200.plans import state8_zeros
ctx = MuonContext(0)
p = torch.zeros(5000, device="cuda"); g = torch.ones(5000, device="cuda"); z = state8_zeros(p)
out = torch.zeros(5000, device="cuda")
m, v = torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda")
q = torch.zeros(5000, device="cuda", dtype=torch.bfloat16)
a = ctx.adamw_plan([p], [g], [z["exp_avg"]], [z["exp_avg_sq"]], [z["exp_avg_scale"]], [z["exp_avg_sq_scale"]])
b = ctx.adamw_plan([q], [g], [m], [v])
n = ctx.grad_norm_plan([g]); u = ctx.state8_plan([out], [z["exp_avg"]], [z["exp_avg_scale"]])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    f = n.run(10.0)
    a.step(1, grad_scale=f[1:], seed=1); b.step(1, seed=2); u.unpack(); u.pack()
graph.replay(); torch.cuda.synchronize()
assert abs(float(f[0]) - 5000 ** 0.5) < 1e-3 and bool((p < 0).all()) and bool((q < 0).all()) and bool((out > 0).all())
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@gpu
@pytest.mark.parametrize("mag", [1e-33, 1e-29, 1e-20, 1e20, 1e36, 1e37, 3e38])
def test_state8_conversion_over_the_range_of_fp32(ctx, mag):
    """Blocks either side of what the fast path takes, up to fp32's largest
    values: codes and scales bit for bit."""
    rng = np.random.default_rng(40)
    m = (rng.uniform(-1, 1, 2100) ** 3 * mag).astype(np.float32)
    v = np.abs(m)
    cm, cv = torch.zeros(2100, dtype=torch.int8, device="cuda"), torch.zeros(2100, dtype=torch.uint8, device="cuda")
    sm, sv = torch.zeros(9, device="cuda"), torch.zeros(9, device="cuda")
    ctx.state8_plan([torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda()], [cm, cv], [sm, sv]).pack()
    torch.cuda.synchronize()
    (c, s), (d, q) = ref.encode_m(m), ref.encode_v(v)
    assert np.array_equal(cm.cpu().numpy(), c) and np.array_equal(sm.cpu().numpy(), s)
    assert np.array_equal(cv.cpu().numpy(), d) and np.array_equal(sv.cpu().numpy(), q)
