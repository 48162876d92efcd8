"""8-bit AdamW on lists so long that a warp works on several blocks of 256
elements: every form of the kernel, codes and scales bit for bit.

A warp takes total / (SMs * 4 * 8) blocks, up to 2 (fp32 parameters and
gradients) to 4 (both bf16).  Two of the tensors end in a warp with one whole
block and 100 elements of the next, whichever of 2, 3 and 4 it is."""

import numpy as np
import pytest

import state8_ref as ref
from test_state_plans import Tensors, check_step

torch = pytest.importorskip("torch")
SIZES = [12 * 256 * 1600 + 356, 12 * 256 * 1080 + 356, 70001, 513, 40]


@pytest.fixture(scope="module")
def ctx():
    import matrix_aware_optimizer_step_b200 as mx
    with mx.MuonContext(0) as c:
        yield c


def test_ends_are_a_whole_block_and_a_ragged_one():
    for n in SIZES[:2]:
        for blocks in (2, 3, 4):
            assert n % (blocks * 256) == 356


def with_moments(T):
    """Random codes and scales in place of zero moments."""
    for i, n in enumerate(T.sizes):
        k = -(-n // 256)
        c = T.rng.integers(-127, 128, n).astype(np.int8)
        d = T.rng.integers(0, 256, n).astype(np.uint8)
        s = (np.exp(T.rng.standard_normal(k)) * 1e-3 / 127.0 ** 2).astype(np.float32)
        q = (np.exp(T.rng.standard_normal(k)) * 1e-3 / 256.0 ** 2).astype(np.float32)
        for t, x in ((T.tm[i], c), (T.tv[i], d), (T.tms[i], s), (T.tvs[i], q)):
            t.copy_(torch.from_numpy(x))
        T.m[i], T.v[i] = ref.decode_m(c, s), ref.decode_v(d, q)
    return T


@pytest.mark.gpu
@pytest.mark.parametrize("gbf16", [True, False])
@pytest.mark.parametrize("seed", [None, 12])
@pytest.mark.parametrize("pbf16,copy,shift", [(False, False, 0), (False, True, 0), (True, False, 0), (False, True, 1),
                                              (True, False, 1)])
def test_several_blocks_a_warp(ctx, pbf16, copy, shift, seed, gbf16):
    import matrix_aware_optimizer_step_b200 as mx
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sum(-(-n // 256) for n in SIZES) // (sms * 32) >= 4
    T = with_moments(Tensors(SIZES, 50, pbf16, gbf16, True, copy, shift, zero=True))
    plan, gs = T.plan(ctx), T.new_grads()
    scale = torch.tensor([0.5], device="cuda")
    plan.step(20, mx.default_adamw_plan_hparams(beta2=0.99), grad_scale=scale, seed=seed)
    torch.cuda.synchronize()
    check_step(T, gs, 20, 0.9, 0.99, 3e-4, 1e-8, 0.01, 0.5, seed)
    T.guards_intact()
