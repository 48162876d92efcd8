"""What the optimizer-state operators compute, and the calls that use them.

Four operators that an AdamW group of many tensors needs each step:

  norm      the 2-norm over every gradient of the group and the factor that
            clips it: norm = sqrt(sum g^2), factor = min(1, max_norm / (norm + 1e-6))
  adamw32   an AdamW step over all tensors with both moments in fp32, on bf16
            parameters or on fp32 parameters with a bf16 working copy
  adamw8    the same step with both moments in 8 bits, one fp32 scale for
            each 256 elements
  state8    the conversion of fp32 moments into the 8-bit form and back

The 8-bit form of 256 consecutive elements of one tensor:

  first moment, signed:     m = c |c| s,           c in -127 .. 127, s = max|m| / 127^2
  second moment, unsigned:  sqrt(v) = (c + 1)^2 s, c in 0 .. 255,    s = max sqrt(v) / 256^2

and a code is floor(y + u), y the exact real-valued code and u = 1/2 (nearest)
or a number in (0, 1) hashed from a seed, the step, the tensor and the element
(stochastic, unbiased in y).

With `own` false, run() computes this with elementary torch operations in
32 bits; with `own` true it makes the calls a training loop makes.
"""

import math

import torch

own = False

BLOCK = 256
LR, BETA1, BETA2, EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.01
M32 = 0xFFFFFFFF
TINY = 2.0 ** -100        # a block whose largest magnitude is below this is stored as zero

_context = None


def _ctx():
    global _context
    if _context is None:
        from matrix_aware_optimizer_step_b200 import MuonContext
        _context = MuonContext(torch.cuda.current_device())
    return _context


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    base = dict(rows=0, cols=0, vectors=0, length=0, ragged=False, grad="bf16", param="f32", copy=False,
                stochastic=False, clip=False, beta2=BETA2, step=10)
    embed = dict(rows=50257, cols=768, vectors=100, length=768)        # a small decoder's embedding, gains and biases
    head = dict(rows=128256, cols=4096, vectors=65, length=4096)       # a large decoder's embedding and RMS-norm gains
    cases = [
        # one gain vector: the least a call can do, all latency
        dict(name="norm one vector", op="norm", vectors=1, length=768),
        # the clipping pass of a small model's aux group
        dict(embed, name="norm small decoder", op="norm"),
        # fp32 gradients accumulated over micro-batches, a large model's aux group
        dict(head, name="norm large decoder f32", op="norm", grad="f32"),
        # every gain of a decoder in pure bf16 training: many short tensors, little work
        dict(name="adamw32 gains bf16", op="adamw32", vectors=65, length=4096, param="bf16"),
        # pure bf16 training with stochastic rounding, clipped
        dict(embed, name="adamw32 small decoder bf16", op="adamw32", param="bf16", stochastic=True, clip=True),
        # fp32 master weights with the bf16 copy that the next forward pass reads
        dict(head, name="adamw32 large decoder copy", op="adamw32", copy=True),
        # one odd-sized tensor: latency again
        dict(name="adamw8 one tensor", op="adamw8", vectors=1, length=1000, grad="f32"),
        # hundreds of ragged biases: tensors that end inside a block
        dict(name="adamw8 ragged biases", op="adamw8", vectors=300, length=5000, ragged=True, grad="f32", beta2=0.999),
        # the ordinary 8-bit step: clipped, rounded stochastically as beta2 = 0.999 needs
        dict(embed, name="adamw8 small decoder", op="adamw8", stochastic=True, clip=True, beta2=0.999),
        # the largest: embedding of a large decoder, master weights and their copy
        dict(head, name="adamw8 large decoder copy", op="adamw8", copy=True),
        # a 32-bit checkpoint taken into 8 bits and read back
        dict(name="state8 ragged biases", op="state8", vectors=300, length=5000, ragged=True),
        dict(embed, name="state8 small decoder", op="state8"),
    ]
    return [dict(base, **c) for c in cases]


def draw(rng):
    op = rng.choice(["norm", "adamw32", "adamw8", "adamw8", "state8"])
    c = dict(op=op, rows=0, cols=0, vectors=0, length=0, ragged=False, grad=rng.choice(["bf16", "f32"]), param="f32",
             copy=False, stochastic=False, clip=False, beta2=rng.choice([0.95, 0.99, 0.999]), step=rng.randint(1, 5000))
    if op in ("adamw32", "adamw8"):
        c["param"] = rng.choice(["f32", "bf16"])
        c["copy"] = c["param"] == "f32" and rng.random() < 0.4
        c["clip"] = rng.random() < 0.4
        c["stochastic"] = (op == "adamw8" or c["param"] == "bf16") and rng.random() < 0.5
    if rng.random() < 0.6:
        # a matrix of up to 2^26 elements (2^24 where the plain form hashes in 64-bit integers)
        total = 2.0 ** rng.uniform(8, 24 if c["stochastic"] else 26)
        c["cols"] = max(1, min(int(2.0 ** rng.uniform(4, 13)), int(total)))
        c["rows"] = max(1, int(total / c["cols"]))
    if not c["rows"] or rng.random() < 0.5:
        c["vectors"] = max(1, int(2.0 ** rng.uniform(0, 9)))
        c["length"] = max(1, int(2.0 ** rng.uniform(0, 14)))
        c["ragged"] = rng.random() < 0.6
    return c


def sizes(case):
    s = [case["rows"] * case["cols"]] if case["rows"] else []
    n = case["length"]
    return s + [1 + (i * 7919 + 13) % n if case["ragged"] else n for i in range(case["vectors"])]


def _layout(case):
    """(numel of each tensor, its place in the flat buffer, the buffer's length): every tensor starts on a block."""
    ns, at, places = sizes(case), 0, []
    for n in ns:
        places.append(at)
        at += (n + BLOCK - 1) // BLOCK * BLOCK
    return ns, places, at


def work(case):
    n = sum(sizes(case))
    g = 2 if case["grad"] == "bf16" else 4
    if case["op"] == "norm":
        return {"bytes": g * n + 8, "flops": 2 * n}
    scales = 2 * 4 * sum((x + BLOCK - 1) // BLOCK for x in sizes(case))
    if case["op"] == "state8":
        return {"bytes": n * 2 * (4 + 1 + 2) + scales, "flops": 12 * n}      # fp32 in; codes and bf16 values out
    p = 2 * (2 if case["param"] == "bf16" else 4) + (2 if case["copy"] else 0)
    if case["op"] == "adamw32":
        return {"bytes": n * (g + p + 16), "flops": 14 * n}
    return {"bytes": n * (g + p + 4 + 4) + 2 * scales, "flops": 30 * n}      # codes in and out, bf16 values out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inputs(case, seed):
    """Flat buffers: gradients with the spread between tensors and the untouched rows that training has, moments that
    fit them, weights."""
    ns, places, total = _layout(case)
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(std=1.0):
        return torch.randn(total, generator=gen, device=dev, dtype=torch.float32).mul_(std)

    inside = torch.zeros(total, device=dev, dtype=torch.bool)
    for n, at in zip(ns, places):
        inside[at:at + n] = True
    row = case["cols"] if case["rows"] else 64
    nrows = (total + row - 1) // row
    # rows of an embedding that this step's tokens do not touch have no gradient
    seen = torch.rand(nrows, generator=gen, device=dev) < 0.6
    level = torch.exp(torch.randn(nrows, generator=gen, device=dev)) * 1e-3
    level = (level * seen).repeat_interleave(row)[:total] * inside
    s = dict(case=case, ns=ns, places=places, total=total, inside=inside)
    grad = normal() * level
    s["grad"] = grad.bfloat16() if case["grad"] == "bf16" else grad
    if case["op"] == "norm":
        return s
    # moments: every row was seen at some time, except a tenth of them
    old = torch.exp(torch.randn(nrows, generator=gen, device=dev)) * 1e-3
    old = old * (torch.rand(nrows, generator=gen, device=dev) < 0.9)
    old = old.repeat_interleave(row)[:total] * inside
    if case["op"] in ("adamw32", "state8"):
        s["m"] = normal(0.3) * old
        s["v"] = (normal().abs_().add_(0.05) * old).square_()
    else:
        blocks = total // BLOCK
        z = (normal() * inside).clamp_(-3.9, 3.9)
        s["m"] = (z.sign() * (z.abs() / 3.9).sqrt().mul_(127.0).round_()).to(torch.int8)
        z = normal().abs_().add_(0.02).clamp_(max=3.9)
        s["v"] = (z / 3.9).sqrt().mul_(255.0).round_().mul_(inside).to(torch.uint8)
        s["m_scale"] = old.view(blocks, BLOCK).amax(1) * (1.2 / 16129.0)
        s["v_scale"] = old.view(blocks, BLOCK).amax(1) * (3.9 / 65536.0)
    if case["op"] != "state8":
        p = normal(0.02) * inside
        s["param"] = p.bfloat16() if case["param"] == "bf16" else p
        if case["copy"]:
            s["copy"] = s["param"].bfloat16()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["step"] = case["step"] - 1
    s["seed"] = int(seed) & 0x7FFFFFFF
    dev = s["grad"].device
    if case["op"] == "state8":
        blocks = s["total"] // BLOCK
        s["m_code"] = torch.zeros(s["total"], device=dev, dtype=torch.int8)
        s["v_code"] = torch.zeros(s["total"], device=dev, dtype=torch.uint8)
        s["m_scale"] = torch.zeros(blocks, device=dev)
        s["v_scale"] = torch.zeros(blocks, device=dev)
    if case["op"] in ("adamw8", "state8"):
        s["m_out"] = torch.zeros(s["total"], device=dev, dtype=torch.bfloat16)
        s["v_out"] = torch.zeros(s["total"], device=dev, dtype=torch.bfloat16)
    if own:
        _plans(s)
    return s


def _plans(s):
    """The handles a training loop builds once over its tensors."""
    case, ctx = s["case"], _ctx()

    def parts(key):
        return [s[key][at:at + n] for n, at in zip(s["ns"], s["places"])]

    def scales(key):
        return [s[key][at // BLOCK:at // BLOCK + (n + BLOCK - 1) // BLOCK] for n, at in zip(s["ns"], s["places"])]

    op = case["op"]
    if op == "norm" or case["clip"]:
        s["norm_plan"] = ctx.grad_norm_plan(parts("grad"))
    if op == "adamw32":
        s["plan"] = ctx.adamw_plan(parts("param"), parts("grad"), parts("m"), parts("v"),
                                   param_copies=parts("copy") if case["copy"] else None)
    if op == "adamw8":
        s["plan"] = ctx.adamw_plan(parts("param"), parts("grad"), parts("m"), parts("v"),
                                   exp_avg_scales=scales("m_scale"), exp_avg_sq_scales=scales("v_scale"),
                                   param_copies=parts("copy") if case["copy"] else None)
        s["values"] = ctx.state8_plan(parts("m_out") + parts("v_out"), parts("m") + parts("v"),
                                      scales("m_scale") + scales("v_scale"))
    if op == "state8":
        s["pack"] = ctx.state8_plan(parts("m") + parts("v"), parts("m_code") + parts("v_code"),
                                    scales("m_scale") + scales("v_scale"))
        s["values"] = ctx.state8_plan(parts("m_out") + parts("v_out"), parts("m_code") + parts("v_code"),
                                      scales("m_scale") + scales("v_scale"))
    if op in ("adamw32", "adamw8"):
        from matrix_aware_optimizer_step_b200 import default_adamw_plan_hparams
        s["hp"] = default_adamw_plan_hparams(lr=LR, beta1=BETA1, beta2=case["beta2"], eps=EPS, weight_decay=DECAY)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    state["step"] += 1
    if own:
        if op == "norm":
            return state["norm_plan"].run(max_norm=1.0)
        if op == "state8":
            state["pack"].pack()
            state["values"].unpack()
            return {"m": state["m_out"], "v": state["v_out"]}
        factor = state["norm_plan"].run(max_norm=1.0) if case["clip"] else None
        state["plan"].step(state["step"], state["hp"], grad_scale=None if factor is None else factor[1:],
                           seed=state["seed"] if case["stochastic"] else None)
        out = {"param": state["param"]}
        if case["copy"]:
            out["copy"] = state["copy"]
        if op == "adamw32":
            out.update(m=state["m"], v=state["v"])
        else:
            state["values"].unpack()
            out.update(m=state["m_out"], v=state["v_out"])
        if factor is not None:
            out["norm"] = factor
        return out
    return _plain(state)


def _plain_norm(grad, max_norm):
    # squares of fp32 gradients below 1e-19 or above 1e19 leave the range of 32 bits, and a sum of 5e8 terms its
    # precision: 64 bits, which bf16 and fp32 values square into exactly
    norm = grad.double().square().sum().sqrt()
    factor = torch.clamp(max_norm / (norm + 1e-6), max=1.0)
    return torch.stack([norm, factor]).float()


def _mix(x):
    """A 32-bit xorshift-multiply mixer on integers kept in 64 bits."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _dither(state):
    """Hashed 16-bit numbers for every element of the flat buffer: (for v, for m, for the parameter)."""
    ns, total = state["ns"], state["total"]
    dev = state["grad"].device
    ids = torch.arange(len(ns), device=dev)
    widths = torch.tensor([(n + BLOCK - 1) // BLOCK * BLOCK for n in ns], device=dev)
    key = _mix((ids + _mix((_mix(torch.tensor(state["seed"], device=dev)) + state["step"]) & M32)) & M32)
    key = key.repeat_interleave(widths, output_size=total)
    start = torch.tensor(state["places"], device=dev).repeat_interleave(widths, output_size=total)
    place = torch.arange(total, device=dev) - start
    pair = place >> 1
    odd = (place & 1) * 16
    word = _mix((((pair & M32) ^ key) + (pair >> 32) * 0x9E3779B9) & M32)
    h = (word >> odd) & 0xFFFF
    hp = (_mix(word ^ 0x5BD1E995) >> odd) & 0xFFFF
    return h, ((h >> 8) | (h << 8)) & 0xFFFF, hp


def _unit(h):
    return 0.5 if h is None else (h.float() + 0.5) * (1.0 / 65536.0)


def _encode(values, u, top, bottom):
    """Codes floor(sqrt(values / s) + u) in bottom .. top and the scales s = max / top^2 of nonnegative values."""
    x = values.view(-1, BLOCK)
    biggest = x.amax(1, keepdim=True)
    fine = (biggest >= TINY) & torch.isfinite(biggest)
    s = biggest * (1.0 / (top * top))
    s = torch.where(fine, s, torch.where(torch.isfinite(biggest), torch.zeros_like(s), torch.full_like(s, math.nan)))
    y = (x * s.reciprocal()).sqrt()
    if not isinstance(u, float):
        u = u.view(-1, BLOCK)
    t = torch.where(fine, torch.floor(y + u).clamp(bottom, top), torch.full_like(y, bottom))
    return t.reshape(-1), s.reshape(-1)


def _encode_m(m, u):
    t, s = _encode(m.abs(), u, 127.0, 0.0)
    return (t * m.sign()).to(torch.int8), s


def _encode_r(r, u):
    t, s = _encode(r, u, 256.0, 1.0)
    return (t - 1.0).to(torch.uint8), s


def _value_m(code, s):
    c = code.float().view(-1, BLOCK)
    return ((c * c.abs()) * s[:, None]).reshape(-1)


def _value_r(code, s):
    c = (code.float() + 1.0).view(-1, BLOCK)
    return ((c * c) * s[:, None]).reshape(-1)


def _round_bf16(p, h):
    """fp32 to bf16: nearest, or up in magnitude with the probability of the dropped bits."""
    if h is None:
        return p.bfloat16()
    bits = (p.view(torch.int32).to(torch.int64) & M32) + h
    bits = (bits & 0xFFFF0000)
    bits = torch.where(bits >= 0x80000000, bits - 0x100000000, bits).to(torch.int32)
    return bits.view(torch.float32).bfloat16()


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(state["grad"], 1.0)
    if op == "state8":
        mc, ms = _encode_m(state["m"], 0.5)
        vc, vs = _encode_r(state["v"].sqrt(), 0.5)
        v = _value_r(vc, vs).square() * state["inside"]
        return {"m": _value_m(mc, ms).bfloat16(), "v": v.bfloat16()}
    g = state["grad"].float()
    norm = None
    if case["clip"]:
        norm = _plain_norm(state["grad"], 1.0)
        g = g * norm[1]
    if op == "adamw32":
        m, v = state["m"], state["v"]
    else:
        m = _value_m(state["m"], state["m_scale"])
        v = _value_r(state["v"], state["v_scale"]).square()
    b1, b2, t = BETA1, case["beta2"], state["step"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = v.sqrt()
    upd = m / (r * (1.0 / math.sqrt(1.0 - b2 ** t)) + EPS)
    p = state["param"].float() * (1.0 - LR * DECAY) - upd * (LR / (1.0 - b1 ** t))
    hv, hm, hp = _dither(state) if case["stochastic"] else (None, None, None)
    state["param"].copy_(_round_bf16(p, hp) if case["param"] == "bf16" else p)
    out = {"param": state["param"]}
    if case["copy"]:
        state["copy"].copy_(p)
        out["copy"] = state["copy"]
    if op == "adamw32":
        state["m"].copy_(m)
        state["v"].copy_(v)
        out.update(m=state["m"], v=state["v"])
    else:
        code, s = _encode_m(m, _unit(hm))
        state["m"].copy_(code)
        state["m_scale"].copy_(s)
        code, s = _encode_r(r, _unit(hv))
        state["v"].copy_(code)
        state["v_scale"].copy_(s)
        v = _value_r(state["v"], state["v_scale"]).square() * state["inside"]
        out.update(m=_value_m(state["m"], state["m_scale"]).bfloat16(), v=v.bfloat16())
    if norm is not None:
        out["norm"] = norm
    return out


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _hash32(x):
    x = torch.bitwise_xor(x, torch.div(x, 1 << 16, rounding_mode="floor"))
    x = (x * 0x7FEB352D) % (1 << 32)
    x = torch.bitwise_xor(x, torch.div(x, 1 << 15, rounding_mode="floor"))
    lo, hi = x % (1 << 16), torch.div(x, 1 << 16, rounding_mode="floor")
    x = (lo * 0x846CA68B + ((hi * 0x846CA68B) % (1 << 16)) * (1 << 16)) % (1 << 32)
    return torch.bitwise_xor(x, torch.div(x, 1 << 16, rounding_mode="floor"))


def _quantised(x, u, levels, low, signed):
    """Values that the 8-bit form keeps of one tensor x (signed: moments; else square roots of second moments)."""
    n = x.numel()
    pad = -n % BLOCK
    x = torch.cat([x, x.new_zeros(pad)]).view(-1, BLOCK)
    u = torch.cat([u, u.new_zeros(pad)]).view(-1, BLOCK) if torch.is_tensor(u) else u
    mag = x.abs()
    big = mag.max(dim=1, keepdim=True).values
    code = torch.floor(levels * torch.sqrt(mag / torch.where(big > 0, big, torch.ones_like(big))) + u)
    code = torch.minimum(torch.maximum(code, torch.full_like(code, low)), torch.full_like(code, levels))
    val = (code / levels) ** 2 * big
    return ((val * torch.sign(x)) if signed else val).reshape(-1)[:n]


def exact(case, seed):
    s = _inputs(case, seed)
    op, t, seed = case["op"], case["step"], int(seed) & 0x7FFFFFFF
    norm = None
    if op == "norm" or case["clip"]:
        total = sum(float((s["grad"][i:i + (1 << 26)].double() ** 2).sum()) for i in range(0, s["total"], 1 << 26))
        norm = torch.tensor([math.sqrt(total), min(1.0, 1.0 / (math.sqrt(total) + 1e-6))], dtype=torch.float64)
        if op == "norm":
            return norm
    names = ["m", "v"] if op == "state8" else ["param", "m", "v"] + (["copy"] if case["copy"] else [])
    out = {k: torch.zeros(s["total"], dtype=torch.float64, device=s["grad"].device) for k in names}
    dev = s["grad"].device
    for k, (n, at) in enumerate(zip(s["ns"], s["places"])):
        for lo in range(0, n, 1 << 26):
            hi = min(n, lo + (1 << 26))
            cut = slice(at + lo, at + hi)
            if op == "state8":
                out["m"][cut] = _quantised(s["m"][cut].double(), 0.5, 127.0, 0.0, True)
                out["v"][cut] = _quantised(s["v"][cut].double().sqrt(), 0.5, 256.0, 1.0, False) ** 2
                continue
            g = s["grad"][cut].double() * (1.0 if norm is None else float(norm[1]))
            if op == "adamw32":
                m, v = s["m"][cut].double(), s["v"][cut].double()
            else:
                blocks = torch.arange(lo, hi, device=dev) // BLOCK + at // BLOCK
                c, d = s["m"][cut].double(), s["v"][cut].double() + 1.0
                m = torch.sign(c) * c ** 2 * s["m_scale"].double()[blocks]
                v = (d ** 2 * s["v_scale"].double()[blocks]) ** 2
            m = BETA1 * m + (1.0 - BETA1) * g
            v = case["beta2"] * v + (1.0 - case["beta2"]) * g ** 2
            step = (m / (1.0 - BETA1 ** t)) / (torch.sqrt(v / (1.0 - case["beta2"] ** t)) + EPS)
            p = s["param"][cut].double()
            p = p - LR * DECAY * p - LR * step
            out["param"][cut] = p
            if case["copy"]:
                out["copy"][cut] = p
            um = uv = 0.5
            if case["stochastic"] and op == "adamw8":
                a = _hash32(torch.tensor(seed, device=dev))
                a = _hash32((a + t) % (1 << 32))
                a = _hash32((a + k) % (1 << 32))
                i = torch.arange(lo, hi, device=dev)
                w = _hash32(torch.bitwise_xor(torch.div(i, 2, rounding_mode="floor"), a))
                h = torch.where(i % 2 == 1, torch.div(w, 1 << 16, rounding_mode="floor"), w % (1 << 16))
                uv = (h.double() + 0.5) / 65536.0
                um = (torch.div(h, 256, rounding_mode="floor") + (h % 256) * 256).double().add(0.5) / 65536.0
            out["m"][cut] = m if op == "adamw32" else _quantised(m, um, 127.0, 0.0, True)
            out["v"][cut] = v if op == "adamw32" else _quantised(torch.sqrt(v), uv, 256.0, 1.0, False) ** 2
    if norm is not None:
        out["norm"] = norm
    return out
