"""Gradient norm and AdamW (32- and 8-bit states) against the formulas in 64
bits. u = 2^-24 is one fp32 rounding; each tolerance counts the roundings on the
path to the value."""
import math

import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
SIZES = [0, 1, 3, 127, 128, 129, 1023, 1024, 2047, 2048, 2049, 8191, 8192, 8193, 30011]
LR, BETAS, EPS, WD = 1e-2, (0.9, 0.95), 1e-8, 0.1
GUARD = 64


def guarded(values, offset=0):
    """The values at an odd place of a larger buffer, and a check that nothing around them changed."""
    n = values.numel()
    fill = 77
    buf = torch.full((n + 2 * GUARD + offset,), fill, dtype=values.dtype, device=DEV) \
        if values.dtype != torch.uint8 else torch.full((n + 2 * GUARD + offset,), 77, dtype=torch.uint8, device=DEV)
    view = buf[GUARD + offset:GUARD + offset + n]
    view.copy_(values)

    def intact():
        return bool((buf[:GUARD + offset] == fill).all()) and bool((buf[GUARD + offset + n:] == fill).all())
    return view, intact


def rand(n, std, seed, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(dtype).to(DEV)


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("offset", [0, 1])
def test_norm_of_all_sizes(dtype, offset):
    grads = [guarded(rand(n, 1.0, n, dtype), offset)[0] for n in SIZES]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    say("norm", dtype, offset)
    for subset in [grads] + [[g] for g in grads]:
        want = math.sqrt(sum(float(g.double().square().sum()) for g in subset))
        ctrl = dps.dp_grad_norm(subset, max_norm=0.5)
        # fp64 sums, one rounding to fp32
        assert abs(float(ctrl.norm) - want) <= 1.01 * U * want
        scale = 0.5 / want if want > 0.5 else 1.0
        assert abs(float(ctrl.scale) - scale) <= 1.01 * U * scale
        assert int(ctrl.step) == 1 and int(ctrl.skipped) == 0


def test_norm_over_many_tensors_and_again():
    """Three launches of one call; the workspace is ready for the next call; the same bits each time."""
    grads = [rand(100 + 37 * i, 1e-3, i, BF16) for i in range(300)]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    plan = dps.GradNorm(grads)
    got = []
    for i in range(4):
        say("norm many", i)
        ctrl = plan.run(max_norm=1e9)
        got.append(ctrl.norm.clone())
        assert abs(float(ctrl.norm) - want) <= 1.01 * U * want
        assert float(ctrl.scale) == 1.0 and int(ctrl.step) == i + 1
    assert all(torch.equal(g, got[0]) for g in got)


def test_norm_extremes():
    one = lambda *v: torch.tensor(v, device=DEV)
    assert float(dps.dp_grad_norm([]).norm) == 0.0
    zero = dps.dp_grad_norm([torch.zeros(5000, device=DEV)], max_norm=1.0)
    assert float(zero.norm) == 0.0 and float(zero.scale) == 1.0
    # squares that leave fp32 both ways
    big = dps.dp_grad_norm([one(3e30, 4e30)], max_norm=1.0)
    assert abs(float(big.norm) - 5e30) <= 2 * U * 5e30 and abs(float(big.scale) - 2e-31) <= 4 * U * 2e-31
    tiny = dps.dp_grad_norm([one(3e-40, 4e-40)], max_norm=1.0)
    assert abs(float(tiny.norm) - 5e-40) <= 2e-45 and float(tiny.scale) == 1.0
    for bad in (float("inf"), float("nan"), -float("inf")):
        g = torch.ones(9000, device=DEV)
        g[8999] = bad
        ctrl = dps.StepCtrl(step=4)
        dps.dp_grad_norm([torch.ones(5, device=DEV), g], ctrl, max_norm=1.0)
        assert float(ctrl.scale) == 0.0 and int(ctrl.step) == 4 and int(ctrl.skipped) == 1
    over = dps.dp_grad_norm([torch.full((9,), 3e38, device=DEV)])       # finite, its norm is not in fp32
    assert float(over.scale) == 0.0 and int(over.skipped) == 1


# ------------------------------------------------------------------ AdamW

def reference(p, g, m, v, t, clip=1.0):
    """The step in 64 bits, and what its fp32 roundings can add up to for each of its values."""
    b1, b2 = BETAS
    p, g, m, v = (x.double() for x in (p, g, m, v))
    g = g * clip
    m2 = b1 * m + (1 - b1) * g
    # beta, product, and for g also the clip: 3 roundings, then the sum
    em = 5 * U * (b1 * m.abs() + (1 - b1) * g.abs()) + 2 ** -149
    v2 = b2 * v + (1 - b2) * g * g
    ev = 7 * U * v2 + 2 ** -149
    den = (v2 / (1 - b2 ** t)).sqrt() + EPS
    lo = ((v2 - ev).clamp(min=0) / (1 - b2 ** t)).sqrt() * (1 - 4 * U) + EPS * (1 - 2 * U)
    step = LR / (1 - b1 ** t)
    new = p * (1 - LR * WD) - step * m2 / den
    ep = 4 * U * (p.abs() + new.abs()) + step * (em / lo + m2.abs() * (1 / lo - 1 / den).abs() + 12 * U * m2.abs() / den)
    return new, m2, v2, ep, em, ev


@pytest.mark.parametrize("p_dtype,g_dtype,copy", [(F32, F32, False), (F32, BF16, True), (BF16, BF16, False),
                                                  (BF16, F32, False)])
@pytest.mark.parametrize("offset", [0, 1])
def test_adamw_against_the_formula(p_dtype, g_dtype, copy, offset):
    ps, gs, ms, vs, cs, guards = [], [], [], [], [], []
    for n in SIZES:
        for into, std, dtype in ((ps, 1.0, p_dtype), (gs, 0.1, g_dtype), (ms, 0.05, F32), (vs, 0.02, F32),
                                 (cs, 1.0, BF16)):
            x = rand(n, std, n + len(guards), dtype)
            x, ok = guarded(x.square() if into is vs else x, offset)
            into.append(x)
            guards.append(ok)
    # an element without any history or gradient, and one whose state is zero
    gs[-1][:5] = 0
    ms[-1][:5] = 0
    vs[-1][:5] = 0
    ps0, ms0, vs0 = ([x.clone() for x in xs] for xs in (ps, ms, vs))
    say("adamw", p_dtype, g_dtype, offset)
    dps.dp_adamw(ps, gs, ms, vs, step=3, copies=cs if copy else None, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
    for i, n in enumerate(SIZES):
        new, m2, v2, ep, em, ev = reference(ps0[i], gs[i], ms0[i], vs0[i], 3)
        assert bool(((ms[i].double() - m2).abs() <= em).all()) and bool(((vs[i].double() - v2).abs() <= ev).all())
        half = 2.0 ** -8 * (new.abs() + ep) if p_dtype == BF16 else 0
        assert bool(((ps[i].double() - new).abs() <= ep + half).all()), n
        if copy:
            assert torch.equal(cs[i], ps[i].bfloat16())
    assert all(ok() for ok in guards)


def test_adamw_many_tensors_and_control_block():
    """Two launches; step number and clip factor from the device equal those given by the host."""
    k = 70
    make = lambda: ([rand(1000 + i, 1.0, i) for i in range(k)], [rand(1000 + i, 0.3, 99 + i) for i in range(k)],
                    [torch.zeros(1000 + i, device=DEV) for i in range(k)], [torch.zeros(1000 + i, device=DEV) for i in range(k)])
    a, b = make(), make()
    kw = dict(lr=LR, betas=BETAS, eps=EPS, weight_decay=WD)
    plan = dps.AdamW(*b, **kw)
    ctrl = dps.StepCtrl()
    norm = dps.GradNorm(b[1], ctrl)
    for t in range(1, 4):
        say("adamw control", t)
        norm.run(max_norm=2.0)
        scale = float(ctrl.scale)
        assert 0 < scale < 1 and int(ctrl.step) == t
        plan.step(ctrl=ctrl)
        dps.dp_adamw(a[0], [g * ctrl.scale for g in a[1]], a[2], a[3], step=t, **kw)
        for x, y in zip(a[0] + a[2] + a[3], b[0] + b[2] + b[3]):
            assert torch.allclose(x, y, rtol=8 * U, atol=1e-30)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_with_a_bad_gradient_changes_nothing(bits):
    p = [rand(5000, 1.0, 1), rand(33, 1.0, 2)]
    g = [rand(5000, 1.0, 3), torch.full((33,), float("nan"), device=DEV)]
    m, v, s = dps.AdamW.new_state(p, bits)
    plan = dps.AdamW(p, g, m, v, scales=s, lr=LR)
    ctrl = dps.StepCtrl()
    norm = dps.GradNorm(g, ctrl)
    before = [x.clone() for x in p + m + v]
    norm.run(1.0)
    plan.step(ctrl=ctrl)
    assert all(torch.equal(x, y) for x, y in zip(before, p + m + v)) and int(ctrl.skipped) == 1
    g[1].fill_(0.5)
    norm.run(1.0)
    plan.step(ctrl=ctrl)
    assert int(ctrl.step) == 1 and not any(torch.equal(x, y) for x, y in zip(before, p + m + v))


# ------------------------------------------------------------------ 8-bit states

def spread(scales, n, at):
    return scales.view(-1, 2)[:, at].double().repeat_interleave(128)[:n]


def held(x, scales, at):
    """What 8-bit codes stand for."""
    return x.view(torch.float8_e4m3fn).float().double() * spread(scales, x.numel(), at)


def eight_bit_state(n, seed):
    m, r = rand(n, 0.05, seed), rand(n, 0.1, seed + 1).abs()
    b = -(-n // 128)
    pad = lambda x: torch.nn.functional.pad(x, (0, 128 * b - n)).view(b, 128)
    s = torch.stack([pad(m).abs().amax(1), pad(r).amax(1)], 1) / 448 if b else torch.zeros(0, 2, device=DEV)
    code = lambda x, at: (x / spread(s, n, at).float().clamp(min=1e-30)).to(torch.float8_e4m3fn).view(torch.uint8)
    return code(m, 0), code(r, 1), s


@pytest.mark.parametrize("seed", [None, 0, 12345])
@pytest.mark.parametrize("p_dtype,g_dtype,offset", [(F32, BF16, 0), (BF16, F32, 1), (F32, F32, 3)])
def test_adamw8_against_the_formula(seed, p_dtype, g_dtype, offset):
    ps, gs, ms, vs, ss, cs, guards = [], [], [], [], [], [], []
    for n in SIZES:
        m, v, s = eight_bit_state(n, 5 * n)
        for into, x in ((ps, rand(n, 1.0, n + 1, p_dtype)), (gs, rand(n, 0.1, n + 2, g_dtype)), (ms, m), (vs, v),
                        (cs, rand(n, 1.0, n + 3, BF16))):
            x, ok = guarded(x, offset)
            into.append(x)
            guards.append(ok)
        s, ok = guarded(s.view(-1), 2)
        ss.append(s)
        guards.append(ok)
    ps0, ms0, vs0, ss0 = ([x.clone() for x in xs] for xs in (ps, ms, vs, ss))
    copies = cs if p_dtype == F32 else None
    kw = dict(scales=ss, copies=copies, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD, seed=seed)
    say("adamw8", seed, p_dtype, g_dtype, offset)
    dps.dp_adamw(ps, gs, ms, vs, step=7, **kw)
    for i, n in enumerate(SIZES):
        if n == 0:
            continue
        m0, v0 = held(ms0[i], ss0[i], 0), held(vs0[i], ss0[i], 1).square()
        new, m2, v2, ep, em, ev = reference(ps0[i], gs[i], m0, v0, 7)
        # the product with the scale, and for v its square, are rounded too
        em, ev = em + 2 * U * m0.abs(), ev + 4 * U * v0
        ep = ep + LR / (1 - BETAS[0] ** 7) * (2 * U * m0.abs() + 4 * U * m2.abs()) / ((v2 / (1 - BETAS[1] ** 7)).sqrt() + EPS)
        half = 2.0 ** -8 * (new.abs() + ep) if p_dtype == BF16 else 0
        assert bool(((ps[i].double() - new).abs() <= ep + half).all()), n
        if copies:
            assert torch.equal(cs[i], ps[i].bfloat16())
        r2 = v2.sqrt()
        blocks = -(-n // 128)
        top = lambda x: torch.nn.functional.pad(x, (0, 128 * blocks - n)).view(blocks, 128).abs().amax(1)
        for at, x, e in ((0, m2, em), (1, r2, 6 * U * r2)):
            s = ss[i].view(-1, 2)[:, at].double()
            assert bool(((s * 448 - top(x)).abs() <= top(e) + 4 * U * top(x)).all())
            codes = (ms, vs)[at][i]
            # half a step to nearest, a whole one at random: 2^-4 of the value or 2^-10 of the scale
            steps = 1 if seed is None else 2
            slack = steps * (2.0 ** -4 * x.abs() + 2.0 ** -10 * spread(ss[i], n, at)) * (1 + 8 * U) + 2 * e
            off = (held(codes, ss[i], at) - x).abs()
            if at == 1:          # raised to the smallest code
                slack = torch.maximum(slack, 2.0 ** -9 * spread(ss[i], n, at) * (x > 0))
                assert bool((codes[x > 0] != 0).all())
            assert bool((off <= slack).all()), (n, at)
    assert all(ok() for ok in guards)


def test_random_rounding_is_reproducible_and_unbiased():
    n = 1 << 20
    p, g = torch.zeros(n, device=DEV), torch.full((n,), 0.1, device=DEV)
    g[::128] = 1.0                                   # the blocks' scale: 0.1 lies between two codes

    def run(seed, step):
        m, v, s = dps.AdamW.new_state([p], 8)
        dps.dp_adamw([p.clone()], [g], m, v, step=step, scales=s, lr=0.0, betas=(0.5, 0.5), seed=seed)
        return m[0], v[0], s[0]
    a, b, c, d = run(1, 1), run(1, 1), run(2, 1), run(1, 2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert not torch.equal(a[0], c[0]) and not torch.equal(a[0], d[0])
    for at, want in ((0, 0.05), (1, math.sqrt(0.5) * 0.1)):
        x = held(a[at], a[2], at)
        x = x[torch.arange(n, device=DEV) % 128 != 0]
        codes = x.unique()
        assert codes.numel() == 2 and codes[0] < want < codes[1]
        # a mean of N draws of two values a step apart: five standard errors, and r's 2^-16 grid
        step = float(codes[1] - codes[0])
        assert abs(float(x.mean()) - want) <= 5 * 0.5 * step / math.sqrt(x.numel()) + step * 2.0 ** -16
    # m and v of an element, and neighbours, draw their own bits
    up = [(held(a[at], a[2], at) > (0.05, math.sqrt(0.5) * 0.1)[at]).double() for at in (0, 1)]
    keep = torch.arange(n, device=DEV) % 128 > 1
    corr = lambda x, y: float(torch.corrcoef(torch.stack([x, y]))[0, 1])
    assert abs(corr(up[0][keep], up[1][keep])) < 0.01
    assert abs(corr(up[0][keep], up[0].roll(1)[keep])) < 0.01


def test_random_rounding_goes_by_a_tensors_place_in_the_call():
    """The second launch of a long list goes on counting: a tensor rounds as it does in a list of empty ones."""
    k, n, one = 70, 700, 66
    g = [rand(n, 0.1, i) for i in range(k)]

    def run(keep):
        gs = [x if keep(i) else x[:0] for i, x in enumerate(g)]
        p = [torch.zeros_like(x) for x in gs]
        m, v, s = dps.AdamW.new_state(p, 8)
        dps.dp_adamw(p, gs, m, v, step=2, scales=s, lr=LR, seed=11)
        return m[one], v[one]
    whole, alone = run(lambda i: True), run(lambda i: i == one)
    assert torch.equal(whole[0], alone[0]) and torch.equal(whole[1], alone[1])
    other = [g[one]] * k
    p = [torch.zeros_like(x) for x in other]
    m, v, s = dps.AdamW.new_state(p, 8)
    dps.dp_adamw(p, other, m, v, step=2, scales=s, lr=LR, seed=11)
    assert torch.equal(m[one], whole[0]) and not torch.equal(m[one], m[one - 64]) and not torch.equal(m[1], m[2])


def test_8_bit_training_follows_32_bit_training():
    """200 steps on a quadratic with beta2 = 0.999: random rounding keeps the second moment moving."""
    n = 4096
    target, curve = rand(n, 1.0, 5), 10 ** rand(n, 0.5, 6)
    ends = []
    for bits, seed in ((32, None), (8, 3)):
        p = [torch.zeros(n, device=DEV)]
        g = [torch.empty(n, device=DEV)]
        m, v, s = dps.AdamW.new_state(p, bits)
        plan = dps.AdamW(p, g, m, v, scales=s, lr=2e-2, betas=(0.9, 0.999), weight_decay=0.0, seed=seed)
        for t in range(1, 201):
            g[0].copy_(curve * (p[0] - target))
            plan.step(step=t)
        ends.append(float((curve * (p[0] - target).square()).mean()))
    start = float((curve * target.square()).mean())
    say("quadratic", start, ends)
    assert ends[0] < 0.01 * start and ends[1] < 0.02 * start


def test_no_state_of_a_zero_block_is_lost_or_invented():
    p, g = [torch.ones(300, device=DEV)], [torch.zeros(300, device=DEV)]
    m, v, s = dps.AdamW.new_state(p, 8)
    dps.dp_adamw(p, g, m, v, step=1, scales=s, lr=LR, weight_decay=0.0)
    assert bool((p[0] == 1).all()) and not bool(m[0].any() | v[0].any()) and not bool(s[0].any())
    g[0][130] = 1e-38                                # below 2^-100: held as zeros, with its root
    dps.dp_adamw(p, g, m, v, step=2, scales=s, lr=LR, weight_decay=0.0)
    assert not bool(m[0].any()) and bool(torch.isfinite(s[0]).all()) and bool(torch.isfinite(p[0]).all())


@pytest.mark.parametrize("seed", [None, 4])
def test_non_finite_gradients_without_a_control_block(seed):
    """NaNs of any payload stay with their element, an infinity spoils its block, and no other block."""
    n = 128 * 6
    g = torch.full((n,), 0.25, device=DEV)
    bits = g.view(torch.int32)
    bits[3], bits[130], bits[131] = 0x7FFFFFFF, 0x7FC00000, -1
    g[400] = float("inf")
    p = [torch.zeros(n, device=DEV)]
    m, v, s = dps.AdamW.new_state(p, 8)
    dps.dp_adamw(p, [g], m, v, step=1, scales=s, lr=LR, seed=seed)
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[3] = bad[130] = bad[131] = bad[384:512] = True
    for at, x in ((0, m[0]), (1, v[0])):
        assert torch.equal(held(x, s[0], at).isnan(), bad)
    bad[384:512] = False
    assert torch.equal(p[0].isnan() | (torch.arange(n, device=DEV) == 400), bad | (torch.arange(n, device=DEV) == 400))


def test_the_step_in_a_graph():
    """Norm and update captured once; each replay counts its step on the device and equals the eager call."""
    def make():
        p = [rand(3000 + 5 * i, 1.0, i) for i in range(3)]
        g = [torch.zeros(3000 + 5 * i, dtype=BF16, device=DEV) for i in range(3)]
        m, v, s = dps.AdamW.new_state(p, 8)
        c = [x.bfloat16() for x in p]
        ctrl = dps.StepCtrl()
        return g, p + m + v + s + c, dps.GradNorm(g, ctrl), dps.AdamW(p, g, m, v, copies=c, scales=s, seed=9, lr=LR), ctrl
    eager, graphed = make(), make()
    dps.lib()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        graphed[2].run(1.0)
        graphed[3].step(ctrl=graphed[4])
    for t in range(5):
        for i in range(3):
            x = rand(3000 + 5 * i, 0.5, 10 * t + i, BF16)
            if t == 2:
                x[7] = float("inf")
            eager[0][i].copy_(x)
            graphed[0][i].copy_(x)
        say("graph replay", t)
        graph.replay()
        torch.cuda.synchronize()
        eager[2].run(1.0)
        eager[3].step(ctrl=eager[4])
        assert torch.equal(eager[4].buf, graphed[4].buf)
        assert all(torch.equal(a, b) for a, b in zip(eager[1], graphed[1]))
    assert int(eager[4].step) == 4 and int(eager[4].skipped) == 1


def test_on_another_stream():
    s = torch.cuda.Stream()
    p, g = [rand(100000, 1.0, 1)], [rand(100000, 1.0, 2)]
    q = [p[0].clone()]
    m, v, _ = dps.AdamW.new_state(p)
    m2, v2, _ = dps.AdamW.new_state(p)
    torch.cuda.synchronize()
    ctrl = dps.dp_grad_norm(g, max_norm=1.0, stream=s)
    dps.dp_adamw(p, g, m, v, ctrl=ctrl, stream=s)
    s.synchronize()
    dps.dp_adamw(q, g, m2, v2, ctrl=ctrl)
    assert torch.equal(p[0], q[0])


def test_beyond_32_bits():
    """A tensor of more than 2^31 elements: its end equals the same elements updated by themselves."""
    n, k = 2 ** 31 + 2048 * 5 + 77, 128 * 50 + 77
    cut = n - k                                      # a multiple of 128
    assert cut % 128 == 0
    p, g = torch.full((n,), 0.5, dtype=BF16, device=DEV), torch.full((n,), 0.25, dtype=BF16, device=DEV)
    p[cut:] = rand(k, 1.0, 1, BF16)
    g[cut:] = rand(k, 1.0, 2, BF16)
    m, v, s = dps.AdamW.new_state([p], 8)
    small = [p[cut:].clone()]
    ms, vs, ss = dps.AdamW.new_state(small, 8)
    say("beyond 32 bits")
    ctrl = dps.dp_grad_norm([g])
    want = math.sqrt(cut * 0.0625 + float(g[cut:].double().square().sum()))
    assert abs(float(ctrl.norm) - want) <= 2 * U * want
    dps.dp_adamw([p], [g], m, v, step=1, scales=s, lr=LR)
    dps.dp_adamw(small, [g[cut:].clone()], ms, vs, step=1, scales=ss, lr=LR)
    assert torch.equal(p[cut:], small[0]) and torch.equal(m[0][cut:], ms[0]) and torch.equal(v[0][cut:], vs[0])
    assert torch.equal(s[0][cut // 128:], ss[0]) and bool((p[:cut] == p[0]).all())
