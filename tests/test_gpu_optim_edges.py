"""Gradient norm and AdamW where fp32 gets thin: subnormal second moments, states that are not numbers,
and clip factors beyond fp32. u = 2^-24 is one fp32 rounding; each tolerance counts them."""
import math

import numpy as np
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def signs(n, seed):
    return 1.0 - 2.0 * torch.randint(0, 2, (n,), generator=torch.Generator().manual_seed(seed))


def uniform(n, lo, hi, seed):
    return lo + (hi - lo) * torch.rand(n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def held(x, scales, at):
    """What 8-bit codes stand for."""
    return x.view(torch.float8_e4m3fn).float().double() * scales.view(-1, 2)[:, at].double().repeat_interleave(128)[:x.numel()]


# ------------------------------------------------------------------ subnormal second moments

def test_root_of_a_subnormal_second_moment():
    """eps = 0 and no gradient, so that the update is -2 lr m / (root(v) / root(1/2)) with m and v halved."""
    n = 100_000
    v0 = torch.exp2(uniform(n, -147, -120, 1)).float()
    m0 = (v0.double().sqrt() * (0.5 + torch.rand(n, generator=torch.Generator().manual_seed(2))) * signs(n, 3)).float()
    p, g, m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), m0.to(DEV), v0.to(DEV)
    say("root of a subnormal")
    dps.dp_adamw([p], [g], [m], [v], step=1, lr=1.0, betas=(0.5, 0.5), eps=0.0, weight_decay=0.0)
    v, p = v.cpu().double(), p.cpu().double()
    assert torch.equal(m.cpu(), m0 * 0.5) and bool(((v - v0.double() / 2).abs() <= 2.0 ** -150).all()) and bool((v > 0).all())
    want = -2.0 * (m0.double() / 2) / (v.sqrt() * math.sqrt(2.0))
    # root 1, its factor 1 and product 1, quotient 3 (a reciprocal to 2 and a product), step size 0 and product 1
    assert bool(((p - want).abs() <= 7.01 * U * want.abs()).all()), float(((p - want).abs() / want.abs()).max())


@pytest.mark.parametrize("seed", [None, 5])
def test_eight_bit_states_of_a_subnormal_second_moment(seed):
    """The root of the smallest second moments is far above 2^-100: it is kept, and the step stays one of lr."""
    n = 128 * 300
    e = uniform(n // 128, -73, -61, 4).repeat_interleave(128) + uniform(n, 0, 1, 5)
    g0 = (torch.exp2(e) * signs(n, 6)).float()
    p, g = torch.zeros(n, device=DEV), g0.to(DEV)
    m, v, s = dps.AdamW.new_state([p], 8)
    say("8-bit subnormal", seed)
    dps.dp_adamw([p], [g], m, v, scales=s, step=1, lr=1.0, betas=(0.5, 0.5), eps=0.0, weight_decay=0.0, seed=seed)
    m2, v2 = g0.double() / 2, ((g0 * g0) * 0.5).double()
    r2 = v2.sqrt()
    assert bool((r2 > 0).all())
    want = -2.0 * m2 / (r2 * math.sqrt(2.0))
    assert bool(((p.cpu().double() - want).abs() <= 7.01 * U * want.abs()).all())
    for at, x in ((0, m2), (1, r2)):
        code, scale = (m, v)[at][0].cpu(), s[0].cpu().double().view(-1, 2)[:, at]
        top = x.abs().view(-1, 128).amax(1)
        assert bool(((scale * 448 - top).abs() <= 4 * U * top).all())
        assert bool((code.view(-1) & 0x7F != 0).all())
        steps = 1 if seed is None else 2
        slack = steps * (2.0 ** -4 * x.abs() + 2.0 ** -10 * scale.repeat_interleave(128)) * (1 + 8 * U)
        assert bool(((held(code, s[0].cpu(), at) - x).abs() <= slack).all())


# ------------------------------------------------------------------ states that are not numbers

@pytest.mark.parametrize("bits", [32, 8])
def test_a_second_moment_that_is_nan_shows_in_the_parameter(bits):
    n, at = 1000, 300
    p, g = [torch.full((n,), 2.0, device=DEV)], [torch.full((n,), 0.5, device=DEV)]
    m, v, s = dps.AdamW.new_state(p, bits)
    if bits == 32:
        v[0][at] = float("nan")
    else:
        s[0].fill_(1.0)
        v[0][at] = 0x7F
    say("NaN second moment", bits)
    dps.dp_adamw(p, g, m, v, scales=s, step=1, lr=0.125, weight_decay=0.0)
    assert bool(torch.isfinite(p[0]).sum() == n - 1) and bool(p[0][at].isnan())
    keep = torch.arange(n, device=DEV) != at
    assert bool((p[0][keep] == p[0][0]).all()) and abs(float(p[0][0]) - 1.875) < 1e-5


# ------------------------------------------------------------------ bit for bit

def test_adamw_with_fp32_states_is_the_formula_rounded_as_written():
    """Every operation rounded to nearest once, in the order of the formula: second moments of every exponent,
    subnormal ones among them, and of random fractions."""
    n, t = 1 << 20, 4
    lr, (b1, b2), eps, wd = 0.01, (0.9, 0.95), 1e-30, 0.1
    gen = torch.Generator().manual_seed(7)
    v0 = torch.randint(1, 0x7F000000, (n,), generator=gen, dtype=torch.int32).view(F32)
    v0[:4096] = torch.arange(1, 4097, dtype=torch.int32).view(F32)
    v0[4096:4200] = 0
    m0 = (v0.double().sqrt() * torch.randn(n, generator=gen, dtype=torch.float64)).float()
    g0 = (v0.double().sqrt() * torch.randn(n, generator=gen, dtype=torch.float64)).float()
    p0 = torch.randn(n, generator=gen)
    p, g, m, v = (x.to(DEV) for x in (p0, g0, m0, v0))
    say("bit for bit")
    dps.dp_adamw([p], [g], [m], [v], step=t, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd)
    f = lambda x: np.float32(x)
    p0, g0, m0, v0 = (x.numpy() for x in (p0, g0, m0, v0))
    with np.errstate(all="ignore"):
        m2 = m0 * f(b1) + g0 * f(1 - b1)
        v2 = v0 * f(b2) + (g0 * g0) * f(1 - b2)
        den = np.sqrt(v2) * f(1 / math.sqrt(1 - b2 ** t)) + f(eps)
        want = p0 * f(1 - lr * wd) - m2 / den * f(lr / (1 - b1 ** t))
    for got, x in ((m, m2), (v, v2), (p, want)):
        assert x.dtype == np.float32 and np.array_equal(got.cpu().numpy(), x)


# ------------------------------------------------------------------ clip factors beyond fp32

@pytest.mark.parametrize("value,most", [(1e30, 1e-30), (1e37, 1e-9), (3.0, 1e-46), (1e20, 1e-300), (2.0, 1e-45)])
def test_a_finite_norm_far_above_the_bound_still_steps(value, most):
    """The factor is max_norm / norm rounded once, and where fp32 has nothing so small its smallest number:
    zero means that the step is skipped, and this one counts."""
    g = [torch.full((100,), value, device=DEV)]
    say("clip", value, most)
    ctrl = dps.dp_grad_norm(g, max_norm=most)
    want = most / (float(torch.tensor(value, dtype=F32)) * 10)
    assert int(ctrl.step) == 1 and int(ctrl.skipped) == 0
    assert abs(float(ctrl.scale) - want) <= U * want + 2.0 ** -149 and float(ctrl.scale) > 0
    p = [torch.full((100,), 4.0, device=DEV)]
    m, v, _ = dps.AdamW.new_state(p)
    dps.dp_adamw(p, g, m, v, ctrl=ctrl, lr=0.5, weight_decay=0.5)
    assert bool((p[0] <= 3.01).all())                # at least the decay was made


def test_a_bound_beyond_fp32_clips_nothing():
    ctrl = dps.dp_grad_norm([torch.full((4,), 1e38, device=DEV)], max_norm=1e39)
    assert float(ctrl.scale) == 1.0 and int(ctrl.step) == 1


# ------------------------------------------------------------------ streams

def test_a_norm_built_behind_other_work_runs_on_another_stream():
    """The workspace's fill is queued behind work on the stream where the norm is built, and the run does not
    wait for that stream."""
    g = [torch.full((1000 + i,), 0.5, device=DEV) for i in range(200)]
    want = math.sqrt(sum(x.numel() for x in g)) * 0.5
    side, ctrl = torch.cuda.Stream(), dps.StepCtrl()
    busy = torch.ones(1 << 28, device=DEV)
    torch.cuda.synchronize()
    for i in range(3):
        for _ in range(20):
            busy.mul_(1.0)
        norm = dps.GradNorm(g, ctrl)
        say("norm on another stream", i)
        norm.run(1.0, stream=side)
        side.synchronize()
        assert int(ctrl.step) == i + 1 and abs(float(ctrl.norm) - want) <= 1.01 * U * want
        torch.cuda.synchronize()


def test_a_norm_dropped_while_its_run_is_on_its_way():
    """Its workspace and control block go to no one else before the run on the other stream has ended."""
    g = [torch.full((1000 + i,), 0.5, device=DEV) for i in range(200)]
    want = math.sqrt(sum(x.numel() for x in g)) * 0.5
    side = torch.cuda.Stream()
    busy = torch.ones(1 << 28, device=DEV)
    torch.cuda.synchronize()
    for i in range(3):
        with torch.cuda.stream(side):
            for _ in range(20):
                busy.mul_(1.0)
        norm = dps.GradNorm(g)
        at, ctrl = norm.workspace.data_ptr(), norm.run(1.0, stream=side)
        say("dropped norm", i)
        del norm
        others = [torch.full((dps.training.GRAD_NORM_WS_BYTES,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
        assert all(o.data_ptr() != at for o in others)
        side.synchronize()
        assert abs(float(ctrl.norm) - want) <= 1.01 * U * want and int(ctrl.step) == 1
        assert all(bool((o == 255).all()) for o in others)
