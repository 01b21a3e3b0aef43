"""The bits of the stochastic rounding of 8-bit states, computed on the CPU from the header's definition, and
the codes they give."""
import numpy as np
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
BETAS = (0.75, 0.875)                                # exact in fp32, and 1 - beta too
MASK = (1 << 64) - 1
G = 0x9E3779B97F4A7C15


def mix(z):
    """SplitMix64's output function, on Python integers of any size."""
    z &= MASK
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK
    return z ^ (z >> 31)


def fractions(seed, t, i, start, n):
    """r / 65536 for m and for sqrt(v) of elements start .. start + n - 1 of tensor i at step t."""
    key = mix(mix(seed + t * G) + (i + 1) * G)
    out = np.zeros((2, n))
    for at in range(start - start % 2, start + n, 2):
        z = mix(key + (at // 2 + 1) * G)
        for odd in (0, 1):
            for which in (0, 1):
                if 0 <= at + odd - start < n:
                    out[which, at + odd - start] = (z >> (32 * odd + 16 * which) & 0xFFFF) / 65536
    return out


def expected(g, r):
    """Of one step from states of zero, for elements that start at a block: the values of the codes in units of
    their scale, for m and sqrt(v), and where they are certain (y is known to a few roundings, 2^-18 of a step)."""
    g = g.float().cpu().numpy()
    n = len(g)
    m, v = g * np.float32(1 - BETAS[0]), g * g * np.float32(1 - BETAS[1])
    out = []
    for at, x in ((0, m), (1, np.sqrt(v))):
        x = x.astype(np.float64)
        top = np.zeros(-(-n // 128) * 128)
        top[:n] = np.abs(x)
        top = top.reshape(-1, 128).max(1).repeat(128)[:n]
        a = np.minimum(np.abs(x) / top * 448, 448)
        if at == 1:
            a = np.where(a > 0, np.maximum(a, 2.0 ** -9), 0)
        u = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6) - 3)
        steps = a / u + r[at]
        sure = np.abs(steps - np.round(steps)) > 2.0 ** -15
        sure |= (a == 0)
        out.append((np.copysign(np.floor(steps) * u, x), sure))
    return out


def check(codes, g, r, what):
    for at in (0, 1):
        want, sure = expected(g, r)[at]
        got = codes[at].view(torch.float8_e4m3fn).float().cpu().double().numpy()
        assert sure.mean() > 0.98
        assert np.array_equal(got[sure], want[sure]), (what, at, int((got != want)[sure].sum()))


def gradient(n, seed, dtype):
    gen = torch.Generator().manual_seed(seed)
    # 12 octaves: the codes' subnormal range too
    return (torch.randn(n, generator=gen) * torch.exp2(-12 * torch.rand(n, generator=gen))).to(dtype).to(DEV)


@pytest.mark.parametrize("seed,t", [(0, 1), (12345, 7), ((1 << 64) - 3, 1000), (1 << 63, 1 << 40)])
@pytest.mark.parametrize("p_dtype,g_dtype", [(F32, BF16), (BF16, F32)])
def test_codes_are_those_of_the_counters(seed, t, p_dtype, g_dtype):
    """Whole chunks (both groups of a thread), short ones, odd ends, and tensors of a call's second launch."""
    sizes = {0: 2048 * 3 + 777, 1: 129, 2: 1, 63: 2048, 64: 300, 66: 4096 + 128, 69: 2047}
    gs = [gradient(sizes.get(i, 0), 100 + i, g_dtype) for i in range(70)]
    ps = [torch.zeros_like(g, dtype=p_dtype) for g in gs]
    m, v, s = dps.AdamW.new_state(ps, 8)
    say("counters", seed, t, p_dtype, g_dtype)
    dps.dp_adamw(ps, gs, m, v, step=t, scales=s, lr=1e-3, betas=BETAS, seed=seed)
    for i, n in sizes.items():
        check((m[i], v[i]), gs[i], fractions(seed, t, i, 0, n), i)


def test_the_step_in_the_counter_is_the_control_blocks():
    g = [gradient(5000, 3, F32)]
    p = [torch.zeros(5000, device=DEV)]
    m, v, s = dps.AdamW.new_state(p, 8)
    dps.dp_adamw(p, g, m, v, ctrl=dps.StepCtrl(step=23), scales=s, betas=BETAS, seed=9)
    check((m[0], v[0]), g[0], fractions(9, 23, 0, 0, 5000), "control")


def test_counters_beyond_32_bits():
    """The last elements of a tensor of more than 2^32: their pair counters are beyond 2^31."""
    n, k = 2 ** 32 + 2048 * 5 + 77, 128 * 50 + 77
    cut = n - k
    assert cut % 128 == 0
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of GPU memory")
    p, g = torch.zeros(n, dtype=BF16, device=DEV), torch.zeros(n, dtype=BF16, device=DEV)
    g[cut:] = gradient(k, 5, BF16)
    m, v, s = dps.AdamW.new_state([p], 8)
    say("counters beyond 32 bits")
    dps.dp_adamw([p], [g], m, v, step=3, scales=s, lr=1e-3, betas=BETAS, seed=77)
    check((m[0][cut:], v[0][cut:]), g[cut:], fractions(77, 3, 0, cut, k), "tail")
    assert not bool(m[0][:cut].any()) and not bool(v[0][:cut].any())
