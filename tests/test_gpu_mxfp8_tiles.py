"""Products of 8-bit operands in the large tiles: values of a normal distribution, scales far apart and blocks that are
NaN, against 64 bits; and the largest finite values."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say
from tests.test_gpu_mxfp8 import check_product, quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def rand(rows, cols, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    size = torch.exp2(torch.randint(-3, 4, (rows, 1), generator=g, device=DEV).float())
    return torch.randn(rows, cols, generator=g, device=DEV) * size


def values(q):
    f = dps.dp_mxfp4_dequantize if isinstance(q, dps.Mxfp4) else dps.dp_mxfp8_dequantize
    return f(q, dtype=F32)


def sample(rows, skip):
    """Rows of every wave's part of a tile and of C's edge."""
    at = sorted({0, 1, 15, 16, 63, 64, 127, 128, 200, 255, 256, rows // 2, rows - 17, rows - 2, rows - 1} - set(skip))
    return torch.tensor(at, device=DEV)


# tiles of 128, of 256 one a workgroup and several: k of one to three fours of 128 and a rest of each kind
SHAPES = [(2049, 2050, 1400), (2100, 4090, 700), (2304, 2304, 1024), (4001, 4090, 1100), (4096, 4096, 1290), (8190, 8191, 1100),
          (8192, 8184, 1400), (8190, 8191, 130)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_of_normal_values(m, n, k, bits):
    a, b = dps.dp_mxfp8_quantize(rand(m, k, 1)), quantize(rand(n, k, 2), bits)
    va, vb = values(a), values(b)
    r, c = sample(m, ()), sample(n, ())
    for dtype in (F32, BF16):
        say("product", m, n, k, bits, dtype)
        out = dps.dp_gemm_mxfp8(a, b, dtype=dtype)
        check_product(out[r], va[r], vb, dtype)
        check_product(out[:, c], va, vb[c], dtype)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product_of_far_scales_and_nan_blocks(m, n, k, bits):
    """Neighbouring blocks 2^130 apart, and NaN in the first, a middle and the last block of a row of either operand, the
    last one's step being loaded again in place of those behind the row's end."""
    a, b = rand(m, k, 3), rand(n, k, 4)
    a[:, 32:64] *= 2.0 ** 60
    b[:, 32:64] *= 2.0 ** -70
    a[:, 64:96] = 0
    a[:, 96:128] *= 2.0 ** -70
    b[:, 96:128] *= 2.0 ** 60
    a[:, k - 2:] *= 2.0 ** 40
    b[:, k - 2:] *= 2.0 ** -50
    bad_a, bad_b = [9, 130, m - 3], [7, 300, n - 4]
    for t, bad in ((a, bad_a), (b, bad_b)):
        t[bad[0], k - 1] = float("nan")
        t[bad[1], 40] = float("inf")
        t[bad[2], 0] = -float("inf")
    qa, qb = dps.dp_mxfp8_quantize(a), quantize(b, bits)
    nan = torch.zeros(m, n, dtype=torch.bool, device=DEV)
    nan[bad_a] = True
    nan[:, bad_b] = True
    va, vb = values(qa), values(qb)
    r, c = sample(m, bad_a), sample(n, bad_b)
    keep_r, keep_c = (torch.tensor([i for i in range(x) if i not in bad], device=DEV) for x, bad in ((m, bad_a), (n, bad_b)))
    for dtype in (F32, BF16):
        say("product, far scales", m, n, k, bits, dtype)
        out = dps.dp_gemm_mxfp8(qa, qb, dtype=dtype)
        assert torch.equal(out.isnan(), nan)
        check_product(out[r][:, keep_c], va[r], vb[keep_c], dtype)
        check_product(out[keep_r][:, c], va[keep_r], vb[c], dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_largest_finite_values(dtype):
    """1.9375 * 2^127, halfway between 240 and 256 times 2^120, and what is above it are held as 2^128 (the even code): beyond
    fp32, so infinite once expanded, but a number to a product."""
    least = 1.9375 * 2.0 ** 127
    below = least - (2.0 ** 104 if dtype == F32 else 2.0 ** 120)
    x = torch.zeros(4, 64, dtype=dtype)
    x[:, 3] = torch.tensor([torch.finfo(dtype).max, least, below, -torch.finfo(dtype).max], dtype=torch.float64).to(dtype)
    held = [2.0 ** 128, 2.0 ** 128, 240 * 2.0 ** 120, -2.0 ** 128]
    q, qt = dps.dp_mxfp8_quantize(x.to(DEV), transposed="also")
    for t in (F32, BF16):
        assert dps.dp_mxfp8_dequantize(q, dtype=t)[:, 3].tolist() == [v if abs(v) < 2.0 ** 128 else v * float("inf") for v in held]
    for codes in (q.codes[:, 3], qt.codes[3, :4]):
        assert codes.tolist() == [0x78, 0x78, 0x77, 0xf8]
    for rows, n in ((4, 5), (70, 50), (2049, 2050), (4001, 4090)):
        a = torch.zeros(rows, 64, dtype=dtype, device=DEV)
        a[rows - 4:] = x.to(DEV)
        say("product of the largest values", rows, n, dtype)
        for bits in (4, 8):
            b = quantize(torch.full((n, 64), 2.0 ** -20, device=DEV), bits)
            out = dps.dp_gemm_mxfp8(dps.dp_mxfp8_quantize(a), b, dtype=F32)
            assert torch.equal(out[rows - 4:].double(), torch.tensor(held, dtype=torch.float64, device=DEV).mul(2.0 ** -20).unsqueeze(1).expand(4, n))
            assert not bool(out[:rows - 4].any())
