"""Gradients of the root-mean-square norm over batches that are read past the caches (128 MiB and more), and beyond 2^31
elements, against 64 bits."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24                  # half a step of fp32, relative
HALF = {F32: 0.0, BF16: 2.0 ** -8}
EPS = 1e-6


def rand(rows, cols, seed, dtype):
    """Rows of different sizes."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    size = torch.exp2(torch.randint(-2, 3, (rows, 1), generator=g, device=DEV).float())
    return (torch.randn(rows, cols, generator=g, device=DEV) * size).to(dtype)


def gamma(n, seed, dtype):
    return (1 + 0.1 * torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)).to(dtype)


def check_dx(dx, dy, h, w, rstd, dr):
    """u, g and their products are a rounding of fp32 each; a row's sum passes at most 8 elements of 2 chunks, 6 steps of a
    wave and 16 waves (40 are counted). A bf16 dx is half a step off besides."""
    dy, h, w, rstd = dy.double(), h.double(), w.double(), rstd.double().unsqueeze(1)
    u, g = h * rstd, dy * w
    mean, size = (g * u).mean(1, keepdim=True), (g * u).abs().mean(1, keepdim=True)
    want = rstd * (g - u * mean)
    tol = rstd * (4 * U * (g.abs() + u.abs() * mean.abs()) + u.abs() * 40 * U * size)
    if dr is not None:
        want = want + dr.double()
        tol += 2 * U * want.abs() + U * dr.double().abs()
    off = (dx.double() - want).abs() - HALF[dx.dtype] * want.abs()
    assert bool((off <= tol).all()), float((off - tol).max())


def check_dw(dw, terms, size, rows):
    """At most rows / 64 + 64 additions of products of two roundings."""
    assert bool(((dw.double() - terms).abs() <= (rows / 64 + 66) * U * size).all())


def check(dx, dw, dy, h, w, rstd, dr):
    check_dx(dx, dy, h, w, rstd, dr)
    terms = dy.double() * h.double() * rstd.double().unsqueeze(1)
    check_dw(dw, terms.sum(0), terms.abs().sum(0), h.shape[0])


# 4 bytes an element of dy and hidden state at least: 128 MiB and more each. A quarter, a half and a whole workgroup of 1024
# threads a row, one chunk and two, whole rows and rows that end inside 8 elements
@pytest.mark.parametrize("dtype,dy_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,cols", [(18000, 2000), (18000, 1997), (9000, 4096), (9000, 4089), (5000, 8192), (5000, 7003),
                                       (2300, 16384), (2300, 16001)])
def test_backward_of_large_batches(rows, cols, dtype, dy_dtype):
    assert rows * cols * 4 >= 128 << 20
    h, dy, dr = rand(rows, cols, 1, dtype), rand(rows, cols, 2, dy_dtype), rand(rows, cols, 3, dtype)
    w = gamma(cols, 4, dy_dtype)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    say("norm backward", rows, cols, dtype, dy_dtype)
    dx, dw = dps.dp_rms_norm_backward(dy, h, w, rstd)
    check(dx, dw, dy, h, w, rstd, None)
    dx, dw = dps.dp_rms_norm_backward(dy, h, w, rstd, dresidual=dr)
    check(dx, dw, dy, h, w, rstd, dr)
    # in the place of each input of its type
    for i, t in enumerate((dy, h, dr)):
        if t.dtype != dtype:
            continue
        a = [t.clone() if j == i else t for j, t in enumerate((dy, h, dr))]
        got = dps.dp_rms_norm_backward(a[0], a[1], w, rstd, dresidual=a[2], out=a[i])
        assert got[0] is a[i] and torch.equal(a[i], dx) and torch.equal(got[1], dw)


def test_backward_of_large_strided_batches():
    """Columns of a wider buffer, with NaN beside them."""
    rows, cols = 9000, 4089
    kept = [torch.full((rows, cols + 13), float("nan"), dtype=BF16, device=DEV) for _ in range(3)]
    for i, t in enumerate(kept):
        t[:, 3:3 + cols] = rand(rows, cols, i + 1, BF16)
    dy, h, dr = (t[:, 3:3 + cols] for t in kept)
    w = gamma(cols, 4, F32)
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    say("norm backward strided", rows, cols)
    dx, dw = dps.dp_rms_norm_backward(dy, h, w, rstd, dresidual=dr)
    check(dx, dw, dy, h, w, rstd, dr)
    got = dps.dp_rms_norm_backward(dy, h, w, rstd, dresidual=dr, out=dr)
    assert torch.equal(dr, dx) and torch.equal(got[1], dw)
    assert bool(kept[2][:, :3].isnan().all()) and bool(kept[2][:, 3 + cols:].isnan().all())


def test_backward_beyond_32_bits():
    """2^31 elements and more: rows from both ends and around the 2^31st element against 64 bits, and dw against all rows'."""
    rows, cols = 131200, 16384
    edge = (1 << 31) // cols
    h, dy = torch.empty(rows, cols, dtype=BF16, device=DEV), torch.empty(rows, cols, dtype=BF16, device=DEV)
    for i in range(0, rows, 16400):
        h[i:i + 16400], dy[i:i + 16400] = rand(16400, cols, i, BF16), rand(16400, cols, i + 1, BF16)
    w = gamma(cols, 4, BF16)
    rstd = torch.cat([(h[i:i + 16400].double().square().mean(1) + EPS).rsqrt().float() for i in range(0, rows, 16400)])
    total, size = (torch.zeros(cols, dtype=torch.float64, device=DEV) for _ in range(2))
    for i in range(0, rows, 16400):
        p = dy[i:i + 16400].double() * h[i:i + 16400].double() * rstd[i:i + 16400].double().unsqueeze(1)
        total += p.sum(0)
        size += p.abs().sum(0)
    at = torch.tensor([0, 1, 1000, edge - 1, edge, edge + 1, rows - 2, rows - 1], device=DEV)
    some = [t[at].clone() for t in (dy, h, rstd)]
    say("norm backward beyond 32 bits")
    dx, dw = dps.dp_rms_norm_backward(dy, h, w, rstd, out=h)
    assert dx is h
    check_dx(dx[at], some[0], some[1], w, some[2], None)
    check_dw(dw, total, size, rows)
