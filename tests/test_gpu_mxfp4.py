"""4-bit block-scaled quantisation and product against their definition in 64
bits, and the training products against the gradient's formula and differences."""
import pytest
import torch

import gradient_sync_amd as dps
from tests.helpers import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def quantized(x):
    """(values of the codes, exponent + 127 per block) of a matrix, from the definition, on the CPU."""
    x = x.detach().cpu().double()
    rows, cols = x.shape
    blocks = -(-cols // 32)
    b = torch.zeros(rows, blocks * 32, dtype=torch.float64)
    b[:, :cols] = x
    b = b.view(rows, blocks, 32)
    top = b.abs().amax(2)
    finite = torch.isfinite(b).all(2)
    top = torch.where(finite, top, 1.0)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(min=-127)
    y = torch.where(finite.unsqueeze(2), b, 0.0) / torch.ldexp(torch.ones_like(top), e).unsqueeze(2)
    a = y.abs().clamp(max=6)
    near = (a.unsqueeze(3) - GRID).abs()
    best = near.amin(3, keepdim=True)
    tied = near == best                              # two neighbours in a tie: the even code
    even = torch.arange(8) % 2 == 0
    pick = torch.where(tied.sum(3, keepdim=True) > 1, tied & even, tied).int().argmax(3)
    value = torch.copysign(GRID[pick], y)
    return value.view(rows, -1), torch.where(finite, e + 127, 255), cols


def unpacked(q):
    """The same pair from a quantised matrix's bytes, by the layout the header states."""
    codes, scales = q.codes.cpu(), q.scales.cpu()
    blocks = -(-q.cols // 32)
    nib = torch.stack([codes & 15, codes >> 4], 2).view(q.rows, -1).long()
    assert not bool(nib[:, blocks * 32:].any())      # zero past the last block
    value = GRID[nib % 8] * torch.where(nib >= 8, -1.0, 1.0)
    r, b = torch.arange(q.rows).view(-1, 1), torch.arange(blocks).view(1, -1)
    at = ((r // 16) * (-(-q.cols // 512)) + b // 16) * 256 + (16 * (b % 4) + r % 16) * 4 + (b % 16) // 4
    return value[:, :blocks * 32], scales.view(-1)[at.view(-1)].view(q.rows, blocks).long()


def same(q, x):
    value, byte, cols = quantized(x)
    got, gbyte = unpacked(q)
    return bool((gbyte == byte).all()) and bool((got == value).all())


def rand(shape, seed, dtype=F32, spread=3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-spread, spread + 1, (shape[0], 1), generator=g).float())
    return x.to(dtype).to(DEV)


def values(q):
    return dps.dp_mxfp4_dequantize(q, dtype=F32).cpu().double()


# ------------------------------------------------------------------ quantisation

SHAPES = [(1, 1), (1, 32), (3, 33), (16, 128), (17, 129), (128, 128), (129, 31), (130, 257), (5, 513), (200, 1000),
          (300, 70)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_both_ways(shape, dtype):
    x = rand(shape, 7, dtype)
    say("quantize", shape, dtype)
    q, qt = dps.dp_mxfp4_quantize(x, transposed="also")
    assert same(q, x) and same(qt, x.t())
    one, other = dps.dp_mxfp4_quantize(x), dps.dp_mxfp4_quantize(x, transposed="only")
    assert torch.equal(one.codes, q.codes) and torch.equal(other.codes, qt.codes)
    assert torch.equal(unpacked(one)[1], unpacked(q)[1]) and torch.equal(unpacked(other)[1], unpacked(qt)[1])
    for q, of in ((q, x), (qt, x.t())):
        v, byte, cols = quantized(of)
        want = (v.view(v.shape[0], -1, 32) * torch.exp2(byte.double() - 127).unsqueeze(2)).view(v.shape[0], -1)[:, :cols]
        for t in (F32, BF16):
            assert torch.equal(dps.dp_mxfp4_dequantize(q, dtype=t).cpu().double(), want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_strided_and_unaligned(dtype):
    big = rand((70, 301), 3, dtype)
    x = big[2:60, 3:203]                             # rows start at odd elements
    q, qt = dps.dp_mxfp4_quantize(x, transposed="also")
    assert same(q, x) and same(qt, x.t())
    with pytest.raises(ValueError):
        dps.dp_mxfp4_quantize(big.t())


def test_quantize_ties_and_saturation():
    """Every midpoint, its neighbours, and everything above the largest value."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = torch.cat([mid, mid * (1 + 2.0 ** -22), mid * (1 - 2.0 ** -22), torch.tensor([7.999, 6.0, 5.5, 0.0, 4.0])])
    x = torch.cat([x, -x, torch.zeros(12)]).view(2, 32)
    x[:, 31] = 7.5                                   # keeps the scale at 1
    rows = torch.cat([x * 2.0 ** e for e in (0, -3, 40, -126, -130, 125)]).to(DEV)
    q, qt = dps.dp_mxfp4_quantize(rows, transposed="also")
    assert same(q, rows) and same(qt, rows.t())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_special_values(dtype):
    x = rand((64, 96), 5, dtype)
    x[0, :32] = 0
    x[1, :32] = -0.0
    x[2, 5] = float("nan")
    x[3, 40] = float("inf")
    x[4, 95] = -float("inf")
    x[5, 0] = torch.finfo(dtype).max
    x[6, :32] = torch.finfo(dtype).tiny * 2.0 ** -5  # subnormal
    x[7, :32] = torch.finfo(dtype).tiny
    q, qt = dps.dp_mxfp4_quantize(x, transposed="also")
    assert same(q, x) and same(qt, x.t())
    v = dps.dp_mxfp4_dequantize(q, dtype=F32)
    bad = torch.zeros(64, 96, dtype=torch.bool, device=DEV)
    bad[2, :32] = bad[3, 32:64] = bad[4, 64:] = True
    assert torch.equal(v.isnan(), bad) and torch.equal(dps.dp_mxfp4_dequantize(q).isnan(), bad)


def test_quantize_leaves_its_surroundings():
    x = rand((33, 200), 1)
    q = dps.Mxfp4(33, 200)
    n, k = q.codes.numel(), q.scales.numel()
    buf = torch.full((n + 512,), 99, dtype=torch.uint8, device=DEV)
    sbuf = torch.full((k + 512,), 99, dtype=torch.uint8, device=DEV)
    q = dps.Mxfp4(33, 200, buf[256:256 + n], sbuf[256:256 + k])
    dps.dp_mxfp4_quantize(x, out=q)
    out = torch.full((33 * 200 + 64,), 9.0, device=DEV)
    dps.dp_mxfp4_dequantize(q, out=out[32:32 + 6600].view(33, 200))
    for b, e in ((buf, 99), (sbuf, 99)):
        assert bool((b[:256] == e).all()) and bool((b[-256:] == e).all())
    assert bool((out[:32] == 9).all()) and bool((out[-32:] == 9).all()) and same(q, x)


def test_quantize_is_idempotent_and_empty_is_fine():
    x = rand((40, 300), 2)
    v = dps.dp_mxfp4_dequantize(dps.dp_mxfp4_quantize(x))
    assert torch.equal(dps.dp_mxfp4_dequantize(dps.dp_mxfp4_quantize(v)), v)
    for shape in ((0, 40), (40, 0)):
        q = dps.dp_mxfp4_quantize(torch.empty(shape, device=DEV))
        assert dps.dp_mxfp4_dequantize(q).shape == shape


def test_quantize_beyond_32_bits():
    rows, cols = 65664, 32768                        # 2^31 elements and more, 4 GiB of bf16
    x = torch.empty(rows, cols, dtype=BF16, device=DEV)
    x.fill_(1.5)
    x[-200:] = rand((200, cols), 4, BF16)
    say("quantize beyond 32 bits")
    q, qt = dps.dp_mxfp4_quantize(x, transposed="also")
    tail = dps.dp_mxfp4_quantize(x[-192:].contiguous())
    assert torch.equal(q.codes[-192:], tail.codes)
    assert torch.equal(dps.dp_mxfp4_dequantize(q)[-192:], dps.dp_mxfp4_dequantize(tail))
    part = dps.dp_mxfp4_quantize(x[-128:].contiguous(), transposed="only")
    assert torch.equal(qt.codes[:, -64:], part.codes)
    del x
    one = dps.dp_mxfp4_quantize(torch.ones(1, cols, device=DEV))
    y = dps.dp_gemm_mxfp4(q, one, dtype=F32)         # sums of the rows, from 2^30 bytes of codes
    assert bool((y[:1000] == 1.5 * cols).all())
    want = dps.dp_mxfp4_dequantize(tail, dtype=F32).double().sum(1)
    assert bool(((y[-192:, 0].double() - want).abs() <= cols * 2.0 ** -23 * dps.dp_mxfp4_dequantize(tail, dtype=F32).double().abs().sum(1)).all())


# ------------------------------------------------------------------ product

def check_product(c, a, b, extra=0.0, dtype=F32):
    """k products are exact; each of at most k fp32 additions may lose 2^-23 of the sum of magnitudes."""
    a, b = a.cpu().double(), b.cpu().double()
    want, mag = a @ b.t(), a.abs() @ b.abs().t()
    tol = a.shape[1] * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if dtype == BF16 else 0) + extra
    assert bool(((c.cpu().double() - want).abs() <= tol).all()), float(((c.cpu().double() - want).abs() - tol).max())


MNK = [(1, 1, 1), (1, 16, 128), (3, 5, 31), (16, 33, 512), (17, 100, 200), (40, 17, 513), (64, 64, 1000), (65, 130, 640),
       (100, 300, 96), (128, 128, 256), (129, 257, 384), (255, 300, 1100), (256, 256, 512), (300, 520, 2080),
       (513, 260, 1024), (1, 2000, 4096), (700, 1, 300), (520, 780, 768)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", MNK)
def test_product(m, n, k, dtype):
    a, b = dps.dp_mxfp4_quantize(rand((m, k), 1)), dps.dp_mxfp4_quantize(rand((n, k), 2))
    buf = torch.full((m * n + 64,), 5.0, dtype=dtype, device=DEV)
    out = buf[32:32 + m * n].view(m, n)
    say("product", m, n, k, dtype)
    dps.dp_gemm_mxfp4(a, b, out=out)
    check_product(out, values(a), values(b), dtype=dtype)
    assert bool((buf[:32] == 5).all()) and bool((buf[-32:] == 5).all())


@pytest.mark.parametrize("m,n,k", MNK)
def test_product_is_exact_for_small_integers(m, n, k):
    """Codes 0..6 at scales 2^-2 .. 2^1: every sum is a multiple of 2^-4 below 2^20, so any order is exact."""
    g = torch.Generator().manual_seed(m + n + k)
    make = lambda r: (GRID[torch.randint(0, 8, (r, k), generator=g)] * (1 - 2 * torch.randint(0, 2, (r, k), generator=g)) *
                      torch.exp2(torch.randint(-1, 1, (r, -(-k // 32)), generator=g).double()).repeat_interleave(32, 1)[:, :k])
    a, b = make(m), make(n)
    qa, qb = dps.dp_mxfp4_quantize(a.float().to(DEV)), dps.dp_mxfp4_quantize(b.float().to(DEV))
    assert torch.equal(values(qa), values(dps.dp_mxfp4_quantize(values(qa).float().to(DEV))))
    c = dps.dp_gemm_mxfp4(qa, qb, dtype=F32)
    assert torch.equal(c.cpu().double(), values(qa) @ values(qb).t())
    before = torch.randint(-50, 50, (m, n), generator=g).float().to(DEV)
    out = before.clone()
    dps.dp_gemm_mxfp4(qa, qb, out=out, accumulate=True)
    assert torch.equal(out, before + c)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n,k", [(4096, 2560, 512), (4001, 2500, 1100), (3900, 2601, 640), (2561, 4090, 130),
                                   (4096, 4096, 1024), (4001, 4090, 1100), (8192, 8192, 200), (8000, 5000, 1400),
                                   (7941, 5099, 1400)])
def test_product_of_large_matrices(m, n, k, dtype):
    """Enough of C for the large tile, one a workgroup or several in turn, with and without edges, rows of C
    on 16 bytes or not."""
    a, b = dps.dp_mxfp4_quantize(rand((m, k), 1)), dps.dp_mxfp4_quantize(rand((n, k), 2))
    buf = torch.full((m * n + 64,), 5.0, dtype=dtype, device=DEV)
    out = buf[32:32 + m * n].view(m, n)
    say("large product", m, n, k, dtype)
    dps.dp_gemm_mxfp4(a, b, out=out)
    first = out.clone()
    va, vb = (dps.dp_mxfp4_dequantize(q, dtype=F32).double() for q in (a, b))
    want, mag = va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()
    tol = k * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if dtype == BF16 else 0)
    assert bool(((out.double() - want).abs() <= tol).all())
    if dtype == F32:
        dps.dp_gemm_mxfp4(a, b, out=out, accumulate=True)
        assert torch.equal(out, first + first)
    assert bool((buf[:32] == 5).all()) and bool((buf[-32:] == 5).all())


def test_product_of_extreme_scales_and_nan_blocks():
    a, b = rand((70, 160), 3), rand((50, 160), 4)
    a[:, 32:64] *= 2.0 ** 60
    b[:, 32:64] *= 2.0 ** -70
    a[:, 64:96] = 0
    a[9, 100] = float("nan")
    b[7, 3] = float("inf")
    qa, qb = dps.dp_mxfp4_quantize(a), dps.dp_mxfp4_quantize(b)
    c = dps.dp_gemm_mxfp4(qa, qb, dtype=F32)
    nan = torch.zeros(70, 50, dtype=torch.bool, device=DEV)
    nan[9] = True
    nan[:, 7] = True
    assert torch.equal(c.isnan(), nan)
    keep_r, keep_c = [i for i in range(70) if i != 9], [j for j in range(50) if j != 7]
    check_product(c[keep_r][:, keep_c], values(qa)[keep_r], values(qb)[keep_c])


@pytest.mark.parametrize("x_dtype", [F32, BF16])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 64, 130])
def test_linear_is_quantize_and_product(m, x_dtype):
    for n, k in ((100, 100), (48, 1024), (33, 2085), (40, 500), (6500, 6000)):
        x = rand((m, k + 3), 5, x_dtype)[:, 1:1 + k] if m > 1 else rand((m, k), 5, x_dtype)
        if k > 1000:
            x[0, 40] = float("nan")
        w = dps.dp_mxfp4_quantize(rand((n, k), 6))
        say("linear", m, n, k, x_dtype)
        for t in (F32, BF16):
            y = dps.dp_mxfp4_linear(x, w, dtype=t)
            want = dps.dp_gemm_mxfp4(dps.dp_mxfp4_quantize(x.contiguous()), w, dtype=t)
            assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.nan_to_num())


def test_linear_on_another_stream_and_in_a_graph():
    x, w = rand((100, 640), 1, BF16), dps.dp_mxfp4_quantize(rand((300, 640), 2))
    want = dps.dp_mxfp4_linear(x, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = dps.dp_mxfp4_linear(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, one = torch.empty_like(want), torch.empty(1, 300, dtype=BF16, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dps.dp_mxfp4_linear(x, w, out=out)
        dps.dp_mxfp4_linear(x[:1], w, out=one)
    for i in range(4):
        x.copy_(rand((100, 640), 10 + i, BF16))
        say("graph replay", i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dps.dp_mxfp4_linear(x, w)) and torch.equal(one, dps.dp_mxfp4_linear(x[:1], w))


def test_binding_refusals_on_the_gpu():
    a, b = dps.dp_mxfp4_quantize(rand((8, 64), 1)), dps.dp_mxfp4_quantize(rand((8, 96), 1))
    with pytest.raises(ValueError):
        dps.dp_gemm_mxfp4(a, b)
    with pytest.raises(ValueError):
        dps.dp_gemm_mxfp4(a, a, accumulate=True)
    with pytest.raises(dps.DpsyncError):
        dps.dp_gemm_mxfp4(a, a, out=torch.empty(8, 8, dtype=BF16, device=DEV), accumulate=True)
    with pytest.raises(ValueError):
        dps.dp_gemm_mxfp4(a, a, out=torch.empty(8, 9, device=DEV))
    with pytest.raises(ValueError):
        dps.dp_mxfp4_linear(rand((3, 65), 1), a)
    with pytest.raises(TypeError):
        dps.dp_mxfp4_dequantize(a, dtype=torch.float16)


# ------------------------------------------------------------------ training products

def training_step(x, w, dy):
    xq, xt = dps.dp_mxfp4_quantize(x, transposed="also")
    wq, wt = dps.dp_mxfp4_quantize(w, transposed="also")
    gq, gt = dps.dp_mxfp4_quantize(dy, transposed="also")
    return (dps.dp_gemm_mxfp4(xq, wq, dtype=F32), dps.dp_gemm_mxfp4(gq, wt, dtype=F32),
            dps.dp_gemm_mxfp4(gt, xt, dtype=F32))


@pytest.mark.parametrize("m,n,k", [(33, 70, 50), (256, 128, 384), (520, 300, 260)])
def test_gradients_equal_the_formula(m, n, k):
    x, w, dy = rand((m, k), 1, spread=0), rand((n, k), 2, spread=0), rand((m, n), 3, spread=0)

    def q(t):
        v, byte, cols = quantized(t)
        return (v.view(v.shape[0], -1, 32) * torch.exp2(byte.double() - 127).unsqueeze(2)).view(v.shape[0], -1)[:, :cols]
    y, dx, dw = training_step(x, w, dy)
    check_product(y, q(x), q(w))
    check_product(dx, q(dy), q(w.t()))
    check_product(dw, q(dy.t()), q(x.t()))


def test_gradients_equal_differences():
    """On values that four bits hold exactly, each of the three matrices moved by one code: the loss
    sum(y * dy) is linear in w and in x, so the difference is the gradient times the move."""
    m, n, k = 64, 96, 160
    g = torch.Generator().manual_seed(8)

    def exact(r, c):
        v = GRID[torch.randint(0, 7, (r, c), generator=g)] * (1 - 2 * torch.randint(0, 2, (r, c), generator=g))
        at = torch.arange(max(r, c))
        v[at % r, at % c] = 4.0                      # a 4 in every block of either orientation
        v[:, ::16] = 4.0
        v[::16, :] = 4.0
        return v.float().to(DEV)
    x, w, dy = exact(m, k), exact(n, k), exact(m, n)
    y, dx, dw = training_step(x, w, dy)
    loss = lambda x, w: float((training_step(x, w, dy)[0].double() * dy.double()).sum())
    base = loss(x, w)
    assert base == float(((x.double() @ w.double().t()) * dy.double()).sum())
    for i, j in ((5, 7), (90, 151), (33, 1)):
        moved = w.clone()
        moved[i, j] = 0.5 if w[i, j] != 0.5 else 1.0
        assert loss(x, moved) - base == float(dw[i, j]) * float(moved[i, j] - w[i, j])
        i, j = i % m, j
        moved = x.clone()
        moved[i, j] = -1.5 if x[i, j] != -1.5 else 2.0
        assert loss(moved, w) - base == float(dx[i, j]) * float(moved[i, j] - x[i, j])
