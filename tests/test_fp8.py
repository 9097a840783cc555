"""The 8-bit block-scaled operators against their definitions in 64 bits, and
their refusals (CPU).

Tolerances. Codes and scales of iqk_fp8_quantize are exact. A product's
float32 sums: every addition on the way (the block sums of up to 128 products
in the tensor cores, whose additions may truncate, so 2^-23 each; two products
with the scales and one addition for each block) is relative to a partial sum
of magnitude at most S = sum |xs ws xq wq|, so |y - exact| <= (cols + 8 blocks
+ 16) 2^-23 S, then half a step of y's type (2^-8 for bfloat16, 2^-24 for
float32) relative to y. gate_up: see check_h.
"""
import math

import numpy as np
import pytest

from gemm_iq2_ks_b200 import binding as B

torch = pytest.importorskip("torch")

E4M3 = torch.float8_e4m3fn


def blocks(n):
    return (n + 127) // 128


def gen(seed):
    return torch.Generator().manual_seed(seed)


def activations(seed, T, cols):
    x = torch.randn((T, cols), generator=gen(seed))
    x[:, torch.rand((cols,), generator=gen(seed + 1)) < 0.02] *= 16
    return x.bfloat16().cuda()


def operand(seed, rows, cols, block_rows):
    """Random e4m3 codes (every finite one occurs) and scales over a few binades."""
    c = torch.randint(0, 256, (rows, cols), generator=gen(seed), dtype=torch.int32)
    c = torch.where((c & 127) == 127, c - 1, c).to(torch.uint8)
    s = torch.exp2(-8 + 2 * torch.randn(((rows + block_rows - 1) // block_rows, blocks(cols)), generator=gen(seed + 1)))
    return c.cuda().view(E4M3), s.cuda()


def value(q, s, block_rows):
    rows, cols = q.shape
    f = s.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return q.double() * f


def product(wq, ws, xq, xs):
    """(exact product, S, the bound of the float32 sums' error)."""
    x, w = value(xq, xs, 1), value(wq, ws, 128)
    S = x.abs() @ w.abs().t()
    cols = wq.shape[1]
    return x @ w.t(), S, (cols + 8 * blocks(cols) + 16) * 2.0 ** -23 * S


# -------------------------------------------------------------- quantisation

def quantized(x):
    """Definition: nearest e4m3 number of 448 x / m (ties to even), from float64."""
    T, cols = x.shape
    q, s = torch.zeros((T, cols), dtype=torch.float64), torch.zeros((T, blocks(cols)), dtype=torch.float32)
    x = x.double().cpu()
    for b in range(blocks(cols)):
        v = x[:, b * 128:(b + 1) * 128]
        m = v.abs().amax(1).clamp(min=2.0 ** -100)
        s[:, b] = m.float() / 448.0
        t = v * 448.0 / m[:, None]
        e = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3)
        q[:, b * 128:(b + 1) * 128] = torch.round(t / step) * step
    return q, s


def same_codes(x, q, s):
    rq, rs = quantized(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu().double(), rq)


@pytest.mark.gpu
@pytest.mark.parametrize("T,cols", [(1, 16), (1, 128), (3, 144), (1, 4096), (7, 2064), (130, 272), (64, 4096), (5, 8192),
                                    (1000, 1008)])
def test_quantize_is_exact(T, cols):
    x = activations(T + cols, T, cols)
    same_codes(x, *B.iqk_fp8_quantize(x))


@pytest.mark.gpu
def test_quantize_borders():
    """Quotients on and next to rounding borders: every pair of a bfloat16
    mantissa and a largest magnitude's mantissa, over the exponents down to
    e4m3's subnormal numbers."""
    a = torch.arange(128, 256, dtype=torch.float64)
    for shift in range(0, 20):
        x = (a[None, :] * 2.0 ** -shift).repeat(128, 1)            # [128 largest][128 mantissas]
        x[:, ::2] *= -1
        top = a[:, None] * 2.0                                     # larger than every one of them
        x = torch.cat([x[:, :112], top, x[:, :15]], 1), torch.cat([x[:, 112:], top, x[:, :111]], 1)
        for v in x:
            v = v.bfloat16().cuda()
            same_codes(v, *B.iqk_fp8_quantize(v.contiguous()))


@pytest.mark.gpu
def test_quantize_extremes():
    x = activations(3, 12, 256)
    x[0] = 0
    x[1] = 0
    x[1, 5] = 2.0 ** -130
    x[2] = torch.finfo(torch.bfloat16).max
    x[3] = -torch.finfo(torch.bfloat16).tiny
    x[4, :128] = 2.0 ** -99
    x[5, 100] = torch.finfo(torch.bfloat16).max
    same_codes(x, *B.iqk_fp8_quantize(x))
    x[7, 3] = math.inf
    x[8, 130] = -math.inf
    x[9, 127] = math.nan
    x[10] = math.nan
    q, s = B.iqk_fp8_quantize(x)
    bad = torch.tensor([[7, 0], [8, 1], [9, 0], [10, 0], [10, 1]])
    mask = torch.zeros((12, 2), dtype=torch.bool)
    mask[bad[:, 0], bad[:, 1]] = True
    assert torch.equal(torch.isnan(s.cpu()), mask)
    q = q.cpu().float().view(12, 2, 128)
    assert (q[mask] == 0).all()
    x = x.clone().view(12, 2, 128)
    x[mask.cuda()] = 0
    rq, _ = quantized(x.view(12, 256))
    assert torch.equal(q.view(12, 256).double(), rq)


@pytest.mark.gpu
def test_quantize_strides_and_neighbours():
    wide = activations(8, 33, 1000)
    q = torch.full((35, 272), 3, dtype=torch.uint8, device="cuda")
    s = torch.full((35, 3), -1.0, device="cuda")
    for off in (0, 8, 200):
        x = wide[:, off:off + 272]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        a, b = B.iqk_fp8_quantize(x, q=q[1:34].view(E4M3), s=s[1:34], stream=st)
        st.synchronize()
        same_codes(x, a, b)
    assert (q[0] == 3).all() and (q[34] == 3).all() and (s[0] == -1).all() and (s[34] == -1).all()
    with pytest.raises(ValueError):
        B.iqk_fp8_quantize(wide[:, 4:276])  # rows not 16-byte aligned


# ------------------------------------------------------------------ products

def check_linear(T, rows, cols, dtype, add, seed=0):
    wq, ws = operand(seed + 1, rows, cols, 128)
    xq, xs = operand(seed + 2, T, cols, 1)
    extra = torch.randn((T, rows), generator=gen(seed + 3)).to(dtype).cuda() if add else None
    buf = torch.full((T * rows + 64,), -5.0, dtype=dtype, device="cuda")
    y = B.iqk_fp8_linear(wq, ws, xq, xs, add=extra, y=buf[:T * rows].view(T, rows))
    assert B.iqk_fp8_status() == B.IQK_OK
    ref, S, tol = product(wq, ws, xq, xs)
    if add:
        ref = ref + extra.double()
        tol = tol + 2.0 ** -23 * ref.abs()
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    err = (y.double() - ref).abs()
    bound = tol * (1 + half) + half * ref.abs()
    assert (err <= bound).all(), float((err / bound).max())
    assert (buf[T * rows:] == -5).all()
    return wq, ws, xq, xs, y


SIZES = [(1, 16, 16), (1, 1, 128), (1, 4096, 2048), (2, 100, 144), (8, 256, 4096), (9, 33, 272), (16, 2048, 1008),
         (17, 128, 128), (17, 20, 16), (33, 1000, 2064), (64, 512, 4096), (127, 129, 400), (128, 128, 256), (129, 257, 1040),
         (200, 4096, 512), (333, 1000, 2064), (700, 4100, 384), (1300, 2050, 272), (2500, 2048, 128), (4000, 1301, 272), (2900, 2100, 400),
         (8200, 700, 144), (513, 8192, 656),
         (3900, 800, 1040)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(T, rows, cols, dtype):
    check_linear(T, rows, cols, dtype, add=False)
    check_linear(T, rows, cols, dtype, add=True, seed=10)


@pytest.mark.gpu
@pytest.mark.parametrize("T", list(range(1, 20)) + [31, 32, 48, 63, 65])
def test_linear_every_small_batch(T):
    check_linear(T, 144, 640, torch.float32, add=False, seed=T)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_linear_adds_in_place_and_repeats_bitwise(T):
    wq, ws, xq, xs, y = check_linear(T, 520, 2064, torch.bfloat16, add=False)
    z = torch.randn((T, 520), generator=gen(4)).bfloat16().cuda()
    a = B.iqk_fp8_linear(wq, ws, xq, xs, add=z)
    w = z.clone()
    assert B.iqk_fp8_linear(wq, ws, xq, xs, add=w, y=w) is w
    assert torch.equal(a.view(torch.int16), w.view(torch.int16))
    for _ in range(3):
        assert torch.equal(B.iqk_fp8_linear(wq, ws, xq, xs).view(torch.int16), y.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 30, 60, 2300])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_outputs_at_any_element(T, dtype):
    """y and add one element off the alignment that wide stores need."""
    rows = 2048
    wq, ws = operand(1, rows, 272, 128)
    xq, xs = operand(2, T, 272, 1)
    z = torch.randn((T * rows + 1,), generator=gen(3)).to(dtype).cuda()[1:].view(T, rows)
    buf = torch.full((T * rows + 3,), -5.0, dtype=dtype, device="cuda")
    a = B.iqk_fp8_linear(wq, ws, xq, xs, add=z, y=buf[1:-2].view(T, rows))
    assert torch.equal(a, B.iqk_fp8_linear(wq, ws, xq, xs, add=z.clone()))
    assert buf[0] == -5 and (buf[-2:] == -5).all()


def far_operands(T, rows, cols, weights=1):
    """Operands whose scales' products leave float32's normal numbers although
    the results do not. Even tokens: 2^130 and more (in every third block),
    under the smallest codes of both operands in one column of the block and
    zeros; odd ones: 2^-142 to 2^-133 (in the block behind), under ordinary
    codes, and scales of 0. Returns xq, xs and (codes, scales) of each weight
    matrix; the scales of the second are ordinary where the first's are not."""
    nkb = blocks(cols)
    kind = torch.arange(nkb) % 3
    xq, xs = operand(1, T, cols, 1)
    x = xq.view(torch.uint8)
    x[::2] &= 0x80         # signed zeros ...
    x[::2, ::128] |= 1     # ... and 2^-9
    r = (1 + torch.rand((T, nkb), generator=gen(2))).cuda()
    xs[::2] = torch.where((kind == 0).cuda(), r[::2] * 2.0 ** 70, torch.zeros(()).cuda())
    xs[1::2] = torch.where((kind == 1).cuda(), r[1::2] * torch.exp2(torch.linspace(-82, -74, nkb)).cuda(), torch.zeros(()).cuda())
    out = []
    for n in range(weights):
        wq, ws = operand(3 + 2 * n, rows, cols, 128)
        w = wq.view(torch.uint8)
        w[:, ::128] &= 0x83    # at most 3 * 2^-9
        r = (1 + torch.rand(ws.shape, generator=gen(8 + n))).cuda()
        far = [(60.0, -60.0), (-60.0, 100.0)][n]
        ws = torch.where((kind == 0).cuda(), r * 2.0 ** far[0], torch.where((kind == 1).cuda(), r * 2.0 ** far[1], ws))
        out.append((wq, ws))
    return (xq, xs, *out)


FAR_SIZES = [(1, 144, 512), (5, 528, 4096), (24, 144, 400), (40, 528, 2064), (300, 1008, 400), (700, 2064, 272),
             (2600, 1104, 400), (5200, 2096, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,rows,cols", FAR_SIZES)
def test_linear_scales_of_any_size(T, rows, cols):
    """Only the result has to be in float32's range. Two roundings for a block
    instead of one (its sum times one scale, then times the other) are within
    the 8 that the bound counts; 2^-148 for each block is what is lost below
    float32's normal numbers."""
    xq, xs, (wq, ws) = far_operands(T, rows, cols)
    y = B.iqk_fp8_linear(wq, ws, xq, xs, dtype=torch.float32)
    ref, S, tol = product(wq, ws, xq, xs)
    assert 2.0 ** 100 < S[::2].max() < 2.0 ** 127 and (T == 1 or 2.0 ** -126 < S[1::2].max() < 2.0 ** -100)
    err = (y.double() - ref).abs()
    assert (err <= tol * (1 + 2.0 ** -24) + 2.0 ** -24 * ref.abs() + 2.0 ** -148 * blocks(cols)).all()
    xq.view(torch.uint8)[0] = 0  # a token of zeros under the largest scales
    assert (B.iqk_fp8_linear(wq, ws, xq, xs, dtype=torch.float32)[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,rows,cols", FAR_SIZES)
def test_gate_up_scales_of_any_size(T, rows, cols):
    """As check_h, with either matrix's products out of range."""
    xq, xs, *w = far_operands(T, rows, cols, 2)
    for (gq, gs), (uq, us) in (w, w[::-1]):
        q, s = B.iqk_fp8_gate_up(gq, gs, uq, us, xq, xs)
        g, _, dg = product(gq, gs, xq, xs)
        u, _, du = product(uq, us, xq, xs)
        dg, du = dg + 2.0 ** -148 * blocks(cols), du + 2.0 ** -148 * blocks(cols)
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -20 * h.abs() + 2.0 ** -148
        for b in range(blocks(rows)):
            c = slice(b * 128, min((b + 1) * 128, rows))
            m, dm = h[:, c].abs().amax(1), dh[:, c].amax(1)
            assert (m > 2.0 ** -100).all()
            assert ((s[:, b].double() - m / 448).abs() <= dm / 448 + 2.0 ** -22 * m / 448).all()
            sb = s[:, b].double()[:, None]
            bound = (2.0 ** -4 * (h[:, c].abs() + dh[:, c]) + 2.0 ** -10 * sb + dh[:, c]) * (1 + 2.0 ** -20)
            assert ((q[:, c].double() * sb - h[:, c]).abs() <= bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 150])
def test_linear_nan_stays_in_its_row(T):
    wq, ws = operand(1, 64, 512, 128)
    xq, xs = operand(2, T, 512, 1)
    xs[1, 2] = math.nan
    y = B.iqk_fp8_linear(wq, ws, xq, xs, dtype=torch.float32)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[torch.arange(T) != 1]).all()


def check_h(T, inter, cols, seed=0):
    """With g and u within their products' bounds dg, du, h = silu(g) u in
    float32 is within dh = 1.1 dg (|u| + du) + |silu(g)| du + 2^-20 |h| of the
    exact one (|silu'| <= 1.1). The scale is then within max dh / 448 and
    2^-22 of exact, and q s within half an e4m3 step of h: 2^-4 of it, or half
    of 2^-9 s for the smallest; the scale's own error moves 448 h / m by the
    same relative amount, covered by dh's share below."""
    gq, gs = operand(seed + 1, inter, cols, 128)
    uq, us = operand(seed + 2, inter, cols, 128)
    xq, xs = operand(seed + 3, T, cols, 1)
    nb = blocks(inter)
    qbuf = torch.full((T * inter + 64,), 3, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((T * nb + 16,), -1.0, device="cuda")
    q, s = B.iqk_fp8_gate_up(gq, gs, uq, us, xq, xs, q=qbuf[:T * inter].view(T, inter).view(E4M3),
                             s=sbuf[:T * nb].view(T, nb))
    assert B.iqk_fp8_status() == B.IQK_OK
    g, _, dg = product(gq, gs, xq, xs)
    u, _, du = product(uq, us, xq, xs)
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -20 * h.abs()
    for b in range(nb):
        c = slice(b * 128, min((b + 1) * 128, inter))
        m, dm = h[:, c].abs().amax(1), dh[:, c].amax(1)
        err = (s[:, b].double() - m.clamp(min=2.0 ** -100) / 448).abs()
        assert (err <= dm / 448 + 2.0 ** -22 * m / 448 + 2.0 ** -120).all()
        sb = s[:, b].double()[:, None]
        got = q[:, c].double() * sb
        bound = (2.0 ** -4 * (h[:, c].abs() + dh[:, c]) + 2.0 ** -10 * sb + dh[:, c]) * (1 + 2.0 ** -20)
        assert ((got - h[:, c]).abs() <= bound).all()
        assert (q[:, c].double().abs().amax(1) == 448).all()  # the largest magnitude is the largest code
    assert (qbuf[T * inter:] == 3).all() and (sbuf[T * nb:] == -1).all()
    return gq, gs, uq, us, xq, xs, q, s


@pytest.mark.gpu
@pytest.mark.parametrize("T,inter,cols", [(1, 16, 16), (1, 128, 128), (1, 2048, 4096), (3, 144, 272), (8, 512, 1008),
                                          (9, 2048, 512), (16, 272, 4096), (17, 128, 128), (17, 16, 16), (40, 2048, 2064),
                                          (128, 256, 1024), (130, 400, 640), (333, 1040, 272), (1500, 2048, 256), (2700, 1040, 272), (1025, 2000, 1040)])
def test_gate_up(T, inter, cols):
    *ops, q, s = check_h(T, inter, cols)
    a, b = B.iqk_fp8_gate_up(*ops)
    assert torch.equal(a.view(torch.uint8), q.view(torch.uint8)) and torch.equal(b, s)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 150])
def test_gate_up_zero_and_not_finite_rows(T):
    gq, gs = operand(1, 256, 512, 128)
    uq, us = operand(2, 256, 512, 128)
    xq, xs = operand(3, T, 512, 1)
    xs[0] = 0
    xs[1, 0] = math.nan
    q, s = B.iqk_fp8_gate_up(gq, gs, uq, us, xq, xs)
    assert (q[0].float() == 0).all() and (s[0] == np.float32(2.0 ** -100) / np.float32(448)).all()
    assert (q[1].float() == 0).all() and torch.isnan(s[1]).all()
    assert torch.isfinite(s[2:]).all()
    assert torch.isnan(B.iqk_fp8_linear(*operand(4, 32, 256, 128), q, s)[1]).all()


@pytest.mark.gpu
def test_no_tokens():
    wq, ws = operand(1, 64, 256, 128)
    xq, xs = operand(2, 4, 256, 1)
    assert B.iqk_fp8_linear(wq, ws, xq[:0], xs[:0]).shape == (0, 64)
    q, s = B.iqk_fp8_gate_up(wq, ws, wq, ws, xq[:0], xs[:0])
    assert q.shape == (0, 64) and s.shape == (0, 1)
    q, s = B.iqk_fp8_quantize(torch.zeros((0, 256), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 elements behind the first row: of y, and of x and q."""
    T, rows, cols = 65536, 33000, 16
    wq, ws = operand(1, rows, cols, 128)
    xq, xs = operand(2, T, cols, 1)
    y = B.iqk_fp8_linear(wq, ws, xq, xs)
    assert y.numel() > 2 ** 31
    at = torch.tensor([0, 1, 40000, 65080, 65081, 65534, 65535], device="cuda")  # 2^31 elements end in row 65075
    ref, _, tol = product(wq, ws, xq[at.cpu()].contiguous(), xs[at.cpu()].contiguous())
    assert ((y[at].double() - ref).abs() <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()).all()
    del y
    T, cols = 140000, 16384
    x = torch.zeros((T, cols), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 131071, 131072, 139999], device="cuda")
    x[at] = activations(5, len(at), cols)
    q, s = B.iqk_fp8_quantize(x)
    same_codes(x[at], q.view(torch.uint8)[at].view(E4M3), s[at])
    assert not q.view(torch.uint8)[1000].any()


@pytest.mark.gpu
def test_products_follow_one_another():
    """Every product kernel right behind every other, many times over: what one
    leaves in an SM's shared or tensor memory is complete when the next takes it."""
    calls, alone = [], []
    for n, (T, rows, cols, gate_up) in enumerate([(1, 1040, 1024, False), (9, 528, 272, True), (40, 1040, 1024, False),
                                                  (40, 528, 640, True), (700, 2050, 144, False), (1300, 2050, 272, False),
                                                  (1300, 2064, 16, True), (2600, 1040, 128, True)]):
        wq, ws = operand(n, rows, cols, 128)
        uq, us = operand(n + 50, rows, cols, 128)
        xq, xs = operand(n + 100, T, cols, 1)
        if gate_up:
            def call(a=(wq, ws, uq, us, xq, xs)):
                q, s = B.iqk_fp8_gate_up(*a)
                return q.view(torch.uint8), s.view(torch.int32)
        else:
            def call(a=(wq, ws, xq, xs)):
                return (B.iqk_fp8_linear(*a).view(torch.int16),)
        calls.append(call)
        alone.append([t.clone() for t in call()])
        torch.cuda.synchronize()
    order = torch.randint(0, len(calls), (40, 25), generator=gen(9)).tolist()
    for some in order:
        outs = [calls[i]() for i in some]
        torch.cuda.synchronize()
        for i, out in zip(some, outs):
            assert all(torch.equal(a, b) for a, b in zip(out, alone[i])), i
    assert B.iqk_fp8_status() == B.IQK_OK


# ------------------------------------------------------------------ refusals

def test_refusals_on_the_host():
    L = B.lib()
    P = 4096

    def quant(x=P, stride=256, T=2, cols=256, q=P, s=P):
        return L.iqk_fp8_quantize(x, stride, T, cols, q, s, None)

    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(x=P + 2), dict(q=P + 4), dict(s=P + 2), dict(T=-1),
               dict(stride=255), dict(stride=260)):
        assert quant(**kw) == B.IQK_EINVAL, kw
    assert quant(cols=0) == quant(cols=24) == quant(cols=-16) == B.IQK_ESHAPE
    assert quant(T=1 << 30, cols=256) == B.IQK_EUNSUPPORTED
    assert quant(T=0, x=None, q=None, s=None) == B.IQK_OK

    def linear(wq=P, ws=P, rows=64, cols=256, xq=P, xs=P, T=2, add=None, y=P, dt=1):
        return L.iqk_fp8_linear(wq, ws, rows, cols, xq, xs, T, add, y, dt, None)

    for kw in (dict(wq=None), dict(ws=None), dict(xq=None), dict(xs=None), dict(y=None), dict(wq=P + 8), dict(xq=P + 8),
               dict(ws=P + 2), dict(xs=P + 2), dict(y=P + 1), dict(add=P + 1), dict(y=P + 2, dt=0), dict(dt=2), dict(T=-1)):
        assert linear(**kw) == B.IQK_EINVAL, kw
    assert linear(rows=0) == linear(cols=0) == linear(cols=100) == B.IQK_ESHAPE
    assert linear(T=65537) == linear(rows=2 ** 30 + 1) == B.IQK_EUNSUPPORTED
    assert linear(T=65536, cols=2 ** 23) == linear(rows=2 ** 26, cols=2 ** 20) == B.IQK_EUNSUPPORTED
    assert linear(cols=2 ** 31 - 16, T=200) == B.IQK_EUNSUPPORTED
    assert linear(T=0, xq=None, xs=None, y=None) == B.IQK_OK

    def gate_up(gq=P, gs=P, uq=P, us=P, inter=64, cols=256, xq=P, xs=P, T=2, hq=P, hs=P):
        return L.iqk_fp8_gate_up(gq, gs, uq, us, inter, cols, xq, xs, T, hq, hs, None)

    for kw in (dict(gq=None), dict(gs=None), dict(uq=None), dict(us=None), dict(xq=None), dict(xs=None), dict(hq=None),
               dict(hs=None), dict(uq=P + 8), dict(hq=P + 4), dict(T=-1)):
        assert gate_up(**kw) == B.IQK_EINVAL, kw
    assert gate_up(inter=8) == gate_up(inter=24) == gate_up(cols=8) == B.IQK_ESHAPE
    assert gate_up(T=65537) == B.IQK_EUNSUPPORTED
    assert gate_up(T=0, xq=None, xs=None, hq=None, hs=None) == B.IQK_OK
    w = torch.zeros((32, 256), dtype=torch.uint8).view(E4M3)
    with pytest.raises(ValueError):
        B.iqk_fp8_linear(w, torch.zeros((1, 2)), w, torch.zeros((32, 2)))  # not on a GPU
    with pytest.raises(ValueError):
        B.iqk_fp8_quantize(torch.zeros((2, 256), dtype=torch.bfloat16))


@pytest.mark.gpu
def test_refusals_of_tensors():
    wq, ws = operand(1, 64, 256, 128)
    xq, xs = operand(2, 4, 256, 1)
    oq, os_ = operand(3, 4, 272, 1)
    uq, us = operand(4, 80, 256, 128)
    bf, f32 = torch.zeros((4, 64), dtype=torch.bfloat16).cuda(), torch.zeros((4, 64)).cuda()
    for bad in (lambda: B.iqk_fp8_linear(wq, ws, oq, os_), lambda: B.iqk_fp8_linear(wq, ws[:, :1], xq, xs),
                lambda: B.iqk_fp8_linear(wq, ws, xq, xs[:3]), lambda: B.iqk_fp8_linear(wq, ws.double(), xq, xs),
                lambda: B.iqk_fp8_linear(wq.view(torch.uint8), ws, xq, xs), lambda: B.iqk_fp8_linear(wq[:, :128], ws, xq, xs),
                lambda: B.iqk_fp8_linear(wq, ws, xq, xs, add=bf, y=f32), lambda: B.iqk_fp8_linear(wq, ws, xq, xs, y=bf[:3]),
                lambda: B.iqk_fp8_linear(wq, ws, xq, xs, dtype=torch.float16),
                lambda: B.iqk_fp8_linear(wq, ws, xq, xs, y=bf.cpu()), lambda: B.iqk_fp8_linear(wq[0], ws, xq, xs),
                lambda: B.iqk_fp8_gate_up(wq, ws, uq, us, xq, xs), lambda: B.iqk_fp8_gate_up(wq, ws, wq, ws, oq, os_),
                lambda: B.iqk_fp8_gate_up(wq, ws, wq, ws, xq, xs, q=torch.empty((4, 64)).cuda()),
                lambda: B.iqk_fp8_quantize(f32), lambda: B.iqk_fp8_quantize(bf.t()),
                lambda: B.iqk_fp8_quantize(torch.zeros((4, 24), dtype=torch.bfloat16).cuda())):
        with pytest.raises(ValueError):
            bad()
