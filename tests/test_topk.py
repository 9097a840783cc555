"""iqk_moe_topk against the definition in 64 bits: ids exactly, weights within
float32's error, masks, ties, groups, layouts; refusals on the host (CPU).

Tolerance of a weight: relative (d + E / 32 + 64) 2^-24 with d the largest
distance between the row's finite logits that enter an exponential. An
exponential's argument is rounded once (d 2^-24 absolute, so relative in the
exponential), expf is within 2 ulp, a sum over E experts adds E / 32 + 5
roundings, and the quotient, the sigmoid's sum and the scale a few more; 64
covers these constants. Below float32's normal range 2^-126 is allowed.
"""
import math

import numpy as np
import pytest

from gemm_iq2_ks_b200 import binding as B

torch = pytest.importorskip("torch")


def reference(x, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """ids [T, k], p [T, k] by sorting each row in float64."""
    x = x.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    T, E = x.shape
    ids, ps = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        r = x[t]
        dead = ~(r > -math.inf)
        with np.errstate(invalid="ignore", over="ignore"):
            if score == "softmax":
                m = r[~dead].max() if (~dead).any() else 0.0
                e = np.where(dead, 0.0, np.where(r == m, 1.0, np.exp(np.where(dead, 0.0, r) - m)))
                s = e / e.sum() if e.sum() > 0 else e
            else:
                s = np.where(dead, 0.0, 1.0 / (1.0 + np.exp(-np.where(dead, 0.0, r))))
        if b is not None:
            dead = dead | ~(b > -math.inf)
        v = np.where(dead, -math.inf, s + b if b is not None else r)
        allowed = list(range(E))
        if groups > 1:
            w = np.where(dead, -math.inf, s + (b if b is not None else 0.0)) if group_top == 2 else v
            n, val = E // groups, []
            for g in range(groups):
                best = sorted((float(z) for z in w[g * n:(g + 1) * n]), reverse=True)[:group_top]
                val.append(best[0] + sum(z for z in best[1:] if z > -math.inf))
            chosen = sorted(range(groups), key=lambda g: (-val[g], g))[:topk_groups]
            allowed = [e for e in range(E) if e // n in chosen]
        pick = sorted(allowed, key=lambda e: (-v[e], e))[:k]
        ids[t] = pick
        p = np.where(dead[pick], 0.0, s[pick])
        if renorm and not dead[pick].all():
            # the ratio in exact arithmetic, through logarithms: scores may lie below float64's range
            z = np.where(dead[pick], 0.0, r[pick])
            with np.errstate(over="ignore", invalid="ignore"):
                if score == "sigmoid":
                    z = np.where(z > 0, -np.log1p(np.exp(-z)), z - np.log1p(np.exp(z)))
                m = z[~dead[pick]].max()
                p = np.where(dead[pick], 0.0, np.where(z == m, 1.0, np.exp(z - m)))
            p = p / p.sum()
        ps[t] = p * scale
    return ids, ps


def check(x, k, what="", **kw):
    ids, p = B.iqk_moe_topk(x, k, **kw)
    ri, rp = reference(x, k, **kw)
    got = ids.cpu().numpy()
    assert np.array_equal(got, ri), f"{what}: rows {np.nonzero((got != ri).any(1))[0][:5]} differ"
    f = x.double()
    f = f[torch.isfinite(f)]
    d = float(f.max() - f.min()) if f.numel() else 0.0
    tol = (min(d, 104.0) + x.shape[1] / 32 + 64) * 2.0 ** -24
    err = np.abs(p.double().cpu().numpy() - rp)
    assert (err <= tol * np.abs(rp) + 2.0 ** -126 * kw.get("scale", 1.0)).all(), f"{what}: {err.max()}"


def logits(seed, T, E, dtype=torch.float32, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, E), generator=g)).to(dtype).cuda()


def bias_of(seed, E):
    return (0.05 * torch.randn((E,), generator=torch.Generator().manual_seed(seed))).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 2, 7, 8, 31, 32, 33, 64, 100, 128, 160, 250, 256, 384, 512, 1000, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_every_width(E, dtype, score):
    for T, k in [(1, min(E, 6)), (37, min(E, 16)), (3, 1)]:
        x = logits(E + T, T, E, dtype)
        for renorm in (True, False):
            check(x, k, f"E {E} T {T}", score=score, renorm=renorm, scale=2.5)
            check(x, k, f"E {E} T {T} bias", score=score, renorm=renorm, bias=bias_of(E, E))


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,topk_groups", [(256, 8, 4), (256, 8, 1), (64, 4, 3), (60, 5, 2), (96, 3, 3), (32, 32, 9),
                                                  (1024, 32, 7), (512, 2, 1), (1008, 7, 5), (26, 13, 6)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups(E, groups, topk_groups, group_top):
    k = min(8, topk_groups * (E // groups))
    for dtype in (torch.float32, torch.bfloat16):
        for score in ("softmax", "sigmoid"):
            for bias in (None, bias_of(3, E)):
                check(logits(E + groups, 65, E, dtype), k, f"{dtype} {score}", score=score, bias=bias, groups=groups,
                      topk_groups=topk_groups, group_top=group_top)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [48, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_and_extremes(score, renorm, E, dtype):
    k = 8
    x = logits(5, 12, E)
    x[0] = -math.inf                      # nothing left
    x[1, 3:] = -math.inf                  # fewer than k
    x[2, ::2] = math.nan
    x[3] = math.nan
    x[4, 7] = math.inf
    x[5, [7, 40, 9]] = math.inf
    x[6] = torch.finfo(torch.float32).min
    x[7, 5:] = torch.finfo(torch.float32).min
    x[8] = -80.0 - torch.arange(E).cuda() / 8  # sigmoid and softmax tails
    x[9] = 0.0
    x[9, ::3] = -0.0                      # the two zeros tie
    x[10] = torch.finfo(torch.float32).max
    open_bias = bias_of(1, E)
    shut_bias = open_bias.clone()
    shut_bias[:E - 4] = -math.inf
    shut_bias[E - 3] = math.nan
    forced = open_bias.clone()
    forced[[2, 30]] = math.inf
    x = x.to(dtype)  # the lowest float32 becomes -inf in bfloat16
    for bias in (None, open_bias, shut_bias, forced):
        check(x, k, "plain", score=score, renorm=renorm, bias=bias)
        for group_top in (1, 2):
            check(x, 6, f"groups {group_top}", score=score, renorm=renorm, bias=bias, groups=8, topk_groups=2,
                  group_top=group_top)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_follow_float64(score):
    """Selection values that float32 cannot tell apart: the bias undoes the
    scores' order but for less than 2^-24, in either direction; and equal ones."""
    E, T = 64, 64
    g = torch.Generator().manual_seed(9)
    x = torch.randn((1, E), generator=g).expand(T, E).contiguous()
    x = x + 2.0 ** -22 * torch.randint(-2, 3, (T, E), generator=g)
    s = torch.softmax(x[0].double(), -1) if score == "softmax" else torch.sigmoid(x[0].double())
    bias = (1.0 - s).float()  # every selection value is 1 but for roundings
    bias[10:20] = bias[9]
    x[:, 10:20] = x[:, 9:10]  # true ties
    check(x.cuda(), 16, "near", score=score, bias=bias.cuda())
    check(x.cuda(), 5, "near, groups", score=score, bias=bias.cuda(), groups=8, topk_groups=3, group_top=2)
    zero = torch.zeros((E,)).cuda()
    check(x.bfloat16().cuda(), 16, "bf16 ties", score=score, bias=zero)
    check(x.bfloat16().cuda(), 6, "bf16 ties, groups", score=score, bias=zero, groups=4, topk_groups=2, group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [32, 256, 1024])
@pytest.mark.parametrize("spread", [1.0, 6.0])
def test_near_ties_of_far_logits(score, E, spread):
    """As above with logits far apart, where the hardware exponential's error is
    largest: selection values that differ by 2^-24 of the largest score to 2^-18."""
    T = 512
    g = torch.Generator().manual_seed(E)
    x = spread * torch.randn((1, E), generator=g)
    s = torch.softmax(x[0].double(), -1) if score == "softmax" else torch.sigmoid(x[0].double())
    top = float(s.max())
    bias = (top - s + top * torch.exp2(torch.randint(-24, -17, (E,), generator=g).double())).float()
    x = (x * (1 + 2.0 ** -22 * torch.randint(-4, 5, (T, 1), generator=g))).cuda()
    check(x, 16, "far", score=score, bias=bias.cuda())
    check(x, 6, "far, groups", score=score, bias=bias.cuda(), groups=8, topk_groups=3, group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_outputs_and_streams(dtype):
    """Rows inside a wider matrix at any offset, on another stream, into given
    outputs with neighbours that stay as they were."""
    T, E, k = 19, 128, 6
    wide = logits(3, T, 300, dtype)
    ids = torch.full((T + 2, k), -7, dtype=torch.int32, device="cuda")
    p = torch.full((T + 2, k), -7.0, device="cuda")
    for off in (0, 1, 8, 37):
        x = wide[:, off:off + E]
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            a, b = B.iqk_moe_topk(x, k, ids=ids[1:T + 1], p=p[1:T + 1])
        c, d = B.iqk_moe_topk(x, k, stream=st)
        st.synchronize()
        ri, _ = reference(x, k)
        assert np.array_equal(a.cpu().numpy(), ri) and torch.equal(a, c) and torch.equal(b, d)
    assert (ids[0] == -7).all() and (ids[-1] == -7).all() and (p[0] == -7).all() and (p[-1] == -7).all()
    e, f = B.iqk_moe_topk(wide[:0], k)
    assert e.shape == (0, k) and f.shape == (0, k)


def choice(x, k, score, bias, groups, topk_groups, group_top):
    """reference()'s ids for many rows at once, for rows with a bias and without masks."""
    x = x.double()
    v = (torch.softmax(x, -1) if score == "softmax" else torch.sigmoid(x)) + bias.double()
    T, E = v.shape
    val = v.view(T, groups, -1).topk(group_top, -1).values.sum(-1)
    best = torch.sort(val, dim=-1, descending=True, stable=True).indices[:, :topk_groups]
    open_ = torch.zeros((T, groups), dtype=torch.bool, device=v.device).scatter_(1, best, True)
    v = torch.where(open_.repeat_interleave(E // groups, 1), v, -math.inf)
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[:, :k].int()


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,off", [(160, 8, 0), (256, 8, 1), (60, 5, 0), (512, 32, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_doubtful_rows_among_ordinary_ones(E, groups, off, dtype):
    """Rows whose groups tie, which the float64 pass orders, between ordinary
    ones: the warps of a block are then at different passes at once."""
    T, k, n = 8192, 6, E // groups
    wide = logits(E, T, E + 8, dtype)
    x = wide[:, off:off + E]
    tied = torch.rand((T,), generator=torch.Generator().manual_seed(1)).cuda() < 0.4
    x[tied] = 0.25
    bias = bias_of(2, n).repeat(groups)  # alike in every group
    for group_top in (1, 2):
        kw = dict(score="sigmoid", bias=bias, groups=groups, topk_groups=groups // 2, group_top=group_top)
        want = choice(x, k, **kw)
        for _ in range(5):
            ids, _ = B.iqk_moe_topk(x, k, **kw)
            assert torch.equal(ids, want)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups,off", [(16, 8, 0), (256, 8, 0), (256, 8, 1), (160, 8, 0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(E, groups, off, score):
    """Groups whose two best values are large and of opposite sign: the sum's
    error follows the two, not the little that is left of them."""
    T, n = 20000, E // groups
    x = logits(E + off, T, E + 8)[:, off:off + E]
    for size in (4096.0, 3.0e38):
        bias = torch.full((E,), -size).cuda()
        bias[::n] = size
        kw = dict(score=score, bias=bias, groups=groups, topk_groups=groups // 2, group_top=2)
        ids, _ = B.iqk_moe_topk(x, 6, **kw)
        assert torch.equal(ids, choice(x, 6, **kw)), size


@pytest.mark.gpu
@pytest.mark.parametrize("E,off", [(16, 0), (256, 0), (256, 1)])
def test_group_sums_past_float32(E, off):
    """A group whose two best values add up to less than float32's lowest
    number is still ahead of one that is masked throughout."""
    T, n = 64, E // 8
    x = logits(E + off, T, E + 8)[:, off:off + E]
    bias = torch.full((E,), -3.0e38).cuda()
    bias[:3 * n] = -math.inf
    for topk_groups in (2, 5, 6):
        check(x, 2 * topk_groups, f"open {topk_groups}", score="sigmoid", bias=bias, groups=8, topk_groups=topk_groups,
              group_top=2)


@pytest.mark.gpu
def test_many_tokens():
    x = logits(11, 65536, 256, torch.bfloat16)
    ids, p = B.iqk_moe_topk(x, 6)
    order = torch.sort(x.float(), dim=-1, descending=True, stable=True)
    assert torch.equal(ids.long(), order.indices[:, :6])
    ref = torch.softmax(order.values[:, :6].double(), -1)
    assert ((p.double() - ref).abs() <= 96 * 2.0 ** -24 * ref).all()


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    """Rows 2^23 elements apart, the last ones more than 2^31 elements behind the first."""
    T, E, stride = 300, 64, 1 << 23
    flat = torch.empty((T * stride,), dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((T, E), (stride, 1))
    x.copy_(logits(4, T, E, torch.bfloat16))
    check(x, 6, "far rows")


@pytest.mark.gpu
def test_as_many_rows_as_an_int_counts():
    """T = 2^31 - 1 rows of one expert: the last block is rounded up past it."""
    T = 2 ** 31 - 1
    x = torch.zeros((T, 1), dtype=torch.bfloat16, device="cuda")
    ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    _, p = B.iqk_moe_topk(x, 1, ids=ids)
    assert int(ids.amin()) == int(ids.amax()) == 0
    assert float(p.amin()) == float(p.amax()) == 1.0


def test_refusals_on_the_host():
    L = B.lib()

    def call(logits=4096, dtype=0, stride=64, T=3, E=64, k=4, score=0, bias=None, groups=1, tg=1, gt=1, ids=4096, p=4096):
        return L.iqk_moe_topk(logits, dtype, stride, T, E, k, score, bias, groups, tg, gt, 1, 1.0, ids, p, None)

    for kw in (dict(dtype=2), dict(score=2), dict(T=-1), dict(E=0), dict(k=0), dict(k=65), dict(groups=0), dict(groups=3),
               dict(tg=0), dict(tg=2), dict(gt=0), dict(gt=3), dict(groups=16, tg=1, k=5), dict(stride=63),
               dict(logits=None), dict(ids=None), dict(p=None), dict(logits=4098), dict(dtype=1, logits=4097),
               dict(bias=4098), dict(ids=4098), dict(p=4097)):
        assert call(**kw) == B.IQK_EINVAL, kw
    for kw in (dict(E=1025, stride=2000), dict(k=17), dict(E=66, stride=66, groups=33, tg=33)):
        assert call(**kw) == B.IQK_EUNSUPPORTED, kw
    assert call(T=0, logits=None, ids=None, p=None) == B.IQK_OK
    with pytest.raises(ValueError):
        B.iqk_moe_topk(torch.zeros((2, 8)), 2)  # not on a GPU


@pytest.mark.gpu
def test_refusals_of_tensors():
    x = logits(1, 4, 64)
    for bad in (lambda: B.iqk_moe_topk(x.half(), 2), lambda: B.iqk_moe_topk(x.t(), 2), lambda: B.iqk_moe_topk(x[0], 2),
                lambda: B.iqk_moe_topk(x, 2, score="tanh"), lambda: B.iqk_moe_topk(x, 65), lambda: B.iqk_moe_topk(x, 0),
                lambda: B.iqk_moe_topk(x, 2, bias=torch.zeros(63, device="cuda")),
                lambda: B.iqk_moe_topk(x, 2, bias=torch.zeros(64)),
                lambda: B.iqk_moe_topk(x, 2, ids=torch.zeros((4, 2), dtype=torch.int64, device="cuda")),
                lambda: B.iqk_moe_topk(x, 2, p=torch.zeros((4, 4), device="cuda")[:, :2]),
                lambda: B.iqk_moe_topk(x[:1].expand(4, 64), 2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        B.iqk_moe_topk(logits(1, 2, 64), 17)
