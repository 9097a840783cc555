"""Measured cases of the routing, 8-bit quantisation and 8-bit product operators.

The operators stand around the routed experts of one layer (256 experts, six
selected, hidden width 4096, expert width 2048 in this repository's benchmark):

  topk      router logits to the experts of each token and their weights
  quantize  bf16 activations to e4m3 with one scale per token and 128 columns
  linear    y = x w^T of two e4m3 operands, the weights scaled per 128 x 128 block
  gate_up   the same product for a gate and an up matrix, silu(gate) * up, and
            its quantisation: what the down product of a dense expert reads

``run`` computes them with elementary torch operations, or, where ``own`` is
set, through the library's entry points. ``exact`` evaluates the definitions
in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128  # columns of a scale
LARGEST = 448.0  # largest e4m3 number
SMALLEST = 2.0 ** -100  # a group's largest magnitude counts as at least this


# ------------------------------------------------------------------- cases

def _topk(name, T, experts, k, dtype="f32", score="softmax", bias=False, groups=1, topk_groups=1, group_top=1,
          renorm=True, scale=1.0, masked=0.0):
    return {"name": name, "op": "topk", "T": T, "experts": experts, "k": k, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "topk_groups": topk_groups, "group_top": group_top, "renorm": renorm,
            "scale": scale, "masked": masked}


def listed():
    return [
        # one decoded token of the benchmark's layer: launch latency
        _topk("topk_1x256_top6", 1, 256, 6),
        # a prompt through grouped, bias-balanced sigmoid routing
        _topk("topk_2048x256_grouped", 2048, 256, 8, score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2,
              scale=2.5),
        # the most tokens a routed prefill takes, logits as a bf16 product leaves them
        _topk("topk_65536x256_bf16", 65536, 256, 6, dtype="bf16"),
        # one token's hidden row
        {"name": "quantize_1x4096", "op": "quantize", "T": 1, "cols": 4096, "pad": 0},
        # a long prompt's rows, a column slice of a wider activation
        {"name": "quantize_8192x4096_slice", "op": "quantize", "T": 8192, "cols": 4096, "pad": 2048},
        # decode: down product of one token, added onto the routed experts' output
        {"name": "linear_1x4096x2048_add", "op": "linear", "T": 1, "rows": 4096, "cols": 2048, "out": "bf16",
         "add": True},
        # a decode batch, the most tokens a routed decode takes
        {"name": "linear_64x4096x4096", "op": "linear", "T": 64, "rows": 4096, "cols": 4096, "out": "bf16",
         "add": False},
        # a short prompt at ragged widths, float32 out
        {"name": "linear_333x1000x2064_f32", "op": "linear", "T": 333, "rows": 1000, "cols": 2064, "out": "f32",
         "add": False},
        # a long prompt
        {"name": "linear_8192x4096x4096", "op": "linear", "T": 8192, "rows": 4096, "cols": 4096, "out": "bf16",
         "add": False},
        # decode and prompt forms of the fused gate/up step
        {"name": "gate_up_1x2048x4096", "op": "gate_up", "T": 1, "inter": 2048, "cols": 4096},
        {"name": "gate_up_16x2048x4096", "op": "gate_up", "T": 16, "inter": 2048, "cols": 4096},
        {"name": "gate_up_2048x2048x4096", "op": "gate_up", "T": 2048, "inter": 2048, "cols": 4096},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number between lo and hi, uniform over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("topk", "quantize", "linear", "gate_up"))
    if op == "topk":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        topk_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, experts // groups * topk_groups))
        c = _topk("", _log(rng, 1, 65536 * 256 // max(256, experts)), experts, k, dtype=rng.choice(("f32", "bf16")),
                  score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups,
                  topk_groups=topk_groups, group_top=rng.choice((1, 2)), renorm=rng.random() < 0.7,
                  scale=rng.choice((1.0, 2.5)), masked=rng.choice((0.0, 0.0, 0.02)))
        del c["name"]
        return c
    if op == "quantize":
        cols = _log(rng, 128, 8192, 16)
        return {"op": "quantize", "T": _log(rng, 1, 8192 * 4096 // max(4096, cols)), "cols": cols,
                "pad": rng.choice((0, 0, 8, 2048))}
    if op == "linear":
        return {"op": "linear", "T": _log(rng, 1, 8192), "rows": _log(rng, 16, 4096), "cols": _log(rng, 128, 4096, 16),
                "out": rng.choice(("bf16", "f32")), "add": rng.random() < 0.3}
    return {"op": "gate_up", "T": _log(rng, 1, 2048), "inter": _log(rng, 64, 2048, 16),
            "cols": _log(rng, 128, 4096, 16)}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    T = case["T"]
    if case["op"] == "topk":
        E, k = case["experts"], case["k"]
        item = 4 if case["dtype"] == "f32" else 2
        # a score and a comparison for each expert
        return {"bytes": T * E * item + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    cols = case["cols"]
    if case["op"] == "quantize":
        return {"bytes": T * cols * 3 + 4 * T * _blocks(cols), "flops": 2 * T * cols}
    x = T * cols + 4 * T * _blocks(cols)
    if case["op"] == "linear":
        rows, item = case["rows"], 2 if case["out"] == "bf16" else 4
        w = rows * cols + 4 * _blocks(rows) * _blocks(cols)
        return {"bytes": x + w + T * rows * item * (2 if case["add"] else 1), "flops": 2 * T * rows * cols}
    inter = case["inter"]
    w = 2 * (inter * cols + 4 * _blocks(inter) * _blocks(cols))
    return {"bytes": x + w + T * inter + 4 * T * _blocks(inter), "flops": 4 * T * inter * cols}


# ------------------------------------------------------------------ inputs

def _activations(g, T, cols):
    """Rows of unit variance with a few loud columns, as hidden states have."""
    x = torch.randn((T, cols), generator=g, device="cuda")
    loud = torch.rand((cols,), generator=g, device="cuda") < 0.01
    return torch.where(loud, 8.0 * x, x).to(torch.bfloat16)


def _quantized(x):
    """e4m3 codes and scales of x, per row and 128 columns."""
    T, cols = x.shape
    pad = _blocks(cols) * BLOCK - cols
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(T, -1, BLOCK)
    most = v.abs().amax(-1).clamp(min=SMALLEST)
    q = (v * LARGEST / most[..., None]).view(T, -1)[:, :cols]
    return q.to(torch.float8_e4m3fn).contiguous(), most / LARGEST


def _weights(g, rows, cols):
    """e4m3 weights with a scale for each 128 x 128 block."""
    w = torch.randn((rows, cols), generator=g, device="cuda") * cols ** -0.5
    r, c = _blocks(rows), _blocks(cols)
    p = torch.nn.functional.pad(w, (0, c * BLOCK - cols, 0, r * BLOCK - rows)).view(r, BLOCK, c, BLOCK)
    s = p.abs().amax((1, 3)).clamp(min=SMALLEST) / LARGEST
    q = (p / s[:, None, :, None]).view(r * BLOCK, c * BLOCK)[:rows, :cols]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = dict(case)
    T = case["T"]
    if case["op"] == "topk":
        E = case["experts"]
        # experts differ in how often they are wanted
        x = 1.5 * torch.randn((T, E), generator=g, device="cuda") + torch.randn((E,), generator=g, device="cuda")
        if case["masked"]:  # experts out of service, and padding tokens that want none
            x[:, torch.rand((E,), generator=g, device="cuda") < case["masked"]] = -math.inf
            x[torch.rand((T,), generator=g, device="cuda") < case["masked"]] = -math.inf
        st["logits"] = x if case["dtype"] == "f32" else x.to(torch.bfloat16)
        st["b"] = 0.05 * torch.randn((E,), generator=g, device="cuda") if case["bias"] else None
        st["ids"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
        st["p"] = torch.empty((T, case["k"]), device="cuda")
        return st
    cols = case["cols"]
    if case["op"] == "quantize":
        st["x"] = _activations(g, T, cols + case["pad"])[:, :cols]
        st["q"] = torch.empty((T, cols), dtype=torch.float8_e4m3fn, device="cuda")
        st["s"] = torch.empty((T, _blocks(cols)), device="cuda")
        return st
    st["xq"], st["xs"] = _quantized(_activations(g, T, cols))
    if case["op"] == "linear":
        st["wq"], st["ws"] = _weights(g, case["rows"], cols)
        dtype = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        st["y"] = torch.empty((T, case["rows"]), dtype=dtype, device="cuda")
        st["more"] = (torch.randn((T, case["rows"]), generator=g, device="cuda").to(dtype) if case["add"] else None)
        return st
    st["gq"], st["gs"] = _weights(g, case["inter"], cols)
    st["uq"], st["us"] = _weights(g, case["inter"], cols)
    st["q"] = torch.empty((T, case["inter"]), dtype=torch.float8_e4m3fn, device="cuda")
    st["s"] = torch.empty((T, _blocks(case["inter"])), device="cuda")
    return st


# ----------------------------------------------------------------- one pass

def run(st):
    if own:
        return _library(st)
    return {"topk": _plain_topk, "quantize": lambda s: _plain_quantize(s["x"].float()), "linear": _plain_linear,
            "gate_up": _plain_gate_up}[st["op"]](st)


def _library(st):
    from gemm_iq2_ks_b200 import binding as B
    if st["op"] == "topk":
        ids, p = B.iqk_moe_topk(st["logits"], st["k"], score=st["score"], bias=st["b"], groups=st["groups"],
                                topk_groups=st["topk_groups"], group_top=st["group_top"], renorm=st["renorm"],
                                scale=st["scale"], ids=st["ids"], p=st["p"])
        return {"ids": ids, "p": p}
    if st["op"] == "quantize":
        q, s = B.iqk_fp8_quantize(st["x"], q=st["q"], s=st["s"])
        return {"q": q, "s": s}
    if st["op"] == "linear":
        return {"y": B.iqk_fp8_linear(st["wq"], st["ws"], st["xq"], st["xs"], add=st["more"], y=st["y"])}
    q, s = B.iqk_fp8_gate_up(st["gq"], st["gs"], st["uq"], st["us"], st["xq"], st["xs"], q=st["q"], s=st["s"])
    return {"q": q, "s": s}


def _plain_topk(st):
    """Experts by descending selection value, ties to the lowest index.

    The value is the logit, or score + bias with a bias; masked experts (a
    logit or bias of -inf or NaN) come last and get no weight. Values that
    decide next to a border are formed in 64 bits.
    """
    k, groups, b = st["k"], st["groups"], st["b"]
    x = st["logits"].float()
    T, E = x.shape
    masked = torch.isnan(x) | (x == -math.inf)
    x = torch.where(masked, -math.inf, x).double()
    if st["score"] == "softmax":
        most = x.amax(-1, keepdim=True)
        e = torch.where(x == most, 1.0, torch.exp(x - most))
        e = torch.where(x == -math.inf, 0.0, e)
        total = e.sum(-1, keepdim=True)
        s = torch.where(total > 0, e / total, 0.0)
    else:
        s = torch.where(x == -math.inf, 0.0, 1.0 / (1.0 + torch.exp(-x)))
    rank = x
    if b is not None:
        masked = masked | torch.isnan(b) | (b == -math.inf)
        rank = s + b.double()
    rank = torch.where(masked, -math.inf, rank)
    allowed = torch.ones_like(masked)
    if groups > 1:
        per = torch.where(masked, -math.inf, rank if st["group_top"] == 1 or b is not None else s)
        per = torch.sort(per.view(T, groups, -1), dim=-1, descending=True).values
        value = per[..., 0]
        if st["group_top"] == 2 and E // groups > 1:
            value = value + torch.where(per[..., 1] == -math.inf, 0.0, per[..., 1])
        best = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, : st["topk_groups"]]
        open_ = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        allowed = open_[:, :, None].expand(T, groups, E // groups).reshape(T, E)
    # two stable orders, the allowed experts first: a closed expert is behind a masked one
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    first = torch.sort(allowed.gather(1, order).to(torch.uint8), dim=-1, descending=True, stable=True).indices
    order = order.gather(1, first)
    ids = order[:, :k]
    p = torch.where(masked.gather(1, ids), 0.0, s.gather(1, ids))
    if st["renorm"]:
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    return {"ids": ids.to(torch.int32), "p": (p * st["scale"]).float()}


def _plain_quantize(x):
    """q = e4m3(448 x / most), s = most / 448 with the largest magnitude of 128 columns."""
    T, cols = x.shape
    v = torch.nn.functional.pad(x, (0, _blocks(cols) * BLOCK - cols)).view(T, -1, BLOCK)
    most = v.abs().amax(-1)
    fine = torch.isfinite(most)
    most = torch.where(fine, most, 1.0).clamp(min=SMALLEST)
    q = torch.where(fine[..., None], v * LARGEST / most[..., None], 0.0)
    return {"q": q.view(T, -1)[:, :cols].to(torch.float8_e4m3fn), "s": torch.where(fine, most / LARGEST, math.nan)}


def _spread(s, n):
    return s.repeat_interleave(BLOCK, -1)[..., :n]


def _product(xq, xs, wq, ws):
    """x w^T of the values that codes and scales stand for, in 32 bits."""
    x = xq.float() * _spread(xs, xq.shape[1])
    w = wq.float() * _spread(ws.repeat_interleave(BLOCK, 0)[: wq.shape[0]], wq.shape[1])
    return torch.matmul(x, w.t())


def _plain_linear(st):
    y = _product(st["xq"], st["xs"], st["wq"], st["ws"])
    if st["more"] is not None:
        y = y + st["more"].float()
    return {"y": y.to(st["y"].dtype)}


def _plain_gate_up(st):
    g = _product(st["xq"], st["xs"], st["gq"], st["gs"])
    u = _product(st["xq"], st["xs"], st["uq"], st["us"])
    return _plain_quantize(g / (1.0 + torch.exp(-g)) * u)


# ---------------------------------------------------------- 64-bit reference

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "topk":
        return _exact_topk(st)
    if case["op"] == "quantize":
        return _exact_quantize(st["x"].double())
    if case["op"] == "linear":
        y = _exact_product(st["xq"], st["xs"], st["wq"], st["ws"])
        return {"y": y if st["more"] is None else y + st["more"].double()}
    g = _exact_product(st["xq"], st["xs"], st["gq"], st["gs"])
    u = _exact_product(st["xq"], st["xs"], st["uq"], st["us"])
    return _exact_quantize(g * torch.sigmoid(g) * u)


def _exact_product(xq, xs, wq, ws):
    """The definition: sum over 128-column blocks of scale times the codes' product."""
    y = torch.zeros((xq.shape[0], wq.shape[0]), dtype=torch.float64, device=xq.device)
    row = torch.arange(wq.shape[0], device=xq.device) // BLOCK
    for b in range(xs.shape[1]):
        c = slice(b * BLOCK, min((b + 1) * BLOCK, xq.shape[1]))
        part = xq[:, c].double() @ wq[:, c].double().t()
        y += part * xs[:, b, None].double() * ws[row, b].double()
    return y


def _exact_quantize(x):
    """Nearest e4m3 number, ties to even: multiples of 2^(e-3) in [2^e, 2^(e+1)), of 2^-9 below 2^-6."""
    q, s = torch.zeros_like(x), torch.zeros((x.shape[0], _blocks(x.shape[1])), dtype=torch.float64, device=x.device)
    for b in range(s.shape[1]):
        v = x[:, b * BLOCK: (b + 1) * BLOCK]
        most = v.abs().amax(-1).clamp(min=SMALLEST)
        s[:, b] = most / LARGEST
        t = v * LARGEST / most[:, None]
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, b * BLOCK: (b + 1) * BLOCK] = torch.round(t / step) * step
    return {"q": q, "s": s}


def _exact_topk(st):
    """Each expert's place is the number of experts ahead of it."""
    E, k, groups = st["experts"], st["k"], st["groups"]
    x = st["logits"].double()
    b = st["b"].double() if st["b"] is not None else torch.zeros((E,), dtype=torch.float64, device=x.device)
    ids, ps = [], []
    at = torch.arange(E, device=x.device)

    def places(v):
        n = torch.arange(v.shape[-1], device=v.device)
        ahead = (v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & (n[None, :] < n[:, None]))
        return ahead.sum(-1)

    for x in x.split(max(1, (1 << 26) // (E * E))):
        dead = ~(x > -math.inf)
        s = torch.sigmoid(x) if st["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, -1))
        s = torch.where(dead, 0.0, s)
        v = torch.where(dead, -math.inf, s + b if st["b"] is not None else x)
        if groups > 1:
            w = torch.where(dead, -math.inf, s + b) if st["group_top"] == 2 or st["b"] is not None else v
            two = w.view(len(x), groups, -1).topk(min(st["group_top"], E // groups), -1).values
            total = torch.where(two[..., 0] == -math.inf, -math.inf, torch.where(two == -math.inf, 0.0, two).sum(-1))
            closed = places(total).repeat_interleave(E // groups, -1) >= st["topk_groups"]
        else:
            closed = torch.zeros_like(dead)
        # a masked expert of an open group stands behind the others there, a closed one behind all
        place = places(torch.where(closed, -1e300, torch.where(dead, -1e200, v)))
        pick = torch.zeros_like(place).scatter_(1, place, at.expand(len(x), E))[:, :k]
        p = s.gather(1, pick)
        if st["renorm"]:
            p = torch.nan_to_num(p / p.sum(-1, keepdim=True))
        ids.append(pick.to(torch.int32))
        ps.append(p * st["scale"])
    return {"ids": torch.cat(ids), "p": torch.cat(ps)}
