"""One layer's feed-forward part with the operators together: router logits to
experts (iqk_moe_topk), the routed experts (iqk_moe_decode / iqk_moe_prefill),
and the shared expert in 8 bits (iqk_fp8_quantize, iqk_fp8_gate_up,
iqk_fp8_linear added onto the routed output in place).

Kernels overlap their launches (each waits for its predecessor before it reads
anything), so the calls made back to back, on other streams and replayed from
a graph must equal, bit for bit, the same calls with the device synchronised
between them; each stage is checked against its definition on its own inputs.
"""
import numpy as np
import pytest

import iqk_synth as S
from oracle import oracle as O
from util import check_block, from_dev_bf16, to_dev_bf16

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_fp8 as F  # noqa: E402
import test_topk as R  # noqa: E402
from gemm_iq2_ks_b200 import binding as B  # noqa: E402

E, H, I, K = 32, 512, 768, 6


class Layer:
    def __init__(self, seed, T, prefill):
        rng = S.rng_for(seed)
        # small row scales keep chained layers (quadratic through SwiGLU) finite
        self.host = [S.random_streams(rng, "iq2_ks", E, r, c, dv_range=(3e-4, 5e-4)) for r, c in ((I, H), (I, H), (H, I))]
        self.gate, self.up, self.down = (B.Weights.from_host(w) for w in self.host)
        self.values = S.value_table("dyadic", 8)
        self.router = (torch.randn((E, H), generator=F.gen(seed)) * H ** -0.5).cuda()
        self.bias = R.bias_of(seed, E)
        self.gq, self.gs = self.dense(seed + 1, I, H)
        self.uq, self.us = self.dense(seed + 2, I, H)
        self.dq, self.ds = self.dense(seed + 3, H, I)
        self.moe = B.iqk_moe_prefill if prefill else B.iqk_moe_decode
        self.ws = B.workspace(B.iqk_moe_workspace_bytes(1 if prefill else 0, T, K, E, H, I))
        f32, bf, dev = torch.float32, torch.bfloat16, "cuda"
        self.logits = torch.empty((T, E), dtype=f32, device=dev)
        self.ids, self.p = torch.empty((T, K), dtype=torch.int32, device=dev), torch.empty((T, K), dtype=f32, device=dev)
        self.routed, self.y = (torch.empty((T, H), dtype=bf, device=dev) for _ in range(2))
        self.xq, self.xs = torch.empty((T, H), dtype=F.E4M3, device=dev), torch.empty((T, H // 128), device=dev)
        self.hq, self.hs = torch.empty((T, I), dtype=F.E4M3, device=dev), torch.empty((T, I // 128), device=dev)

    def dense(self, seed, rows, cols):
        w = torch.randn((rows, cols), generator=F.gen(seed)) * cols ** -0.5
        s = torch.full(((rows + 127) // 128, cols // 128), 0.01)
        return (w / 0.01).to(F.E4M3).cuda(), s.cuda()

    def run(self, x, sync=False):
        def step():
            if sync:
                torch.cuda.synchronize()
        torch.matmul(x.float(), self.router.t(), out=self.logits)
        step()
        B.iqk_moe_topk(self.logits, K, score="sigmoid", bias=self.bias, groups=8, topk_groups=4, group_top=2,
                       ids=self.ids, p=self.p)
        step()
        self.moe(self.gate, self.up, self.down, self.values, x, self.ids, self.p, y=self.y, ws=self.ws)
        step()
        if sync:
            self.routed.copy_(self.y)
        B.iqk_fp8_quantize(x, q=self.xq, s=self.xs)
        step()
        B.iqk_fp8_gate_up(self.gq, self.gs, self.uq, self.us, self.xq, self.xs, q=self.hq, s=self.hs)
        step()
        B.iqk_fp8_linear(self.dq, self.ds, self.hq, self.hs, add=self.y, y=self.y)
        step()
        return self.y


@pytest.mark.parametrize("T,prefill", [(1, False), (12, False), (40, False), (150, True)])
def test_layer(T, prefill):
    L = Layer(30 + T, T, prefill)
    xb = S.random_bf16(S.rng_for(7), (T, H))
    x = to_dev_bf16(xb)
    y = L.run(x, sync=True).clone()
    kept = [t.clone() for t in (L.ids, L.p, L.xq.view(torch.uint8), L.xs, L.hq.view(torch.uint8), L.hs)]

    # every stage against its definition
    ids, _ = R.reference(L.logits, K, score="sigmoid", bias=L.bias, groups=8, topk_groups=4, group_top=2)
    assert np.array_equal(L.ids.cpu().numpy(), ids)
    p = L.p.cpu().numpy()
    ref = O.moe(*L.host, L.values, xb, ids.astype(np.int32), p)
    check_block(from_dev_bf16(L.routed), None, ref, L.host[2], L.values, ids.astype(np.int32), p, f"layer T {T}")
    F.same_codes(x, L.xq, L.xs)
    g, _, dg = F.product(L.gq, L.gs, L.xq, L.xs)
    u, _, du = F.product(L.uq, L.us, L.xq, L.xs)
    h = g * torch.sigmoid(g) * u
    dh = 1.1 * dg * (u.abs() + du) + (g * torch.sigmoid(g)).abs() * du + 2.0 ** -20 * h.abs()
    got = F.value(L.hq, L.hs, 1)
    step = L.hs.double().repeat_interleave(128, 1)
    assert ((got - h).abs() <= (2.0 ** -4 * (h.abs() + dh) + 2.0 ** -10 * step + dh) * (1 + 2.0 ** -20)).all()
    d, _, tol = F.product(L.dq, L.ds, L.hq, L.hs)
    d = d + L.routed.double()
    err = (y.double() - d).abs()
    assert (err <= (tol + 2.0 ** -23 * d.abs()) * (1 + 2.0 ** -8) + 2.0 ** -8 * d.abs()).all()

    def same(what):
        torch.cuda.synchronize()
        assert torch.equal(L.y.view(torch.int16), y.view(torch.int16)), what
        now = (L.ids, L.p, L.xq.view(torch.uint8), L.xs, L.hq.view(torch.uint8), L.hs)
        assert all(torch.equal(a, b) for a, b in zip(now, kept)), what

    for _ in range(3):
        L.run(x)
    same("back to back")
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        L.run(x)
    same("another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            for _ in range(2):
                L.run(x)
    for t in (L.y, L.ids, L.p, L.xs, L.hs):
        t.zero_()
    graph.replay()
    graph.replay()
    same("replayed")
    assert B.iqk_moe_status(L.ws) == B.IQK_OK and B.iqk_fp8_status() == B.IQK_OK


@pytest.mark.parametrize("T", [2, 40, 700])
def test_two_streams_and_two_graphs_at_once(T):
    """The operators keep no state between calls: equal calls on two streams and
    in two graphs running together give what they give alone."""
    wq, ws = F.operand(1, 1040, 1024, 128)
    uq, us = F.operand(2, 1040, 1024, 128)
    xs = [F.operand(3 + i, T, 1024, 1) for i in range(2)]
    lg = [R.logits(5 + i, T, 96) for i in range(2)]

    def run(i):
        q, s = B.iqk_fp8_gate_up(wq, ws, uq, us, *xs[i])
        return [B.iqk_fp8_linear(wq, ws, *xs[i]).view(torch.int16), q.view(torch.uint8), s, *B.iqk_moe_topk(lg[i], 5)]

    alone = []
    for i in range(2):
        alone.append([t.clone() for t in run(i)])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(run(i))
    torch.cuda.synchronize()
    graphs, held = [], []
    for i, st in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(st), torch.cuda.graph(g, stream=st):
            held.append([run(i) for _ in range(3)])
        graphs.append(g)
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i] + held[i]:
            assert all(torch.equal(a, b) for a, b in zip(o, alone[i]))


def pool_of(t):
    """The stream whose pool of the caching allocator a tensor's memory is from."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_memory_of_a_call_is_from_its_streams_pool():
    """What a call on a given stream allocates is ordered by that stream: a
    block of the current stream's pool may still be written to there."""
    T = 40
    wq, ws = F.operand(1, 528, 512, 128)
    xq, xs = F.operand(2, T, 512, 1)
    x, lg = F.activations(3, T, 512), R.logits(4, T, 96)
    rng = S.rng_for(3)
    w = B.Weights.from_host(S.random_streams(rng, "iq2_ks", 4, 512, 512))
    values = S.value_table("dyadic", 8)
    ids = torch.zeros((T, 2), dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    calls = [lambda **k: B.iqk_moe_topk(lg, 5, **k), lambda **k: B.iqk_fp8_quantize(x, **k),
             lambda **k: [B.iqk_fp8_linear(wq, ws, xq, xs, **k)], lambda **k: B.iqk_fp8_gate_up(wq, ws, wq, ws, xq, xs, **k),
             lambda **k: [B.iqk_dequant(w, 1, values, **k)], lambda **k: [B.iqk_gemv(w, 1, values, x[:2], **k)],
             lambda **k: [B.iqk_switch_linear(w, values, x, ids, **k)], lambda **k: B.iqk_moe_route(ids, 4, **k)[:3]]
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        got = call(stream=st)
        assert all(pool_of(t) == st.cuda_stream for t in got)
        assert all(pool_of(t) != st.cuda_stream for t in want)
        st.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("T", [1, 9, 300])
def test_weights_written_just_before_the_call_are_read(T):
    """Stream order holds for weights and scales, too."""
    wq, ws = F.operand(1, 520, 1024, 128)
    vq, vs = F.operand(2, 520, 1024, 128)
    xq, xs = F.operand(3, T, 1024, 1)
    a = B.iqk_fp8_linear(wq, ws, xq, xs).clone()
    b = B.iqk_fp8_linear(vq, vs, xq, xs).clone()
    torch.cuda.synchronize()
    q, s = torch.empty_like(wq), torch.empty_like(ws)
    outs = []
    for i in range(6):
        src = (wq, ws) if i % 2 == 0 else (vq, vs)
        q.view(torch.uint8).copy_(src[0].view(torch.uint8))
        s.copy_(src[1])
        outs.append(B.iqk_fp8_linear(q, s, xq, xs))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o.view(torch.int16), (a if i % 2 == 0 else b).view(torch.int16)), i


FIRST = """
import sys
import torch
sys.path[:0] = [{root!r}, {tests!r}]
from gemm_iq2_ks_b200 import binding as B
import test_fp8 as F, test_topk as R
T = int(sys.argv[1])
wq, ws = F.operand(1, 512, 512, 128)
xq, xs = F.operand(2, T, 512, 1)
x, lg = F.activations(3, T, 512), R.logits(4, T, 96)
y = torch.empty((T, 512), dtype=torch.bfloat16, device="cuda")
q, s = torch.empty((T, 512), dtype=F.E4M3, device="cuda"), torch.empty((T, 4), device="cuda")
h, hs = torch.empty_like(q), torch.empty_like(s)
ids, p = torch.empty((T, 5), dtype=torch.int32, device="cuda"), torch.empty((T, 5), device="cuda")
def run():
    B.iqk_moe_topk(lg, 5, groups=4, topk_groups=2, ids=ids, p=p)
    B.iqk_fp8_quantize(x, q=q, s=s)
    B.iqk_fp8_linear(wq, ws, xq, xs, y=y)
    B.iqk_fp8_gate_up(wq, ws, wq, ws, xq, xs, q=h, s=hs)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
a = [t.clone() for t in (y, q.view(torch.uint8), s, h.view(torch.uint8), hs, ids, p)]
run()
torch.cuda.synchronize()
assert all(torch.equal(u, v) for u, v in zip(a, (y, q.view(torch.uint8), s, h.view(torch.uint8), hs, ids, p)))
print("captured")
"""


@pytest.mark.parametrize("T", [1, 20, 100, 3000])
def test_a_process_may_capture_its_first_calls(T):
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(root=os.path.dirname(tests), tests=tests)
    r = subprocess.run([sys.executable, "-c", code, str(T)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
