"""GPU: the grouped products and the adapters as a program uses them: a training step of a layer of experts and
a serving step (adapters, then block-scaled experts), the offsets written on the device; the same calls
captured into a graph and replayed; calls on another stream, and two at once with a workspace each."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import check
from test_gpu_grouped_mx import codes
from gpu_util import say

pytestmark = pytest.mark.gpu


class Step:
    """One layer: tokens x (T, K) each sent to two of E experts with weights w1 (E, H, K) and w2 (E, K, H) and no
    activation between, so that its gradients are products: y = x w1^T w2^T summed over a token's experts."""

    def __init__(self, T=150, K=136, H=264, E=7, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.K, self.H, self.E = T, K, H, E
        grid = lambda *s: (torch.randint(-4, 5, s, generator=g) / 4).bfloat16().cuda()
        self.x, self.w1, self.w2 = grid(T, K), grid(E, H, K), grid(E, K, H)
        self.dy = grid(2 * T, K)
        self.choice = torch.stack([torch.randperm(E, generator=g)[:2] for _ in range(T)]).flatten().cuda()
        self.choice[self.choice == 3] = 4                     # expert 3 gets no row
        n = 2 * T
        self.offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        e = lambda *s, dt=torch.bfloat16: torch.full(s, float("nan"), dtype=dt, device="cuda")
        self.xs, self.h, self.dh = e(n, K), e(n, H), e(n, H)
        self.y, self.dx = e(n, K, dt=torch.float32), e(n, K, dt=torch.float32)
        self.dw1, self.dw2 = e(E, H, K, dt=torch.float32), e(E, K, H, dt=torch.float32)

    def route(self):
        """The router's part, in torch: rows sorted by expert and the experts' offsets, all on the device."""
        order = torch.argsort(self.choice, stable=True)
        counts = torch.zeros(self.E, dtype=torch.int32, device="cuda").scatter_add_(
            0, self.choice, torch.ones_like(self.choice, dtype=torch.int32))
        self.offsets[1:] = torch.cumsum(counts, 0)
        self.xs.copy_(self.x[order // 2])

    def products(self, stream=None):
        n, K, H, E, o = 2 * self.T, self.K, self.H, self.E, self.offsets
        g = lambda *a, **k: bsm.bsm_gemm_grouped(n, *a, stream=stream, **k)
        g(H, K, E, o, "bf16", self.xs, K, self.w1, K, "k", H * K, "bf16", self.h, H)
        g(K, H, E, o, "bf16", self.h, H, self.w2, H, "k", K * H, "f32", self.y, K)
        g(H, K, E, o, "bf16", self.dy, K, self.w2, H, "n", K * H, "bf16", self.dh, H)
        g(K, H, E, o, "bf16", self.dh, H, self.w1, K, "n", H * K, "f32", self.dx, K)
        w = lambda *a: bsm.bsm_gemm_grouped_wgrad(n, *a, stream=stream)
        w(K, H, E, o, "bf16", self.dy, K, self.h, H, "f32", self.dw2, H, K * H)
        w(H, K, E, o, "bf16", self.dh, H, self.xs, K, "f32", self.dw1, K, H * K)

    def outputs(self):
        return {k: getattr(self, k).clone() for k in ("h", "y", "dh", "dx", "dw1", "dw2")}

    def poison(self):
        for k in ("h", "y", "dh", "dx", "dw1", "dw2"):
            getattr(self, k).fill_(float("nan"))


def test_training_step():
    s = Step()
    s.route()
    s.products()
    torch.cuda.synchronize()
    off = s.offsets.tolist()
    cpu = lambda t: t.double().cpu()
    for e in range(s.E):
        a, b = off[e], off[e + 1]
        x, h, dy, dh = cpu(s.xs[a:b]), cpu(s.h[a:b]), cpu(s.dy[a:b]), cpu(s.dh[a:b])
        w1, w2 = cpu(s.w1[e]), cpu(s.w2[e])
        p = lambda u, v: (u @ v, u.abs() @ v.abs())
        check(s.h[a:b], *p(x, w1.T), s.K, "bf16", "h")
        check(s.y[a:b], *p(h, w2.T), s.H, "f32", "y")
        check(s.dh[a:b], *p(dy, w2), s.K, "bf16", "dh")
        check(s.dx[a:b], *p(dh, w1), s.H, "f32", "dx")
        check(s.dw2[e], *p(dy.T, h), b - a, "f32", "dw2")
        check(s.dw1[e], *p(dh.T, x), b - a, "f32", "dw1")
    assert off[3] == off[4] and not s.dw1[3].any() and not s.dw2[3].any()


def test_training_step_in_a_graph_and_on_another_stream():
    """A captured step with a new routing before each replay equals the eager step on the same routing, bit for
    bit; so does the step on a stream of its own."""
    s = Step(seed=3)
    side = torch.cuda.Stream()
    s.route()
    s.products()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.products()
    for k in range(4):
        say("graph replay", k)
        s.choice = (s.choice + 1) % s.E if k else s.choice
        s.route()
        s.poison()
        s.products()
        torch.cuda.synchronize()
        want = s.outputs()
        s.poison()
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.poison()
        torch.cuda.synchronize()
        s.products(stream=side)
        side.synchronize()
        other = s.outputs()
        for name in want:
            assert torch.equal(got[name], want[name]), (k, name)
            assert torch.equal(other[name], want[name]), (k, name)


class Serve:
    """A projection with adapters, then block-scaled experts on codes of their own."""

    def __init__(self, T, seed):
        g = torch.Generator().manual_seed(seed)
        self.T, self.K, self.N, self.R, self.L = T, 200, 136, 12, 5
        mk = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
        self.x, self.w = mk(T, 200), mk(136, 200)
        self.la, self.lb = mk(5, 12, 200), mk(5, 136, 16)
        self.ids = (torch.randint(0, 6, (T,), generator=g) - 1).int().cuda()
        self.scale = torch.rand(5, generator=g).cuda()
        self.ws = torch.full((bsm.bsm_gemm_lora_workspace(T, 12),), 255, dtype=torch.uint8, device="cuda")
        self.d = torch.empty(T, 136, dtype=torch.bfloat16, device="cuda")
        self.xq, self.xqs, _ = (t.cuda() for t in codes(g, (T,), 192, "e4m3"))
        self.wq, self.wqs, _ = (t.cuda() for t in codes(g, (3, 72), 192, "e2m1"))
        self.off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
        self.q = torch.empty(T, 72, dtype=torch.bfloat16, device="cuda")

    def go(self, stream=None):
        bsm.bsm_gemm_lora(self.T, 136, 200, 12, 5, self.ids, "bf16", self.x, 200, self.w, 200, self.la, 200, 2400, self.lb, 16,
                          136 * 16, self.scale, self.ws, "bf16", self.d, 136, stream=stream)
        bsm.bsm_gemm_grouped_block_scale(self.T, 72, 192, 3, self.off, "e4m3", self.xq, 192, self.xqs, self.xqs.stride(0), "e2m1",
                                         self.wq, 192, 72 * 192, self.wqs, self.wqs.stride(1), self.wqs.stride(0), 0, "bf16",
                                         self.q, 72, stream=stream)

    def poison(self):
        self.d.fill_(float("nan"))
        self.q.fill_(float("nan"))


@pytest.mark.parametrize("T", [1, 20, 64, 90, 400])
def test_serving_step_in_graphs_and_two_at_once(T):
    a, b = Serve(T, 1), Serve(T, 2)
    for s in (a, b):
        s.go()
    torch.cuda.synchronize()
    want = [(s.d.clone(), s.q.clone()) for s in (a, b)]
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.go()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def same(what):
        torch.cuda.synchronize()
        for s, (d, q) in zip((a, b), want):
            assert torch.equal(s.d, d) and torch.equal(s.q, q), what
            s.poison()
        torch.cuda.synchronize()

    same("eager")
    for k in range(3):
        say("serve", T, k)
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        same("two graphs at once")
        for s, st in zip((a, b), streams):
            s.go(stream=st)
        same("two streams at once")
