"""GPU: a training step of a layer of experts as a program makes it: the router's counts, offsets and balance loss; rows
kept in 8 bits, the experts' products, their activation, the head's cross entropy and its gradients; then backward through
the activation and into the weights from what was kept. Captured into a graph and replayed with new routings and
labels between; on other streams; two at once with a workspace each."""
import pytest
import torch

import block_scaled_matrix_amd as bsm
from grouped_util import check, up
from test_gpu_checkpoint import F8, values
from test_gpu_router import reference as balance_reference
from xent_util import reference as head_reference
from gpu_util import say

pytestmark = pytest.mark.gpu
OUT = ("counts", "offsets", "balance", "xq", "xf", "zq", "zf", "a", "y", "loss", "lse", "dy", "dwo", "da", "dw2", "dz", "dw1", "dx", "dl")


class Step:
    """T tokens to k of E experts, w1 (E, H, K), silu, w2 (E, K, H), a head wo (V, K) on every expert's row."""

    def __init__(self, T=150, K=136, H=264, E=7, V=1003, k=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.K, self.H, self.E, self.V, self.k, self.n = T, K, H, E, V, k, T * k
        r = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).bfloat16().cuda()
        self.x, self.w1, self.w2, self.wo = r(T, K), r(E, H, K, by=K ** -0.5), r(E, K, H, by=H ** -0.5), r(V, K, by=K ** -0.5)
        self.logits = torch.randn(T, E, generator=g).cuda()
        self.labels = torch.randint(-1, V, (self.n,), generator=g, dtype=torch.int32).cuda()
        self.dloss = (torch.rand(self.n, generator=g) / self.n).cuda()
        self.coef = torch.tensor([0.01], device="cuda")
        e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")
        n, u8, f32 = self.n, torch.uint8, torch.float32
        self.ids = e(T, k, dt=torch.int32)
        self.counts, self.offsets, self.balance = e(E + 1, dt=torch.int32), e(E + 1, dt=torch.int32), e(1, dt=f32)
        self.xs, self.xq, self.xf = e(n, K), e(n, up(K, 16), dt=u8), e(n, up(up(K, 32) // 32, 4), dt=u8)
        self.z, self.zq, self.zf, self.a = e(n, H), e(n, up(H, 16), dt=u8), e(n, up(up(H, 32) // 32, 4), dt=u8), e(n, H)
        self.y, self.loss, self.lse, self.dy = e(n, K), e(n, dt=f32), e(n, dt=f32), e(n, K)
        self.dwo, self.dw2, self.dw1 = e(V, K, dt=f32), e(E, K, H, dt=f32), e(E, H, K, dt=f32)
        self.da, self.dz, self.dx, self.dl = e(n, H), e(n, H), e(n, K), e(T, E, dt=f32)
        self.wb = e(bsm.bsm_router_balance_workspace(T, E), dt=u8)
        self.wl = e(bsm.bsm_gemm_cross_entropy_workspace(n, V), dt=u8)
        self.wg = e(bsm.bsm_gemm_cross_entropy_grad_workspace(n, V, K, 512), dt=u8)

    def choose(self):
        """The router's choice in torch; the last tokens are padding and go nowhere."""
        self.ids.copy_(torch.topk(self.logits, self.k, dim=1).indices)
        self.ids[-self.T // 10:] = -1

    def sort(self):
        """Rows sorted by expert, those of none behind (their values are of no matter)."""
        flat = self.ids.flatten().long()
        self.order = torch.argsort(torch.where(flat < 0, self.E, flat), stable=True)
        self.xs.copy_(self.x[self.order // self.k])
        self.last = int((flat >= 0).sum())
        self.labels[self.last:] = -1

    def go(self, stream=None):
        T, K, H, E, V, n, o, st = self.T, self.K, self.H, self.E, self.V, self.n, self.offsets, dict(stream=stream)
        ew = bsm.ewise_desc("silu_affine", 1.25, 0.0)
        kept = lambda q, f: (q, q.stride(0), f, f.stride(0))
        bsm.bsm_router_balance(T, E, self.k, "f32", self.logits, E, self.ids, 1.0, self.counts, o, self.balance, self.wb, **st)
        bsm.bsm_block_scale_save(n, K, "bf16", self.xs, K, "e4m3", *kept(self.xq, self.xf), **st)
        bsm.bsm_gemm_grouped(n, H, K, E, o, "bf16", self.xs, K, self.w1, K, "k", H * K, "bf16", self.z, H, **st)
        bsm.bsm_block_scale_save(n, H, "bf16", self.z, H, "e5m2", *kept(self.zq, self.zf), **st)
        bsm.bsm_block_scale_restore(n, H, "e5m2", *kept(self.zq, self.zf), "bf16", self.a, H, ew, **st)
        bsm.bsm_gemm_grouped(n, K, H, E, o, "bf16", self.a, H, self.w2, H, "k", K * H, "bf16", self.y, K, **st)
        bsm.bsm_gemm_cross_entropy(n, V, K, "bf16", self.y, K, self.wo, K, self.labels, self.loss, self.lse, self.wl, **st)
        bsm.bsm_gemm_cross_entropy_grad(n, V, K, "bf16", self.y, K, self.wo, K, self.labels, self.lse, self.dloss, 512, self.wg, "bf16",
                                        self.dy, K, "f32", self.dwo, K, **st)
        bsm.bsm_gemm_grouped(n, H, K, E, o, "bf16", self.dy, K, self.w2, H, "n", K * H, "bf16", self.da, H, **st)
        bsm.bsm_gemm_grouped_wgrad(n, K, H, E, o, "bf16", self.dy, K, self.a, H, "f32", self.dw2, H, K * H, **st)
        bsm.bsm_block_scale_ewise_grad(n, H, "e5m2", *kept(self.zq, self.zf), "bf16", self.da, H, self.dz, H, ew, **st)
        bsm.bsm_gemm_grouped_wgrad_block_scale(n, H, K, E, o, "bf16", self.dz, H, "e4m3", *kept(self.xq, self.xf), "f32", self.dw1, K,
                                               H * K, **st)
        bsm.bsm_gemm_grouped(n, K, H, E, o, "bf16", self.dz, H, self.w1, K, "n", H * K, "bf16", self.dx, K, **st)
        bsm.bsm_router_balance_grad(T, E, self.k, "f32", self.logits, E, self.ids, self.counts, 1.0, self.coef, "f32", self.dl, E, **st)

    def outputs(self):
        """What the step wrote (rows of no expert hold what the buffers held)."""
        rows = ("z", "a", "y", "da", "dz", "dx", "zq", "zf")
        return {k: (getattr(self, k)[:self.last] if k in rows or k in ("xq", "xf") else getattr(self, k)).clone() for k in OUT}

    def poison(self):
        """Values of another step in every output and workspace (finite: rows of no expert pass through the head's W gradient)."""
        for k in OUT + ("z",):
            getattr(self, k).fill_(3)
        for k in ("wb", "wl", "wg"):
            getattr(self, k).fill_(255)


def test_step():
    s = Step()
    s.choose()
    s.sort()
    s.poison()
    s.go()
    torch.cuda.synchronize()
    cpu = lambda t: t.double().cpu()
    loss, counts, ends, grad, lb, gb = balance_reference(s.logits.cpu(), s.ids.cpu(), s.E, s.k, 1.0, float(s.coef))
    assert torch.equal(s.counts.cpu().long(), counts) and torch.equal(s.offsets.cpu().long(), ends) and int(ends[-1]) == s.last
    assert abs(float(s.balance) - float(loss)) <= lb + 2.0 ** -24 * abs(float(loss))
    assert ((cpu(s.dl) - grad).abs() <= gb + 2.0 ** -24 * grad.abs() + 2.0 ** -126).all()
    x = values(s.xq.cpu()[:, :s.K].contiguous().view(F8["e4m3"]).double(), s.xf.cpu()[:, :(s.K + 31) // 32], s.K)
    z = values(s.zq.cpu()[:, :s.H].contiguous().view(F8["e5m2"]).double(), s.zf.cpu()[:, :(s.H + 31) // 32], s.H)
    # half a step of the formats, and half a subnormal one of the block's scale
    assert ((x - cpu(s.xs)).abs() <= 2.0 ** -4 * cpu(s.xs).abs() + 2.0 ** -17 * cpu(s.xs).abs().amax(1, keepdim=True))[:s.last].all()
    zr, lse, el, lref = (head_reference(s.y, s.wo, s.labels)[i] for i in (1, 2, 3, 4))
    assert ((s.lse.double() - lse).abs() <= el).all() and ((s.loss.double() - lref).abs() <= zr + el + 1e-6 * lref.abs()).all()
    off = s.offsets.tolist()
    for e in range(s.E):
        a, b = off[e], off[e + 1]
        p = lambda u, v: (u @ v, u.abs() @ v.abs())
        act, dy, dz, da = cpu(s.a[a:b]), cpu(s.dy[a:b]), cpu(s.dz[a:b]), cpu(s.da[a:b])
        check(s.y[a:b], *p(act, cpu(s.w2[e]).T), s.H, "bf16", "y")
        check(s.da[a:b], *p(dy, cpu(s.w2[e])), s.K, "bf16", "da")
        check(s.dw2[e], *p(dy.T, act), b - a, "f32", "dw2")
        check(s.dw1[e], *p(dz.T, x[a:b]), b - a, "f32", "dw1")
        check(s.dx[a:b], *p(dz, cpu(s.w1[e])), s.H, "bf16", "dx")
        sg = torch.sigmoid(z[a:b])
        slope = 1.25 * sg * (1 + z[a:b] * (1 - sg))
        assert ((dz - da * slope).abs() <= 2.0 ** -8 * (da * slope).abs() * 1.01 + 2.0 ** -17 * da.abs() * (1 + z[a:b].abs())).all()


def test_step_in_a_graph_and_on_another_stream():
    """A captured step with a new routing, labels and inputs before each replay equals the eager step, bit for bit; so does
    the step on a stream of its own, its workspaces full of other values."""
    s = Step(seed=3)
    side = torch.cuda.Stream()
    s.choose()
    s.sort()
    s.go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.go()
    g = torch.Generator(device="cuda").manual_seed(1)
    for r in range(4):
        say("graph replay", r)
        if r:
            s.logits.normal_(generator=g)
            s.labels.random_(0, s.V, generator=g)
            s.x.normal_(generator=g)
        s.choose()
        s.sort()
        s.poison()
        s.go()
        torch.cuda.synchronize()
        want = s.outputs()
        s.poison()
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.poison()
        torch.cuda.synchronize()
        s.go(stream=side)
        side.synchronize()
        other = s.outputs()
        for name in want:
            assert torch.equal(got[name], want[name]), (r, name)
            assert torch.equal(other[name], want[name]), (r, name)


@pytest.mark.parametrize("T,V", [(8, 40000), (90, 300), (700, 5000)])
def test_two_steps_at_once(T, V):
    """Two steps, each with buffers of its own, on two streams and as two graphs at once."""
    both = [Step(T=T, V=V, seed=i, E=5 + i) for i in (1, 2)]
    graphs, want = [], []
    for s in both:
        s.choose()
        s.sort()
        s.poison()
        s.go()
        torch.cuda.synchronize()
        want.append(s.outputs())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.go()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def same(what):
        torch.cuda.synchronize()
        for s, w in zip(both, want):
            got = s.outputs()
            for name in w:
                assert torch.equal(got[name], w[name]), (what, name)
            s.poison()
        torch.cuda.synchronize()

    same("eager")
    for r in range(3):
        say("two at once", T, r)
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        same("graphs")
        for s, st in zip(both, streams):
            s.go(stream=st)
        same("streams")
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s.go()
        same("current streams")


def test_kept_rows_feed_the_block_scaled_product():
    """Codes saved from rows of a multiple of 32 are the block-scaled products' operands: x W^T on the codes is the product of
    the restored rows."""
    g = torch.Generator().manual_seed(2)
    rows, K, N = 70, 256, 136
    mk = lambda *s: torch.randn(*s, generator=g).bfloat16().cuda()
    x, w = mk(rows, K), mk(N, K)
    q = [torch.empty(r, K, dtype=torch.uint8, device="cuda") for r in (rows, N)]
    f = [torch.empty(r, K // 32, dtype=torch.uint8, device="cuda") for r in (rows, N)]
    D = torch.empty(rows, N, device="cuda")
    for t, c, s in zip((x, w), q, f):
        bsm.bsm_block_scale_save(t.shape[0], K, "bf16", t, K, "e4m3", c, K, s, K // 32)
    bsm.bsm_gemm_block_scale(rows, N, K, "e4m3", q[0], K, f[0], K // 32, "e4m3", q[1], K, f[1], K // 32, D, N)
    v = [values(c.cpu().view(F8["e4m3"]).double(), s.cpu(), K) for c, s in zip(q, f)]
    ref, mag = v[0] @ v[1].T, v[0].abs() @ v[1].abs().T
    assert ((D.cpu().double() - ref).abs() <= 1e-5 * mag + 2.0 ** -24 * ref.abs()).all()
