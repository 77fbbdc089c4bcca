"""A training step's operators around the products, measured: the router's counts and balance loss, activations kept
in 8 bits and used in the backward pass, and the cross entropy of a projection onto a large vocabulary.

listed() names the cases, draw() makes more of the same ranges, prepare() makes what a program has in hand
before the call, run() is one pass: in plain torch operations in 32 bits, or, where `own` is set, through the
library's entry points. exact() is the same in 64 bits. Row-major tensors throughout; rows of an odd length are
padded to the leading dimension that the library asks for, as its callers keep them.

Operators ("op"):
  balance      counts, offsets and balance loss of a router's choices, and the loss's gradient in the logits
  checkpoint   rows of activations to 8-bit codes with an E8M0 scale per 32 values, and back
  activation   gradient of silu_affine, its input kept as such codes: dX = dY f'(x)
  wgrad        weight gradient D_g = Y_g^T X_g over the rows of group g, X kept as such codes
  head         cross entropy of X W^T against labels: losses and log-sum-exps ("loss"), and with them both
               gradients ("step")
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
F8_TOP = {"e4m3": 9, "e5m2": 16}     # the largest finite value of both formats is 0.875 * 2^top
SILU_SCALE, SILU_BIAS = 1.25, 0.5


def listed():
    return [
        # a few tokens of a short sequence routed to 6 of 64 experts: the smallest call, latency counts
        dict(name="balance few tokens", op="balance", rows=16, experts=64, k=6, fmt="f32", pad=0.0, split=1),
        # an odd number of tokens, an odd number of experts, the batch's last part padding
        dict(name="balance odd", op="balance", rows=8191, experts=60, k=4, fmt="f32", pad=0.1, split=2),
        # a training batch of tokens, 8 of 128 experts, 16-bit logits
        dict(name="balance batch", op="balance", rows=32768, experts=128, k=8, fmt="bf16", pad=0.03, split=3),
        # a layer's activations kept for the backward pass and restored there
        dict(name="checkpoint layer", op="checkpoint", rows=8190, K=8192, x="bf16", fmt="e4m3", split=4),
        # few rows of an odd length, the wide-range format
        dict(name="checkpoint small", op="checkpoint", rows=515, K=1000, x="f16", fmt="e5m2", split=5),
        # backward pass through the activation of a feed-forward layer
        dict(name="activation gradient", op="activation", rows=8190, K=8192, x="bf16", fmt="e4m3", split=6),
        # the same with a few short segments, float32 gradients
        dict(name="activation gradient small", op="activation", rows=77, K=1416, x="f32", fmt="e5m2", split=7),
        # weight gradient of a training step from kept activations, summed in and kept as float32
        dict(name="experts weight gradient", op="wgrad", rows=16381, groups=8, M=4096, N=2048, ab="bf16", fmt="e4m3", d="f32",
             split=8),
        # few rows over many experts, some without any, odd sizes, 16-bit gradients
        dict(name="experts weight gradient small", op="wgrad", rows=1021, groups=32, M=1000, N=520, ab="f16", fmt="e5m2", d="f16",
             split=9),
        # the losses of a few rows, as an evaluation of short answers takes them
        dict(name="head loss few rows", op="head", rows=24, N=50021, K=2048, ab="bf16", d="bf16", step=False, split=10),
        # a short micro-batch with an odd vocabulary and width, 16-bit floats, float32 gradients
        dict(name="head step small", op="head", rows=200, N=10007, K=1000, ab="f16", d="f32", step=True, split=11),
        # a training step's head, losses and both gradients
        dict(name="head step", op="head", rows=8190, N=32001, K=4096, ab="bf16", d="bf16", step=True, split=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["balance", "checkpoint", "activation", "wgrad", "head", "head"])
        split = rng.randrange(1 << 30)
        if op == "balance":
            c = dict(op=op, rows=_log(rng, 1, 65536), experts=_log(rng, 2, 512), k=rng.randint(1, 8),
                     fmt=rng.choice(["f32", "bf16", "f16"]), pad=rng.choice([0.0, 0.1, 0.5]), split=split)
            c["k"] = min(c["k"], c["experts"])
        elif op in ("checkpoint", "activation"):
            c = dict(op=op, rows=_log(rng, 1, 16384), K=_log(rng, 32, 16384), x=rng.choice(["bf16", "f16", "f32"]),
                     fmt=rng.choice(["e4m3", "e5m2"]), split=split)
        elif op == "wgrad":
            c = dict(op=op, rows=_log(rng, 1, 16384), groups=_log(rng, 1, 64), M=_log(rng, 256, 4096), N=_log(rng, 256, 4096),
                     ab=rng.choice(["bf16", "f16"]), fmt=rng.choice(["e4m3", "e5m2"]), d=rng.choice(["same", "f32"]), split=split)
            c["d"] = c["ab"] if c["d"] == "same" else "f32"
        else:
            c = dict(op=op, rows=_log(rng, 1, 8192), N=_log(rng, 1000, 131072), K=_log(rng, 256, 4096),
                     ab=rng.choice(["bf16", "f16"]), d=rng.choice(["same", "f32"]), step=rng.choice([True, False]), split=split)
            c["d"] = c["ab"] if c["d"] == "same" else "f32"
        if all(work(c)[k] <= top[k] for k in top):
            return c


def _counts(case):
    """Rows of each group: a router's uneven split, the same for every seed of the case."""
    r = random.Random(case["split"])
    n = case["groups"]
    share = [r.expovariate(1.0) + 0.25 for _ in range(n)]
    got = [0] * n
    for g in r.choices(range(n), share, k=case["rows"]):
        got[g] += 1
    return got


def work(case):
    """What the operator cannot do without: each input read once, each output written once (kept codes both), and the
    multiplications and additions of its products (the logits of a head once)."""
    size = {"bf16": 2, "f16": 2, "f32": 4}
    rows, code = case["rows"], 1 + 1 / 32
    if case["op"] == "balance":
        E = case["experts"]
        return {"bytes": rows * (2 * E * size[case["fmt"]] + 4 * case["k"]) + 8 * E, "flops": 10 * rows * E}
    if case["op"] == "checkpoint":
        return {"bytes": rows * case["K"] * 2 * (size[case["x"]] + code), "flops": 3 * rows * case["K"]}
    if case["op"] == "activation":
        return {"bytes": rows * case["K"] * (2 * size[case["x"]] + code), "flops": 10 * rows * case["K"]}
    if case["op"] == "wgrad":
        M, N = case["M"], case["N"]
        return {"bytes": rows * (2 * M + code * N) + case["groups"] * M * N * size[case["d"]], "flops": 2 * rows * M * N}
    N, K = case["N"], case["K"]
    grads = (rows * K * size[case["ab"]] + N * K * size[case["d"]]) if case["step"] else 0
    return {"bytes": 2 * K * (rows + N) + 12 * rows + grads, "flops": (6 if case["step"] else 2) * rows * N * K}


def _up(n, to):
    return -(-n // to) * to


def _rows_of(gen, shape, ld, dtype, scale=1.0):
    """Normal values of `shape` in rows of `ld` elements, the last axis a view of its first values."""
    t = torch.empty(*shape[:-1], ld, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
    return t[..., :shape[-1]]


def _blocks(x):
    """x in 32 bits as (rows, blocks, 32), the last block filled up with zeros."""
    return torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % 32)).unflatten(-1, (-1, 32))


def _save(x, fmt):
    """Codes as the 8-bit type's values, and scale codes, of rows x: the scale is the smallest power of two that brings
    the block's largest finite value inside the format."""
    b = _blocks(x)
    top = torch.where(torch.isfinite(b), b.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - F8_TOP[fmt] + (m > 0.875), -127).clamp(-127, 127)
    y = torch.ldexp(b, -e[..., None])
    if fmt == "e4m3":
        y = torch.where(torch.isfinite(y), y, torch.nan)
    return y.flatten(-2)[..., :x.shape[-1]].to(F8[fmt]), (e + 127).to(torch.uint8)


def _kept(x, fmt):
    """Rows x as a program keeps them: codes in rows of whole 16 bytes, scales in rows of whole words."""
    q, s = _save(x, fmt)
    codes = torch.zeros(x.shape[0], _up(x.shape[1], 16), dtype=torch.uint8, device=x.device)
    scales = torch.full((x.shape[0], _up(s.shape[1], 4)), 127, dtype=torch.uint8, device=x.device)
    codes[:, :x.shape[1]] = q.view(torch.uint8)
    scales[:, :s.shape[1]] = s
    return codes, scales


def _values(q, s):
    """The 32-bit values that 8-bit codes (as their type) and scale codes stand for."""
    b = _blocks(q)
    return torch.ldexp(b, s[..., :b.shape[1], None].int() - 127).flatten(-2)[..., :q.shape[-1]]


class State:
    pass


def _activations(gen, rows, K, x):
    """Activations: normal values, some channels much larger, as the layers of a model have them, in padded rows."""
    t = _rows_of(gen, (rows, K), _up(K, 4 if x == "f32" else 8), DT[x])
    t *= torch.exp(torch.empty(K, device="cuda").normal_(0.0, 1.0, generator=gen)).to(t.dtype)
    return t


def prepare(case, seed):
    s = State()
    s.case = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows = case["op"], case["rows"]
    if op == "balance":
        E, k = case["experts"], case["k"]
        s.logits = torch.empty(rows, E, device="cuda").normal_(0.0, 1.5, generator=gen)
        s.logits += torch.empty(E, device="cuda").normal_(0.0, 0.5, generator=gen)
        s.logits = s.logits.to(DT[case["fmt"]])
        # the router chooses with noise; rows behind the last sequence are padding and go to no expert
        noise = torch.empty(rows, E, device="cuda").normal_(0.0, 0.2, generator=gen)
        s.ids = torch.topk(s.logits.float() + noise, k, dim=1).indices.to(torch.int32)
        s.ids[rows - int(rows * case["pad"]):] = -1
        s.dloss = torch.rand(1, device="cuda", generator=gen) * 0.02 + 0.01
        return s
    if op in ("checkpoint", "activation"):
        s.x = _activations(gen, rows, case["K"], case["x"])
        if op == "activation":
            s.codes, s.scales = _kept(s.x, case["fmt"])
            s.dy = _rows_of(gen, (rows, case["K"]), s.x.stride(0), DT[case["x"]])
            del s.x
        return s
    t = DT[case["ab"]]
    if op == "wgrad":
        counts = _counts(case)
        ends = [sum(counts[:i + 1]) for i in range(len(counts))]
        s.groups = [(ends[g] - n, ends[g]) for g, n in enumerate(counts)]
        s.offsets = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
        s.y = _rows_of(gen, (rows, case["M"]), _up(case["M"], 8), t)
        s.codes, s.scales = _kept(_activations(gen, rows, case["N"], case["ab"]), case["fmt"])
        return s
    N, K = case["N"], case["K"]
    s.x = _rows_of(gen, (rows, K), _up(K, 8), t)
    s.w = _rows_of(gen, (N, K), _up(K, 8), t, 2.0 * K ** -0.5)
    s.labels = torch.randint(0, N, (rows,), dtype=torch.int32, device="cuda", generator=gen)
    # one row in sixteen is a prompt's or padding: no label
    s.labels[torch.rand(rows, device="cuda", generator=gen) < 1 / 16] = -1
    s.dloss = (torch.rand(rows, device="cuda", generator=gen) + 0.5) / rows
    return s


def _plain(s):
    c = s.case
    op = c["op"]
    if op == "balance":
        E, k, x = c["experts"], c["k"], s.logits.float()
        experts = torch.arange(E, device=x.device)
        mine = sum((s.ids[:, j, None] == experts).int() for j in range(k))
        keep = mine.sum(1, keepdim=True) > 0
        counts, n = mine.sum(0), keep.sum()
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = torch.where(keep, p / p.sum(1, keepdim=True), 0.0)
        f, over = counts.float() / (k * n).clamp_min(1), n.clamp_min(1)
        loss = E * (f * p.sum(0) / over).sum()
        d = s.dloss * E / over * p * (f - (f * p).sum(1, keepdim=True))
        ends = counts.cumsum(0)
        return loss[None], torch.cat((counts, n[None])).int(), torch.cat((ends[:1] * 0, ends)).int(), d.to(s.logits.dtype)
    if op == "checkpoint":
        d = DT[c["x"]]
        return _values(*_save(s.x, c["fmt"])).clamp(-torch.finfo(d).max, torch.finfo(d).max).to(d)
    if op == "activation":
        z = _values(s.codes.view(F8[c["fmt"]])[:, :c["K"]], s.scales)
        a = 1 / (1 + torch.exp(-z))
        return (s.dy.float() * (SILU_SCALE * a * (1 + z * (1 - a)))).to(s.dy.dtype)
    if op == "wgrad":
        x = _values(s.codes.view(F8[c["fmt"]])[:, :c["N"]], s.scales)
        return torch.stack([s.y[a:b].float().T @ x[a:b] for a, b in s.groups]).to(DT[c["d"]])
    x, w = s.x.float(), s.w.float()
    z = x @ w.T
    top = z.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(z - top).sum(1, keepdim=True))
    has = s.labels[:, None] >= 0
    at = s.labels[:, None].clamp_min(0).long()
    loss = torch.where(has, lse - z.gather(1, at), 0.0)
    if not c["step"]:
        return loss[:, 0], lse[:, 0]
    g = torch.exp(z - lse)
    g.scatter_add_(1, at, torch.full_like(loss, -1.0))
    g *= torch.where(has, s.dloss[:, None], 0.0)
    return loss[:, 0], lse[:, 0], (g @ w).to(s.x.dtype), (g.T @ x).to(DT[c["d"]])


def _out(lead, n, d):
    """An output of rows of n values of type d, in rows of the leading dimension that the library asks for."""
    return torch.empty(*lead, _up(n, 4 if d == "f32" else 8), dtype=DT[d], device="cuda")


def _bytes(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _own(s):
    import block_scaled_matrix_amd as bsm
    c = s.case
    op, rows = c["op"], c["rows"]
    if op == "balance":
        E, k, fmt = c["experts"], c["k"], c["fmt"]
        counts, offsets = (torch.empty(E + 1, dtype=torch.int32, device="cuda") for _ in range(2))
        loss = torch.empty(1, device="cuda")
        bsm.bsm_router_balance(rows, E, k, fmt, s.logits, E, s.ids, 1.0, counts, offsets, loss,
                               _bytes(bsm.bsm_router_balance_workspace(rows, E)))
        d = torch.empty_like(s.logits)
        bsm.bsm_router_balance_grad(rows, E, k, fmt, s.logits, E, s.ids, counts, 1.0, s.dloss, fmt, d, E)
        return loss, counts, offsets, d
    if op == "checkpoint":
        K = c["K"]
        q, sf = _bytes((rows, _up(K, 16))), _bytes((rows, _up(_up(K, 32) // 32, 4)))
        bsm.bsm_block_scale_save(rows, K, c["x"], s.x, s.x.stride(0), c["fmt"], q, q.stride(0), sf, sf.stride(0))
        d = _out((rows,), K, c["x"])
        bsm.bsm_block_scale_restore(rows, K, c["fmt"], q, q.stride(0), sf, sf.stride(0), c["x"], d, d.stride(0))
        return d[:, :K]
    if op == "activation":
        K = c["K"]
        d = _out((rows,), K, c["x"])
        bsm.bsm_block_scale_ewise_grad(rows, K, c["fmt"], s.codes, s.codes.stride(0), s.scales, s.scales.stride(0), c["x"], s.dy,
                                       s.dy.stride(0), d, d.stride(0), bsm.ewise_desc("silu_affine", SILU_SCALE, SILU_BIAS))
        return d[:, :K]
    if op == "wgrad":
        out = _out((c["groups"], c["M"]), c["N"], c["d"])
        bsm.bsm_gemm_grouped_wgrad_block_scale(rows, c["M"], c["N"], c["groups"], s.offsets, c["ab"], s.y, s.y.stride(0), c["fmt"],
                                               s.codes, s.codes.stride(0), s.scales, s.scales.stride(0), c["d"], out, out.stride(1),
                                               out.stride(0))
        return out[..., :c["N"]]
    N, K, ab = c["N"], c["K"], c["ab"]
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    bsm.bsm_gemm_cross_entropy(rows, N, K, ab, s.x, s.x.stride(0), s.w, s.w.stride(0), s.labels, loss, lse,
                               _bytes(bsm.bsm_gemm_cross_entropy_workspace(rows, N)))
    if not c["step"]:
        return loss, lse
    dx, dw = _out((rows,), K, ab), _out((N,), K, c["d"])
    bsm.bsm_gemm_cross_entropy_grad(rows, N, K, ab, s.x, s.x.stride(0), s.w, s.w.stride(0), s.labels, lse, s.dloss, 0,
                                    _bytes(bsm.bsm_gemm_cross_entropy_grad_workspace(rows, N, K, 0)), ab, dx, dx.stride(0), c["d"],
                                    dw, dw.stride(0))
    return loss, lse, dx[:, :K], dw[:, :K]


def run(s):
    return _own(s) if own else _plain(s)


def _exact_values(codes, scales, fmt, K):
    """The 64-bit values from the formats' definition: sign, exponent and fraction bits of each code."""
    codes = codes[:, :K].to(torch.int64)
    eb, mb = (4, 3) if fmt == "e4m3" else (5, 2)
    e, m = (codes >> mb) % 2 ** eb, (codes % 2 ** mb).double() / 2 ** mb
    v = torch.where(e == 0, m * 2.0 ** (2 - 2 ** (eb - 1)), (1 + m) * torch.exp2((e + 1 - 2 ** (eb - 1)).double()))
    v = torch.where(codes >= 128, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :K]


def exact(case, seed):
    s = prepare(case, seed)
    op, rows = case["op"], case["rows"]
    if op == "balance":
        E, x, ids = case["experts"], s.logits.double(), s.ids.long()
        kept = torch.nonzero((ids >= 0).any(1)).flatten()
        counts = torch.bincount(ids[ids >= 0], minlength=E)
        n = len(kept)
        d = torch.zeros_like(x)
        loss = torch.zeros(1, dtype=torch.float64, device="cuda")
        if n:
            p = torch.exp(x[kept] - torch.logsumexp(x[kept], 1)[:, None])
            f = counts.double() / (case["k"] * n)
            loss += E * torch.dot(f, p.mean(0))
            d[kept] = s.dloss.double() * E / n * (p * f - p * (p @ f)[:, None])
        ends = [0] + torch.cumsum(counts, 0).tolist()
        return loss, torch.tensor(counts.tolist() + [n], device="cuda"), torch.tensor(ends, device="cuda"), d
    if op == "checkpoint":
        x, (mb, low, most) = s.x.double(), {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}[case["fmt"]]
        out = torch.empty_like(x)
        for k in range(0, case["K"], 32):
            b = x[:, k:k + 32]
            top = b.abs().amax(1, keepdim=True)
            e = torch.where(top > 0, torch.ceil(torch.log2(top / most)), -127.0).clamp(-127, 127)
            y = b * torch.exp2(-e)
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** low))).clamp_min(low) - mb)
            out[:, k:k + 32] = torch.round(y / step) * step * torch.exp2(e)
        return out
    if op == "activation":
        z = _exact_values(s.codes, s.scales, case["fmt"], case["K"])
        return s.dy.double() * SILU_SCALE * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    if op == "wgrad":
        x = _exact_values(s.codes, s.scales, case["fmt"], case["N"])
        out = torch.zeros(case["groups"], case["M"], case["N"], dtype=torch.float64, device="cuda")
        for g, (a, b) in enumerate(s.groups):
            if b > a:
                torch.matmul(s.y[a:b].double().T.contiguous(), x[a:b], out=out[g])
        return out
    x, w = s.x.double(), s.w.double()
    z = torch.matmul(x, w.T.contiguous())
    lse = torch.logsumexp(z, 1)
    rows_with = torch.nonzero(s.labels >= 0).flatten()
    at = s.labels[rows_with].long()
    loss = torch.zeros(rows, dtype=torch.float64, device="cuda")
    loss[rows_with] = lse[rows_with] - z[rows_with, at]
    if not case["step"]:
        return loss, lse
    g = z.sub_(lse[:, None]).exp_()
    g[rows_with, at] -= 1.0
    weight = torch.zeros(rows, dtype=torch.float64, device="cuda")
    weight[rows_with] = s.dloss[rows_with].double()
    g *= weight[:, None]
    return loss, lse, torch.matmul(g, w), torch.matmul(g.T.contiguous(), x)
