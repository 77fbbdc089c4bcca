"""Ragged products with a weight per group of rows, measured: products grouped by expert (forward, input
gradient, weight gradient, block scaled) and low-rank adapters of many requests beside a shared projection.

listed() names the cases, draw() makes more of the same ranges, prepare() makes what a program has in hand
before the call, run() is one pass: in plain torch operations in 32 bits, or, where `own` is set, through the
library's entry points. exact() is the same product in 64 bits. Row-major tensors throughout; rows of an
odd length are padded to the leading dimension that the library asks for, as its callers keep them.

Operators ("op"):
  grouped      D[r, :] = X[r, :] W_g^T for the rows r of group g; W_g is (N, K) ('k') or, for the input
               gradient dX = dY W, stored (K, N) ('n')
  wgrad        D_g = Y_g^T X_g over the rows of group g, float32 or 16-bit; a group without rows gives zeros
  mx           grouped with block-scaled operands (one E8M0 scale per 32 K elements)
  adapters     D[t, :] = X[t, :] W^T + s_a (X[t, :] A_a^T) B_a^T, a = the adapter of row t (-1: none)
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MX_BITS = {"e4m3": 8, "e5m2": 8, "e2m1": 4}
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decoder sent to 8 of 64 experts: the smallest call, latency counts
        dict(name="experts one token", op="grouped", rows=8, groups=64, N=1024, K=2048, ab="bf16", d="bf16", major="k", split=1),
        # a decode batch of 96 tokens, 4 experts each: every expert's weights are read once
        dict(name="experts decode", op="grouped", rows=384, groups=32, N=4096, K=2048, ab="f16", d="f16", major="k", split=2),
        # an odd number of prompt rows over 16 experts
        dict(name="experts prompt", op="grouped", rows=16381, groups=16, N=4096, K=8192, ab="bf16", d="bf16", major="k", split=3),
        # input gradient of a training step: the same weights read the other way
        dict(name="experts input gradient", op="grouped", rows=8190, groups=8, N=2048, K=8192, ab="bf16", d="bf16", major="n", split=4),
        # many small experts and odd sizes, float32 out
        dict(name="experts input gradient small", op="grouped", rows=4099, groups=64, N=1000, K=1416, ab="f16", d="f32", major="n",
             split=5),
        # weight gradient of a training step, summed in and kept as float32
        dict(name="experts weight gradient", op="wgrad", rows=16381, groups=8, M=4096, N=2048, ab="bf16", d="f32", split=6),
        # few rows over many experts, some without any, odd sizes, 16-bit gradients
        dict(name="experts weight gradient small", op="wgrad", rows=1021, groups=32, M=1000, N=520, ab="f16", d="f16", split=7),
        # decode with 8-bit activations on 4-bit weights, exact products
        dict(name="experts mx decode", op="mx", rows=64, groups=32, N=4096, K=4096, a="e4m3", b="e2m1", fast=0, d="bf16", split=8),
        # prompt rows in MXFP8, sums at the full 8-bit rate
        dict(name="experts mxfp8 prompt", op="mx", rows=8190, groups=16, N=8192, K=4096, a="e4m3", b="e4m3", fast=1, d="bf16", split=9),
        # prompt rows in MXFP4
        dict(name="experts mxfp4 prompt", op="mx", rows=16381, groups=8, N=4096, K=8192, a="e2m1", b="e2m1", fast=0, d="bf16", split=10),
        # a decode batch of 48 requests over 24 adapters of rank 16, some requests without one
        dict(name="adapters decode", op="adapters", rows=48, adapters=24, R=16, N=4096, K=4096, ab="bf16", d="bf16", split=11),
        # prompts of requests with 8 adapters of rank 64
        dict(name="adapters prompt", op="adapters", rows=8190, adapters=8, R=64, N=8192, K=4096, ab="bf16", d="bf16", split=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    top = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["grouped", "grouped", "wgrad", "mx", "adapters"])
        split = rng.randrange(1 << 30)
        if op == "grouped":
            c = dict(op=op, rows=_log(rng, 1, 16384), groups=_log(rng, 1, 128), N=_log(rng, 256, 8192), K=_log(rng, 256, 8192),
                     ab=rng.choice(["bf16", "f16"]), d=rng.choice(["same", "f32"]), major=rng.choice("kn"), split=split)
            c["d"] = c["ab"] if c["d"] == "same" else "f32"
        elif op == "wgrad":
            c = dict(op=op, rows=_log(rng, 64, 16384), groups=_log(rng, 1, 64), M=_log(rng, 256, 4096), N=_log(rng, 256, 4096),
                     ab=rng.choice(["bf16", "f16"]), d=rng.choice(["same", "f32"]), split=split)
            c["d"] = c["ab"] if c["d"] == "same" else "f32"
        elif op == "mx":
            a, b, fast = rng.choice([("e4m3", "e4m3", 1), ("e4m3", "e2m1", 0), ("e2m1", "e2m1", 0), ("e4m3", "e4m3", 0)])
            c = dict(op=op, rows=_log(rng, 1, 16384), groups=_log(rng, 1, 64), N=_log(rng, 256, 8192), K=32 * _log(rng, 8, 256),
                     a=a, b=b, fast=fast, d="bf16", split=split)
        else:
            c = dict(op=op, rows=_log(rng, 1, 8192), adapters=_log(rng, 1, 64), R=_log(rng, 4, 128), N=_log(rng, 256, 8192),
                     K=_log(rng, 256, 8192), ab=rng.choice(["bf16", "f16"]), d="same", split=split)
            c["d"] = c["ab"]
        if all(work(c)[k] <= top[k] for k in top):
            return c


def _counts(case):
    """Rows of each group: a router's uneven split, the same for every seed of the case."""
    r = random.Random(case["split"])
    n = case.get("groups")
    share = [r.expovariate(1.0) + 0.25 for _ in range(n)]
    got = [0] * n
    for g in r.choices(range(n), share, k=case["rows"]):
        got[g] += 1
    return got


def _adapters(case):
    """The adapter of each row: requests of many rows each where there are many rows; about one in eight without."""
    r = random.Random(case["split"])
    got, left = [], case["rows"]
    while left:
        n = min(left, 1 if case["rows"] <= 128 else r.randint(1, max(1, case["rows"] // 8)))
        got += [r.randrange(case["adapters"]) if r.random() < 0.875 else -1] * n
        left -= n
    return got


def work(case):
    """What the operator cannot do without: each input that a row needs read once, each output written once, and the
    multiplications and additions of its products."""
    rows, N = case["rows"], case["N"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "adapters":
        K, R = case["K"], case["R"]
        ids = _adapters(case)
        with_one = sum(a >= 0 for a in ids)
        n = rows * K + N * K + len({a for a in ids if a >= 0}) * R * (K + N)
        return {"bytes": 2 * n + rows * N * size[case["d"]] + 4 * rows, "flops": 2 * rows * N * K + 2 * with_one * R * (K + N)}
    counts = _counts(case)
    used = sum(c > 0 for c in counts)
    if case["op"] == "wgrad":
        M = case["M"]
        return {"bytes": 2 * rows * (M + N) + case["groups"] * M * N * size[case["d"]], "flops": 2 * rows * M * N}
    K = case["K"]
    if case["op"] == "mx":
        a, b = MX_BITS[case["a"]] / 8 + 1 / 32, MX_BITS[case["b"]] / 8 + 1 / 32
    else:
        a = b = size[case["ab"]]
    return {"bytes": a * rows * K + b * used * N * K + rows * N * size[case["d"]], "flops": 2 * rows * N * K}


def _up(n, to):
    return -(-n // to) * to


def _rows_of(gen, shape, ld, dtype, scale=1.0):
    """Normal values of `shape` in rows of `ld` elements, the last axis a view of its first values."""
    t = torch.empty(*shape[:-1], ld, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)
    return t[..., :shape[-1]]


def _mx_rows(gen, shape, fmt, scale=1.0):
    """Normal values in blocks of 32 as their elements' codes and E8M0 scale codes. The scale is the power of two that
    brings the block's largest value to the format's largest exponent."""
    lead, K = shape[:-1], shape[-1]
    ld_sf = _up(K // 32, 4)
    codes = torch.empty(*lead, _up(K * MX_BITS[fmt] // 8, 16), dtype=torch.uint8, device="cuda")
    scales = torch.full((*lead, ld_sf), 127, dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 26) // (lead[-1] * K))  # groups at once, to hold few 32-bit temporaries
    flat_c, flat_s = codes.view(-1, lead[-1], codes.shape[-1]), scales.view(-1, lead[-1], ld_sf)
    for g in range(0, flat_c.shape[0], per):
        n = min(per, flat_c.shape[0] - g)
        x = torch.empty(n, lead[-1], K // 32, 32, device="cuda").normal_(0.0, scale, generator=gen)
        top = {"e4m3": 8, "e5m2": 15, "e2m1": 2}[fmt]
        e = torch.floor(torch.log2(x.abs().amax(-1).clamp_min(1e-30))) - top
        y = (x * torch.exp2(-e)[..., None]).view(n, lead[-1], K)
        if fmt == "e2m1":
            edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
            v = torch.bucketize(y.abs(), edges).to(torch.uint8) + 8 * (y < 0).to(torch.uint8)
            v = v[..., 0::2] + 16 * v[..., 1::2]
        else:
            f8 = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
            v = y.clamp(-448.0, 448.0).to(f8).view(torch.uint8)
        flat_c[g:g + n, :, :v.shape[-1]] = v
        flat_s[g:g + n, :, :K // 32] = (e + 127).to(torch.uint8)
    return codes, scales


class State:
    pass


def prepare(case, seed):
    s = State()
    s.case = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, N = case["op"], case["rows"], case["N"]
    if op == "adapters":
        K, R, L = case["K"], case["R"], case["adapters"]
        t = DT[case["ab"]]
        s.x = _rows_of(gen, (rows, K), _up(K, 8), t)
        s.w = _rows_of(gen, (N, K), _up(K, 8), t, K ** -0.5)
        s.la = _rows_of(gen, (L, R, K), _up(K, 8), t, K ** -0.5)
        s.lb = _rows_of(gen, (L, N, R), _up(R, 8), t, R ** -0.5)
        s.scale = torch.rand(L, device="cuda", generator=gen) * 1.5 + 0.5
        s.ids = _adapters(case)
        s.adapter = torch.tensor(s.ids, dtype=torch.int32, device="cuda")
        return s
    counts = _counts(case)
    ends = [sum(counts[:i + 1]) for i in range(len(counts))]
    s.groups = [(g, ends[g] - n, ends[g]) for g, n in enumerate(counts)]
    s.offsets = torch.tensor([0] + ends, dtype=torch.int32, device="cuda")
    if op == "mx":
        s.x, s.xs = _mx_rows(gen, (rows, case["K"]), case["a"])
        s.w, s.ws = _mx_rows(gen, (case["groups"], N, case["K"]), case["b"], case["K"] ** -0.5)
        return s
    t = DT[case["ab"]]
    if op == "wgrad":
        s.y = _rows_of(gen, (rows, case["M"]), _up(case["M"], 8), t)
        s.x = _rows_of(gen, (rows, N), _up(N, 8), t)
        return s
    K = case["K"]
    s.x = _rows_of(gen, (rows, K), _up(K, 8), t)
    lead = (N, K) if case["major"] == "k" else (K, N)
    s.w = _rows_of(gen, (case["groups"], *lead), _up(lead[1], 8), t, K ** -0.5)
    return s


def _values(codes, scales, fmt, K):
    """The 32-bit values that element codes and their scales stand for."""
    if fmt == "e2m1":
        table = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), device=codes.device)
        codes = codes[..., :K // 2]
        v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    else:
        v = codes[..., :K].view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float()
    s = torch.exp2(scales[..., :K // 32].float() - 127)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _plain(s):
    c = s.case
    op, d = c["op"], DT[c["d"]]
    if op == "adapters":
        # every adapter's A beside the others: a row keeps its own adapter's R values of the L * R
        L, R = c["adapters"], c["R"]
        x = s.x.float()
        mine = torch.arange(L, device=x.device) == s.adapter[:, None]
        u = (x @ s.la.float().flatten(0, 1).T).unflatten(1, (L, R))
        u = torch.where(mine[..., None], u * s.scale[:, None], 0.0).flatten(1)
        return (x @ s.w.float().T + u @ s.lb.float().transpose(0, 1).flatten(1).T).to(d)
    used = [g for g in s.groups if g[2] > g[1]]
    if op == "wgrad":
        return torch.stack([s.y[a:b].float().T @ s.x[a:b].float() for _, a, b in s.groups]).to(d)
    if op == "mx":
        x = _values(s.x, s.xs, c["a"], c["K"])
        return torch.cat([x[a:b] @ _values(s.w[g], s.ws[g], c["b"], c["K"]).T for g, a, b in used]).to(d)
    x = s.x.float()
    if c["major"] == "k":
        return torch.cat([x[a:b] @ s.w[g].float().T for g, a, b in used]).to(d)
    return torch.cat([x[a:b] @ s.w[g].float() for g, a, b in used]).to(d)


def _out(lead, n, d):
    """An output of rows of n values of type d, in rows of the leading dimension that the library asks for."""
    return torch.empty(*lead, _up(n, 4 if d == "f32" else 8), dtype=DT[d], device="cuda")


def _own(s):
    import block_scaled_matrix_amd as bsm
    c = s.case
    op, d, rows, N = c["op"], c["d"], c["rows"], c["N"]
    if op == "wgrad":
        out = _out((c["groups"], c["M"]), N, d)
        bsm.bsm_gemm_grouped_wgrad(rows, c["M"], N, c["groups"], s.offsets, c["ab"], s.y, s.y.stride(0), s.x, s.x.stride(0),
                                   d, out, out.stride(1), out.stride(0))
        return out[..., :N]
    out = _out((rows,), N, d)
    if op == "adapters":
        work = torch.empty(bsm.bsm_gemm_lora_workspace(rows, c["R"]), dtype=torch.uint8, device="cuda")
        bsm.bsm_gemm_lora(rows, N, c["K"], c["R"], c["adapters"], s.adapter, c["ab"], s.x, s.x.stride(0), s.w, s.w.stride(0),
                          s.la, s.la.stride(1), s.la.stride(0), s.lb, s.lb.stride(1), s.lb.stride(0), s.scale, work,
                          d, out, out.stride(0))
    elif op == "mx":
        per_a, per_b = 8 // MX_BITS[c["a"]], 8 // MX_BITS[c["b"]]
        bsm.bsm_gemm_grouped_block_scale(rows, N, c["K"], c["groups"], s.offsets, c["a"], s.x, s.x.stride(0) * per_a, s.xs,
                                         s.xs.stride(0), c["b"], s.w, s.w.stride(1) * per_b, s.w.stride(0) * per_b, s.ws,
                                         s.ws.stride(1), s.ws.stride(0), c["fast"], d, out, out.stride(0))
    else:
        bsm.bsm_gemm_grouped(rows, N, c["K"], c["groups"], s.offsets, c["ab"], s.x, s.x.stride(0), s.w, s.w.stride(1),
                             c["major"], s.w.stride(0), d, out, out.stride(0))
    return out[:, :N]


def run(s):
    return _own(s) if own else _plain(s)


def _exact_values(codes, scales, fmt, K):
    """The 64-bit values from the formats' definition: sign, exponent and fraction bits of each code."""
    if fmt == "e2m1":
        codes = codes[..., :K // 2].to(torch.int64)
        codes = torch.stack((codes % 16, codes // 16), -1).flatten(-2)
        eb, mb = 2, 1
    else:
        codes = codes[..., :K].to(torch.int64)
        eb, mb = (4, 3) if fmt == "e4m3" else (5, 2)
    bias = 2 ** (eb - 1) - 1
    e, m = (codes >> mb) % 2 ** eb, codes % 2 ** mb
    v = torch.where(e == 0, m.double() * 2.0 ** (1 - bias - mb), (1 + m.double() / 2 ** mb) * torch.exp2((e - bias).double()))
    v = torch.where(codes >> (eb + mb) == 1, -v, v)
    return v * torch.exp2(scales[..., :K // 32].double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op, rows, N = case["op"], case["rows"], case["N"]
    if op == "wgrad":
        out = torch.zeros(case["groups"], case["M"], N, dtype=torch.float64, device="cuda")
        for g, a, b in s.groups:
            if b > a:
                torch.matmul(s.y[a:b].double().T.contiguous(), s.x[a:b].double(), out=out[g])
        return out
    out = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
    if op == "adapters":
        torch.matmul(s.x.double(), s.w.double().T, out=out)
        ids = torch.tensor(s.ids, device="cuda")
        for a in sorted(set(s.ids) - {-1}):
            at = torch.nonzero(ids == a).flatten()
            u = s.x[at].double() @ s.la[a].double().T
            out[at] += s.scale[a].double() * (u @ s.lb[a].double().T)
        return out
    for g, a, b in s.groups:
        if b > a:
            if op == "mx":
                x = _exact_values(s.x[a:b], s.xs[a:b], case["a"], case["K"])
                w = _exact_values(s.w[g], s.ws[g], case["b"], case["K"]).T
            else:
                x, w = s.x[a:b].double(), s.w[g].double()
                w = w.T if case["major"] == "k" else w
            out[a:b] = x @ w
    return out
