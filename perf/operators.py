"""Measured cases of the operators around and inside the expert layer.

Three kinds of work, each with a plain form in elementary torch operations and the framework's
own call:

* ``norm`` / ``norm_backward``: layer norm (or its root-mean-square form) of token rows, the step
  in front of the router and the experts, and its gradients with the weight's reduction;
* ``dropout`` / ``dropout_backward`` / ``combine_dropout``: dropout of the layer's output from a
  counter-based generator (Philox4x32-10), added to the residual stream, alone or in the combine;
* ``matvec``: the experts' products at decode sizes on 4-bit weights with group scales.

``own`` false computes the plain form, true calls ``grouped_gemm_histogram_amd``.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5

# the values of the sixteen 4-bit floating codes (1 sign, 2 exponent, 1 mantissa bit)
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token in front of a decode-size gpt-oss-20b layer: latency of a single row
        dict(name="norm_one_token", op="norm", rms=True, T=1, H=2880, dtype="bf16", wdtype="bf16", bias=False,
             stats=False),
        # a prefill or training batch at the width of the DeepSeek-V3 layer
        dict(name="norm_batch", op="norm", rms=False, T=8192, H=7168, dtype="bf16", wdtype="f32", bias=True,
             stats=True),
        # odd width and row count in f32: rows that start off every alignment
        dict(name="norm_odd_f32", op="norm", rms=False, T=1531, H=2881, dtype="f32", wdtype="f32", bias=True,
             stats=True),
        # training at the gpt-oss-20b layer's shape, with the weight's and the bias' gradients
        dict(name="norm_backward", op="norm_backward", rms=False, T=4096, H=2880, dtype="bf16", wdtype="f32",
             bias=True),
        # training at the DeepSeek-V3 layer's shape
        dict(name="norm_backward_batch", op="norm_backward", rms=True, T=8192, H=7168, dtype="bf16", wdtype="f32",
             bias=False),
        # the Mixtral-8x7B layer's output dropped and added to the residual stream
        dict(name="dropout_batch", op="dropout", T=8192, H=4096, dtype="bf16", rdtype="bf16", p=0.1),
        # gradient of the dropped branch, odd sizes in f32
        dict(name="dropout_backward_odd", op="dropout_backward", T=1021, H=2881, dtype="f32", p=0.25),
        # the gpt-oss-20b layer's combine with dropout and the residual in one pass
        dict(name="combine_dropout", op="combine_dropout", T=4096, H=2880, E=32, k=4, dtype="bf16", p=0.1),
        # one token of a gpt-oss-20b layer on 4-bit floating weights: latency and four experts' weights
        dict(name="matvec_one_token", op="matvec", fmt="mxfp4", group=32, T=1, k=4, E=32, N=5760, K=2880,
             silu=True, valid=1.0),
        # a small decode batch through the DeepSeek-V3 layer's down projection, 128-channel groups
        dict(name="matvec_down", op="matvec", fmt="int4", group=128, T=16, k=8, E=256, N=7168, K=2048,
             silu=False, valid=1.0),
        # a larger decode batch, a quarter of it padding, over many small experts with fine groups
        dict(name="matvec_padded", op="matvec", fmt="int4", group=32, T=64, k=8, E=128, N=1536, K=2048,
             silu=True, valid=0.75),
        # a decode batch that reads every expert of the Mixtral-8x7B layer's gate/up projection
        dict(name="matvec_all_experts", op="matvec", fmt="mxfp4", group=32, T=32, k=2, E=8, N=28672, K=4096,
             silu=True, valid=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "dropout", "dropout_backward", "combine_dropout", "matvec", "matvec"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_backward"):
        H = rng.choice([rng.randrange(64, 8193), 16 * rng.randrange(4, 513)])
        T = _log(rng, 1, min(16384, 50_000_000 // H))
        case = dict(op=op, rms=rng.random() < 0.5, T=T, H=H, dtype=dtype, wdtype=rng.choice(["bf16", "f32"]),
                    bias=rng.random() < 0.5)
        if op == "norm":
            case["stats"] = rng.random() < 0.5
        if dtype == "f32":
            case["T"] = max(1, T // 2)
        return case
    if op in ("dropout", "dropout_backward"):
        H = rng.choice([rng.randrange(1, 8193), 16 * rng.randrange(4, 513)])
        T = _log(rng, 1, min(16384, 30_000_000 // H))
        case = dict(op=op, T=T, H=H, dtype=dtype, p=rng.choice([0.0, 0.1, 0.5, rng.random()]))
        if op == "dropout":
            case["rdtype"] = rng.choice(["none", "bf16", "f32"])
        if dtype == "f32":
            case["T"] = max(1, T // 2)
        return case
    if op == "combine_dropout":
        k = rng.choice([1, 2, 4, 8])
        H = 8 * rng.randrange(8, 513)
        return dict(op=op, T=_log(rng, 1, max(1, 40_000_000 // (H * (k + 2)))), H=H, E=rng.choice([8, 32, 128]), k=k,
                    dtype=dtype, p=rng.choice([0.1, rng.random()]))
    fmt = rng.choice(["mxfp4", "int4"])
    group = 32 if fmt == "mxfp4" else rng.choice([32, 64, 128])
    k = rng.choice([1, 2, 4, 8])
    E = rng.choice([8, 32, 64, 128])
    K = group * rng.randrange(max(1, 256 // group), 4096 // group + 1)
    # rows of the output are whole 16-byte units: a multiple of 8 columns after SiLU * up
    N = 16 * rng.randrange(4, 513)
    while E * N * K > 900_000_000:
        E //= 2
    return dict(op=op, fmt=fmt, group=group, T=_log(rng, 1, 128), k=min(k, E), E=E, N=N, K=K,
                silu=rng.random() < 0.5, valid=rng.choice([1.0, 1.0, rng.random()]))


# ------------------------------------------------------------------------------------ the inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _routing(g, T, E, k, valid):
    """Top-k routing of random logits with the flat rows past the valid ones as sentinels."""
    R = T * k
    V = int(round(valid * R))
    logits = _randn(g, T, E)
    top = torch.topk(logits, k, dim=1)
    w = torch.softmax(top.values, dim=1).reshape(-1)
    ids = top.indices.reshape(-1)
    flat = torch.arange(R, device=DEV)
    ids = torch.where(flat < V, ids, torch.full_like(ids, E))
    w = torch.where(flat < V, w, torch.zeros_like(w))
    sorted_rows = torch.argsort(ids, stable=True)
    row_pos = torch.empty_like(sorted_rows)
    row_pos[sorted_rows] = flat
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    i32 = lambda t: t.to(torch.int32).contiguous()
    return dict(offsets=i32(offsets), sorted_rows=i32(sorted_rows), row_pos=i32(row_pos),
                weights=w.reshape(T, k).contiguous(), seg=[int(v) for v in offsets.tolist()])


def _quantised(g, E, N, K, fmt, group):
    """4-bit codes [E, N, K/2] (even channel in the low nibble) and group scales of normal weights."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // group, dtype=torch.uint8 if fmt == "mxfp4" else torch.float32, device=DEV)
    for e in range(E):
        w = (_randn(g, N, K) * 0.02).view(N, K // group, group)
        amax = w.abs().amax(dim=2)
        if fmt == "int4":
            s = torch.where(amax > 0, amax / 7.0, torch.ones_like(amax))
            c = (torch.round(w / s[..., None]).clamp_(-8, 7) + 8).to(torch.uint8)
            scales[e] = s
        else:
            ex = torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2.0
            v = w / torch.exp2(ex)[..., None]
            a = v.abs()
            c = torch.zeros_like(a)
            for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
                c += (a > edge).to(torch.float32)
            c = (c + 8.0 * (v < 0).to(torch.float32)).to(torch.uint8)
            scales[e] = (ex + 127.0).to(torch.uint8)
        c = c.view(N, K // 2, 2)
        codes[e] = c[..., 0] | (c[..., 1] << 4)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op == "matvec":
        T, k, E, N, K = case["T"], case["k"], case["E"], case["N"], case["K"]
        st.update(_routing(g, T, E, k, case["valid"]))
        # SiLU * up products read token rows through the permutation, the others permuted rows
        st["a"] = (_randn(g, T if case["silu"] else T * k, K)).to(torch.bfloat16)
        st["codes"], st["scales"] = _quantised(g, E, N, K, case["fmt"], case["group"])
        return st
    T, H, dt = case["T"], case["H"], _DT[case["dtype"]]
    if op in ("norm", "norm_backward"):
        wdt = _DT[case["wdtype"]]
        # hidden states: a few channels much larger than the rest, and an offset
        chan = 1.0 + 4.0 * (torch.rand(H, generator=g, device=DEV) < 0.01)
        st["x"] = (_randn(g, T, H) * chan + 0.3).to(dt)
        st["weight"] = (1.0 + 0.1 * _randn(g, H)).to(wdt)
        st["bias"] = (0.1 * _randn(g, H)).to(wdt) if case["bias"] else None
        if op == "norm_backward":
            st["dy"] = _randn(g, T, H).to(dt)
            xf = st["x"].double()
            mean = xf.mean(1) if not case["rms"] else torch.zeros(T, dtype=torch.float64, device=DEV)
            var = ((xf - mean[:, None]) ** 2).mean(1)
            st["mean"] = None if case["rms"] else mean.float()
            st["rstd"] = (1.0 / torch.sqrt(var + EPS)).float()
        return st
    st["rng"] = torch.tensor([(seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 63), seed * 1000003],
                             dtype=torch.int64, device=DEV)
    if op == "combine_dropout":
        r = _routing(g, T, case["E"], case["k"], 1.0)
        st.update(r)
        st["y"] = _randn(g, T * case["k"], H).to(dt)
        st["residual"] = _randn(g, T, H).to(dt)
        return st
    st["x"] = _randn(g, T, H).to(dt)
    if op == "dropout" and case["rdtype"] != "none":
        st["residual"] = _randn(g, T, H).to(_DT[case["rdtype"]])
    return st


# -------------------------------------------------------------------------------- the plain forms

def _plain_norm(st):
    case = st["case"]
    x = st["x"].float()
    if case["rms"]:
        mean = None
        d = x
    else:
        mean = x.mean(dim=1)
        d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + EPS)
    y = d * rstd[:, None] * st["weight"].float()
    if st["bias"] is not None:
        y = y + st["bias"].float()
    y = y.to(st["x"].dtype)
    if not case["stats"]:
        return y
    return (y, rstd) if mean is None else (y, mean, rstd)


def _plain_norm_backward(st):
    case = st["case"]
    x, dy = st["x"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    xhat = (x if case["rms"] else x - st["mean"][:, None]) * rstd
    wdy = dy * st["weight"].float()
    dx = wdy - xhat * (wdy * xhat).mean(dim=1, keepdim=True)
    if not case["rms"]:
        dx = dx - wdy.mean(dim=1, keepdim=True)
    dx = (dx * rstd).to(st["x"].dtype)
    dw = (dy * xhat).sum(dim=0)
    return (dx, dw, dy.sum(dim=0)) if case["bias"] else (dx, dw)


def _philox(blocks, word2, seed):
    """Philox4x32-10 of the counters (block low, block high, word2, 0): four words each, in int64."""
    m = 0xFFFFFFFF
    c0, c1 = blocks & m, (blocks >> 32) & m
    c2 = torch.full_like(c0, word2)
    c3 = torch.zeros_like(c0)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return torch.stack([c0, c1, c2, c3], dim=1)


def _plain_keep(rng, n, p):
    """The kept elements of n: a 32-bit uniform each, its high half and its low half 16-bit pieces of
    two Philox blocks that eight consecutive elements share, not below p * 2^32."""
    blocks = torch.arange((n + 7) // 8, device=DEV, dtype=torch.int64) + rng[1]
    halves = []
    for word2 in (0, 1):
        w = _philox(blocks, word2, rng[0])
        halves.append(torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:n])
    return ((halves[0] << 16) | halves[1]) >= round(p * 4294967296.0)


def _plain_dropout(x, rng, p, residual):
    keep = _plain_keep(rng, x.numel(), p).view(x.shape)
    scale = 0.0 if p >= 1.0 else 1.0 / (1.0 - p)
    out = torch.where(keep, x * scale, torch.zeros_like(x))
    return out if residual is None else out + residual.float()


def _plain_combine_dropout(st):
    case = st["case"]
    T, k = case["T"], case["k"]
    pos = st["row_pos"].long().view(T, k)
    valid = pos < st["offsets"][-1]
    acc = torch.zeros(T, case["H"], dtype=torch.float32, device=DEV)
    for j in range(k):
        w = torch.where(valid[:, j], st["weights"][:, j], torch.zeros_like(st["weights"][:, j]))
        acc = acc + w[:, None] * st["y"][pos[:, j]].float()
    return _plain_dropout(acc, st["rng"], case["p"], st["residual"]).to(st["y"].dtype)


def _plain_dequant(codes, scales, fmt, group, dtype):
    N, half = codes.shape
    c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(N, half * 2)
    if fmt == "int4":
        v = c.to(dtype) - 8.0
        s = scales.to(dtype)
    else:
        v = torch.tensor(_E2M1, dtype=dtype, device=codes.device)[c.long()]
        s = torch.exp2(scales.to(dtype) - 127.0)
    return (v.view(N, -1, group) * s[..., None]).view(N, half * 2)


def _plain_matvec(st):
    case = st["case"]
    N, k, silu, seg = case["N"], case["k"], case["silu"], st["seg"]
    R = st["sorted_rows"].numel()
    out = torch.zeros(R, N // 2 if silu else N, dtype=torch.float32, device=DEV)
    for e in range(case["E"]):
        lo, hi = seg[e], seg[e + 1]
        if lo == hi:
            continue
        w = _plain_dequant(st["codes"][e], st["scales"][e], case["fmt"], case["group"], torch.float32)
        a = st["a"][st["sorted_rows"][lo:hi].long() // k] if silu else st["a"][lo:hi]
        acc = a.float() @ w.t()
        if silu:
            gate, up = acc[:, :N // 2], acc[:, N // 2:]
            acc = gate / (1.0 + torch.exp(-gate)) * up
        out[lo:hi] = acc
    return out.to(torch.bfloat16)


# ----------------------------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(st)
    if op == "norm_backward":
        return _plain_norm_backward(st)
    if op == "combine_dropout":
        return _plain_combine_dropout(st)
    if op == "matvec":
        return _plain_matvec(st)
    residual = st.get("residual")
    out = _plain_dropout(st["x"].float(), st["rng"], case["p"], residual)
    return out.to(st["x"].dtype if residual is None else residual.dtype)


def _run_own(st):
    import grouped_gemm_histogram_amd as g
    case = st["case"]
    op = case["op"]
    if op == "norm":
        res = g.layer_norm(st["x"], st["weight"], st["bias"], eps=EPS, rms=case["rms"], return_stats=case["stats"])
        if not case["stats"]:
            return res
        y, stats = res
        return (y, stats.rstd) if case["rms"] else (y, stats.mean, stats.rstd)
    if op == "norm_backward":
        stats = g.NormStats(mean=st["mean"], rstd=st["rstd"])
        gr = g.layer_norm_backward(st["dy"], st["x"], stats, st["weight"], bias_grad=case["bias"])
        return (gr.dx, gr.dweight, gr.dbias) if case["bias"] else (gr.dx, gr.dweight)
    if op == "dropout":
        return g.dropout_add(st["x"], st["rng"], case["p"], residual=st.get("residual"))
    if op == "dropout_backward":
        return g.dropout_add_backward(st["x"], st["rng"], case["p"])
    if op == "combine_dropout":
        return g.unpermute_combine_dropout(st["y"], st["row_pos"], st["weights"], st["offsets"], case["k"],
                                           st["rng"], case["p"], residual=st["residual"])
    if case["silu"]:
        return g.grouped_matvec_fourbit(st["a"], st["codes"], st["scales"], st["offsets"], "silu_mul",
                                        gather_rows=st["sorted_rows"], gather_div=case["k"])
    return g.grouped_matvec_fourbit(st["a"], st["codes"], st["scales"], st["offsets"])


# ------------------------------------------------------------------------------------ the work

def work(case):
    op = case["op"]
    if op == "matvec":
        R = case["T"] * case["k"]
        V = int(round(case["valid"] * R))
        E, N, K = case["E"], case["N"], case["K"]
        # experts that V random routes reach, on average
        active = E * (1.0 - (1.0 - 1.0 / E) ** V)
        per = N * K // 2 + N * (K // case["group"]) * (1 if case["fmt"] == "mxfp4" else 4)
        a_rows = math.ceil(V / case["k"]) if case["silu"] else V
        n_out = N // 2 if case["silu"] else N
        return {"bytes": int(active * per) + 2 * a_rows * K + 2 * R * n_out, "flops": 2 * V * N * K}
    T, H = case["T"], case["H"]
    n, b = T * H, _BYTES[case["dtype"]]
    if op == "norm":
        params = H * _BYTES[case["wdtype"]] * (2 if case["bias"] else 1)
        stats = 0 if not case["stats"] else 4 * T * (1 if case["rms"] else 2)
        return {"bytes": 2 * n * b + params + stats, "flops": 8 * n}
    if op == "norm_backward":
        stats = 4 * T * (1 if case["rms"] else 2)
        grads = 4 * H * (2 if case["bias"] else 1)
        return {"bytes": 3 * n * b + stats + H * _BYTES[case["wdtype"]] + grads, "flops": 14 * n}
    if op == "combine_dropout":
        return {"bytes": n * b * (case["k"] + 2) + 8 * T * case["k"], "flops": n * (2 * case["k"] + 2)}
    if op == "dropout" and case["rdtype"] != "none":
        return {"bytes": n * (b + 2 * _BYTES[case["rdtype"]]), "flops": 2 * n}
    return {"bytes": 2 * n * b, "flops": n}


# ------------------------------------------------------------------------- the definition in 64 bits

def _host(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def _exact_keep(rng, n, p):
    """The generator from its definition, on the host in unsigned arithmetic."""
    seed, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in rng.tolist())
    nb = -(-n // 8)
    pieces = []
    for stream in range(2):
        ctr = np.arange(nb, dtype=np.uint64) + np.uint64(offset)
        x = [ctr & np.uint64(0xFFFFFFFF), ctr >> np.uint64(32), np.full(nb, stream, np.uint64), np.zeros(nb, np.uint64)]
        key = [seed & 0xFFFFFFFF, seed >> 32]
        for r in range(10):
            a = np.uint64(0xD2511F53) * x[0]
            b = np.uint64(0xCD9E8D57) * x[2]
            x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF),
                 b & np.uint64(0xFFFFFFFF),
                 (a >> np.uint64(32)) ^ x[3] ^ np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF),
                 a & np.uint64(0xFFFFFFFF)]
        words = np.empty((nb, 4, 2), np.uint64)
        for i in range(4):
            words[:, i, 0] = x[i] & np.uint64(0xFFFF)
            words[:, i, 1] = x[i] >> np.uint64(16)
        pieces.append(words.reshape(-1)[:n])
    return pieces[0] * np.uint64(65536) + pieces[1] >= np.uint64(round(p * 2.0 ** 32))


def _exact_drop(v, rng, p, residual):
    keep = _exact_keep(rng, v.size, p).reshape(v.shape)
    out = np.where(keep, v / (1.0 - p) if p < 1.0 else 0.0, 0.0)
    return torch.from_numpy(out if residual is None else out + residual)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        x, w = st["x"].double(), st["weight"].double()
        n = case["H"]
        if op == "norm":
            mu = x.sum(1, keepdim=True) / n * (0.0 if case["rms"] else 1.0)
            inv = torch.rsqrt(((x - mu) ** 2).sum(1, keepdim=True) / n + EPS)
            y = torch.addcmul(st["bias"].double() if case["bias"] else torch.zeros_like(w), (x - mu) * inv, w)
            if not case["stats"]:
                return y
            return (y, inv[:, 0]) if case["rms"] else (y, mu[:, 0], inv[:, 0])
        # the transposed Jacobian of the normalised row applied to w * dy
        dy = st["dy"].double()
        inv = st["rstd"].double()[:, None]
        mu = 0.0 if case["rms"] else st["mean"].double()[:, None]
        z = (x - mu) * inv
        gz = dy * w
        dx = inv * (gz - z * ((gz * z).sum(1, keepdim=True) / n))
        if not case["rms"]:
            dx = dx - inv * (gz.sum(1, keepdim=True) / n)
        out = [dx, torch.einsum("th,th->h", dy, z)]
        if case["bias"]:
            out.append(dy.sum(0))
        return tuple(out)
    if op == "combine_dropout":
        T, k = case["T"], case["k"]
        y = st["y"].double()
        pos = st["row_pos"].long()
        wt = st["weights"].double().reshape(-1) * (pos < st["offsets"][-1])
        acc = (y[pos] * wt[:, None]).view(T, k, -1).sum(1)
        return _exact_drop(_host(acc), st["rng"], case["p"], _host(st["residual"]))
    if op in ("dropout", "dropout_backward"):
        return _exact_drop(_host(st["x"]), st["rng"], case["p"], _host(st.get("residual")))
    N, K = case["N"], case["K"]
    table = torch.arange(16, device=DEV, dtype=torch.float64) - 8.0
    if case["fmt"] == "mxfp4":
        c = torch.arange(16, device=DEV)
        ex, man = ((c >> 1) & 3).double(), (c & 1).double()
        mag = torch.where(ex > 0, (1.0 + man / 2) * 2.0 ** (ex - 1), man / 2)
        table = torch.where(c >= 8, -mag, mag)
    R = st["sorted_rows"].numel()
    out = torch.zeros(R, N // 2 if case["silu"] else N, dtype=torch.float64, device=DEV)
    rows = torch.arange(R, device=DEV)
    expert = torch.searchsorted(st["offsets"][1:].contiguous(), rows.to(torch.int32), right=True)
    src = st["sorted_rows"].long() // case["k"] if case["silu"] else rows
    for e in sorted(set(expert.tolist())):
        if e >= case["E"]:
            continue
        sel = (expert == e).nonzero()[:, 0]
        w = torch.empty(N, K, dtype=torch.float64, device=DEV)
        w[:, 0::2] = table[(st["codes"][e] % 16).long()]
        w[:, 1::2] = table[torch.div(st["codes"][e], 16, rounding_mode="floor").long()]
        sc = st["scales"][e].double()
        sc = torch.pow(2.0, sc - 127.0) if case["fmt"] == "mxfp4" else sc
        w *= sc.repeat_interleave(case["group"], dim=1)
        acc = torch.matmul(st["a"][src[sel]].double(), w.T)
        if case["silu"]:
            acc = acc[:, :N // 2] * torch.sigmoid(acc[:, :N // 2]) * acc[:, N // 2:]
        out[sel] = acc
    return out
