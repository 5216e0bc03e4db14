"""Measured cases of the expert layer's 8-bit products, its form for a few tokens and its optimizer.

* ``gemm``: the grouped product of 8-bit integers with a scale for each token and each output
  channel, with and without SiLU(gate) * up, rows read directly or through the permutation;
* ``layer8``: the whole layer on such weights (tokens and hidden rows quantised on the way);
* ``decode``: the whole layer for a few tokens, on bf16, 8-bit or 4-bit weights;
* ``adamw``: an AdamW step over many tensors, with states in 32 bits or in 8.

``own`` false computes the plain form, true calls ``grouped_gemm_histogram_amd``.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda:0"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
# elements that share a scale of an 8-bit optimizer state; tensors start at multiples of it
BLOCK = 128
# rows and blocks whose largest value is below this are held as zeros: 448 over it is still finite
TINY = 2.0 ** -100

# the values of the sixteen 4-bit floating codes (1 sign, 2 exponent, 1 mantissa bit)
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # a decode batch through the DeepSeek-V3 layer's down projection, a quarter of its experts
        dict(name="int8_decode", op="gemm", T=16, k=8, E=64, N=7168, K=2048, silu=False, valid=1.0, out="bf16"),
        # the sentinel sweep's layer with an odd number of tokens, a quarter of the rows padding
        dict(name="int8_ragged", op="gemm", T=1031, k=8, E=128, N=1536, K=2048, silu=True, valid=0.75, out="f32"),
        # a prefill or training batch through the gpt-oss-20b layer's gate/up projection
        dict(name="int8_prefill", op="gemm", T=4096, k=4, E=32, N=5760, K=2880, silu=True, valid=1.0, out="bf16"),
        # small batch of the sentinel sweep's layer, half of its rows valid
        dict(name="int8_layer_small", op="layer8", T=64, H=2048, I=768, E=128, k=8, valid=0.5),
        # prefill through the Mixtral-8x7B layer
        dict(name="int8_layer_prefill", op="layer8", T=2048, H=4096, I=14336, E=8, k=2, valid=1.0),
        # one token of the gpt-oss-20b layer: four experts' weights, latency
        dict(name="decode_one_token", op="decode", fmt="bf16", group=0, T=1, H=2880, I=2880, E=32, k=4, valid=1.0),
        # a few sequences of it on 4-bit floating weights
        dict(name="decode_mxfp4", op="decode", fmt="mxfp4", group=32, T=4, H=2880, I=2880, E=32, k=4, valid=1.0),
        # a padded batch over many small experts with fine int4 groups
        dict(name="decode_int4_padded", op="decode", fmt="int4", group=32, T=16, H=2048, I=768, E=128, k=8,
             valid=0.75),
        # eight sequences of the DeepSeek-V3 layer, an eighth of its experts, e4m3 weights
        dict(name="decode_fp8", op="decode", fmt="fp8", group=128, T=8, H=7168, I=2048, E=32, k=8, valid=1.0),
        # the small parameters of six layers: norm weights, biases and router rows, odd sizes among them
        dict(name="adamw_small", op="adamw", sizes="2880,2880,92160,32,5761,2881", repeat=4, param="f32", grad="f32",
             bits=32, master=False, random=False),
        # the experts' weights of an eighth of the gpt-oss-20b layer: bf16 weights without a copy, 8-bit states
        dict(name="adamw_experts_8bit", op="adamw", sizes="66355200,33177600", repeat=1, param="bf16", grad="bf16",
             bits=8, master=False, random=True),
        # experts of the sentinel sweep's layer with a 32-bit copy of the weights
        dict(name="adamw_experts_master", op="adamw", sizes="50331648,25165824", repeat=1, param="bf16", grad="f32",
             bits=32, master=True, random=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gemm", "gemm", "layer8", "decode", "decode", "decode", "adamw", "adamw"])
    if op == "gemm":
        E = rng.choice([1, 8, 32, 128])
        K = 16 * _log(rng, 4, 448)
        N = 16 * _log(rng, 4, 512)
        while E * N * K > 700_000_000:
            E //= 2
        k = min(E, rng.choice([1, 2, 4, 8]))
        T = _log(rng, 1, min(16384 // k, max(1, 400_000_000_000 // (2 * N * K * k))))
        return dict(op=op, T=T, k=k, E=E, N=N, K=K, silu=rng.random() < 0.5, valid=rng.choice([1.0, rng.random()]),
                    out=rng.choice(["bf16", "f32"]))
    if op == "layer8":
        E = rng.choice([8, 32, 128])
        H, I = 16 * _log(rng, 8, 256), 16 * _log(rng, 8, 512)
        while E * H * I > 300_000_000:
            E //= 2
        k = min(E, rng.choice([1, 2, 4, 8]))
        T = _log(rng, 1, min(16384 // k, max(1, 400_000_000_000 // (6 * H * I * k))))
        return dict(op=op, T=T, H=H, I=I, E=E, k=k, valid=rng.choice([1.0, rng.random()]))
    if op == "decode":
        fmt = rng.choice(["bf16", "int8", "fp8", "int4", "mxfp4"])
        group = {"bf16": 0, "int8": 0, "fp8": 128, "mxfp4": 32, "int4": rng.choice([32, 64, 128])}[fmt]
        unit = {"bf16": 8, "int8": 16}.get(fmt, group)
        size = lambda lo, hi: unit * _log(rng, max(1, lo // unit), hi // unit)
        H, I = size(256, 7168), size(256, 4096)
        E = rng.choice([8, 32, 128])
        while E * H * I > 400_000_000:
            E //= 2
        return dict(op=op, fmt=fmt, group=group, T=rng.randrange(1, 17), H=H, I=I, E=E,
                    k=min(E, rng.choice([1, 2, 4, 8])), valid=rng.choice([1.0, 1.0, rng.random()]))
    bits = rng.choice([8, 32])
    param = rng.choice(["bf16", "f32"])
    master = param == "bf16" and rng.random() < 0.4
    sizes = [_log(rng, 1, 8_000_000) for _ in range(rng.randrange(1, 7))]
    return dict(op=op, sizes=",".join(str(s) for s in sizes), repeat=rng.choice([1, 1, 2]), param=param,
                grad=rng.choice(["bf16", "f32"]), bits=bits, master=master,
                random=rng.random() < 0.5 and (bits == 8 or (param == "bf16" and not master)))


# ------------------------------------------------------------------------------------ the inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _quantise_rows(x):
    """8-bit codes and a scale for each row: scale = amax / 127, code = round(x * (127 / amax)); a row
    below TINY counts as zeros, with scale 1."""
    x = x.float()
    amax = x.abs().amax(dim=-1)
    some = amax >= TINY
    scale = torch.where(some, amax / 127.0, torch.ones_like(amax))
    inv = torch.where(some, 127.0 / amax, torch.zeros_like(amax))
    return torch.round(x * inv[..., None]).to(torch.int8), scale


def _weights(g, E, N, K, fmt, group):
    """(weights, scales) of a format from normal values, an expert at a time."""
    shape, dt = {"bf16": ((N, K), torch.bfloat16), "int8": ((N, K), torch.int8),
                 "fp8": ((N, K), torch.float8_e4m3fn)}.get(fmt, ((N, K // 2), torch.uint8))
    w = torch.empty(E, *shape, dtype=dt, device=DEV)
    if fmt == "bf16":
        s = None
    elif fmt == "int8":
        s = torch.empty(E, N, dtype=torch.float32, device=DEV)
    elif fmt == "fp8":
        s = torch.empty(E, N // 128, K // 128, dtype=torch.float32, device=DEV)
    else:
        s = torch.empty(E, N, K // group, dtype=torch.uint8 if fmt == "mxfp4" else torch.float32, device=DEV)
    for e in range(E):
        v = _randn(g, N, K) * 0.02
        if fmt == "bf16":
            w[e] = v.to(dt)
        elif fmt == "int8":
            w[e], s[e] = _quantise_rows(v)
        elif fmt == "fp8":
            b = v.view(N // 128, 128, K // 128, 128)
            s[e] = b.abs().amax(dim=(1, 3)) / 448.0
            w[e] = (b / s[e][:, None, :, None]).clamp(-448, 448).view(N, K).to(dt)
        else:
            v = v.view(N, K // group, group)
            amax = v.abs().amax(dim=2)
            if fmt == "int4":
                s[e] = amax / 7.0
                c = (torch.round(v / s[e][..., None]).clamp_(-8, 7) + 8).to(torch.uint8)
            else:
                ex = torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2.0
                s[e] = (ex + 127.0).to(torch.uint8)
                v = v / torch.exp2(ex)[..., None]
                edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
                c = (torch.bucketize(v.abs(), edges) + 8 * (v < 0)).to(torch.uint8)
            c = c.view(N, K // 2, 2)
            w[e] = c[..., 0] | (c[..., 1] << 4)
    return w, s


def _prepare_gemm(case, g, st):
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    V = int(round(case["valid"] * R))
    ids = torch.topk(_randn(g, T, E), k, dim=1).indices.reshape(-1)
    flat = torch.arange(R, device=DEV)
    ids = torch.where(flat < V, ids, torch.full_like(ids, E))
    st["sorted_rows"] = torch.argsort(ids, stable=True).to(torch.int32)
    counts = torch.bincount(ids, minlength=E + 1)[:E]
    st["offsets"] = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)
    st["most"] = int(counts.max())
    # SiLU * up products read token rows through the permutation, the others permuted rows
    chan = 1.0 + 4.0 * (torch.rand(case["K"], generator=g, device=DEV) < 0.01)
    st["a"], st["a_scale"] = _quantise_rows(_randn(g, T if case["silu"] else R, case["K"]) * chan)
    st["b"], st["b_scale"] = _weights(g, E, case["N"], case["K"], "int8", 0)


def _prepare_adamw(case, g, st, seed):
    sizes = [int(s) for s in case["sizes"].split(",")] * case["repeat"]
    starts, n = [], 0
    for s in sizes:
        starts.append(n)
        n += -(-s // BLOCK) * BLOCK
    keep = torch.zeros(n, dtype=torch.bool, device=DEV)
    for a, s in zip(starts, sizes):
        keep[a:a + s] = True
    flat = lambda scale, dt: (_randn(g, n) * scale * keep).to(dt)
    w = flat(0.02, torch.float32)
    st["p"] = w.to(_DT[case["param"]])
    st["master"] = w if case["master"] else None
    st["g"] = flat(1e-3, _DT[case["grad"]])
    m = flat(3e-4, torch.float32)
    u = (flat(1e-3, torch.float32).abs() + 1e-4) * keep   # root of the second moment
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", u)):
            b = x.view(-1, BLOCK)
            amax = b.abs().amax(dim=1)
            s = torch.where(amax >= TINY, amax / 448.0, torch.ones_like(amax))
            st[name] = (b / s[:, None]).clamp(-448, 448).view(-1).to(torch.float8_e4m3fn)
            st[name + "_scale"] = s
    else:
        st["m"], st["v"] = m, u * u
    cut = lambda t: [t[a:a + s] for a, s in zip(starts, sizes)]
    st["params"], st["grads"] = cut(st["p"]), cut(st["g"])
    st["rng"] = None
    if case["random"]:
        st["rng"] = torch.tensor([(seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 63), seed * 1000003],
                                 dtype=torch.int64, device=DEV)
    # the factor of a norm clip, left on the GPU
    st["grad_scale"] = torch.full((1,), 0.5, device=DEV) + 0.25 * torch.rand(1, generator=g, device=DEV)
    st["hyper"] = dict(lr=3e-4, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, step=20 + seed % 50)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "gemm":
        _prepare_gemm(case, g, st)
    elif case["op"] == "adamw":
        _prepare_adamw(case, g, st, seed)
    else:
        T, H, I, E = case["T"], case["H"], case["I"], case["E"]
        fmt = case.get("fmt", "int8")
        st["x"] = _randn(g, T, H).to(torch.bfloat16)
        st["logits"] = _randn(g, T, E)
        st["w13"], st["w13_scale"] = _weights(g, E, 2 * I, H, fmt, case.get("group", 0))
        st["w2"], st["w2_scale"] = _weights(g, E, H, I, fmt, case.get("group", 0))
        st["valid"] = int(round(case["valid"] * T * case["k"]))
    return st


# -------------------------------------------------------------------------------- the plain forms

def _silu_mul(acc):
    gate, up = acc.chunk(2, dim=-1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_grouped(a, a_scale, b, b_scale, expert, within, most):
    """Rows a [R, K] (codes) of experts `expert`, each row the `within`-th of its expert's: one
    batched product over experts of their rows padded to `most`, scaled by rows and channels."""
    E, _, K = b.shape
    pad = torch.zeros(E + 1, most, K, dtype=torch.float32, device=DEV)
    pad[expert, within] = a.float()
    acc = torch.bmm(b.float(), pad[:E].transpose(1, 2).contiguous()).transpose(1, 2)
    e = expert.clamp(max=E - 1)
    return acc[e, within] * a_scale[:, None] * b_scale[e]


def _plain_gemm(st):
    case = st["case"]
    E, most = case["E"], max(1, st["most"])
    rows = torch.arange(st["sorted_rows"].numel(), device=DEV)
    off = st["offsets"].long()
    expert = torch.searchsorted(off[1:].contiguous(), rows, right=True)
    within = torch.where(expert < E, rows - off[expert.clamp(max=E - 1)], rows % most)
    src = st["sorted_rows"].long() // case["k"] if case["silu"] else rows
    acc = _plain_grouped(st["a"][src], st["a_scale"][src], st["b"], st["b_scale"], expert, within, most)
    if case["silu"]:
        acc = _silu_mul(acc)
    return torch.where((expert < E)[:, None], acc, torch.zeros_like(acc)).to(_DT[case["out"]])


def _plain_route(st):
    """(ids [T, k], weights [T, k]): softmax over the k largest logits; id E and weight 0 past the valid rows."""
    case = st["case"]
    top = torch.topk(st["logits"], case["k"], dim=1)
    ex = torch.exp(top.values - top.values[:, :1])
    w = ex / ex.sum(dim=1, keepdim=True)
    flat = torch.arange(case["T"] * case["k"], device=DEV).view(case["T"], case["k"])
    ok = flat < st["valid"]
    return torch.where(ok, top.indices, torch.full_like(top.indices, case["E"])), torch.where(ok, w, torch.zeros_like(w))


def _plain_layer8(st):
    case = st["case"]
    T, E, k = case["T"], case["E"], case["k"]
    ids, w = _plain_route(st)
    ids = ids.reshape(-1)
    order = torch.argsort(ids, stable=True)
    expert = ids[order]
    counts = torch.bincount(ids, minlength=E + 1)
    start = torch.cumsum(counts, 0) - counts
    most = max(1, int(counts[:E].max()))
    within = torch.where(expert < E, torch.arange(T * k, device=DEV) - start[expert], torch.zeros_like(expert))
    xq, xs = _quantise_rows(st["x"])
    tok = order // k
    h = _silu_mul(_plain_grouped(xq[tok], xs[tok], st["w13"], st["w13_scale"], expert, within, most))
    hq, hs = _quantise_rows(h.to(torch.bfloat16))
    y = _plain_grouped(hq, hs, st["w2"], st["w2_scale"], expert, within, most).to(torch.bfloat16).float()
    y = torch.where((expert < E)[:, None], y, torch.zeros_like(y))
    out = torch.empty_like(y)
    out[order] = y
    return (out.view(T, k, -1) * w[..., None]).sum(dim=1).to(torch.bfloat16)


def _plain_values(w, s, fmt, group):
    """The values [n, N, K] in f32 that the weights of some experts stand for."""
    if fmt == "bf16":
        return w.float()
    if fmt == "int8":
        return w.float() * s[..., None]
    n, N = w.shape[:2]
    if fmt == "fp8":
        return (w.float().view(n, N // 128, 128, -1, 128) * s[:, :, None, :, None]).view(n, N, -1)
    c = torch.stack([w & 15, w >> 4], dim=3).view(n, N, -1, group)
    if fmt == "int4":
        return ((c.float() - 8.0) * s[..., None]).view(n, N, -1)
    v = torch.tensor(_E2M1, device=DEV)[c.long()]
    return (v * torch.exp2(s.float() - 127.0)[..., None]).view(n, N, -1)


def _plain_decode(st):
    case = st["case"]
    T, E, k, fmt, group = case["T"], case["E"], case["k"], case["fmt"], case["group"]
    ids, w = _plain_route(st)
    pick = lambda t, at: None if t is None else (t.view(torch.uint8)[at].view(t.dtype) if at is not None else t)
    if T * k < E:   # the routed experts only, one for each routed row
        at = ids.reshape(-1).clamp(max=E - 1)
        gate = torch.zeros(T, k, T, device=DEV)
        gate[torch.arange(T, device=DEV), :, torch.arange(T, device=DEV)] = w
        gate = gate.view(T * k, T)
    else:
        at = None
        gate = torch.zeros(T, E + 1, device=DEV).scatter(1, ids, w)[:, :E].t().contiguous()
    scale = lambda s: None if s is None else (s if at is None else s[at])
    w13 = _plain_values(pick(st["w13"], at), scale(st["w13_scale"]), fmt, group)
    acc = torch.matmul(w13, st["x"].float().t().contiguous()).transpose(1, 2)          # [n, T, 2I]
    h = _silu_mul(acc).to(torch.bfloat16).float()
    w2 = _plain_values(pick(st["w2"], at), scale(st["w2_scale"]), fmt, group)
    y = torch.bmm(w2, h.transpose(1, 2).contiguous()).transpose(1, 2)                  # [n, T, H]
    return (y * gate[..., None]).sum(dim=0).to(torch.bfloat16)


def _philox16(rng, n):
    """n 16-bit pieces of Philox4x32-10 with counters (block low, block high, 2, 0), in int64."""
    m = 0xFFFFFFFF
    block = torch.arange((n + 7) // 8, device=DEV, dtype=torch.int64) + rng[1]
    c0, c1 = block & m, (block >> 32) & m
    c2, c3 = torch.full_like(c0, 2), torch.zeros_like(c0)
    k0, k1 = rng[0] & m, (rng[0] >> 32) & m
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & m) ^ c1 ^ k0, p1 & m, ((p0 >> 32) & m) ^ c3 ^ k1, p0 & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    w = torch.stack([c0, c1, c2, c3], dim=1)
    return torch.stack([w & 0xFFFF, w >> 16], dim=2).reshape(-1)[:n]


def _plain_e4m3(x, piece, least):
    """x (within +-448) as e4m3, rounded up with the chance of the piece (None: to nearest); `least`: a
    value above zero keeps the smallest code at least."""
    if piece is None:
        q = x.to(torch.float8_e4m3fn)
    else:
        a = x.abs()
        small = a < 2.0 ** -6   # codes below the smallest normal have its step: add it to round there
        bits = torch.where(small, a + 2.0 ** -6, a).view(torch.int32)
        code = ((bits + (piece.to(torch.int32) << 4) + 8) >> 20) - torch.where(small, 968, 960)
        code = code.clamp(max=126)
        q = torch.where(x < 0, code | 128, code).to(torch.uint8).view(torch.float8_e4m3fn)
    if least:
        q = torch.where((x > 0) & (q.view(torch.uint8) == 0), torch.ones_like(q.view(torch.uint8)),
                        q.view(torch.uint8)).view(torch.float8_e4m3fn)
    return q


def _plain_adamw(st):
    case, h = st["case"], st["hyper"]
    b1, b2 = h["betas"]
    small = case["bits"] == 8
    g = st["g"].float() * st["grad_scale"]
    if small:
        m = (st["m"].float().view(-1, BLOCK) * st["m_scale"][:, None]).view(-1)
        u = (st["v"].float().view(-1, BLOCK) * st["v_scale"][:, None]).view(-1)
        v = u * u
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    u = torch.sqrt(v)
    upd = m / (u * (1.0 / math.sqrt(1.0 - b2 ** h["step"])) + h["eps"])
    p = st["p"].float() if st["master"] is None else st["master"]
    p = p * (1.0 - h["lr"] * h["weight_decay"]) - upd * (h["lr"] / (1.0 - b1 ** h["step"]))
    piece = None if st["rng"] is None else _philox16(st["rng"], p.numel())
    out = dict(p=st["p"], m=st["m"], v=st["v"])
    if st["master"] is not None:
        st["master"].copy_(p)
        out["master"] = st["master"]
    if st["p"].dtype == torch.bfloat16 and st["master"] is None and piece is not None:
        bits = p.view(torch.int32) + piece.to(torch.int32)
        p = (bits & -65536).view(torch.float32)
    st["p"].copy_(p)
    if small:
        for name, x in (("m", m), ("v", u)):
            b = x.view(-1, BLOCK)
            amax = b.abs().amax(dim=1)
            some = amax >= TINY
            scale = torch.where(some, amax / 448.0, torch.ones_like(amax))
            inv = torch.where(some, 448.0 / amax, torch.zeros_like(amax))
            q = (b * inv[:, None]).clamp(-448.0, 448.0).view(-1)
            st[name].copy_(_plain_e4m3(q, piece, name == "v"))
            st[name + "_scale"].copy_(scale)
            out[name + "_scale"] = st[name + "_scale"]
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    return out


# ----------------------------------------------------------------------------------- one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    return {"gemm": _plain_gemm, "layer8": _plain_layer8, "decode": _plain_decode, "adamw": _plain_adamw}[
        st["case"]["op"]](st)


def _run_own(st):
    import grouped_gemm_histogram_amd as g
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        more = dict(gather_rows=st["sorted_rows"], gather_div=case["k"]) if case["silu"] else {}
        return g.grouped_gemm_eightbit(st["a"], st["a_scale"], st["b"], st["b_scale"], st["offsets"],
                                       "silu_mul" if case["silu"] else "none", out_dtype=_DT[case["out"]], **more)
    if op == "layer8":
        return g.forward_eightbit(st["x"], st["logits"], st["w13"], st["w13_scale"], st["w2"], st["w2_scale"],
                                  case["k"], num_valid_rows=st["valid"])
    if op == "decode":
        return g.forward_decode(st["x"], st["logits"], st["w13"], st["w2"], case["k"], num_valid_rows=st["valid"],
                                w13_scale=st["w13_scale"], w2_scale=st["w2_scale"])
    state = g.AdamWState(m=st["m"], v=st["v"], m_scale=st.get("m_scale"), v_scale=st.get("v_scale"),
                         master=st["master"])
    g.adamw_step(st["params"], st["grads"], state, grad_scale=st["grad_scale"], rng=st["rng"], **st["hyper"])
    out = dict(p=st["p"], m=st["m"], v=st["v"])
    out.update({name: st[name] for name in ("m_scale", "v_scale", "master") if st.get(name) is not None})
    return out


# ------------------------------------------------------------------------------------ the work

def _weight_bytes(N, K, fmt, group):
    """Bytes of one expert's [N, K]."""
    if fmt == "bf16":
        return 2 * N * K
    if fmt == "int8":
        return N * K + 4 * N
    if fmt == "fp8":
        return N * K + N * K // 4096
    return N * K // 2 + N * (K // group) * (1 if fmt == "mxfp4" else 4)


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(int(s) for s in case["sizes"].split(",")) * case["repeat"]
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        weights = 2 * _BYTES[case["param"]] if not case["master"] else 8 + _BYTES[case["param"]]
        return {"bytes": int(n * (state + weights + _BYTES[case["grad"]])), "flops": 16 * n}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    V = int(round(case["valid"] * R))
    active = E * (1.0 - (1.0 - 1.0 / E) ** V)   # experts that V random routes reach, on average
    if op == "gemm":
        N, K = case["N"], case["K"]
        n_out = N // 2 if case["silu"] else N
        a_rows = math.ceil(V / k) if case["silu"] else V
        return {"bytes": int(active * _weight_bytes(N, K, "int8", 0)) + a_rows * (K + 4) + R * n_out * _BYTES[case["out"]],
                "flops": 2 * V * N * K}
    H, I = case["H"], case["I"]
    fmt, group = case.get("fmt", "int8"), case.get("group", 0)
    per = _weight_bytes(2 * I, H, fmt, group) + _weight_bytes(H, I, fmt, group)
    return {"bytes": int(active * per) + 4 * T * E + 4 * T * H, "flops": 6 * V * H * I}


# ------------------------------------------------------------------------- the definition in 64 bits

def _exact_values(w, s, fmt, group):
    """[N, K] in f64 of one expert."""
    if fmt == "bf16":
        return w.double()
    if fmt == "int8":
        return w.double() * s.double()[:, None]
    if fmt == "fp8":
        return w.to(torch.float32).double() * s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    N, half = w.shape
    code = torch.empty(N, 2 * half, dtype=torch.int64, device=DEV)
    code[:, 0::2] = (w % 16).long()
    code[:, 1::2] = torch.div(w, 16, rounding_mode="floor").long()
    if fmt == "int4":
        table = torch.arange(16, device=DEV, dtype=torch.float64) - 8.0
        return table[code] * s.double().repeat_interleave(group, dim=1)
    c = torch.arange(16, device=DEV)
    ex, man = ((c >> 1) & 3).double(), (c & 1).double()
    mag = torch.where(ex > 0, (1.0 + man / 2) * 2.0 ** (ex - 1), man / 2)
    table = torch.where(c >= 8, -mag, mag)
    return table[code] * torch.pow(2.0, s.double() - 127.0).repeat_interleave(group, dim=1)


def _exact_glu(acc):
    n = acc.shape[1] // 2
    return acc[:, :n] * torch.sigmoid(acc[:, :n]) * acc[:, n:]


def _exact_codes(x):
    """Dequantised rows of the 8-bit quantiser, whose decisions are taken in 32 bits."""
    x = x.float()
    top = x.abs().max(dim=1, keepdim=True).values
    inv = torch.where(top >= TINY, 127.0 / top, torch.zeros_like(top))
    step = torch.where(top >= TINY, top / 127.0, torch.ones_like(top))
    return (x * inv).round().double() * step.double()


def _exact_layer(case, st):
    T, E, k, fmt, group = case["T"], case["E"], case["k"], case.get("fmt", "int8"), case.get("group", 0)
    order = torch.argsort(st["logits"].double(), dim=1, descending=True, stable=True)[:, :k]
    w = torch.softmax(torch.gather(st["logits"].double(), 1, order), dim=1)
    flat = torch.arange(T * k, device=DEV).view(T, k)
    out = torch.zeros(T, case["H"], dtype=torch.float64, device=DEV)
    x = _exact_codes(st["x"]) if case["op"] == "layer8" else st["x"].double()
    for e in range(E):
        t, j = ((order == e) & (flat < st["valid"])).nonzero(as_tuple=True)
        if not t.numel():
            continue
        one = lambda s: None if s is None else s[e]
        h = _exact_glu(x[t] @ _exact_values(st["w13"][e], one(st["w13_scale"]), fmt, group).T)
        if case["op"] == "layer8":
            h = _exact_codes(h.to(torch.bfloat16))
        y = h @ _exact_values(st["w2"][e], one(st["w2_scale"]), fmt, group).T
        out.index_add_(0, t, y * w[t, j][:, None])
    return out


def _exact_gemm(case, st):
    R, silu = st["sorted_rows"].numel(), case["silu"]
    off = st["offsets"].tolist()
    out = torch.zeros(R, case["N"] // 2 if silu else case["N"], dtype=torch.float64, device=DEV)
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        src = torch.div(st["sorted_rows"][lo:hi].long(), case["k"], rounding_mode="floor") if silu else slice(lo, hi)
        acc = st["a"][src].double() @ st["b"][e].double().T
        acc = acc * torch.outer(st["a_scale"][src].double(), st["b_scale"][e].double())
        out[lo:hi] = _exact_glu(acc) if silu else acc
    return out


def _exact_pieces(rng, n):
    """The generator's 16-bit pieces from its definition: products split into halves of 32 bits."""
    seed, offset = (int(v) & 0xFFFFFFFFFFFFFFFF for v in rng.tolist())
    low = torch.tensor(0xFFFFFFFF, dtype=torch.int64, device=DEV)
    ctr = torch.arange(-(-n // 8), dtype=torch.int64, device=DEV) + offset
    x = [ctr & low, (ctr >> 32) & low, torch.full_like(ctr, 2), torch.zeros_like(ctr)]
    for r in range(10):
        hi0, hi1 = (x[0] * 0xD2511F53 >> 32) & low, (x[2] * 0xCD9E8D57 >> 32) & low
        lo0, lo1 = (x[0] * 0xD2511F53) & low, (x[2] * 0xCD9E8D57) & low
        x = [hi1 ^ x[1] ^ ((seed + r * 0x9E3779B9) & 0xFFFFFFFF), lo1,
             hi0 ^ x[3] ^ (((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF), lo0]
    out = torch.empty(ctr.numel(), 8, dtype=torch.int64, device=DEV)
    for i in range(4):
        out[:, 2 * i], out[:, 2 * i + 1] = x[i] % 65536, torch.div(x[i], 65536, rounding_mode="floor")
    return out.view(-1)[:n]


def _exact_round(x, piece, mantissa, least_exp, add):
    """|x| to a float of `mantissa` stored bits and least exponent `least_exp`: down, or up where the
    fraction of a step and the piece's share of one reach 1."""
    a = x.abs()
    ex = torch.floor(torch.log2(a.clamp_min(1e-300))).clamp_min(least_exp)
    step = torch.pow(2.0, ex - mantissa)
    return torch.copysign(torch.floor(a / step + (piece.double() + add) / 65536.0) * step, x)


def _exact_adamw(case, st):
    hy = st["hyper"]
    (b1, b2), t = hy["betas"], hy["step"]
    grad = st["g"].double() * st["grad_scale"].double()
    wide = lambda c, s: (c.float().double().view(-1, BLOCK) * s.double()[:, None]).view(-1)
    small = case["bits"] == 8
    m = wide(st["m"], st["m_scale"]) if small else st["m"].double()
    v = wide(st["v"], st["v_scale"]) ** 2 if small else st["v"].double()
    m = b1 * m + (1 - b1) * grad
    v = b2 * v + (1 - b2) * grad ** 2
    p = (st["p"] if st["master"] is None else st["master"]).double()
    p = p - hy["lr"] * (hy["weight_decay"] * p + (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + hy["eps"]))
    out = dict(p=p, m=m, v=v)
    if st["master"] is not None:
        out["master"] = p
    piece = _exact_pieces(st["rng"], p.numel()) if st["rng"] is not None else None
    if piece is not None and case["param"] == "bf16" and st["master"] is None:
        out["p"] = _exact_round(p, piece, 7, -126, 0.0)
    if small:
        for name, x in (("m", m), ("v", torch.sqrt(v))):
            top = x.view(-1, BLOCK).abs().max(dim=1).values
            scale = torch.where(top >= TINY, top / 448.0, torch.ones_like(top))
            q = (x.view(-1, BLOCK) / scale[:, None]).view(-1)
            if piece is not None:
                q = _exact_round(q, piece, 3, -6, 0.5)
                if name == "v":
                    q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
            out[name], out[name + "_scale"] = q, scale
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"gemm": _exact_gemm, "layer8": _exact_layer, "decode": _exact_layer, "adamw": _exact_adamw}[case["op"]](case, st)
