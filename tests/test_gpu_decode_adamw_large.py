"""The layer for few tokens at every number of tokens an expert can have; far ends of large arrays; every mantissa
through the AdamW step's square root; and the operators one after the other as a run uses them."""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, say
from oracle import adamw as oa
from test_gpu_decode import Case, FORMATS, UNIT

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_number_of_tokens_of_an_expert(fmt):
    """1 to 16 tokens of one expert, and as many split between it and the next one in the list, with rows of a step and a
    part of one."""
    u = UNIT[fmt]
    H, I = max(u, 128) + 5 * u, max(u, 128) + 3 * u
    case = Case(fmt, 16, H, I, 3, 2)
    for n in range(1, 17):
        case_n = Case.__new__(Case)
        case_n.__dict__.update(case.__dict__)
        case_n.x = case.x[:n]
        for split in (n, n // 2):
            logits = np.zeros((n, 3), np.float32)
            logits[:, 2] = 5.0
            logits[:split, 0] = 3.0
            logits[split:, 1] = 3.0
            case_n.logits = logits
            say("tokens", fmt, n, split)
            case_n.check(out=torch.float32)


def exact(x, rows13, cols2):
    """(out, tolerance) of one token with x of 128 elements, on one expert of which only some hidden columns live: rows13
    their gate and up rows.  Tolerance as in test_gpu_decode: sums of 128 products, then of two."""
    u = 2.0 ** -24
    gate, up = (rows13.double() @ x.double()).reshape(2, -1)
    eg, eu = (2 * 128 + 40) * u * (rows13.double().abs() @ x.double().abs()).reshape(2, -1)
    silu = gate / (1 + torch.exp(-gate))
    h = silu * up
    eh = 1.1 * up.abs() * eg + (silu.abs() + 1.1 * eg) * eu + h.abs() * ((8 + 1.5 * gate.abs()) * u + 2.0 ** -8)
    return cols2.double() @ h, cols2.double().abs() @ (eh + 64 * u * (h.abs() + eh)) + 1e-30


def test_weights_at_the_far_end_of_4_gib():
    """One expert's W13 of just under 4 GiB (bf16), and routed experts behind 4 GiB: first and last rows and columns
    count, all others are zeros."""
    for E, H, I in ((1, 32760, 32760), (70, 4096, 4000)):
        say("far", E, H, I)
        gen = torch.Generator(device=DEV).manual_seed(3)
        w13 = torch.zeros(E, 2 * I, H, dtype=BF, device=DEV)
        w2 = torch.zeros(E, H, I, dtype=BF, device=DEV)
        live = [0, I - 1]
        e = E - 1
        rows = torch.randn(4, H, device=DEV, generator=gen).mul_(0.2).to(BF)
        cols = torch.randn(H, 2, device=DEV, generator=gen).to(BF)
        w13[e, live] = rows[:2]
        w13[e, [I + i for i in live]] = rows[2:]
        w2[e][:, live] = cols
        ends = [*range(64), *range(H - 64, H)]
        x = torch.zeros(2, H, dtype=BF, device=DEV)
        x[:, ends] = torch.randn(2, 128, device=DEV, generator=gen).to(BF)
        logits = torch.zeros(2, E, device=DEV)
        logits[:, e] = 9.0
        got = g.forward_decode(x, logits, w13, w2, 1, out_dtype=torch.float32).double()
        for t in range(2):
            ref, tol = exact(x[t, ends], rows[:, ends], cols)
            assert bool(((got[t] - ref).abs() <= tol).all())
        assert float(got.abs().max()) > 0
        del w13, w2, got


def test_many_rows_quantised():
    """More rows than a launch's axis has waves, and codes behind 2 GiB."""
    H, rows = 32, 70_000_000
    some = torch.randn(1000, H, device=DEV).to(BF)
    x = some.repeat(rows // 1000, 1)
    codes, scales = g.quantize_rows_eightbit(x)
    few, fscales = g.quantize_rows_eightbit(some)
    for at in (0, rows // 2, rows - 1000):
        assert torch.equal(codes[at:at + 1000], few) and torch.equal(scales[at:at + 1000], fscales)
    assert bool((scales.reshape(-1, 1000) == fscales).all())


def test_eight_bit_products_behind_4_gib():
    """Experts' weights behind 4 GiB."""
    E, N, K = 70, 4096, 16384
    b = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    b[E - 1] = torch.randint(-127, 128, (N, K), device=DEV, dtype=torch.int8)
    sb = torch.ones(E, N, device=DEV)
    a = torch.randint(-127, 128, (3, K), device=DEV, dtype=torch.int8)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[E] = 3
    got = g.grouped_gemm_eightbit(a, torch.ones(3, device=DEV), b, sb, off, out_dtype=torch.float32)
    assert torch.equal(got.double(), (a.double() @ b[E - 1].double().T).float().double())


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_tensor_of_more_than_2_31_elements(bits):
    n, part = (1 << 31) + 4096 + 77, 4096
    tile = lambda s: (s * torch.randn(part, device=DEV)).to(BF).repeat(n // part + 1)[:n].contiguous()
    p, gr = tile(0.5), tile(0.02)
    first, last = p[:part].clone(), p[n - 77:].clone()
    state = g.adamw_init([p], bits=bits)
    g.adamw_step([p], [gr], state, lr=1e-2, step=1)
    for sl, old in ((slice(0, part), first), (slice(n - 77, n), last)):
        small, gs = old.clone(), gr[sl].clone()
        st = g.adamw_init([small], bits=bits)
        g.adamw_step([small], [gs], st, lr=1e-2, step=1)
        assert torch.equal(p[sl], small)
        m = state.m.view(torch.uint8) if bits == 8 else state.m
        ms = st.m.view(torch.uint8) if bits == 8 else st.m
        assert torch.equal(m[sl], ms[:small.numel()])
    assert bool((p.reshape(-1)[:n // part * part].reshape(-1, part) == p[:part]).all())


def test_square_roots_of_every_mantissa():
    """v halves (g = 0, beta2 = 0.5), so each float32 mantissa at both parities of the exponent passes the root; a wave of
    values below 2^-96 takes the other form of it.  To the bit against the oracle."""
    r = np.random.default_rng(0)
    n = 1 << 24
    i = np.arange(n, dtype=np.uint32)
    for low, high in ((32, 126), (1, 16)):     # exponent fields / 2
        field = (r.integers(low, high, n).astype(np.uint32) * 2 + (i >> 23)).astype(np.uint32)
        v = ((field << 23) | (i & 0x7fffff)).view(np.float32)
        m = np.full(n, 3.0, np.float32)
        zero = np.zeros(n, np.float32)
        p = torch.zeros(n, device=DEV)
        st = g.adamw_init([p])
        st.v.copy_(torch.from_numpy(v))
        st.m.copy_(torch.from_numpy(m))
        hyper = dict(lr=0.5, betas=(0.5, 0.5), eps=1e-30, weight_decay=0.0, step=1)
        g.adamw_step([p], [torch.zeros(n, device=DEV)], st, **hyper)
        rp, rm, rv = oa.step_f32(zero, zero, m, v, 0.5, 0.5, 0.5, 1e-30, 0.0, 1)[:3]
        assert (np32(st.v) == rv).all() and (np32(p) == rp).all()


def test_trained_quantised_and_served():
    """A training step on the experts, their quantisation, and the layer on the codes at many tokens and few: all of them
    captured as one graph and replayed, equal to the eager calls after each replay."""
    torch.manual_seed(0)
    T, H, I, E, k = 48, 64, 32, 8, 2
    x = torch.randn(T, H, device=DEV).to(BF)
    few = torch.randn(5, H, device=DEV).to(BF)
    logits, few_logits = torch.randn(T, E, device=DEV), torch.randn(5, E, device=DEV)
    w13 = (0.1 * torch.randn(E, 2 * I, H, device=DEV)).to(BF)
    w2 = (0.1 * torch.randn(E, H, I, device=DEV)).to(BF)
    state = g.adamw_init([w13, w2], bits=8)
    rng = torch.tensor([11, 0], dtype=torch.int64, device=DEV)
    schedule = torch.tensor(g.adamw_schedule(1e-2, 1), device=DEV)

    def step():
        out, aux = g.forward(x, logits, w13, w2, k, return_aux=True)
        gr = g.backward(x, w13, w2, out, aux.topk_weights, aux.offsets, aux.sorted_rows, aux.row_pos, grad_dtype=BF)
        g.adamw_step([w13, w2], [gr.dw13, gr.dw2], state, lr=1e-2, step=1, schedule=schedule, rng=rng)
        q13, s13 = g.quantize_rows_eightbit(w13)
        q2, s2 = g.quantize_rows_eightbit(w2)
        many = g.forward_eightbit(few, few_logits, q13, s13, q2, s2, k)
        return many, g.forward_decode(few, few_logits, q13, q2, k, w13_scale=s13, w2_scale=s2)

    tensors = [w13, w2, state.m.view(torch.uint8), state.v.view(torch.uint8), state.m_scale, state.v_scale]
    start = [t.clone() for t in tensors]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    for t, s in zip(tensors, start):
        t.copy_(s)
    eager = []
    for i in range(3):
        rng[1] = 1000 * i
        many, served = step()
        eager.append([t.clone() for t in (*tensors, many, served)])
    # activations in 8 bits (2^-8 of a row's largest value, twice) against activations as they are
    a, b = eager[0][-2].double(), eager[0][-1].double()
    assert float((a - b).abs().max()) <= 0.05 * float(b.abs().max())
    assert not torch.equal(eager[0][0], eager[1][0])
    for t, s in zip(tensors, start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        many, served = step()
    for i in range(3):
        rng[1] = 1000 * i
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip((*tensors, many, served), eager[i]):
            assert torch.equal(got, want), i
        torch.randn(1000, device=DEV).sum().item()   # the program's own work between replays
