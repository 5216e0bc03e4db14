"""AdamW on the GPU against the oracle's float32 steps, to the bit: every operation is one rounding in a
defined order, and so are the states' codes; the oracle's own distance from the formula in 64 bits is bounded in
test_oracle_eightbit_adamw."""
import numpy as np
import pytest
import torch

import grouped_gemm_histogram_amd as g
from helpers import np32, npu8, say
from oracle import adamw as oa, e4m3
from oracle.eightbit import bf16

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F = np.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.97), eps=1e-8, weight_decay=0.1, step=4)


def same(a, b):
    a, b = np.asarray(a), np.asarray(b)
    return a.shape == b.shape and ((a == b) | (np.isnan(a) & np.isnan(b))).all()


class Run:
    """Tensors with gradients and states in the middle of a run, and what the oracle makes of them."""

    def __init__(self, sizes, p_dtype, g_dtype, bits, master, seed=0, rng=None):
        r = np.random.default_rng(seed)
        self.sizes, self.bits, self.rng = sizes, bits, rng
        new = lambda n, s, dt: torch.from_numpy((s * r.normal(size=n)).astype(F)).to(dt).to(DEV)
        self.params = [new(n, 0.5, p_dtype) for n in sizes]
        self.grads = [new(n, 0.02, g_dtype) for n in sizes]
        self.state = g.adamw_init(self.params, bits=bits, master=master)
        *self.starts, total = g.adamw_starts(self.params)
        used = np.zeros(total, bool)
        for a, n in zip(self.starts, sizes):
            used[a:a + n] = True
        m = np.where(used, 0.01 * r.normal(size=total), 0).astype(F)
        v = np.where(used, 1e-4 * r.random(total) ** 4, 0).astype(F)
        if bits == 8:
            for name, x in (("m", m), ("v", np.sqrt(v))):
                pairs = [oa.code_block(b, None, name == "v") for b in x.reshape(-1, 128)]
                code = torch.from_numpy(np.concatenate([c for c, _ in pairs]).astype(np.uint8))
                getattr(self.state, name).copy_(code.to(DEV).view(torch.float8_e4m3fn))
                getattr(self.state, name + "_scale").copy_(torch.tensor([float(s) for _, s in pairs]).to(DEV))
        else:
            self.state.m.copy_(torch.from_numpy(m))
            self.state.v.copy_(torch.from_numpy(v))
            self.state.m[torch.from_numpy(~used).to(DEV)] = 7.0     # between the tensors: not ours to touch
        if master:
            self.state.master += torch.from_numpy(np.where(used, 1e-4 * r.normal(size=total), 3.0).astype(F)).to(DEV)
        self.used = used

    def expected(self, grad_scale=1.0, schedule=None, **hyper):
        h = dict(HYPER, **hyper)
        b1, b2 = h.pop("betas")
        st = self.state
        host = lambda t: None if t is None else t.detach().cpu()
        small = self.bits == 8
        m, v = host(st.m), host(st.v)
        if small:
            sm, sv = host(st.m_scale).numpy(), host(st.v_scale).numpy()
            m = (e4m3.decode(npu8(m)).astype(F).reshape(-1, 128) * sm[:, None]).reshape(-1).astype(F)
            u = (e4m3.decode(npu8(v)).astype(F).reshape(-1, 128) * sv[:, None]).reshape(-1).astype(F)
            v = u * u
        else:
            m, v = m.numpy().copy(), v.numpy().copy()
        ms = None if st.master is None else host(st.master).numpy().copy()
        seed = off = 0
        if self.rng is not None:
            seed, off = (int(x) & oa.dropout.M64 for x in self.rng.tolist())
        out = dict(p=[], m=m, v=v, master=ms)
        if small:
            out.update(m=np.zeros(m.size, np.uint8), v=np.zeros(m.size, np.uint8), sm=np.empty(m.size // 128, F),
                       sv=np.empty(m.size // 128, F))
        for a, n, p, gr in zip(self.starts, self.sizes, self.params, self.grads):
            p0 = np32(p) if ms is None else ms[a:a + n]
            p1, m1, v1, u1 = oa.step_f32(p0, np32(gr), m[a:a + n], v[a:a + n], beta1=b1, beta2=b2, grad_scale=grad_scale,
                                         schedule=schedule, **h)
            piece = None if self.rng is None else oa.pieces(a, n, seed, off)
            if ms is not None:
                ms[a:a + n] = p1
            if p.dtype == torch.bfloat16:
                if ms is None and piece is not None:
                    p1 = oa.by_chance(p1, piece, 7, -126, 0.0)
                else:
                    p1 = bf16(p1)
            out["p"].append(p1)
            if not small:
                m[a:a + n], v[a:a + n] = m1, v1
                continue
            for at in range(0, n, 128):
                cut = slice(at, min(n, at + 128))
                q = None if piece is None else piece[cut]
                for name, x in (("m", m1), ("v", u1)):
                    code, scale = oa.code_block(x[cut], q, name == "v")
                    out[name][a + at:a + at + code.size] = code
                    out["s" + name][(a + at) // 128] = scale
        return out

    def check(self, want):
        st = self.state
        for i, (p, w) in enumerate(zip(self.params, want["p"])):
            assert same(np32(p), w), ("param", i, int((np32(p) != w).sum()))
        if self.bits == 8:
            for name in ("m", "v"):
                got = npu8(getattr(st, name))
                assert (got == want[name]).all(), (name, int((got != want[name]).sum()))
                assert (np32(getattr(st, name + "_scale")) == want["s" + name]).all(), name
        else:
            assert same(np32(st.m), want["m"]) and same(np32(st.v), want["v"])
        if st.master is not None:
            assert same(np32(st.master), want["master"])

    def step(self, **more):
        g.adamw_step(self.params, self.grads, self.state, rng=self.rng, **dict(HYPER, **more))
        torch.cuda.synchronize()


SIZES = [[1], [8, 127, 128, 129], [2047, 1, 0, 2048, 2049, 5], [0, 4100]]
KINDS = [(p, gr, bits, master) for p in (torch.float32, torch.bfloat16) for gr in (torch.float32, torch.bfloat16)
         for bits in (32, 8) for master in (False, True) if not (master and p == torch.float32)]


@pytest.mark.parametrize("random", [False, True])
@pytest.mark.parametrize("p,gr,bits,master", KINDS)
@pytest.mark.parametrize("sizes", SIZES)
def test_step(sizes, p, gr, bits, master, random):
    say("adamw", sizes, p, gr, bits, master, random)
    rng = torch.tensor([0x1234567890ABCDEF, (1 << 33) + 5], dtype=torch.int64, device=DEV) if random else None
    run = Run(sizes, p, gr, bits, master, seed=sum(sizes), rng=rng)
    for t in (4, 5):
        want = run.expected(step=t)
        run.step(step=t)
        run.check(want)


def test_many_tensors():
    """More than one launch's 64 tensors, some empty."""
    run = Run([(i * 37) % 300 for i in range(150)], torch.bfloat16, torch.bfloat16, 8, False)
    want = run.expected()
    run.step()
    run.check(want)


def test_first_step_from_zeros():
    for bits in (8, 32):
        run = Run([1000], torch.float32, torch.float32, bits, False)
        run.state = g.adamw_init(run.params, bits=bits)
        want = run.expected(step=1)
        run.step(step=1)
        run.check(want)


def test_grad_scale_schedule_and_skip():
    for bits in (8, 32):
        run = Run([700, 33], torch.bfloat16, torch.float32, bits, True)
        scale = torch.tensor([0.37], device=DEV)
        sched = torch.tensor(g.adamw_schedule(2e-3, 9, HYPER["betas"]), device=DEV)
        want = run.expected(grad_scale=F(0.37), schedule=sched.cpu().numpy())
        run.step(grad_scale=scale, schedule=sched)
        run.check(want)
        for bad in (float("nan"), float("inf")):
            before = [t.clone() for t in run.params] + [run.state.m.clone(), run.state.v.clone(), run.state.master.clone()]
            run.step(grad_scale=torch.tensor([bad], device=DEV))
            after = run.params + [run.state.m, run.state.v, run.state.master]
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(before, after))


def test_blocks_without_values_and_extremes():
    """Gradients of zero from zero states, blocks below the least scale, values far below their block's largest."""
    run = Run([128 * 5], torch.float32, torch.float32, 8, False)
    run.state = g.adamw_init(run.params, bits=8)
    gr = run.grads[0]
    gr[:128] = 0
    gr[128:256] = 1e-36
    gr[256:384] *= torch.logspace(-30, 3, 128, device=DEV)
    gr[384:512] = 1e15
    for t in (1, 2, 3):
        want = run.expected(step=t)
        run.step(step=t)
        run.check(want)
    # a gradient below 2^-75 has a square below 2^-150, zero in f32; from 2^-70 on the second moment is above it
    seen = np.abs(np32(gr)[256:384]) >= 2.0 ** -70
    assert seen.any() and not seen.all()
    assert (npu8(run.state.v)[256:384][seen] >= 1).all() and (npu8(run.state.v)[256:384][np32(gr)[256:384] == 0] == 0).all()


@pytest.mark.parametrize("random", [False, True])
def test_bad_gradients_stay_where_they_are(random):
    rng = torch.tensor([5, 6], dtype=torch.int64, device=DEV) if random else None
    for bits in (32, 8):
        run = Run([512], torch.bfloat16, torch.float32, bits, False, rng=rng)
        clean = run.expected()
        run.grads[0][130] = float("nan")
        run.grads[0][300] = float("inf")
        run.step()
        p = np32(run.params[0])
        bad = np.zeros(512, bool)
        bad[[130, 300]] = True
        assert np.isnan(p[bad]).all() and same(p[~bad], clean["p"][0][~bad])
        if bits == 32:
            assert not np.isfinite(np32(run.state.m)[bad]).any() and same(np32(run.state.m)[~bad], clean["m"][~bad])
            continue
        m = e4m3.decode(npu8(run.state.m)).reshape(-1, 128) * np32(run.state.m_scale)[:, None]
        assert np.isnan(m[1, 2]) and np.isfinite(np.delete(m[1], 2)).all()        # a NaN: its element
        assert np.isnan(m[2]).all() or not np.isfinite(m[2, 44])                  # an infinity: its block
        assert (npu8(run.state.m)[:128] == clean["m"][:128]).all() and (npu8(run.state.m)[384:] == clean["m"][384:]).all()


def test_slow_averages_move_by_chance():
    """beta2 = 0.999 at a constant gradient: to nearest, the codes stand still; by chance they go where the
    formula goes, on average (16384 elements; a step of 1/8 to 1/16 has a deviation below 1/16 of the value)."""
    n = 1 << 14
    moved = {}
    for random in (False, True):
        rng = torch.tensor([99, 0], dtype=torch.int64, device=DEV) if random else None
        p = [torch.zeros(n, device=DEV)]
        gr = [torch.full((n,), 0.5, device=DEV)]
        gr[0][::128] = 1.0                                  # keeps the scales
        st = g.adamw_init(p, bits=8)
        st.v.copy_(torch.full((n,), 224.0, device=DEV).to(torch.float8_e4m3fn))
        st.v.view(-1)[::128] = torch.full((n // 128,), 448.0, device=DEV).to(torch.float8_e4m3fn)
        st.v_scale.fill_(1.0 / 448.0)                       # sqrt(v) = 0.5 and 1
        gr[0][torch.arange(n, device=DEV) % 128 != 0] = 0.0
        for t in range(100):
            g.adamw_step(p, gr, st, lr=0.0, step=1000 + t, betas=(0.9, 0.999), weight_decay=0.0, rng=rng)
            if rng is not None:
                rng[1] += g.adamw_counters(p)
        u = st.v.float() * st.v_scale.repeat_interleave(128)
        moved[random] = float(u[torch.arange(n, device=DEV) % 128 != 0].double().mean())
    say("mean of sqrt(v)", moved)
    want = 0.5 * 0.999 ** 50                                # sqrt of 0.25 * 0.999^100
    assert moved[False] == 0.5
    # 100 steps add at most 100 variances of (1/16 of 0.5) * 0.5 * sqrt(share): below 0.01 an element; / sqrt(16256) * 5
    # and 1/65536 of a step's centre
    assert abs(moved[True] - want) < 5 * 0.1 / 16256 ** 0.5 + 1e-3


def test_bf16_params_move_by_chance():
    n = 1 << 15
    p = [torch.ones(n, dtype=torch.bfloat16, device=DEV)]
    gr = [torch.ones(n, dtype=torch.bfloat16, device=DEV)]
    st = g.adamw_init(p, bits=32)
    rng = torch.tensor([3, 1 << 40], dtype=torch.int64, device=DEV)
    g.adamw_step(p, gr, st, lr=2.0 ** -11, step=1, weight_decay=0.0, rng=rng)
    # 1 - 2^-11 lies 1/8 of a step of 2^-8 below 1
    share = float((p[0].float() == 1.0 - 2.0 ** -8).double().mean())
    assert abs(share - 0.125) < 5 * (0.125 * 0.875 / n) ** 0.5 and bool(((p[0] == 1) | (p[0] == 1 - 2.0 ** -8)).all())


def test_replayed_graph_takes_new_values():
    run = Run([3000, 40], torch.bfloat16, torch.bfloat16, 8, False,
              rng=torch.tensor([1, 2], dtype=torch.int64, device=DEV))
    other = Run([3000, 40], torch.bfloat16, torch.bfloat16, 8, False, rng=run.rng)
    sched = torch.tensor(g.adamw_schedule(1e-3, 1, HYPER["betas"]), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.adamw_step(other.params, other.grads, other.state, schedule=sched, rng=run.rng, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.adamw_step(run.params, run.grads, run.state, schedule=sched, rng=run.rng, **HYPER)
    for t in (1, 2, 3):
        sched.copy_(torch.tensor(g.adamw_schedule(1e-3 * t, t, HYPER["betas"])))
        run.rng[1] += g.adamw_counters(run.params)
        for gr in run.grads:
            gr.copy_(0.01 * torch.randn(gr.shape, device=DEV))
        want = run.expected(schedule=sched.cpu().numpy())
        graph.replay()
        torch.cuda.synchronize()
        run.check(want)


def test_after_the_layers_backward():
    """Route, forward, backward and a step on both weights: the step is the oracle's for the layer's gradients."""
    torch.manual_seed(0)
    T, H, I, E, k = 48, 64, 32, 4, 2
    x = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T, E, device=DEV)
    w13 = (0.1 * torch.randn(E, 2 * I, H, device=DEV)).to(torch.bfloat16)
    w2 = (0.1 * torch.randn(E, H, I, device=DEV)).to(torch.bfloat16)
    run = Run([w13.numel(), w2.numel()], torch.bfloat16, torch.bfloat16, 32, True)
    run.params = [w13, w2]
    run.state = g.adamw_init(run.params, bits=32, master=True)
    for t in (1, 2):
        out, aux = g.forward(x, logits, w13, w2, k, return_aux=True)
        gr = g.backward(x, w13, w2, out, aux.topk_weights, aux.offsets, aux.sorted_rows, aux.row_pos,
                        grad_dtype=torch.bfloat16)
        run.grads = [gr.dw13, gr.dw2]
        flat = Run.expected.__get__(_Flat(run))(step=t)
        run.step(step=t)
        assert same(np32(w13).reshape(-1), flat["p"][0]) and same(np32(w2).reshape(-1), flat["p"][1])
        assert same(np32(run.state.master), flat["master"])


class _Flat:
    """A run's tensors without their shapes, for the oracle."""

    def __init__(self, run):
        self.__dict__.update(run.__dict__)
        self.params = [p.reshape(-1) for p in run.params]
        self.grads = [p.reshape(-1) for p in run.grads]


def test_refusals():
    f = lambda n, dt=torch.float32: torch.zeros(n, dtype=dt, device=DEV)
    st = g.adamw_init([f(8)])
    ok = dict(lr=1e-3, step=1)
    with pytest.raises(ValueError):
        g.adamw_step([f(8)], [], st, **ok)
    with pytest.raises(ValueError):
        g.adamw_step([f(8)], [f(9)], st, **ok)
    with pytest.raises(ValueError):
        g.adamw_step([f(8), f(8, torch.bfloat16)], [f(8), f(8)], st, **ok)
    with pytest.raises(ValueError):
        g.adamw_step([f(8).cpu()], [f(8).cpu()], st, **ok)
    with pytest.raises(ValueError):
        g.adamw_step([f(200)], [f(200)], st, **ok)
    with pytest.raises(ValueError):
        g.adamw_step([f(16)[::2]], [f(8)], st, **ok)
    with pytest.raises(RuntimeError):
        g.adamw_step([f(8)], [f(8)], g.adamw_init([f(8)], master=True), **ok)
    with pytest.raises(RuntimeError):
        g.adamw_step([f(9)[1:]], [f(8)], st, **ok)      # not 16-byte aligned
    for bad in (dict(lr=-1.0), dict(step=0), dict(eps=0.0), dict(betas=(1.0, 0.9)), dict(weight_decay=float("nan"))):
        with pytest.raises(RuntimeError):
            g.adamw_step([f(8)], [f(8)], st, **dict(ok, **bad))
    with pytest.raises(ValueError):
        g.adamw_init([f(8)], bits=4)
