"""A step raises the version counters of what it writes, as torch's own in-place operations do."""
import pytest
import torch

import grouped_gemm_histogram_amd as g

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def test_autograd_notices_a_step():
    """A backward through values that were saved before the step and overwritten by it is refused, not wrong."""
    w = torch.nn.Parameter(torch.randn(64, device=DEV))
    state = g.adamw_init([w])
    x = torch.randn(64, device=DEV, requires_grad=True)
    loss = (w * x).sum()
    g.adamw_step([w], [torch.ones_like(w)], state, lr=0.1, step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.parametrize("bits", [8, 32])
def test_all_that_is_written_counts(bits):
    params = [torch.nn.Parameter(torch.randn(n, device=DEV).to(torch.bfloat16)) for n in (40, 0, 300)]
    grads = [torch.randn_like(p) for p in params]
    state = g.adamw_init(params, bits=bits, master=True)
    written = params + [t for t in vars(state).values() if t is not None]
    before = [t._version for t in written]
    g.adamw_step(params, grads, state, lr=0.1, step=1)
    assert all(t._version > b for t, b in zip(written, before))
    still = [t._version for t in grads]
    with torch.no_grad():
        g.adamw_step(params, grads, state, lr=0.1, step=2)
    assert [t._version for t in grads] == still and all(p.requires_grad and p.is_leaf for p in params)


def test_tensors_without_a_counter():
    """Tensors made in inference mode have none."""
    with torch.inference_mode():
        p = [torch.ones(32, device=DEV)]
        state = g.adamw_init(p)
    g.adamw_step(p, [torch.ones(32, device=DEV)], state, lr=0.1, step=1, weight_decay=0.0)
    assert bool((p[0] < 0.95).all())
