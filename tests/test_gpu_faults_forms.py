"""Bounded device-side waits of every tensor-core form, as in test_gpu_faults: a spin limit
below what a load takes is reported at most, what a CTA has in flight lands before it
ends, and the next call gives the bits of the one before the fault.
"""

import pytest
import torch

from linear_attention_la2_b200 import inputs as la2_inputs
from test_gpu_faults import la2  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

FORMS = ["causal64", "causal128", "noncausal", "backward64", "backward128", "decay", "decay_backward", "state"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,H,N", [(1, 4, 4096), (2, 100, 130)])
def test_wait_limit_recovers(la2, form, B, H, N):  # noqa: F811
    ins = la2_inputs.make_custom(B, H, N, 128, 128, "bf16", seed=N, with_grad_out=True)
    q, k, v, do = (ins[n].cuda() for n in ("q", "k", "v", "do"))
    lam = torch.linspace(0.9, 1.0, H, device="cuda")

    def call():
        if form.startswith("causal"):
            return (la2.forward(q, k, v, block=int(form[6:])),)
        if form == "noncausal":
            return (la2.forward(q, k, v, causal=False),)
        if form.startswith("backward"):
            return la2.backward(q, k, v, do, block=int(form[8:]))
        if form == "decay":
            return (la2.forward_decay(q, k, v, lam),)
        if form == "decay_backward":
            return la2.backward_decay(q, k, v, do, lam)
        return (la2.kv_state(k, v),)

    ref = call()
    la2.check()
    assert la2.la2_set_spin_limit(1) == la2.LA2_OK
    try:
        call()
        assert la2.la2_check(la2._stream_handle(None)) in (la2.LA2_OK, la2.LA2_ERR_TIMEOUT)
    finally:
        la2.la2_set_spin_limit(0)
    assert la2.la2_check(la2._stream_handle(None)) == la2.LA2_OK
    again = call()
    la2.check()
    assert all(torch.equal(x, y) for x, y in zip(ref, again))
