"""Bounded device-side waits of the gated kernels: a wait that runs out is reported by
la2_check, what the CTA had in flight lands before it ends, and the next call is as if
nothing had been. The fault is a spin limit below what a load takes, as in test_gpu_faults.
"""

import pytest
import torch

from test_gpu_gated import behind, la2, make  # noqa: F401 (la2: a fixture)

pytestmark = pytest.mark.gpu


# short sequences: all loads are under way when the first wait gives up
@pytest.mark.parametrize("N,H", [(4096, 8), (190, 150), (64, 300), (2100, 40)])
@pytest.mark.parametrize("d", [128, 64])
def test_wait_limit_reports_and_recovers(la2, N, H, d):  # noqa: F811
    ins = {n: t.cuda() for n, t in make("bf16", 1, H, N, d, d, N).items()}
    args = [ins[n] for n in ("q", "k", "v", "gate")]

    def calls(status):
        outs = [behind(t.shape, t.dtype) for t in (ins["v"], *args)]
        pool = torch.zeros(1, H, d, d, device="cuda")
        la2.forward_gated(*args, out=outs[0][1])
        status.append(la2.la2_check(la2._stream_handle(None)))
        la2.backward_gated(*args, ins["do"], outs=tuple(x for _, x in outs[1:]))
        status.append(la2.la2_check(la2._stream_handle(None)))
        la2.kv_state_gated(*args[1:], pool)
        status.append(la2.la2_check(la2._stream_handle(None)))
        for buf, x in outs:
            assert torch.all(buf[x.numel():] == 7.25)
        return [x for _, x in outs] + [pool]

    status = []
    ref = calls(status)
    assert status == [la2.LA2_OK] * 3
    assert la2.la2_set_spin_limit(1) == la2.LA2_OK
    try:
        status = []
        calls(status)
        assert set(status) <= {la2.LA2_OK, la2.LA2_ERR_TIMEOUT}
        if N == 4096:  # (a try of the hardware's outlasts the waits of short pieces)
            assert status[:2] == [la2.LA2_ERR_TIMEOUT] * 2
    finally:
        la2.la2_set_spin_limit(0)
    status = []
    again = calls(status)
    assert status == [la2.LA2_OK] * 3
    assert all(torch.equal(x, y) for x, y in zip(ref, again))
