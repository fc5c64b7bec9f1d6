"""The q/k norm without an epsilon, which the calls allow: rows that are no zeros have
finite gradients whatever the rest of their warp holds. Token and head counts leave groups
of lanes without a row. Tolerances as in test_gpu_rope.
"""

import pytest
import torch

import oracle
from test_gpu_rope import DT, close, la2, num  # noqa: F401 (la2: a fixture)

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, B, N, H, Hkv, d, rot
    ("bf16", 1, 100, 4, 4, 128, 128),   # few tokens: most head places of a CTA are idle
    ("bf16", 1, 7109, 2, 1, 128, 128),  # 16 tokens a tile, the last tile is not full
    ("bf16", 3, 1, 3, 1, 64, 64),
    ("bf16", 1, 77, 3, 2, 128, 50),     # pairs that meet in shared memory
    ("bf16", 1, 33, 3, 1, 90, 90),      # a warp a row
    ("f32", 1, 100, 4, 4, 128, 128),
    ("f32", 2, 41, 5, 3, 64, 24),
    ("f32", 1, 9, 3, 1, 50, 30),
]


@pytest.mark.parametrize("eps", [0.0, 1e-60])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_no_epsilon(la2, case, eps):  # noqa: F811
    dt, B, N, H, Hkv, d, rot = case
    g = torch.Generator().manual_seed(N + d)
    x = torch.randn(B, N, H + Hkv, d, generator=g).to(DT[dt])
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(DT[dt]) for _ in range(2)]
    dy = [torch.randn(B, h, N, d, generator=g).to(DT[dt]) for h in (H, Hkv)]
    dev = x.cuda()
    q, k, wc = dev[:, :, :H], dev[:, :, H:], [t.cuda() for t in w]
    out = la2.qk_norm_rope(q, k, *wc, rot=rot, eps=eps)
    got = la2.qk_norm_rope_backward(dy[0].cuda(), dy[1].cuda(), q, k, *wc, rot=rot, eps=eps)
    la2.check()
    pos = torch.arange(N).expand(1, B, N).numpy()
    args = (pos, 10000.0, rot, (rot // 2,), eps)
    for i, rows in enumerate((x[:, :, :H], x[:, :, H:])):
        rows = rows.double().numpy()
        assert close(out[i], oracle.qk_norm_rope(rows, num(w[i]), *args, 1.0), dt)
        dx, dw = oracle.qk_norm_rope_backward(num(dy[i]), rows, num(w[i]), *args, 1.0)
        assert close(got[i], dx, dt)
        assert close(got[2 + i], dw, dt)
