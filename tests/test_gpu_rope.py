"""GPU parity of la2_qk_norm_rope and its gradients with the float64 oracle.

Tolerances, relative Frobenius. An output rounds once: bf16 2^-8, fp32 2^-24. In fp32
a row's sum of d <= 256 squares is off by at most 2^-24 * 256 / 2 relative, halved by the
root, and the angle's cosine by 2^-22 (a fraction of a turn kept to 2^-25, times 2 pi):
1e-5 covers both. dw sums up to a few thousand rows in fp32 before fp64: sums of
random signs, 1e-5 of the norm again, and one rounding.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 2.0 ** -8 + 1e-5}


@pytest.fixture(scope="module")
def la2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_la2_b200 import build

    build.build()
    from linear_attention_la2_b200 import la2 as lib

    return lib


CASES = [
    # dtype, B, N, H, Hkv, d, rot, sections, far, weights
    ("bf16", 2, 100, 4, 2, 128, 128, (64,), 0, True),
    ("bf16", 1, 1, 1, 1, 64, 64, (32,), 0, True),
    ("bf16", 64, 1, 8, 2, 128, 128, (64,), 1 << 20, True),
    ("bf16", 1, 333, 3, 3, 64, 32, (16,), 1 << 30, False),
    ("bf16", 2, 77, 2, 1, 128, 128, (24, 20, 20), 0, True),
    ("bf16", 1, 50, 2, 2, 48, 48, (24,), 100, True),       # 6 pieces a row
    ("bf16", 1, 50, 2, 2, 100, 50, (25,), 100, True),      # rows of no whole pieces
    ("bf16", 1, 9, 5, 1, 256, 256, (60, 34, 34), 5, True),
    ("bf16", 1, 9, 5, 1, 250, 250, (125,), 5, True),
    ("f32", 2, 65, 4, 2, 128, 128, (64,), 1 << 20, True),
    ("f32", 1, 40, 2, 2, 64, 40, (5, 10, 5), 9, True),
    ("f32", 2, 33, 3, 1, 17, 10, (5,), 0, True),
    ("f32", 1, 5, 2, 2, 1, 0, (0,), 0, True),
    ("f32", 1, 20, 2, 2, 32, 0, (0,), 0, False),           # norm alone
    ("f32", 3, 4099, 2, 1, 64, 64, (32,), 0, True),
    ("f32", 1, 70, 2, 2, 200, 180, (30, 30, 20, 10), 50, True),
    ("f32", 1, 30, 2, 0, 64, 64, (32,), 0, True),
    ("f32", 1, 30, 0, 2, 64, 64, (32,), 0, True),
]


def make(case):
    dt, B, N, H, Hkv, d, rot, sections, far, weights = case
    g = torch.Generator().manual_seed(B + 3 * N + d)
    proj = torch.randn(B, N, H + 2 * Hkv + 1, d, generator=g).to(DT[dt])
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(DT[dt]) if weights else None for _ in range(2)]
    pos = torch.randint(0, far + N + 1, (len(sections), B, N), generator=g).to(torch.int32)
    dy = [torch.randn(B, h, N, d, generator=g).to(DT[dt]) for h in (H, Hkv)]
    return proj, w, pos, dy


def num(t):
    return None if t is None else t.double().numpy()


def close(got, want, dt):
    return want.size == 0 or oracle.relative_frobenius(got.double().cpu().numpy(), want) <= TOL[dt]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(la2, case):
    dt, B, N, H, Hkv, d, rot, sections, far, weights = case
    proj, w, pos, dy = make(case)
    dev = proj.cuda()
    q, k = dev[:, :, :H], dev[:, :, H:H + Hkv]
    wc = [None if x is None else x.cuda() for x in w]
    kw = dict(base=1000.0, rot=rot, sections=sections, eps=1e-5, q_scale=0.25, k_scale=1.5)
    outs = [torch.full((B * h * N * d + 64,), 3.5, dtype=DT[dt], device="cuda") for h in (H, Hkv)]
    views = [o[:B * h * N * d].view(B, h, N, d) for o, h in zip(outs, (H, Hkv))]
    la2.qk_norm_rope(q, k, *wc, pos.cuda(), outs=tuple(views), **kw)
    la2.check()
    args = (pos.numpy(), 1000.0, rot, sections, 1e-5)
    for got, x, weight, scale in ((views[0], q, w[0], 0.25), (views[1], k, w[1], 1.5)):
        want = oracle.qk_norm_rope(x.double().cpu().numpy(), num(weight), *args, scale)
        assert close(got, want, dt)
    for o, v in zip(outs, views):
        assert torch.all(o[v.numel():] == 3.5)
    got = la2.qk_norm_rope_backward(dy[0].cuda(), dy[1].cuda(), q, k, *wc, pos.cuda(), **kw)
    again = la2.qk_norm_rope_backward(dy[0].cuda(), dy[1].cuda(), q, k, *wc, pos.cuda(), **kw)
    la2.check()
    for i, (x, weight, scale) in enumerate(((q, w[0], 0.25), (k, w[1], 1.5))):
        dx, dw = oracle.qk_norm_rope_backward(num(dy[i]), x.double().cpu().numpy(), num(weight), *args, scale)
        # with one value a row the norm leaves nothing but the sign: dx is 0 up to eps
        if d > 1:
            assert close(got[i], dx, dt)
        if weights:
            assert close(got[2 + i], dw, dt)
        else:
            assert got[2 + i] is None
    for a, b in zip(got, again):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(dev.cpu(), proj)


def test_unaligned_and_transposed_inputs(la2):
    """Other strides and alignments take other loads and give the same bits."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(2, 30, 4, 128, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(128, generator=g).to(torch.bfloat16).cuda()
    a, b = la2.qk_norm_rope(x[:, :, :2], x[:, :, 2:], w, w)
    heads_first = x.transpose(1, 2).contiguous().transpose(1, 2)
    c, d = la2.qk_norm_rope(heads_first[:, :, :2], heads_first[:, :, 2:], w, w)
    assert torch.equal(a, c) and torch.equal(b, d)
    odd = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
    odd.copy_(x)
    e, f = la2.qk_norm_rope(odd[:, :, :2], odd[:, :, 2:], w, w)
    # a warp a row instead of half a warp: sums in another order, at most one rounding apart
    assert oracle.relative_frobenius(e.double().cpu().numpy(), a.double().cpu().numpy()) <= 2.0 ** -8
    assert oracle.relative_frobenius(f.double().cpu().numpy(), b.double().cpu().numpy()) <= 2.0 ** -8
    one = x[:, :1].expand(2, 30, 4, 128)  # one token's row for all positions
    e, _ = la2.qk_norm_rope(one[:, :, :2], one[:, :, 2:], w, w)
    f, _ = la2.qk_norm_rope(one[:, :, :2].contiguous(), one[:, :, 2:].contiguous(), w, w)
    assert torch.equal(e, f)


def test_zero_rows_and_default_positions(la2):
    x = torch.zeros(1, 70, 2, 64, device="cuda")
    q, k = la2.qk_norm_rope(x, x, eps=1e-6)
    assert not q.any() and not k.any()
    y = torch.randn(2, 70, 2, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    pos = torch.arange(70, dtype=torch.int32, device="cuda").expand(2, 70).contiguous()
    a, b = la2.qk_norm_rope(y, y), la2.qk_norm_rope(y, y, positions=pos)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_same_bits_on_another_stream_and_from_a_graph(la2):
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(2, 300, 6, 128, device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randn(128, device="cuda", generator=g).to(torch.bfloat16)
    dy = torch.randn(2, 3, 300, 128, device="cuda", generator=g).to(torch.bfloat16)

    def calls(stream=None):
        q, k = x[:, :, :3], x[:, :, 3:]
        return la2.qk_norm_rope(q, k, w, w, stream=stream) + la2.qk_norm_rope_backward(dy, dy, q, k, w, w, stream=stream)

    ref = calls()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = calls(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    x.copy_(x.flip(1))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(calls(), got))
    la2.check()


def test_empty(la2):
    x = torch.zeros(2, 0, 3, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    q, k = la2.qk_norm_rope(x, x, w, w)
    assert q.shape == (2, 3, 0, 64) and k.shape == (2, 3, 0, 64)
    dq, dk, dwq, dwk = la2.qk_norm_rope_backward(q, k, x, x, w, w)
    assert dq.shape == x.shape and not dwq.any() and not dwk.any()
    la2.check()
