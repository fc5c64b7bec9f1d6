"""GPU parity of the gated form (la2_forward_gated, la2_backward_gated) and of its
inference calls (la2_kv_state_gated, la2_decode_step_gated) with the float64 oracle.

Tolerances, relative Frobenius. fp32: 1e-5, the plain op's (sums of at most 128
products and a few hundred rows, each 2^-24 off per addition at random signs). bf16:
an output rounding is at most 2^-8; on the tensor cores the scores, the scaled keys
and the copy of the state are rounded to bf16 as well, four roundings that add up at
random: 1e-2, the plain op's bound. States are fp32 sums of exact bf16 products: 1e-5.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 1e-2}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def la2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from linear_attention_la2_b200 import build

    build.build()
    from linear_attention_la2_b200 import la2 as lib

    lib.la2_set_chunk_len(0)
    yield lib
    lib.la2_set_chunk_len(0)


@pytest.fixture()
def chunk(la2):
    def set_to(n):
        assert la2.la2_set_chunk_len(n) == la2.LA2_OK

    yield set_to
    la2.la2_set_chunk_len(0)


def rel(x, ref):
    return oracle.relative_frobenius(x.detach().float().cpu().numpy(), ref)


def make(dt, B, H, N, d, dv, seed, kind="soft"):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(B, H, N, w, generator=g) / d ** 0.5 for w in (d, d, dv, dv))
    gate = torch.nn.functional.logsigmoid(torch.randn(B, H, N, generator=g) + 2.0)
    if kind == "weak":
        gate = gate * 0.01
    elif kind == "strong":
        gate = gate * 20.0
    elif kind == "restarts":
        gate = gate.masked_fill(torch.rand(B, 1, N, generator=g) < 0.05, -torch.inf)
    elif kind == "closed":
        gate = torch.full_like(gate, -torch.inf)
    elif kind == "open":
        gate = torch.zeros_like(gate)
    elif kind == "lowest":
        gate = gate.masked_fill(torch.rand(B, H, N, generator=g) < 0.2, torch.finfo(DT[dt]).min)
    return {n: t.to(DT[dt]) for n, t in zip(("q", "k", "v", "gate", "do"), (q, k, v, gate, do))}


def double(ins):
    return {n: t.double().numpy() for n, t in ins.items()}


def behind(shape, dtype):
    """A tensor with a margin behind it that must stay as it is."""
    n = int(np.prod(shape))
    buf = torch.full((n + 256,), 7.25, dtype=dtype, device="cuda")
    return buf, buf[:n].view(shape)


CASES = [
    # dtype, B, H, N, d, dv, chunk length (0: the library's), gates
    ("f32", 1, 1, 1, 64, 64, 0, "soft"),
    ("f32", 1, 2, 2, 1, 1, 0, "soft"),
    ("f32", 2, 3, 63, 17, 33, 0, "restarts"),
    ("f32", 1, 2, 65, 128, 128, 0, "strong"),
    ("f32", 2, 3, 777, 48, 80, 0, "soft"),
    ("f32", 1, 2, 640, 64, 32, 64, "weak"),
    ("f32", 1, 1, 300, 16, 24, 128, "closed"),
    ("f32", 1, 2, 513, 64, 64, 0, "open"),
    ("f32", 1, 2, 200, 32, 32, 64, "lowest"),
    ("bf16", 1, 2, 1, 64, 64, 0, "soft"),
    ("bf16", 2, 2, 1000, 64, 64, 128, "restarts"),
    ("bf16", 1, 3, 650, 128, 64, 0, "soft"),
    ("bf16", 1, 2, 1, 128, 128, 0, "soft"),
    ("bf16", 1, 1, 2, 128, 128, 0, "soft"),
    ("bf16", 1, 2, 63, 128, 128, 0, "restarts"),
    ("bf16", 2, 2, 64, 128, 128, 0, "soft"),
    ("bf16", 1, 3, 65, 128, 128, 0, "strong"),
    ("bf16", 1, 2, 130, 128, 128, 64, "soft"),
    ("bf16", 2, 2, 1537, 128, 128, 0, "soft"),
    ("bf16", 1, 2, 2100, 128, 128, 512, "restarts"),
    ("bf16", 1, 1, 3001, 128, 128, 256, "weak"),
    ("bf16", 1, 2, 700, 128, 128, 0, "closed"),
    ("bf16", 1, 2, 900, 128, 128, 0, "open"),
    ("bf16", 1, 2, 500, 128, 128, 128, "lowest"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(la2, chunk, case):
    dt, B, H, N, d, dv, length, kind = case
    ins = make(dt, B, H, N, d, dv, N + d + H, kind)
    chunk(length)
    dev = {n: t.cuda() for n, t in ins.items()}
    keep = {n: t.clone() for n, t in dev.items()}
    buf, o = behind((B, H, N, dv), DT[dt])
    la2.forward_gated(dev["q"], dev["k"], dev["v"], dev["gate"], out=o)
    la2.check()
    outs = [behind(dev[n].shape, DT[dt]) for n in ("q", "k", "v", "gate")]
    la2.backward_gated(*(dev[n] for n in ("q", "k", "v", "gate", "do")), outs=tuple(x for _, x in outs))
    la2.check()
    ref = double(ins)
    args = (ref["q"], ref["k"], ref["v"])
    want = oracle.forward_gated(*args, ref["gate"])
    assert rel(o, want) <= TOL[dt]
    grads = oracle.backward_gated(*args, ref["do"], ref["gate"])
    for (_, got), w, name in zip(outs, grads, ("dq", "dk", "dv", "dgate")):
        if not np.any(w):
            assert not got.float().any(), name
        else:
            assert rel(got, w) <= TOL[dt], name
    # every row on its own at the edges of blocks and chunks
    for r in sorted({x for e in range(0, N, length or 64) for x in (max(0, e - 1), e)} | {N - 1}):
        assert rel(o[:, :, r], want[:, :, r]) <= 4 * TOL[dt]
    for b, x in [(buf, o)] + outs:
        assert torch.all(b[x.numel():] == 7.25)
    for n in dev:
        assert torch.equal(dev[n], keep[n])


def test_gate_gradient_by_differences(la2):
    """dgate against differences of the kernel's own forward in fp32. With a loss of
    about 1, a step of 2^-7 and third derivatives of the same size, central
    differences are 2^-14 / 6 = 1e-5 off and rounding adds 2^-24 * 2^7 = 8e-6 times
    sqrt(terms): 1e-3 of the largest entry is allowed."""
    ins = {n: t.cuda() for n, t in make("f32", 1, 1, 40, 8, 8, 3).items()}
    q, k, v, gate, do = (ins[n] for n in ("q", "k", "v", "gate", "do"))
    dgate = la2.backward_gated(q, k, v, gate, do)[3]
    num = torch.zeros_like(gate)
    for t in range(40):
        e = torch.zeros_like(gate)
        e[..., t] = 2.0 ** -7
        f = [(la2.forward_gated(q, k, v, gate + s * e).double() * do.double()).sum() for s in (1, -1)]
        num[..., t] = ((f[0] - f[1]) / 2.0 ** -6).float()
    assert float((num - dgate).abs().max()) <= 1e-3 * float(dgate.abs().max())


def test_open_gates_are_the_plain_op(la2):
    ins = {n: t.cuda() for n, t in make("bf16", 2, 2, 1500, 128, 128, 5, "open").items()}
    o = la2.forward_gated(ins["q"], ins["k"], ins["v"], ins["gate"])
    p = la2.forward(ins["q"], ins["k"], ins["v"])
    assert rel(o, p.double().cpu().numpy()) <= 1e-2


def test_restart_hides_what_was_before(la2):
    """Values before a restart, of any finite size, leave what follows bit for bit;
    the gate of the first token decides nothing."""
    for dt, d in (("f32", 32), ("bf16", 128)):
        ins = {n: t.cuda() for n, t in make(dt, 1, 2, 300, d, d, 9).items()}
        ins["gate"][..., 130] = -torch.inf
        a = la2.forward_gated(ins["q"], ins["k"], ins["v"], ins["gate"])
        k2, g2 = ins["k"].clone(), ins["gate"].clone()
        k2[:, :, :130] = 3.0
        b = la2.forward_gated(ins["q"], k2, ins["v"], g2)
        g2[..., 0] = -torch.inf
        c = la2.forward_gated(ins["q"], k2, ins["v"], g2)
        assert torch.equal(a[:, :, 130:], b[:, :, 130:])
        assert torch.equal(b, c)


def test_nan_stays_in_its_sequence(la2):
    for dt, d in (("f32", 32), ("bf16", 128)):
        ins = {n: t.cuda() for n, t in make(dt, 2, 2, 200, d, d, 11).items()}
        ref = la2.forward_gated(ins["q"], ins["k"], ins["v"], ins["gate"])
        ins["gate"][1, 0, 100] = torch.nan
        o = la2.forward_gated(ins["q"], ins["k"], ins["v"], ins["gate"])
        assert torch.isnan(o[1, 0, 100:]).all()
        assert torch.equal(o[1, 0, :64], ref[1, 0, :64])
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1, 1], ref[1, 1])


@pytest.mark.parametrize("dt,d,N", [("f32", 40, 600), ("bf16", 128, 1300)])
def test_same_bits_on_another_stream_and_from_a_graph(la2, dt, d, N):
    ins = {n: t.cuda() for n, t in make(dt, 2, 3, N, d, d, 17).items()}
    args = [ins[n] for n in ("q", "k", "v", "gate")]
    o, grads = la2.forward_gated(*args), la2.backward_gated(*args, ins["do"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, grads2 = la2.forward_gated(*args, stream=s), la2.backward_gated(*args, ins["do"], stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(grads, grads2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, grads3 = la2.forward_gated(*args), la2.backward_gated(*args, ins["do"])
    new = {n: t.cuda() for n, t in make(dt, 2, 3, N, d, d, 18).items()}
    for n in ins:
        ins[n].copy_(new[n])
    graph.replay()
    torch.cuda.synchronize()
    la2.check()
    o, grads = la2.forward_gated(*args), la2.backward_gated(*args, ins["do"])
    assert torch.equal(o, o3) and all(torch.equal(a, b) for a, b in zip(grads, grads3))


def test_empty(la2):
    for B, H, N in ((0, 2, 5), (2, 0, 5), (2, 2, 0)):
        x = torch.zeros(B, H, N, 64, device="cuda")
        g = torch.zeros(B, H, N, device="cuda")
        assert la2.forward_gated(x, x, x, g).shape == x.shape
        assert [t.shape for t in la2.backward_gated(x, x, x, g, x)] == [x.shape] * 3 + [g.shape]
        s = torch.ones(B, H, 64, 64, device="cuda")
        la2.kv_state_gated(x, x, g, s)
        assert torch.all(s == 1)
    la2.check()


STATES = [
    # dtype, B, H, N, d, dv, chunk length, gates
    ("f32", 2, 2, 300, 30, 20, 0, "soft"),
    ("f32", 1, 3, 1, 64, 64, 0, "soft"),
    ("f32", 2, 1, 129, 128, 128, 64, "restarts"),
    ("bf16", 2, 2, 700, 64, 128, 128, "soft"),
    ("bf16", 3, 2, 1001, 128, 128, 0, "soft"),
    ("bf16", 1, 2, 2000, 128, 128, 256, "restarts"),
    ("bf16", 1, 2, 64, 128, 128, 0, "weak"),
    ("bf16", 1, 2, 5, 128, 128, 0, "strong"),
]


@pytest.mark.parametrize("case", STATES, ids=lambda c: "-".join(map(str, c)))
def test_prefill_state_in_slots(la2, chunk, case):
    dt, B, H, N, d, dv, length, kind = case
    ins = make(dt, B, H, N, d, dv, 3 * N + d, kind)
    chunk(length)
    pool = torch.randn(B + 3, H, d, dv, generator=torch.Generator().manual_seed(N)).cuda()
    before = pool.clone()
    slots = torch.arange(B + 2, 2, -1, dtype=torch.int32, device="cuda")
    la2.kv_state_gated(*(ins[n].cuda() for n in ("k", "v", "gate")), pool, slots=slots)
    la2.check()
    ref = double(ins)
    want = oracle.kv_state_gated(ref["k"], ref["v"], ref["gate"], before[slots.long()].double().cpu().numpy())
    assert rel(pool[slots.long()], want) <= 1e-5
    assert torch.equal(pool[:3], before[:3])


@pytest.mark.parametrize("dt,d,dv", [("bf16", 128, 128), ("f32", 128, 128), ("f32", 33, 50), ("f32", 1, 4),
                                     ("bf16", 96, 30), ("bf16", 200, 64), ("f32", 160, 36)])
def test_decode_in_slots(la2, dt, d, dv):
    B, H, S = 5, 3, 8
    ins = make(dt, B, H, 1, d, dv, d + dv)
    ins["gate"][1, 0] = -torch.inf
    x = {n: t[:, :, 0].contiguous().cuda() for n, t in ins.items()}
    pool = torch.randn(S, H, d, dv, generator=torch.Generator().manual_seed(d)).cuda()
    before = pool.clone()
    slots = torch.tensor([6, 0, -1, 3, 7], dtype=torch.int32, device="cuda")
    out = torch.full((B, H, dv), 9.0, dtype=DT[dt], device="cuda")
    la2.decode_step_gated(x["q"], x["k"], x["v"], x["gate"], pool, slots=slots, out=out)
    la2.check()
    on = slots >= 0
    at = slots[on].long()
    g = x["gate"][on].double().exp()[..., None, None]
    want = before[at].double() * g + x["k"][on].double()[..., :, None] * x["v"][on].double()[..., None, :]
    assert rel(pool[at], want.cpu().numpy()) <= 1e-6
    o = (x["q"][on].double()[..., None, :] @ want)[..., 0, :]
    assert rel(out[on], o.cpu().numpy()) <= (2.0 ** -8 if dt == "bf16" else 1e-5)
    assert torch.all(out[2] == 9.0)
    idle = [s for s in range(S) if s not in slots.tolist()]
    assert torch.equal(pool[idle], before[idle])
    # without slots row b works on slot b
    pool2 = before[:B].clone()
    o2 = la2.decode_step_gated(x["q"], x["k"], x["v"], x["gate"], pool2)
    pool3 = before[:B].clone()
    o3 = la2.decode_step_gated(x["q"], x["k"], x["v"], x["gate"], pool3,
                               slots=torch.arange(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(o2, o3) and torch.equal(pool2, pool3)


@pytest.mark.parametrize("slots", [[1, 1, 2], [0, 3, 1], [0, 1, 1 << 30]])
def test_refused_slots_are_skipped_and_reported(la2, slots):
    """A slot named twice or out of the pool: the later or bad row is skipped, the
    others are carried out, la2_check reports it once."""
    B, H, d, S = 3, 2, 32, 3
    x = {n: t[:, :, 0].contiguous().cuda() for n, t in make("f32", B, H, 1, d, d, 1).items()}
    seq = {n: t.cuda() for n, t in make("f32", B, H, 9, d, d, 2).items()}
    bad = next(b for b in range(B) if slots[b] >= S or slots[b] in slots[:b])
    good = [b for b in range(B) if b != bad]
    idx = torch.tensor(slots, dtype=torch.int32, device="cuda")
    pool = torch.randn(S, H, d, d, device="cuda")
    for call in ("decode", "prefill"):
        p, ref = pool.clone(), pool.clone()
        out = torch.full((B, H, d), 5.0, device="cuda")
        sub = idx[good].contiguous()
        if call == "decode":
            la2.decode_step_gated(x["q"], x["k"], x["v"], x["gate"], p, slots=idx, out=out)
        else:
            la2.kv_state_gated(seq["k"], seq["v"], seq["gate"], p, slots=idx)
        assert la2.la2_check(la2._stream_handle(None)) == la2.LA2_ERR_INVALID_ARG
        assert la2.la2_check(la2._stream_handle(None)) == la2.LA2_OK
        pick = {n: t[good].contiguous() for n, t in (x if call == "decode" else seq).items()}
        if call == "decode":
            o = la2.decode_step_gated(pick["q"], pick["k"], pick["v"], pick["gate"], ref, slots=sub)
            assert torch.equal(out[good], o) and torch.all(out[bad] == 5.0)
        else:
            la2.kv_state_gated(pick["k"], pick["v"], pick["gate"], ref, slots=sub)
        assert torch.equal(p, ref)
        la2.check()


def test_far_slots(la2):
    """Slots whose element offsets pass 32 bits: 70000 slots of 64 K values (17 GB)."""
    S, d = 70000, 256
    pool = torch.zeros(S, 1, d, d, device="cuda")
    slots = torch.tensor([S - 1, 32768], dtype=torch.int32, device="cuda")
    x = {n: t[:, :, 0].contiguous().cuda() for n, t in make("f32", 2, 1, 1, d, d, 4).items()}
    la2.decode_step_gated(x["q"], x["k"], x["v"], x["gate"], pool, slots=slots)
    la2.state_copy(pool, slots, torch.tensor([S - 2, 65536], dtype=torch.int32, device="cuda"))
    la2.check()
    want = x["k"][..., :, None] * x["v"][..., None, :]
    for at, b in ((S - 1, 0), (32768, 1), (S - 2, 0), (65536, 1)):
        assert torch.equal(pool[at], want[b])
    assert int((pool.flatten(1).abs().amax(1) > 0).sum()) == 4


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 48)])
def test_layer_in_training_and_serving(la2, dt, d):
    """The calls together: projections -> norm and rotation -> gated forward; and the
    same tokens as a prefill into slots, single steps, a fork of one sequence and a
    compaction of the pool, each step giving the forward's rows."""
    B, N, H, P = 3, 90, 4, 70
    g = torch.Generator().manual_seed(d)
    proj = torch.randn(B, N, 3 * H, d, generator=g).to(DT[dt]).cuda()
    gate = torch.nn.functional.logsigmoid(torch.randn(B, H, N, generator=g) + 2).to(DT[dt]).cuda()
    wq, wk = (torch.randn(d, generator=g).to(DT[dt]).cuda() for _ in range(2))
    v = proj[:, :, 2 * H:].transpose(1, 2).contiguous()
    q, k = la2.qk_norm_rope(proj[:, :, :H], proj[:, :, H:2 * H], wq, wk, q_scale=d ** -0.5, k_scale=d ** -0.5)
    o = la2.forward_gated(q, k, v, gate)
    pool = torch.full((8, H, d, d), 3.0, device="cuda")
    slots = torch.tensor([5, 1, 7], dtype=torch.int32, device="cuda")
    la2.state_copy(pool, torch.full_like(slots, -1), slots)
    la2.kv_state_gated(k[:, :, :P].contiguous(), v[:, :, :P].contiguous(), gate[:, :, :P].contiguous(), pool,
                       slots=slots)
    pos = torch.empty(B, 1, dtype=torch.int32, device="cuda")
    scale = float(o.float().norm()) / o.numel() ** 0.5
    # two outputs of one value: twice the bound of either
    tol = 2 * TOL[dt]
    for t in range(P, N):
        if t == P + 4:  # sequence 1 continues in slot 2 as well; both give the same rows
            la2.state_copy(pool, slots[1:2].contiguous(), torch.tensor([2], dtype=torch.int32, device="cuda"))
            slots[1] = 2
        if t == P + 9:
            live = torch.zeros(8, dtype=torch.int32, device="cuda")
            live[slots.long()] = 1
            moved = la2.state_compact(pool, live)
            slots = moved[slots.long()].contiguous()
            assert sorted(slots.tolist()) == [0, 1, 2]
        pos.fill_(t)
        qt, kt = la2.qk_norm_rope(proj[:, t:t + 1, :H], proj[:, t:t + 1, H:2 * H], wq, wk, pos,
                                  q_scale=d ** -0.5, k_scale=d ** -0.5)
        assert torch.equal(qt, q[:, :, t:t + 1]) and torch.equal(kt, k[:, :, t:t + 1])
        got = la2.decode_step_gated(qt[:, :, 0], kt[:, :, 0], v[:, :, t].contiguous(), gate[:, :, t].contiguous(),
                                    pool, slots=slots)
        err = float((got.float() - o[:, :, t].float()).norm()) / got.numel() ** 0.5
        assert err <= tol * max(scale, float(got.float().norm()) / got.numel() ** 0.5)
    la2.check()
