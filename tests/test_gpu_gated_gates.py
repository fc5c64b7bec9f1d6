"""The gated form where its gates are extreme: heads that forget within a few tokens, long
chunks, many restarts in a block, restarts with growing gates behind them. The reference
is the recurrence in float64 on the GPU, 64 tokens at a time, with restarts as cuts
rather than as large numbers, and with the gates' gradient summed over pairs.
"""

import pytest
import torch

import oracle
from test_gpu_gated import DT, chunk, la2, make  # noqa: F401 (la2, chunk: fixtures)

pytestmark = pytest.mark.gpu

R = 64


def blocks(x):
    """[B,H,N,...] -> float64 [T,B,H,64,...], zeros behind the last token."""
    B, H, N = x.shape[:3]
    T = (N + R - 1) // R
    y = torch.zeros(B, H, T * R, *x.shape[3:], dtype=torch.float64, device=x.device)
    y[:, :, :N] = x
    return y.view(B, H, T, R, *x.shape[3:]).movedim(2, 0)


def whole(parts, N):
    x = torch.stack(parts).movedim(0, 2)
    return x.flatten(2, 3)[:, :, :N]


class Weights:
    """Decays inside a block: pairs, from the state before it, to its end, over all of it."""

    def __init__(self, gate):
        cut = gate == -torch.inf
        c = gate.masked_fill(cut, 0.0).cumsum(-1)
        part = cut.long().cumsum(-1)
        t = torch.arange(R, device=gate.device)
        same = (part[..., :, None] == part[..., None, :]) & (t[:, None] >= t)
        self.pair = torch.where(same, c[..., :, None] - c[..., None, :], -torch.inf).exp()
        self.head = torch.where(part == 0, c, -torch.inf).exp()
        self.tail = self.pair[..., -1, :]
        self.all = self.head[..., -1]


def reference(q, k, v, gate, do, state=None):
    """(o, dq, dk, dv, dgate, state behind the last token) in float64."""
    N = q.shape[2]
    q, k, v, gate, do = (blocks(x) for x in (q, k, v, gate, do))
    w = [Weights(g) for g in gate]
    T = len(w)
    S = torch.zeros(*q.shape[1:3], q.shape[-1], v.shape[-1], dtype=torch.float64, device=q.device)
    if state is not None:
        S = S + state
    before, o, dq, dk, dv, dg = [], [], [], [], [], []
    for t in range(T):
        before.append(S)
        P = (q[t] @ k[t].mT) * w[t].pair
        o.append(P @ v[t] + w[t].head[..., None] * (q[t] @ S))
        S = w[t].all[..., None, None] * S + (k[t] * w[t].tail[..., None]).mT @ v[t]
    U = torch.zeros_like(S)
    upper = torch.ones(R, R, device=q.device, dtype=torch.bool).tril(-1)
    for t in reversed(range(T)):
        A, P = (do[t] @ v[t].mT) * w[t].pair, (q[t] @ k[t].mT) * w[t].pair
        q_far = w[t].head[..., None] * (do[t] @ before[t].mT)
        k_far = w[t].tail[..., None] * (v[t] @ U.mT)
        dq.append(A @ k[t] + q_far)
        dk.append(A.mT @ q[t] + k_far)
        dv.append(P.mT @ do[t] + w[t].tail[..., None] * (k[t] @ U))
        pairs = A * (q[t] @ k[t].mT)
        inside = (pairs.flip(-2).cumsum(-2).flip(-2) * upper).sum(-1)  # i >= t > j of the block
        a, b = (q[t] * q_far).sum(-1), (k[t] * k_far).sum(-1)
        across = w[t].all * (before[t] * U).sum((-1, -2))
        dg.append(inside + a.flip(-1).cumsum(-1).flip(-1) + (b.cumsum(-1) - b) + across[..., None])
        U = w[t].all[..., None, None] * U + (q[t] * w[t].head[..., None]).mT @ do[t]
    back = [whole(x[::-1], N) for x in (dq, dk, dv, dg)]
    back[3][:, :, 0] = 0.0  # nothing comes before the first token
    return whole(o, N), *back, S


def by_head(x, ref):
    """Largest relative Frobenius error of a head."""
    x, ref = x.double().movedim(1, 0).flatten(1), ref.movedim(1, 0).flatten(1)
    return float(((x - ref).norm(dim=1) / ref.norm(dim=1)).max())


def test_reference():
    """The float64 reference against the oracle, token by token (no kernel runs)."""
    ins = make("f32", 1, 2, 150, 6, 5, 1, "restarts")
    args = [ins[n].double() for n in ("q", "k", "v")]
    gate, do = ins["gate"].double(), ins["do"].double()
    got = reference(*args, gate, do)
    n = [t.numpy() for t in args]
    want = (oracle.forward_gated(*n, gate.numpy()), *oracle.backward_gated(*n, do.numpy(), gate.numpy()))
    for x, y in zip(got, want):
        assert oracle.relative_frobenius(x.numpy(), y) <= 1e-12


# ------------------------------------------------- the gradient of the gates, head by head
#
# fp32: a row's dot of q and dq is off by a few 2^-24 of the pairs behind it, and a gate's
# gradient adds up to 512 such rows (a chunk), at random signs: 512^0.5 * 2 * 4 * 2^-24
# = 1.1e-5 of the pairs across it, which is what the gradient of a head that forgets at
# once consists of; 5e-5 is allowed. bf16: a score is rounded alike in both passes (2^-9
# of each pair), the output once (2^-9), states to 2^-17 a row, which over 8192 rows adds
# 8192^0.5 * 2^-17 = 7e-4: 1e-2, the bound of the other gradients.
GATE_TOL = {"f32": 5e-5, "bf16": 1e-2}

FORGETTING = [
    # dtype, N, d, dv, chunk length, restarts
    ("f32", 500, 64, 64, 512, False),
    ("f32", 777, 48, 80, 0, False),
    ("f32", 300, 128, 128, 512, True),
    ("bf16", 500, 128, 128, 512, False),
    ("bf16", 8192, 128, 128, 8192, False),
    ("bf16", 8192, 128, 128, 8192, True),
    ("bf16", 6001, 64, 64, 4096, True),
    ("bf16", 3000, 64, 128, 0, False),
    ("bf16", 2500, 128, 64, 128, True),  # more chunks than add their states up: scanned
]


@pytest.mark.parametrize("case", FORGETTING, ids=lambda c: "-".join(map(str, c)))
def test_gate_gradient_of_each_head(la2, chunk, case):  # noqa: F811
    dt, N, d, dv, length, restarts = case
    g = torch.Generator().manual_seed(N + d)
    level = torch.tensor([-0.001, -0.05, -1.0, -4.0, -8.0, -10.0, -12.0, -20.0])
    H = len(level)
    q, k, v, do = (torch.randn(1, H, N, w, generator=g) / w ** 0.5 for w in (d, d, dv, dv))
    gate = level[:, None] * (0.9 + 0.2 * torch.rand(1, H, N, generator=g))
    if restarts:
        gate = gate.masked_fill(torch.rand(1, 1, N, generator=g) < 0.02, -torch.inf)
    ins = [x.to(DT[dt]).cuda() for x in (q, k, v, gate, do)]
    chunk(length)
    got = la2.backward_gated(*ins)
    la2.check()
    want = reference(*ins)[1:5]
    for x, y, name in zip(got, want, ("dq", "dk", "dv", "dgate")):
        assert by_head(x, y) <= (GATE_TOL[dt] if name == "dgate" else 1e-5 if dt == "f32" else 1e-2), name
    assert not got[3][ins[3] == -torch.inf].any()


@pytest.mark.parametrize("dt,d", [("f32", 64), ("bf16", 128), ("bf16", 64)])
def test_gate_gradient_does_not_cross_a_restart(la2, chunk, dt, d):  # noqa: F811
    """The last document's gradients, of any size, leave those of the gates before it bit
    for bit; two tokens before a restart the gradient is that of one pair."""
    N = 400
    ins = {n: t.cuda() for n, t in make(dt, 1, 2, N, d, d, 5).items()}
    ins["gate"][..., 200] = -torch.inf
    chunk(512)
    a = la2.backward_gated(*(ins[n] for n in ("q", "k", "v", "gate", "do")))[3]
    big = ins["do"].clone()
    big[:, :, 200:] *= 2.0 ** 20
    b = la2.backward_gated(*(ins[n] for n in ("q", "k", "v", "gate")), big)[3]
    la2.check()
    assert torch.equal(a[..., :201], b[..., :201])
    assert not torch.equal(a[..., 201:], b[..., 201:])
    want = reference(*(ins[n] for n in ("q", "k", "v", "gate", "do")))[4]
    few = slice(190, 200)
    assert by_head(a[..., few], want[..., few]) <= (1e-5 if dt == "f32" else 1e-2)


@pytest.mark.parametrize("dt,d,N", [("bf16", 128, 65536)])
def test_one_chunk_of_many_rows(la2, chunk, dt, d, N):  # noqa: F811
    """A sequence that one CTA walks from end to end: 65536^0.5 * 2^-17 = 2e-3 beside the
    roundings above."""
    g = torch.Generator(device="cuda").manual_seed(3)
    level = torch.tensor([-0.0005, -0.02, -1.0, -6.0], device="cuda")
    q, k, v, do = (torch.randn(1, 4, N, d, generator=g, device="cuda") / d ** 0.5 for _ in range(4))
    gate = level[:, None] * (0.5 + torch.rand(1, 4, N, generator=g, device="cuda"))
    ins = [x.to(DT[dt]) for x in (q, k, v, gate, do)]
    chunk(N)
    got = la2.backward_gated(*ins)
    la2.check()
    for x, y in zip(got, reference(*ins)[1:5]):
        assert by_head(x, y) <= 1e-2


# --------------------------------------------------------------------- restarts in a block


@pytest.mark.parametrize("rate", [0.05, 0.3])
@pytest.mark.parametrize("dt,d,length", [("bf16", 128, 64), ("bf16", 128, 256), ("bf16", 64, 0), ("f32", 48, 64)])
def test_state_behind_restarts(la2, chunk, dt, d, length, rate):  # noqa: F811
    """Restarts among the first 40 rows of every block leave the states of what comes
    behind them as exact as those of a block without: 1e-5, the bound of all states."""
    B, H, N = 2, 3, 512
    ins = make(dt, B, H, N, d, d, 8, "weak")
    g = torch.Generator().manual_seed(1)
    cut = (torch.rand(B, H, N, generator=g) < rate) & (torch.arange(N) % 64 < 40)
    ins["gate"] = ins["gate"].masked_fill(cut, -torch.inf)
    dev = [ins[n].cuda() for n in ("q", "k", "v", "gate", "do")]
    chunk(length)
    pool = torch.randn(B, H, d, d, generator=g).cuda()
    want = reference(*dev, state=pool)[5]
    la2.kv_state_gated(*dev[1:4], pool)
    la2.check()
    assert by_head(pool, want) <= 1e-5


@pytest.mark.parametrize("kind", ["soft", "weak", "strong", "restarts"])
@pytest.mark.parametrize("B,H,N,d,dv,length", [(3, 4, 3001, 128, 128, 0), (1, 2, 512, 128, 128, 512),
                                               (1, 3, 777, 64, 64, 0), (2, 2, 300, 64, 128, 128)])
def test_pool_states_are_fp32(la2, chunk, B, H, N, d, dv, length, kind):  # noqa: F811
    """A pool's state from bf16 keys and values holds fp32's digits, not those of a pair of bf16
    values. Its products are exact to 2^-24. A tensor core's sum over 512 rows, the longest
    piece here, adds 32 times, each cut off by at most 2^-23 and 2^-24 on average, of a sum
    that grows like a root: 32 * 2/3 * 2^-24 = 1.3e-6; the smaller parts' sum and the gates'
    exponentials (2^-22) add 2^-22 and 3 * 2^-24: 2e-6 in all, where pairs leave 4.5e-6."""
    ins = make("bf16", B, H, N, d, dv, N, kind)
    dev = [ins[n].cuda() for n in ("q", "k", "v", "gate", "do")]
    chunk(length)
    pool = torch.randn(B, H, d, dv, generator=torch.Generator().manual_seed(7)).cuda()
    want = reference(*dev, state=pool)[5]
    la2.kv_state_gated(*dev[1:4], pool)
    la2.check()
    assert by_head(pool, want) <= 2e-6


@pytest.mark.parametrize("dt,d,length", [("bf16", 128, 0), ("bf16", 64, 64), ("bf16", 128, 128), ("f32", 40, 0),
                                         ("f32", 33, 64)])
@pytest.mark.parametrize("at,n,up", [(0, 70, 0.25), (3, 30, 0.5), (70, 200, 0.5)])
def test_restart_with_growing_gates_drops_what_a_slot_held(la2, chunk, dt, d, length, at, n, up):  # noqa: F811
    """Gates above 0 behind a restart do not bring back what a slot held, be it no number."""
    ins = {x: t.cuda() for x, t in make(dt, 2, 2, n, d, d, d).items()}
    ins["gate"] = torch.full_like(ins["gate"], up)
    ins["gate"][:, :, :at] = -0.5
    ins["gate"][:, :, at] = -torch.inf
    chunk(length)
    worst = torch.full((2, 2, d, d), float("nan"), device="cuda")
    worst[1] = float("inf")
    zero = torch.zeros_like(worst)
    la2.kv_state_gated(ins["k"], ins["v"], ins["gate"], worst)
    la2.kv_state_gated(ins["k"], ins["v"], ins["gate"], zero)
    la2.check()
    assert torch.equal(worst, zero) and bool(torch.isfinite(zero).all())


@pytest.mark.parametrize("dt,d,length", [("bf16", 128, 0), ("bf16", 128, 64), ("bf16", 64, 128), ("f32", 32, 0)])
@pytest.mark.parametrize("at", [10, 63, 130])
def test_restart_with_growing_gates_hides_what_was_before(la2, chunk, dt, d, length, at):  # noqa: F811
    """Values before a restart, of any finite size, leave all outputs and gradients behind
    it bit for bit, however small those are and whatever the gates behind it."""
    N = 200
    ins = {n: t.cuda() for n, t in make(dt, 1, 2, N, d, d, 9).items()}
    ins["gate"] = torch.full_like(ins["gate"], -0.5)
    ins["gate"][..., at] = -torch.inf
    ins["gate"][..., at + 1:at + 60] = 1.0
    chunk(length)
    ins["k"][:, :, at:] *= 2.0 ** -60
    far = {n: ins[n].clone() for n in ("k", "v")}
    far["k"][:, :, :at] *= 2.0 ** 50
    far["v"][:, :, :at] *= 2.0 ** 50
    q, gate, do = ins["q"], ins["gate"], ins["do"]
    a = (la2.forward_gated(q, ins["k"], ins["v"], gate), *la2.backward_gated(q, ins["k"], ins["v"], gate, do))
    b = (la2.forward_gated(q, far["k"], far["v"], gate), *la2.backward_gated(q, far["k"], far["v"], gate, do))
    la2.check()
    for x, y, name in zip(a, b, ("o", "dq", "dk", "dv", "dgate")):
        assert torch.equal(x[:, :, at:], y[:, :, at:]), name
    assert bool(torch.isfinite(a[0].float()).all())


@pytest.mark.parametrize("dt,d,length", [("bf16", 128, 0), ("bf16", 128, 1024), ("bf16", 128, 64), ("bf16", 64, 256),
                                         ("f32", 32, 0), ("f32", 48, 1024)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_no_numbers_end_at_a_restart(la2, chunk, dt, d, length, bad):  # noqa: F811
    """A document whose values are no numbers leaves the others bit for bit, but for the
    64-row blocks in which it begins and ends, and the gates' gradients of the document before it."""
    N, begin, end = 1000, 200, 700  # blocks 3 and 10: rows 192-255 and 640-703
    ins = {n: t.cuda() for n, t in make(dt, 1, 2, N, d, d, 15).items()}
    ins["gate"][..., [begin, end]] = -torch.inf
    chunk(length)

    def calls():
        q, k, v, gate, do = (ins[n] for n in ("q", "k", "v", "gate", "do"))
        pool = torch.full((1, 2, d, d), 2.0, device="cuda")
        la2.kv_state_gated(k, v, gate, pool)
        return (la2.forward_gated(q, k, v, gate), *la2.backward_gated(q, k, v, gate, do), pool)

    a = calls()
    for n in ("q", "k", "v", "do"):
        ins[n][:, :, 300:310] = bad
    b = calls()
    la2.check()
    assert not torch.isfinite(b[0][:, :, 300:310].float()).any()
    for x, y, name in zip(a, b, ("o", "dq", "dk", "dv", "dgate")):
        assert torch.equal(x[:, :, 704:], y[:, :, 704:]), name
        if name != "dgate":
            assert torch.equal(x[:, :, :192], y[:, :, :192]), name
    assert torch.equal(a[5], b[5])


@pytest.mark.parametrize("low", [-105.0, -150.0, -9000.0])
@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 32)])
def test_gates_that_are_zero_in_fp32_are_restarts(la2, dt, d, low):  # noqa: F811
    """A gate below -104 is one of -infinity in every call, growing gates behind it or not:
    large values before it and small ones behind would show the difference."""
    N = 150
    ins = {n: t.cuda() for n, t in make(dt, 1, 2, N, d, d, 4).items()}
    ins["gate"][..., 21:60] = 2.0
    ins["k"][:, :, 20:] *= 2.0 ** -20
    got = []
    for x in (low, -torch.inf):
        gate = ins["gate"].clone()
        gate[..., 20] = x
        args = (ins["q"], ins["k"], ins["v"], gate)
        pool = torch.full((1, 2, d, d), 1e38, device="cuda")
        la2.kv_state_gated(*args[1:], pool)
        one = [t[:, :, 20].contiguous() for t in args]
        step = la2.decode_step_gated(*one, pool)
        got.append((la2.forward_gated(*args), *la2.backward_gated(*args, ins["do"]), pool, step))
    la2.check()
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_gradients_hold_the_same_bits_on_every_call(la2):  # noqa: F811
    """Pieces of many lengths, chunks that add them up (both state passes run side by
    side) and scanned ones, gates of very different sizes."""
    for B, H, N in ((1, 8, 9000), (2, 16, 2048), (1, 1, 5000)):
        ins = {n: t.cuda() for n, t in make("bf16", B, H, N, 128, 128, 2, "strong").items()}
        ins["gate"][..., ::7] *= 2.0 ** -20
        args = [ins[n] for n in ("q", "k", "v", "gate", "do")]
        first = la2.backward_gated(*args)
        for _ in range(10):
            assert all(torch.equal(x, y) for x, y in zip(first, la2.backward_gated(*args)))
    la2.check()


def test_two_streams_many_times(la2):  # noqa: F811
    """Calls on two streams share the memory system and the instruction caches, so that a
    CTA's roles meet at other times than alone: no wait runs out, and the bits stay."""
    sets = [{n: t.cuda() for n, t in make("bf16", 1, 8, 2000, 128, 128, 30 + s, "restarts").items()} for s in range(2)]
    args = [[s[n] for n in ("q", "k", "v", "gate")] for s in sets]
    alone = [(la2.forward_gated(*a),) + la2.backward_gated(*a, s["do"]) for a, s in zip(args, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(200):
        got = [[(la2.forward_gated(*a, stream=st),) + la2.backward_gated(*a, s["do"], stream=st) for _ in range(3)]
               for a, s, st in zip(args, sets, streams)]
        torch.cuda.synchronize()
        la2.check()
        for want, many in zip(alone, got):
            for one in many:
                assert all(torch.equal(x, y) for x, y in zip(want, one))
