"""The gated form's shapes at the borders of its plans: chunks of one block, chunks added
up by their readers and scanned, widths of 64 beside 128, widths that are no multiple of
four; and restarts on slots that hold no numbers. Tolerances as in test_gpu_gated.
"""

import pytest
import torch

import oracle
from test_gpu_gated import DT, TOL, behind, double, la2, make, rel  # noqa: F401 (la2: a fixture)

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, B, H, N, d, dv, gates
    ("f32", 1, 1, 256, 64, 64, "soft"),
    ("f32", 1, 2, 830, 128, 128, "restarts"),  # 13 chunks: scanned
    ("f32", 2, 1, 1500, 36, 100, "soft"),
    ("f32", 1, 1, 200, 3, 2, "strong"),
    ("f32", 1, 1, 129, 125, 127, "weak"),
    ("f32", 5, 31, 70, 65, 68, "soft"),
    ("f32", 1, 150, 64, 16, 12, "soft"),
    ("bf16", 1, 1, 900, 64, 128, "soft"),
    ("bf16", 2, 3, 1111, 128, 64, "restarts"),
    ("bf16", 1, 2, 4100, 64, 64, "weak"),
    ("bf16", 4, 40, 100, 64, 64, "strong"),
    ("bf16", 1, 1, 9, 64, 64, "closed"),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_forward_gradients_and_state(la2, case):  # noqa: F811
    dt, B, H, N, d, dv, kind = case
    ins = make(dt, B, H, N, d, dv, 7 * N + d, kind)
    dev = {n: t.cuda() for n, t in ins.items()}
    args = [dev[n] for n in ("q", "k", "v", "gate")]
    buf, o = behind((B, H, N, dv), DT[dt])
    la2.forward_gated(*args, out=o)
    outs = [behind(dev[n].shape, DT[dt]) for n in ("q", "k", "v", "gate")]
    la2.backward_gated(*args, dev["do"], outs=tuple(x for _, x in outs))
    pool = torch.randn(B + 1, H, d, dv, generator=torch.Generator().manual_seed(N)).cuda()
    before = pool.clone()
    slots = torch.arange(B, 0, -1, dtype=torch.int32, device="cuda")
    la2.kv_state_gated(dev["k"], dev["v"], dev["gate"], pool, slots=slots)
    la2.check()
    ref = double(ins)
    qkv = (ref["q"], ref["k"], ref["v"])
    assert rel(o, oracle.forward_gated(*qkv, ref["gate"])) <= TOL[dt]
    for (_, got), w, name in zip(outs, oracle.backward_gated(*qkv, ref["do"], ref["gate"]), ("dq", "dk", "dv", "dgate")):
        if w.any():
            assert rel(got, w) <= TOL[dt], name
        else:
            assert not got.float().any(), name
    want = oracle.kv_state_gated(ref["k"], ref["v"], ref["gate"], before[slots.long()].double().cpu().numpy())
    assert rel(pool[slots.long()], want) <= 1e-5
    assert torch.equal(pool[0], before[0])
    for b, x in [(buf, o)] + outs:
        assert torch.all(b[x.numel():] == 7.25)


@pytest.mark.parametrize("dt,d,dv", [("f32", 33, 20), ("f32", 17, 5), ("bf16", 128, 128), ("bf16", 64, 64)])
def test_restart_drops_what_a_slot_held(la2, dt, d, dv):  # noqa: F811
    """A gate of -inf opens a new sequence: a slot's infinities and NaN do not reach it,
    and the state is the one of a zeroed slot, bit for bit."""
    B, H, N = 2, 2, 70
    ins = {n: t.cuda() for n, t in make(dt, B, H, N, d, dv, d).items()}
    ins["gate"][:, :, 0] = -torch.inf
    worst = torch.full((B, H, d, dv), float("nan"), device="cuda")
    worst[1] = float("inf")
    zero = torch.zeros_like(worst)
    one = [ins[n][:, :, 0].contiguous() for n in ("q", "k", "v", "gate")]
    got, want = worst.clone(), zero.clone()
    o = la2.decode_step_gated(*one, got)
    assert torch.equal(o, la2.decode_step_gated(*one, want)) and torch.equal(got, want)
    got, want = worst.clone(), zero.clone()
    la2.kv_state_gated(ins["k"], ins["v"], ins["gate"], got)
    la2.kv_state_gated(ins["k"], ins["v"], ins["gate"], want)
    la2.check()
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_calls_in_a_row_share_a_workspace(la2, dt, d):  # noqa: F811
    """Forward and backward calls queued on one stream with one workspace: each starts
    when the one before is done with it, so all give what a call by itself gives."""
    B, H, N = 2, 4, 1000
    sets = [{n: t.cuda() for n, t in make(dt, B, H, N, d, d, s).items()} for s in range(3)]
    code = la2._dtype_code(sets[0]["q"])
    ws = torch.empty(max(la2.workspace_bytes_gated(B, H, N, d, d, code, b) for b in (False, True)), dtype=torch.uint8,
                     device="cuda")
    args = [[s[n] for n in ("q", "k", "v", "gate")] for s in sets]
    alone = []
    for a, s in zip(args, sets):
        alone.append((la2.forward_gated(*a),) + la2.backward_gated(*a, s["do"]))
        torch.cuda.synchronize()
    for _ in range(5):
        got = [(la2.forward_gated(*a, workspace=ws),) + la2.backward_gated(*a, s["do"], workspace=ws)
               for a, s in zip(args, sets)]
        for x, y in zip(alone, got):
            assert all(torch.equal(u, w) for u, w in zip(x, y))
    la2.check()


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("f32", 64)])
def test_two_streams_at_once(la2, dt, d):  # noqa: F811
    """Calls on two streams, each with what it allocates there, give what they give alone."""
    sets = [{n: t.cuda() for n, t in make(dt, 1, 8, 2000, d, d, 20 + s, "restarts").items()} for s in range(2)]
    args = [[s[n] for n in ("q", "k", "v", "gate")] for s in sets]
    alone = [(la2.forward_gated(*a),) + la2.backward_gated(*a, s["do"]) for a, s in zip(args, sets)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            got[i].append((la2.forward_gated(*args[i], stream=st),)
                          + la2.backward_gated(*args[i], sets[i]["do"], stream=st))
    torch.cuda.synchronize()
    la2.check()
    for want, many in zip(alone, got):
        for one in many:
            assert all(torch.equal(x, y) for x, y in zip(want, one))
