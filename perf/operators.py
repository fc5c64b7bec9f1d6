"""Cases for the gated recurrence, the q/k preparation and the state slots.

The operators of a layer whose KV state decays by a gate that each token brings,
in training and in serving, each in its plain form (elementary torch operations,
32 bits, 64 for cumulative gates and rotation angles) and as the library's calls:

* ``gated_fwd``, ``gated_bwd``: ``KV_t = exp(gate_t) KV_(t-1) + k_t^T v_t``,
  ``o_t = q_t KV_t`` over whole sequences, and the gradients of <dO, O> by q, k, v
  and the log gate;
* ``gated_state``: the state that a prefill leaves, into the slots of a pool;
* ``decode``: one token a sequence on the states of a pool's slots;
* ``rope_fwd``, ``rope_bwd``: RMS norm of every query and key head and the
  rotation of its pairs by one or three position axes, written as the [B,H,N,d]
  tensors that the attention reads; and the gradients;
* ``fork``, ``compact``: copies between a pool's slots (one prompt into several
  continuations, fresh slots zeroed) and the live slots moved to the front.
"""

import math

import torch

own = False

_CHUNK = 64  # rows that the plain form treats as one block
_LOG_ZERO = -1.0e4  # stands for log 0 in the plain form: exp of it is 0


def listed():
    return [
        # the smallest call: one head of 256 tokens, where launches count
        dict(name="gated_fwd_f32_n256", kind="gated_fwd", dt="f32", B=1, H=1, N=256, d=64, dv=64, packed=False),
        # one training layer, forward
        dict(name="gated_fwd_b4h16_n2k", kind="gated_fwd", dt="bf16", B=4, H=16, N=2048, d=128, dv=128, packed=False),
        # a long prompt of one sequence (several documents packed into it)
        dict(name="gated_fwd_b1h32_n16k", kind="gated_fwd", dt="bf16", B=1, H=32, N=16384, d=128, dv=128, packed=True),
        # gradients of a short odd batch in 32 bits, odd head widths
        dict(name="gated_bwd_f32_odd", kind="gated_bwd", dt="f32", B=2, H=3, N=777, d=48, dv=80, packed=False),
        # gradients of a long-context layer
        dict(name="gated_bwd_b2h32_n8k", kind="gated_bwd", dt="bf16", B=2, H=32, N=8192, d=128, dv=128, packed=True),
        # a ragged prefill's states, into slots of a serving pool
        dict(name="gated_state_b3h16_n3001", kind="gated_state", dt="bf16", B=3, H=16, N=3001, d=128, dv=128, packed=False),
        # one token of one sequence: latency
        dict(name="decode_b1h8", kind="decode", dt="bf16", B=1, H=8, d=128, dv=128, slots=4, pad=0),
        # one token of a full batch with a few padded rows
        dict(name="decode_b64h32", kind="decode", dt="bf16", B=64, H=32, d=128, dv=128, slots=72, pad=3),
        # queries and keys of a decode batch at far positions
        dict(name="rope_fwd_decode_b64", kind="rope_fwd", dt="bf16", B=64, N=1, H=32, Hkv=8, d=128, rot=128, axes=1, far=1 << 20),
        # queries and keys of a training layer over text and images, with gradients
        dict(name="rope_bwd_b4_n2k_3axes", kind="rope_bwd", dt="bf16", B=4, N=2048, H=16, Hkv=16, d=128, rot=128, axes=3, far=0),
        # one prompt's state into the slots of its continuations, some fresh slots zeroed
        dict(name="fork_s32h32", kind="fork", H=32, d=128, dv=128, slots=32, n=24),
        # a pool after a third of its sequences ended
        dict(name="compact_s48h32", kind="compact", H=32, d=128, dv=128, slots=48, n=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["gated_fwd", "gated_bwd", "gated_state", "decode", "rope_fwd", "rope_bwd", "fork", "compact"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind in ("gated_fwd", "gated_bwd", "gated_state"):
        if dt == "bf16":
            d, dv, most, longest = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64)]) + (1 << 19, 1 << 16)
            if d == 64:
                most, longest = 1 << 15, 4096
        else:
            d, dv, most, longest = rng.randint(16, 128), rng.randint(16, 128), 1 << 15, 4096
        N = _log_int(rng, 1, longest)
        B = _log_int(rng, 1, max(1, min(8, most // N)))
        H = _log_int(rng, 1, max(1, min(32, most // (N * B))))
        return dict(kind=kind, dt=dt, B=B, H=H, N=N, d=d, dv=dv, packed=rng.random() < 0.3)
    if kind == "decode":
        d, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (rng.randint(8, 160), rng.randint(8, 160))])
        B = _log_int(rng, 1, 64)
        return dict(kind=kind, dt=dt, B=B, H=rng.randint(1, 32), d=d, dv=dv, slots=B + rng.randint(0, 8), pad=rng.randint(0, B // 4))
    if kind in ("rope_fwd", "rope_bwd"):
        d = rng.choice([128, 128, 64, 2 * rng.randint(8, 64)])
        Hkv = _log_int(rng, 1, 16)
        H = Hkv * rng.choice([1, 1, 2, 4])
        N = _log_int(rng, 1, 16384)
        B = _log_int(rng, 1, max(1, min(64, (1 << 18) // (N * (H + Hkv)))))
        axes = rng.choice([1, 1, 3])
        rot = d if rng.random() < 0.6 else 2 * rng.randint(3, d // 2)
        return dict(kind=kind, dt=dt, B=B, N=N, H=H, Hkv=Hkv, d=d, rot=rot, axes=axes, far=rng.choice([0, 0, 1 << 17, 1 << 20]))
    d, dv = rng.choice([(128, 128), (128, 128), (64, 64), (rng.randint(8, 128), rng.randint(8, 128))])
    slots = _log_int(rng, 4, 64)
    return dict(kind=kind, H=rng.randint(1, 32), d=d, dv=dv, slots=slots, n=rng.randint(1, slots - 1))


def _dtype(case):
    return torch.float32 if case.get("dt") == "f32" else torch.bfloat16


def _gates(g, B, H, N, dt, packed):
    # log sigmoid of a projection, sharpened less in some heads than in others (a
    # head's memory is from a few to a few hundred tokens); packed documents start
    # with a gate of 0
    head = torch.logspace(0.0, -2.0, H, device="cuda").view(1, H, 1)
    x = torch.nn.functional.logsigmoid(torch.randn(B, H, N, device="cuda", generator=g) + 1.0) * head
    if packed:
        starts = torch.rand(B, 1, N, device="cuda", generator=g) < 1.0 / 512
        x = x.masked_fill(starts, float("-inf"))
    return x.to(dt)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    kind = case["kind"]
    s = {"case": case}

    def rand(*shape, scale=1.0, dt=None):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dt or torch.float32)

    if kind in ("gated_fwd", "gated_bwd", "gated_state"):
        B, H, N, d, dv, dt = case["B"], case["H"], case["N"], case["d"], case["dv"], _dtype(case)
        if kind != "gated_state":
            s["q"] = rand(B, H, N, d, scale=d ** -0.5, dt=dt)
        s["k"] = rand(B, H, N, d, scale=d ** -0.5, dt=dt)
        s["v"] = rand(B, H, N, dv, dt=dt)
        s["gate"] = _gates(g, B, H, N, dt, case["packed"])
        if kind == "gated_bwd":
            s["do"] = rand(B, H, N, dv, dt=dt)
        if kind == "gated_state":
            s["pool"] = rand(B + 2, H, d, dv, scale=0.1)
            s["slots"] = torch.randperm(B + 2, generator=g, device="cuda")[:B].to(torch.int32)
    elif kind == "decode":
        B, H, d, dv, dt = case["B"], case["H"], case["d"], case["dv"], _dtype(case)
        s["q"], s["k"] = (rand(B, H, d, scale=d ** -0.5, dt=dt) for _ in range(2))
        s["v"] = rand(B, H, dv, dt=dt)
        s["gate"] = _gates(g, B, H, 1, dt, False)[..., 0].contiguous()
        s["pool"] = rand(case["slots"], H, d, dv, scale=0.1)
        s["slots"] = torch.randperm(case["slots"], generator=g, device="cuda")[:B].to(torch.int32)
        if case["pad"]:
            s["slots"][B - case["pad"]:] = -1
        s["out"] = torch.zeros(B, H, dv, dtype=dt, device="cuda")
    elif kind in ("rope_fwd", "rope_bwd"):
        B, N, H, Hkv, d, dt = case["B"], case["N"], case["H"], case["Hkv"], case["d"], _dtype(case)
        proj = rand(B, N, H + 2 * Hkv, d, dt=dt)  # the fused q, k, v projection
        s["proj"] = proj
        s["q"], s["k"] = proj[:, :, :H], proj[:, :, H:H + Hkv]
        s["wq"], s["wk"] = ((1.0 + rand(d, scale=0.1)).to(dt) for _ in range(2))
        t = torch.arange(N, device="cuda", dtype=torch.int64)
        start = torch.randint(0, case["far"] + 1, (B, 1), device="cuda", generator=g)
        if case["axes"] == 1:
            pos = (t + start)[None]
        else:  # frames of 16 x 16 patches
            pos = torch.stack([(t // 256).expand(B, N) + start, (t // 16 % 16).expand(B, N) + 0 * start,
                               (t % 16).expand(B, N) + 0 * start])
        s["pos"] = pos.to(torch.int32).contiguous()
        half = case["rot"] // 2
        first = half - 2 * (half * 3 // 8) if case["axes"] == 3 else half
        s["sections"] = (first, half * 3 // 8, half * 3 // 8) if case["axes"] == 3 else (half,)
        if kind == "rope_bwd":
            s["dyq"], s["dyk"] = rand(B, H, N, d, dt=dt), rand(B, Hkv, N, d, dt=dt)
    else:
        H, d, dv, S, n = case["H"], case["d"], case["dv"], case["slots"], case["n"]
        s["pool"] = rand(S, H, d, dv, scale=0.1)
        order = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
        if kind == "fork":  # the first quarter of the slots (at least one) into the next n; the last of these are fresh
            few = max(1, S // 4)
            n = min(n, S - few)
            src = order[torch.arange(n, device="cuda") % few].clone()
            src[n - n // 4:] = -1
            s["src"], s["dst"] = src, order[few:few + n].clone()
        else:
            live = torch.zeros(S, dtype=torch.int32, device="cuda")
            live[order[:n].long()] = 1
            s["live"] = live
    return s


# ------------------------------------------------------------------ plain forms


def _blocks(x, T):
    # [B,H,N,w] -> float32 [BH,T,CHUNK,w], zero rows behind the last token
    B, H, N, w = x.shape
    x = x.reshape(B * H, N, w).float()
    return torch.nn.functional.pad(x, (0, 0, 0, T * _CHUNK - N)).view(B * H, T, _CHUNK, w)


class _Gates:
    """Cumulative log gates of every block and the decay weights made of them."""

    def __init__(self, gate):
        B, H, N = gate.shape
        self.T = T = (N + _CHUNK - 1) // _CHUNK
        x = gate.reshape(B * H, N).double().clamp_min(_LOG_ZERO)
        x = torch.nn.functional.pad(x, (0, T * _CHUNK - N)).view(B * H, T, _CHUNK)
        c = x.cumsum(-1)
        self.dead = x <= _LOG_ZERO
        i = torch.arange(_CHUNK, device=gate.device)
        pair = torch.where(i[:, None] >= i[None, :], c[..., :, None] - c[..., None, :], -math.inf)
        self.intra = pair.exp().float()  # [BH,T,t,s]: from the state after s to the one after t
        self.head = c.exp().float()  # from the state before the block to the one after t
        self.tail = (c[..., -1:] - c).exp().float()  # from the state after s to the block's last
        total = c[..., -1].cumsum(-1)  # [BH,T]
        before = torch.cat([torch.zeros_like(total[:, :1]), total[:, :-1]], 1)
        j = torch.arange(T, device=gate.device)
        # block m's own state as the state before block n sees it
        self.inter = torch.where(j[:, None] > j[None, :], before[:, :, None] - total[:, None, :],
                                 -math.inf).exp().float()
        self.whole = c[..., -1].exp().float()


def _prefix(a, b, w):
    """The state a^T b before every block."""
    own_state = (a * w.tail[..., None]).transpose(-1, -2) @ b
    return (w.inter @ own_state.flatten(2)).view_as(own_state)


def _suffix(a, b, w):
    """sum a_t^T b_t of the tokens behind every block, decayed back to its last token."""
    own_state = (a * w.head[..., None]).transpose(-1, -2) @ b
    return (w.inter.transpose(-1, -2) @ own_state.flatten(2)).view_as(own_state)


def _unblock(x, like, dt):
    B, H, N = like.shape[:3]
    return x.reshape(B, H, -1, x.shape[-1])[:, :, :N].to(dt).contiguous()


def _plain_gated_fwd(s):
    w = _Gates(s["gate"])
    q, k, v = (_blocks(s[x], w.T) for x in "qkv")
    o = ((q @ k.transpose(-1, -2)) * w.intra) @ v + w.head[..., None] * (q @ _prefix(k, v, w))
    return _unblock(o, s["q"], s["q"].dtype)


def _plain_gated_bwd(s):
    w = _Gates(s["gate"])
    q, k, v, do = (_blocks(s[x], w.T) for x in ("q", "k", "v", "do"))
    before, after = _prefix(k, v, w), _suffix(q, do, w)
    p = (q @ k.transpose(-1, -2)) * w.intra
    a = (do @ v.transpose(-1, -2)) * w.intra
    dq_far = w.head[..., None] * (do @ before.transpose(-1, -2))
    dk_far = w.tail[..., None] * (v @ after.transpose(-1, -2))
    dq = a @ k + dq_far
    dk = a.transpose(-1, -2) @ q + dk_far
    dv = p.transpose(-1, -2) @ do + w.tail[..., None] * (k @ after)
    # d<dO,O> / d gate_t: all pairs (i, j) with j < t <= i, with no difference of large sums
    pairs = (q @ k.transpose(-1, -2)) * a
    i = torch.arange(_CHUNK, device=q.device)
    inside = (pairs.flip(-2).cumsum(-2).flip(-2) * (i[:, None] > i[None, :])).sum(-1)
    from_before = (q * dq_far).sum(-1).flip(-1).cumsum(-1).flip(-1)
    to_after = (k * dk_far).sum(-1)
    to_after = to_after.cumsum(-1) - to_after
    across = (before * after).sum((-1, -2)) * w.whole
    dg = (inside + from_before + to_after + across[..., None]).masked_fill(w.dead, 0.0)
    dt = s["q"].dtype
    return {"dq": _unblock(dq, s["q"], dt), "dk": _unblock(dk, s["q"], dt), "dv": _unblock(dv, s["q"], dt),
            "dgate": _unblock(dg[..., None], s["q"], dt)[..., 0]}


def _plain_gated_state(s):
    w = _Gates(s["gate"])
    k, v = (_blocks(s[x], w.T) for x in "kv")
    B, H, N, d = s["k"].shape
    own_state = (k * w.tail[..., None]).transpose(-1, -2) @ v
    last = _prefix(k, v, w)[:, -1] * w.whole[:, -1, None, None] + own_state[:, -1]
    decay = s["gate"].double().clamp_min(_LOG_ZERO).sum(-1).exp().float()
    at = s["slots"].long()
    s["pool"][at] = s["pool"][at] * decay[..., None, None] + last.view(B, H, d, -1)
    return s["pool"]


def _plain_decode(s):
    B = s["q"].shape[0] - s["case"]["pad"]
    at = s["slots"][:B].long()
    q, k, v, gate = (s[x][:B].float() for x in ("q", "k", "v", "gate"))
    state = s["pool"][at] * gate.exp()[..., None, None] + k[..., :, None] * v[..., None, :]
    s["pool"][at] = state
    s["out"][:B] = (q[..., None, :] @ state)[..., 0, :].to(s["out"].dtype)
    return {"o": s["out"], "pool": s["pool"]}


_EPS, _BASE = 1e-6, 10000.0


def _rotation(s):
    """cos and sin of every pair's angle, [B,1,N,rot/2]."""
    rot = s["case"]["rot"]
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=rot // 2)
    angle = s["pos"].double()[axis].permute(1, 2, 0) * _BASE ** (-2.0 * i / rot)
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _plain_rope(x, weight, cos, sin, scale):
    x = x.float().transpose(1, 2)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * weight.float()
    h = cos.shape[-1]
    a, b = y[..., :h], y[..., h:2 * h]
    return torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., 2 * h:]], -1) * scale


def _plain_rope_bwd(dy, x, weight, cos, sin, scale):
    dy = dy.float() * scale
    h = cos.shape[-1]
    a, b = dy[..., :h], dy[..., h:2 * h]
    dz = torch.cat([a * cos + b * sin, b * cos - a * sin, dy[..., 2 * h:]], -1)
    x = x.float().transpose(1, 2)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
    xh = x * r
    dxh = dz * weight.float()
    dx = r * (dxh - xh * (dxh * xh).mean(-1, keepdim=True))
    return dx.transpose(1, 2), (dz * xh).sum((0, 1, 2))


def _scale(s):
    return s["case"]["d"] ** -0.5


def _plain_rope_fwd_pass(s):
    cos, sin = _rotation(s)
    dt = s["q"].dtype
    return {"q": _plain_rope(s["q"], s["wq"], cos, sin, _scale(s)).to(dt),
            "k": _plain_rope(s["k"], s["wk"], cos, sin, 1.0).to(dt)}


def _plain_rope_bwd_pass(s):
    cos, sin = _rotation(s)
    dt = s["q"].dtype
    dq, dwq = _plain_rope_bwd(s["dyq"], s["q"], s["wq"], cos, sin, _scale(s))
    dk, dwk = _plain_rope_bwd(s["dyk"], s["k"], s["wk"], cos, sin, 1.0)
    return {"dq": dq.to(dt).contiguous(), "dk": dk.to(dt).contiguous(), "dwq": dwq.to(dt), "dwk": dwk.to(dt)}


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    rows = s["pool"][src.clamp_min(0)]
    s["pool"][dst] = torch.where((src >= 0).view(-1, 1, 1, 1), rows, 0.0)
    return s["pool"]


def _plain_compact(s):
    live = s["live"] != 0
    S = live.numel()
    at = torch.arange(S, device="cuda")
    front = at < live.sum()
    # the k-th live slot behind the front goes into the k-th hole of it
    hole, mover = front & ~live, live & ~front
    rank = torch.where(hole, hole.cumsum(0) - 1, S)
    place = torch.full((S + 1,), -1, dtype=torch.int64, device="cuda").scatter(0, rank, at)
    moved = torch.where(live, torch.where(mover, place[mover.cumsum(0) - 1], at), -1)
    source = torch.full((S + 1,), -1, dtype=torch.int64, device="cuda").scatter(0, torch.where(mover, moved, S), at)[:S]
    keep = torch.where(hole, source, at)
    s["pool"].copy_(s["pool"][keep])
    return {"pool": s["pool"], "moved": moved.to(torch.int32)}


def run(state):
    s, kind = state, state["case"]["kind"]
    if own:
        from linear_attention_la2_b200 import la2

        if kind == "gated_fwd":
            return la2.forward_gated(s["q"], s["k"], s["v"], s["gate"])
        if kind == "gated_bwd":
            dq, dk, dv, dgate = la2.backward_gated(s["q"], s["k"], s["v"], s["gate"], s["do"])
            return {"dq": dq, "dk": dk, "dv": dv, "dgate": dgate}
        if kind == "gated_state":
            return la2.kv_state_gated(s["k"], s["v"], s["gate"], s["pool"], slots=s["slots"])
        if kind == "decode":
            o = la2.decode_step_gated(s["q"], s["k"], s["v"], s["gate"], s["pool"], slots=s["slots"], out=s["out"])
            return {"o": o, "pool": s["pool"]}
        if kind == "rope_fwd":
            q, k = la2.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], base=_BASE, rot=s["case"]["rot"],
                                    sections=s["sections"], eps=_EPS, q_scale=_scale(s))
            return {"q": q, "k": k}
        if kind == "rope_bwd":
            dq, dk, dwq, dwk = la2.qk_norm_rope_backward(
                s["dyq"], s["dyk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], base=_BASE, rot=s["case"]["rot"],
                sections=s["sections"], eps=_EPS, q_scale=_scale(s))
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if kind == "fork":
            return la2.state_copy(s["pool"], s["src"], s["dst"])
        moved = la2.state_compact(s["pool"], s["live"])
        return {"pool": s["pool"], "moved": moved}
    return {"gated_fwd": _plain_gated_fwd, "gated_bwd": _plain_gated_bwd, "gated_state": _plain_gated_state,
            "decode": _plain_decode, "rope_fwd": _plain_rope_fwd_pass, "rope_bwd": _plain_rope_bwd_pass,
            "fork": _plain_fork, "compact": _plain_compact}[kind](s)


def work(case):
    kind = case["kind"]
    es = 4 if case.get("dt") == "f32" else 2
    if kind in ("gated_fwd", "gated_bwd", "gated_state"):
        B, H, N, d, dv = case["B"], case["H"], case["N"], case["d"], case["dv"]
        rows = B * H * N
        if kind == "gated_state":
            return {"bytes": rows * (d + dv + 1) * es + 2 * B * H * d * dv * 4, "flops": 2.0 * rows * d * dv}
        # the recurrence itself: k^T v into the state, q times the state; a
        # gradient pass forms two states and three products with them
        if kind == "gated_fwd":
            return {"bytes": rows * (2 * d + 2 * dv + 1) * es, "flops": 4.0 * rows * d * dv}
        return {"bytes": rows * (4 * d + 3 * dv + 2) * es, "flops": 10.0 * rows * d * dv}
    if kind == "decode":
        rows = (case["B"] - case["pad"]) * case["H"]
        return {"bytes": rows * (2 * case["d"] * case["dv"] * 4 + (2 * case["d"] + 2 * case["dv"] + 1) * es),
                "flops": 5.0 * rows * case["d"] * case["dv"]}
    if kind in ("rope_fwd", "rope_bwd"):
        rows, d = case["B"] * case["N"] * (case["H"] + case["Hkv"]), case["d"]
        more = case["axes"] * case["B"] * case["N"] * 4 + 2 * d * es
        if kind == "rope_fwd":
            return {"bytes": 2 * rows * d * es + more, "flops": 10.0 * rows * d}
        return {"bytes": 3 * rows * d * es + more + 2 * d * es, "flops": 20.0 * rows * d}
    one = case["H"] * case["d"] * case["dv"] * 4
    if kind == "fork":
        few = max(1, case["slots"] // 4)
        n = min(case["n"], case["slots"] - few)
        return {"bytes": one * (n + min(few, n - n // 4)), "flops": 0.0}
    # on average (1 - n / slots) of the n front slots are holes
    return {"bytes": one * 2.0 * max(1.0, case["n"] * (1 - case["n"] / case["slots"])) + 8 * case["slots"], "flops": 0.0}


# ------------------------------------------------------------------ in 64 bits


def _exact_rows(case, s, rows):
    """Row blocks of the left product ((Q K^T) * D) V and its gradients, one head at a time."""
    bwd = case["kind"] == "gated_bwd"
    B, H, N = case["B"], case["H"], case["N"]
    q, k, v, gate = (s[x].double() for x in ("q", "k", "v", "gate"))
    do = s["do"].double() if bwd else None
    out = {x: torch.zeros_like(y) for x, y in (("dq", q), ("dk", k), ("dv", v), ("dgate", gate))} if bwd else None
    o = torch.zeros(B, H, N, case["dv"], dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            g = gate[b, h]
            zero = torch.isneginf(g)
            resets, c = zero.long().cumsum(-1), g.masked_fill(zero, 0.0).cumsum(-1)
            flux = torch.zeros(N + 1, dtype=torch.float64, device="cuda") if bwd else None
            for t0 in range(0, N, rows):
                t1 = min(N, t0 + rows)
                t = torch.arange(t0, t1, device="cuda")[:, None]
                e = torch.arange(0, t1, device="cuda")[None, :]
                on = (t >= e) & (resets[t0:t1, None] == resets[None, :t1])
                D = torch.where(on, c[t0:t1, None] - c[None, :t1], -math.inf).exp()
                S = (q[b, h, t0:t1] @ k[b, h, :t1].T) * D
                if not bwd:
                    o[b, h, t0:t1] = S @ v[b, h, :t1]
                    continue
                raw = do[b, h, t0:t1] @ v[b, h, :t1].T
                A = raw * D
                out["dq"][b, h, t0:t1] = A @ k[b, h, :t1]
                out["dk"][b, h, :t1] += A.T @ q[b, h, t0:t1]
                out["dv"][b, h, :t1] += S.T @ do[b, h, t0:t1]
                # a pair (i, j) counts for every token t with j < t <= i
                W = S * raw
                flux[:t1] -= W.sum(0)
                flux[t0:t1] += W.sum(1)
            if bwd:
                out["dgate"][b, h] = flux[:N].flip(0).cumsum(0).flip(0).masked_fill(zero, 0.0)
    return out if bwd else o


def exact(case, seed):
    kind = case["kind"]
    s = prepare(case, seed)
    if kind in ("gated_fwd", "gated_bwd"):
        if float(case["B"] * case["H"]) * case["N"] ** 2 * (1 if kind == "gated_fwd" else 3) > 3.0e10:
            return None  # too long in 64 bits
        return _exact_rows(case, s, 2048)
    if kind == "gated_state":
        B, H, N = case["B"], case["H"], case["N"]
        k, v, gate = (s[x].double() for x in ("k", "v", "gate"))
        pool = s["pool"].double()
        zero = torch.isneginf(gate)
        # log of the product of the gates behind every token; -inf where one of them is 0
        behind = gate.masked_fill(zero, 0.0).flip(-1).cumsum(-1).flip(-1)
        cut = zero.long().flip(-1).cumsum(-1).flip(-1)
        after = torch.cat([behind[..., 1:], torch.zeros_like(behind[..., :1])], -1).exp()
        after = after * (torch.cat([cut[..., 1:], torch.zeros_like(cut[..., :1])], -1) == 0)
        whole = behind[..., 0].exp() * (cut[..., 0] == 0)
        for b, at in enumerate(s["slots"].tolist()):
            pool[at] = pool[at] * whole[b, :, None, None] + torch.einsum("hnc,hn,hne->hce", k[b], after[b], v[b])
        return pool
    if kind == "decode":
        pool, out = s["pool"].double(), s["out"].double()
        for b, at in enumerate(s["slots"].tolist()):
            if at >= 0:
                q, k, v, g = (s[x][b].double() for x in ("q", "k", "v", "gate"))
                pool[at] = pool[at] * g.exp()[:, None, None] + torch.einsum("hc,he->hce", k, v)
                out[b] = torch.einsum("hc,hce->he", q, pool[at])
        return {"o": out, "pool": pool}
    if kind in ("rope_fwd", "rope_bwd"):
        return _exact_rope(case, s)
    pool = s["pool"].double()
    if kind == "fork":
        old = pool.clone()
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[b] = old[a] if a >= 0 else 0.0
        return pool
    live = s["live"].tolist()
    n, moved = sum(live), [-1] * len(live)
    holes = [i for i in range(n) if not live[i]]
    for i, on in enumerate(live):
        if on:
            moved[i] = i if i < n else holes.pop(0)
            if moved[i] != i:
                pool[moved[i]] = pool[i].clone()
    return {"pool": pool, "moved": torch.tensor(moved, dtype=torch.int32)}


def _exact_rope(case, s):
    d, rot, half = case["d"], case["rot"], case["rot"] // 2
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    freq = torch.tensor([_BASE ** (-2.0 * i / rot) for i in range(half)], dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.stack([s["pos"][a].double() for a in axis], -1) * freq)[:, :, None]  # [B,N,1,half]

    def forward(x, w, scale):
        y = x / (x.square().mean(-1, keepdim=True) + _EPS).sqrt() * w
        z = torch.complex(y[..., :half].contiguous(), y[..., half:rot].contiguous()) * turn
        return (torch.cat([z.real, z.imag, y[..., rot:]], -1) * scale).transpose(1, 2)

    done = {}
    for name, scale in (("q", d ** -0.5), ("k", 1.0)):
        x, w = s[name].double(), s["w" + name].double()
        if case["kind"] == "rope_fwd":
            done[name] = forward(x, w, scale)
        else:
            x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
            done["d" + name], done["dw" + name] = torch.autograd.grad(forward(x, w, scale), (x, w), s["dy" + name].double())
    return done
