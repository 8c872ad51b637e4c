"""The linear-attention block where a value is not finite, a sequence is empty,
rows lie far apart or a call is replayed: what a bad value may reach, what
stays the bits of a call without it, and the Python entry points' refusals."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import linattn_reference as R
from tests.test_linattn import attention_inputs, count, near, on_gpu
from tests.test_ssm import DEV, EPS32, HALF, TYPES, dev, gen
from tests.test_ssm_edges import same

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


# ------------------------------------------------------- what a value reaches

@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("at", [0, 15, 16, 37, 63, 64, 100, 130])
def test_bad_value_reaches_no_earlier_token(at, which, bad, io):
    """q[t] is read by o[t] alone; k[t] by o from t on; v[t] by one value of o from t on.  Everything else keeps its bits."""
    t = TYPES[io]
    B, L, N, Dk, Dv = 2, 131, 2, 24, 40
    a, _, _ = attention_inputs((B, L, (N, N, N), Dk, Dv, True, None, "slow", "dense"), t, 5)
    on = on_gpu(a)
    clean, last = H.linear_attention(**on, return_state=True)
    on[which] = on[which].clone()
    on[which][1, at, 1, 7] = bad
    o, s = H.linear_attention(**on, return_state=True)
    reach = torch.zeros(B, L, N, Dv, dtype=torch.bool, device=DEV)
    reach[1, at:at + 1 if which == "q" else L, 1, 7 if which == "v" else slice(None)] = True
    same(o[~reach], clean[~reach], "o elsewhere")
    assert not bool(o[reach].isfinite().any())
    behind = torch.zeros(B, N, Dk, Dv, dtype=torch.bool, device=DEV)
    if which == "k":
        behind[1, 1, 7] = True
    if which == "v":
        behind[1, 1, :, 7] = True
    same(s[~behind], last[~behind], "state elsewhere")
    assert not bool(s[behind].isfinite().any())


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("at", [0, 40, 64, 99])
def test_bad_gradient_reaches_no_later_token(at, io):
    """go[t] is read by gq[t] and by gk and gv up to t."""
    t = TYPES[io]
    B, L, N, Dk, Dv = 1, 100, 2, 32, 16
    a, go, gso = attention_inputs((B, L, (N, N, N), Dk, Dv, True, None, "slow", "dense"), t, 6)
    on, go = on_gpu(a), dev(go)
    clean = H.linear_attention_backward(**on, go=go, gstate_out=dev(gso))
    go = go.clone()
    go[0, at, 0, 3] = NAN
    got = H.linear_attention_backward(**on, go=go, gstate_out=dev(gso))
    same(got["gq"][:, :at], clean["gq"][:, :at], "gq before")
    same(got["gq"][:, at + 1:], clean["gq"][:, at + 1:], "gq behind")
    for k in ("gk", "gv"):
        same(got[k][:, at + 1:], clean[k][:, at + 1:], k)
        same(got[k][:, :, 1], clean[k][:, :, 1], k)
    assert bool(got["gk"][0, :at + 1, 0].isnan().all()) and bool(got["gv"][0, :at + 1, 0, 3].isnan().all())


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("L", [5, 70, 4100])
def test_empty_sequence_hands_its_state_on(L, io):
    t = TYPES[io]
    B, N, Dk, Dv = 3, 1, 16, 24
    a, go, gso = attention_inputs((B, L, (N, N, N), Dk, Dv, True, [L, 0, L // 2], "slow", "dense"), t, L)
    a["state"][1, 0, ::2], a["state"][1, 0, 1::2] = NAN, INF
    a["state"][1, 0, 3, 3] = -0.0
    on = on_gpu(a)
    o, s = H.linear_attention(**on, return_state=True)
    same(s[1], on["state"][1], "the state of an empty sequence")
    assert not bool(o[1].any()) and bool(o[0].isfinite().all()) and bool(s[0].isfinite().all())
    gso[1, 0, 2] = NAN
    got = H.linear_attention_backward(**on, go=dev(go), gstate_out=dev(gso))
    same(got["gstate"][1], dev(gso)[1], "gstate of an empty sequence")
    for k in ("gq", "gk", "gv"):
        assert not bool(got[k][1].any()) and bool(got[k].isfinite().all()), k


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_group_norm_bad_value_stays_in_its_group(io):
    t, r = TYPES[io], gen(2)
    x, z, gy, w, b = r(9, 96).to(t), r(9, 96).to(t), r(9, 96).to(t), dev(r(96)), dev(r(96))
    xb = x.clone()
    xb[4, 40] = NAN
    y, yb = (H.group_norm(dev(v), 4, w, b, z=dev(z)) for v in (x, xb))
    keep = torch.ones(9, 96, dtype=torch.bool)
    keep[4, 24:48] = False
    same(y.cpu()[keep], yb.cpu()[keep], "y of other groups")
    assert bool(yb.cpu()[~keep].isnan().all())
    g, gb = (H.group_norm_backward(dev(v), 4, dev(gy), w, b, z=dev(z)) for v in (x, xb))
    for k in ("gx", "gz"):
        same(g[k].cpu()[keep], gb[k].cpu()[keep], k)
    cols = torch.ones(96, dtype=torch.bool)
    cols[24:48] = False
    same(g["gweight"].cpu()[cols], gb["gweight"].cpu()[cols], "gweight of other groups")


def test_group_norm_backward_without_eps():
    """eps = 0 on groups that are not constant: places behind the last row or group add nothing."""
    r = gen(3)
    for rows, G, Dg in ((1, 3, 24), (5, 7, 40), (3, 1, 300), (17, 12, 128), (2, 1, 1030)):
        x, gy, w = r(rows, G * Dg), r(rows, G * Dg), 1 + 0.1 * r(G * Dg)
        g = H.group_norm_backward(dev(x), G, dev(gy), dev(w), eps=0.0)
        v = x.double().requires_grad_()
        u = w.double().requires_grad_()
        (R.group_norm(v, G, u, eps=0.0) * gy).sum().backward()
        # the counts of test_group_norm, sizes of normal values
        c = 8 * (Dg / 256 + 24) + rows
        near(g["gx"], v.grad, 8 * float(gy.abs().max()), c, 0, "gx")
        near(g["gweight"], u.grad, (gy.abs() * 6).sum(0).double(), c, 0, "gweight")


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_bad_value_stays_in_its_pair(interleaved):
    x = dev(gen(4)(2, 9, 3, 64))
    freq, _ = H.rotary_frequencies(48, device=DEV)
    y = H.rotary(x, freq, interleaved=interleaved)
    xb = x.clone()
    xb[1, 4, 2, 6], xb[0, 1, 1, 60] = NAN, INF
    yb = H.rotary(xb, freq, interleaved=interleaved)
    reach = torch.zeros_like(x, dtype=torch.bool)
    reach[1, 4, 2, [6, 7] if interleaved else [6, 30]] = True
    reach[0, 1, 1, 60] = True
    same(yb[~reach], y[~reach], "other values")
    assert bool(yb[1, 4, 2][reach[1, 4, 2]].isnan().all()) and float(yb[0, 1, 1, 60]) == INF


# ------------------------------------------------------------ views and places

@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_views_give_the_bits_of_copies(io):
    """Heads first, time first, parts of rows at odd places, one sequence for a whole batch, one token for all of them."""
    t, r = TYPES[io], gen(8)
    B, L, N, Dk, Dv = 3, 90, 2, 40, 48
    q, k, v = (dev(r(B, L, N, d).to(t)) for d in (Dk, Dk, Dv))
    g, go = dev(-torch.tensor([0.01, 0.3])), dev(r(B, L, N, Dv).to(t))
    want, grads = H.linear_attention(q, k, v, g), H.linear_attention_backward(q, k, v, go, g)
    odd = torch.zeros(B, L, 7 + N * (2 * Dk + Dv) + 5, dtype=t, device=DEV)
    at = 7
    parts = []
    for x, d in ((q, Dk), (k, Dk), (v, Dv)):
        odd[..., at:at + N * d] = x.flatten(2)
        parts.append(odd[..., at:at + N * d].unflatten(-1, (N, d)))
        at += N * d
    first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    time = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    for views in (parts, first, time):
        assert not views[0].is_contiguous()
        same(H.linear_attention(*views, g), want, "o")
        for name, x in H.linear_attention_backward(*views, go, g).items():
            if x is not None:
                same(x, grads[name], name)
    one = k[:1].expand(B, -1, -1, -1)
    same(H.linear_attention(q, one, v, g), H.linear_attention(q, one.contiguous(), v, g), "one sequence's k")
    still = q[:, :1].expand(-1, L, -1, -1)
    same(H.linear_attention(still, k, v, g), H.linear_attention(still.contiguous(), k, v, g), "one token's q")


def test_rows_behind_two_to_the_31_values():
    """A token's row is so wide that the last ones lie beyond 2^32 bytes, and a block of 64 beyond 32 bits of offsets."""
    N, D = 1, 16
    wide = (1 << 23) + 8                                # the kernel for far rows; 300 of them are 4.7 GiB of bf16
    r = gen(10)
    q, k, v = (r(1, 300, N, D).to(torch.bfloat16) for _ in range(3))
    room = torch.empty(300 * wide, dtype=torch.bfloat16, device=DEV)
    rows = room.view(1, 300, wide)
    views = []
    for i, x in enumerate((q, k, v)):
        rows[:, :, 32 * i:32 * i + D] = dev(x)[:, :, 0]
        views.append(rows[:, :, 32 * i:32 * i + D].unflatten(-1, (N, D)))
    want = H.linear_attention(dev(q), dev(k), dev(v))
    got = H.linear_attention(*views)
    near(got, *R.linear_attention(q, k, v)["o"], count(300, D, D), 1, "o")
    near(got, want.double().cpu(), R.linear_attention(q, k, v)["o"][1], count(300, D, D), 2, "o of rows that are near")
    freq, _ = H.rotary_frequencies(D, device=DEV)
    same(H.rotary(views[0], freq), H.rotary(dev(q), freq), "rotary")
    last = rows[:, -1:, :D].unflatten(-1, (N, D))
    pos = torch.tensor([[299]], dtype=torch.int32, device=DEV)
    turned = H.rotary(last, freq, pos, out=last)
    same(turned, H.rotary(dev(q[:, -1:]), freq, pos), "in place at the end")


# -------------------------------------------------------- replays and streams

def block_calls():
    t, r = torch.bfloat16, gen(12)
    B, L, N, D = 2, 1100, 2, 64                         # long enough for a split time axis
    q, k, v, go = (dev(r(B, L, h, D).to(t)) for h in (N, 1, 1, N))
    g, n = dev(-torch.tensor([0.01, 0.2])), torch.tensor([1100, 77], dtype=torch.int32, device=DEV)
    freq, _ = H.rotary_frequencies(D, device=DEV)
    pos = torch.arange(L, device=DEV, dtype=torch.int32)
    w, b, z = dev(r(N * D)), dev(r(N * D)), dev(r(B, L, N * D).to(t))
    need = H.linear_attention_backward_workspace_bytes(B, L, N, N, 1, 1, D, D)
    assert H.linear_attention_workspace_bytes(B, L, N, D, D) > 0 and need > 0

    def run():
        o, s = H.linear_attention(q, k, v, g, lengths=n, return_state=True)
        gr = H.linear_attention_backward(q, k, v, go, g, lengths=n)
        y = H.group_norm(o.flatten(2), N, w, b, z=z)
        gn = H.group_norm_backward(o.flatten(2), N, y, w, b, z=z)
        return [o, s, gr["gq"], gr["gk"], gr["gv"], H.rotary(q, freq, pos), y, gn["gx"], gn["gweight"], gn["gbias"], gn["gz"]]
    return run


def test_calls_replay_from_a_graph():
    run = block_calls()
    want = [x.clone() for x in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        for x in out:
            x.zero_()
        again = run()                                   # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (x, y, e) in enumerate(zip(out, want, again)):
            same(x, y, f"output {k} of replay {i}")
            same(e, y, f"output {k}, eager")


def test_calls_on_two_streams_at_once():
    run = block_calls()
    want = [x.clone() for x in run()]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([run() for _ in range(3)])
    torch.cuda.synchronize()
    for o in outs:
        for rep in o:
            for k, (x, y) in enumerate(zip(rep, want)):
                same(x, y, f"output {k}")


def test_steps_replay_from_a_graph():
    r = gen(13)
    q, k, v = dev(r(3, 4, 64)), dev(r(3, 2, 64)), dev(r(3, 2, 32))
    g, state = dev(-r(4).abs()), dev(r(3, 4, 64, 32))
    eager, o = state.clone(), torch.empty(3, 4, 32, device=DEV)
    H.linear_attention_step(q, k, v, eager.clone(), g, out=o)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H.linear_attention_step(q, k, v, state, g, out=o)
    for i in range(3):
        want = H.linear_attention_step(q, k, v, eager, g)
        graph.replay()
        torch.cuda.synchronize()
        same(o, want, f"o of replay {i}")
        same(state, eager, f"state of replay {i}")


def test_many_tokens_of_a_slow_decay():
    """4000 tokens one at a time: a decay that was rounded once would bend the state by 4000 half steps."""
    r = gen(14)
    L, D = 4000, 16
    q, k, v = (r(1, L, 1, D) for _ in range(3))
    g = torch.tensor([-1e-4])
    ref = R.linear_attention(q, k, v, g)
    state = torch.zeros(1, 1, D, D, device=DEV)
    qd, kd, vd, gd = map(dev, (q, k, v, g))
    for i in range(L):
        o = H.linear_attention_step(qd[:, i], kd[:, i], vd[:, i], state, gd)
    # a token adds one rounding to the state, of half a step of its size then: sqrt(L) of the largest of them in all, for which
    # 4 sqrt(L) is a bound that chance does not reach; every one of them the same way would be L
    big = float(ref["state"][0].abs().max())
    assert float((state.cpu().double() - ref["state"][0]).abs().max()) <= 4 * L ** 0.5 * EPS32 * 2 * big
    near(o, ref["o"][0][:, -1], ref["o"][1][:, -1], 4 * L ** 0.5, 0, "the last o")


# ------------------------------------------------------------------- refusals

def test_entry_points_ask_for_their_tensors():
    r = gen(15)
    x, row, s = dev(r(2, 6, 4, 8)), dev(r(2, 4, 8)), dev(r(2, 4, 8, 8))
    freq, _ = H.rotary_frequencies(8, device=DEV)
    flat = x.flatten(2)
    calls = {
        "linear_attention": (H.linear_attention, dict(q=x, k=x, v=x)),
        "linear_attention_step": (H.linear_attention_step, dict(q=row, k=row, v=row, state=s)),
        "linear_attention_backward": (H.linear_attention_backward, dict(q=x, k=x, v=x, go=x)),
        "rotary": (H.rotary, dict(x=x, freq=freq)),
        "group_norm": (H.group_norm, dict(x=flat, groups=4)),
        "group_norm_backward": (H.group_norm_backward, dict(x=flat, groups=4, gy=flat)),
    }
    for name, (f, args) in calls.items():
        f(**args)
        for k, t in args.items():
            if not isinstance(t, torch.Tensor):
                continue
            for bad in ([1.0], t.cpu()):
                with pytest.raises(TypeError):
                    f(**dict(args, **{k: bad}))
            with pytest.raises((TypeError, H.HyenaError)) as e:
                f(**dict(args, **{k: None}))
            assert e.type is TypeError or e.value.code == 1, (name, k)
            with pytest.raises((TypeError, ValueError)):
                f(**dict(args, **{k: t.half()}))


def test_entry_points_refuse_shapes():
    r = gen(16)
    x, row = dev(r(2, 6, 4, 8)), dev(r(2, 4, 8))
    att = H.linear_attention
    freq, _ = H.rotary_frequencies(8, device=DEV)
    for call in (
            lambda: att(x, x[:, :5], x), lambda: att(x, x[:1], x), lambda: att(x, x[..., :4], x), lambda: att(x[:, :, :3], x, x),
            lambda: att(row, row, row), lambda: att(x[..., ::2], x[..., ::2], x), lambda: att(x, x, x, log_decay=dev(r(3))),
            lambda: att(x, x, x, state=dev(r(2, 4, 8, 9))), lambda: att(x, x, x, lengths=torch.zeros(3, dtype=torch.int32, device=DEV)),
            lambda: att(x, x, x, out=dev(r(2, 6, 4, 9))), lambda: H.linear_attention_step(row, row, row, dev(r(2, 4, 8, 4))),
            lambda: H.linear_attention_backward(x, x, x, x[:, :5].contiguous()),
            lambda: H.rotary(x, freq, torch.zeros(5, dtype=torch.int32, device=DEV)), lambda: H.rotary(row, freq),
            lambda: H.rotary(x.transpose(1, 2), freq, out=x), lambda: H.rotary(x, freq, out=x[:, :3]),
            lambda: H.group_norm(row, 3), lambda: H.group_norm(row, 0), lambda: H.group_norm(row, 2, z=row, silu=True),
            lambda: H.group_norm(row, 2, weight=dev(r(7))), lambda: H.group_norm(row.transpose(0, 1), 2)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: att(x, x.bfloat16(), x), lambda: att(x, x, x, lengths=torch.zeros(2, dtype=torch.int64, device=DEV)),
                 lambda: H.rotary(x, freq.float()), lambda: H.rotary(x, freq, torch.zeros(2, 6, dtype=torch.int64, device=DEV))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: att(dev(r(1, 2, 1, 257)), dev(r(1, 2, 1, 257)), dev(r(1, 2, 1, 8))), lambda: att(x, x, x, scale=float("nan")),
                 lambda: H.rotary(x[..., :4], freq), lambda: H.rotary(x[:1].expand(2, -1, -1, -1), freq, out="same")):
        with pytest.raises((H.HyenaError, TypeError)):
            call()
    wide = x[:1].expand(2, -1, -1, -1)
    with pytest.raises(H.HyenaError):
        H.rotary(wide, freq, out=wide)                  # one memory for two sequences


# ------------------------------------------------------ the caller's own memory

def test_rotary_positions_for_a_whole_batch():
    """No positions, one row of them for all sequences, and one for each give the same bits where they say the same."""
    x = dev(gen(17)(3, 21, 2, 32))
    freq, _ = H.rotary_frequencies(16, device=DEV)
    row = torch.arange(21, device=DEV, dtype=torch.int32)
    want = H.rotary(x, freq)
    same(H.rotary(x, freq, row), want, "one row")
    same(H.rotary(x, freq, row.expand(3, -1).contiguous()), want, "a row each")
    same(H.rotary(x, freq, row + 7)[2], H.rotary(x[2:], freq, row + 7)[0], "the last sequence")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
def test_outputs_and_workspaces_of_the_caller(io):
    """A workspace that holds anything, larger than asked for and used again, and outputs that are given."""
    t, r = TYPES[io], gen(18)
    B, L, N, D = 1, 2000, 2, 64
    q, k, v, go = (dev(r(B, L, h, D).to(t)) for h in (N, 1, N, N))
    want, last = H.linear_attention(q, k, v, return_state=True)
    grads = H.linear_attention_backward(q, k, v, go)
    need = max(H.linear_attention_workspace_bytes(B, L, N, D, D), H.linear_attention_backward_workspace_bytes(B, L, N, N, 1, N, D, D))
    assert H.linear_attention_workspace_bytes(B, L, N, D, D) > 0
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    o, s = torch.empty_like(want), torch.empty_like(last)
    for _ in range(2):
        got = H.linear_attention(q, k, v, return_state=True, out=o, state_out=s, workspace=ws)
        assert got[0] is o and got[1] is s
        same(o, want, "o")
        same(s, last, "state")
        for name, x in H.linear_attention_backward(q, k, v, go, workspace=ws).items():
            same(x, grads[name], name)
    with pytest.raises(H.HyenaError):
        H.linear_attention(q, k, v, workspace=ws[:16])
    x, w = dev(r(50, 96).to(t)), dev(r(96))
    a, b = H.group_norm_backward(x, 3, x, w), H.group_norm_backward(x, 3, x, w, workspace=torch.full(
        (H.group_norm_backward_workspace_bytes(50, 96, 3),), 255, dtype=torch.uint8, device=DEV))
    for name in a:
        same(a[name], b[name], name)
