"""The state-space block's operators at the sizes whose launches loop: several
channel tiles to a workgroup, several chunks to a segment, several sequences
or rows to a workgroup, long columns of partial sums.  Every value and every
parameter's gradient is compared within its own terms' sizes, so that a part
that is left out of a sum shows.  tests/test_ssm_plans.py holds each case to
the launch it is there for."""
import pytest
import torch

import hyena_long_conv_amd as H
from tests import ssm_reference as R
from tests.test_ssm import TYPES, close, dev, gen, leaves, scan_inputs, scan_on_gpu, spoil

pytestmark = pytest.mark.gpu

# name -> (B, D, G, N, L), what its launches have to be
SCAN = {
    "tiles": ((32, 192, 8, 5, 500), dict(split=1, segs=1, chunks_per_seg=4, waves=4, splits=1, tiles_per=2)),
    "tiles_splits": ((10, 1280, 10, 6, 300), dict(split=1, chunks_per_seg=3, waves=4, splits=4, tiles_per=2)),
    "tiles_one_chunk": ((64, 384, 16, 5, 40), dict(waves=4, chunks=1, splits=1, tiles_per=2)),
    "waves_8": ((32, 1120, 16, 37, 130), dict(waves=8, chunks=2, splits=1, tiles_per=3)),
    "waves_8_one_chunk": ((64, 1120, 16, 37, 20), dict(waves=8, chunks=1, splits=1, tiles_per=3)),
    "waves_8_splits": ((9, 4000, 16, 33, 129), dict(waves=8, chunks=2, splits=4, tiles_per=2)),
    "all_states_to_a_wave": ((2, 2100, 1, 16, 400), dict(split=1, segs=1, chunks_per_seg=4)),
    "segments": ((1, 768, 1, 16, 8192), dict(split=1, segs=32, chunks_per_seg=2, tiles_per=3)),
    "shared_states": ((1, 1000, 1, 32, 600), dict(split=4, segs=1, chunks_per_seg=5)),
    "shared_states_64": ((4, 250, 1, 64, 500), dict(split=4, segs=1, chunks_per_seg=4, waves=8, splits=8)),
    "a_channel_to_a_group": ((2, 40, 40, 40, 300), dict(tiles_per=1, chunks=3)),
    "parts": ((48, 20, 1, 4, 384), dict(parts=144)),
}


def ragged(B, L, seed):
    """Lengths over the whole range, a full sequence and an empty one among them."""
    n = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    n[0] = L
    if B > 2:
        n[B // 2] = 0
    return n


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("name", SCAN)
def test_selective_scan_wide(name, io):
    """Roundings that a term of the state passes: 8 steps of a lane at 3, 4 steps of a row's scan at 3, then for
    each later chunk its decay and another row's scan, 15, the segments' or chunks' joins, 4 each, at most as many;
    16 for the input (softplus, products) and 10 for the decays' exponents, in the sizes' half decay."""
    B, D, G, N, L = SCAN[name][0]
    t = TYPES[io]
    a, _, _ = scan_inputs((B, D, G, N, L, True, True, True, True, True, None), t, L + N)
    lengths = ragged(B, L, L) if B > 1 else None
    r = gen(L * 3 + N)
    gy, gso = r(B, D, L).to(t), r(B, D, N)
    on = scan_on_gpu(a, lengths, True)
    ref = R.selective_scan_with_sizes(**{k: dev(v) for k, v in a.items()}, softplus=True, lengths=dev(lengths), gy=dev(gy),
                                      gstate_out=dev(gso))
    chunks = -(-L // 128)
    c_h = 24 + 12 + 24 + 19 * chunks + 16 + 10
    y, h = H.selective_scan(**on, return_state=True)
    cpu = lambda p: (p[0].cpu(), p[1].cpu())  # noqa: E731
    for got, key, c in ((y, "y", c_h + N + 16), (h, "h", c_h)):
        want, size = cpu(ref[key])
        close(got, want, c, size, key)
    g = H.selective_scan_backward(**on, gy=dev(spoil(gy, lengths)), gstate_out=dev(gso))
    c = 2 * c_h + N + 40                                # both recurrences, the gates and the sums over states
    for key, got in g.items():
        # channels: a tile at a time, then the splits; time: 8 steps, a row's tree, then partials in 32 columns
        more = D // G // 4 + 64 if key in ("gB", "gC") else 64 + B * chunks / 32 if key in ("gA", "gskip", "gdelta_bias") else 0
        want, size = cpu(ref[key])
        close(got, want, c + more, size, key)


# walks over sequences: a workgroup takes several of them, one or many at a time
CONV = {"long_rows": ((5, 2100, 2100, 4), 5), "short_rows": ((300, 2100, 20, 4), 3), "many_taps": ((70, 2100, 70, 13), 5)}


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("name", CONV)
def test_short_conv_backward_walks_over_sequences(name, io):
    (B, D, L, T), _ = CONV[name]
    t, r = TYPES[io], gen(L)
    lengths = ragged(B, L, B)
    x, w, bias = r(B, D, L).to(t), r(D, T) / T ** 0.5, r(D)
    state, gy, gso = r(B, D, T - 1).to(t), r(B, D, L).to(t), r(B, D, T - 1).to(t)
    got = H.short_conv_backward(dev(spoil(x, lengths)), dev(w), dev(spoil(gy, lengths)), dev(bias), silu=True, state=dev(state),
                                lengths=dev(lengths), gstate_out=dev(gso))
    up = lambda v: dev(v).double()  # noqa: E731
    inside = torch.arange(L, device=got[0].device) < dev(lengths).view(B, 1, 1)
    zero = torch.zeros((), dtype=torch.float64, device=got[0].device)
    xe = torch.cat((up(state), torch.where(inside, up(x), zero)), -1)
    tap = lambda j: xe[..., T - 1 - j:T - 1 - j + L]  # noqa: E731
    p = up(bias)[:, None] + sum(up(w)[:, j:j + 1] * tap(j) for j in range(T))
    p_size = up(bias).abs()[:, None] + sum((up(w)[:, j:j + 1] * tap(j)).abs() for j in range(T))
    s = 1 / (1 + torch.exp(-p))
    gp = torch.where(inside, up(gy) * s * (1 + p * (1 - s)), zero)
    # silu' is at most 1.1 and changes by at most half of what p does: p's T + 1 roundings, 14 of its own
    gp_size = torch.where(inside, up(gy).abs() * (1.1 + 0.5 * p_size), zero)
    c = T + 16
    gxe, size = torch.zeros_like(xe), torch.zeros_like(xe)
    for j in range(T):
        gxe[..., T - 1 - j:T - 1 - j + L] += up(w)[:, j:j + 1] * gp
        size[..., T - 1 - j:T - 1 - j + L] += up(w)[:, j:j + 1].abs() * gp_size
    at = (dev(lengths).long().view(B, 1, 1) + torch.arange(T - 1, device=xe.device)).expand(-1, D, -1)
    gxe.scatter_add_(2, at, up(gso))
    size.scatter_add_(2, at, up(gso).abs())
    close(got[0], gxe[..., T - 1:].cpu(), c + T + 2, size[..., T - 1:].cpu(), "gx")
    close(got[3], gxe[..., :T - 1].cpu(), c + T + 2, size[..., :T - 1].cpu(), "gstate")
    # 8 or 16 steps of a lane, again for each word and sequence that it walks over, and 10 of the trees
    more = 16 * (-(-L // 2048) + 1) * CONV[name][1] + 10
    gw = torch.stack([(gp * tap(j)).sum((0, 2)) for j in range(T)], 1)
    gw_size = torch.stack([(gp_size * tap(j).abs()).sum((0, 2)) for j in range(T)], 1)
    close(got[1], gw.cpu(), c + more, gw_size.cpu(), "gw")
    close(got[2], gp.sum((0, 2)).cpu(), c + more, gp_size.sum((0, 2)).cpu(), "gbias")


@pytest.mark.parametrize("io", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,D", [(4500, 40), (5000, 777), (2500, 1030), (1030, 5000), (1500, 8200)])
def test_norm_backward_strides_over_rows(rows, D, io):
    """More rows than workgroups: each adds up several, at every width of the kernels."""
    t, r = TYPES[io], gen(rows + D)
    s, w, gy, gs = r(rows, D).to(t), 1 + 0.2 * r(D), r(rows, D).to(t), r(rows, D).to(t)
    eps = 1e-5
    S, W, g = dev(s).double(), dev(w).double(), dev(gy).double()
    rr = 1 / torch.sqrt((S * S).mean(-1, keepdim=True) + eps)
    gx = rr * (g * W - S * rr * (g * W * S * rr).mean(-1, keepdim=True)) + dev(gs).double()
    got, gw = H.rms_norm_backward(dev(s), dev(w), dev(gy), gs=dev(gs), eps=eps)
    # the counts of test_rms_norm; rows to a workgroup, then partials in 32 columns
    c = (D / 256 + 16) / 2 + 8
    big = rr * (W.abs() * g.abs()).amax(-1, keepdim=True) * 4 + dev(gs).double().abs()
    close(got, gx.cpu(), 4 * c + 16, big.cpu(), "gx")
    close(gw, (g * S * rr).sum(0).cpu(), c + 8 + rows / 1024 + 1 + 32 + 16, (g.abs() * (S * rr).abs()).sum(0).cpu(), "gw")
