"""The layer's activation between its two products, value by value: the down product takes differences
of channels that are nearly alike, so that what rounding the output leaves visible is the activation's
own rounding.

Bounds: a value keeps 10 bits (2^-10 of it), and next to a larger one of its 8 not less than a step of
fp16's least numbers without their last bit, 2^-23 + 2^-25 where the largest is 2^14 and more: 2^-36 of
it covers that.  For 8-bit weights it is brought to fp16 once more beside the largest of 128, twice off
by at most 2^-25 where that is 2^14 and more: 2^-38 of it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_moe_layer import F8, Layer  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    mlg.mlg_read_device_errors(clear=True)
    yield
    torch.cuda.synchronize()
    assert mlg.mlg_read_device_errors(clear=True) == 0


def _largest(v, of):
    """The largest of each run of `of` values, beside each of them."""
    n = v.shape[-1]
    padded = np.zeros(-(-n // of) * of)
    padded[:n] = v
    return np.repeat(padded.reshape(-1, of).max(1), of)[:n]


def _pairs(layer, seed):
    """Channels 2 i and 2 i + 1 alike but for a few of the up rows' weights, and down rows that take
    their difference."""
    g = torch.Generator().manual_seed(seed)
    E, inter, H = layer.E, layer.inter, layer.H
    w = layer.gate_up.float().cpu().view(E, 2, inter // 2, 2, H)
    w[:, :, :, 1] = w[:, :, :, 0]
    w[:, 1, :, 1, :4] *= 1 + torch.rand(E, inter // 2, 4, generator=g) / 8
    layer.gate_up = w.view(E, 2 * inter, H).to(layer.gate_up.dtype).cuda()
    down = torch.zeros(E, H, inter)
    for r in range(H):
        down[:, r, 2 * r % inter], down[:, r, (2 * r + 1) % inter] = 1, -1
    layer.down = down.to(layer.down.dtype).cuda()
    if layer.f8:
        layer.down_scales.fill_(1.0)


def _exact(layer, eight_bits):
    """(out, bound) in 64 bits; with eight_bits, out of activations rounded to bf16."""
    up, down = layer.values()
    x = layer.x.double().cpu().numpy()
    idx, w, bound = operator_refs.route(layer.logits.double().cpu().numpy(), layer.K, layer.renorm)
    out, err = np.zeros((layer.T, layer.H)), np.zeros((layer.T, layer.H))
    for t in range(layer.T):
        for j, e in enumerate(idx[t]):
            h, most = up[e] @ x[t], np.abs(up[e]) @ np.abs(x[t])
            dh = operator_refs.sum_bound(layer.H + 4 * refs.blocks(layer.H), most)
            # hidden states beside 8-bit weights: fp16, off by half its least number, 2^-25, where the
            # largest is 2^14 and more
            dh = dh + 2.0 ** -39 * np.abs(up[e]).sum(1) * np.abs(x[t]).max()
            g, u = np.split(h, 2)
            dg, du = np.split(dh, 2)
            silu = g / (1 + np.exp(-g))
            a = silu * u
            da = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + refs.ACT_REL * np.abs(a)
            size = np.abs(a) + da
            da = da + 2.0 ** -10 * size + 2.0 ** -36 * _largest(size, 8) + 2.0 ** -38 * _largest(size, 128)
            if eight_bits:
                a = torch.from_numpy(a).to(torch.bfloat16).double().numpy()
            mag = np.abs(down[e]) @ size
            out[t] += w[t, j] * (down[e] @ a)
            err[t] += w[t, j] * (np.abs(down[e]) @ da
                                 + operator_refs.sum_bound(layer.inter * layer.K + 64, mag))
            err[t] += (bound[t, j] + 2 * refs.U * w[t, j]) * mag
    return out, err


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,E,K,H,inter", [(1, 4, 1, 64, 128), (5, 4, 1, 128, 256), (16, 6, 2, 96, 192),
                                           (64, 3, 2, 208, 416)])
def test_ten_bits_of_every_value(T, E, K, H, inter, f8):
    layer = Layer(T, E, K, H, inter, f8, T + H)
    _pairs(layer, T)
    layer.run()
    ref, err = _exact(layer, False)
    operator_refs.assert_within(layer.out[:T].double().cpu().numpy(), ref, err, True, "out")
    assert (layer.act[-1] == 77).all()
    # the bound would show an activation of 8 bits
    coarse, _ = _exact(layer, True)
    if T > 1:
        assert (np.abs(coarse - ref) > err + 2.0 ** -8 * np.abs(ref)).any()


def test_values_far_below_their_neighbours():
    """Two channels of each 16 are 2^20 times the others (2^6 in 8 bits): those keep their bits as far
    as fp16 reaches beside them."""
    for f8 in (False, True):
        layer = Layer(6, 2, 1, 64, 128, f8, 3)
        _pairs(layer, 4)
        w = layer.gate_up.float().cpu().view(2, 2, 128, 64)
        if f8:  # by a whole block's scale: channels 0 to 127 of up, whose x is the same
            w[:, 1] /= 2.0 ** 6
            w[:, 1, ::16], w[:, 1, 1::16] = w[:, 1, ::16] * 2.0 ** 6, w[:, 1, 1::16] * 2.0 ** 6
        else:
            w[:, 1] *= 2.0 ** -20
            w[:, 1, ::16], w[:, 1, 1::16] = w[:, 1, ::16] * 2.0 ** 20, w[:, 1, 1::16] * 2.0 ** 20
        layer.gate_up = w.view(2, 256, 64).to(layer.gate_up.dtype).cuda()
        layer.run()
        ref, err = _exact(layer, False)
        operator_refs.assert_within(layer.out[:6].double().cpu().numpy(), ref, err, True, "out")


@pytest.mark.parametrize("f8", [False, True])
def test_groups_far_below_the_largest_of_their_block(f8):
    """Eight channels of a block of 128 are 2^10 to 2^70 times the others, which the down product
    takes alone.  All products are of small integers, so that gates and ups are exact."""
    T, H, inter = 4, 128, 128
    layer = Layer(T, 1, 1, H, inter, f8, 1)
    x = torch.tensor([0.5, 0.75, 1.0, 1.5]).view(T, 1)
    layer.x = x.expand(T, H).to(torch.bfloat16).contiguous().cuda()
    channel = torch.arange(inter)
    gate = torch.where(channel < 8, 448.0, -16.0 - 2 * (channel // 8 % 8))
    up = 1.0 + channel % 5
    w = torch.cat([gate, up]).view(1, 2 * inter, 1).expand(1, 2 * inter, H)
    down = torch.eye(inter).view(1, H, inter).clone()
    down[:, :8] = 0
    if f8:
        layer.gate_up, layer.down = w.to(F8).cuda(), down.to(F8).cuda()
        layer.gate_up_scales.fill_(1 / H)
        layer.down_scales.fill_(1.0)
    else:
        layer.gate_up, layer.down = (w / H).to(torch.bfloat16).cuda(), down.to(torch.bfloat16).cuda()
    layer.run()
    g, u = (v.double().numpy() * x.double().numpy() for v in (gate, up))
    a = g / (1 + np.exp(-g)) * u
    err = (2.0 ** -10 + refs.ACT_REL) * np.abs(a)
    err = err + np.stack([2.0 ** -36 * _largest(np.abs(v), 8) for v in a])
    if f8:
        err = err + np.stack([2.0 ** -38 * _largest(np.abs(v), 128) for v in a])
    a[:, :8], err[:, :8] = 0, 0
    operator_refs.assert_within(layer.out[:T].double().cpu().numpy(), a, err, True, "out")
