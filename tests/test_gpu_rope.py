"""GPU parity: rotary positions against the definition in 64 bits (angles reduced in exact integers)."""
import numpy as np
import pytest
import torch

import attn_reference as R
from bit_quantized_decode_amd import binding as B
from helpers import device

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
EXTREME = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 20, 999_999_937, 12345]


def make(tokens, heads, d, dtype, seed=0, pad=0):
    """[tokens][heads][d] inside rows that are `pad` elements wider."""
    g = torch.Generator().manual_seed(seed)
    return torch.randn(tokens, heads * d + pad, generator=g).to(dtype)[:, :heads * d].unflatten(1, (heads, d))


def check(y, x, pos, table, inverse=False, what=""):
    want, size = R.rope(x.double().numpy(), pos, table.freqs.cpu().numpy(), table.layout == B.NVFP4_ROPE_INTERLEAVED,
                        table.magnitude, inverse)
    got = y.double().cpu().numpy()
    bound = R.ROPE_STEPS * size + HALF_STEP[y.dtype] * np.abs(want) + 1e-38
    err = np.abs(got - want)
    assert (err <= bound).all(), (what, (err / bound).max(), np.argwhere(err > bound)[:4])
    rot = table.rot_dim
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:].to(y.dtype)), what


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,d,rot", [(1, 48, 128, 128), (8, 1, 16, 16), (7, 3, 80, 48), (33, 5, 128, 64),
                                                (129, 2, 256, 256), (65, 1, 64, 0), (5, 7, 192, 176), (300, 11, 96, 96)])
def test_shapes(layout, tokens, heads, d, rot):
    dev = device()
    table = B.rope_table(rot, base=1e6, layout=layout, device=dev)
    rng = np.random.default_rng(tokens)
    pos = np.concatenate([EXTREME, rng.integers(0, 1 << 20, size=tokens)])[:tokens].astype(np.int32)
    p = torch.from_numpy(pos).to(dev)
    for xt in (torch.float32, torch.bfloat16):
        for yt in (torch.float32, torch.bfloat16):
            x = make(tokens, heads, d, xt, seed=d)
            y = B.rope(x.to(dev), p, table, dtype=yt)
            assert y.dtype == yt
            check(y, x, pos, table, what=(xt, yt))


@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("yarn", 8.0, 32768), ("yarn", 64.0, 4096, 32.0, 1.0)])
def test_scalings_strides_and_in_place(scaling):
    dev = device()
    table = B.rope_table(128, base=1e4, scaling=scaling, device=dev)
    assert (table.magnitude > 1) == (scaling is not None and scaling[0] == "yarn")
    pos = np.array(EXTREME + list(range(1000, 1009)), np.int32)
    p = torch.from_numpy(pos).to(dev)
    x = make(len(pos), 6, 128, torch.bfloat16, seed=3, pad=256)
    wide = torch.randn(len(pos), 6 * 128 + 256).to(torch.bfloat16).to(dev)
    rows = wide[:, :768].unflatten(1, (6, 128))
    rows.copy_(x)
    tail = wide[:, 768:].clone()
    y = B.rope(rows, p, table)
    check(y, x, pos, table)
    back = B.rope(rows, p, table, out=rows)
    assert back.data_ptr() == rows.data_ptr() and torch.equal(rows, y)
    assert torch.equal(wide[:, 768:], tail)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_inverse_is_the_gradient(layout):
    """<dy, rope(dx)> = <rope inverse(dy), dx> for the linear map, and differences along dx agree with it."""
    dev = device()
    table = B.rope_table(64, base=1e4, layout=layout, scaling=("yarn", 4.0, 1024), device=dev)
    pos = np.array([0, 3, 4000, 70000, -5], np.int32)
    p = torch.from_numpy(pos).to(dev)
    x, dx, dy = (make(5, 4, 96, torch.float32, seed=s) for s in (1, 2, 3))
    grad = B.rope(dy.to(dev), p, table, inverse=True)
    check(grad, dy, pos, table, inverse=True)
    y0, y1 = B.rope(x.to(dev), p, table), B.rope((x + dx).to(dev), p, table)
    forward = ((y1 - y0).double().cpu() * dy.double()).sum(-1)
    backward = (grad.double().cpu() * dx.double()).sum(-1)
    # Each side: ROPE_STEPS of the summands, for values up to |x| + |dx|, and the rounding of x + dx and y1 - y0.
    scale = (table.magnitude * 2 * dy.abs().double().sum(-1) * (x.abs() + dx.abs()).double().amax(-1)) * (2 * R.ROPE_STEPS + 4 * R.U24)
    assert ((forward - backward).abs() <= scale).all()
    # At magnitude 1 it undoes the turn.
    plain = B.rope_table(64, base=1e4, layout=layout, device=dev)
    z = B.rope(B.rope(x.to(dev), p, plain), p, plain, inverse=True).cpu()
    assert ((z - x).abs() <= 2 * 2 * R.ROPE_STEPS * 2 * x.abs().amax()).all()


def test_no_rows():
    dev = device()
    table = B.rope_table(64, device=dev)
    y = B.rope(torch.empty(0, 4, 64, device=dev), torch.empty(0, dtype=torch.int32, device=dev), table)
    assert y.shape == (0, 4, 64)
