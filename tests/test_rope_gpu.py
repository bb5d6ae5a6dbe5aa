"""Rotary positions on the GPU: the table against 64 bits, the rotation bit
for bit against the f32 steps that the header defines (and so within two
roundings of the formula), its inverse as the gradient."""
import numpy as np
import pytest

import decode_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402


def rand_table(n, rot, seed):
    a = np.random.default_rng(seed).uniform(0, 6.3, (n, rot // 2))
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("scaling", [None, "linear", "base", "ramp"])
@pytest.mark.parametrize("positions,rot", [(1, 8), (131072, 64), (1001, 128)])
def test_table(scaling, positions, rot):
    base, factor, orig, fast, slow = 10000.0, 4.0, 2048, 32.0, 1.0
    mag = 1.25 if scaling == "ramp" else 1.0
    got = kq.rope_table(positions, rot, base, scaling=scaling, factor=factor, orig=orig, fast=fast,
                        slow=slow, magnitude=mag).cpu().numpy()
    i = np.arange(rot // 2)
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "ramp":
        turns = orig * f / (2 * np.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        f = f / factor * (1 - keep) + f * keep
    a = np.arange(positions)[:, None] * f
    want = np.stack([np.cos(a), np.sin(a)], -1) * mag
    # one rounding to f32; an angle up to 131072 is off by a few 2^-53 of itself
    assert np.abs(got - want).max() <= mag * (2.0 ** -24 + positions * 2.0 ** -49)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,dim,rot", [(1, 32, 128, 128), (5, 3, 128, 64), (37, 1, 96, 24),
                                             (3, 2, 8, 8), (260, 7, 256, 256), (2, 1, 1024, 16)])
def test_rotation(n, heads, dim, rot, inter, inverse):
    rng = np.random.default_rng(n * dim + rot)
    x = rng.standard_normal((n, heads, dim)).astype(np.float32)
    x[0, 0, :4] = [np.inf, -0.0, 1e38, 1e-40]
    table = rand_table(50, rot, rot)
    pos = rng.integers(0, 50, n).astype(np.int32)
    with np.errstate(all="ignore"):
        want = R.rotate(x, pos, table, inter, inverse, np.float32)
    xd, td, pd = dev(x), dev(table), dev(pos)
    got = kq.rope(xd, pd, td, interleaved=inter, inverse=inverse)
    assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)
    # slices of a wider row, in and out, and in place
    wide = torch.full((n, (heads + 2) * dim), 7.0, device="cuda")
    cut = wide[:, dim:(heads + 1) * dim].view(n, heads, dim) if n == 1 else \
        wide.view(n, heads + 2, dim)[:, 1:heads + 1]
    cut.copy_(xd)
    kq.rope(cut, pd, td, interleaved=inter, inverse=inverse, out=cut)
    assert np.array_equal(cut.cpu().numpy(), want, equal_nan=True)
    rest = wide.view(n, heads + 2, dim)
    assert (rest[:, 0] == 7).all() and (rest[:, -1] == 7).all()


def test_positions_outside_the_table_give_nan():
    x, table = torch.ones(4, 2, 64, device="cuda"), dev(rand_table(10, 32, 1))
    y = kq.rope(x, dev(np.array([0, 10, -1, 9], np.int32)), table).cpu()
    assert torch.isnan(y[1:3]).all() and not torch.isnan(y[[0, 3]]).any()
    assert kq.rope(x[:0], dev(np.zeros(0, np.int32)), table).shape == (0, 2, 64)


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(inter):
    rng = np.random.default_rng(5)
    n, heads, dim, rot = 9, 4, 128, 64
    x, g, e = (rng.standard_normal((n, heads, dim)).astype(np.float32) for _ in range(3))
    table, pos = rand_table(30, rot, 2), rng.integers(0, 30, n).astype(np.int32)
    td, pd = dev(table), dev(pos)
    grad = kq.rope(dev(g), pd, td, interleaved=inter, inverse=True).cpu().numpy().astype(float)
    want = R.rotate(g, pos, table, inter, True)
    # two products and a sum: three roundings of at most |a| + |b|
    assert np.abs(grad - want).max() <= 3 * 2.0 ** -24 * 2 * np.abs(g).max()
    # differences of the kernel itself along e: linear, so only rounding is left
    up, dn = (kq.rope(dev(x + s * e), pd, td, interleaved=inter).cpu().numpy().astype(float)
              for s in (np.float32(1), np.float32(-1)))
    diff = ((up - dn) / 2 * g).sum()
    size = (np.abs(x) + np.abs(e)).max()
    assert abs(diff - (grad * e).sum()) <= 8 * 2.0 ** -24 * size * np.abs(g).sum() * 2


def test_refusals_and_streams():
    x, table = torch.ones(4, 2, 64, device="cuda"), dev(rand_table(10, 32, 1))
    pos = dev(np.arange(4, dtype=np.int32))
    with pytest.raises(ValueError):
        kq.rope(x, pos.long(), table)
    with pytest.raises(ValueError):
        kq.rope(x.transpose(0, 1), pos[:2], table)
    with pytest.raises(ValueError):
        kq.rope(x.half(), pos, table)
    with pytest.raises(kq.KQError, match="KQ_ERR_SHAPE"):
        kq.rope(x[..., :16].contiguous(), pos, table)
    with pytest.raises(kq.KQError, match="KQ_ERR_ALIAS"):
        buf = torch.ones(5, 2, 64, device="cuda")
        kq.rope(buf[:4], pos, table, out=buf[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = kq.rope(x, pos, table, stream=side)
    side.synchronize()
    assert torch.equal(y, kq.rope(x, pos, table))
