"""The quantised cache on the GPU: codes, scales and layout bit for bit
against the f32 steps and the byte layout that the header defines; reading
back; moving accepted drafts; bad pages, positions and values."""
import numpy as np
import pytest

import decode_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

FMTS = [R.F16, R.Q8, R.Q4]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Setup:
    """Sequences over scattered pages; every cache byte starts as 0xA5."""

    def __init__(self, fmt, heads, dim, new, ctx, seed=0, extra=2):
        self.rng = rng = np.random.default_rng(seed)
        self.new, self.ctx = list(new), list(ctx)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        need = [-(-(n + c) // 64) for n, c in zip(new, ctx)]
        self.pages = sum(need) + extra
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(new), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.ntok = int(self.start[-1])
        nb = kq.KVCache(fmt, heads, dim, 1).page_bytes
        self.cache = kq.KVCache(fmt, heads, dim, self.pages,
                                torch.full((nb * self.pages,), 0xA5, dtype=torch.uint8, device="cuda"))
        self.batch = self.make(self.start, self.ctx)
        self.k, self.v = (rng.standard_normal((self.ntok, heads, dim)).astype(np.float32)
                          for _ in range(2))

    def make(self, start, ctx, table=None, max_new=None):
        return kq.KVBatch(dev(np.asarray(start, np.int32)), dev(np.asarray(ctx, np.int32)),
                          dev(self.table if table is None else table), int(start[-1]),
                          max_new or max(1, max(np.diff(start))))

    def slots(self):
        """(page, token in it) of every new token."""
        return [(self.table[b, (c + j) // 64], (c + j) % 64)
                for b, (n, c) in enumerate(zip(self.new, self.ctx)) for j in range(n)]


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("heads,dim,new,ctx", [
    (1, 64, [1], [0]), (2, 128, [5, 1, 70], [63, 1000, 3]), (3, 256, [16], [1003]),
    (2, 64, [129, 2], [7, 62]), (1, 128, [1, 1, 1], [64, 127, 66])])
def test_append_bits(fmt, heads, dim, new, ctx):
    s = Setup(fmt, heads, dim, new, ctx)
    if fmt != R.F16:  # codes over what 0xA5 bytes stand for
        s.k[0, 0, :32] = 0
        s.v[-1, 0, :32] *= 1e-9
    else:
        s.k[0, 0, 0] = 1e6  # an infinity in f16
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v))
    # the pages before, byte for byte as the layout says, with the new tokens in place
    shape = (s.pages, 64, heads, dim)
    old = {R.F16: np.uint16(0xA5A5), R.Q8: np.int8(0xA5 - 256)}
    if fmt == R.Q4:
        kc = np.tile(np.array([5, -6], np.int8), (s.pages, 64, heads, dim // 2))
        # the values' nibbles alternate from token to token
        vc = np.tile(np.array([5, -6], np.int8)[:, None, None], (s.pages, 32, heads, dim))
    else:
        kc = np.full(shape, old[fmt])
        vc = kc.copy()
    if fmt == R.F16:
        kc, vc = kc.view(np.float16), vc.view(np.float16)
        ks = vs = None
    else:
        ks = np.full((s.pages, 64, heads, dim // 32), np.uint16(0xA5A5)).view(np.float16)
        vs = ks.copy()
    with np.errstate(over="ignore"):
        qk, qv = R.quantise(s.k, fmt), R.quantise(s.v, fmt)
    for i, (p, t) in enumerate(s.slots()):
        kc[p, t], vc[p, t] = qk[0][i], qv[0][i]
        if fmt != R.F16:
            ks[p, t], vs[p, t] = qk[1][i], qv[1][i]
    assert np.array_equal(s.cache.data.cpu().numpy(), R.pack(kc, ks, vc, vs, fmt))
    k, v = kq.kv_read(s.cache, s.batch)
    assert np.array_equal(k.cpu().numpy(), R.values(*qk))
    assert np.array_equal(v.cpu().numpy(), R.values(*qv))
    # what a code stands for is within half a step (Q4: a value at the far end
    # of the range within one) of the value; a scale below 2^-14 is rounded to
    # within 2^-25, which counts as many times as the code
    if fmt != R.F16:
        step = np.repeat(np.abs(qv[1]).astype(float), 32, -1)
        off = np.abs(R.values(*qv).astype(float) - s.v)
        least = 2.0 ** -25 * (127 if fmt == R.Q8 else 8)
        assert (off <= step * (0.5 + 2.0 ** -9 * 127 if fmt == R.Q8 else 1.01) + least).all()


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (64, 24), (256, 128)])
def test_append_rotates_keys(fmt, dim, rot, inter):
    s = Setup(fmt, 2, dim, [9, 66], [5, 62], seed=rot)
    a = s.rng.uniform(0, 6.3, (40, rot // 2))
    table = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)
    pos = s.rng.integers(0, 40, s.ntok).astype(np.int32)
    # keys and values as slices of a fused projection's rows
    qkv = torch.zeros(s.ntok, 7, dim, device="cuda")
    qkv[:, 3:5], qkv[:, 5:7] = dev(s.k), dev(s.v)
    kq.kv_append(s.cache, s.batch, qkv[:, 3:5], qkv[:, 5:7], dev(pos), dev(table), inter)
    k, v = kq.kv_read(s.cache, s.batch)
    want = R.rotate(s.k, pos, table, inter, False, np.float32)
    assert np.array_equal(k.cpu().numpy(), R.values(*R.quantise(want, fmt)))
    assert np.array_equal(v.cpu().numpy(), R.values(*R.quantise(s.v, fmt)))
    pos[1], pos[2] = 40, -1
    kq.kv_append(s.cache, s.batch, qkv[:, 3:5], qkv[:, 5:7], dev(pos), dev(table), inter)
    k2 = kq.kv_read(s.cache, s.batch)[0].cpu().numpy()
    assert np.isnan(k2[1:3, :, :rot // 32 * 32 or rot]).all()
    assert np.array_equal(k2[[0] + list(range(3, s.ntok))], k.cpu().numpy()[[0] + list(range(3, s.ntok))])


@pytest.mark.parametrize("fmt", [R.Q8, R.Q4], ids=R.NAMES.get)
def test_extreme_groups(fmt):
    s = Setup(fmt, 1, 128, [4], [0])
    s.k[:] = 0
    s.k[0, 0, :32] = 3e38          # the scale stops at 65504
    s.k[0, 0, 32], s.k[0, 0, 64], s.k[0, 0, 96] = np.nan, np.inf, -np.inf
    s.k[1, 0, :32] = 1e-38         # the scale rounds to zero
    s.k[2, 0, 5], s.k[2, 0, 6] = 2.0, -2.0   # a tie of magnitudes
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v))
    k = kq.kv_read(s.cache, s.batch)[0].cpu().numpy()
    assert np.array_equal(k, R.values(*R.quantise(s.k, fmt)), equal_nan=True)
    assert np.isnan(k[0, 0, 32:]).all() and (k[1] == 0).all()
    assert k[0, 0, 0] == (127 * 65504.0 if fmt == R.Q8 else 8 * 65504.0)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_bad_pages_and_lengths_touch_nothing(fmt):
    s = Setup(fmt, 2, 64, [3, 70, 2], [62, 10, 5])
    before = s.cache.data.clone()
    table = s.table.copy()
    table[0, 1], table[1, 0] = s.pages, -5        # sequence 0's tokens 64.., 1's first page
    b = s.make(s.start, s.ctx, table)
    kq.kv_append(s.cache, b, dev(s.k), dev(s.v))
    k, v = (x.cpu().numpy() for x in kq.kv_read(s.cache, b))
    want = R.values(*R.quantise(s.k, fmt))
    bad = [i for i, (n, c) in enumerate([(j, c) for n, c in zip(s.new, s.ctx) for j in range(n)])
           if (i < 3 and c + n >= 64) or (3 <= i < 73 and c + n < 64)]
    good = [i for i in range(s.ntok) if i not in bad]
    assert np.isnan(k[bad]).all() and np.isnan(v[bad]).all()
    assert np.array_equal(k[good], want[good])
    # starts that fall or pass the end, a negative ctx, places past the table
    s.cache.data.copy_(before)
    b = kq.KVBatch(dev(np.array([5, 2, 2, 900], np.int32)), dev(np.array([-7, 3, 1 << 30], np.int32)),
                   dev(s.table), s.ntok, 70)
    kq.kv_append(s.cache, b, dev(s.k), dev(s.v))
    out = torch.full((s.ntok, 2, 64), 3.0, device="cuda")
    kq.kv_read(s.cache, b, k=out, v=torch.empty_like(out))
    assert torch.equal(s.cache.data, before)
    assert (out[:2] == 3).all() and torch.isnan(out[2:72]).all() and (out[72:] == 3).all()


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_move(fmt, dim):
    s = Setup(fmt, 2, dim, [9, 4, 40], [60, 3, 100])
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v))
    k0, v0 = kq.kv_read(s.cache, s.batch)
    path = np.full(s.ntok, -1, np.int32)
    path[0:4] = [0, 3, 5, 8]
    path[9:11] = [0, 1]
    path[13:16] = [0, 2, 39]
    count = np.array([4, 2, 3], np.int32)
    kq.kv_move(s.cache, s.batch, dev(path), dev(count))
    k1, v1 = kq.kv_read(s.cache, s.batch)
    src = list(range(s.ntok))
    src[1:4], src[14:16] = [3, 5, 8], [15, 52]
    assert torch.equal(k1, k0[src]) and torch.equal(v1, v0[src])
    # entries that do not rise, or are no new tokens, end the list
    path[0:4], count[:] = [2, 1, 5, 8], [4, 0, 99]
    path[13:16] = [0, 40, 3]
    kq.kv_move(s.cache, s.batch, dev(path), dev(count))
    k2, _ = kq.kv_read(s.cache, s.batch)
    want = k1.clone()
    want[0] = k1[2]
    assert torch.equal(k2, want)


def test_large_offsets():
    """Pages past 4 GiB of cache."""
    heads, dim = 8, 256
    nb = kq.KVCache(kq.KV_F16, heads, dim, 1).page_bytes
    pages = (9 << 29) // nb
    cache = kq.KVCache(kq.KV_F16, heads, dim, pages)
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    b = kq.KVBatch(dev(np.array([0, 70], np.int32)), dev(np.array([61], np.int32)), dev(table), 70, 70)
    x = torch.randn(70, heads, dim, device="cuda").half().float()
    kq.kv_append(cache, b, x, -x)
    k, v = kq.kv_read(cache, b)
    assert torch.equal(k, x) and torch.equal(v, -x)
    assert int(cache.data.view(torch.int64).count_nonzero()) == 2 * 70 * heads * dim // 4 or \
        bool((cache.data[-nb:] != 0).any())


def test_refusals():
    s = Setup(R.Q8, 2, 64, [3], [0])
    with pytest.raises(ValueError):
        kq.KVCache(5, 2, 64, 4)
    with pytest.raises(ValueError):
        kq.KVCache(kq.KV_Q8, 2, 64, 4, data=torch.zeros(7, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kq.kv_append(s.cache, s.batch, dev(s.k[:2]), dev(s.v))
    with pytest.raises(ValueError):
        kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v), table=torch.zeros(4, 4, 2, device="cuda"))
    with pytest.raises(kq.KQError, match="KQ_ERR_NTOK"):
        kq.kv_move(s.cache, s.make([0, 3], [0], max_new=65), dev(np.zeros(3, np.int32)),
                   dev(np.zeros(1, np.int32)))
    pinned = torch.zeros(3, 2, 64).pin_memory()
    with pytest.raises(ValueError):
        kq.kv_append(s.cache, s.batch, pinned, dev(s.v))


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_pages_past_32_bits(fmt):
    """The last pages of a cache of more than 2^32 bytes: written, read back,
    attended by few and by many rows and moved as those of a small one."""
    heads, dim, new, ctx = 16, 128, 8, 130
    each = kq.KVCache(fmt, heads, dim, 1).page_bytes
    gen = torch.Generator(device="cuda").manual_seed(5)
    n = ctx + new

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    k, v = normal(n, heads, dim), normal(n, heads, dim)
    q1, q4 = normal(1, heads, dim), normal(new, 4 * heads, dim)
    path = torch.tensor([0, 2, 5, 6, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    count = torch.tensor([4], dtype=torch.int32, device="cuda")
    out = []
    for pages in (3, (1 << 32) // each + 40):
        cache = kq.KVCache(fmt, heads, dim, pages)
        assert pages == 3 or cache.data.numel() > (1 << 32) + 30 * each

        def batch(held, m):
            return kq.KVBatch(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (
                [0, m], [held], [[pages - 2, pages - 1, pages - 3]])), m, m)

        kq.kv_append(cache, batch(0, n), k, v)
        kept = list(kq.kv_read(cache, batch(0, n)))
        one, many = kq.tree_attention(cache, batch(n - 1, 1), q1), kq.tree_attention(cache, batch(ctx, new), q4)
        kq.kv_move(cache, batch(ctx, new), path, count)
        out.append(kept + [one, many] + list(kq.kv_read(cache, batch(0, n))))
        del cache
    for a, b in zip(*out):
        assert torch.equal(a, b)
    assert torch.isfinite(out[0][2]).all() and torch.isfinite(out[0][3]).all()
    assert not torch.equal(out[0][0], out[0][4])


def test_descriptors_follow_values_and_refuse_other_tensors():
    s = Setup(R.Q8, 2, 64, [3], [10])
    with pytest.raises(AttributeError):
        s.batch.ctx = dev(np.array([20], np.int32))
    with pytest.raises(AttributeError):
        s.batch.ntok = 2  # (the kernels would read three tokens of k and v)
    with pytest.raises(AttributeError):
        s.cache.data = torch.zeros_like(s.cache.data)
    assert s.batch.ntok == 3 and (s.batch.nseq, s.batch.max_new) == (1, 3)
    with pytest.raises(ValueError):
        kq.kv_append(s.cache, s.batch, dev(s.k[:2]), dev(s.v[:2]))
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v))
    want = kq.kv_read(s.cache, s.batch)
    s.batch.ctx.fill_(12)  # values may change
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v))
    got = kq.kv_read(s.cache, s.batch)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    s.batch.ctx.fill_(10)
    assert torch.equal(kq.kv_read(s.cache, s.batch)[0][2], want[0][0])


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 32), (64, 24), (256, 128), (128, 128)])
def test_a_bad_position_stores_a_key_of_nan(fmt, inter, dim, rot):
    """The whole key, as kq_rope gives it, also where a part of it is not
    rotated; its value, and the other tokens, are as ever."""
    s = Setup(fmt, 2, dim, [9, 66], [5, 62], seed=rot)
    a = s.rng.uniform(0, 6.3, (40, rot // 2))
    table = np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)
    pos = s.rng.integers(0, 40, s.ntok).astype(np.int32)
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v), dev(pos), dev(table), inter)
    k, v = (x.cpu().numpy() for x in kq.kv_read(s.cache, s.batch))
    bad = [1, 2, 70]
    pos[bad] = [40, -1, 1 << 30]
    kq.kv_append(s.cache, s.batch, dev(s.k), dev(s.v), dev(pos), dev(table), inter)
    k2, v2 = (x.cpu().numpy() for x in kq.kv_read(s.cache, s.batch))
    assert np.isnan(k2[bad]).all()
    rest = [i for i in range(s.ntok) if i not in bad]
    assert np.array_equal(k2[rest], k[rest]) and np.array_equal(v2, v)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_only_the_sequences_pages_are_written(fmt):
    """Of a cache of more than 4 GiB nothing but the pages that the calls are
    about is touched."""
    heads, dim = 8, 256
    each = kq.KVCache(fmt, heads, dim, 1).page_bytes
    pages = (9 << 29) // each
    cache = kq.KVCache(fmt, heads, dim, pages)
    table = np.array([[pages - 1, 0, pages - 2]], np.int32)
    b = kq.KVBatch(dev(np.array([0, 62], np.int32)), dev(np.array([66], np.int32)), dev(table), 62, 62)
    x = torch.randn(62, heads, dim, device="cuda")
    path = torch.full((62,), -1, dtype=torch.int32, device="cuda")
    path[:4] = torch.tensor([0, 3, 30, 61])
    kq.kv_append(cache, b, x, -x)
    kq.kv_move(cache, b, path, torch.tensor([4], dtype=torch.int32, device="cuda"))
    k, _ = kq.kv_read(cache, b)
    y = kq.tree_attention(cache, b, torch.randn(62, 2 * heads, dim, device="cuda"))
    assert torch.isfinite(y).all() and (k != 0).any()
    held = cache.data.view(pages, each)
    assert (held[0] != 0).any()
    assert not (held[pages - 1] != 0).any() and not (held[pages - 2] != 0).any()
    held[0] = 0  # places 66..127 are the second page's
    assert int(cache.data.view(torch.int64).count_nonzero()) == 0
