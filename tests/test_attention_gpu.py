"""Attention of new tokens over the paged cache, against the formula in 64
bits with the error bound that decode_ref.attention derives: every format,
head layout and width, lengths from one token on, masks that leave a row
empty, NaN and infinities in masked places, bad pages, long offsets."""
import numpy as np
import pytest

import decode_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

FMTS = [R.F16, R.Q8, R.Q4]


@pytest.fixture(autouse=True)
def no_expired_wait():
    """Every wait inside the kernels is bounded; none may have run out."""
    yield
    assert not kq.device_error()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """Sequences whose every place has been appended; k and v as the cache
    holds them, per sequence."""

    def __init__(self, fmt, hkv, g, dim, new, ctx, masks=None, seed=0, spread=1.0, garbage=0xFF,
                 first_page=0, pages=None):
        self.rng = rng = np.random.default_rng(seed)
        self.new, self.ctx, self.fmt, self.dim = list(new), list(ctx), fmt, dim
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.ntok = int(self.start[-1])
        need = [-(-(n + c) // 64) for n, c in zip(new, ctx)]
        self.pages = pages or sum(need) + 2
        order = first_page + rng.permutation(sum(need) + 2).astype(np.int32)
        self.table = np.full((len(new), max(max(need), 1)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        nb = kq.KVCache(fmt, hkv, dim, 1).page_bytes
        data = torch.full((nb * self.pages,), garbage, dtype=torch.uint8, device="cuda")
        self.cache = kq.KVCache(fmt, hkv, dim, self.pages, data)
        self.hq = hkv * g
        self.q = (spread * rng.standard_normal((self.ntok, self.hq, dim))).astype(np.float32)
        # all places are written through a batch whose new tokens they are
        total = [n + c for n, c in zip(new, ctx)]
        starts = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
        n = int(starts[-1])
        self.k, self.v = (rng.standard_normal((n, hkv, dim)).astype(np.float32) for _ in range(2))
        self.starts = starts
        self.whole = kq.KVBatch(dev(starts), dev(np.zeros(len(new), np.int32)), dev(self.table), n,
                                max(total))
        self.batch = kq.KVBatch(dev(self.start), dev(np.asarray(ctx, np.int32)), dev(self.table),
                                self.ntok, max(new))
        if masks is None:  # random sets of the sequence's own new tokens
            masks = [int(rng.integers(0, 1 << min(m, 62))) | 1 << j
                     for m in new for j in range(m)]
        self.masks = masks
        self.write()

    def write(self):
        kq.kv_append(self.cache, self.whole, dev(self.k), dev(self.v))

    def mask(self):
        return dev(np.array([m - (1 << 64) if m >> 63 else m for m in self.masks], np.int64))

    def run(self, **kw):
        kw.setdefault("mask", self.mask())
        return kq.tree_attention(self.cache, self.batch, dev(self.q), **kw)

    def want(self, masks=None, scale=None):
        masks = self.masks if masks is None else masks
        ks, vs = (R.values(*R.quantise(x, self.fmt)) for x in (self.k, self.v))
        outs, bounds = [], []
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            lo, hi = self.starts[b], self.starts[b + 1]
            seen = np.ones((n, n + c), bool)
            for i in range(n):
                for j in range(n):
                    seen[i, c + j] = masks[self.start[b] + i] >> j & 1
            o, e = R.attention(self.q[self.start[b]:self.start[b] + n], ks[lo:hi], vs[lo:hi], seen,
                               self.dim ** -0.5 if scale is None else scale)
            outs.append(o)
            bounds.append(e)
        return np.concatenate(outs), np.concatenate(bounds)

    def check(self, got, want=None):
        out, bound = self.want() if want is None else want
        off = np.abs(got.cpu().numpy().astype(float) - out)
        assert np.isfinite(off).all()
        assert (off <= bound).all(), (float((off / np.maximum(bound, 1e-30)).max()))


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("hkv,g,new,ctx", [
    (1, 1, [1], [0]), (2, 16, [1], [777]), (2, 4, [5, 1, 3], [63, 64, 0]),
    (1, 8, [16], [1]), (3, 5, [7, 2], [190, 65]), (1, 16, [17], [300]), (8, 1, [1, 1], [62, 511])])
def test_against_64_bits(fmt, dim, hkv, g, new, ctx):
    c = Case(fmt, hkv, g, dim, new, ctx, seed=dim + g)
    got = c.run()
    c.check(got)
    assert torch.equal(got, c.run())  # the same bits again


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("hkv,g,new,ctx", [
    (1, 1, [64], [0]), (1, 4, [64, 33], [31, 64]), (1, 16, [64], [100]), (2, 7, [61], [3])])
def test_many_new_tokens(fmt, hkv, g, new, ctx):
    c = Case(fmt, hkv, g, 128, new, ctx, seed=g)
    c.check(c.run())
    causal = [(2 << j) - 1 for n in new for j in range(n)]
    c.check(c.run(mask=None), c.want(causal))


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_long_and_ragged(fmt):
    c = Case(fmt, 2, 4, 128, [2, 1, 4, 1, 1, 3], [9000, 1, 4097, 0, 2999, 640], seed=3, spread=4.0)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("g,new", [(17, 1), (8, 4), (11, 3), (16, 4), (13, 5), (16, 8), (43, 3)])
def test_many_rows(fmt, dim, g, new):
    """17..129 rows a key head, blocks of 32, 64 and 128: one sequence whose
    pages are shared by CTAs, one of a few, one with nothing committed."""
    c = Case(fmt, 2, g, dim, [new, new, 1], [1500, 130, 0], seed=g)
    got = c.run()
    c.check(got)
    assert torch.equal(got, c.run())


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g,new", [(9, 1), (3, 4), (2, 6), (13, 1)])
def test_some_rows(fmt, dim, g, new):
    """9..13 rows a key head, tiles of four rows that are full and that are not."""
    c = Case(fmt, 2, g, dim, [new, 1, new], [1500, 0, 129], seed=g)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("g,new", [(4, 1), (8, 1), (16, 1), (5, 5), (12, 5), (16, 6)])
def test_many_pages_a_cta(fmt, g, new):
    """Enough pages that every ring goes round several times."""
    c = Case(fmt, 1, g, 64, [new], [150000], seed=g, spread=3.0)
    c.q[:, 1:] = c.q[:, :1]  # (the reference takes one head's time)
    got = c.run()
    assert torch.equal(got, got[:, :1].expand_as(got))
    c.q, c.hq = c.q[:, :1], 1
    c.check(got[:, :1])


def test_a_batch_of_many_sequences():
    rng = np.random.default_rng(8)
    new, ctx = rng.integers(0, 4, 300).tolist(), rng.integers(0, 200, 300).tolist()
    new[0] = 3
    c = Case(R.Q8, 1, 4, 64, new, ctx, seed=9)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
def test_empty_rows_are_zero(fmt):
    c = Case(fmt, 2, 4, 128, [3, 2], [0, 5], masks=[0, 1, 0, 0, 0])
    got = c.run()
    assert (got[0] == 0).all() and (got[2] == 0).all()
    c.check(got)
    # bits beyond the sequence's own new tokens say nothing
    c.masks = [~0 << 3 & (1 << 64) - 1, ~0 << 3 & (1 << 64) - 1 | 1, ~0 << 3 & (1 << 64) - 1,
               1 << 63, 1 << 2]
    assert torch.equal(c.run(), got)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx", [0, 61, 130])
def test_masked_places_do_not_reach_any_of_many_rows(fmt, bad, ctx):
    """The same with 48 rows a key head."""
    test_masked_places_do_not_reach_a_row(fmt, bad, ctx, g=8)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("g", [1, 2])
def test_masked_places_do_not_reach_any_of_few_rows(fmt, g):
    """The same with 6 and 12 rows a key head."""
    for ctx in (0, 61):
        test_masked_places_do_not_reach_a_row(fmt, float("nan"), ctx, g=g)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx", [0, 61, 130])
def test_masked_places_do_not_reach_a_row(fmt, bad, ctx, g=4):
    """New token 2's key and value hold a NaN or an infinity; rows that attend
    it show it, others are as without it."""
    c = Case(fmt, 1, g, 128, [6], [ctx], masks=[1, 3, 7, 9, 17, 37], seed=4)
    clean = c.run()
    c.k[ctx + 2, 0, 3], c.v[ctx + 2, 0, 40] = bad, bad
    c.write()
    got = c.run()
    sees = [2, 5]
    others = [0, 1, 3, 4]
    assert torch.equal(got[others], clean[others])
    assert torch.isnan(got[sees]).any(-1).all()
    # the value alone: only the places of its own scale group (f16: itself)
    c.k[ctx + 2, 0, 3] = 0.25
    c.write()
    got = c.run().cpu()
    hit = torch.zeros(128, dtype=torch.bool)
    hit[40 if fmt == R.F16 else slice(32, 64)] = True
    if fmt == R.F16:
        assert (~torch.isfinite(got[sees][..., hit])).all()
        if bad == bad:
            assert (got[sees][..., hit] == bad).all()
    else:
        assert torch.isnan(got[sees][..., hit]).all()
    assert torch.isfinite(got[sees][..., ~hit]).all()
    assert torch.isfinite(got[others]).all()


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("g", [2, 20])
def test_extreme_logits(fmt, g):
    c = Case(fmt, 1, g, 64, [2], [200], seed=6, spread=3000.0)
    c.check(c.run())
    c.q[:] = 0
    c.check(c.run())
    c.q[:] = 1e-30
    c.check(c.run())
    c.q[0, 0, 5], c.q[1, 1, 7] = np.nan, np.inf
    got = c.run()
    assert torch.isnan(got[0, 0]).all() and torch.isnan(got[1, 1]).all()
    assert torch.isfinite(got[0, 1]).all() and torch.isfinite(got[1, 0]).all()


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("g", [4, 20])
def test_bad_pages(fmt, g):
    c = Case(fmt, 2, g, 64, [2, 1], [150, 150], masks=[1, 2, 1])
    good = c.run()
    table = c.table.copy()
    table[0, 1] = c.pages
    b = kq.KVBatch(c.batch.start, c.batch.ctx, dev(table), c.ntok, 2)
    got = kq.tree_attention(c.cache, b, dev(c.q), mask=c.mask())
    assert torch.isnan(got[:2]).all() and torch.equal(got[2], good[2])
    # places past the table's end; lengths that are no lengths
    b = kq.KVBatch(dev(np.array([0, 2, 9], np.int32)), dev(np.array([-3, 1 << 30], np.int32)),
                   dev(c.table), c.ntok, 2)
    out = torch.full((c.ntok, 2 * g, 64), 5.0, device="cuda")
    kq.tree_attention(c.cache, b, dev(c.q), mask=c.mask(), out=out)
    assert torch.isfinite(out[:2]).all() and torch.isnan(out[2]).all()
    # a token of no sequence is left alone
    b = kq.KVBatch(dev(np.array([0, 1, 1], np.int32)), c.batch.ctx, dev(c.table), c.ntok, 2)
    out.fill_(5.0)
    kq.tree_attention(c.cache, b, dev(c.q), mask=c.mask(), out=out)
    assert (out[1:] == 5).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("dim", [64, 256])
def test_masked_bad_page_is_not_attended(dim):
    c = Case(R.Q8, 1, 4, dim, [40], [50], masks=[1] * 40, seed=2)
    good = c.run()
    table = c.table.copy()
    table[0, 1] = -1  # new tokens 14.. : none of them is attended
    b = kq.KVBatch(c.batch.start, c.batch.ctx, dev(table), c.ntok, 40)
    assert torch.equal(kq.tree_attention(c.cache, b, dev(c.q), mask=c.mask()), good)


def test_large_offsets():
    hkv, dim = 8, 256
    nb = kq.KVCache(kq.KV_F16, hkv, dim, 1).page_bytes
    pages = (9 << 29) // nb
    c = Case(R.F16, hkv, 2, dim, [2], [700], first_page=pages - 14, pages=pages, garbage=0)
    c.check(c.run())


def test_strides_scale_out_and_workspace():
    c = Case(R.Q4, 2, 4, 128, [3, 2], [700, 90], seed=11)
    want = c.run()
    wide = torch.zeros(c.ntok, c.hq + 4, 128, device="cuda")
    wide[:, 2:2 + c.hq] = dev(c.q)
    out = torch.empty_like(want)
    ws = torch.full((kq.attention_workspace_bytes(c.cache, c.batch, c.hq) + 256,), 0xFF,
                    dtype=torch.uint8, device="cuda")
    got = kq.tree_attention(c.cache, c.batch, wide[:, 2:2 + c.hq], mask=c.mask(), out=out,
                            workspace=ws)
    assert got is out and torch.equal(got, want)
    c.check(c.run(scale=0.7), c.want(scale=0.7))
    c.check(c.run(scale=-0.3), c.want(scale=-0.3))
    c.check(c.run(scale=0.0), c.want(scale=0.0))
    d = Case(R.Q8, 1, 24, 128, [2], [200], seed=14)  # many rows
    d.check(d.run(scale=-0.3), d.want(scale=-0.3))
    d.check(d.run(scale=0.0), d.want(scale=0.0))
    need = kq.attention_workspace_bytes(c.cache, c.batch, c.hq)
    if need:
        with pytest.raises(kq.KQError, match="KQ_ERR_LIMIT"):
            c.run(workspace=ws[:need - 1])


def test_graph_serves_a_growing_sequence():
    c = Case(R.Q8, 2, 8, 128, [2, 2], [500, 40], seed=12)
    ws = torch.empty(max(256, kq.attention_workspace_bytes(c.cache, c.batch, c.hq)),
                     dtype=torch.uint8, device="cuda")
    q, m, out = dev(c.q), c.mask(), torch.empty(c.ntok, c.hq, 128, device="cuda")
    kq.tree_attention(c.cache, c.batch, q, mask=m, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.tree_attention(c.cache, c.batch, q, mask=m, out=out, workspace=ws)
    for ctx in ([500, 40], [130, 0], [64, 39]):
        c.batch.ctx.copy_(dev(np.asarray(ctx, np.int32)))
        out.zero_()
        graph.replay()
        assert torch.equal(out, c.run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, out)


@pytest.mark.parametrize("g", [4, 24])
def test_an_expired_wait_is_reported(g):
    """With a limit far below the time a page takes to arrive the call reports
    it, gives NaN where it shows, and the next call is as always."""
    c = Case(R.F16, 4, g, 128, [2], [60000], seed=15)
    want = c.run()
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    torch.cuda.synchronize()
    lib.kq_set_wait_limit_ns(1)
    try:
        # (a page may come before its first test: then nothing expires)
        got = c.run()
        torch.cuda.synchronize()
    finally:
        lib.kq_set_wait_limit_ns(0)
    expired = kq.device_error()
    same = (got == want) | torch.isnan(got)
    assert same.all()
    assert torch.isnan(got).any() == expired
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("g,new", [(4, 1), (16, 2), (16, 4), (16, 8)])
def test_an_expired_wait_in_each_kernel(fmt, g, new):
    """The same for few rows and for one, two and four warps of rows; NaN only
    where the wait ran out, and nothing of it stays."""
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    c = Case(fmt, 2, g, 128, [new], [40000], seed=16)
    want = c.run()
    torch.cuda.synchronize()
    lib.kq_set_wait_limit_ns(1)
    try:
        got = c.run()
        torch.cuda.synchronize()
    finally:
        lib.kq_set_wait_limit_ns(0)
    expired = kq.device_error()
    assert ((got == want) | torch.isnan(got)).all()
    assert torch.isnan(got).any() == expired
    assert torch.equal(c.run(), want)


def test_refusals():
    c = Case(R.Q8, 2, 4, 64, [3], [10])
    with pytest.raises(ValueError):
        kq.tree_attention(c.cache, c.batch, dev(c.q)[:2])
    with pytest.raises(ValueError):
        kq.tree_attention(c.cache, c.batch, dev(c.q), mask=c.mask().int())
    with pytest.raises(kq.KQError, match="KQ_ERR_SHAPE"):
        kq.tree_attention(c.cache, c.batch, dev(c.q)[:, :7].contiguous())
    with pytest.raises(kq.KQError, match="KQ_ERR_ALIAS"):
        x = dev(c.q)
        kq.tree_attention(c.cache, c.batch, x, out=x)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("hkv,g,new,ctx,dim", [
    (1, 4, [1], [64 * 152 - 1], 64), (1, 4, [1], [64 * 152], 64), (2, 8, [3], [64 * 300 + 7], 64),
    (4, 1, [1] * 8, [2000, 0, 3000, 64, 1, 4000, 700, 63], 64), (1, 20, [2, 1], [64 * 200, 64 * 90], 128)])
def test_few_items_cut_by_themselves(fmt, hkv, g, new, ctx, dim):
    """Pages of few items, about as many as CTAs and some more: runs of one
    item's pages, of lengths that differ by one."""
    c = Case(fmt, hkv, g, dim, new, ctx, seed=hkv + g, spread=2.0)
    c.check(c.run())


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("nseq,hkv,most", [(116, 4, 200), (116, 4, 900), (160, 4, 600)])
def test_many_items(fmt, nseq, hkv, most):
    """More items than SMs have: groups in CTAs of their own, items cut by
    themselves or not."""
    ctx = [(37 * b * b + 11 * b) % most for b in range(nseq)]
    c = Case(fmt, hkv, 2, 64, [1 + b % 2 for b in range(nseq)], ctx, seed=nseq)
    c.check(c.run())


def _expire(c, tries=8):
    """The case's call with a limit far below the time a page takes to arrive,
    over data that is not in L2: rows are NaN where a wait ran out, else as
    always, the call ends at once, and nothing of it stays.  Returns how often
    a wait ran out."""
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    want = c.run()
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    q, mask, out = dev(c.q), c.mask(), torch.empty_like(want)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    times = 0
    for _ in range(tries):
        flush.fill_(1)
        out.fill_(5.0)
        torch.cuda.synchronize()
        lib.kq_set_wait_limit_ns(1)
        try:
            ends[0].record()
            kq.tree_attention(c.cache, c.batch, q, mask=mask, out=out)
            ends[1].record()
            torch.cuda.synchronize()
        finally:
            lib.kq_set_wait_limit_ns(0)
        expired = kq.device_error()
        times += expired
        assert ends[0].elapsed_time(ends[1]) < 1000.0
        assert ((out == want) | torch.isnan(out)).all()
        assert torch.isnan(out).any() == expired
        for _ in range(2):  # the same SMs again, at once
            assert torch.equal(c.run(), want)
    return times


def _many_segments(fmt, g, dim, nseq=600, most=900):
    """A batch of which each CTA has several items, some of them of one page."""
    ctx = [(37 * b * b + 11 * b) % most for b in range(nseq)]
    return Case(fmt, 2, g, dim, [1 + b % 2 for b in range(nseq)], ctx, seed=18)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim,g", [(64, 2), (128, 4), (128, 7), (256, 8)])
def test_expired_waits_with_few_rows(fmt, dim, g):
    _expire(Case(fmt, 2, g, dim, [2], [40000], seed=19))
    _expire(_many_segments(fmt, g, dim))


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim,g", [(64, 20), (128, 20), (128, 50), (64, 100), (128, 100)])
def test_expired_waits_in_batches_of_many_rows(fmt, dim, g):
    """Blocks of 32, 64 and 128 rows, and several items a CTA: those after
    the one whose wait ran out wait for nothing."""
    _expire(_many_segments(fmt, g, dim, nseq=300, most=300))


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim,g", [(64, 20), (128, 10), (128, 50), (64, 100), (128, 100)])
def test_expired_waits_with_many_rows(fmt, dim, g):
    """One item's pages in every CTA: its copies and MMAs end with the call
    (the next one takes the same shared and tensor memory at once)."""
    _expire(Case(fmt, 2, g, dim, [2], [30000], seed=20))


@pytest.mark.parametrize("g", [4, 20])
def test_the_limit_is_a_waits_not_the_calls(g):
    """A call whose items take several times the limit each, no wait of which
    is long: nothing expires.  (One page stands for all 800000 of a sequence.)"""
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    nseq, hkv = 4, torch.cuda.get_device_properties(0).multi_processor_count // 4
    pages = 800000 if g == 4 else 100000
    cache = kq.KVCache(kq.KV_Q4, hkv, 64, 1)
    one = kq.KVBatch(dev(np.array([0, 64], np.int32)), dev(np.zeros(1, np.int32)),
                     dev(np.zeros((1, 1), np.int32)), 64, 64)
    gen = torch.Generator(device="cuda").manual_seed(21)
    kq.kv_append(cache, one, *(torch.randn(64, hkv, 64, generator=gen, device="cuda") for _ in range(2)))
    batch = kq.KVBatch(dev(np.arange(nseq + 1, dtype=np.int32)),
                       dev(np.full(nseq, 64 * pages - 1, np.int32)),
                       torch.zeros(nseq, pages, dtype=torch.int32, device="cuda"), nseq, 1)
    q = torch.randn(nseq, hkv * g, 64, generator=gen, device="cuda")
    want = kq.tree_attention(cache, batch, q)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda.synchronize()
    lib.kq_set_wait_limit_ns(20 * 10 ** 6)
    try:
        ends[0].record()
        got = kq.tree_attention(cache, batch, q)
        ends[1].record()
        torch.cuda.synchronize()
    finally:
        lib.kq_set_wait_limit_ns(0)
    assert ends[0].elapsed_time(ends[1]) > 60.0  # ms
    assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim,g", [(64, 2), (128, 4), (128, 7), (256, 8), (64, 20), (128, 10),
                                   (128, 20), (128, 50), (64, 100), (128, 100)])
def test_a_short_limit_is_kept(fmt, dim, g):
    """1 ns is shorter than any page takes: each kernel's waits do run out,
    where CTAs have one item of many pages and where they have several."""
    c = Case(fmt, 2, g, dim, [2], [62], seed=22)
    pages = 20000  # one page stands for all of them
    c.batch = kq.KVBatch(dev(c.start), dev(np.array([64 * pages - 2], np.int32)),
                         dev(np.full((1, pages), c.table[0, 0], np.int32)), 2, 2)
    assert _expire(c, tries=3) == 3
    c = Case(fmt, 2, g, dim, [1] * 200, [63] * 200, seed=23)
    c.batch = kq.KVBatch(dev(c.start), dev(np.full(200, 64 * 200 - 1, np.int32)),
                         dev(np.repeat(c.table, 200, 1)), 200, 1)
    assert _expire(c, tries=3) == 3


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("by", ["query", "scale"])
@pytest.mark.parametrize("top", [2.0 ** 24 + 10, 2.0 ** 25 + 4, 1e8, 2.0 ** 27, 3e9, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_past_24_bits(fmt, dim, by, top, sign, g=2):
    """Finite logits (in units of log 2) that f32 holds in steps of 2 and
    more: the row is the mean of the values at its largest logit, of which
    three are the same to the bit, in three pages.

    Queries and keys have one factor of a logit that is not zero, so equal
    keys give equal logits, whatever their size, and the other logits are
    smaller by half the largest: their probabilities are 0 in f32.  What is
    left of the error is the sums', as decode_ref.attention derives it with
    logits that are exact."""
    c = Case(fmt, 2, g, dim, [2], [200], seed=17)
    at = [5, 70, 130]
    c.k[..., 0] = 0.5 if sign > 0 else 1.0
    c.k[..., 1:] *= 0.01
    c.k[at, :, 0] = 1.0 if sign > 0 else 0.5
    c.write()
    big = sign * top / 1.4427 / (1.0 if sign > 0 else 0.5)
    c.q[:] = 0
    c.q[..., 0] = big if by == "query" else 1.0
    got = c.run(scale=1.0 if by == "query" else big, mask=None).cpu().numpy().astype(float)
    v = R.values(*R.quantise(c.v, fmt)).astype(float)
    want, size = (np.repeat(f(v)[at].mean(0), g, 0) for f in (np.asarray, np.abs))
    bound = size * (2 * 2.0 ** -21 + (64 + 4 + 304) * 2.0 ** -22) + 202 * 2.0 ** -38 * np.abs(v).max()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("g", [10, 30, 60])
@pytest.mark.parametrize("top", [2.0 ** 24 + 10, 2.0 ** 25 + 4, 1e8, 2.0 ** 27, 3e9, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
def test_logits_past_24_bits_in_many_rows(fmt, dim, top, sign, g):
    """The same with 20, 60 and 120 rows a key head."""
    for by in ("query", "scale"):
        test_logits_past_24_bits(fmt, dim, by, top, sign, g=g)


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("g,new", [(1, 3), (3, 2), (5, 2), (2, 8)])
@pytest.mark.parametrize("most", [150, 700])
def test_many_items_of_each_tile(fmt, dim, g, new, most):
    """More items than three an SM, so that an SM's groups stand in CTAs of
    their own, for each number of tiles of four rows and each width."""
    nseq = 120
    ctx = [(37 * b * b + 11 * b) % most for b in range(nseq)]
    c = Case(fmt, 4, g, dim, [1 + (b + new - 1) % new for b in range(nseq)], ctx, seed=nseq + g)
    got = c.run()
    assert torch.equal(got, c.run())
    # (the reference takes one head of the first and the last key head's time)
    heads = [0, c.hq - 1]
    c.q, c.hq = np.ascontiguousarray(c.q[:, heads]), 2
    c.k, c.v = (np.ascontiguousarray(x[:, [0, -1]]) for x in (c.k, c.v))
    c.check(got[:, heads])


@pytest.mark.parametrize("fmt", FMTS, ids=R.NAMES.get)
@pytest.mark.parametrize("dim,g", [(64, 2), (128, 7), (256, 4), (64, 20), (128, 50)])
@pytest.mark.parametrize("scale", [3e38, -3e38, 1e-38])
def test_scales_at_the_ends_of_f32(fmt, dim, g, scale):
    """Any finite scale, as long as its product with a query is finite."""
    scale = float(np.float32(scale))
    c = Case(fmt, 1, g, dim, [2], [200], seed=24, spread=0.25 / abs(scale))
    got = c.run(scale=scale)
    c.check(got, c.want(scale=scale))
