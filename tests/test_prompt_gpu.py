"""Attention of whole prompts on the GPU, against 64 bits."""
import numpy as np
import pytest

import prompt_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
KINDS = [F32, F16, BF16]
INF, NAN = float("inf"), float("nan")


def starts(lens):
    return [0] + np.cumsum(lens).tolist()


def dev(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def inputs(new, ctx, hq, hkv, dim, kind, seed, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    held = [a + b for a, b in zip(new, ctx)]

    def normal(n, h):
        return torch.randn(n, h, dim, generator=g, device="cuda")

    q = (2 * size * normal(sum(new), hq)).to(kind)
    k = (normal(sum(held), hkv) + 0.3 * normal(1, hkv)).to(kind)
    v = normal(sum(held), hkv).to(kind)
    return q, k, v, starts(new), starts(held)


def check(got, q, k, v, s, ks, scale=None):
    want, bound, seen = R.attention(q, k, v, s, ks, q.shape[2] ** -0.5 if scale is None else scale)
    of = seen >= 0
    assert got.dtype is q.dtype and got.shape == q.shape
    d = (got.double() - want).abs()[of]
    assert torch.isfinite(got[of]).all()
    worst = (d / bound[of].clamp(min=1e-300)).max().item() if d.numel() else 0.0
    assert (d <= bound[of]).all(), worst
    assert (got[seen == 0] == 0).all()


SHAPES = [  # new, ctx, hq, hkv, dim
    ([1], [0], 1, 1, 64),
    ([1], [0], 32, 2, 128),
    ([77], [0], 32, 2, 128),
    ([64], [0], 8, 8, 64),
    ([129], [0], 4, 4, 128),
    ([300], [0], 5, 1, 64),
    ([200], [0], 6, 2, 256),
    ([5, 1, 130, 64, 33], [0, 0, 0, 0, 0], 8, 2, 128),
    ([40, 3, 100], [100, 777, 28], 4, 2, 64),
    ([17, 90], [333, 0], 16, 4, 256),
    ([1, 1, 1], [50, 0, 300], 40, 8, 128),
    ([1000], [24], 8, 1, 128),
    ([9], [3000], 8, 2, 128),
    ([3], [2049], 4, 4, 64),
    ([2], [5000], 2, 1, 256),
    ([50], [10], 200, 1, 64),
    ([30], [0], 260, 2, 64),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_against_64_bits(i, kind):
    new, ctx, hq, hkv, dim = SHAPES[i]
    q, k, v, s, ks = inputs(new, ctx, hq, hkv, dim, kind, i)
    got = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    check(got, q, k, v, s, ks)
    if not any(ctx):
        assert torch.equal(kq.prompt_attention(q, k, v, dev(s)), got)
    assert not kq.device_error()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_every_length_about_a_tile(dim, kind):
    """Prompts of 1..140 tokens packed into one call, and continued ones."""
    new = [n for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 140)]
    ctx = [(37 * i) % 150 for i in range(len(new))]
    for c in ([0] * len(new), ctx):
        q, k, v, s, ks = inputs(new, c, 4, 2, dim, kind, dim)
        check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long(dim, kind):
    q, k, v, s, ks = inputs([2100, 700], [0, 1500], 4, 1, dim, kind, 11)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,hq,hkv", [(64, 8, 8), (128, 8, 4), (256, 4, 4)])
def test_several_items_a_cta_on_new_inputs(dim, hq, hkv, kind):
    """More items than SMs, of all lengths, on inputs that no call has seen:
    copies come late and out of order, and a CTA's roles lie an item apart."""
    for seed in range(4):
        new = [1 + (197 * (i + 3 * seed) * (i + 5)) % 1001 for i in range(16)]
        q, k, v, s, ks = inputs(new, [(91 * i) % 300 for i in range(16)], hq, hkv, dim, kind, seed)
        sd, kd = dev(s), dev(ks)
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(seed)
        torch.cuda.synchronize()
        check(kq.prompt_attention(q, k, v, sd, kd), q, k, v, s, ks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_attend_nothing(dim, kind):
    """Fewer keys than queries: the first queries' rows are zero; and no keys
    at all."""
    q, k, v, _, _ = inputs([150, 40, 20], [0, 0, 0], 4, 2, dim, kind, 3)
    s, ks = [0, 150, 190, 210], [0, 70, 70, 80]
    got = kq.prompt_attention(q, k[:80], v[:80], dev(s), dev(ks))
    check(got, q, k[:80], v[:80], s, ks)
    assert (got[:80] == 0).all() and (got[150:200] == 0).all() and (got[80] != 0).any()
    got = kq.prompt_attention(q, k[:0], v[:0], dev(s), dev([0, 0, 0, 0]))
    assert (got == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,new,ctx", [(128, [100, 30], [0, 90]), (64, [20], [3000]), (256, [70, 9], [5, 5])])
def test_strides_and_rows_left_alone(dim, new, ctx, kind):
    q, k, v, s, ks = inputs(new, ctx, 8, 2, dim, kind, 5)
    n, m = q.shape[0], k.shape[0]
    want = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    wide = torch.full((n + 6, 12, dim), NAN, dtype=kind, device="cuda")
    wide[3:n + 3, 2:10] = q
    kv = torch.full((m + 9, 7, dim), NAN, dtype=kind, device="cuda")
    kv[4:m + 4, 1:3], kv[4:m + 4, 4:6] = k, v
    out = torch.full((n + 6, 8, dim), 7.0, dtype=kind, device="cuda")
    got = kq.prompt_attention(wide[:, 2:10], kv[:, 1:3], kv[:, 4:6], dev([x + 3 for x in s]),
                              dev([x + 4 for x in ks]), out=out)
    assert got is out
    assert torch.equal(out[3:n + 3], want)
    assert (out[:3] == 7).all() and (out[n + 3:] == 7).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,ctx", [([90, 70], [30, 0]), ([8], [2500])])
def test_what_is_not_attended_does_not_matter(dim, new, ctx, kind):
    """NaN and infinities in later tokens, in other sequences and behind the
    last one."""
    q, k, v, s, ks = inputs(new, ctx, 4, 2, dim, kind, 6)
    want = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    n, m = q.shape[0], k.shape[0]
    at = m - 5  # a token of the last sequence: its rows from n - 5 on see it
    for value in (NAN, INF, -INF):
        k2, v2 = k.clone(), v.clone()
        v2[at, :, 3] = value
        k2[at] = value
        got = kq.prompt_attention(q, k2, v2, dev(s), dev(ks))
        assert torch.equal(got[:n - 5], want[:n - 5])
        # values alone: the column gets what the formula gives, no other does
        got = kq.prompt_attention(q, k, v2, dev(s), dev(ks))
        assert torch.equal(got[:n - 5], want[:n - 5])
        others = [c for c in range(dim) if c != 3]
        assert torch.equal(got[:, :, others], want[:, :, others])
        tail = got[n - 5:, :, 3]
        assert tail.isnan().all() if value != value else (tail == value).all()
    # behind the last sequence (other sizes may cut the keys otherwise)
    kk = torch.cat([k, torch.full_like(k[:100], NAN)])
    vv = torch.cat([v, torch.full_like(v[:100], INF)])
    check(kq.prompt_attention(q, kk, vv, dev(s), dev(ks)), q, kk, vv, s, ks)
    q2 = torch.cat([q, torch.full_like(q[:9], NAN)])
    check(kq.prompt_attention(q2, kk, vv, dev(s), dev(ks))[:n], q, kk, vv, s, ks)


@pytest.mark.parametrize("kind", KINDS)
def test_early_value_that_is_not_finite(kind):
    """An infinite value that every row attends, far from the diagonal."""
    q, k, v, s, ks = inputs([10], [600], 2, 1, 128, kind, 8, size=0.1)
    v[3, 0, 7] = INF
    got = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    assert (got[:, :, 7] == INF).all()
    assert torch.isfinite(got[:, :, 8:]).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", [1.0, -0.2, 0.0, 1e-30, 30.0])
def test_scales(scale, dim, kind):
    q, k, v, s, ks = inputs([100, 20], [0, 300], 4, 2, dim, kind, 9)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks), scale=scale), q, k, v, s, ks, scale)


@pytest.mark.parametrize("kind,size", [(F32, 1e10), (F32, 1e30), (BF16, 1e10), (BF16, 1e30), (F16, 5e3)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_logits(dim, kind, size):
    """Logits far past 24 bits: each row is the value of its largest score,
    as long as no other comes near it."""
    q, k, v, s, ks = inputs([120], [50], 4, 2, dim, kind, 10, size=size)
    got = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    assert torch.isfinite(got).all()
    x = torch.einsum("thgd,jhd->thgj", q.double().view(120, 2, 2, dim), k.double()) * dim ** -0.5
    limit = torch.arange(120, device="cuda") + 50
    x = x.masked_fill((torch.arange(170, device="cuda") > limit[:, None])[:, None, None], -INF)
    top = x.topk(2, -1)
    # (f32: q to 2^-21 of itself, sums of up to 256 products)
    clear = (top.values[..., 0] - top.values[..., 1]) > 40 + top.values[..., 0].abs() * 2.0 ** -9
    want = torch.gather(v.double().view(170, 2, 1, dim).permute(1, 2, 0, 3).expand(2, 2, 170, dim), 2,
                        top.indices[..., 0].permute(1, 2, 0)[..., None].expand(2, 2, 120, dim))
    want = want.permute(2, 0, 1, 3)
    assert clear.any()
    err = (got.double().view(120, 2, 2, dim) - want).abs()[clear]
    assert (err <= want.abs()[clear] * 2.0 ** -20).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("levels", ["all", "every second", "falling", "up and down"])
def test_maxima_that_grow_from_tile_to_tile(levels, dim, kind):
    """Scores whose level changes by more than 2^8 every 64 keys, from the last
    to the first: what was summed before is corrected each time, or never."""
    q, k, v, s, ks = inputs([150, 70], [800, 100], 4, 2, dim, kind, 21, size=0.25)
    n = torch.cat([torch.arange(m - 1, -1, -1, device="cuda") // 64 for m in (950, 170)])
    level = {"all": 9 * n, "every second": 18 * (n // 2), "falling": -9 * n,
             "up and down": 3 * n + 9 * (n % 2)}[levels]
    q[..., 0] = 4.0
    k[..., 0] = (level[:, None] * dim ** 0.5 / 4.0).to(kind)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)


def test_sizes_of_f32_far_apart():
    """Keys and values of tokens and queries of rows whose sizes differ."""
    q, k, v, s, ks = inputs([200], [100], 4, 2, 128, F32, 12)
    g = torch.Generator(device="cuda").manual_seed(1)
    q *= 10 ** (2 * torch.rand(200, 1, 1, generator=g, device="cuda") - 1.5)
    v *= 1e20
    v[::2] *= 1e-3
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)
    check(kq.prompt_attention(q * 1e15, k * 1e-15, v * 1e-30, dev(s), dev(ks)), q * 1e15, k * 1e-15,
          v * 1e-30, s, ks)


@pytest.mark.parametrize("kind", KINDS)
def test_starts_that_are_not_in_order(kind):
    """Each start counts as the largest so far, within what there is."""
    q, k, v, _, _ = inputs([200], [0], 4, 2, 64, kind, 13)
    bad, good = [-5, 60, 20, 300, 90], [0, 60, 60, 200, 200]
    want = kq.prompt_attention(q, k, v, dev(good), dev(good))
    assert torch.equal(kq.prompt_attention(q, k, v, dev(bad), dev(bad)), want)
    kbad, kgood = [50, 10, 180, -1, 1 << 30], [50, 50, 180, 180, 200]
    want = kq.prompt_attention(q, k, v, dev(good), dev(kgood))
    assert torch.equal(kq.prompt_attention(q, k, v, dev(good), dev(kbad)), want)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    new = [(7 * i) % 5 for i in range(1500)]
    q, k, v, s, ks = inputs(new, [(i * i) % 3 for i in range(1500)], 4, 2, 64, kind, 14)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim", [64, 256])
def test_the_most_sequences(dim, kind):
    """4096 sequences, most of them empty or of one token: far fewer items than
    the grid has CTAs for."""
    new = [1 + i % 2 if i % 3 == 0 else 0 for i in range(4095)] + [70]
    q, k, v, s, ks = inputs(new, [i % 5 if n else 0 for i, n in enumerate(new)], 2, 1, dim, kind, 18)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)
    # and none at all
    out = torch.full_like(q, 3.0)
    kq.prompt_attention(q, k, v, torch.zeros_like(dev(s)), torch.zeros_like(dev(s)), out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,hkv", [(1024, 1), (1024, 1024), (130, 1)])
def test_many_heads(hq, hkv, kind):
    q, k, v, s, ks = inputs([3, 2], [5, 0], hq, hkv, 64, kind, 19)
    check(kq.prompt_attention(q, k, v, dev(s), dev(ks)), q, k, v, s, ks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,new,ctx", [(128, [50], [20]), (64, [9], [4000]), (256, [9], [4000])])
def test_without_a_workspace(dim, new, ctx, kind):
    """The C call takes a stream-ordered temporary; also in a captured graph."""
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    q, k, v, s, ks = inputs(new, ctx, 4, 2, dim, kind, 21)
    sd, kd = dev(s), dev(ks)
    want = kq.prompt_attention(q, k, v, sd, kd)
    got = torch.empty_like(q)

    def call():
        return lib.kq_prompt_attention(
            {F32: 0, F16: 1, BF16: 30}[kind], 1, q.shape[0], k.shape[0], sd.data_ptr(), kd.data_ptr(),
            q.data_ptr(), 4 * dim, 4, k.data_ptr(), 2 * dim, v.data_ptr(), 2 * dim, 2, dim, dim ** -0.5,
            got.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)

    assert call() == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert call() == 0
    got.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,new,ctx", [(128, [700, 300], [0, 0]), (128, [16], [4000]), (256, [90], [800]),
                                         (64, [333, 5], [9, 400])])
def test_streams_graphs_and_workspaces(dim, new, ctx, kind):
    q, k, v, s, ks = inputs(new, ctx, 8, 2, dim, kind, 15)
    sd, kd = dev(s), dev(ks)
    want = kq.prompt_attention(q, k, v, sd, kd)
    need = kq.prompt_workspace_bytes(q, k, len(new))
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(kq.prompt_attention(q, k, v, sd, kd, workspace=ws), want)
    assert (ws[need:] == 255).all()
    if need:
        with pytest.raises(kq.KQError, match="LIMIT"):
            kq.prompt_attention(q, k, v, sd, kd, workspace=ws[:need - 256])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = kq.prompt_attention(q, k, v, sd, kd, stream=other)
    other.synchronize()
    assert torch.equal(got, want)
    # two graphs that share a workspace, replayed in turn; lengths change
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kq.prompt_attention(q, k, v, sd, kd, workspace=ws))
        graphs.append(g)
    for g, out in zip(graphs, outs):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    sd[1:] -= 3
    kd[1:] -= 3
    shorter = kq.prompt_attention(q, k, v, sd, kd)
    for g, out in zip(graphs, outs):
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out[:s[-1] - 3], shorter[:s[-1] - 3])
    assert not kq.device_error()


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    sets = [inputs([600], [0], 8, 2, 128, kind, 20 + i) for i in range(2)]
    d = [(dev(x[3]), dev(x[4])) for x in sets]
    want = [kq.prompt_attention(*x[:3], *y) for x, y in zip(sets, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for st, x, y in zip(streams, sets, d):
            got.append(kq.prompt_attention(*x[:3], *y, stream=st))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(kind):
    """A token stride that puts the last tokens beyond 2^32 bytes."""
    n, dim = 160, 64
    stride = (1 << 31) // 128
    size = 2 if kind is not F32 else 4
    q, k, v, s, ks = inputs([n], [0], 2, 1, dim, kind, 16)
    want = kq.prompt_attention(q, k, v, dev(s), dev(ks))
    big = torch.zeros(n * stride + 4 * dim, dtype=kind, device="cuda")
    assert big.numel() * size > 1 << 32
    qs = big.as_strided((n, 2, dim), (stride, dim, 1))
    kk = big.as_strided((n, 1, dim), (stride, dim, 1), 2 * dim)
    vv = big.as_strided((n, 1, dim), (stride, dim, 1), 3 * dim)
    qs.copy_(q), kk.copy_(k), vv.copy_(v)
    assert torch.equal(kq.prompt_attention(qs, kk, vv, dev(s), dev(ks)), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dim,new,ctx", [(128, [300, 200], [0, 9]), (64, [16], [4000]), (256, [300], [0]),
                                         (64, [9000], [0]), (128, [9000], [0]), (256, [5000], [0])])
def test_expired_waits(dim, new, ctx, kind):
    """A limit below the time that copies and products take: the call ends in
    time, the error word is set where a wait ran out, rows are NaN or right, and
    the next calls are right.  (Waits of a microsecond or two may end before
    the clock is looked at; with several items a CTA some are longer.)"""
    from quant_quantized_matvec_gb300 import _binding
    lib = _binding.load()
    q, k, v, s, ks = inputs(new, ctx, 8, 2, dim, kind, 17)
    sd, kd = dev(s), dev(ks)
    want = kq.prompt_attention(q, k, v, sd, kd)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(want)
    ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    times = 0
    for _ in range(5):
        flush.fill_(1)
        got.fill_(5.0)
        torch.cuda.synchronize()
        lib.kq_set_wait_limit_ns(1)
        try:
            ends[0].record()
            kq.prompt_attention(q, k, v, sd, kd, out=got)
            ends[1].record()
            torch.cuda.synchronize()
        finally:
            lib.kq_set_wait_limit_ns(0)
        expired = kq.device_error()
        times += expired
        assert ends[0].elapsed_time(ends[1]) < 1000.0
        assert ((got == want) | torch.isnan(got)).all()
        assert torch.isnan(got).any() == expired
        for _ in range(2):
            assert torch.equal(kq.prompt_attention(q, k, v, sd, kd), want)
    assert times or sum(new) < 5000


@pytest.mark.parametrize("kind", KINDS)
def test_wrong_arguments(kind):
    q, k, v, s, ks = inputs([30], [10], 4, 2, 64, kind, 22)
    sd, kd = dev(s), dev(ks)
    with pytest.raises(kq.KQError, match="ALIAS"):
        kq.prompt_attention(q, k, v, sd, kd, out=q)
    with pytest.raises(kq.KQError, match="NTOK"):
        kq.prompt_attention(q, k, v, sd)  # more keys than queries, and no starts of theirs
    with pytest.raises(kq.KQError, match="SHAPE"):
        kq.prompt_attention(q[:, :3], k, v, sd, kd)
    with pytest.raises(kq.KQError, match="COUNT"):
        kq.prompt_attention(q, k, v, sd[:1], kd[:1])
    for bad in (dict(q=q.double()), dict(k=k.double()), dict(v=v[:5]), dict(start=sd.long()), dict(v=v.cpu()),
                dict(q=q[..., ::2]), dict(out=torch.empty_like(q)[:5]), dict(start=sd.cpu())):
        args = dict(q=q, k=k, v=v, start=sd, key_start=kd)
        args.update(bad)
        with pytest.raises(ValueError):
            kq.prompt_attention(**args)
    got = kq.prompt_attention(q[:0], k, v, torch.zeros_like(sd), kd)
    assert got.shape == (0, 4, 64)


def test_agrees_with_the_cache():
    """A prompt's path: norms and rotation, the cache's write, attention of the
    prompt; then a second piece attends the keys that were read back, and its
    last tokens agree with attention over the cache."""
    hq, hkv, dim, n, new = 8, 2, 128, 200, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn(n, hq + 2 * hkv, dim, generator=g, device="cuda")
    w = [1 + 0.1 * torch.randn(dim, generator=g, device="cuda") for _ in range(2)]
    table = kq.rope_table(n, dim)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, k = kq.norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], *w, pos, table)
    v = qkv[:, hq + hkv:]
    cache = kq.KVCache(kq.KV_F16, hkv, dim, 8)
    pages = torch.tensor([[3, 1, 7, 0]], dtype=torch.int32, device="cuda")
    kq.kv_append(cache, kq.KVBatch(dev([0, n]), dev([0]), pages, n, n), k, v.contiguous())
    kk, vv = kq.kv_read(cache, kq.KVBatch(dev([0, n]), dev([0]), pages, n, n))
    last = q[n - new:]
    y = kq.prompt_attention(last, kk, vv, dev([0, new]), dev([0, n]))
    z = kq.tree_attention(cache, kq.KVBatch(dev([0, new]), dev([n - new]), pages, new, new), last.contiguous())
    want, bound, _ = R.attention(last, kk, vv, [0, new], [0, n], dim ** -0.5)
    assert ((y.double() - want).abs() <= bound).all()
    assert ((z.double() - want).abs() <= bound).all()
    whole = kq.prompt_attention(q, kk, vv, dev([0, n]))
    assert ((whole[n - new:].double() - want).abs() <= bound).all()
    logits = whole.view(n, -1)
    logp, ent, tl, tt = kq.token_logprobs(logits, pos % logits.shape[1], top=4)
    p = torch.softmax(logits.double(), -1)
    assert ((logp.double().exp() - p.gather(-1, (pos % logits.shape[1]).long()[:, None])[:, 0]).abs() < 1e-6).all()
    assert (tl[:, 0].double() - p.amax(-1).log()).abs().max() < 1e-5
