"""Head norms with rotary positions on the GPU, against 64 bits."""
import pytest

import prompt_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def inputs(n, hq, hk, dim, rot, kind, seed, extra=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(n, hq + hk + extra, dim, generator=g, device="cuda")
    qkv = (qkv * (0.1 + 4 * torch.rand(n, 1, 1, generator=g, device="cuda"))).to(kind)
    w = [1 + 0.3 * torch.randn(dim, generator=g, device="cuda") for _ in range(2)]
    a = 6.3 * torch.rand(50, rot // 2, generator=g, device="cuda")
    table = torch.stack([a.cos(), a.sin()], -1).contiguous()
    pos = torch.randint(0, 50, (n,), generator=g, device="cuda", dtype=torch.int32)
    return qkv[:, :hq], qkv[:, hq:hq + hk], w, pos, table


def check(got, x, w, pos, table, inter, eps, dtype):
    assert got.dtype is dtype
    want, size = R.norm_rope(x, w, pos, table, inter, eps)
    assert ((got.double() - want).abs() <= R.norm_bound(want, size, dtype)).all()


@pytest.mark.parametrize("kind,dtype", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hk,dim,rot", [(1, 32, 2, 128, 128), (5, 3, 1, 128, 64), (37, 1, 1, 96, 24),
                                             (3, 2, 2, 8, 8), (131, 7, 7, 256, 256), (2, 1, 1, 1024, 16),
                                             (9, 5, 2, 520, 520), (4, 40, 8, 40, 8), (70, 2, 1, 64, 64)])
def test_against_64_bits(n, hq, hk, dim, rot, inter, kind, dtype):
    q, k, w, pos, table = inputs(n, hq, hk, dim, rot, kind, n * dim + rot, extra=hk)
    yq, yk = kq.norm_rope(q, k, *w, pos, table, interleaved=inter, dtype=dtype)
    check(yq, q, w[0], pos, table, inter, 1e-6, dtype)
    check(yk, k, w[1], pos, table, inter, 1e-6, dtype)


@pytest.mark.parametrize("kind,dtype", [(F32, F32), (F32, BF16), (F16, F16)])
@pytest.mark.parametrize("n,hq,hk,dim,rot,inter", [(9001, 9, 2, 128, 64, False), (5003, 6, 5, 256, 256, True),
                                                   (16001, 7, 3, 96, 40, False), (20011, 5, 4, 64, 64, True)])
def test_many_tokens(n, hq, hk, dim, rot, inter, kind, dtype):
    """Sizes at which a group of lanes goes through four heads, or what is left
    of them."""
    q, k, w, pos, table = inputs(n, hq, hk, dim, rot, kind, n, extra=1)
    pos[n // 2] = 50
    q[5, 1, 3], k[7, 0] = float("inf"), 0
    yq, yk = kq.norm_rope(q, k, *w, pos, table, interleaved=inter, dtype=dtype)
    assert yq[n // 2].isnan().all() and yk[n // 2].isnan().all() and yq[5, 1].isnan().any()
    assert (yk[7, 0] == 0).all()
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[5, n // 2]] = False
    for y, x, weight in ((yq, q, w[0]), (yk, k, w[1])):
        check(y[keep], x[keep], weight, pos[keep], table, inter, 1e-6, dtype)
    assert torch.equal(kq.norm_rope(q[5:6], None, w[0], None, pos[5:6], table, interleaved=inter,
                                    dtype=dtype)[0][0, 2:], yq[5, 2:])


def test_without_weights_table_or_keys():
    q, k, w, pos, table = inputs(11, 4, 2, 128, 128, F32, 3)
    yq, none = kq.norm_rope(q)
    assert none is None
    check(yq, q, None, None, None, False, 1e-6, F32)
    yq, yk = kq.norm_rope(q, k, None, w[1], pos, table, eps=0.5)
    check(yq, q, None, pos, table, False, 0.5, F32)
    check(yk, k, w[1], pos, table, False, 0.5, F32)


@pytest.mark.parametrize("kind", [F32, F16, BF16])
def test_in_place_in_a_fused_buffer(kind):
    q, k, w, pos, table = inputs(23, 8, 2, 64, 64, kind, 4, extra=2)
    want = kq.norm_rope(q, k, *w, pos, table)
    q.mul_(1)
    got = kq.norm_rope(q, k, *w, pos, table, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_outputs_that_meet_are_refused():
    q, k, w, pos, table = inputs(5, 4, 2, 64, 64, F32, 5)
    other = torch.zeros(5, 8, 64, device="cuda")
    with pytest.raises(kq.KQError, match="ALIAS"):
        kq.norm_rope(q, k, *w, pos, table, q_out=other[:, :4], k_out=other[:, 3:5])
    with pytest.raises(kq.KQError, match="ALIAS"):
        kq.norm_rope(q, k, *w, pos, table, q_out=q[:, :4], k_out=q[:, :2])
    kq.norm_rope(q, k, *w, pos, table, q_out=other[:, :4], k_out=other[:, 4:6])


def test_sizes_whose_squares_f32_does_not_hold():
    x = torch.randn(6, 2, 128, device="cuda")
    for i, f in enumerate([1e30, 1e-30, 3e37, 1e-38, 1.0, 0.0]):
        x[i] *= f
    # (1e-38 times a normal number is partly subnormal: still exact in x)
    got, _ = kq.norm_rope(x, eps=0.0)
    want, size = R.norm_rope(x[:5], None, None, None, False, 0.0)
    assert ((got[:5].double() - want).abs() <= R.norm_bound(want, size, F32) + 2.0 ** -22).all()
    assert got[5].isnan().all()  # 0 / 0
    got, _ = kq.norm_rope(x, eps=1e-6)
    want, size = R.norm_rope(x, None, None, None, False, 1e-6)
    assert ((got.double() - want).abs() <= R.norm_bound(want, size, F32)).all()


def test_bad_positions_and_values_stay_in_their_token():
    q, k, w, pos, table = inputs(9, 4, 2, 128, 64, F32, 6)
    want = kq.norm_rope(q, k, *w, pos, table)
    pos2, q2 = pos.clone(), q.clone()
    pos2[2], pos2[7] = -1, 50
    q2[4, 1, 5] = float("nan")
    q2[5, 2, 100] = float("inf")
    got = kq.norm_rope(q2, k, *w, pos2, table)
    for i in (2, 7):
        assert got[0][i].isnan().all() and got[1][i].isnan().all()
    assert got[0][4, 1].isnan().all()
    assert got[0][5, 2, 100].isnan() and (got[0][5, 2, 64:100] == 0).all()
    keep = [0, 1, 3, 6, 8]
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep + [4, 5]], want[1][keep + [4, 5]])
    assert torch.equal(got[0][4, [0, 2, 3]], want[0][4, [0, 2, 3]])


def test_it_is_rope_of_the_norm():
    """Bit for bit with interleaved pairs, whose lanes hold the values that
    they hold without a rotation.  With halves the squares are summed in another
    order, so that both are within the bound of 64 bits only."""
    q, k, w, pos, table = inputs(33, 6, 1, 128, 128, F32, 7)
    y, _ = kq.norm_rope(q, None, w[0])
    for inter in (False, True):
        z, _ = kq.norm_rope(q, None, w[0], None, pos, table, interleaved=inter)
        turned = kq.rope(y, pos, table, interleaved=inter)
        if inter:
            assert torch.equal(turned, z)
        want, size = R.norm_rope(q, w[0], pos, table, inter, 1e-6)
        assert ((turned.double() - z.double()).abs() <= 2 * R.norm_bound(want, size, F32)).all()


def test_streams_and_graphs():
    q, k, w, pos, table = inputs(300, 8, 2, 128, 128, F32, 8)
    want = kq.norm_rope(q, k, *w, pos, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kq.norm_rope(q, k, *w, pos, table, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kq.norm_rope(q, k, *w, pos, table)
    q.mul_(2)
    pos.add_(-1).clamp_(min=0)
    g.replay()
    want = kq.norm_rope(q, k, *w, pos, table)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
