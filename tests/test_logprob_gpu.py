"""Log probabilities, entropies and alternatives on the GPU, against 64 bits."""
import pytest

import prompt_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def normal(n, v, kind, seed, size=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (size * torch.randn(n, v, generator=g, device="cuda")).to(kind)
    return x, torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)


def check(x, tokens, top):
    logp, ent, tl, tt = kq.token_logprobs(x, tokens, top=top)
    want = R.logprobs(x, tokens, top)
    # weights' errors move the entropy by the spread of the distances at most
    spread = 30.0
    for got, ref in ((logp, want[0]), (ent, want[1])) + (((tl, want[2]),) if top else ()):
        assert torch.equal(got.isnan(), ref.isnan())
        inf = ref.isinf()
        assert torch.equal(got[inf].double(), ref[inf])
        ok = torch.isfinite(ref)
        bound = R.logprob_bound(ref, spread if ref is want[1] else 0.0, x.shape[1])
        # the logit's distance to the maximum is a rounding of its own
        assert ((got.double() - ref).abs()[ok] <= bound[ok]).all()
    if top:
        assert torch.equal(tt, want[3])
    else:
        assert tl is None and tt is None


@pytest.mark.parametrize("kind", [F32, F16, BF16])
@pytest.mark.parametrize("n,v,top", [(1, 1, 1), (3, 2, 2), (1, 31, 20), (5, 33, 32), (2, 1000, 0),
                                     (7, 4097, 5), (1, 202048, 20), (3, 50001, 32), (40, 32000, 20),
                                     (400, 1003, 8), (160, 8190, 1), (1, 524288, 32)])
def test_against_64_bits(n, v, top, kind):
    check(*normal(n, v, kind, n + v + top), top)


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_rows_that_begin_and_end_off_lines(kind, shift):
    x, t = normal(6, 5000, kind, shift)
    check(x[:, shift:5000 - 2 * shift], t.clamp(max=4000), 7)
    y = x.flatten()[shift:shift + 3 * 4999].view(3, 4999)  # odd stride
    check(y, t[:3].clamp(max=4998), 7)


@pytest.mark.parametrize("order", ["rising", "falling", "equal", "steps"])
@pytest.mark.parametrize("n,v", [(2, 20011), (320, 5003)])
def test_orders(order, n, v):
    i = torch.arange(v, device="cuda", dtype=F32)
    row = {"rising": i / 1000, "falling": -i / 1000, "equal": 0 * i, "steps": (i // 700) % 3}[order]
    x = row.repeat(n, 1).contiguous()
    check(x, torch.full((n,), v - 1, device="cuda", dtype=torch.int32), 32)


def test_minus_zero_is_zero_and_lowest_tokens_come_first():
    x = torch.full((1, 300), -1.0, device="cuda")
    x[0, [7, 100, 200]] = torch.tensor([-0.0, 0.0, -0.0], device="cuda")
    assert kq.token_logprobs(x, top=4)[3].tolist() == [[7, 100, 200, 0]]


@pytest.mark.parametrize("v", [50, 40000])
def test_masked_words(v):
    x, t = normal(5, v, F32, v)
    x[0, 3:] = -INF
    x[1, ::2] = -INF
    x[2] = -INF
    x[2, v - 1] = 2.0
    x[3] = torch.finfo(F32).min
    x[3, 5] = 0.0
    x[4] = -INF
    t = torch.tensor([1, 0, v - 1, 5, 0], device="cuda", dtype=torch.int32)
    check(x, t, 20)
    logp, ent, tl, tt = kq.token_logprobs(x, t, top=20)
    assert logp[2] == 0 and ent[2] == 0 and logp[1] == -INF
    assert logp[4].isnan() and ent[4].isnan() and tl[4].isnan().all() and tt[4].tolist() == list(range(20))
    assert tt[0, :3].sort().values.tolist() == [0, 1, 2] and tt[0, 3:].tolist() == list(range(3, 20))


def test_not_finite():
    x, t = normal(4, 9000, F32, 1)
    want = kq.token_logprobs(x, t, top=3)
    x[1, 17] = NAN
    x[1, 4000] = NAN
    x[2, 8999] = INF
    logp, ent, tl, tt = kq.token_logprobs(x, t, top=3)
    for i in (1, 2):
        assert logp[i].isnan() and ent[i].isnan() and tl[i].isnan().all()
    assert tt[1, :2].tolist() == [17, 4000] and tt[2, 0] == 8999
    for i in (0, 3):
        assert all(torch.equal(a[i], b[i]) for a, b in zip((logp, ent, tl, tt), want))


@pytest.mark.parametrize("size", [1e-3, 50.0, 1e4, 1e30])
def test_sizes(size):
    check(*normal(3, 30000, F32, 9, size), 10)


def test_tokens_outside_and_parts_left_out():
    x, t = normal(3, 777, F32, 2)
    t[0], t[1] = -1, 777
    check(x, t, 0)
    assert kq.token_logprobs(x, t)[0].isnan().tolist() == [True, True, False]
    logp, ent, tl, tt = kq.token_logprobs(x, None, top=2, entropy=False)
    assert logp is None and ent is None and tt.shape == (3, 2)
    a, b, *_ = kq.token_logprobs(x, t, entropy=False)
    assert b is None and torch.equal(a[2:], kq.token_logprobs(x, t)[0][2:])
    none = kq.token_logprobs(x[:0], t[:0], top=2)
    assert [tuple(z.shape) for z in none] == [(0,), (0,), (0, 2), (0, 2)]


def test_streams_and_graphs():
    x, t = normal(20, 30001, BF16, 3)
    want = kq.token_logprobs(x, t, top=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kq.token_logprobs(x, t, top=6, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = kq.token_logprobs(x, t, top=6)
    x.copy_(x.flip(1))
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, kq.token_logprobs(x, t, top=6)))


@pytest.mark.parametrize("top", [1, 12, 13, 24, 25, 32])
@pytest.mark.parametrize("n,v", [(1, 9001), (2, 150001), (400, 20011)])
def test_alternatives_of_few_values(n, v, top):
    """Many equal logits, in rows as they come, rising and falling, and rows of
    one value: the lower token first, whatever the order of the merging."""
    g = torch.Generator(device="cuda").manual_seed(v + top)
    x = torch.randint(-40, 9, (n, v), generator=g, device="cuda").float()
    x[0, :] = torch.arange(v, device="cuda") // 7 % 1000 if n == 1 else 3.0
    if n > 2:
        x[1] = x[1].sort().values
        x[2] = x[2].sort(descending=True).values
        x[3, 5:] = -float("inf")
    logp, ent, tl, tt = kq.token_logprobs(x, None, top=top)
    want = x.sort(dim=1, descending=True, stable=True)
    assert torch.equal(tt.long(), want.indices[:, :top])
    ref = want.values[:, :top].double() - torch.logsumexp(x.double(), 1, keepdim=True)
    at = torch.isfinite(ref)
    # (2^-21: the sum, its logarithm below 16, and a difference below 1100)
    assert ((tl.double() - ref)[at].abs() <= 2.0 ** -21 * (16 + ref[at].abs())).all()
    assert (tl[~at] == -float("inf")).all()
