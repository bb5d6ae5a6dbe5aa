"""Verification of drafted tokens against the definition in whole numbers:
chains, trees, drafts with and without a distribution, numbers on a bound,
bad tokens and parents; and that what comes out is distributed as the target."""
import numpy as np
import pytest

import decode_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import quant_quantized_matvec_gb300 as kq  # noqa: E402


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Case:
    def __init__(self, new, vocab, kind, near=0.7, seed=0):
        self.rng = rng = np.random.default_rng(seed)
        self.new, self.vocab = list(new), vocab
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n = int(self.start[-1])
        self.parent = np.array([-1 if j == 0 else j - 1 if kind == "chain" else
                                int(rng.integers(max(0, j - 4), j)) if kind == "tree" else 0
                                for m in new for j in range(m)], np.int32)
        x = 2 * rng.standard_normal((self.n, vocab))
        self.p, self.q = softmax(x), softmax(x + near * rng.standard_normal(x.shape))
        self.token = np.zeros(self.n, np.int32)
        for b, m in enumerate(new):
            for j in range(1, m):
                i = self.start[b] + j
                cdf = np.cumsum(self.q[self.start[b] + self.parent[i]].astype(float))
                self.token[i] = min(np.searchsorted(cdf, rng.uniform() * cdf[-1]), vocab - 1)
        self.u = rng.uniform(size=self.n).astype(np.float32)
        self.un = rng.uniform(size=len(new)).astype(np.float32)

    def run(self, q=True, **kw):
        out = kq.verify_tree(dev(self.start), dev(self.token), dev(self.parent), dev(self.p),
                             dev(self.q) if q else None, dev(self.u), dev(self.un),
                             max(1, max(self.new)), **kw)
        return [x.cpu().numpy() for x in out]

    def check(self, q=True):
        path, count, nxt = self.run(q)
        for b, m in enumerate(self.new):
            lo, hi = self.start[b], self.start[b + 1]
            if m == 0:
                assert count[b] == 0 and nxt[b] == -1
                continue
            want, t = R.verify(m, self.token[lo:hi], self.parent[lo:hi], self.p[lo:hi],
                               self.q[lo:hi] if q else None, self.u[lo:hi], self.un[b])
            assert count[b] == len(want) and nxt[b] == t, (b, count[b], want, nxt[b], t)
            assert path[lo:hi].tolist() == want + [-1] * (m - len(want))


@pytest.mark.parametrize("q", [True, False], ids=["probs", "tokens"])
@pytest.mark.parametrize("kind", ["chain", "tree", "star"])
@pytest.mark.parametrize("new,vocab", [([1], 5), ([6], 1000), ([4, 0, 16, 1, 9], 333),
                                       ([64], 77), ([3, 5], 1), ([8, 8], 30011)])
def test_against_the_definition(new, vocab, kind, q):
    for seed in range(4):
        Case(new, vocab, kind, seed=seed).check(q)


def test_large_vocabulary():
    Case([6, 16], 202048, "tree", seed=1).check()
    Case([5], 202048, "star", seed=2, near=3.0).check()
    Case([3], 1 << 19, "star", seed=3, near=3.0).check()


def test_bounds_of_the_random_numbers():
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, 2.0 ** -31):
        c = Case([4, 3], 1001, "chain", seed=5)
        c.un[:] = u
        c.u[:] = u
        want = c.run()
        c.un[:] = np.clip(c.un, 0, 1 - 2.0 ** -24)
        c.u[:] = np.clip(c.u, 0, 1)
        got = c.run()
        if u != 1.0 and u != 2.0:
            assert all(np.array_equal(a, b) for a, b in zip(want, got))
        assert (want[2] >= 0).all() and (want[2] < 1001).all()
        c.check()


def test_point_masses_and_equal_distributions():
    c = Case([5], 100, "chain", seed=6)
    c.p[:] = 0
    c.p[:, 7] = 1
    c.token[1:] = [7, 7, 3, 7]
    c.check()
    path, count, nxt = c.run()
    assert count[0] == 3 and nxt[0] == 7   # the third draft has no mass
    c.check(q=False)
    d = Case([4], 100, "star", seed=7)
    d.q[:] = d.p                            # every draft is accepted
    d.u[:] = np.minimum(d.u, 0.999)
    assert d.run()[1][0] == 2
    d.u[:] = 1.0                            # on the bound: rejected, nothing left: p stays
    d.check()
    d.p[:] = 0                              # no mass at all
    assert d.run()[2][0] == 99


def test_bad_entries():
    c = Case([8], 50, "chain", seed=8)
    c.u[:] = 0
    c.token[2], c.token[5] = -1, 50         # the chain ends before node 2
    assert c.run()[1][0] == 2
    c.check()
    c = Case([8], 50, "tree", seed=9)
    c.u[:] = 0
    c.parent[3], c.parent[4], c.parent[6] = 3, 99, -7
    c.check()
    c.p[2, 3], c.q[1, 4], c.p[0, 5] = np.nan, 2.0, -1.0
    path, count, nxt = c.run()
    assert 1 <= count[0] <= 8 and 0 <= nxt[0] < 50
    # starts that fall or pass the end
    c.start = np.array([5, 2, 100], np.int32)
    c.un = np.full(2, 0.5, np.float32)
    c.new = [8, 8]
    path, count, nxt = c.run()
    assert count[0] == 0 and nxt[0] == -1 and count[1] >= 1


def test_rows_apart_and_streams():
    c = Case([5, 4], 999, "tree", seed=10)
    want = c.run()
    wide = torch.zeros(2, c.n, 1203, device="cuda")
    wide[0, :, 100:1099], wide[1, :, 100:1099] = dev(c.p), dev(c.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = [dev(x) for x in (c.start, c.token, c.parent, c.u, c.un)]
    torch.cuda.synchronize()
    got = kq.verify_tree(*args[:3], wide[0, :, 100:1099], wide[1, :, 100:1099], *args[3:], 5,
                         stream=side)
    side.synchronize()
    assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(want, got))


@pytest.mark.parametrize("q", [True, False], ids=["probs", "tokens"])
def test_first_token_is_distributed_as_the_target(q):
    """4096 sequences of one node and three drafts of it: the first token after
    the node (the accepted draft, or the one drawn) has the target's
    distribution: each frequency within five standard deviations."""
    n, vocab, rng = 4096, 12, np.random.default_rng(11)
    p = softmax(1.5 * rng.standard_normal(vocab))
    d = softmax(1.5 * rng.standard_normal(vocab))
    c = Case([4] * n, vocab, "star", seed=12)
    c.p[:], c.q[:] = p, d
    if q:
        c.token[:] = rng.choice(vocab, c.n, p=d.astype(float) / d.astype(float).sum())
    else:
        c.token[:] = np.tile([0, 3, 5, 7], n)
    path, count, nxt = c.run(q)
    second = path.reshape(n, 4)[:, 1]
    first = np.where(second >= 0, c.token.reshape(n, 4)[np.arange(n), second], nxt)
    got = np.bincount(first, minlength=vocab) / n
    assert (np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / n) + 1e-9).all()
    # and the token after an accepted draft too
    more = nxt[second >= 0]
    got = np.bincount(more, minlength=vocab) / len(more)
    assert (np.abs(got - p) <= 5 * np.sqrt(p * (1 - p) / len(more)) + 1e-9).all()


def test_refusals():
    c = Case([3], 20, "chain")
    a = [dev(x) for x in (c.start, c.token, c.parent, c.p, c.q, c.u, c.un)]
    with pytest.raises(ValueError):
        kq.verify_tree(a[0], a[1].long(), *a[2:], 3)
    with pytest.raises(ValueError):
        kq.verify_tree(*a[:4], a[4][:, :10], *a[5:], 3)
    with pytest.raises(kq.KQError, match="KQ_ERR_NTOK"):
        kq.verify_tree(*a, 65)


@pytest.mark.parametrize("q", [True, False], ids=["probs", "tokens"])
def test_no_nodes_in_any_sequence(q):
    """A step whose sequences are all idle: count 0 and next -1 for each, as
    for one idle sequence among others."""
    c = Case([0, 0, 0], 100, "chain")
    count, nxt = (torch.full((3,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    path, _, _ = c.run(q, count=count, next_token=nxt)
    assert path.shape == (0,)
    assert count.tolist() == [0, 0, 0] and nxt.tolist() == [-1, -1, -1]
    many = Case([0] * 4096, 5, "chain")
    _, got, nxt = many.run(q)
    assert (got == 0).all() and (nxt == -1).all()


def test_no_nodes_with_torchs_strides_and_starts_of_any_kind():
    c = Case([0, 0], 100, "chain")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    p = torch.empty(0, 100, device="cuda")
    for start in ([0, 0, 0], [7, 3, 1 << 30]):  # (cut to the ntok tokens there are)
        out = kq.verify_tree(dev(np.array(start, np.int32)), none, none, p, None, p[:, 0], dev(c.un), 4)
        assert [x.tolist() for x in out] == [[], [0, 0], [-1, -1]]
    with pytest.raises(kq.KQError, match="KQ_ERR_ALIAS"):
        kq.verify_tree(dev(c.start), none, none, p, None, p[:, 0], dev(c.un), 4,
                       count=out[2], next_token=out[2])
