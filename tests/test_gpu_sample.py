"""Token probabilities and the verification of drafts on the GPU against oracle/steps.py."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
DEV = "cuda"
INF = float("inf")


def probs(logits, temperature=None, out=None):
    R, T, V = logits.shape
    p = ssd.make_probs_problem(R, T, V, logits.dtype)
    out = torch.full((R, T, V), 7.0, device=DEV) if out is None else out
    t = None if temperature is None else torch.tensor(temperature, dtype=F32, device=DEV)
    ssd.token_probs(p, logits.to(DEV), t, out, ssd.alloc_probs_workspace(p, DEV))
    return out


def check_probs(out, logits, temperature=None):
    t = None if temperature is None else np.float32(temperature).astype(np.float64)
    want, tol = os_.probs(logits, t)
    got = out.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    bad = ~(np.abs(got - want) <= tol) & ~np.isnan(want)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("ti", [BF, F32])
@pytest.mark.parametrize("R,T,V", [(1, 1, 1), (1, 1, 2), (2, 3, 7), (3, 1, 100), (2, 2, 1023), (1, 2, 4097),
                                   (5, 3, 8191), (1, 1, 50257), (2, 1, 131072), (40, 4, 3001), (1, 1, 300001)])
def test_probs(ti, R, T, V):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(R, T, V, generator=g) * 4).to(ti)
    check_probs(probs(x), x)
    temp = [[0.7, 0.0, 1.3, 1e-3, 50.0][r % 5] for r in range(R)]
    out = probs(x, temp)
    check_probs(out, x, temp)
    s = out.double().sum(-1).cpu()
    assert float((s - 1).abs().max()) < (V / 64 + 80) * 2.0 ** -24 + 1e-7


def test_greedy_takes_the_first_of_equals():
    for V in (5, 300, 5000, 70001):
        x = torch.zeros(1, 4, V)
        x[0, 1, V // 2:] = 1
        x[0, 2, [1, V - 1]] = 3
        x[0, 3, V - 1] = 1
        out = probs(x, [0.0]).cpu()
        assert torch.equal(out.argmax(-1)[0], torch.tensor([0, V // 2, 1, V - 1]))
        assert torch.equal(out.sum(-1), torch.ones(1, 4)) and torch.equal(out.amax(-1), torch.ones(1, 4))
        assert torch.equal(probs(x.to(BF), [-1.0]).cpu(), out) and torch.equal(probs(x, [float("nan")]).cpu(), out)


@pytest.mark.parametrize("V", [9, 2000, 66000])
def test_masked_and_non_finite(V):
    x = torch.randn(1, 7, V, generator=torch.Generator().manual_seed(V))
    x[0, 1, :V // 2] = -INF
    x[0, 2] = -INF
    x[0, 3] = -INF
    x[0, 3, V - 2] = -5.0
    x[0, 4, 3] = float("nan")
    x[0, 5, V - 1] = INF
    x[0, 6] = torch.finfo(F32).min
    for temp in ([1.0], [0.0], [0.3]):
        check_probs(probs(x, temp), x, temp)
    out = probs(x).cpu()
    assert bool((out[0, 2] == 0).all()) and float(out[0, 3, V - 2]) == 1 and bool((out[0, 1, :V // 2] == 0).all())


@pytest.mark.parametrize("V", [50, 3000, 9000, 40000])
def test_ends_of_temperature(V):
    """Temperatures so high that all but masked logits are equal, and so low that the largest alone counts."""
    x = torch.randn(6, 2, V, generator=torch.Generator().manual_seed(V))
    x[:, :, ::3] = -INF
    x[:, 1, V - 1] = 9.0
    temp = [1e30, 1e37, 3e38, INF, 1e-30, 1e-40]
    for ti in (BF, F32):
        check_probs(probs(x.to(ti), temp), x.to(ti), temp)


@pytest.mark.parametrize("ti", [BF, F32])
@pytest.mark.parametrize("V", [511, 1025, 2047, 2049, 4095, 4097, 8193, 16383, 16385, 32767, 32769])
def test_probs_of_every_form(ti, V):
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(2, 3, V, generator=g) * 3).to(ti)
    x[1, 1, : V // 3] = -INF
    x[0, 2, V - 1] = float("nan")
    for temp in ([0.6, 1.0], [0.0, 2.0]):
        check_probs(probs(x, temp), x, temp)


@pytest.mark.parametrize("ti", [BF, F32])
def test_probs_strides(ti):
    R, T, V = 2, 2, 301
    x = torch.randn(R * T, V + 7, generator=torch.Generator().manual_seed(1)).to(ti).to(DEV)
    out = torch.full((R * T, V + 5), 7.0, device=DEV)
    p = ssd.make_probs_problem(R, T, V, ti)
    ssd.token_probs(p, x[:, 3:3 + V], None, out[:, 1:1 + V], ssd.alloc_probs_workspace(p, DEV))
    check_probs(out[:, 1:1 + V].unflatten(0, (R, T)), x[:, 3:3 + V].cpu().unflatten(0, (R, T)))
    out[:, 1:1 + V] = 7.0
    assert bool((out == 7.0).all())


def test_probs_past_4gb():
    R, V = 9000, 131072                                    # 4.7 GB of probabilities
    x = torch.zeros(R, 1, V, dtype=BF, device=DEV)
    a = torch.randn(2, 1, V, generator=torch.Generator().manual_seed(3)).to(BF)
    x[-1], x[8500] = a[0].to(DEV), a[1].to(DEV)
    out = probs(x)
    check_probs(out[[R - 1, 8500]], a)
    assert bool((out[8501] == 2.0 ** -17).all())


def drafts_for(seed, R, T, V, q=True, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, T, V, generator=g) * sharp
    p = torch.softmax(x, -1)
    dq = torch.softmax(x[:, :T - 1] + torch.randn(R, T - 1, V, generator=g), -1)
    d = torch.multinomial(dq.flatten(0, 1), 1, generator=g).view(R, T - 1).to(I32) if T > 1 else \
        torch.zeros(R, 0, dtype=I32)
    return p, (dq.contiguous() if q and T > 1 else None), d, torch.rand(R, T, generator=g)


def verify(p, q, d, n, u):
    R, T, V = p.shape
    dev = lambda t: None if t is None else t.to(DEV)                            # noqa: E731
    pr = ssd.make_verify_problem(R, T, V)
    acc, tok = torch.full((R,), -9, dtype=I32, device=DEV), torch.full((R, T), -9, dtype=I32, device=DEV)
    ssd.verify_drafts(pr, dev(p), dev(q), dev(d), dev(n), dev(u), acc, tok, ssd.alloc_verify_workspace(pr, DEV))
    return acc.cpu().numpy(), tok.cpu().numpy()


def check_verify(p, q, d, n, u):
    acc, tok = verify(p, q, d, n, u)
    wa, wt = os_.verify(p, q, d, n, u)
    assert np.array_equal(acc, wa), (acc, wa)
    assert np.array_equal(tok, wt), (tok, wt)
    return acc, tok


@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("R,T,V", [(1, 1, 1), (1, 2, 2), (3, 1, 10), (7, 4, 50), (64, 3, 33), (5, 8, 300), (2, 65, 20)])
def test_verify(R, T, V, q):
    p, dq, d, u = drafts_for(R * T + V, R, T, V, q)
    acc, _ = check_verify(p, dq, d, None, u)
    n = torch.randint(-1, T + 1, (R,), generator=torch.Generator().manual_seed(1)).to(I32)
    check_verify(p, dq, d, n, u)


@pytest.mark.parametrize("V", [1023, 1025, 4096, 8193, 16383, 16384, 16385, 20000, 38913])
def test_verify_long_rows(V):
    """Rows of one block and of many grains, ends inside and on them."""
    p, dq, d, u = drafts_for(V, 4, 3, V)
    check_verify(p, dq, d, None, u)
    check_verify(p, None, d, None, u)
    u[:, -1] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5, 0.999])
    check_verify(p, dq, d, torch.tensor([0, 1, 2, 0], dtype=I32), u)


@pytest.mark.parametrize("V", [4, 20000])
def test_verify_borders_of_sums(V):
    """Draws that lie on a border of the sums, past it by the least, or at an end."""
    p = torch.zeros(9, 1, V)
    at = [0, V // 4, V // 2, V - 1]
    p[:, 0, at] = torch.tensor([0.25, 0.5, 0.0, 0.25])
    u = torch.tensor([[0.0], [0.2], [0.25], [0.5], [0.75], [0.76], [0.74999], [0.9999], [1.0]])
    _, tok = verify(p, None, None, None, u)
    assert tok[:, 0].tolist() == [at[i] for i in [0, 0, 1, 1, 3, 3, 1, 3, 3]]


def test_verify_borders():
    """Drafts whose test is an equality."""
    # u q < p is strict; a probability of zero is never accepted, one of the draft's zero always
    p = torch.tensor([[[0.5, 0.5, 0.0], [0.0, 1.0, 0.0]]]).repeat(4, 1, 1)
    q = torch.tensor([[[0.5, 0.25, 0.25]]]).repeat(4, 1, 1)
    q[3] = torch.tensor([0.0, 1.0, 0.0])
    d = torch.tensor([[0], [2], [1], [0]], dtype=I32)
    acc, tok = check_verify(p, q, d, None, torch.tensor([[0.99, 0.0], [0.0, 0.0], [0.5, 0.0], [0.99, 0.0]]))
    assert acc.tolist() == [1, 0, 1, 1]
    # equal distributions: turned down (u = 1 is past the range), nothing is left, the target's row counts
    same = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]])
    _, tok = check_verify(same, same[:, :1].contiguous(), torch.tensor([[0]], dtype=I32), None,
                          torch.tensor([[1.0, 0.5]]))
    assert tok[0].tolist() == [1, -1]


def test_verify_odd_probabilities():
    """Tokens outside the vocabulary, rows of zeros, negatives and NaN: no entry of these is drawn."""
    p, q, d, u = drafts_for(5, 6, 3, 40)
    d[0, 0], d[1, 1], d[2, 0], d[3, 0] = -1, 40, 2 ** 31 - 1, -2 ** 31
    check_verify(p, q, d, None, u)
    check_verify(p, None, d, None, u)
    p[4] = 0
    p[5, :, ::2] = float("nan")
    p[5, :, 1] = -3.0
    q[5, :, 5] = float("nan")
    acc, tok = check_verify(p, q, d, None, u)
    assert acc[4] == 0 and tok[4].tolist() == [-1, -1, -1]
    check_verify(p, None, d, None, u)
    for V in (5000, 50000):
        pr = torch.zeros(2, 1, V)
        pr[0, 0, V - 1] = 1e-38
        _, tok = verify(pr, None, None, None, torch.tensor([[0.999], [0.5]]))
        assert tok[:, 0].tolist() == [V - 1, -1]


def test_verify_strides():
    R, T, V = 3, 3, 77
    p, q, d, u = drafts_for(8, R, T, V)
    wp, wq = torch.full((R * T, V + 5), 9.0), torch.full((R * (T - 1), V + 1), 9.0)
    wp[:, 2:2 + V], wq[:, 1:] = p.flatten(0, 1), q.flatten(0, 1)
    pr = ssd.make_verify_problem(R, T, V)
    acc, tok = torch.empty(R, dtype=I32, device=DEV), torch.empty(R, T, dtype=I32, device=DEV)
    ssd.verify_drafts(pr, wp.to(DEV)[:, 2:2 + V], wq.to(DEV)[:, 1:], d.to(DEV), None, u.to(DEV), acc, tok,
                      ssd.alloc_verify_workspace(pr, DEV))
    wa, wt = os_.verify(p, q, d, None, u)
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)


def test_verify_past_4gb():
    """The last request's rows lie past 2^32 bytes."""
    R, T, V = 3000, 3, 131072                              # 4.7 GB
    p = torch.zeros(R, T, V, device=DEV)
    p[:, :, 7] = 1
    d = torch.full((R, T - 1), 7, dtype=I32)
    d[R - 1, 1] = 9
    p[R - 1, 1, 100000] = 3.0
    u = torch.full((R, T), 0.5)
    acc, tok = verify(p, None, d, None, u)
    assert acc[:-1].min() == 2 and acc[-1] == 1
    assert (tok[:-1] == 7).all() and tok[-1].tolist() == [7, 100000, -1]


def test_drawn_tokens_follow_the_probabilities():
    """Draws of many requests at once against the row's probabilities: a count's variance is n p
    (1 - p), five of its roots are taken."""
    n, V = 20000, 12
    g = torch.Generator().manual_seed(4)
    row = torch.softmax(torch.randn(V, generator=g), 0)
    q = torch.softmax(torch.randn(V, generator=g), 0)
    d = torch.multinomial(q, n, replacement=True, generator=g).to(I32)[:, None]
    p = row.repeat(n, 2, 1)
    _, tok = verify(p, q.repeat(n, 1, 1), d, None, torch.rand(n, 2, generator=g))
    count = np.bincount(tok[:, 0], minlength=V)
    pr = row.double().numpy()
    assert np.all(np.abs(count - n * pr) < 5 * np.sqrt(n * pr * (1 - pr)) + 1)


def test_streams_and_graphs():
    R, T, V = 6, 3, 9001
    p, q, d, u = (t.to(DEV) for t in drafts_for(2, R, T, V))
    x = torch.randn(R, T, V, device=DEV)
    pp, pr = ssd.make_probs_problem(R, T, V, F32), ssd.make_verify_problem(R, T, V)
    w1, w2 = ssd.alloc_probs_workspace(pp, DEV), ssd.alloc_verify_workspace(pr, DEV)
    out, acc = torch.empty(R, T, V, device=DEV), torch.empty(R, dtype=I32, device=DEV)
    tok = torch.empty(R, T, dtype=I32, device=DEV)
    temp = torch.tensor([1.0, 0.5, 0.0, 2.0, 1.0, 0.1], device=DEV)

    def go():
        ssd.token_probs(pp, x, temp, out, w1)
        ssd.verify_drafts(pr, out, q, d, None, u, acc, tok, w2)

    go()
    want = [t.clone() for t in (out, acc, tok)]
    wa, wt = os_.verify(out.cpu(), q.cpu(), d.cpu(), None, u.cpu())
    assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)

    def same():
        assert all(torch.equal(a, b) for a, b in zip((out, acc, tok), want))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        tok.zero_()
        go()
    side.synchronize()
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        out.zero_()
        acc.zero_()
        tok.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same()


def test_no_requests():
    e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device=DEV)          # noqa: E731
    probs(torch.empty(0, 3, 9))
    ssd.verify_drafts(ssd.make_verify_problem(0, 2, 9), e(0, 2, 9), None, e(0, 1, dtype=I32), None, e(0, 2),
                      e(0, dtype=I32), e(0, 2, dtype=I32))


def test_tensors_that_are_turned_down():
    """Tensors that do not fit are told on the host; a parameter is a tensor too; a stream is taken."""
    p = ssd.make_probs_problem(1, 1, 64, F32)
    x = torch.randn(1, 1, 64, device=DEV)
    out = torch.empty_like(x)
    with pytest.raises(ValueError, match="GPU"):
        ssd.token_probs(p, x, torch.ones(1), out)
    with pytest.raises(ValueError, match="shape"):
        ssd.token_probs(p, x[..., :32], None, out)
    with pytest.raises(ValueError, match="float32"):
        ssd.token_probs(p, x, None, out.half())
    with pytest.raises(ValueError, match="contiguous"):
        ssd.token_probs(p, x, None, torch.empty(1, 1, 128, device=DEV)[..., ::2])
    ssd.token_probs(p, torch.nn.Parameter(x), None, out)
    check_probs(out, x.cpu())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    ssd.token_probs(p, x, None, out, stream=side)
    side.synchronize()
    check_probs(out, x.cpu())
