"""The references of oracle/layers.py against independent forms of the same definitions."""
import numpy as np
import torch

import oracle
from oracle import layers as ol


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_conv_is_torch_conv1d_and_continues():
    g = gen(1)
    T, C, W = 37, 6, 4
    x = torch.randn(T, C, generator=g, dtype=torch.float64)
    w, b = torch.randn(C, W, generator=g), torch.randn(C, generator=g)
    cache = torch.zeros(3, W - 1, C, dtype=torch.float64)
    y, left, _ = ol.conv(x, w, b, [0, T], cache, [1], None, silu=False)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.t()[None], (W - 1, 0)),
                                      w.double()[:, None], b.double(), groups=C)[0].t()
    assert np.allclose(y, want.numpy(), rtol=0, atol=1e-12)
    assert np.array_equal(left[1], x[-3:].numpy())
    # cut anywhere, the second part continued from the slot
    for cut in (0, 1, 2, 3, 20, 36):
        y1, c1, _ = ol.conv(x[:cut], w, b, [0, cut], cache, [1], None)
        y2, c2, _ = ol.conv(x[cut:], w, b, [0, T - cut], torch.as_tensor(c1), [1], [1])
        full, cf, _ = ol.conv(x, w, b, [0, T], cache, [1], None)
        assert np.allclose(np.concatenate([y1, y2]), full, rtol=0, atol=1e-12)
        assert np.array_equal(c2, cf)


def test_scan_with_one_decay_a_head_is_the_ssd_recurrence():
    g = gen(2)
    T, H, P, N, G = 29, 4, 16, 16, 2
    x = torch.randn(T, H, P, generator=g)
    dt = torch.rand(T, H, generator=g) * 0.1
    A = -torch.rand(H, generator=g) * 4
    B, C = torch.randn(T, G, N, generator=g), torch.randn(T, G, N, generator=g)
    D = torch.randn(H, generator=g)
    cu = torch.tensor([0, 10, 29], dtype=torch.int32)
    cache = torch.randn(3, H, P, N, generator=g)
    idx, has = torch.tensor([2, 0], dtype=torch.int32), torch.tensor([0, 1], dtype=torch.uint8)
    want = oracle.prefill(x, dt, A, B, C, D, cu, idx, has, cache, 64, checkpoints=False)
    wide = lambda v: v[..., None].expand(*v.shape, P).reshape(*v.shape[:-1], H * P)   # noqa: E731
    y, _, left, *_ = ol.scan(x.reshape(T, H * P), wide(dt), wide(A)[:, None].expand(H * P, N), B, C,
                             wide(D), None, cu, cache.reshape(3, H * P, N), idx, has)
    assert np.allclose(y, np.asarray(want["y"]).reshape(T, H * P), rtol=0, atol=1e-9)
    assert np.allclose(left[[0, 2]], want["cache"].double().numpy().reshape(3, H * P, N)[[0, 2]],
                       rtol=0, atol=1e-6)


def test_scan_closed_forms():
    # no decay, unit steps: the state counts tokens; gate of a large z is z
    T, ch, N = 5, 3, 16
    one = torch.ones(T, ch)
    y, st, *_ = ol.scan(one, one, torch.zeros(ch, N), torch.ones(T, 1, N), torch.ones(T, 1, N), None,
                        None, [0, T], torch.zeros(1, ch, N), [0], None)
    assert np.allclose(y, N * np.arange(1, T + 1)[:, None])
    raw = torch.full((1, ch), -3.0)
    y, *_ = ol.scan(one[:1], raw, torch.zeros(ch, N), torch.ones(1, 1, N), torch.ones(1, 1, N), None,
                    torch.full((1, ch), 50.0), [0, 1], torch.zeros(1, ch, N), [0], None,
                    torch.zeros(ch), 0.0, 1e9)
    assert np.allclose(y, N * 50.0 * np.log1p(np.exp(-3.0)))


def test_attention_forms():
    g = gen(3)
    q, k, v = (torch.randn(n, h, 8, generator=g, dtype=torch.float64)
               for n, h in ((7, 4), (9, 2), (9, 2)))
    out, lse, mag, top = ol.attention(q, k, v, [0, 7], [0, 9])
    kk, vv = (t.repeat_interleave(2, 1).transpose(0, 1) for t in (k, v))
    mask = torch.ones(7, 9, dtype=torch.bool).tril(2)
    sc = (q.transpose(0, 1) @ kk.transpose(1, 2)) / 8 ** 0.5
    sc = sc.masked_fill(~mask, -torch.inf)
    want = (torch.softmax(sc, -1) @ vv).transpose(0, 1)
    assert np.allclose(out, want.numpy(), rtol=0, atol=1e-12)
    assert np.allclose(lse, torch.logsumexp(sc, -1).t().numpy(), rtol=0, atol=1e-12)
    # equal keys: the mean; more queries than keys: the first ones see nothing
    out, lse, *_ = ol.attention(q[:3], k[:1].expand(2, 2, 8), v[:2], [0, 3], [0, 2])
    assert np.all(out[0] == 0) and np.all(np.isinf(lse[0]))
    assert np.allclose(out[2, 0], v[:2, 0].mean(0).numpy())


def test_codes_and_rows():
    t = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ol.CODES, t, equal_nan=True)
    v, b = ol.encode_row([448.0, -1.0, 0.0, 2.0 ** -9])
    assert b == 127 and list(v) == [448.0, -1.0, 0.0, 2.0 ** -9]
    v, b = ol.encode_row([449.0, 17.0, 19.0])       # one past the largest: the scale doubles
    assert b == 128 and v[0] == 224.0 and v[1] == 8.0 and v[2] == 10.0     # ties to the even code
    assert ol.encode_row([0.0, 0.0]) [1] == 1
    v, b = ol.encode_row([np.inf, 1.0, np.nan])
    assert np.isnan(v[0]) and np.isnan(v[2]) and v[1] == 256.0 and b == 119
    g = gen(4)
    x = torch.randn(64, generator=g)
    v, b = ol.encode_row(x.numpy())
    want = (x * 2.0 ** (127 - b)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, want)
