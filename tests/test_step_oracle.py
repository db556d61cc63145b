"""The references of oracle/steps.py, pinned by hand-worked values and invariants (no GPU)."""
import numpy as np
import torch

from oracle import steps as os_


def test_norm_by_hand():
    x = torch.tensor([[3.0, 4.0, 0.0, 0.0]])
    out, v, _ = os_.rms_norm(x, eps=0.0)
    assert np.array_equal(out, [[1.2, 1.6, 0, 0]]) and np.array_equal(v, x.numpy())
    out, v, _ = os_.rms_norm(x, torch.tensor([2.0, 1, 1, 1]), residual=torch.tensor([[1.0, -4, 0, 0]]), eps=0.0)
    assert np.array_equal(v, [[4, 0, 0, 0]]) and np.array_equal(out, [[4, 0, 0, 0]])
    out, _, _ = os_.rms_norm(torch.tensor([[1.0, 1.0, 5.0, -5.0]]), groups=2, eps=0.0)
    assert np.array_equal(out, [[1, 1, 1, -1]])
    # silu(0) = 0, silu(v) - silu(-v) = v
    a = os_.rms_norm(torch.ones(1, 2), gate=torch.tensor([[0.0, 3.0]]))[1]
    b = os_.rms_norm(torch.ones(1, 2), gate=torch.tensor([[0.0, -3.0]]))[1]
    assert a[0, 0] == 0 and abs(a[0, 1] - b[0, 1] - 3.0) < 1e-15
    assert np.array_equal(os_.rms_norm(torch.zeros(1, 3))[0], np.zeros((1, 3)))


def test_four_bits_by_hand():
    codes = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe] + [0] * 8], dtype=torch.uint8)
    w = os_.weights(codes, torch.tensor([[128]], dtype=torch.uint8))[0]
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert np.array_equal(w[:16], 2 * np.array(want + [-v for v in want]))
    assert np.isnan(os_.weights(codes, torch.tensor([[255]], dtype=torch.uint8))).all()
    # between two values the even place: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 2.5 -> 2, 5 -> 4
    row = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -5.0] + [0] * 22)
    got, b = os_.encode_weights(row)
    assert b == 127 and np.array_equal(got[:10], [6, 0, 1, 1, 2, 2, 4, 4, 0, -4])
    assert os_.encode_weights(np.full(32, 6.01))[1] == 128 and os_.encode_weights(np.full(32, 3.0))[1] == 126
    assert os_.encode_weights(np.zeros(32))[1] == 1
    got, b = os_.encode_weights(np.array([np.inf, np.nan, -np.inf, 1.5] + [0] * 28))
    assert b == 125 and np.array_equal(got[:4], [1.5, 0, -1.5, 1.5])


def test_probs_by_hand():
    x = torch.log(torch.tensor([[[1.0, 2.0, 5.0]]]).double())
    out, _ = os_.probs(x)
    assert np.allclose(out, [[[0.125, 0.25, 0.625]]], rtol=1e-15)
    out, _ = os_.probs(x, [0.5])
    assert np.allclose(out, np.array([[[1, 4, 25]]]) / 30, rtol=1e-15)
    out, _ = os_.probs(torch.tensor([[[1.0, 7.0, 7.0]]]), [0.0])
    assert np.array_equal(out, [[[0, 1, 0]]])
    inf = float("inf")
    assert np.array_equal(os_.probs(torch.tensor([[[-inf, 0.0, -inf]]]))[0], [[[0, 1, 0]]])
    assert np.array_equal(os_.probs(torch.full((1, 1, 3), -inf))[0], np.zeros((1, 1, 3)))
    assert np.isnan(os_.probs(torch.tensor([[[inf, 0.0]]]))[0]).all()


def test_verify_by_hand():
    t = torch.tensor
    p = t([[[0.5, 0.25, 0.25], [0.25, 0.5, 0.25], [0.0, 0.0, 1.0]]])
    q = t([[[0.25, 0.5, 0.25], [0.25, 0.25, 0.5]]])
    both = lambda *a: [v.tolist() for v in os_.verify(*a)]                     # noqa: E731
    # token 0: 0.99 * 0.25 < 0.5; token 2: 0.5 * 0.5 < 0.25 is not: weights (0, 0.25, 0)
    assert both(p, q, t([[0, 2]]), None, t([[0.99, 0.5, 0.9]])) == [[1], [[0, 1, -1]]]
    assert both(p, q, t([[0, 2]]), None, t([[0.99, 0.49, 0.0]])) == [[2], [[0, 2, 2]]]
    # fewer drafts: the row behind them
    assert both(p, q, t([[0, 2]]), [1], t([[0.5, 0.0, 0.74]])) == [[1], [[0, 1, -1]]]
    assert both(p, q, t([[0, 2]]), [1], t([[0.5, 0.0, 0.75]])) == [[1], [[0, 2, -1]]]
    # certain drafts: 0.5 < 0.5 is not; the others' weights (., 0.25, 0.25)
    assert both(p, None, t([[0, 2]]), None, t([[0.5, 0.0, 0.49]])) == [[0], [[1, -1, -1]]]
    assert both(p, None, t([[0, 2]]), None, t([[0.5, 0.0, 0.5]])) == [[0], [[2, -1, -1]]]
    # turned down where nothing is left over: the target's own row
    assert both(p[:, :2], p[:, :1], t([[7]]), None, t([[0.5, 0.5]])) == [[0], [[1, -1]]]
    assert both(t([[[0.0, -1.0]]]), None, None, None, t([[0.5]])) == [[0], [[-1]]]


def test_verified_tokens_are_the_targets():
    """Over all uniform numbers the first token is distributed as the target says: p(v) = q(v) times
    the chance of acceptance + the chance of none times the rest's share."""
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.2, 0.6])
    n, count = 64, np.zeros(3)
    for d in range(3):
        for i in range(n):
            for j in range(n):
                u = torch.tensor([[(i + 0.5) / n, (j + 0.5) / n]])
                tok = os_.verify(torch.tensor(np.array([[p, p]])), torch.tensor(np.array([[q]])), np.array([[d]]), None, u)[1]
                count[tok[0, 0]] += q[d] / n ** 2
    assert np.abs(count - p).max() < 1.0 / n
