"""The convolution's and the scan's tests once more, where a result that is NaN is wrong (their own
comparison, a difference larger than the tolerance, does not see one)."""
import numpy as np
import pytest
import torch

import test_gpu_conv as conv
import test_gpu_scan as scan

pytestmark = pytest.mark.gpu
BF, F32, F16 = torch.bfloat16, torch.float32, torch.float16


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    plain, close = conv.check, scan.close

    def number(got):
        assert bool(torch.isfinite(got).all())

    monkeypatch.setattr(conv, "check", lambda got, *a: (number(got), plain(got, *a)))
    monkeypatch.setattr(scan, "close", lambda got, *a: (number(got), close(got, *a)))


def test_the_comparison_sees_nan():
    one = torch.full((1, 1), float("nan"))
    with pytest.raises(AssertionError):
        conv.check(one, np.ones((1, 1)), np.ones((1, 1)), 4, F32)
    with pytest.raises(AssertionError):
        scan.close(one, np.ones((1, 1)), np.ones((1, 1)), 4, F32, "")


@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, BF), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv(ti, ts, W):
    for C in (520, 513):
        conv.run(conv.make(W, [15, 33, 1, 0, 64, 16], C, W, ti, ts))


@pytest.mark.parametrize("ti,ts", [(F32, F32), (BF, F32), (BF, BF), (BF, F16), (F32, BF), (F32, F16)])
@pytest.mark.parametrize("N", [16, 32, 64])
def test_scan(ti, ts, N):
    scan.run(scan.make(N, [31, 0, 33, 64, 200], 80, N, 1, ti, ts), [31, 0, 33, 64, 200])
    lens = [3 + (7 * i) % 11 for i in range(40)] + [37]
    scan.run(scan.make(19, lens, 900, N, 1, ti, ts), lens)


@pytest.mark.parametrize("ti,ts", [(BF, BF), (F32, F32), (BF, F16)])
@pytest.mark.parametrize("R,T,C,N", [(3, 3, 65, 16), (5, 4, 64, 32), (2, 6, 48, 64)])
def test_scan_update(ti, ts, R, T, C, N):
    scan.test_update(ti, ts, R, T, C, N)
