"""Products with 4-bit weights on the GPU against oracle/steps.py: small whole numbers, whose sums
are exact in any order, bit for bit; others within linear_tolerance."""
import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, E4, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
DEV = "cuda"


def make(seed, T, K, N, xt, whole):
    """Codes and scales, rows, and what they stand for."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=U8)
    ws = torch.randint(126, 129, (N, K // 32), generator=g, dtype=U8)
    if whole:
        x = torch.randint(-4, 5, (T, K), generator=g).float()
        lo, hi = 126, 129
    else:
        x = torch.randn(T, K, generator=g)
        ws -= 3
        lo, hi = 115, 135
    xs = None
    if xt == E4:
        xs = torch.randint(lo, hi, (T, K // 32), generator=g, dtype=U8)
        if not whole:
            x = x * 60
    x = x.to(xt)
    xv = os_.rows8(x, xs) if xt == E4 else os_.f64(x)
    return codes, ws, x, xs, os_.weights(codes, ws), xv


def run(codes, ws, x, xs, N, to, bias=None, out=None):
    T, K = x.shape
    p = ssd.make_linear_problem(T, K, N, x.dtype, to)
    out = torch.full((T, N), 7.0, dtype=to, device=DEV) if out is None else out
    dev = lambda t: None if t is None else t.to(DEV)                            # noqa: E731
    ssd.linear_w4(p, dev(x), dev(codes), dev(ws), out, dev(xs), dev(bias), ssd.alloc_linear_workspace(p, DEV))
    return out


def check(out, xv, w, bias=None, xt=BF):
    y, mag = os_.linear(xv, w, bias)
    cut = os_.cut_products(xv, w) if xt == E4 and out.dtype == BF else 0.0
    got = out.cpu().double().numpy()
    bad = ~(np.abs(got - y) <= os_.linear_tolerance(y, mag, w.shape[1], out.dtype, cut))
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - y))))


SIZES = [(1, 32, 1), (1, 2560, 100), (1, 4864, 40), (4, 4352, 16), (8, 768, 50), (2, 96, 17), (3, 160, 33), (5, 1056, 64), (16, 512, 48), (17, 544, 65),
         (31, 256, 16), (33, 64, 257), (48, 1024, 130), (64, 320, 31), (65, 128, 96), (77, 1056, 111),
         (100, 32, 300), (127, 96, 129), (128, 256, 256), (129, 288, 255), (200, 2080, 70), (256, 224, 513),
         (300, 128, 40), (513, 160, 272), (1000, 64, 20)]


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_whole_numbers(T, K, N, xt):
    codes, ws, x, xs, w, xv = make(T + K + N, T, K, N, xt, True)
    y, mag = os_.linear(xv, w)
    # multiples of 2^-3 (8-bit rows: 2^-4 with their own scales) below 2^20: every partial sum is exact;
    # within a block of 32 products the largest is at most 48 times the smallest
    assert mag.max() < 2.0 ** 20
    for to in (F32, BF):
        got = run(codes, ws, x, xs, N, to).cpu()
        assert torch.equal(got, torch.from_numpy(y).to(to)), (to, np.argwhere(got.double().numpy() != y)[:5])


# a size for each tile that is built (per type of the rows), K ending inside a step or not
TILES = {"few": (4, 2560, 300), "16x16": (12, 4096, 300), "16x32": (16, 512, 9000), "32x32": (64, 1024, 2600),
         "64x64": (32, 256, 9000), "128x128": (200, 256, 9000), "256x256": (1700, 512, 9000), "192x256": (1150, 512, 9000),
         "128x256": (384, 640, 18560)}           # (of 8-bit rows alone)


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("to", [BF, F32])
@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("odd", [0, 1])
def test_every_tile(tile, xt, to, odd):
    T, K, N = TILES[tile]
    if odd:
        T, K, N = max(1, T - 3), K - 96 if K > 512 else K + 32, N - 7
    took = exact_in_any_order(T, K, N, xt, to)
    if not odd and (xt == E4 or tile != "128x256"):
        assert took == tile


@pytest.mark.parametrize("K", [512, 1024, 1536, 2560, 4096])
@pytest.mark.parametrize("shift", [0, 4])
def test_scales_of_four_stages(K, shift):
    """The tile that loads scales for four stages of K at once, where their arrays allow it, and not."""
    assert exact_in_any_order(301, K, 18553, E4, BF, shift) == "128x256"


def exact_in_any_order(T, K, N, xt, to, shift=0):
    """Runs whole numbers and compares bit for bit; scales begin `shift` bytes behind 16. Returns the kernel."""
    p = ssd.make_linear_problem(T, K, N, xt, to)
    took = ssd.linear_w4_kernel(p)
    g = torch.Generator(DEV).manual_seed(K)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=U8, device=DEV)
    ws = torch.randint(126, 129, (N, K // 32), generator=g, dtype=U8, device=DEV)
    x = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float()
    xs = torch.randint(126, 129, (T, K // 32), generator=g, dtype=U8, device=DEV) if xt == E4 else None
    if shift:
        ws, xs = (torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape) for t in (ws, xs))
    out = torch.empty(T, N, dtype=to, device=DEV)
    ssd.linear_w4(p, x.to(xt), codes, ws, out, xs, None, ssd.alloc_linear_workspace(p, DEV))
    # the same sums in float32, exact in any order: whole multiples of 2^-4 below 2^20
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(1).int()
    w = torch.where(c >= 8, -1.0, 1.0) * lut[c & 7] * torch.exp2(ws.float() - 127).repeat_interleave(32, 1)
    if xt == E4:
        x = x * torch.exp2(xs.float() - 127).repeat_interleave(32, 1)
    want = torch.cat([(x[a:a + 512].double() @ w.double().t()) for a in range(0, T, 512)])
    assert float((x.abs().amax(0) * w.abs().amax(0)).sum()) < 2.0 ** 20
    assert torch.equal(out, want.to(to)), took
    return took


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("to", [BF, F32])
@pytest.mark.parametrize("T,K,N", [(1, 2560, 200), (4, 1056, 50), (20, 512, 64), (77, 1056, 111), (130, 320, 300)])
def test_values(T, K, N, xt, to):
    codes, ws, x, xs, w, xv = make(T * K, T, K, N, xt, False)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1))
    check(run(codes, ws, x, xs, N, to), xv, w, xt=xt)
    check(run(codes, ws, x, xs, N, to, bias), xv, w, bias, xt)


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T", [1, 20, 150])
def test_strides(T, xt):
    """Rows of x and out inside wider ones; what lies beside them is left as it was."""
    K, N = 160, 75
    codes, ws, x, xs, w, xv = make(T, T, K, N, xt, True)
    wide = torch.zeros(T, 3 * K, device=DEV).to(xt)
    wide[:, K:2 * K] = x.to(DEV)
    out = torch.full((T, N + 9), 7.0, dtype=F32, device=DEV)
    p = ssd.make_linear_problem(T, K, N, xt, F32)
    ssd.linear_w4(p, wide[:, K:2 * K], codes.to(DEV), ws.to(DEV), out[:, 4:4 + N], None if xs is None else xs.to(DEV),
                  None, ssd.alloc_linear_workspace(p, DEV))
    assert np.array_equal(out[:, 4:4 + N].cpu().double().numpy(), os_.linear(xv, w)[0])
    out[:, 4:4 + N] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T", [1, 40, 200])
def test_odd_output_rows(T, xt):
    """Output rows that start on their element alone."""
    K, N = 64, 33
    codes, ws, x, xs, w, xv = make(T, T, K, N, xt, True)
    buf = torch.full((T * N + 3,), 7.0, dtype=BF, device=DEV)
    run(codes, ws, x, xs, N, BF, out=buf[1:1 + T * N].view(T, N))
    check(buf[1:1 + T * N].view(T, N), xv, w, xt=xt)
    assert float(buf[0]) == 7 and bool((buf[-2:] == 7).all())


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T", [3, 90, 140])
def test_non_finite_stay_in_their_rows(T, xt):
    """A NaN weight makes its output NaN for every token, a NaN or infinite value its token's
    outputs; nothing else. K ends inside a step, so that what is filled in is seen to be nothing."""
    K, N = 96, 40
    codes, ws, x, xs, w, xv = make(T, T, K, N, xt, True)
    ws[7, 1] = 255
    x = x.float()
    x[1, 90] = float("nan")
    if xt == BF:
        x[2] = 0
        x[2, 5] = float("inf")
        codes[:, 2] = 0x22                  # 1 at k = 4 and 5
    x = x.to(xt)
    got = run(codes, ws, x, xs, N, F32).cpu().double().numpy()
    xv = os_.rows8(x, xs) if xt == E4 else os_.f64(x)
    clean = np.ones((T, N), dtype=bool)
    clean[1], clean[:, 7] = False, False
    if xt == BF:
        clean[2] = False
        assert np.all(np.isposinf(got[2, np.arange(N) != 7]))
    assert np.isnan(got[1]).all() and np.isnan(got[:, 7]).all()
    with np.errstate(invalid="ignore"):
        want = os_.linear(np.nan_to_num(xv, nan=0, posinf=0), np.nan_to_num(os_.weights(codes, ws)))[0]
    assert np.array_equal(got[clean], want[clean])


@pytest.mark.parametrize("to", [BF, F32])
@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T", [1, 6, 30, 100, 1100])
def test_scales_of_nan(T, xt, to):
    """A scale byte of 255 is NaN whatever it scales, zeros too; the rest is untouched."""
    K, N = 160, 300
    codes, ws, x, xs, w, xv = make(T, T, K, N, xt, True)
    codes[9, 16:32] = 0
    ws[9, 1] = ws[130, 4] = 255
    rows = torch.ones(T, dtype=torch.bool)
    if xt == E4 and T > 1:
        x = x.float()
        x[2, 64:96] = 0
        x = x.to(E4)
        xs[2, 2] = xs[T - 1, 0] = 255
        rows[2] = rows[T - 1] = False
    outs = torch.ones(N, dtype=torch.bool)
    outs[9] = outs[130] = False
    got = run(codes, ws, x, xs, N, to).cpu()
    assert bool(got[:, ~outs].isnan().all()) and bool(got[~rows].isnan().all())
    want = torch.from_numpy(os_.linear(np.nan_to_num(xv), np.nan_to_num(w))[0])
    assert torch.equal(got[rows][:, outs], want[rows][:, outs].to(to))


@pytest.mark.parametrize("xt", [BF, E4])
def test_ends_of_the_scales(xt):
    """Scale bytes over their whole range, one weight block each: results in float32's range are
    right, powers below and above it 0 or infinite as float32 has it."""
    T, K = 2, 32
    ws = torch.arange(0, 255, dtype=torch.int32).to(U8)[:, None]
    N = ws.shape[0]
    codes = torch.zeros(N, K // 2, dtype=U8)
    codes[:, 3] = 0x07                      # 6 at k = 6
    x = torch.zeros(T, K)
    x[0, 6], x[1, 6] = 1.0, -0.25
    xs = torch.full((T, 1), 127, dtype=U8) if xt == E4 else None
    got = run(codes, ws, x.to(xt), xs, N, F32).cpu().double().numpy()
    want = np.outer([6.0, -1.5], 2.0 ** (ws[:, 0].double().numpy() - 127))
    fits = (np.abs(want) < 2.0 ** 127) & (np.abs(want) >= 2.0 ** -126)
    fits[:, 252:] = False                   # 6 2^126 and more is past bfloat16's and float32's range
    assert np.array_equal(got[fits], want[fits])
    tiny = np.abs(want) < 2.0 ** -126
    assert np.all(np.abs(got[tiny]) <= 2.0 ** -125)


@pytest.mark.parametrize("dt", [BF, F32])
def test_encode(dt):
    g = torch.Generator().manual_seed(2)
    N, K = 37, 96
    w = torch.randn(N, K, generator=g) * torch.exp2(torch.randint(-60, 60, (N, 1), generator=g).float())
    w[0] = 0
    w[1, :32] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5] * 4) * torch.tensor([1.0, -1.0]).repeat(16)
    w[2, 0], w[2, 40], w[2, 70] = float("inf"), float("nan"), float("-inf")
    w[3] = float("nan")
    w[4] = 1e-39
    w[5] = 3e38
    w = w.to(dt)
    p = ssd.make_linear_problem(1, K, N, BF, F32)
    c = ssd.alloc_linear_weights(p, DEV)
    ssd.linear_w4_encode(p, w.to(DEV), **c)
    codes, ws = c["weight"].cpu(), c["weight_scale"].cpu()
    got = os_.weights(codes, ws)
    for n in range(N):
        for b in range(K // 32):
            want, byte = os_.encode_weights(w[n, 32 * b:32 * b + 32].double().numpy())
            assert int(ws[n, b]) == byte, (n, b)
            assert np.array_equal(got[n, 32 * b:32 * b + 32], want), (n, b)
    # and the product with them
    x = torch.randint(-4, 5, (5, K), generator=g).to(BF)
    ok = torch.arange(6, N)
    out = run(codes[ok], ws[ok], x, None, len(ok), F32)
    check(out, os_.f64(x), got[6:])


def test_weights_past_2gb():
    """Weight and output rows past 2^31 bytes."""
    K, N, T = 65536, 70000, 2
    codes = torch.zeros(N, K // 2, dtype=U8, device=DEV)       # 2.3 GB
    ws = torch.full((N, K // 32), 127, dtype=U8, device=DEV)
    rows = torch.tensor([0, 65535, 65537, N - 1])
    codes[rows.to(DEV), 5] = torch.tensor([0x21, 0x32, 0x43, 0x54], dtype=U8, device=DEV)
    codes[N - 1, -1] = 0x70
    x = torch.ones(T, K, dtype=BF, device=DEV)
    x[1] = 2
    out = torch.empty(T, N, dtype=F32, device=DEV)
    p = ssd.make_linear_problem(T, K, N, BF, F32)
    ssd.linear_w4(p, x, codes, ws, out, workspace=ssd.alloc_linear_workspace(p, DEV))
    want = torch.zeros(N)
    want[rows] = torch.tensor([1.5, 2.5, 3.5, 5.0 + 6.0])
    assert torch.equal(out[0].cpu(), want) and torch.equal(out[1].cpu(), 2 * want)


@pytest.mark.parametrize("xt", [BF, E4])
@pytest.mark.parametrize("T", [1, 50, 300])
def test_streams_graphs_and_repeats(T, xt):
    K, N = 544, 200
    codes, ws, x, xs, w, xv = make(4, T, K, N, xt, False)
    d = [None if t is None else t.to(DEV) for t in (codes, ws, x, xs)]
    p = ssd.make_linear_problem(T, K, N, xt, F32)
    out, wsp = torch.empty(T, N, device=DEV), ssd.alloc_linear_workspace(p, DEV)
    go = lambda: ssd.linear_w4(p, d[2], d[0], d[1], out, d[3], None, wsp)       # noqa: E731
    go()
    want = out.clone()
    check(want, xv, w, xt=xt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        go()
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_no_tokens():
    p = ssd.make_linear_problem(0, 64, 8, BF, F32)
    ssd.linear_w4(p, torch.empty(0, 64, dtype=BF, device=DEV), torch.zeros(8, 32, dtype=U8, device=DEV),
                  torch.zeros(8, 2, dtype=U8, device=DEV), torch.empty(0, 8, device=DEV))
