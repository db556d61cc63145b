"""Every kernel of the 4-bit products with a bias, rows inside wider ones, neighbours that stay as they
were, outputs on and off 16 bytes, and scales over a wide range: bit for bit, as all sums are exact in
float32 in any order."""
import pytest
import torch

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, E4, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
DEV = "cuda"
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])
# the type of the rows and of the results, and whether products may be cut
MODES = {"bf16": (BF, BF, False), "bf16-f32": (BF, F32, False), "8": (E4, BF, False), "8-f32": (E4, F32, False),
         "8-cut": (E4, BF, True)}
TILES = {"few": (4, 2560, 300), "16x16": (12, 4096, 300), "16x32": (16, 512, 9000), "32x32": (64, 1024, 2600),
         "64x64": (32, 256, 9000), "128x128": (200, 256, 9000), "256x256": (1700, 512, 9000), "192x256": (1150, 512, 9000),
         "128x256": (384, 640, 18560)}


def case(T, K, N, xt, seed, far):
    """x, codes, scales, bias, result. Each column block of 32 k has a power of two 2^e, in the rows'
    scales (8-bit) or values (bfloat16), and its inverse in the weights' scales, so that products stay
    multiples of 1/2 up to 24: sums below 24 K + 2^10 < 2^20 whatever the powers, e up to `far` each way."""
    assert 24 * K + 2 ** 10 < 2 ** 20
    g = torch.Generator(DEV).manual_seed(seed)
    e = torch.randint(-far, far + 1, (K // 32,), generator=g, device=DEV)
    x = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float()
    codes = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=U8)
    w = VALUES.to(DEV)[(codes & 7).int()] * torch.where(codes >= 8, -1.0, 1.0)
    bias = torch.randint(-1024, 1025, (N,), generator=g, device=DEV).float()
    want = torch.cat([x[a:a + 512].double() @ w.double().t() for a in range(0, T, 512)]) + bias.double()
    ws = (127 - e).to(U8).repeat(N, 1)
    if xt == E4:
        return x.to(E4), (127 + e).to(U8).repeat(T, 1), codes, ws, bias, want
    return (x * torch.exp2(e.float()).repeat_interleave(32)).to(BF), None, codes, ws, bias, want


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("tile", list(TILES))
def test_bias_slices_and_scales(tile, mode, odd):
    xt, to, cut = MODES[mode]
    T, K, N = TILES[tile]
    if odd:
        T, K, N = T - 3, K - 96 if K > 512 else K + 32, N - 7
    x, xs, codes, ws, bias, want = case(T, K, N, xt, T + K + N, 100)
    p = ssd.make_linear_problem(T, K, N, xt, to, cut_products=cut)
    if not odd and (xt == E4 or tile != "128x256"):
        assert ssd.linear_w4_kernel(p) == tile
    side = 32                                               # (keeps rows of either type on 16 bytes)
    wide = torch.full((T, K + 2 * side), float("nan"), device=DEV).to(xt)     # read by mistake, it would show
    wide[:, side:side + K] = x
    left, right = (8, 8) if not odd else (3, 6)             # rows of the result on and off 16 bytes
    out = torch.full((T, left + N + right), 7.0, dtype=to, device=DEV)
    part = out[:, left:left + N]
    ssd.linear_w4(p, wide[:, side:side + K], codes[:, 0::2] | codes[:, 1::2] << 4, ws, part, xs, bias)
    assert torch.equal(part, want.to(to)), (ssd.linear_w4_kernel(p), float((part.double() - want).abs().max()))
    part.fill_(7.0)
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("tile", ["32x32", "64x64", "128x128", "192x256", "256x256"])
def test_nan_stays_in_its_row_and_column(tile, mode):
    xt, to, cut = MODES[mode]
    T, K, N = TILES[tile]
    x, xs, codes, ws, bias, want = case(T, K, N, xt, 5, 0)
    x, codes = x.float(), codes.clone()
    x[T // 2, K - 1] = float("nan")
    bias[N // 3] = float("nan")
    ws[N - 1, K // 32 - 1] = 255
    out = torch.empty(T, N, dtype=to, device=DEV)
    p = ssd.make_linear_problem(T, K, N, xt, to, cut_products=cut)
    ssd.linear_w4(p, x.to(xt), codes[:, 0::2] | codes[:, 1::2] << 4, ws, out, xs, bias)
    rows, outs = torch.ones(T, dtype=torch.bool, device=DEV), torch.ones(N, dtype=torch.bool, device=DEV)
    rows[T // 2] = False
    outs[[N // 3, N - 1]] = False
    assert bool(out[~rows].isnan().all()) and bool(out[:, ~outs].isnan().all())
    assert torch.equal(out[rows][:, outs], want.to(to)[rows][:, outs])


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("T,K,N", [(200, 256, 9000), (1150, 512, 9000)])
def test_large_tiles_in_a_graph(T, K, N, mode):
    xt, to, cut = MODES[mode]
    x, xs, codes, ws, bias, want = case(T, K, N, xt, 9, 20)
    weight, out = codes[:, 0::2] | codes[:, 1::2] << 4, torch.empty(T, N, dtype=to, device=DEV)
    p = ssd.make_linear_problem(T, K, N, xt, to, cut_products=cut)
    go = lambda: ssd.linear_w4(p, x, weight, ws, out, xs, bias)                 # noqa: E731
    go()
    assert torch.equal(out, want.to(to))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want.to(to))
