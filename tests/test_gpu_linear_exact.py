"""Products of 8-bit rows: exact whatever else their block holds, unless the caller lets them be cut.
Sums that are exact in float32 in any order are compared bit for bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ssd = pytest.importorskip("state_space_model_varlen_amd")
BF, F32, E4, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
DEV = "cuda"
VALUES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def values(codes):
    return VALUES.to(DEV)[(codes & 7).int()] * torch.where(codes >= 8, -1.0, 1.0)


def packed(codes):
    return codes[:, 0::2] | codes[:, 1::2] << 4


def product(x, w):
    return torch.cat([x[a:a + 512].double() @ w.double().t() for a in range(0, x.shape[0], 512)])


def run(x, weight, scale, xs, to, cut=False):
    T, K, N = x.shape[0], x.shape[1], weight.shape[0]
    p = ssd.make_linear_problem(T, K, N, E4, to, cut_products=cut)
    out = torch.empty(T, N, dtype=to, device=DEV)
    ssd.linear_w4(p, x, weight, scale, out, xs, None, ssd.alloc_linear_workspace(p, DEV))
    return out, ssd.linear_w4_kernel(p)


def cancelling(T, K, N, seed):
    """8-bit rows, their values, codes, and the exact results. One block of every row of x holds 448
    twice, where the weights are 6 and -6 (of other sign in every second weight row); everything else
    is a whole multiple of 2^-9 up to 7 of them. Products are multiples of 2^-10, and no partial sum of
    any order passes 2688 + 6 7 2^-9 K < 2^12 (K up to 16384): 22 bits."""
    assert K <= 16384
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randint(-7, 8, (T, K), generator=g, device=DEV).float() * 2.0 ** -9
    codes = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=U8)
    block = torch.randint(0, K // 32, (T,), generator=g, device=DEV)
    codes[:, 5::32], codes[:, 22::32] = 7, 15                   # 6 and -6
    codes[1::2, 5::32], codes[1::2, 22::32] = 15, 7
    rows = torch.arange(T, device=DEV)
    x[rows, 32 * block + 5] = 448.0
    x[rows, 32 * block + 22] = 448.0
    return x, codes, product(x, values(codes))


# every kernel: few tokens, and a size of each tile, K ending inside a step or not
SIZES = [(1, 2560, 40), (8, 4096, 50), (12, 4096, 300), (16, 512, 9000), (64, 1024, 2600), (32, 256, 9000),
         (200, 256, 9000), (1700, 512, 9000), (1150, 512, 9000), (384, 640, 18560), (77, 1056, 111), (301, 512, 18553)]


@pytest.mark.parametrize("to", [BF, F32])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_large_products_that_cancel(T, K, N, to):
    x, codes, want = cancelling(T, K, N, T + N)
    one = lambda n: torch.full((n, K // 32), 127, dtype=U8, device=DEV)         # noqa: E731
    got, took = run(x.to(E4), packed(codes), one(N), one(T), to)
    assert torch.equal(got, want.to(to)), (took, float((got.double() - want).abs().max()))


@pytest.mark.parametrize("T,K,N", [(8, 4096, 50), (12, 4096, 300), (301, 512, 18553)])
def test_cut_products_stay_within_their_bound(T, K, N):
    """Cut by 2^-13 of the largest factors' product a block at most, then rounded to bfloat16."""
    x, codes, want = cancelling(T, K, N, T + N)
    one = lambda n: torch.full((n, K // 32), 127, dtype=U8, device=DEV)         # noqa: E731
    top = lambda v: v.abs().unflatten(1, (-1, 32)).amax(-1)                     # noqa: E731
    bound = 32 * 2.0 ** -13 * product(top(x), top(values(codes)))
    got, took = run(x.to(E4), packed(codes), one(N), one(T), BF, cut=True)
    assert bool(((got.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all()), took
    # float32 results are not cut by that choice
    got, _ = run(x.to(E4), packed(codes), one(N), one(T), F32, cut=True)
    assert torch.equal(got, want.float())


def whole(T, K, N, shift=0, cut=True):
    """Rows of -4 to 4 with scales of 1/2 to 2: the largest product of a block is at most 48 times the
    smallest, which is not cut; sums are multiples of 2^-4 below 2^20. Scales begin `shift` bytes behind 16."""
    g = torch.Generator(DEV).manual_seed(T + K)
    codes = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=U8)
    x = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float()
    ws, xs = (torch.randint(126, 129, (n, K // 32), generator=g, dtype=U8, device=DEV) for n in (N, T))
    if shift:
        ws, xs = (torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape) for t in (ws, xs))
    wide = lambda v, s: v * torch.exp2(s.float() - 127).repeat_interleave(32, 1)        # noqa: E731
    want = product(wide(x, xs), wide(values(codes), ws))
    got, took = run(x.to(E4), packed(codes), ws, xs, BF, cut)
    assert torch.equal(got, want.to(BF)), took
    return took


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_cut_products_of_every_kernel(T, K, N, odd):
    whole(max(1, T - 3 * odd), K - 96 * odd if K > 512 else K + 32 * odd, N - 7 * odd)


@pytest.mark.parametrize("K", [512, 1024, 1536, 2560, 4096])
@pytest.mark.parametrize("shift", [0, 4])
def test_cut_products_with_scales_of_four_stages(K, shift):
    """The tile that loads scales for four stages of K at once, where their arrays allow it, and not."""
    assert whole(301, K, 18553, shift) == "128x256"


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("T", [1, 6, 30, 100, 1100])
def test_scales_of_nan(T, cut):
    """A scale byte of 255, and a NaN among a row's values, make NaN of what they enter and of nothing else."""
    K, N = 160, 300
    g = torch.Generator(DEV).manual_seed(T)
    codes = torch.randint(0, 16, (N, K), generator=g, device=DEV, dtype=U8)
    x = torch.randint(-4, 5, (T, K), generator=g, device=DEV).float()
    ws, xs = (torch.full((n, K // 32), 127, dtype=U8, device=DEV) for n in (N, T))
    want = product(x, values(codes)).to(BF)
    codes[9, 32:64] = 0
    ws[9, 1] = ws[130, 4] = 255
    rows, outs = torch.ones(T, dtype=torch.bool, device=DEV), torch.ones(N, dtype=torch.bool, device=DEV)
    outs[9] = outs[130] = False
    if T > 1:
        x[2, 64:96] = 0
        xs[2, 2] = 255
        x[T - 1, 159] = float("nan")
        x[4, 0] = float("nan")
        codes[:, 0] = codes[:, 159] = 0             # (zero times NaN)
        want = product(torch.nan_to_num(x), values(codes)).to(BF)
        rows[[2, 4, T - 1]] = False
    got, took = run(x.to(E4), packed(codes), ws, xs, BF, cut)
    assert bool(got[:, ~outs].isnan().all()) and bool(got[~rows].isnan().all()), took
    assert torch.equal(got[rows][:, outs], want[rows][:, outs]), took


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("T", [2, 12, 200])
def test_ends_of_the_scales(T, cut):
    """Scale bytes of the weights over their whole range, and of the rows so that results stay in range."""
    K = 32
    ws = torch.arange(0, 253, dtype=torch.int32, device=DEV).to(U8)[:, None]
    N = ws.shape[0]
    codes = torch.zeros(N, K, dtype=U8, device=DEV)
    codes[:, 6] = 7
    x = torch.zeros(T, K, device=DEV)
    x[:, 6] = torch.tensor([1.0, -0.25], device=DEV).repeat(T // 2)
    for byte in (27, 127, 227):
        xs = torch.full((T, 1), byte, dtype=U8, device=DEV)
        got, took = run(x.to(E4), packed(codes), ws.contiguous(), xs, BF, cut)
        want = np.outer(x[:, 6].cpu().double() * 6, 2.0 ** (ws[:, 0].cpu().double().numpy() - 127 + byte - 127))
        fits = (np.abs(want) < 2.0 ** 127) & (np.abs(want) >= 2.0 ** -126)
        got = got.cpu().double().numpy()
        assert np.array_equal(got[fits], want[fits]), took
        assert np.all(np.abs(got[np.abs(want) < 2.0 ** -126]) <= 2.0 ** -125), took
