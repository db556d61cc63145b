"""The norm, the 4-bit products, the token probabilities and the verification together, as
examples/hybrid_stack.py answers with them behind its layers."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import steps as os_

pytestmark = pytest.mark.gpu
pytest.importorskip("state_space_model_varlen_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location(
        "hybrid_stack", os.path.join(ROOT, "examples", "hybrid_stack.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("lens,tokens", [((70, 1, 133), 3), ((300, 17), 1), ((2, 64, 65, 200), 4)])
def test_parts_and_verify_steps_give_the_whole(lens, tokens):
    """Both ways round the same values, but not in the same order of sums. Where they differ by d
    relative (2^-9 for each of about six bfloat16 roundings a layer, added as independent errors:
    d = 2^-9 sqrt(6) = 5e-3), rounding to 8 bits with steps of about 2^-3.5 of a value takes a share
    d / 2^-3.5 of them to the other side, by a step each: sqrt(d 2^-3.5) = 2e-2 of the row's size.
    Three such roundings, and as much again for the gated norm's and the cache's: 2e-2 sqrt(6) = 5e-2; a
    wrong state, row or scale is of the result's own size."""
    for e in load().check(256, lens, 3, tokens, four_bit=True):
        assert e < 5e-2


@pytest.mark.parametrize("drafts", [0, 1, 3])
@pytest.mark.parametrize("four_bit", [False, True])
def test_answers(drafts, four_bit):
    """Every step's decision is the reference's on the probabilities that it saw, greedy requests get
    the largest logit's token, and the slots hold what was accepted."""
    m = load()
    R, V = 3, 500
    st = m.Stack(256, R, 400, seed=1, four_bit=four_bit, vocab=V)
    g = torch.Generator("cuda").manual_seed(2)
    lens = [40, 1, 77]
    prompt = torch.randint(0, V, (sum(lens),), generator=g, device="cuda")
    st.prompt(st.emb[prompt], [2, 0, 1], lens)
    slots = [2, 0, 1]
    temp = torch.tensor([1.0, 0.0, 0.7], device="cuda")
    last = torch.randint(0, V, (R,), generator=g, device="cuda").to(torch.int32)
    held = list(lens)
    for _ in range(4):
        got, (target, draft, tokens, uniform, acc, out) = st.speculate(last, slots, drafts, temp, g)
        wa, wt = os_.verify(target.cpu(), None if draft is None else draft.cpu(),
                            None if tokens is None else tokens.cpu(), None, uniform.cpu())
        assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(out.cpu().numpy(), wt)
        assert float((target.sum(-1) - 1).abs().max()) < 1e-4
        for r in range(R):
            assert len(got[r]) == int(wa[r]) + 1 and all(0 <= t < V for t in got[r])
            held[r] += len(got[r])
            assert int(st.lens[slots[r]]) == held[r]
        # temperature 0: one at the largest, so accepted or corrected to it
        best = target[1].argmax(-1).tolist()
        assert got[1] == best[:len(got[1])]
        last = torch.tensor([t[-1] for t in got], dtype=torch.int32, device="cuda")


def test_chain_in_a_graph():
    """Norm, product, probabilities and verification captured together, on a stream of its own, next to
    the same calls made eagerly on another batch; replayed with new inputs each time."""
    import state_space_model_varlen_amd as ssd
    R, T, K, V, dev = 5, 3, 512, 40000, "cuda"
    rows, bf, u8, i32 = R * T, torch.bfloat16, torch.uint8, torch.int32
    g = torch.Generator(dev).manual_seed(11)
    np_ = ssd.make_norm_problem(rows, K, bf, torch.float8_e4m3fn, residual_dtype=torch.float32)
    lp = ssd.make_linear_problem(rows, K, V, torch.float8_e4m3fn, bf)
    pp, vp = ssd.make_probs_problem(R, T, V, bf), ssd.make_verify_problem(R, T, V)
    w = ssd.alloc_linear_weights(lp, dev)
    ssd.linear_w4_encode(lp, torch.randn(V, K, generator=g, device=dev) * 0.1, **w)
    temp = torch.tensor([1.0, 0.0, 0.5, 2.0, 1.0], device=dev)

    def batch():
        b = dict(x=torch.empty(rows, K, dtype=bf, device=dev), res=torch.empty(rows, K, device=dev),
                 kept=torch.empty(rows, K, device=dev), rows8=torch.empty(rows, K, device=dev).to(torch.float8_e4m3fn),
                 scale=torch.empty(rows, K // 32, dtype=u8, device=dev), logits=torch.empty(rows, V, dtype=bf, device=dev),
                 probs=torch.empty(R, T, V, device=dev), drafts=torch.empty(R, T - 1, dtype=i32, device=dev),
                 uniform=torch.empty(R, T, device=dev), acc=torch.empty(R, dtype=i32, device=dev),
                 out=torch.empty(R, T, dtype=i32, device=dev), ws=ssd.alloc_probs_workspace(pp, dev),
                 wv=ssd.alloc_verify_workspace(vp, dev))
        fill(b)
        return b

    def fill(b):
        b["x"].copy_(torch.randn(rows, K, generator=g, device=dev))
        b["res"].copy_(torch.randn(rows, K, generator=g, device=dev))
        b["drafts"].copy_(torch.randint(0, V, (R, T - 1), generator=g, device=dev))
        b["uniform"].copy_(torch.rand(R, T, generator=g, device=dev))

    def run(b):
        ssd.rms_norm(np_, b["x"], None, b["rows8"], residual=b["res"], residual_out=b["kept"], out_scale=b["scale"])
        ssd.linear_w4(lp, b["rows8"], w["weight"], w["weight_scale"], b["logits"], b["scale"])
        ssd.token_probs(pp, b["logits"].view(R, T, V), temp, b["probs"], b["ws"])
        ssd.verify_drafts(vp, b["probs"], None, b["drafts"], None, b["uniform"], b["acc"], b["out"], b["wv"])

    a, other = batch(), batch()
    run(a), run(other)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(a)
    side = torch.cuda.Stream()
    for _ in range(4):
        fill(a), fill(other)
        run(a)
        want = {k: a[k].clone() for k in ("kept", "rows8", "scale", "logits", "probs", "acc", "out")}
        for k in want:
            a[k].view(u8).fill_(0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        run(other)                              # at the same time, on buffers of its own
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(a[k].view(u8), v.view(u8)), k
        wa, wt = os_.verify(a["probs"].cpu(), None, a["drafts"].cpu(), None, a["uniform"].cpu())
        assert np.array_equal(a["acc"].cpu().numpy(), wa) and np.array_equal(a["out"].cpu().numpy(), wt)
        wa, wt = os_.verify(other["probs"].cpu(), None, other["drafts"].cpu(), None, other["uniform"].cpu())
        assert np.array_equal(other["acc"].cpu().numpy(), wa) and np.array_equal(other["out"].cpu().numpy(), wt)
