"""nvfp4_route_topk and nvfp4_route_topk_backward on the GPU against the CPU
reference in 64 bits.

Choice.  Without a bias keys are the logits, so ids are equal, ties included.
With fp32 keys (score + bias) the kernel's key differs from
the exact one by at most the rounding of the score and of the sum, |key| *
2^-22 in all for |key| < 4 (exp within 1 ulp, the sum and the division half an
ulp each, the bias sum half an ulp; group scores add one more sum): tokens whose
margin is above KEY_TOL must agree, and of the others there are few.
Weights.  Each chosen score has relative error below 8 * 2^-24, the sum of up
to 32 of them 5 roundings more, the division and the scale one each:
W_TOL = 2^-19 relative covers it.  Softmax over a row sums E <= 1024 terms in
32 + 5 steps and forms x - m, whose rounding enters the exponential as
|x - m| * 2^-24: the tests' logits stay within 32 of each other, 2^-18 in all.
Gradients: the same factors, but d - c cancels: the error is relative to the
sum of the absolute terms (computed beside the reference)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from oracle import mxfp4_oracle as mo

pytestmark = pytest.mark.gpu

KEY_TOL = 2.0 ** -19
W_TOL = 2.0 ** -18


def make_logits(T, E, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) * spread).astype(np.float32)
    return torch.from_numpy(x).to(dtype).cuda()


def host(x):
    return x.float().cpu().numpy().astype(np.float64)


def check_route(x, k, bias=None, **form):
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    got = nv.nvfp4_route_topk(x, k, bias=b, **form)
    ids, w = got["expert_ids"].cpu().numpy(), got["weights"].cpu().numpy().astype(np.float64)
    want_ids, want_w, margin = mo.route_topk(host(x), k, bias=None if bias is None else bias.astype(np.float32),
                                             **form)
    sure = margin > KEY_TOL         # (infinite where nothing rounds: keys that are the logits themselves)
    assert sure.mean() > 0.95
    assert np.array_equal(ids[sure], want_ids[sure])
    err = np.abs(w[sure] - want_w[sure])
    assert np.all(err <= W_TOL * np.abs(want_w[sure]) + 1e-30), float(np.max(err))
    assert np.all(ids < x.shape[1]) and np.all(ids >= -1)
    return ids, w


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (2, 16, 4), (129, 63, 6), (33, 64, 8), (40, 100, 7),
                                   (257, 128, 8), (65, 160, 6), (1000, 256, 8), (31, 255, 32), (17, 384, 8),
                                   (9, 513, 3), (21, 1024, 10), (5, 1000, 32)])
def test_route_sizes(T, E, k, dtype, score):
    x = make_logits(T, E, dtype, 7 * T + E)
    for renorm in (True, False):
        check_route(x, k, score=score, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_bias(dtype, score):
    rng = np.random.default_rng(3)
    for T, E, k in [(64, 256, 8), (33, 40, 4), (15, 1024, 16)]:
        check_route(make_logits(T, E, dtype, E), k, bias=rng.standard_normal(E) * 0.3, score=score, scale=1.5)


@pytest.mark.parametrize("score,group_top", [("sigmoid", 2), ("sigmoid", 1), ("softmax", 1), ("softmax", 2)])
@pytest.mark.parametrize("E,G,kg,k", [(256, 8, 4, 8), (160, 8, 3, 6), (24, 3, 2, 4), (32, 32, 9, 8), (1000, 5, 1, 7),
                                      (62, 31, 4, 8), (256, 8, 8, 8), (64, 1, 1, 8)])
def test_route_groups(E, G, kg, k, score, group_top):
    rng = np.random.default_rng(E + G)
    for dtype in (torch.bfloat16, torch.float32):
        for bias in (None, rng.standard_normal(E) * 0.1):
            check_route(make_logits(67, E, dtype, 5 * E + k), k, bias=bias, score=score, num_groups=G, topk_groups=kg,
                        group_top=group_top)


@pytest.mark.parametrize("T", [3, 700, 12011])
@pytest.mark.parametrize("E,G,kg", [(256, 1, 1), (100, 1, 1), (264, 8, 4), (128, 4, 2)])
def test_route_close_keys_in_every_list_length(T, E, G, kg):
    """Keys that differ in their last bits only, more of them than a list holds,
    and equal ones: lists of 8 and of 16 choose as the whole keys do."""
    rng = np.random.default_rng(E + T)
    low = 1.0 + rng.integers(0, 4 * E, (T, E)) * 2.0 ** -23
    x = torch.from_numpy(np.where(rng.random((T, E)) < 0.02, -low, low).astype(np.float32)).cuda()
    bias = rng.integers(0, 8, E) * 2.0 ** -24
    for k in (1, 5, 8, 9, 12, 16):
        check_route(x, k, score="sigmoid", renormalize=True, num_groups=G, topk_groups=kg, group_top=1)
        form = dict(bias=torch.from_numpy(bias.astype(np.float32)).cuda(), score="sigmoid", num_groups=G,
                    topk_groups=kg, group_top=2)
        ids = nv.nvfp4_route_topk(x, k, **form)["expert_ids"]
        # the same choices as the first ones of a longer list, which another kernel makes
        longer = nv.nvfp4_route_topk(x, 20, **form)["expert_ids"]
        assert torch.equal(ids, longer[:, :k])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(5, 16, 16), (70, 40, 10), (300, 256, 9), (11003, 64, 12), (10501, 250, 16)])
def test_route_nine_to_sixteen(T, E, k, dtype, score):
    rng = np.random.default_rng(k + E)
    for bias in (None, rng.standard_normal(E) * 0.2):
        check_route(make_logits(T, E, dtype, T + k), k, bias=bias, score=score, renormalize=bias is not None)
    # fewer usable experts than choices
    x = make_logits(T, E, dtype, T)
    x[:, 3:] = float("-inf")
    x[::2, 1] = float("nan")
    ids, w = check_route(x, k, score=score)
    assert np.all((ids >= 0).sum(1) == np.where(np.arange(T) % 2 == 0, 2, 3)) and np.all(w[ids < 0] == 0)


@pytest.mark.parametrize("score,group_top", [("sigmoid", 2), ("softmax", 1)])
@pytest.mark.parametrize("T,E,G,kg,k", [(67, 22, 2, 1, 6), (67, 44, 4, 3, 8), (33, 72, 8, 5, 7), (9, 508, 4, 2, 8),
                                        (40, 264, 8, 4, 8), (25, 16, 16, 3, 3), (5, 32 * 31, 32, 2, 8), (7, 6, 2, 1, 3),
                                        (20011, 66, 2, 1, 8), (10007, 264, 8, 4, 8)])
def test_route_groups_of_any_size(T, E, G, kg, k, score, group_top):
    """Groups whose experts do not divide among their lanes."""
    rng = np.random.default_rng(E + T)
    for dtype in (torch.bfloat16, torch.float32):
        for bias in (None, rng.standard_normal(E) * 0.1):
            check_route(make_logits(T, E, dtype, 3 * E + k), k, bias=bias, score=score, num_groups=G, topk_groups=kg,
                        group_top=group_top, renormalize=bias is None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_ties_go_to_the_lowest_index(dtype):
    for E, k in [(256, 8), (64, 8), (100, 6), (512, 10)]:
        rng = np.random.default_rng(E)
        x = torch.from_numpy(rng.integers(-2, 3, (50, E)).astype(np.float32)).to(dtype).cuda()
        x[0] = 0.0
        x[1, ::2], x[1, 1::2] = 0.0, -0.0       # the two zeros are equal
        for score in ("sigmoid", "softmax"):
            want, _, _ = mo.route_topk(host(x), k, score=score)
            ids = nv.nvfp4_route_topk(x, k, score=score)["expert_ids"].cpu().numpy()
            assert np.array_equal(ids, want)
    # equal keys under a bias as well: equal logits, equal bias
    x = torch.zeros(4, 256, dtype=dtype, device="cuda")
    ids = nv.nvfp4_route_topk(x, 8, bias=torch.full((256,), 0.25, device="cuda"), num_groups=8,
                              topk_groups=2)["expert_ids"]
    assert torch.equal(ids.cpu(), torch.arange(8, dtype=torch.int32).repeat(4, 1))


def test_route_neighbouring_fp32_keys():
    """Keys that differ only in bits below the packed index: one fp32 ulp apart."""
    E, k = 256, 8
    base = np.float32(0.7)
    ulps = np.random.default_rng(1).permuted(np.tile(np.arange(E, dtype=np.uint32), (32, 1)), axis=1)
    x = (base.view(np.uint32) + ulps).view(np.float32)
    xt = torch.from_numpy(x).cuda()
    want, _, _ = mo.route_topk(x.astype(np.float64), k)
    assert np.array_equal(nv.nvfp4_route_topk(xt, k)["expert_ids"].cpu().numpy(), want)
    xn = torch.from_numpy(-x).cuda()
    want, _, _ = mo.route_topk(-x.astype(np.float64), k)
    assert np.array_equal(nv.nvfp4_route_topk(xn, k)["expert_ids"].cpu().numpy(), want)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_masked_infinite_and_extreme_logits(dtype, score):
    E, k = 96, 6
    x = make_logits(12, E, dtype, 11)
    inf = float("inf")
    x[0] = -inf                                  # nothing can be chosen
    x[1] = float("nan")
    x[2, 3:] = -inf                              # three left of six
    x[3, 1::2] = float("nan")
    x[4, 5] = x[4, 90] = inf                     # count as the largest finite value
    x[5] = torch.finfo(dtype).min                # the type's lowest value is an ordinary logit
    x[6] = torch.finfo(dtype).min
    x[6, 40] = 1.0
    x[7] *= 1e30
    for bias in (None, np.linspace(-0.2, 0.2, E)):
        for form in (dict(), dict(num_groups=4, topk_groups=2, group_top=2 if score == "sigmoid" else 1)):
            for renorm in (True, False):
                b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
                got = nv.nvfp4_route_topk(x, k, bias=b, score=score, renormalize=renorm, **form)
                ids, w = got["expert_ids"].cpu().numpy(), got["weights"].cpu().numpy()
                want_ids, want_w, margin = mo.route_topk(host(x), k, None if bias is None else bias.astype(np.float32),
                                                         score, renormalize=renorm, **form)
                assert np.all(np.isfinite(w))
                assert np.all(ids[0] == -1) and np.all(ids[1] == -1) and np.all(w[:2] == 0)
                assert np.array_equal(ids[2] == -1, want_ids[2] == -1)
                assert np.all((ids[3] % 2 == 0) | (ids[3] == -1))
                if bias is None and not form:
                    assert np.array_equal(ids, want_ids)
                for t in (2, 3, 4, 6, 8, 9, 10, 11):
                    if margin[t] > KEY_TOL:
                        assert np.array_equal(ids[t], want_ids[t]), t
                        assert np.allclose(w[t], want_w[t], rtol=W_TOL, atol=1e-30), t


def test_route_strided_rows_and_no_write_past_the_ends():
    big = make_logits(50, 300, torch.float32, 2)
    for off, E in [(0, 256), (4, 256), (1, 255), (3, 64)]:
        x = big[:, off:off + E]
        a = nv.nvfp4_route_topk(x, 8)
        b = nv.nvfp4_route_topk(x.contiguous(), 8)
        assert torch.equal(a["expert_ids"], b["expert_ids"]) and torch.equal(a["weights"], b["weights"])
        g = torch.randn(50, 8, device="cuda")
        out = torch.full((50, 300), 7.0, device="cuda")
        nv.nvfp4_route_topk_backward(x, a["expert_ids"], g, out=out[:, off:off + E])
        want = nv.nvfp4_route_topk_backward(x.contiguous(), a["expert_ids"], g)
        assert torch.equal(out[:, off:off + E], want)
        assert torch.all(out[:, :off] == 7.0) and torch.all(out[:, off + E:] == 7.0)


def backward_scale(x, ids, grad, score, renorm, scale):
    """Sum of the absolute terms of each gradient element's formula."""
    s = mo.scores(x, score)
    out = np.zeros_like(s)
    for t in range(s.shape[0]):
        j = np.flatnonzero((ids[t] >= 0) & (ids[t] < s.shape[1]))
        e, d = ids[t, j], np.abs(grad[t, j]) * scale
        total = s[t, e].sum()
        if renorm and total > 0:
            ds = (d + (d * s[t, e]).sum() / total) / total
        else:
            ds = d
        if score == "sigmoid":
            out[t, e] = ds * s[t, e] * (1 - s[t, e])
        elif renorm:
            out[t, e] = ds * s[t, e]
        else:
            out[t] = s[t] * (d * s[t, e]).sum()
            out[t, e] += s[t, e] * d
    return out


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (70, 63, 6), (33, 160, 6), (300, 256, 8), (9, 1024, 32),
                                   (6, 1001, 10)])
def test_route_backward(T, E, k, dtype, renorm, score):
    x = make_logits(T, E, dtype, 13 * T + E, spread=2.0)
    ids = nv.nvfp4_route_topk(x, k, score=score)["expert_ids"]
    if T > 2:
        ids[1, 0] = -1                           # a slot without an expert
        ids[2, 0] = E + 3                        # out of range: contributes nothing
    g = torch.from_numpy(np.random.default_rng(5).standard_normal((T, k)).astype(np.float32)).cuda()
    got = host(nv.nvfp4_route_topk_backward(x, ids, g, score=score, renormalize=renorm, scale=2.5))
    xh, ih, gh = host(x), ids.cpu().numpy(), host(g)
    want = mo.route_topk_backward(xh, ih, gh, score, renorm, 2.5)
    tol = 2.0 ** -17 * backward_scale(xh, ih, gh, score, renorm, 2.5) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)     # the result's own rounding
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(score, renorm):
    """Central differences of the 64-bit forward pass, step h: truncation h^2/6
    of the third derivative (below 8 |grad| scale), rounding 2^-52 / h."""
    T, E, k, h = 3, 24, 4, 1e-4
    x = make_logits(T, E, torch.float32, 77)
    got_f = nv.nvfp4_route_topk(x, k, score=score, renormalize=renorm)
    g = torch.from_numpy(np.random.default_rng(6).standard_normal((T, k)).astype(np.float32)).cuda()
    got = host(nv.nvfp4_route_topk_backward(x, got_f["expert_ids"], g, score=score, renormalize=renorm))
    xh, ids, gh = host(x), got_f["expert_ids"].cpu().numpy(), host(g)

    def loss(v):
        s = mo.scores(v, score)
        w = np.take_along_axis(s, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (w * gh).sum(1)

    for e in range(E):
        up, down = xh.copy(), xh.copy()
        up[:, e] += h
        down[:, e] -= h
        diff = (loss(up) - loss(down)) / (2 * h)
        assert np.all(np.abs(diff - got[:, e]) <= 8 * h * h * np.abs(gh).sum(1) + 1e-5 * np.abs(gh).sum(1))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_backward_large_and_masked_logits_stay_finite(score):
    x = make_logits(6, 64, torch.float32, 4)
    x[0] = -float("inf")
    x[1, 10:] = -float("inf")
    x[2] = 80.0
    x[3] = -80.0
    x[4, 7] = float("inf")
    for renorm in (True, False):
        r = nv.nvfp4_route_topk(x, 8, score=score, renormalize=renorm)
        g = torch.ones(6, 8, device="cuda") * torch.arange(8, device="cuda")
        out = nv.nvfp4_route_topk_backward(x, r["expert_ids"], g, score=score, renormalize=renorm)
        assert bool(torch.isfinite(out).all())
        assert bool((out[0] == 0).all()) and bool((out[1, 10:] == 0).all())


def test_route_on_another_stream_and_in_a_graph():
    x = make_logits(512, 256, torch.bfloat16, 9)
    want = nv.nvfp4_route_topk(x, 8)
    s = torch.cuda.Stream()
    got = nv.nvfp4_route_topk(x, 8, stream=s)
    s.synchronize()
    assert torch.equal(got["expert_ids"], want["expert_ids"])
    call, out = nv.prepare_route_topk(x, 8)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(make_logits(512, 256, torch.bfloat16, 10))
    graph.replay()
    torch.cuda.synchronize()
    want = nv.nvfp4_route_topk(x.clone(), 8)
    assert torch.equal(out["expert_ids"], want["expert_ids"]) and torch.equal(out["weights"], want["weights"])


def test_route_refusals():
    x = make_logits(4, 64, torch.float32, 1)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(x, 65)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(make_logits(2, 1025, torch.float32, 1), 4)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(x, 33)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(x, 4, num_groups=5, topk_groups=2)       # 64 % 5
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(x, 9, num_groups=8, topk_groups=1)       # 8 experts left
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_topk(x[:0], 4)
    with pytest.raises(TypeError):
        nv.nvfp4_route_topk(x.half(), 4)
    with pytest.raises(TypeError):
        nv.nvfp4_route_topk(x.cpu(), 4)
    with pytest.raises(ValueError):
        nv.nvfp4_route_topk(x.t(), 4)
    with pytest.raises(ValueError):
        nv.nvfp4_route_topk(x, 4, bias=torch.zeros(63, device="cuda"))
    ids = torch.zeros(4, 4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        nv.nvfp4_route_topk_backward(x, ids, torch.zeros(4, 4, device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k", [(64, 6), (63, 6), (256, 8), (250, 8), (1024, 20), (1001, 20)])
def test_route_backward_softmax_at_any_offset(E, k, dtype):
    """The dense softmax gradient of rows far from zero: all logits equal, two
    equal largest ones over the others, and a spread of ordinary size around
    the offset, for rows in whole vectors and not.  The differences of a row's
    logits are exact in fp32 or so large that their exponential is 0, so the
    tolerance of test_route_backward holds unchanged."""
    top = float(torch.finfo(dtype).max)
    offsets = [0.0] + [s * v for v in (100.0, 3e4, 1e6, 3e10, 1.0007e12, 1e15, 1e30, 2.5e38, top) for s in (1, -1)]
    rng = np.random.default_rng(E)
    rows = []
    for v in offsets:
        rows.append(np.full(E, v))
        tied = np.full(E, v / 2 if v > 0 else max(2 * v, -top))
        tied[[3, E - 2]] = v
        rows.append(tied)
        rows.append(np.clip(v + rng.standard_normal(E) * 2.0, -top, top))
    x = torch.from_numpy(np.array(rows)).to(dtype).cuda()
    T = x.shape[0]
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    ids[::2, 0], ids[::2, 1] = 3, E - 2
    for t in range(T):                       # one of each (a duplicate of the two above counts as missing)
        seen = set()
        for j in range(k):
            if ids[t, j] in seen:
                ids[t, j] = -1
            seen.add(ids[t, j])
    g = rng.standard_normal((T, k)).astype(np.float32)
    got = host(nv.nvfp4_route_topk_backward(x, torch.from_numpy(ids.astype(np.int32)).cuda(),
                                            torch.from_numpy(g).cuda(), score="softmax", renormalize=False, scale=2.5))
    xh = host(x)
    want = mo.route_topk_backward(xh, ids, g.astype(np.float64), "softmax", False, 2.5)
    tol = 2.0 ** -17 * backward_scale(xh, ids, g.astype(np.float64), "softmax", False, 2.5) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    bad = np.argwhere(~(np.abs(got - want) <= tol))
    assert bad.size == 0, (len(bad), sorted({offsets[r // 3] for r in bad[:, 0]}), got[tuple(bad[0])],
                           want[tuple(bad[0])])


@pytest.mark.parametrize("E,k", [(64, 8), (63, 5), (96, 12), (95, 16), (256, 20)])
def test_route_infinity_ties_with_the_largest_finite_logit(E, k):
    """+inf counts as the largest finite fp32: beside logits of that value it takes
    its place by index, among experts and among groups."""
    top, inf = float(np.finfo(np.float32).max), float("inf")
    x = make_logits(9, E, torch.float32, 17)
    x[0, [0, 5]] = torch.tensor([top, inf], device="cuda")
    x[1, [0, 5]] = torch.tensor([inf, top], device="cuda")
    x[2, ::3], x[2, 1::3] = top, inf
    x[3, E - 1], x[3, 2] = inf, top
    x[4], x[4, 7] = top, inf
    x[5], x[5, 7] = inf, top
    x[6, 1], x[6, 0], x[6, 3] = float("nan"), top, inf
    x[7] = -inf
    x[7, [2, 30]] = torch.tensor([top, inf], device="cuda")
    forms = [dict()]
    for G in (2, 3, 4, 8):
        if E % G == 0:
            for kg in (1, 2):
                forms += [dict(num_groups=G, topk_groups=kg, group_top=t) for t in (1, 2) if k <= kg * (E // G)]
    for score in ("sigmoid", "softmax"):
        for form in forms:
            want, want_w, margin = mo.route_topk(host(x), k, score=score, **form)
            got = nv.nvfp4_route_topk(x, k, score=score, **form)
            sure = margin > KEY_TOL
            if form.get("group_top") == 2:       # equal sums of two scores go to the lowest group in both
                sure |= margin == 0
            ids = got["expert_ids"].cpu().numpy()
            assert np.array_equal(ids[sure], want[sure]), (score, form, np.argwhere(ids != want)[:4])
            assert np.allclose(got["weights"].cpu().numpy()[sure], want_w[sure], rtol=W_TOL, atol=1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k,bias", [(64, 8, False), (63, 5, True), (256, 12, False), (1000, 20, True), (8, 8, False),
                                      (12, 12, False), (20, 20, True)])
def test_route_sigmoid_far_below_zero(E, k, bias, dtype):
    """Renormalised sigmoid weights and their gradient where the scores reach fp32's
    smallest values: their ratios are those of the definition down to the largest
    score's own underflow (logits of -103.9), below which all weights are 0."""
    rng = np.random.default_rng(E)
    # (largest logit, spread below it); the spread's rounding in x - max stays below 2^-19
    rows = [(-70.0, 6.0), (-79.5, 6.0), (-81.0, 6.0), (-86.0, 6.0), (-88.5, 6.0), (-19.0, 60.0), (-21.0, 60.0),
            (-35.0, 60.0), (-75.0, 20.0), (-79.9, 15.0), (-95.0, 6.0), (-103.0, 6.0)]
    x = -200.0 - rng.random((len(rows) + 2, E))
    for t, (v, spread) in enumerate(rows):
        x[t] = v - rng.random(E) * spread
        x[t, rng.integers(E)] = v
    x[-2], x[-1] = -110.0 - rng.random(E), -3e38
    xt = torch.from_numpy(x).to(dtype).cuda()
    b = np.zeros(E) if bias else None
    got = nv.nvfp4_route_topk(xt, k, bias=None if b is None else torch.zeros(E, device="cuda"), scale=2.5)
    ids, w = got["expert_ids"].cpu().numpy(), host(got["weights"])
    xh = host(xt)
    # (with a bias the choice is by the fp32 scores, equal ones by index)
    zero = np.take_along_axis(xh, ids, 1).max(1) < -103.9
    assert zero[-2:].all() and not zero[:5].any()
    s = np.take_along_axis(mo.scores(xh, "sigmoid"), ids, 1)[~zero]
    want = 2.5 * s / s.sum(1, keepdims=True)
    assert np.all(np.abs(w[~zero] - want) <= W_TOL * want)
    assert np.all(w[zero] == 0)
    g = rng.standard_normal(w.shape).astype(np.float32)
    d = host(nv.nvfp4_route_topk_backward(xt, got["expert_ids"], torch.from_numpy(g).cuda(), scale=2.5))
    gh = g.astype(np.float64)
    want = mo.route_topk_backward(xh, ids, gh, "sigmoid", True, 2.5)[~zero]
    tol = 2.0 ** -17 * backward_scale(xh, ids, gh, "sigmoid", True, 2.5)[~zero] + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(d[~zero] - want) <= tol) and np.all(d[zero] == 0)
