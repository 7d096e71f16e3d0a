"""Attention over the key-value cache where a block works through many key tiles:
many sequences over the same pages, scores that climb, fall and jump between
tiles and within one, very large scores, NaN values.

Reference in 64 bits by torch on the GPU, from the packed bytes; the tolerances
are those that test_kv_gpu.py derives."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from oracle import kv_oracle as ko
from test_kv_gpu import normal, scales

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))


class Shared:
    """`lens` sequences of qn new tokens each (qn: a number or one per sequence), all on the same pages, which hold
    the keys k and values v, bf16 [n, kv heads, head_dim]."""

    def __init__(self, k, v, lens, qn, G, page=64, seed=0, g=None, q=None):
        n, H, hd = k.shape
        self.lens, self.H, self.G, self.hd, self.page = list(lens), H, G, hd, page
        self.qlens = [qn] * len(lens) if isinstance(qn, int) else list(qn)
        pages = (n + page - 1) // page
        order = np.random.default_rng(seed).permutation(pages + 1)[:pages]
        self.row = order.astype(np.int32)
        self.gk, self.gv = (scales(H, seed + 1), scales(H, seed + 2)) if g is None else (np.full(H, g, np.float32),) * 2
        self.dgk, self.dgv = torch.from_numpy(self.gk).cuda(), torch.from_numpy(self.gv).cuda()
        self.cache = nv.nvfp4_kv_cache(pages + 1, H, page, hd)
        j = np.arange(n)
        self.slots = torch.from_numpy(order[j // page].astype(np.int64) * page + j % page).cuda()
        nv.nvfp4_kv_write(k, v, self.slots, self.cache, self.dgk, self.dgv)
        self.offsets = np.concatenate([[0], np.cumsum(self.qlens)]).astype(np.int32)
        self.q = normal((int(self.offsets[-1]), H * G, hd), seed + 5) if q is None else q
        self.values()

    def values(self):
        """What the packed rows stand for, in 64 bits, [n, heads, hd]."""
        rows = self.slots.cpu().numpy()
        at, off = rows // self.page, rows % self.page
        c = {m: t.cpu().numpy() for m, t in self.cache.items()}
        self.k, self.v = (torch.from_numpy(ko.values(c[m + "_codes"][at, :, off], c[m + "_sf"][at, :, off], g)).cuda()
                          for m, g in (("k", self.gk), ("v", self.gv)))

    def prepare(self, **form):
        B = len(self.lens)
        table = torch.from_numpy(self.row)[None].expand(B, -1).contiguous().cuda()
        return nv.prepare_kv_attention(
            self.q, self.cache, self.dgk, self.dgv, table, torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
            q_offsets=torch.from_numpy(self.offsets).cuda(), max_q_len=max(self.qlens), want_lse=True, **form)

    def run(self, **form):
        call, got = self.prepare(**form)
        call()
        assert nv.read_device_status(call.workspace) == 0
        return got

    def scores(self, b, scale, causal, window):
        """[tokens, kv heads, group, keys] in 64 bits, -inf where a row does not see a key."""
        n, nq = self.lens[b], self.qlens[b]
        q = self.q[self.offsets[b]:self.offsets[b + 1]].double().reshape(nq, self.H, self.G, self.hd)
        s = torch.einsum("tkgd,nkd->tkgn", q, self.k[:n]) * scale
        j, pos = torch.arange(n, device="cuda"), (n - nq + torch.arange(nq, device="cuda"))[:, None]
        see = j <= pos if causal else torch.ones(nq, n, dtype=torch.bool, device="cuda")
        if window:
            see = see & (j > pos - window)
        return s.masked_fill(~see[:, None, None], -float("inf")), see, q

    def check(self, got, causal=True, window=0, scale=None, seqs=None):
        scale = self.hd ** -0.5 if scale is None else scale
        for b in (range(len(self.lens)) if seqs is None else seqs):
            rows = slice(int(self.offsets[b]), int(self.offsets[b + 1]))
            s, see, q = self.scores(b, scale, causal, window)
            k, v = self.k[:self.lens[b]], self.v[:self.lens[b]]
            top = s.amax(-1, keepdim=True)
            e = torch.exp(s - top)
            total = e.sum(-1, keepdim=True)
            w = e / total
            want = torch.einsum("tkgn,nkd->tkgd", w, v)
            lse = (top + torch.log(total)).squeeze(-1)
            S = torch.einsum("tkgn,nkd->tkgd", w, v.abs())
            V = torch.einsum("tn,nkd->tkd", see.double(), v.abs())[:, :, None] / total
            qk = torch.einsum("tkgd,nkd->tkgn", q.abs(), k.abs()).masked_fill(~see[:, None, None], 0).amax(-1)
            n = self.lens[b]
            d = (self.hd / 16 + 2) * 2.0 ** -22 * scale * qk + 2.0 ** -22 * (lse.abs() + np.log(max(n, 2)) + 2)
            tol = ((2.0 ** -11 + 2 * d[..., None] + (n / 16 + 2) * 2.0 ** -22) * S + 2.0 ** -25 * V
                   + 2.0 ** -8 * want.abs())
            y, z = got[0][rows].double().reshape(want.shape), got[1][rows].double().reshape(lse.shape)
            bad = ~((y - want).abs() <= tol * 1.0001)
            assert not bool(bad.any()), (b, int(bad.sum()), bad.nonzero()[:3], y[bad][:4], want[bad][:4], tol[bad][:4])
            far = ~((z - lse).abs() <= d + 2.0 ** -21 * (lse.abs() + 2))
            assert not bool(far.any()), (b, z[far][:4], lse[far][:4])


def along(height, H, hd):
    """Keys whose first channel is `height` [n], bf16: with a query of ones there, their scores."""
    k = torch.zeros(len(height), H, hd)
    k[:, :, 0] = height[:, None]
    return k.to(torch.bfloat16).cuda()


def first_channel(rows, heads, hd, value=1.0):
    q = torch.zeros(rows, heads, hd, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = value
    return q


# ------------------------------------------------------------- large scores --

@pytest.mark.parametrize("power", [20, 24, 27, 28, 29, 31, 34, 40, 60, 90])
@pytest.mark.parametrize("qn,G,hd", [(1, 4, 128), (3, 8, 64), (8, 8, 128), (32, 8, 64), (5, 64, 128)])
def test_large_scores(qn, G, hd, power):
    """Scores about 2^power: the softmax is 1 at the largest, 0 elsewhere, where the largest leads by more than what
    fp32 sums of such products can be off by (d, twice) and 40.  The result is that key's value: the numerator's
    rounding to f16 (2^-11) and the result's to bf16 (2^-8), 1000 others times e^-40 times less than 2^8; the
    logarithm is its score, to d and three roundings."""
    n, H, B = 1000, 2, 6
    k, v = normal((n, H, hd), power), normal((n, H, hd), power + 1)
    c = Shared(k, v, [n, n, 700, 513, 129, 64], qn, G, seed=power)
    size = c.q.float() * 2.0 ** (power - 4 + 4 * torch.rand(c.q.shape[:2], device="cuda"))[..., None]
    c.q = size.to(torch.bfloat16)
    scale = hd ** -0.5
    out, lse = c.run(scale=scale, causal=False)
    checked = 0
    for b in range(B):
        rows = slice(int(c.offsets[b]), int(c.offsets[b + 1]))
        s, _, q = c.scores(b, scale, False, 0)
        qk = scale * torch.einsum("tkgd,nkd->tkgn", q.abs(), c.k[:c.lens[b]].abs()).amax(-1)
        two, at = s.topk(2, -1)
        d = (hd / 16 + 4) * 2.0 ** -22 * qk
        sure = two[..., 0] - two[..., 1] > 2 * d + 40
        checked += int(sure.sum())
        want = c.v[:c.lens[b]].permute(1, 0, 2)[torch.arange(H, device="cuda")[None, :, None], at[..., 0]]
        y, z = out[rows].double().reshape(want.shape), lse[rows].double().reshape(sure.shape)
        ok = ((y - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * 1.001 * want.abs() + 2.0 ** -39).all(-1)
        assert bool(ok[sure].all()), (b, int((~ok & sure).sum()), int(sure.sum()))
        assert bool(((z - two[..., 0]).abs() <= d + 2.0 ** -22 * two[..., 0].abs())[sure].all())
    assert checked > 0.9 * c.q.shape[0] * H * G


@pytest.mark.parametrize("qn,G", [(1, 8), (5, 4)])
@pytest.mark.parametrize("low,step", [(14, 8), (18, 8), (18, 10), (19, 8), (20, 8), (21, 16), (23, 64)])
@pytest.mark.parametrize("H,n,B", [(4, 1024, 120), (2, 4096, 130)])
def test_exact_steps_between_large_scores(H, n, B, low, step, qn, G):
    """Scores 96 * 2^low, and `step` more from some key on, which fp32 holds exactly (its spacing there is
    2^(low - 17)), but not sums of a score and 7 or 15.  In powers of two (scale ln 2, all factors exact)."""
    k = torch.zeros(n, H, 64)
    k[:, :, 0], k[:, :, 16] = 96.0, 6.0           # blocks' scale bytes 16 and 1
    late = torch.arange(n) % 512 >= 300
    k[late, :, 17] = 4.0
    q = first_channel(B * qn, H * G, 64, 2.0 ** low)
    q[:, :, 17] = step / 4
    c = Shared(k.to(torch.bfloat16).cuda(), normal((n, H, 64), 1), [n - 7 * (i % 5) for i in range(B)], qn, G, g=1.0, q=q)
    assert torch.equal(c.k.float().cpu(), k)
    out, lse = c.run(scale=LN2, causal=False)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    for b in (0, 1, B // 2, B - 2, B - 1):
        rows = slice(int(c.offsets[b]), int(c.offsets[b + 1]))
        e = torch.exp2(step * late[:c.lens[b]].double() - step).cuda()
        v = c.v[:c.lens[b]]
        want = torch.einsum("n,nkd->kd", e, v) / e.sum()
        bound = torch.einsum("n,nkd->kd", e, v.abs()) / e.sum()
        y = out[rows].double().reshape(-1, H, G, 64)
        # every difference of scores is exact: the numerators' rounding, the sums', the result's
        tol = (2.0 ** -11 + (n / 16 + 4) * 2.0 ** -22) * bound + 2.0 ** -25 * v.abs().sum(0) / e.sum() + 2.0 ** -8 * want.abs()
        assert bool(((y - want[None, :, None]).abs() <= tol[None, :, None] * 1.0001).all())


# --------------------------------------------- references that have to follow --

@pytest.mark.parametrize("low", [20.25, 21.0])
@pytest.mark.parametrize("hd", [64, 128])
def test_many_keys_below_many_of_the_largest(hd, low):
    """A tile whose 128 keys are all the row's largest, after a tile slightly below, both without a value, and
    thousands of keys 2^-low of them: the whole result is theirs."""
    n = 8192
    height = torch.full((n,), -low)
    height[:128], height[128:256] = -2.0, 0.0
    v = torch.zeros(n, 1, hd, dtype=torch.bfloat16, device="cuda")
    v[256:] = 6.0
    c = Shared(along(height, 1, hd), v, [n] * 170, 32, 8, g=1.0, q=first_channel(170 * 32, 8, hd))
    c.check(c.run(scale=LN2, causal=False), causal=False, scale=LN2, seqs=range(0, 170, 13))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("top", [13.5, 20.0, 27.0, 39.0])
def test_a_jump_behind_others_in_a_tile(hd, top):
    """Within one tile 96 keys of 2^6.75 and then one of 2^top: the first ones' numerators, written already, follow
    the reference, and the result is theirs (the top key has no value)."""
    n = 256
    height = torch.zeros(n)
    height[128:224], height[240] = 6.75, top
    v = torch.zeros(n, 2, hd, dtype=torch.bfloat16, device="cuda")
    v[128:224] = 6.0
    c = Shared(along(height, 2, hd), v, [n] * 300, 32, 8, g=1.0, q=first_channel(300 * 32, 16, hd))
    c.check(c.run(scale=LN2, causal=False), causal=False, scale=LN2, seqs=range(0, 300, 17))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("size", [-30, -70, -100, -120, -126])
@pytest.mark.parametrize("qn,G", [(1, 8), (12, 8)])
def test_small_queries_under_a_large_scale(qn, G, hd, size):
    """Queries of 2^size under a scale of 2^-size: the products are ordinary.  (bf16 holds less than eight bits of
    numbers below 2^-126: the reference takes what it holds.)"""
    n = 300
    c = Shared(normal((n, 2, hd), 1), normal((n, 2, hd), 2), [n, 100], qn, G, seed=3)
    c.q = (c.q.double() * 2.0 ** size).to(torch.bfloat16)
    scale = 2.0 ** -size * hd ** -0.5
    c.check(c.run(scale=scale), scale=scale)


# --------------------------------------------------------------- NaN values --

def test_nan_of_one_sequence_does_not_hold_up_the_others():
    """A value with a NaN scale in two long sequences among others: its channels of the rows that see it are NaN,
    every other row has the same bits as without it, and no wait runs out that is far longer than the work."""
    n, H, hd, qn = 32768, 2, 128, 32
    lens = [n - 64 * (b % 12) for b in range(96)]
    c = Shared(normal((n, H, hd), 1), normal((n, H, hd), 2), lens, qn, 8)
    page = torch.arange(c.cache["k_codes"].shape[0], device="cuda")
    spare = int(page[~torch.isin(page, torch.from_numpy(c.row).cuda())][0])
    call, (out, lse) = c.prepare()
    call()
    assert nv.read_device_status(call.workspace) == 0
    want = out.clone(), lse.clone()
    # page 40 of the third sequence and of another becomes a copy whose key 7 has a NaN in head 1, channels 48 to 63
    at = 40
    for t in c.cache.values():
        t[spare] = t[int(c.row[at])]
    c.cache["v_sf"][spare, 1, 7, 3] = 0x7F
    table = torch.from_numpy(c.row)[None].expand(len(lens), -1).contiguous().cuda()
    table[[2, 60], at] = spare
    call, (out, lse) = nv.prepare_kv_attention(
        c.q, c.cache, c.dgk, c.dgv, table, torch.tensor(lens, dtype=torch.int32, device="cuda"),
        q_offsets=torch.from_numpy(c.offsets).cuda(), max_q_len=qn, want_lse=True)
    old = nv.set_wait_timeout_ns(2_000_000)
    try:
        call()
        assert nv.read_device_status(call.workspace) == 0
    finally:
        nv.set_wait_timeout_ns(old)
    hit = torch.zeros_like(out, dtype=torch.bool)
    for b in (2, 60):
        hit[b * qn:(b + 1) * qn, 8:, 48:64] = True
    assert bool(torch.isnan(out[hit]).all())
    assert torch.equal(out[~hit], want[0][~hit]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 700), (False, 0)])
@pytest.mark.parametrize("qn,G", [(1, 8), (3, 8), (40, 8)])
def test_nan_values_in_long_sequences(qn, G, causal, window, hd):
    """NaN scales at tiles' borders, in the first key and the last: NaN for the rows that see them, in their
    16 channels, and the other channels right."""
    n, H = 1500, 2
    c = Shared(normal((n, H, hd), 1), normal((n, H, hd), 2), [n, 1400, 513, 300] * 12, qn, G, seed=hd)
    spots = [(0, 0, 0), (127, 1, 1), (128, 0, hd // 16 - 1), (777, 1, 2), (1399, 0, 1), (1485, 0, 0), (1499, 1, 3)]
    for j, h, block in spots:
        slot = int(c.slots[j])
        c.cache["v_sf"][slot // c.page, h, slot % c.page, block] = 0x7F
    out, lse = c.run(causal=causal, window=window)
    for b in range(len(c.lens)):
        rows, m = slice(int(c.offsets[b]), int(c.offsets[b + 1])), c.lens[b]
        s, see, _ = c.scores(b, hd ** -0.5, causal, window)
        y = out[rows].double().reshape(qn, H, G, hd)
        nan = torch.zeros(qn, H, G, hd, dtype=torch.bool, device="cuda")
        for j, h, block in spots:
            if j < m:
                nan[:, h, :, 16 * block:16 * block + 16] |= see[:, j, None, None]
        assert torch.equal(torch.isnan(y), nan)
        w = torch.softmax(s, -1)
        want = torch.einsum("tkgn,nkd->tkgd", w, c.v[:m])
        # unit scores: f16 numerators, bf16 results, the sums of some thousand fp32 terms (2^-12 in all)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12) * torch.einsum("tkgn,nkd->tkgd", w, c.v[:m].abs())
        assert bool(((y - want).abs() <= tol)[~nan].all())


# ------------------------------------------------------------- wide windows --

@pytest.mark.parametrize("window", [2 ** 31, 2 ** 40, 2 ** 63 - 1])
@pytest.mark.parametrize("qn,G", [(1, 8), (5, 4), (400, 8)])
def test_windows_wider_than_any_sequence(qn, G, window):
    """They are no window, with more new tokens than keys too."""
    n = 390
    c = Shared(normal((n, 2, 64), 1), normal((n, 2, 64), 2), [n, 3, 200], qn, G)
    want, got = c.run(), c.run(window=window)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------- heads outermost --

@pytest.mark.parametrize("lens,qn,G", [([300, 40], 1, 4), ([300, 40], 5, 4), ([700, 128], 60, 8)])
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_with_heads_outermost(lens, qn, G, hd):
    """Queries, keys, values and results as transposes of [heads, tokens, head_dim] give the same bits."""
    n, H = 700, 3
    k, v = normal((n, H, hd), 1), normal((n, H, hd), 2)
    c = Shared(k, v, lens, qn, G)
    want, before = c.run(), {m: t.clone() for m, t in c.cache.items()}
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v, c.q)]
    assert turned[0].stride(0) == hd
    for t in c.cache.values():
        t.zero_()
    nv.nvfp4_kv_write(turned[0], turned[1], c.slots, c.cache, c.dgk, c.dgv)
    assert all(torch.equal(c.cache[m][c.row], before[m][c.row]) for m in before)
    c.q = turned[2]
    out = torch.full((H * G, len(lens) * qn + 2, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    got = c.run(out=out[:, 1:-1].transpose(0, 1))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((out[:, 0] == 7).all()) and bool((out[:, -1] == 7).all())
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((2, H, n + 2, hd), 7.0, dtype=dtype, device="cuda")
        rows = nv.nvfp4_kv_read(c.slots, c.cache, c.dgk, c.dgv, out=tuple(t[:, 1:-1].transpose(0, 1) for t in wide))
        plain = nv.nvfp4_kv_read(c.slots, c.cache, c.dgk, c.dgv, out_dtype=dtype)
        assert all(torch.equal(a, b) for a, b in zip(rows, plain))
        assert bool((wide[:, :, 0] == 7).all()) and bool((wide[:, :, -1] == 7).all())
