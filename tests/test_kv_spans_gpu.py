"""Attention over the key-value cache where every block works through several
segments of many key tiles each (5 places of the line a block and more, two
segments in some), compared with 64 bits: references that follow climbing,
falling and jumping scores, ragged prompts and windows whose queries replace one
another, offsets that do not fit.  Reference and tolerances: test_kv_scores_gpu.py."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from test_kv_gpu import Case, normal
from test_kv_scores_gpu import LN2, Shared

pytestmark = pytest.mark.gpu


def steps(n, every, by):
    return (torch.arange(n) // every).float() * by


def saw(n):
    j = torch.arange(n)
    return torch.where(j // 512 % 2 == 0, (j % 512) * 0.12, 60 - (j % 512) * 0.12)


def chunk_jumps(n):
    """20 more in a later chunk of 32 of every third tile of 128, another one each time."""
    j = torch.arange(n)
    return 20.0 * sum((j >= 384 * t + 32 * ((t + 1) % 4)).float() for t in range(1, n // 384 + 1))


def hills(height, qn, G, lens, H, hd, seed=0):
    """Keys whose scores are `height` (in powers of two) and random ones of a few units, by queries of that kind."""
    n = len(height)
    k = normal((n, H, hd), seed + 1)
    k[:, :, :16] = 0
    k[:, :, 0] = height[:, None].to(torch.bfloat16).cuda()
    c = Shared(k, normal((n, H, hd), seed + 2), lens, qn, G, g=1.0, seed=seed)
    c.q = (c.q.float() * (2.0 / hd ** 0.5)).to(torch.bfloat16)
    c.q[:, :, 0] = 1.0
    return c


# A row's first keys leave it 2^3 to 2^4 for the largest numerator.  Steps of 5 from tile to tile: sums of 2^14 to
# 2^16, raised before the next tile.  Of 14 and 40, and the jumps within a tile: a chunk's sum is beyond f16.
SHAPES = {
    "raised between tiles": lambda n: steps(n, 128, 5.0),
    "chunks done again": lambda n: steps(n, 128, 14.0),
    "far steps": lambda n: steps(n, 128, 40.0),
    "jumps within tiles": chunk_jumps,
    "slow climb": lambda n: torch.arange(n) * 0.02,
    "fall": lambda n: 300 - torch.arange(n) * 0.07,
    "up and down": saw,
}


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("hd", [64, 128])
def test_many_rows_over_many_tiles(shape, hd):
    n = 4096
    c = hills(SHAPES[shape](n), 256, 8, [n], 8, hd)
    for causal, window in ((False, 0), (True, 0), (True, 1500)):
        c.check(c.run(scale=LN2, causal=causal, window=window), causal=causal, window=window, scale=LN2)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("qn,G", [(1, 8), (1, 1), (3, 8), (5, 2)])
@pytest.mark.parametrize("H,n,B", [(2, 4096, 130), (4, 1024, 120)])
def test_few_rows_over_many_units(H, n, B, qn, G, shape):
    """19 units of 32 keys a warp, that all warps of a block share, or 32 of a warp's own head; scores climb by more
    than 15 within them."""
    # (as steep for a quarter of the keys)
    height = SHAPES[shape](4 * n)[::4] if n < 4096 else SHAPES[shape](n)
    c = hills(height, qn, G, [n - 13 * (i % 9) for i in range(B)], H, 64)
    c.check(c.run(scale=LN2, causal=False), causal=False, scale=LN2, seqs=(0, 1, 7, B // 2, B - 1))
    c.check(c.run(scale=LN2), scale=LN2, seqs=(0, 5, B - 1))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 200), (False, 0)])
def test_ragged_prompts(hd, causal, window):
    """Whole prompts, most blocks with several segments, tiles with one and with two halves of rows."""
    lens = [1500, 129, 700, 3, 256, 31, 1023, 65]
    c = Shared(normal((1500, 8, hd), 1), normal((1500, 8, hd), 2), lens, lens, 4, seed=hd)
    c.check(c.run(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("hd", [64, 128])
def test_later_chunks_of_several_sequences(hd):
    """Chunks over longer contexts beside single tokens and drafted ones: both kernels in one call."""
    lens, qlens = [3000, 2900, 1, 700, 2000, 130, 2999], [300, 1, 1, 5, 77, 130, 33]
    c = Shared(normal((3000, 4, hd), 1), normal((3000, 4, hd), 2), lens, qlens, 8, page=16, seed=hd)
    for window in (0, 333):
        c.check(c.run(window=window), window=window)


def test_rows_around_a_climbing_one_keep_their_bits():
    """With many rows a row's result does not depend on the others' scores."""
    n = 2048
    c = hills(SHAPES["chunks done again"](n), 64, 8, [n] * 4, 4, 64)
    climbs = torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(0)).cuda() < 0.3
    large = torch.rand(c.q.shape[:2], generator=torch.Generator().manual_seed(1)).cuda() < 0.1
    c.q[:, :, 0] = 0
    flat = c.run(scale=LN2, causal=False)
    c.q[:, :, 0] = climbs.to(torch.bfloat16) * torch.where(large, 2.0 ** 20, 1.0).to(torch.bfloat16)
    got = c.run(scale=LN2, causal=False)
    for a, b in zip(got, flat):
        assert torch.equal(a[~climbs], b[~climbs])
        assert bool(torch.isfinite(a).all()) and not bool((a[climbs] == b[climbs]).all())


@pytest.mark.parametrize("most", [48, 8, 1])
@pytest.mark.parametrize("G", [1, 8])
def test_status_of_offsets_that_do_not_fit(G, most):
    """Offsets that overlap, descend or leave q: no wait runs out and no index is out of range, by the call's own
    status word; those that do fit give their rows."""
    c = Case([100] * 6, [8] * 6, 2, G, 128, 16)
    table, lens = torch.from_numpy(c.table).cuda(), torch.tensor([100] * 6, dtype=torch.int32, device="cuda")
    offsets = torch.empty(7, dtype=torch.int32, device="cuda")
    out = torch.empty_like(c.q)
    call, (out, lse) = nv.prepare_kv_attention(c.q, c.cache, c.dgk, c.dgv, table, lens, q_offsets=offsets,
                                               max_q_len=most, want_lse=True, out=out)
    for values in ([0, 48, 0, 48, 0, 48, 0], [-5, 10, 1000, 3, 2, 60, 48], [48, 40, 30, 20, 10, 5, 0],
                   [2 ** 31 - 1] * 7, [-2 ** 31] * 7):
        offsets.copy_(torch.tensor(values))
        call()
        assert nv.read_device_status(call.workspace) == 0
    fit = [0, 5, 9, 17, 20, 30, 41]
    offsets.copy_(torch.tensor(fit))
    out.fill_(7.0)
    call()
    assert nv.read_device_status(call.workspace) == 0
    assert bool((out[41:] == 7).all())
    c.qlens, c.offsets = list(np.diff(fit)), np.array(fit, np.int32)
    if most >= max(c.qlens):
        c.check((out, lse))
        return
    full = nv.nvfp4_kv_attention(c.q, c.cache, c.dgk, c.dgv, table, lens, q_offsets=offsets, max_q_len=48)
    at = torch.cat([torch.arange(a, a + min(most, b - a)) for a, b in zip(fit, fit[1:])]).cuda()
    kept = torch.ones(48, dtype=torch.bool, device="cuda")
    kept[at] = False
    assert bool((out[kept] == 7).all())
    # the same rows by another kernel or split: two roundings to bf16, numerators to f16
    assert torch.allclose(out[at].float(), full[at].float(), atol=2e-3, rtol=2.0 ** -7)
