"""Where the key-value cache's attention can go wrong: masks that leave rows
empty, device data that do not fit, NaN and stale bytes where nothing looks,
scores that grow, strides, buffers past 32 bits, graphs, streams, workspaces that
hold old results.  Cases, reference and tolerances: test_kv_gpu.py."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from nvfp4_block_scaled_06_gb300._binding import ERR_TIMEOUT
from test_kv_gpu import Case, normal, scales

pytestmark = pytest.mark.gpu

# (new tokens, heads per key-value head): the kernel for few rows with one to three row tiles, the one for many, both
SHAPES = [([1, 1, 1], 4), ([2, 1, 2], 8), ([5, 3, 5], 4), ([40, 1, 70], 8), ([1, 1, 1], 64)]


@pytest.mark.parametrize("qlens,G", SHAPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_rows_without_keys(qlens, G, hd):
    """Lengths of 0 (and below), and more queries than keys: zeros and -inf."""
    c = Case([70, 90, 130], qlens, 2, G, hd, 16, seed=G)
    lens = torch.tensor([0, -7, 33], dtype=torch.int32, device="cuda")
    c.check(c.run(kv_lens=lens), lens=[0, 0, 33])
    c.check(c.run(kv_lens=lens, causal=False), causal=False, lens=[0, 0, 33])
    c.check(c.run(kv_lens=lens, window=5), window=5, lens=[0, 0, 33])


@pytest.mark.parametrize("qlens,G", SHAPES)
@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_cache(qlens, G, page):
    """Keys of such pages are left out; lengths beyond the table end with it."""
    c = Case([300, 200, 260], qlens, 2, G, 128, page, seed=page)
    table = c.table.copy()
    pages = c.cache["k_codes"].shape[0]
    table[0, 1], table[1, 0], table[2, -1], table[2, 2] = -1, pages, 1 << 30, -(1 << 31)
    width = table.shape[1] * page
    lens = [300, 200, 10 ** 9]
    got = c.run(page_table=torch.from_numpy(table).cuda(), kv_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    c.check(got, table=table, lens=[300, 200, width])
    nothing = np.full_like(table, -1)
    c.check(c.run(page_table=torch.from_numpy(nothing).cuda()), table=nothing)


def test_offsets_that_do_not_fit():
    """They are clamped: no access outside the buffers, rows of no sequence stay as they were."""
    c = Case([100] * 6, [8] * 6, 2, 8, 128, 16)
    guard = torch.full((80, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    for offsets in ([0, 48, 0, 48, 0, 48, 0], [-5, 10, 1000, 3, 2, 60, 48], [48, 40, 30, 20, 10, 5, 0],
                    [2 ** 31 - 1] * 7, [-2 ** 31] * 7, [0, 5, 9, 17, 20, 30, 41]):
        guard.fill_(7.0)
        t = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        for most in (48, 8, 1):
            out, lse = c.run(q_offsets=t, max_q_len=most, out=guard[16:64])
            assert out.data_ptr() == guard[16:64].data_ptr()
            assert nv.read_device_status(None) == 0
            assert bool((guard[:16] == 7).all()) and bool((guard[64:] == 7).all())
    assert bool((guard[16 + 41:64] == 7).all()) and not bool((guard[16:16 + 41] == 7).all())


@pytest.mark.parametrize("G", [1, 4, 8, 16])
def test_rows_beyond_the_sequences_and_the_bound(G):
    """Rows past the last offset, and of a sequence past max_q_len, are left as they were; the others are right."""
    c = Case([90, 64, 200], [12, 1, 7], 2, G, 64, 16, seed=G)
    q = torch.cat([c.q, normal((9, 2 * G, 64), 77)])
    out = torch.full_like(q, 3.0)
    got, lse = c.run(q=q, out=out)
    c.check((got[:20], lse[:20]))
    assert bool((got[20:] == 3).all())
    whole = got[:20].clone()
    out.fill_(3.0)
    got, _ = c.run(q=q, out=out, max_q_len=5)
    first = torch.tensor([i < 5 for i in range(12)] + [True] + [i < 5 for i in range(7)], device="cuda")
    assert bool((got[:20][~first] == 3).all())
    assert torch.allclose(got[:20][first].float(), whole[first].float(), atol=2e-2, rtol=2e-2)
    assert not bool((got[:20][first] == 3).all(-1).any())


@pytest.mark.parametrize("qlens,G", SHAPES)
@pytest.mark.parametrize("hd", [64, 128])
def test_stale_bytes(qlens, G, hd):
    """Bytes behind a sequence's end and in pages that no table names do not reach a row."""
    lens = [37, 129, 300]
    c = Case(lens, qlens, 2, G, hd, 32, seed=3)
    want = [t.clone() for t in c.run()]
    seen = torch.zeros(c.cache["k_codes"].shape[0], 32, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        j = np.arange(n)
        seen[torch.from_numpy(c.table[b][j // 32]).long().cuda(), torch.from_numpy(j % 32).cuda()] = True
    for t in c.cache.values():
        t.copy_(torch.where(seen[:, None, :, None], t, torch.full_like(t, 0xFF)))
    for a, b in zip(c.run(), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("qlens,G", [([1, 1], 4), ([6, 3], 4), ([3, 2], 8), ([90, 30], 8), ([64, 200], 3)])
@pytest.mark.parametrize("window", [0, 9])
@pytest.mark.parametrize("what", ["k", "v"])
def test_nan_reaches_the_rows_that_see_it(qlens, G, window, what):
    """A key with a NaN scale makes the rows that see it NaN; a value's its 16 channels of them."""
    lens = [qlens[0] + 20, qlens[1] + 111]
    c = Case(lens, qlens, 2, G, 128, 16, seed=5)
    for b, h, j, blk in ((0, 1, lens[0] - 1, 3), (0, 0, max(0, lens[0] - 3), 0), (1, 1, 60, 7), (1, 0, lens[1] - 2, 5)):
        c.cache[what + "_sf"][int(c.table[b, j // 16]), h, j % 16, blk] = 0x7F
    c.check(c.run(window=window), window=window)
    c.check(c.run(causal=False), causal=False)


@pytest.mark.parametrize("qlens,G", [([1, 1], 8), ([5, 2], 4), ([40, 90], 8), ([16, 1], 16)])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("shape", ["up", "down", "jump", "far"])
def test_growing_scores(qlens, G, hd, shape):
    """Scores that climb along the keys, by steps and by far more than f16's range, or fall, or jump in the middle."""
    n = 700
    c = Case([n, n], qlens, 1, G, hd, 16, seed=hd)
    j = torch.arange(n, device="cuda") / n
    height = {"up": 60 * j, "down": 60 * (1 - j), "jump": 90 * (j > 0.37).float(), "far": 3000 * j}[shape]
    # keys along one direction, as steep as the cache's scale allows (4 to 16 a channel), queries with it
    for b in range(2):
        slots = torch.from_numpy(c.table[b].astype(np.int64)).cuda()[torch.arange(n, device="cuda") // 16] * 16
        slots = slots + torch.arange(n, device="cuda") % 16
        top = float(c.gk[0]) * 2688 / 1.05
        rows = (height / height.max() * top)[:, None, None].expand(n, 1, hd).to(torch.bfloat16).contiguous()
        nv.nvfp4_kv_write(rows, normal((n, 1, hd), b), slots, c.cache, c.dgk, c.dgv)
    c.q = (float(height.max()) / (top * hd ** 0.5) * (1 + 0.01 * c.q.float())).to(torch.bfloat16)
    c.check(c.run(causal=False), causal=False)
    c.check(c.run())


@pytest.mark.parametrize("qn,G", [(1, 4), (3, 8), (40, 8)])
def test_many_keys_far_below_the_largest(qn, G):
    """65535 keys of 2^-27 each beside one of 1 are a 2^-11 part of the sum, and of the result too.
    Tolerance: f16 holds the numerators, lifted by 2^4 or more, exactly up to the scores' error (2^-18, then
    half a step of the smallest f16 rounds it away); sums over 2^12 steps of 2^-22; bf16's half step 2^-8."""
    n, pages = 65536, 1024
    one = torch.ones(1, device="cuda")
    cache = nv.nvfp4_kv_cache(pages, 1, 64, 64)
    k = torch.zeros((n, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[1:, 0, 0], v[1:] = -27.0, 6.0
    nv.nvfp4_kv_write(k, v, torch.arange(n, device="cuda"), cache, one, one)
    q = torch.zeros((qn, G, 64), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    out, lse = nv.nvfp4_kv_attention(q, cache, one, one, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                                     q_offsets=torch.tensor([0, qn], dtype=torch.int32, device="cuda"), max_q_len=qn,
                                     scale=float(np.log(2.0)), causal=False, want_lse=True)
    part = (n - 1) * 2.0 ** -27
    want = 6.0 * part / (1 + part)
    assert float((out.double() - want).abs().max()) <= (2.0 ** -8 + 2.0 ** -9) * want
    assert float((lse.double() - np.log1p(part)).abs().max()) <= 2.0 ** -18


def test_extreme_queries():
    """Rows of tiny, huge and zero queries, and an infinity and a NaN in rows of their own."""
    c = Case([200, 90], [40, 1], 2, 4, 128, 16)
    q = c.q.clone()
    q[0], q[1], q[2] = 0, q[2] * 1e-30, q[3] * 1e4
    q[40] *= 1e-38
    c.q = q
    c.check(c.run(), what="finite")
    bad = q.clone()
    bad[3, 0, 5], bad[4, 7, 100], bad[40, 3, 0] = float("inf"), float("nan"), float("nan")
    want, got = c.run()[0], c.run(q=bad)[0]
    broken = torch.zeros(41, 8, dtype=torch.bool, device="cuda")
    broken[3, 0] = broken[4, 7] = broken[40, 3] = True
    assert bool(torch.isnan(got[broken]).all())
    assert torch.equal(got[~broken], want[~broken])


@pytest.mark.parametrize("qlens,G", SHAPES)
def test_strides_and_pitches(qlens, G):
    """q and out as parts of wider buffers, a cache that is one layer of a larger one, a wider page table."""
    c = Case([70, 20, 200], qlens, 3, G, 64, 32, seed=9)
    want = c.run()
    T, H = c.q.shape[:2]
    wide_q = torch.full((T, 2 * H + 1, 72), 9.0, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 1:H + 1, :64] = c.q
    wide_o = torch.full((T + 2, H + 3, 80), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide_o[1:T + 1, 2:H + 2, :64]
    table = torch.full((3, c.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = torch.from_numpy(c.table)
    store = {n: torch.full((t.shape[0], 3, *t.shape[1:]), 0xFF, dtype=torch.uint8, device="cuda")
             for n, t in c.cache.items()}
    for n, t in c.cache.items():
        store[n][:, 1] = t
    c.cache = {n: t[:, 1] for n, t in store.items()}
    got = c.run(q=wide_q[:, 1:H + 1, :64], out=out, page_table=table[:, :c.table.shape[1]])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide_o[1:T + 1, 2:H + 2, :64] = 5
    assert bool((wide_o == 5).all())


@pytest.mark.parametrize("qlens", [[1, 1], [60, 1]])
def test_caches_past_32_bits(qlens):
    """Pages a megabyte apart: byte offsets past 2^32, for writing, reading and attention."""
    P, H, page, hd = 4600, 2, 16, 128
    c = Case([100, 90], qlens, H, 8, hd, page, seed=4)
    want = c.run()
    far = np.array([P - 1 - 13 * i for i in range(c.cache["k_codes"].shape[0])])
    far[1], far[2] = 0, 4096
    near, c_table = c.cache, c.table
    big = {n: torch.zeros(P << 20, dtype=torch.uint8, device="cuda").as_strided(
        (P, H, page, t.shape[3]), (1 << 20, page * t.shape[3], t.shape[3], 1)) for n, t in near.items()}
    for n, t in near.items():
        big[n][torch.from_numpy(far).cuda()] = t
    c.cache, c.table = big, np.where(c_table >= 0, far[np.maximum(c_table, 0)], -1).astype(np.int32)
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    slots = torch.from_numpy(far * page + 5).cuda()
    k, v = normal((len(far), H, hd), 1), normal((len(far), H, hd), 2)
    nv.nvfp4_kv_write(k, v, slots, big, c.dgk, c.dgv)
    small = nv.nvfp4_kv_cache(len(far), H, page, hd)
    at = torch.arange(len(far), device="cuda") * page + 5
    nv.nvfp4_kv_write(k, v, at, small, c.dgk, c.dgv)
    for a, b in zip(nv.nvfp4_kv_read(slots, big, c.dgk, c.dgv), nv.nvfp4_kv_read(at, small, c.dgk, c.dgv)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("qlens,G,lens", [([1] * 300, 4, None), ([1] * 40, 1, None), ([300, 1, 1, 17], 8, [4000, 9, 900, 40]),
                                          ([5] * 7, 4, [3000, 10, 64, 65, 700, 6, 5])])
def test_repeatable_and_independent_of_the_workspace(qlens, G, lens):
    """The same bits from call to call, whatever the workspace holds."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(1, 400, len(qlens))] if lens is None else lens
    c = Case(lens, qlens, 4, G, 128, 16)
    call, (out, lse) = nv.prepare_kv_attention(
        c.q, c.cache, c.dgk, c.dgv, torch.from_numpy(c.table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
        q_offsets=torch.from_numpy(c.offsets).cuda(), want_lse=True)
    call()
    want = out.clone(), lse.clone()
    for fill in (0xFF, 0x7F, 0x00, 0x55):
        call.workspace[256:].fill_(fill)
        out.zero_()
        lse.zero_()
        call()
        assert nv.read_device_status(call.workspace) == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("qlens", [[1, 1, 1], [70, 1, 9]])
def test_graph_replay_with_new_lengths(qlens):
    """A captured step replays with other lengths, tables, queries and offsets, as the eager call computes them."""
    c = Case([200, 300, 150], qlens, 2, 8, 128, 16)
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    table, offsets, q = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.offsets).cuda(), c.q.clone()
    slots = torch.tensor([3, 40, -1], device="cuda")
    k, v = normal((3, 2, 128), 1), normal((3, 2, 128), 2)
    form = dict(q_offsets=offsets, max_q_len=max(qlens), want_lse=True)
    w, _ = nv.prepare_kv_write(k, v, slots, c.cache, c.dgk, c.dgv)
    call, (out, lse) = nv.prepare_kv_attention(q, c.cache, c.dgk, c.dgv, table, lens, **form)
    w()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w()
        call()
    for step in range(3):
        lens.copy_(torch.tensor([200 - 60 * step, 17 + step, 150]))
        q.copy_(normal(q.shape, 50 + step))
        k.copy_(normal(k.shape, 60 + step))
        slots[0] = 5 + step
        table[0, :2] = table[0, :2].flip(0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = nv.nvfp4_kv_attention(q, c.cache, c.dgk, c.dgv, table, lens, **form)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_other_stream_and_two_at_once():
    """Calls on streams of their own, two in flight, give what the current stream's do."""
    a, b = Case([900, 40], [1, 1], 4, 8, 128, 16, seed=1), Case([500, 80], [128, 33], 4, 8, 128, 16, seed=2)
    want = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        ga, gb = a.run(stream=s1), b.run(stream=s2)
        s1.synchronize()
        s2.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ga + gb, want[0] + want[1]))


def test_waits_run_out_and_the_next_call_recovers():
    c = Case([300], [100], 2, 4, 128, 16)
    want = c.run()
    call, (out, lse) = nv.prepare_kv_attention(
        c.q, c.cache, c.dgk, c.dgv, torch.from_numpy(c.table).cuda(), torch.tensor([300], dtype=torch.int32).cuda(),
        q_offsets=torch.from_numpy(c.offsets).cuda(), want_lse=True)
    old = nv.set_wait_timeout_ns(0)
    try:
        call()
        assert nv.read_device_status(call.workspace) == ERR_TIMEOUT
    finally:
        nv.set_wait_timeout_ns(old)
    call()
    assert nv.read_device_status(call.workspace) == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_binding_refusals():
    c = Case([40], [1], 2, 4, 64, 16)
    t, n = torch.from_numpy(c.table).cuda(), torch.tensor([40], dtype=torch.int32).cuda()
    ok = dict(q=c.q, cache=c.cache, k_global_scale=c.dgk, v_global_scale=c.dgv, page_table=t, kv_lens=n)
    nv.nvfp4_kv_attention(**ok)
    other = {**c.cache, "v_codes": c.cache["v_codes"][:, :, :8]}
    split = {**c.cache, "k_codes": c.cache["k_codes"].transpose(1, 2).contiguous().transpose(1, 2)}
    for bad, err in ((dict(q=c.q.float()), TypeError), (dict(q=c.q[:, :, :32]), ValueError), (dict(q=c.q[0]), ValueError),
                     (dict(q=torch.cat([c.q, c.q])), ValueError), (dict(kv_lens=n.long()), TypeError),
                     (dict(page_table=t.long()), TypeError), (dict(k_global_scale=c.dgk[:1]), ValueError),
                     (dict(cache=other), ValueError), (dict(cache=split), ValueError),
                     (dict(q_offsets=torch.zeros(1, dtype=torch.int32).cuda()), ValueError),
                     (dict(out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")), ValueError),
                     (dict(scale=-1.0), nv.NVFP4Error), (dict(window=3, causal=False), nv.NVFP4Error)):
        with pytest.raises(err):
            nv.nvfp4_kv_attention(**{**ok, **bad})
    k = normal((3, 2, 64), 1)
    s = torch.arange(3, device="cuda")
    for bad in ((k, k[:2], s), (k, k, s[:2]), (k, k[:, :1], s), (k, k, s.float())):
        with pytest.raises((ValueError, TypeError)):
            nv.nvfp4_kv_write(*bad, c.cache, c.dgk, c.dgv)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_read(s, c.cache, c.dgk, c.dgv, out=(k[:2].clone(), k.clone()))


def test_a_layer_step():
    """Projections by nvfp4_gemm, keys and values into the cache, attention over it, the output projection: as
    bf16 attention over the rows read back computes it."""
    hidden, Hq, Hkv, hd, page = 256, 8, 2, 64, 16
    g = torch.tensor([8 / 2688] * Hkv, device="cuda")
    wqkv = nv.nvfp4_quantize(normal(((Hq + 2 * Hkv) * hd, hidden), 1, 0.06))
    wo = nv.nvfp4_quantize(normal((hidden, Hq * hd), 2, 0.06))
    cache = nv.nvfp4_kv_cache(40, Hkv, page, hd)
    table = torch.randperm(40, generator=torch.Generator().manual_seed(0)).int().reshape(4, 10).cuda()
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    for step, new in enumerate(([50, 3, 17, 1], [1, 1, 1, 1], [1, 1, 1, 1], [4, 1, 30, 2])):
        T = sum(new)
        x = normal((T, hidden), 10 + step)
        qkv = nv.nvfp4_gemm(wqkv["codes_row"], wqkv["sf_row"], wqkv["global_scale"], (Hq + 2 * Hkv) * hd, hidden,
                            a_bf16=x).reshape(T, Hq + 2 * Hkv, hd)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        seq = torch.repeat_interleave(torch.arange(4), torch.tensor(new)).cuda()
        offs = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        pos = lens[seq].long() + torch.arange(T, device="cuda") - offs[seq].long()
        slots = table[seq, pos // page].long() * page + pos % page
        nv.nvfp4_kv_write(k, v, slots, cache, g, g)
        lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        y = nv.nvfp4_kv_attention(q, cache, g, g, table, lens, q_offsets=offs, max_q_len=max(new))
        out = nv.nvfp4_gemm(wo["codes_row"], wo["sf_row"], wo["global_scale"], hidden, Hq * hd,
                            a_bf16=y.reshape(T, Hq * hd))
        assert out.shape == (T, hidden) and bool(torch.isfinite(out).all())
        for b in range(4):
            n = int(lens[b])
            j = torch.arange(n, device="cuda")
            kk, vv = nv.nvfp4_kv_read(table[b, j // page].long() * page + j % page, cache, g, g, out_dtype=torch.float32)
            rows = q[offs[b]:offs[b + 1]].double()
            s = torch.einsum("thd,nhd->htn", rows, kk.double().repeat_interleave(Hq // Hkv, 1)) * hd ** -0.5
            hide = j[None] > (n - new[b] + torch.arange(new[b], device="cuda"))[:, None]
            p = torch.softmax(s.masked_fill(hide[None], -float("inf")), -1)
            want = torch.einsum("htn,nhd->thd", p, vv.double().repeat_interleave(Hq // Hkv, 1))
            # rounding to bf16, P's to f16: half steps of the terms' sum of magnitudes
            bound = torch.einsum("htn,nhd->thd", p, vv.double().abs().repeat_interleave(Hq // Hkv, 1))
            assert bool(((y[offs[b]:offs[b + 1]].double() - want).abs() <= 2 ** -8 * want.abs() + 2 ** -10 * bound).all())


@pytest.mark.parametrize("Hkv,G,hd", [(4, 4, 128), (5, 1, 64), (6, 3, 64), (8, 8, 128)])
def test_many_short_sequences(Hkv, G, hd):
    """Enough of them that a sequence's heads go to one warp each, longer ones among them."""
    rng = np.random.default_rng(Hkv)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(120), 500))]
    lens[7], lens[300] = 900, 1500
    c = Case(lens, [1] * 500, Hkv, G, hd, 16, seed=Hkv, offsets=False)
    c.check(c.run())
