"""The NVFP4 key-value cache on the GPU: writing, reading back, attention,
against the CPU reference in 64 bits.

Codes and scales are whole numbers and equal.  Values read back are one fp32
product of exact factors (byte * g, rounded) and the rounding to the output
type: 2^-8 (bf16) or 2^-23 (fp32, two roundings) relative.

Attention.  With S = sum_j w_j |v_j| per output channel, from the reference:
  P's rounding to f16, half a step 2^-11 of each term:         2^-11 S
  of terms below 2^-14 (subnormal f16), 2^-25 each, the sum of
  the numerators being at least sum_j exp(s_j - max):          2^-25 sum_j |v_j| / sum_j exp(s_j - max)
  the scores' error d (below), on numerators and sums:         2 d S
  fp32 accumulation, one step per 16 keys, 2^-22 each:         (n / 16 + 2) 2^-22 S
  the result's rounding to bf16, half a step:                  2^-8 |out|
d: hd / 16 accumulation steps of 2^-22 of sum_d |q_d k_jd|, q's rounding 2^-28 of
its row's maximum, three roundings of the product with the scale and exp2's 2^-22:
  d = (hd / 16 + 2) 2^-22 scale max_j sum_d |q_d k_jd| + 2^-22 (|s| + 2)
lse: d + 2^-21 (|lse| + 2)."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from oracle import kv_oracle as ko
from oracle import nvfp4_oracle as o

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def scales(H, seed):
    rng = np.random.default_rng(seed)
    return (rng.uniform(4, 16, H) / 2688).astype(np.float32)


def normal(shape, seed, spread=1.0):
    x = np.random.default_rng(seed).standard_normal(shape) * spread
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()


def np_cache(cache):
    return {n: t.cpu().numpy() for n, t in cache.items()}


# ------------------------------------------------------------ write and read --

@pytest.mark.parametrize("T,H,hd,page", [(1, 1, 64, 16), (1, 1, 128, 16), (3, 2, 128, 32), (17, 5, 64, 16),
                                         (130, 8, 128, 64), (67, 3, 64, 1024), (1000, 4, 128, 128)])
def test_write_and_read(T, H, hd, page):
    pages = (T + page - 1) // page + 2
    cache = nv.nvfp4_kv_cache(pages, H, page, hd)
    for t in cache.values():
        t.fill_(0xA5)
    rng = np.random.default_rng(T)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    dropped = np.array([-1, pages * page, -(1 << 40), 1 << 40])[:max(0, T // 3)]
    live = T - len(dropped)
    slots[live:] = dropped
    k, v = normal((T, H, hd), 1), normal((T, H, hd), 2, 3.0)
    k[0, 0, :16] = 0
    k[-1, -1, 16:32] *= 1e-6
    v[0, 0, 3] = 1e5
    gk, gv = scales(H, 3), scales(H, 4)
    ds = torch.from_numpy(slots).cuda()
    dgk, dgv = torch.from_numpy(gk).cuda(), torch.from_numpy(gv).cuda()
    assert nv.nvfp4_kv_write(k, v, ds, cache, dgk, dgv) is cache
    got = np_cache(cache)
    read = {d: nv.nvfp4_kv_read(ds, cache, dgk, dgv, out_dtype=d) for d in (torch.bfloat16, torch.float32)}
    for i, (name, x, g) in enumerate((("k", k, gk), ("v", v, gv))):
        codes, sf = ko.pack_rows(bits(x), g)
        want_c = np.full(got[name + "_codes"].shape, 0xA5, np.uint8)
        want_s = np.full(got[name + "_sf"].shape, 0xA5, np.uint8)
        s = slots[:live]
        want_c[s // page, :, s % page], want_s[s // page, :, s % page] = codes[:live], sf[:live]
        assert np.array_equal(got[name + "_codes"], want_c) and np.array_equal(got[name + "_sf"], want_s)
        exact = ko.values(codes, sf, g)[:live]
        for d, tol in ((torch.bfloat16, 2.0 ** -8 * 1.001), (torch.float32, 2.0 ** -23)):
            y = read[d][i][:live].double().cpu().numpy()
            assert np.all(np.abs(y - exact) <= tol * np.abs(exact))
    # the packed rows are the matrix quantizer's under a static scale
    q = nv.nvfp4_quantize(k[:, H - 1].contiguous(), sf_layout="linear", global_scale=dgk[H - 1:])
    s = slots[:live]
    assert np.array_equal(got["k_codes"][s // page, H - 1, s % page], q["codes_row"].cpu().numpy()[:live])
    assert np.array_equal(got["k_sf"][s // page, H - 1, s % page].reshape(-1),
                          q["sf_row"].cpu().numpy().reshape(T, hd // 16)[:live].reshape(-1))


def test_strided_rows_and_pages():
    """k and v as parts of one projection's rows, the cache as one layer of a larger one, outputs into a
    wider buffer; what lies between stays as it was."""
    T, H, hd, page, layers = 37, 3, 128, 16, 3
    qkv = normal((T, 5 * H, hd), 1)
    k, v = qkv[:, H:4 * H:1][:, :H], qkv[:, 4 * H:]
    store = {n: torch.full((9, layers, H, page, w), 0x77, dtype=torch.uint8, device="cuda")
             for n, w in (("k_codes", 64), ("k_sf", 8), ("v_codes", 64), ("v_sf", 8))}
    cache = {n: t[:, 1] for n, t in store.items()}
    g = torch.from_numpy(scales(H, 5)).cuda()
    slots = torch.randperm(9 * page, generator=torch.Generator().manual_seed(1))[:T].cuda()
    nv.nvfp4_kv_write(k, v, slots, cache, g, g)
    plain = nv.nvfp4_kv_cache(9, H, page, hd)
    for t in plain.values():
        t.fill_(0x77)
    nv.nvfp4_kv_write(k.contiguous(), v.contiguous(), slots, plain, g, g)
    for n in cache:
        assert torch.equal(cache[n], plain[n])
        assert bool((store[n][:, 0] == 0x77).all()) and bool((store[n][:, 2] == 0x77).all())
    wide = torch.full((T, 2 * H + 1, hd), 5.0, dtype=torch.bfloat16, device="cuda")
    out = (wide[:, :H], wide[:, H:2 * H])
    some = slots.clone()
    some[5] = -1
    nv.nvfp4_kv_read(some, cache, g, g, out=out)
    ref = nv.nvfp4_kv_read(slots, plain, g, g)
    keep = torch.arange(T, device="cuda") != 5
    for a, b in zip(out, ref):
        assert torch.equal(a[keep], b[keep])
    assert bool((wide[5] == 5).all()) and bool((wide[:, 2 * H] == 5).all())


def test_special_values():
    """Infinities saturate, a NaN makes its own block NaN and no other."""
    g = torch.full((1,), 4 / 2688, device="cuda")
    k = normal((2, 1, 64), 1)
    k[0, 0, 0], k[0, 0, 17], k[1, 0, 40] = float("inf"), -float("inf"), float("nan")
    cache = nv.nvfp4_kv_cache(1, 1, 16, 64)
    slots = torch.tensor([3, 9], device="cuda")
    nv.nvfp4_kv_write(k, k, slots, cache, g, g)
    r = nv.nvfp4_kv_read(slots, cache, g, g, out_dtype=torch.float32)[0]
    assert abs(float(r[0, 0, 0]) - 4.0) < 1e-5 and abs(float(r[0, 0, 17]) + 4.0) < 1e-5
    bad = torch.isnan(r[1, 0])
    assert bool(bad[32:48].all()) and int(bad.sum()) == 16 and not bool(torch.isnan(r[0]).any())


# ----------------------------------------------------------------- attention --

class Case:
    """A cache filled by nvfp4_kv_write and a batch over it."""

    def __init__(self, lens, qlens, Hkv, G, hd, page, seed=0, spread=1.0, offsets=True):
        self.lens, self.qlens, self.Hkv, self.G, self.hd, self.page = lens, qlens, Hkv, G, hd, page
        rng = np.random.default_rng(seed)
        need = [(n + page - 1) // page for n in lens]
        pages = sum(need) + 1
        order = rng.permutation(pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.gk, self.gv = scales(Hkv, seed + 1), scales(Hkv, seed + 2)
        self.cache = nv.nvfp4_kv_cache(pages, Hkv, page, hd)
        k, v = normal((pages * page, Hkv, hd), seed + 3), normal((pages * page, Hkv, hd), seed + 4)
        self.dgk, self.dgv = torch.from_numpy(self.gk).cuda(), torch.from_numpy(self.gv).cuda()
        nv.nvfp4_kv_write(k, v, torch.arange(pages * page, device="cuda"), self.cache, self.dgk, self.dgv)
        self.offsets = np.concatenate([[0], np.cumsum(qlens)]).astype(np.int32)
        self.q = normal((int(self.offsets[-1]), Hkv * G, hd), seed + 5, spread)
        self.use_offsets = offsets

    def run(self, **form):
        form.setdefault("want_lse", True)
        if self.use_offsets:
            form.setdefault("q_offsets", torch.from_numpy(self.offsets).cuda())
        form.setdefault("kv_lens", torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        form.setdefault("page_table", torch.from_numpy(self.table).cuda())
        q = form.pop("q", self.q)
        return nv.nvfp4_kv_attention(q, self.cache, self.dgk, self.dgv, **form)

    def check(self, got, causal=True, window=0, scale=None, lens=None, table=None, what=""):
        out, lse = got
        c = np_cache(self.cache)
        scale = self.hd ** -0.5 if scale is None else scale
        lens = self.lens if lens is None else lens
        table = self.table if table is None else table
        for b, (n, nq) in enumerate(zip(lens, self.qlens)):
            if nq == 0:
                continue
            r0 = self.offsets[b]
            q = self.q[r0:r0 + nq].double().cpu().numpy()
            k, ok = ko.gather(c["k_codes"], c["k_sf"], self.gk, table[b], n, self.page)
            v, _ = ko.gather(c["v_codes"], c["v_sf"], self.gv, table[b], n, self.page)
            w_out, w_lse, S, V, qk = ko.attention(q, k, v, ok, n - nq + np.arange(nq), scale, causal, window)
            y = out[r0:r0 + nq].double().cpu().numpy()
            z = lse[r0:r0 + nq].double().cpu().numpy()
            empty, undefined = np.isinf(w_lse), np.isnan(w_out)
            assert np.array_equal(np.isneginf(z), empty), what
            assert np.all(y[empty] == 0)
            assert np.array_equal(np.isnan(y), undefined), what
            assert np.array_equal(np.isnan(z), np.isnan(w_lse)), what
            empty, y, w_out = empty | np.isnan(w_lse), np.where(undefined, 0, y), np.where(undefined, 0, w_out)
            s_max = np.where(empty, 0, np.abs(w_lse) + np.log(max(n, 2)))
            d = (self.hd / 16 + 2) * 2.0 ** -22 * scale * qk + 2.0 ** -22 * (s_max + 2)
            s_max, d = np.where(empty, 0, s_max), np.where(empty, 0, d)
            assert np.all(np.abs(z[~empty] - w_lse[~empty]) <= (d + 2.0 ** -21 * (np.abs(w_lse) + 2))[~empty]), what
            tol = ((2.0 ** -11 + 2 * d[..., None] + (n / 16 + 2) * 2.0 ** -22) * S + 2.0 ** -25 * V
                   + 2.0 ** -8 * np.abs(w_out))
            bad = ~(np.abs(y - w_out) <= tol * 1.0001 + 1e-30) & ~undefined
            assert not bad.any(), (what, b, np.argwhere(bad)[:4], y[bad][:4], w_out[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 200, 1021])
def test_decode_lengths(n, hd):
    c = Case([n], [1], 2, 4, hd, 16, seed=n, offsets=False)
    c.check(c.run())


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("hd", [64, 128])
def test_decode_groups(G, hd):
    c = Case([77, 1, 300], [1, 1, 1], 2, G, hd, 32, seed=G, offsets=False)
    c.check(c.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
def test_decode_ragged_batch(page, Hkv):
    rng = np.random.default_rng(page + Hkv)
    lens = [int(x) for x in rng.integers(1, 700, 33)]
    c = Case(lens, [1] * 33, Hkv, 4, 128, page, seed=Hkv, offsets=False)
    c.check(c.run())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("G,qlens", [(1, [5, 1, 8]), (4, [5, 5, 1]), (8, [2, 1, 0, 3]), (3, [7, 1, 11]),
                                     (16, [1, 3, 2]), (5, [40, 1, 17]), (8, [130, 0, 33]), (12, [1, 64, 200]),
                                     (1, [257, 1, 128])])
def test_several_new_tokens(G, qlens, causal):
    lens = [max(1, q + 37 * i) for i, q in enumerate(qlens)]
    c = Case(lens, qlens, 2, G, 128, 16, seed=G)
    c.check(c.run(causal=causal), causal)
    c.check(c.run(causal=causal, max_q_len=max(qlens)), causal)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000])
def test_windows(window, hd):
    c = Case([300, 40, 129], [1, 7, 60], 2, 4, hd, 16, seed=window)
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("hd", [64, 128])
def test_whole_prompts(hd):
    lens = [1, 200, 129, 3]
    c = Case(lens, lens, 2, 4, hd, 32, seed=hd)
    c.check(c.run())
    c.check(c.run(causal=False), causal=False)
