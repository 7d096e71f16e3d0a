"""The MXFP4 entry points on the GPU against the CPU reference in 64 bits.

Quantize and dequantize are exact operations up to the one rounding that the
format defines: bit-equal.  Products: codes times powers of two are exact, so
only the fp32 accumulation rounds: the tolerance of the other products of the
library, 2e-5 of the sum of absolute terms (fp32 out), one bf16 ulp more for
bf16 out.  The down-projection stores its expert outputs in bf16 before the
weighted sum, as nvfp4_moe_down_combine does, and has its tolerance."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv
from helpers import assert_bits_equal, assert_gemm_close, dev_bf16, host_bits, u8
from oracle import mxfp4_oracle as mo
from oracle import nvfp4_oracle as o
from synth import f32_to_bf16_bits, make_case

pytestmark = pytest.mark.gpu


def bits(rng, *shape, scale=1.0):
    return f32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


def packed(b):
    """bf16 bits -> (codes, linear sf, device codes, device swizzled sf)."""
    codes, byte = mo.quantize(b)
    return codes, byte, torch.from_numpy(codes).cuda(), torch.from_numpy(mo.sf_swizzle(byte)).cuda()


def special_rows(rng, cols):
    """Rows of the values where a block scale or a code can go wrong."""
    x = rng.standard_normal((12, cols)).astype(np.float32)
    x[0] = 0.0
    x[1] = -0.0
    x[2] *= 1e-38                               # bf16 subnormals among them
    x[3] *= 2.0 ** 127 / np.abs(x[3]).max()     # the largest exponent
    x[4] = np.resize(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], dtype=np.float32), cols)   # ties, X = 1
    x[5] = -x[4]
    x[6] = np.resize(np.array([7.984375, 7.0, 6.0, 5.015625, 4.984375, 0.24902344], dtype=np.float32), cols)
    x[7] = 2.0 ** -133                          # the smallest bf16
    x[8, 3] = np.inf
    x[9, cols - 1] = np.nan
    x[10, ::2] = 0.0
    x[11, 32:64] = 0.0
    return f32_to_bf16_bits(x)


@pytest.mark.parametrize("layout", ["linear", "swizzled"])
@pytest.mark.parametrize("R,Cc", [(1, 32), (1, 2080), (12, 128), (37, 96), (128, 4096), (130, 2048), (300, 6144),
                                  (77, 8224)])
def test_quantize_bits(R, Cc, layout):
    rng = np.random.default_rng(R + Cc)
    b = bits(rng, R, Cc)
    if R >= 12 and Cc >= 64:
        b[:12] = special_rows(rng, Cc)
    got = nv.nvfp4_mxfp4_quantize(dev_bf16(b), sf_layout=layout)
    codes, byte = mo.quantize(b)
    assert_bits_equal(u8(got["sf"]), byte if layout == "linear" else mo.sf_swizzle(byte), "scales")
    assert_bits_equal(u8(got["codes"]), codes, "codes")


def test_quantize_every_bf16_exponent_and_mantissa():
    """Every positive finite bf16 value once as a block's maximum, with its
    neighbours' fractions in the block."""
    top = np.arange(0, 0x7F80, dtype=np.uint16)
    frac = np.arange(32, dtype=np.float64) / 31.0
    f = o.bf16_to_f32(top).astype(np.float64)[:, None] * frac
    b = f32_to_bf16_bits(f.astype(np.float32)).reshape(-1, 32 * 8)
    got = nv.nvfp4_mxfp4_quantize(dev_bf16(b), sf_layout="linear")
    codes, byte = mo.quantize(b)
    assert_bits_equal(u8(got["sf"]), byte, "scales")
    assert_bits_equal(u8(got["codes"]), codes, "codes")


def test_quantize_strided_batch():
    rng = np.random.default_rng(5)
    big = dev_bf16(bits(rng, 3, 50, 200))
    for sl, off in ((slice(8, 136), 8), (slice(0, 160), 0), (slice(16, 176), 16)):
        x = big[:, 3:45, sl]
        got = nv.nvfp4_mxfp4_quantize(x)
        for i in range(3):
            codes, byte = mo.quantize(host_bits(x[i]))
            assert_bits_equal(u8(got["codes"][i]), codes, "codes")
            assert_bits_equal(u8(got["sf"][i]), mo.sf_swizzle(byte), "scales")


def random_packed(rng, R, Cc, lo=0, hi=256):
    codes = rng.integers(0, 256, (R, Cc // 2), dtype=np.uint8)
    byte = rng.integers(lo, hi, (R, Cc // 32)).astype(np.uint8)
    return codes, byte


@pytest.mark.parametrize("layout", ["linear", "swizzled"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,Cc", [(1, 32), (5, 96), (128, 256), (129, 160), (200, 2048)])
def test_dequantize_every_scale(R, Cc, transpose, layout):
    """Random codes under random scale bytes, 0 and 255 among them: the exact
    value rounded to bf16 (a rounding only where 6 * 2^127 overflows)."""
    rng = np.random.default_rng(R * Cc)
    codes, byte = random_packed(rng, R, Cc)
    byte[0, 0] = 255
    if Cc > 32:
        byte[0, 1] = 0
    sf = byte if layout == "linear" else mo.sf_swizzle(byte)
    got = nv.nvfp4_mxfp4_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(sf).cuda(), transpose, layout)
    want = mo.dequantize(codes, byte)
    want = want.T if transpose else want
    with np.errstate(over="ignore"):
        ref = torch.from_numpy(np.ascontiguousarray(want)).to(torch.float32).to(torch.bfloat16)
    g = got.cpu().contiguous()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan)
    assert torch.equal(g.view(torch.int16)[~nan], ref.contiguous().view(torch.int16)[~nan])


def test_dequantize_into_strided_rows():
    rng = np.random.default_rng(8)
    codes, byte = random_packed(rng, 40, 64, 100, 140)
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(byte).cuda()
    want = torch.from_numpy(mo.dequantize(codes, byte)).to(torch.bfloat16)
    for transpose, shape in ((False, (40, 64)), (True, (64, 40))):
        out = torch.full((shape[0], shape[1] + 24), 3.0, dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_mxfp4_dequantize(c, s, transpose, "linear", out=out[:, 8:8 + shape[1]])
        assert torch.equal(out[:, 8:8 + shape[1]].cpu(), want.t() if transpose else want)
        assert bool((out[:, :8] == 3.0).all()) and bool((out[:, 8 + shape[1]:] == 3.0).all())


# ----------------------------------------------------------------- product --

def product(a, b):
    return a @ b.T, np.abs(a) @ np.abs(b).T


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 136, 96), (7, 256, 512), (32, 1000, 2080), (1, 512, 16384),
                                   (33, 128, 64), (100, 264, 352), (128, 256, 8192), (255, 384, 1056),
                                   (256, 256, 256), (257, 136, 96), (300, 520, 2048), (1024, 768, 800)])
def test_gemm_quantized_in_the_call_and_packed(M, N, K, out_dtype):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    x, w = bits(rng, M, K), bits(rng, N, K, scale=0.02)
    ac, ab, ac_d, asf_d = packed(x)
    wc, wb, wc_d, wsf_d = packed(w)
    y, S = product(mo.dequantize(ac, ab), mo.dequantize(wc, wb))
    for form in (dict(a_bf16=dev_bf16(x)), dict(a_codes=ac_d, a_sf=asf_d)):
        call, got = nv.prepare_mxfp4_gemm(wc_d, wsf_d, N, K, out_dtype=out_dtype, **form)
        call()
        assert nv.read_device_status(call.workspace) == 0
        assert_gemm_close(got, y, S, what=f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 20488, 352), (5, 20480, 544), (8, 19464, 2080), (3, 256, 8448), (8, 128, 3104),
                                   (2, 392, 14336)])
def test_gemm_few_rows_packed_by_the_kernel(M, N, K):
    """Rows that the operand-swapped kernel packs itself: more weight tiles than
    SMs (the packed rows serve every unit of a CTA), long K ranges, K ranges whose
    last tile is partly outside K; strided rows."""
    rng = np.random.default_rng(M + N + K)
    big = dev_bf16(bits(rng, M, K + 32))
    x = big[:, 16:16 + K]
    wc, wb, wc_d, wsf_d = packed(bits(rng, N, K, scale=0.02))
    y, S = product(mo.dequantize(*mo.quantize(host_bits(x))), mo.dequantize(wc, wb))
    call, got = nv.prepare_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=x, out_dtype=torch.float32)
    for _ in range(3):
        call()
    assert nv.read_device_status(call.workspace) == 0
    assert_gemm_close(got, y, S)


def test_gemm_scales_of_every_size():
    """Scales spread over 2^-40 .. 2^40 between blocks: each block's scale, not
    a neighbour's, multiplies its codes (K steps of both halves of an atom)."""
    rng = np.random.default_rng(2)
    for M, N, K in [(16, 256, 512), (64, 128, 416), (512, 256, 768)]:
        ac, ab = random_packed(rng, M, K, 87, 167)
        wc, wb = random_packed(rng, N, K, 87, 167)
        y, S = product(mo.dequantize(ac, ab), mo.dequantize(wc, wb))
        got = nv.nvfp4_mxfp4_gemm(torch.from_numpy(wc).cuda(), torch.from_numpy(mo.sf_swizzle(wb)).cuda(), N, K,
                                  a_codes=torch.from_numpy(ac).cuda(),
                                  a_sf=torch.from_numpy(mo.sf_swizzle(ab)).cuda(), out_dtype=torch.float32)
        assert_gemm_close(got, y, S)


@pytest.mark.parametrize("M", [4, 64, 300])
def test_gemm_one_block_at_a_time(M):
    """One non-zero block of K per run: its products alone reach the result."""
    N, K = 256, 512
    for blk in range(K // 32):
        x = np.zeros((M, K), dtype=np.float32)
        w = np.zeros((N, K), dtype=np.float32)
        x[:, blk * 32] = 1.0 + np.arange(M) % 3
        w[:, blk * 32] = 2.0 ** (np.arange(N) % 5)
        got = nv.nvfp4_mxfp4_gemm(*packed(f32_to_bf16_bits(w))[2:], N, K, a_bf16=dev_bf16(f32_to_bf16_bits(x)),
                                  out_dtype=torch.float32)
        assert np.array_equal(got.cpu().numpy(), np.outer(x[:, blk * 32], w[:, blk * 32])), blk


@pytest.mark.parametrize("M", [8, 96, 512])
def test_gemm_non_finite_rows_stay_in_their_rows(M):
    rng = np.random.default_rng(M)
    N, K = 256, 384
    x = (rng.standard_normal((M, K))).astype(np.float32)
    x[1, 5], x[3, 383] = np.inf, np.nan
    xb, wb_ = f32_to_bf16_bits(x), bits(rng, N, K)
    wc, wb, wc_d, wsf_d = packed(wb_)
    got = nv.nvfp4_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=dev_bf16(xb), out_dtype=torch.float32).cpu().numpy()
    assert np.isnan(got[[1, 3]]).all()
    rest = np.delete(np.arange(M), [1, 3])
    a = mo.dequantize(*mo.quantize(xb))[rest]
    y, S = product(a, mo.dequantize(wc, wb))
    assert np.all(np.abs(got[rest] - y) <= 2e-5 * S)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,pad,shift", [(256, 1000, 24, 0), (300, 1004, 4, 0), (511, 1002, 14, 0), (300, 416, 8, 8),
                                           (700, 2088, 3, 0), (257, 512, 8, 1), (290, 33, 7, 0)])
def test_gemm_writes_its_columns_and_rows_only(M, N, pad, shift, out_dtype):
    """Outputs inside a larger buffer, rows that end off a 16-byte or 32-column
    boundary: nothing outside [M, N] is written.  A pitch or base that is no
    multiple of 16 bytes is refused."""
    rng = np.random.default_rng(M + N)
    K = 160
    xb = bits(rng, M, K)
    wc, wb, wc_d, wsf_d = packed(bits(rng, N, K))
    buf = torch.full((M + 40, N + pad + shift), 5.0, device="cuda", dtype=out_dtype)
    if (buf.stride(0) * buf.element_size()) % 16 or (shift * buf.element_size()) % 16:
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=dev_bf16(xb), out=buf[:M, shift:shift + N])
        assert bool((buf == 5.0).all())
        return
    nv.nvfp4_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=dev_bf16(xb), out=buf[:M, shift:shift + N])
    y, S = product(mo.dequantize(*mo.quantize(xb)), mo.dequantize(wc, wb))
    assert_gemm_close(buf[:M, shift:shift + N], y, S)
    buf[:M, shift:shift + N] = 5.0
    assert bool((buf == 5.0).all())


def test_gemm_strided_x_padded_out_and_full_size_sampled():
    rng = np.random.default_rng(4)
    M, N, K = 200, 136, 512
    big = dev_bf16(bits(rng, M, K + 64))
    x = big[:, 32:32 + K]
    wc, wb, wc_d, wsf_d = packed(bits(rng, N, K))
    out = torch.full((M, N + 16), 5.0, device="cuda")
    nv.nvfp4_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=x, out=out[:, :N])
    y, S = product(mo.dequantize(*mo.quantize(host_bits(x))), mo.dequantize(wc, wb))
    assert_gemm_close(out[:, :N], y, S)
    assert bool((out[:, N:] == 5.0).all())
    # the prefill shape of the benchmark, sampled rows
    M, N, K = 8192, 2048, 6144
    xt = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    wt = torch.randn(N, K, device="cuda", dtype=torch.bfloat16) * 0.02
    w = nv.nvfp4_mxfp4_quantize(wt)
    got = nv.nvfp4_mxfp4_gemm(w["codes"], w["sf"], N, K, a_bf16=xt, out_dtype=torch.float32)
    rows = np.array([0, 1, 127, 128, 255, 256, 4095, 5000, 8064, 8191])
    wv = mo.dequantize(*mo.quantize(host_bits(wt)))
    y, S = product(mo.dequantize(*mo.quantize(host_bits(xt[rows.tolist()]))), wv)
    assert_gemm_close(got[rows.tolist()], y, S)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (5, 72, 96), (130, 264, 320), (255, 128, 64), (256, 512, 512),
                                   (700, 1032, 288)])
def test_dgrad(M, N, K, out_dtype):
    rng = np.random.default_rng(M + N + K)
    dy = bits(rng, M, N, scale=0.01)
    wc, wb, wc_d, wsf_d = packed(bits(rng, N, K, scale=0.02))
    call, got = nv.prepare_mxfp4_dgrad(dev_bf16(dy), wc_d, wsf_d, N, K, out_dtype=out_dtype)
    call()
    assert nv.read_device_status(call.workspace) == 0
    y, S = product(o.bf16_to_f32(dy).astype(np.float64), mo.dequantize(wc, wb).T)
    assert_gemm_close(got, y, S, what="dgrad")


def test_dgrad_ragged_contraction_and_difference_of_the_forward():
    """N that is no multiple of 8 (dY's rows padded), and the gradient as the
    change of sum(dY * Y): the product is linear in X's decoded values."""
    rng = np.random.default_rng(12)
    M, N, K = 40, 77, 64
    dy = dev_bf16(bits(rng, M, 80, scale=0.01))[:, :N]
    wc, wb, wc_d, wsf_d = packed(bits(rng, N, K, scale=0.02))
    got = nv.nvfp4_mxfp4_dgrad(dy, wc_d, wsf_d, N, K, out_dtype=torch.float32)
    w = mo.dequantize(wc, wb)
    dyh = o.bf16_to_f32(host_bits(dy)).astype(np.float64)
    y, S = product(dyh, w.T)
    assert_gemm_close(got, y, S, what="ragged dgrad")
    x = mo.dequantize(*mo.quantize(bits(rng, M, K)))
    step = 0.5
    for m, k in [(0, 0), (3, 63), (39, 31)]:
        up = x.copy()
        up[m, k] += step
        diff = ((dyh * (up @ w.T)).sum() - (dyh * (x @ w.T)).sum()) / step
        assert abs(diff - float(got[m, k])) <= 2e-5 * S[m, k] + 1e-9


# ----------------------------------------------------------------- experts --

def grouped_reference(xv, ids, wl):
    """fp64 (rows in grouped order, error scale, perm, offsets)."""
    T, k = ids.shape
    E, N = len(wl), wl[0].shape[0]
    flat = ids.reshape(-1)
    perm = np.concatenate([np.flatnonzero(flat == e) for e in range(E)]).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[(flat >= 0) & (flat < E)], minlength=E))])
    d, S = np.zeros((len(perm), N)), np.zeros((len(perm), N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        d[r], S[r] = product(xv[perm[r] // k], wl[e])
    return d, S, perm, offsets


def expert_case(T, E, k, N, K, seed=0):
    rng = np.random.default_rng(seed + T)
    w = bits(rng, E * N, K, scale=0.02)
    wc, wb, wc_d, wsf_d = packed(w)
    wl = list(mo.dequantize(wc, wb).reshape(E, N, K))
    ids = np.argsort(-(rng.standard_normal((T, E)) - 1.1 * np.log(1 + rng.permutation(E))), axis=1)[:, :k]
    return rng, wl, wc_d, wsf_d, ids.astype(np.int32)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 4, 2, 256, 64), (7, 5, 3, 256, 352), (96, 16, 4, 512, 256),
                                       (300, 8, 2, 256, 544), (513, 31, 8, 256, 128)])
def test_grouped_forms(T, E, k, N, K, out_dtype):
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K)
    x = bits(rng, T, K)
    ac, ab = mo.quantize(x)
    d, S, perm, offsets = grouped_reference(mo.dequantize(ac, ab), ids, wl)
    ids_d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    call, (got, p, offs) = nv.prepare_mxfp4_grouped(ids_d, dev_bf16(x), wc_d, wsf_d, N, K, E, out_dtype=out_dtype)
    call()
    assert nv.read_device_status(call.workspace) == 0
    assert np.array_equal(p.cpu().numpy(), perm) and np.array_equal(offs.cpu().numpy(), offsets)
    assert_gemm_close(got, d, S, what="grouped")
    xp = (torch.from_numpy(ac).cuda(), torch.from_numpy(ab).cuda())
    for form in (dict(x_bf16=None, x_packed=xp, expert_ids=ids_d),
                 dict(x_bf16=dev_bf16(x), expert_ids=None, routing=(offs, p), top_k=k),
                 dict(x_bf16=None, x_packed=xp, expert_ids=None, routing=(offs, p), top_k=k)):
        form = dict(form)
        r = nv.nvfp4_mxfp4_grouped_gemm(form.pop("expert_ids"), form.pop("x_bf16"), wc_d, wsf_d, N, K, E,
                                        out_dtype=out_dtype, **form)
        assert torch.equal(r[0], got)


@pytest.mark.parametrize("T,E,k,N,K,heavy", [(93, 64, 2, 2048, 736, 0), (150, 64, 2, 512, 352, 150),
                                             (500, 40, 1, 256, 1056, 300), (32, 32, 8, 1024, 2048, 0)])
def test_grouped_few_rows_per_expert(T, E, k, N, K, heavy):
    """Few rows per expert on average (the operand-swapped kernel), with more
    units than the GPU's CTAs, K that wraps its stages, and one expert that takes
    `heavy` of the tokens: several groups of 32 rows and more than one m-tile."""
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=21)
    for t in range(heavy):
        if 3 not in ids[t]:
            ids[t, t % k] = 3
    x = bits(rng, T, K)
    d, S, perm, offsets = grouped_reference(mo.dequantize(*mo.quantize(x)), ids, wl)
    ids_d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    call, (got, p, offs) = nv.prepare_mxfp4_grouped(ids_d, dev_bf16(x), wc_d, wsf_d, N, K, E,
                                                    out_dtype=torch.float32)
    for _ in range(3):
        call()
    assert nv.read_device_status(call.workspace) == 0
    assert np.array_equal(p.cpu().numpy(), perm) and np.array_equal(offs.cpu().numpy(), offsets)
    assert_gemm_close(got, d, S)
    # the down-projection's form: rows already grouped, weighted back to the tokens
    h = bits(rng, T * k, K)
    hv = mo.dequantize(*mo.quantize(h))
    dd, SS = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        dd[r], SS[r] = product(hv[r], wl[e])
    w = rng.random((T, k)).astype(np.float32)
    y = nv.nvfp4_mxfp4_moe_down_combine(dev_bf16(h), p, offs, torch.from_numpy(w).cuda(), wc_d, wsf_d, N, K, E)
    want = o.moe_combine(dd, perm, w, k)
    tol = o.moe_combine(2.0 ** -8 * np.abs(dd) + 2e-5 * SS, perm, np.abs(w), k) + o.bf16_ulp(np.abs(want) + 1e-30)
    assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("T,E,k,N,K,heavy,empty", [(300, 4, 2, 256, 96, 0, 1), (513, 5, 2, 512, 1312, 513, 0),
                                                   (1100, 9, 4, 2048, 160, 0, 8), (700, 40, 3, 768, 416, 690, 5)])
def test_grouped_many_rows_per_expert(T, E, k, N, K, heavy, empty):
    """Tiles of 256 rows: experts that end in a tile's first half, in its second or
    on its edge, one row past it, an expert without rows (its choices dropped),
    and more units than CTA pairs, the last ones as halves."""
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=33)
    for t in range(heavy):
        if 3 not in ids[t]:
            ids[t, t % k] = 3
    ids[ids == empty] = -1
    x = bits(rng, T, K)
    d, S, perm, offsets = grouped_reference(mo.dequantize(*mo.quantize(x)), ids, wl)
    n = len(perm)
    ids_d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
    for out_dtype in (torch.float32, torch.bfloat16):
        call, (got, p, offs) = nv.prepare_mxfp4_grouped(ids_d, dev_bf16(x), wc_d, wsf_d, N, K, E, out_dtype=out_dtype)
        got.fill_(-7.0)
        call()
        assert nv.read_device_status(call.workspace) == 0
        assert np.array_equal(p[:n].cpu().numpy(), perm) and np.array_equal(offs.cpu().numpy(), offsets)
        assert_gemm_close(got[:n], d, S)
        assert torch.all(got[n:] == -7.0)
    h = bits(rng, T * k, K)
    hv = mo.dequantize(*mo.quantize(h))
    dd, SS = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        dd[r], SS[r] = product(hv[r], wl[e])
    w = rng.random((T, k)).astype(np.float32)
    y = nv.nvfp4_mxfp4_moe_down_combine(dev_bf16(h), p, offs, torch.from_numpy(w).cuda(), wc_d, wsf_d, N, K, E)
    want, tol = np.zeros((T, N)), np.zeros((T, N))
    for i, pair in enumerate(perm):
        want[pair // k] += w[pair // k, pair % k] * dd[i]
        tol[pair // k] += w[pair // k, pair % k] * (2.0 ** -8 * np.abs(dd[i]) + 2e-5 * SS[i])
    tol += o.bf16_ulp(np.abs(want) + 1e-30)
    assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol)


def test_grouped_drops_missing_choices():
    """ids of -1 (the router's missing choices) take no row."""
    T, E, k, N, K = 40, 6, 4, 256, 96
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=3)
    ids[::3, 2:] = -1
    ids[5] = -1
    x = bits(rng, T, K)
    d, S, perm, offsets = grouped_reference(mo.dequantize(*mo.quantize(x)), ids, wl)
    got, p, offs = nv.nvfp4_mxfp4_grouped_gemm(torch.from_numpy(np.ascontiguousarray(ids)).cuda(), dev_bf16(x), wc_d,
                                               wsf_d, N, K, E, out_dtype=torch.float32)
    n = len(perm)
    assert np.array_equal(offs.cpu().numpy(), offsets) and np.array_equal(p[:n].cpu().numpy(), perm)
    assert_gemm_close(got[:n], d, S)


@pytest.mark.parametrize("T,E,k", [(12, 8, 4), (300, 8, 4), (3000, 16, 8)])
def test_missing_choices_through_router_and_both_products(T, E, k):
    """Tokens whose masked logits leave fewer than k experts, or none: their
    slots take no grouped row, the rest is as if they were not there, and a
    token without experts gets zeros (small and large routing paths)."""
    N, K = 256, 64
    rng, wl, wc_d, wsf_d, _ = expert_case(T, E, k, N, K, seed=33)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[::3, 2:] = -np.inf
    logits[1::7] = -np.inf
    r = nv.nvfp4_route_topk(torch.from_numpy(logits).cuda(), k, score="softmax")
    ids = r["expert_ids"].cpu().numpy()
    assert (ids[1::7] == -1).all() and (ids[0, 2:] == -1).all()
    x = bits(rng, T, K)
    d, S, perm, offsets = grouped_reference(mo.dequantize(*mo.quantize(x)), ids, wl)
    got, p, offs = nv.nvfp4_mxfp4_grouped_gemm(r["expert_ids"], dev_bf16(x), wc_d, wsf_d, N, K, E,
                                               out_dtype=torch.float32)
    n = len(perm)
    assert np.array_equal(offs.cpu().numpy(), offsets) and np.array_equal(p[:n].cpu().numpy(), perm)
    assert bool((p[n:] == -1).all())
    assert_gemm_close(got[:n], d, S)
    h = bits(rng, T * k, K)
    hv = mo.dequantize(*mo.quantize(h))
    dd, SS = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        s = slice(offsets[e], offsets[e + 1])
        dd[s], SS[s] = product(hv[s], wl[e])
    w = r["weights"].cpu().numpy().astype(np.float64)
    want, tol = np.zeros((T, N)), np.zeros((T, N))
    for i in range(n):
        t, j = divmod(int(perm[i]), k)
        want[t] += w[t, j] * dd[i]
        tol[t] += abs(w[t, j]) * (2.0 ** -8 * np.abs(dd[i]) + 2e-5 * SS[i])
    y = nv.nvfp4_mxfp4_moe_down_combine(dev_bf16(h), p, offs, r["weights"], wc_d, wsf_d, N, K, E)
    y = y.float().cpu().numpy()
    assert np.all(np.abs(y - want) <= tol + o.bf16_ulp(np.abs(want) + 1e-30))
    assert (y[1::7] == 0).all()


@pytest.mark.parametrize("T,E,k,N,K", [(1, 4, 2, 256, 64), (32, 32, 8, 512, 352), (200, 40, 4, 256, 256)])
def test_moe_down(T, E, k, N, K):
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=9)
    h = bits(rng, T * k, K)                       # grouped order
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    hv = mo.dequantize(*mo.quantize(h))
    d, S = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        d[r], S[r] = product(hv[r], wl[e])
    w = rng.random((T, k)).astype(np.float32)
    call, y = nv.prepare_mxfp4_moe_down(dev_bf16(h), torch.from_numpy(perm.astype(np.int32)).cuda(),
                                        torch.from_numpy(offsets.astype(np.int32)).cuda(),
                                        torch.from_numpy(w).cuda(), wc_d, wsf_d, N, K, E)
    call()
    assert nv.read_device_status(call.workspace) == 0
    want = o.moe_combine(d, perm, w, k)
    tol = o.moe_combine(2.0 ** -8 * np.abs(d) + 2e-5 * S, perm, np.abs(w), k) + o.bf16_ulp(np.abs(want) + 1e-30)
    assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol)


# ------------------------------------------------------------ calls, limits --

def test_graph_replay_and_another_stream():
    rng = np.random.default_rng(1)
    for M, N, K in [(1, 768, 8192), (8, 256, 512), (384, 512, 1024)]:
        wc, wb, wc_d, wsf_d = packed(bits(rng, N, K))
        x = dev_bf16(bits(rng, M, K))
        call, y = nv.prepare_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=x)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        x.copy_(dev_bf16(bits(rng, M, K)))
        g.replay()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        want = nv.nvfp4_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=x.clone(), stream=s)
        s.synchronize()
        assert torch.equal(y, want)


def test_expired_wait_is_reported_and_the_next_call_recovers():
    rng = np.random.default_rng(6)
    for M, N, K in [(8, 256, 512), (64, 256, 512), (512, 512, 512)]:
        wc, wb, wc_d, wsf_d = packed(bits(rng, N, K))
        x = dev_bf16(bits(rng, M, K))
        call, y = nv.prepare_mxfp4_gemm(wc_d, wsf_d, N, K, a_bf16=x)
        call()
        want = y.clone()
        old = nv.set_wait_timeout_ns(0)
        try:
            call()
            st = nv.read_device_status(call.workspace)
        finally:
            nv.set_wait_timeout_ns(old)
        assert st == 6
        call()
        assert nv.read_device_status(call.workspace) == 0 and torch.equal(y, want)


def test_refusals():
    x = torch.randn(16, 64, device="cuda", dtype=torch.bfloat16)
    w = nv.nvfp4_mxfp4_quantize(torch.randn(256, 64, device="cuda", dtype=torch.bfloat16))
    c, sf = w["codes"], w["sf"]
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_mxfp4_quantize(x[:, :48])                       # 48 columns
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_mxfp4_quantize(x.reshape(-1)[1:33].reshape(1, 32))   # misaligned
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_mxfp4_quantize(x[:0])
    with pytest.raises(TypeError):
        nv.nvfp4_mxfp4_quantize(x.float())
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_gemm(c, sf, 256, 64)                      # no A
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_gemm(c, sf, 512, 64, a_bf16=x)            # fewer codes than N asks for
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_gemm(c, sf[:100], 256, 64, a_bf16=x)
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_gemm(c, sf, 256, 64, a_bf16=x[:, :32])
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_dgrad(x, c, sf, 256, 64)                  # dY has 64 columns, N = 256
    ids = torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        nv.nvfp4_mxfp4_grouped_gemm(ids.long(), x, c, sf, 256, 64, 1)
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_mxfp4_grouped_gemm(ids, x, c, sf, 128, 64, 2)   # N % 256
    with pytest.raises(ValueError):
        nv.nvfp4_mxfp4_moe_down_combine(x, ids.reshape(-1), ids.reshape(-1)[:2],
                                        torch.ones(16, 2, device="cuda"), c, sf, 256, 64, 1)


@pytest.mark.parametrize("T,E,k,N,K", [(5, 8, 4, 256, 96), (32, 32, 8, 512, 352), (300, 8, 8, 256, 544),
                                       (700, 24, 12, 512, 160)])
def test_moe_down_rounds_once(T, E, k, N, K):
    """The expert outputs reach the weighted sum in fp32 and the sum is rounded
    to bf16 once, also where slots of opposite weights cancel: 2e-5 of the
    absolute terms per product as everywhere, k + 1 roundings of the sum in fp32
    (2^-24 of its absolute terms each), half a bf16 ulp of the result."""
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=51)
    h = bits(rng, T * k, K)
    flat = ids.reshape(-1)
    perm = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    hv = mo.dequantize(*mo.quantize(h))
    d, S = np.zeros((T * k, N)), np.zeros((T * k, N))
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        d[r], S[r] = product(hv[r], wl[e])
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    y = nv.nvfp4_mxfp4_moe_down_combine(dev_bf16(h), torch.from_numpy(perm.astype(np.int32)).cuda(),
                                        torch.from_numpy(offsets.astype(np.int32)).cuda(),
                                        torch.from_numpy(w).cuda(), wc_d, wsf_d, N, K, E)
    want, term = o.moe_combine(d, perm, w, k), o.moe_combine(np.abs(d), perm, np.abs(w), k)
    before = 2e-5 * o.moe_combine(S, perm, np.abs(w), k) + (k + 1) * 2.0 ** -24 * term
    err = np.abs(y.float().cpu().numpy() - want)
    assert np.all(err <= before + 0.5 * o.bf16_ulp(np.abs(want) + before)), float(np.max(err / np.abs(want).max()))


@pytest.mark.parametrize("M,N,K", [(0, 64, 64), (8, 0, 64), (8, 64, 0), (300, 0, 64), (0, 0, 0), (8, -64, 64)])
def test_empty_sizes_are_refused(M, N, K):
    """As an error of the call, from every entry point that asks for its workspace first."""
    x = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    codes, sf = (torch.zeros(1 << 15, device="cuda", dtype=torch.uint8) for _ in range(2))
    with pytest.raises((nv.NVFP4Error, RuntimeError)):
        nv.nvfp4_mxfp4_gemm(codes, sf, N, K, a_bf16=x)
    with pytest.raises((nv.NVFP4Error, RuntimeError)):
        nv.nvfp4_mxfp4_dgrad(torch.zeros(M, max(N, 0), device="cuda", dtype=torch.bfloat16), codes, sf, max(N, 0), K)
    ids = torch.zeros(M, 1, device="cuda", dtype=torch.int32)
    with pytest.raises((nv.NVFP4Error, RuntimeError)):
        nv.nvfp4_mxfp4_grouped_gemm(ids, x, codes, sf, N, K, 1)


@pytest.mark.parametrize("T,E,k,N,K,heavy", [(64, 64, 2, 2048, 736, 0), (128, 64, 1, 512, 352, 128),
                                             (120, 40, 1, 256, 1056, 70), (16, 32, 8, 1024, 2048, 16),
                                             (42, 16, 3, 768, 96, 42), (1, 256, 8, 256, 4128, 0), (65, 16, 1, 256, 64, 33),
                                             (250, 32, 1, 512, 480, 190)])
def test_grouped_decode(T, E, k, N, K, heavy):
    """Few routed rows (the operand-swapped kernel), with more units than CTAs, K
    that wraps its stages, and one expert that takes `heavy` of the tokens: its rows
    in one to four groups of 32 and in two m-tiles; some choices dropped in the
    second run."""
    rng, wl, wc_d, wsf_d, ids = expert_case(T, E, k, N, K, seed=61)
    for t in range(heavy):
        if 3 not in ids[t]:
            ids[t, t % k] = 3
    x, h = bits(rng, T, K), bits(rng, T * k, K)
    hv = mo.dequantize(*mo.quantize(h))
    w = rng.uniform(-1, 1, (T, k)).astype(np.float32)
    for drop in (0, 1):
        if drop:
            ids[::3, k - 1] = -1
        d, S, perm, offsets = grouped_reference(mo.dequantize(*mo.quantize(x)), ids, wl)
        n = len(perm)
        ids_d = torch.from_numpy(np.ascontiguousarray(ids)).cuda()
        for out_dtype in (torch.float32, torch.bfloat16):
            call, (got, p, offs) = nv.prepare_mxfp4_grouped(ids_d, dev_bf16(x), wc_d, wsf_d, N, K, E,
                                                            out_dtype=out_dtype)
            got.fill_(-7.0)
            for _ in range(3):
                call()
            assert nv.read_device_status(call.workspace) == 0
            assert np.array_equal(p[:n].cpu().numpy(), perm) and np.array_equal(offs.cpu().numpy(), offsets)
            if n:
                assert_gemm_close(got[:n], d, S)
            assert torch.all(got[n:] == -7.0)
        want, term, prod = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N))
        for e in range(E):
            r = slice(offsets[e], offsets[e + 1])
            de, Se = product(hv[r], wl[e])
            for i, pair in enumerate(perm[r]):
                want[pair // k] += w[pair // k, pair % k] * de[i]
                term[pair // k] += abs(w[pair // k, pair % k]) * np.abs(de[i])
                prod[pair // k] += abs(w[pair // k, pair % k]) * Se[i]
        y = nv.nvfp4_mxfp4_moe_down_combine(dev_bf16(h), p, offs, torch.from_numpy(w).cuda(), wc_d, wsf_d, N, K, E)
        before = 2e-5 * prod + (k + 1) * 2.0 ** -24 * term
        tol = before + 0.5 * o.bf16_ulp(np.abs(want) + before + 1e-30)
        assert np.all(np.abs(y.float().cpu().numpy() - want) <= tol)
