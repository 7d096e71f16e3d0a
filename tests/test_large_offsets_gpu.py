"""Routing and MXFP4 calls on buffers of more than 2^32 bytes and 2^31 elements:
blocks of rows from the start, the middle and the end against the same call on
those rows alone, bit for bit (a row's result depends on no other row)."""
import pytest
import torch

import nvfp4_block_scaled_06_gb300 as nv

pytestmark = pytest.mark.gpu


def blocks(rows, size):
    return [slice(a, a + size) for a in (0, rows // 2 - 3, rows - size)]


def rand_bf16(rows, cols, scale=1.0):
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    for s in range(0, rows, 1 << 15):
        x[s:s + (1 << 15)].normal_(0, scale)
    return x


def test_quantize_and_dequantize():
    R, Cc = (1 << 17) + 40, 1 << 15              # 2^32 elements and more
    x = rand_bf16(R, Cc)
    for layout in ("linear", "swizzled"):
        q = nv.nvfp4_mxfp4_quantize(x, sf_layout=layout)
        for b in blocks(R, 8):
            want = nv.nvfp4_mxfp4_quantize(x[b], sf_layout="linear")
            assert torch.equal(q["codes"][b], want["codes"])
            if layout == "linear":
                assert torch.equal(q["sf"][b], want["sf"])
        y = nv.nvfp4_mxfp4_dequantize(q["codes"], q["sf"], sf_layout=layout)
        for b in blocks(R, 8):
            want = nv.nvfp4_mxfp4_quantize(x[b], sf_layout="linear")
            assert torch.equal(y[b], nv.nvfp4_mxfp4_dequantize(want["codes"], want["sf"], sf_layout="linear"))
        del y
    t = nv.nvfp4_mxfp4_dequantize(q["codes"], q["sf"], transpose=True)
    for b in blocks(R, 8):
        want = nv.nvfp4_mxfp4_quantize(x[b], sf_layout="linear")
        assert torch.equal(t[:, b].t(), nv.nvfp4_mxfp4_dequantize(want["codes"], want["sf"], sf_layout="linear"))


def test_routing_and_its_gradient():
    T, E, k = (1 << 22) + 5, 1000, 8             # 4.2e9 logits
    x = rand_bf16(T, E)
    r = nv.nvfp4_route_topk(x, k, score="softmax", renormalize=False)
    g = torch.randn(T, k, device="cuda")
    d = nv.nvfp4_route_topk_backward(x, r["expert_ids"], g, score="softmax", renormalize=False)
    for b in blocks(T, 64):
        want = nv.nvfp4_route_topk(x[b], k, score="softmax", renormalize=False)
        assert torch.equal(r["expert_ids"][b], want["expert_ids"])
        assert torch.allclose(r["weights"][b], want["weights"], rtol=2.0 ** -18, atol=0)   # (another order of sums)
        assert torch.equal(d[b], nv.nvfp4_route_topk_backward(x[b], r["expert_ids"][b], g[b], score="softmax",
                                                              renormalize=False))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_gemm(out_dtype):
    M, N, K = (1 << 18) + 77, 16392, 64          # 4.3e9 elements of D
    x = rand_bf16(M, K)
    w = nv.nvfp4_mxfp4_quantize(rand_bf16(N, K, 0.02))
    y = nv.nvfp4_mxfp4_gemm(w["codes"], w["sf"], N, K, a_bf16=x, out_dtype=out_dtype)
    for b in blocks(M, 300):
        assert torch.equal(y[b], nv.nvfp4_mxfp4_gemm(w["codes"], w["sf"], N, K, a_bf16=x[b], out_dtype=out_dtype))


def test_routed_products():
    T, E, k, N, K = 1 << 16, 16, 8, 8192, 64     # 4.3e9 elements of D
    ids = torch.rand(T, E, device="cuda").argsort(1)[:, :k].int().contiguous()
    x = rand_bf16(T, K)
    w = nv.nvfp4_mxfp4_quantize(rand_bf16(E * N, K, 0.02))
    d, perm, offs = nv.nvfp4_mxfp4_grouped_gemm(ids, x, w["codes"], w["sf"], N, K, E)
    for t in (0, T // 2, T - 1):
        want, p, o = nv.nvfp4_mxfp4_grouped_gemm(ids[t:t + 1], x[t:t + 1], w["codes"], w["sf"], N, K, E)
        inv = torch.empty(T * k, dtype=torch.int64, device="cuda")
        inv[perm.long()] = torch.arange(T * k, device="cuda")
        for i in range(k):
            assert torch.equal(d[inv[t * k + int(p[i])]], want[i])
    del d, want, inv
    rw = torch.rand(T, k, device="cuda")
    h = rand_bf16(T * k, K)
    y = nv.nvfp4_mxfp4_moe_down_combine(h, perm, offs, rw, w["codes"], w["sf"], N, K, E)
    inv = torch.empty(T * k, dtype=torch.int64, device="cuda")
    inv[perm.long()] = torch.arange(T * k, device="cuda")
    for t in (0, T // 2, T - 1):
        order = ids[t].long().argsort()
        rows = h[inv[t * k + order]].contiguous()
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.bincount(ids[t].long(), minlength=E).cumsum(0).int()
        want = nv.nvfp4_mxfp4_moe_down_combine(rows, order.int(), offsets, rw[t:t + 1].contiguous(), w["codes"],
                                               w["sf"], N, K, E)
        assert torch.equal(y[t:t + 1], want)
