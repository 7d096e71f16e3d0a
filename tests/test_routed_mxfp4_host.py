"""Host side of the routing and MXFP4 entry points, no GPU: the ctypes structs
mirror the header, bad arguments are refused before any device work, size
queries; and the CPU reference against independent derivations."""
import ctypes as C
import math
import multiprocessing

import numpy as np
import pytest

import test_abi_layout as abi
from nvfp4_block_scaled_06_gb300 import _binding as B
from oracle import mxfp4_oracle as mo
from oracle.nvfp4_oracle import bf16_to_f32
from synth import f32_to_bf16_bits

P = 4096                 # an aligned stand-in pointer, never dereferenced

MIRRORS = {
    "nvfp4_route_topk_args": B.RouteTopkArgs,
    "nvfp4_route_topk_backward_args": B.RouteTopkBackwardArgs,
    "nvfp4_mxfp4_quant_args": B.MxQuantArgs,
    "nvfp4_mxfp4_dequant_args": B.MxDequantArgs,
    "nvfp4_mxfp4_gemm_args": B.MxGemmArgs,
    "nvfp4_mxfp4_dgrad_args": B.MxDgradArgs,
    "nvfp4_mxfp4_grouped_args": B.MxGroupedArgs,
    "nvfp4_mxfp4_moe_down_args": B.MxMoeDownArgs,
}


@pytest.fixture(scope="module")
def clib():
    from nvfp4_block_scaled_06_gb300 import build as b
    b.build()
    return B.load()


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    was = abi.MIRRORS
    abi.MIRRORS = MIRRORS
    try:
        return abi.c_layout.__wrapped__(tmp_path_factory)
    finally:
        abi.MIRRORS = was


@pytest.mark.parametrize("cname", sorted(MIRRORS))
def test_struct_mirrors_header(cname, layout):
    cls = MIRRORS[cname]
    assert [f for f, _ in cls._fields_] == abi.header_fields(cname)
    for fname, _ in cls._fields_:
        assert getattr(cls, fname).offset == layout[(cname, fname)], fname
    assert C.sizeof(cls) == layout[(cname, ".")]


BASES = {
    "nvfp4_route_topk": (B.RouteTopkArgs, dict(num_tokens=4, num_experts=16, top_k=2, logits=P, ld=16, logits_dtype=1,
                                               num_groups=1, scale=1.0, expert_ids=P, route_weights=P)),
    "nvfp4_route_topk_backward": (B.RouteTopkBackwardArgs,
                                  dict(num_tokens=4, num_experts=16, top_k=2, logits=P, ld=16, expert_ids=P,
                                       grad_weights=P, grad_logits=P, ld_grad=16)),
    "nvfp4_mxfp4_quantize": (B.MxQuantArgs, dict(src=P, batch=1, rows=4, cols=64, ld=64, codes=P, sf=P)),
    "nvfp4_mxfp4_dequantize": (B.MxDequantArgs, dict(codes=P, sf=P, batch=1, rows=4, cols=64, out=P, ldo=64)),
    "nvfp4_mxfp4_gemm": (B.MxGemmArgs, dict(M=8, N=8, K=64, a_bf16=P, lda=64, b_codes=P, b_sf=P, d=P, ldd=8)),
    "nvfp4_mxfp4_dgrad": (B.MxDgradArgs, dict(M=8, N=64, K=64, dy=P, lddy=64, w_codes=P, w_sf=P, dx=P, lddx=64)),
    "nvfp4_mxfp4_grouped_gemm": (B.MxGroupedArgs, dict(num_tokens=4, top_k=2, num_experts=8, N=256, K=64,
                                                       expert_ids=P, x_bf16=P, w_codes=P, w_sf=P, d=P, perm_out=P)),
    "nvfp4_mxfp4_moe_down_combine": (B.MxMoeDownArgs, dict(num_tokens=4, top_k=2, num_experts=8, N=256, K=64, h=P,
                                                           perm=P, expert_offsets=P, route_weights=P, w_codes=P,
                                                           w_sf=P, y=P)),
}
REFUSED = (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED_SHAPE, B.ERR_ALIGNMENT)


def status(clib, name, **kw):
    cls, base = BASES[name]
    return getattr(clib, name)(C.byref(cls(**dict(base, **kw))), None)


@pytest.mark.parametrize("name", sorted(BASES))
def test_base_arguments_pass_and_null_and_empty_are_refused(clib, name):
    """The arguments themselves are accepted (the call then fails for the
    missing device or workspace); each pointer missing, each size 0 is not."""
    cls, base = BASES[name]
    assert status(clib, name) not in REFUSED
    assert getattr(clib, name)(C.cast(None, C.POINTER(cls)), None) == B.ERR_INVALID_ARG
    for field, value in base.items():
        if value == P or field in ("num_tokens", "num_experts", "top_k", "batch", "rows", "cols", "M", "N", "K"):
            assert status(clib, name, **{field: None if value == P else 0}) == B.ERR_INVALID_ARG, field
        if field.startswith("ld"):
            assert status(clib, name, **{field: value - 8}) == B.ERR_INVALID_ARG, field


@pytest.mark.parametrize("name,kw,want", [
    ("nvfp4_route_topk", dict(num_experts=1025, ld=1025), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_route_topk", dict(num_experts=64, ld=64, top_k=33), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_route_topk", dict(top_k=17), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_route_topk", dict(num_groups=3, topk_groups=1, group_top=1), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_route_topk", dict(num_groups=16, topk_groups=1, group_top=1), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_route_topk", dict(num_groups=4, topk_groups=5, group_top=1), B.ERR_INVALID_ARG),
    ("nvfp4_route_topk", dict(num_groups=4, topk_groups=2, group_top=3), B.ERR_INVALID_ARG),
    ("nvfp4_route_topk", dict(score=2), B.ERR_INVALID_ARG),
    ("nvfp4_route_topk", dict(logits_dtype=2), B.ERR_INVALID_ARG),
    ("nvfp4_route_topk", dict(logits=P + 2), B.ERR_ALIGNMENT),
    ("nvfp4_route_topk", dict(bias=P + 1), B.ERR_ALIGNMENT),
    ("nvfp4_route_topk_backward", dict(grad_logits=P + 1), B.ERR_ALIGNMENT),
    ("nvfp4_route_topk_backward", dict(score=-1), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_quantize", dict(cols=48), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_quantize", dict(ld=68), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_quantize", dict(src=P + 8), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_quantize", dict(sf_layout=2), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_quantize", dict(batch=2, batch_stride=128), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_quantize", dict(batch=65536, batch_stride=256), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_dequantize", dict(cols=96, ldo=96 + 4), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_dequantize", dict(transpose=1, ldo=5), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_dequantize", dict(transpose=1, ldo=2), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_gemm", dict(K=48), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_gemm", dict(ldd=12), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_gemm", dict(a_codes=P, a_sf=P), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_gemm", dict(a_bf16=None, a_codes=P), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_gemm", dict(K=(1 << 24) + 32, lda=(1 << 24) + 32), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_dgrad", dict(K=48), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_dgrad", dict(N=60, lddy=60), B.ERR_ALIGNMENT),
    ("nvfp4_mxfp4_grouped_gemm", dict(N=128), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_grouped_gemm", dict(top_k=9), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_grouped_gemm", dict(offsets_in=P, perm_in=P), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_grouped_gemm", dict(x_codes=P, x_sf=P), B.ERR_INVALID_ARG),
    ("nvfp4_mxfp4_grouped_gemm", dict(num_tokens=1 << 40), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_moe_down_combine", dict(K=40), B.ERR_UNSUPPORTED_SHAPE),
    ("nvfp4_mxfp4_moe_down_combine", dict(y=P + 8), B.ERR_ALIGNMENT),
])
def test_refusals(clib, name, kw, want):
    assert status(clib, name, **kw) == want


def test_size_queries(clib):
    assert clib.nvfp4_mxfp4_sf_bytes(2048, 6144, 0) == 2048 * 192
    assert clib.nvfp4_mxfp4_sf_bytes(37, 160, 1) == 128 * 8
    a = B.MxGemmArgs(M=8192, N=2048, K=6144, a_bf16=P, lda=6144, b_codes=P, b_sf=P, d=P, ldd=2048)
    assert clib.nvfp4_mxfp4_gemm_workspace_bytes(C.byref(a)) >= 8192 * 6144 // 2 + 8192 * 192
    d = B.MxDgradArgs(M=64, N=77, K=64, dy=P, lddy=80, w_codes=P, w_sf=P, dx=P, lddx=64)
    assert clib.nvfp4_mxfp4_dgrad_workspace_bytes(C.byref(d)) >= 64 * 80 * 2


@pytest.mark.parametrize("name,field", [
    (n, f) for n in ("nvfp4_grouped_gemm", "nvfp4_mxfp4_grouped_gemm")
    for f in ("expert_ids", "perm_out", "expert_offsets_out")] + [
    (n, f) for n in ("nvfp4_moe_down_combine", "nvfp4_mxfp4_moe_down_combine")
    for f in ("perm", "expert_offsets", "route_weights")])
def test_misaligned_routing_pointers_are_refused(clib, name, field):
    """Pointers to 32-bit elements off a word, which a kernel would fault on."""
    cls, base = BASES.get(name) or {
        "nvfp4_grouped_gemm": (B.GroupedArgs, dict(num_tokens=4, top_k=2, num_experts=8, N=256, K=64, expert_ids=P,
                                                   x_bf16=P, w_codes=P, w_sf=P, w_global_scale=P, d=P, perm_out=P)),
        "nvfp4_moe_down_combine": (B.MoeDownArgs, dict(num_tokens=4, top_k=2, num_experts=8, N=256, K=64, h=P, perm=P,
                                                       expert_offsets=P, route_weights=P, w_codes=P, w_sf=P,
                                                       w_global_scale=P, y=P)),
    }[name]
    for offset, refused in ((4, False), (2, True), (1, True)):
        args = cls(**dict(base, **{field: P + offset}))
        assert (getattr(clib, name)(C.byref(args), None) == B.ERR_ALIGNMENT) == refused, offset


QUERIES = {
    "nvfp4_quantize": (B.QuantArgs, ("batch", "rows", "cols"), ("src",)),
    "nvfp4_gemm": (B.GemmArgs, ("M", "N", "K"), ("a_bf16",)),
    "nvfp4_grouped": (B.GroupedArgs, ("num_tokens", "top_k", "num_experts", "N", "K"), ("expert_ids", "x_bf16")),
    "nvfp4_lora": (B.LoraArgs, ("M", "N", "K"), ("x",)),
    "nvfp4_dgrad": (B.DgradArgs, ("M", "N", "K"), ("dy",)),
    "nvfp4_wgrad": (B.WgradArgs, ("M", "N", "K"), ("dy", "x")),
    "nvfp4_moe_down": (B.MoeDownArgs, ("num_tokens", "top_k", "num_experts", "N", "K"), ("h",)),
    "nvfp4_mxfp4_gemm": (B.MxGemmArgs, ("M", "N", "K"), ("a_bf16",)),
    "nvfp4_mxfp4_dgrad": (B.MxDgradArgs, ("M", "N", "K"), ("dy",)),
    "nvfp4_mxfp4_grouped": (B.MxGroupedArgs, ("num_tokens", "top_k", "num_experts", "N", "K"),
                            ("expert_ids", "x_bf16")),
    "nvfp4_mxfp4_moe_down": (B.MxMoeDownArgs, ("num_tokens", "top_k", "num_experts", "N", "K"), ("h",)),
}


def ask_every_query(out):
    """Sends (query, field, value, answer) of every answer that is wrong."""
    lib, bad = B.load(), []
    for name, (cls, sizes, pointers) in QUERIES.items():
        query = getattr(lib, f"{name}_workspace_bytes")
        for given in (pointers, ()):
            base = dict({f: 64 if f == "K" else 8 for f in sizes}, **{f: P for f in given})
            if name in ("nvfp4_lora", "nvfp4_gemm"):
                base["rank"] = 32
            for field in sizes:
                for value in (0, -1, -200, base[field]):
                    n = query(C.byref(cls(**dict(base, **{field: value}))))
                    if (n != 0 if value < 1 else n >= 1 << 32):
                        bad.append((name, field, value, n))
    out.send(bad)


def test_workspace_queries_of_empty_and_negative_sizes(clib):
    """A size query is made before the call refuses an empty operand: it answers 0.
    (Asked in a process of its own, which a division by zero would end.)"""
    assert {f"{n}_workspace_bytes" for n in QUERIES} == {n for n in B.EXPORTS if n.endswith("_workspace_bytes")}
    ctx = multiprocessing.get_context("spawn")
    here, there = ctx.Pipe(duplex=False)
    child = ctx.Process(target=ask_every_query, args=(there,))
    child.start()
    child.join(120)
    assert child.exitcode == 0
    assert here.recv() == []


# --------------------------------------------------------- reference pinned --

def test_reference_codes_against_hand_ties_and_brute_force():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 6.5: 7, 100.0: 7, 0.0: 0, 5.01: 7, 0.2501: 1}
    assert mo.e2m1_round(np.array(list(ties))).tolist() == list(ties.values())
    for v in np.linspace(0, 8, 4001):
        c = int(mo.e2m1_round(np.array([v]))[0])
        best = min(abs(v - g) for g in mo.E2M1)
        assert math.isclose(abs(v - mo.E2M1[c]), best, abs_tol=0)


def test_reference_round_trip_and_scale_rule():
    rng = np.random.default_rng(0)
    b = f32_to_bf16_bits((rng.standard_normal((64, 256)) * 10.0 ** rng.integers(-20, 20, (64, 1))).astype(np.float32))
    x = bf16_to_f32(b).astype(np.float64)
    codes, byte = mo.quantize(b)
    v = mo.dequantize(codes, byte)
    blocks = np.abs(x.reshape(64, 8, 32)).max(-1)
    X = np.ldexp(1.0, byte.astype(int) - 127)
    assert np.all((blocks / X >= 4) & (blocks / X < 8))            # 2^(floor(log2 amax) - 2)
    again = mo.quantize(f32_to_bf16_bits(v.astype(np.float32)))
    assert np.array_equal(mo.dequantize(*again), v)                # representable values come back
    # each value is within half a grid step (1 at the top of the range; saturation adds up to 2)
    err = np.abs(v - x).reshape(64, 8, 32) / X[..., None]
    assert np.all(err <= np.where(np.abs(x.reshape(64, 8, 32)) / X[..., None] <= 6, 1.0, 2.0))


def test_reference_swizzle_matches_the_nvfp4_layout():
    from oracle.nvfp4_oracle import sf_swizzle
    byte = np.random.default_rng(1).integers(0, 255, (200, 12)).astype(np.uint8)
    assert np.array_equal(mo.sf_swizzle(byte), np.asarray(sf_swizzle(byte)).reshape(-1))


def test_reference_routing_by_hand():
    x = np.array([[0.0, 2.0, 1.0, 2.0], [-np.inf, np.nan, 0.0, -np.inf]])
    ids, w, _ = mo.route_topk(x, 2)
    s = lambda v: 1 / (1 + math.exp(-v))  # noqa: E731
    assert ids.tolist() == [[1, 3], [2, -1]]
    assert np.allclose(w, [[0.5, 0.5], [1.0, 0.0]])
    ids, w, _ = mo.route_topk(x[:1], 2, bias=np.array([1.0, 0, 0.5, 0]), renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[2 * s(0.0), 2 * s(1.0)]])
    # groups {0,1}, {2,3}: by the largest logit group 0 wins the tie, by the sum of two group 1
    assert mo.route_topk(x[:1], 1, num_groups=2, topk_groups=1, group_top=1)[0].tolist() == [[1]]
    assert mo.route_topk(x[:1], 1, num_groups=2, topk_groups=1, group_top=2)[0].tolist() == [[3]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    x, g, h = rng.standard_normal((4, 12)), rng.standard_normal((4, 3)), 1e-5
    ids, _, _ = mo.route_topk(x, 3, score=score)
    got = mo.route_topk_backward(x, ids, g, score, renorm, 1.5)
    for e in range(12):
        out = []
        for sign in (1, -1):
            v = x.copy()
            v[:, e] += sign * h
            w = np.take_along_axis(mo.scores(v, score), ids, 1)
            out.append(((w / w.sum(1, keepdims=True) if renorm else w) * g * 1.5).sum(1))
        assert np.allclose((out[0] - out[1]) / (2 * h), got[:, e], atol=1e-8)
