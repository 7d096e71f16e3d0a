"""Cases of the routed MXFP4 expert layer: expert routing and its gradient, the
MXFP4 round trip, the MXFP4 linear and its input gradient, and the routed
experts' products.

Every operator has a plain form here (elementary torch operations in fp32, one
rounding at the end) and the call a user makes of the package (`own`).  MXFP4
is the OCP microscaled form: E2M1 codes, one E8M0 scale (a power of two) per
32 consecutive elements of a row.
"""
import math

import numpy as np
import torch

#: False: the plain forms.  True: the package's calls.
own = False

DEV = "cuda"
_DTYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one serving step of 8 requests through a 256-expert router with group-limited selection
        dict(name="route decode 8x256", op="route", T=8, E=256, k=8, dtype="fp32", score="sigmoid", bias=True,
             groups=8, topk_groups=4, renorm=True, scale=2.5),
        # a large training batch, softmax scores, an odd number of tokens
        dict(name="route batch 65521x256", op="route", T=65521, E=256, k=8, dtype="bf16", score="softmax",
             bias=False, groups=1, topk_groups=1, renorm=True, scale=1.0),
        # the router's gradient for one prefill-sized batch
        dict(name="route grad 4096x256", op="route_grad", T=4096, E=256, k=8, dtype="fp32", score="sigmoid",
             renorm=True, scale=2.5),
        # the router's gradient where every expert's logit gets one (softmax, weights not renormalised)
        dict(name="route grad 65521x160", op="route_grad", T=65521, E=160, k=6, dtype="bf16", score="softmax",
             renorm=False, scale=1.0),
        # a few rows of activations, a row length that is no multiple of the kernel's tile
        dict(name="round trip 37x2080", op="round_trip", B=1, R=37, C=2080),
        # a layer's expert weights, the quantisation sweep of a checkpoint conversion
        dict(name="round trip 32x2048x6144", op="round_trip", B=32, R=2048, C=6144),
        # single-token decode through the attention output projection
        dict(name="linear decode 1x6144x16384", op="linear", M=1, N=6144, K=16384, out="bf16"),
        # prefill / training forward of the shared linear
        dict(name="linear 8192x2048x6144", op="linear", M=8192, N=2048, K=6144, out="bf16"),
        # input gradient of the frozen linear, odd number of tokens, fp32 out
        dict(name="linear grad 1021x2048x6144", op="linear_grad", M=1021, N=2048, K=6144, out="fp32"),
        # input gradient of the frozen linear, a training batch
        dict(name="linear grad 8192x2048x6144", op="linear_grad", M=8192, N=2048, K=6144, out="bf16"),
        # a serving step of 32 tokens through 32 experts' down-projection with the weighted sum over slots
        dict(name="experts down 32 of 32", op="experts_down", T=32, k=8, E=32, N=6144, K=2048),
        # prefill through 256 experts' up-projection, skewed routing
        dict(name="experts up 4096 of 256", op="experts_up", T=4096, k=8, E=256, N=2048, K=6144, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(rng, lo, hi, step):
    """A multiple of `step`, spread over the logarithm of [lo, hi]."""
    n = max(lo, min(hi, _log(rng, lo, hi) // step * step))
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(("route", "route", "route_grad", "round_trip", "linear", "linear", "linear_grad", "experts_up",
                     "experts_down"))
    if op in ("route", "route_grad"):
        score = rng.choice(("sigmoid", "softmax"))
        groups = rng.choice((1, 1, 2, 4, 8)) if op == "route" else 1
        per = _log(rng, 4, 512 // groups)
        E = groups * per
        topk_groups = rng.randint(1, groups)
        c = dict(op=op, T=_log(rng, 1, 65521), E=E, k=rng.randint(1, min(10, topk_groups * per)),
                 dtype=rng.choice(("bf16", "fp32")), score=score, renorm=rng.random() < 0.7,
                 scale=rng.choice((1.0, 2.5)))
        if op == "route":
            c.update(bias=score == "sigmoid" and rng.random() < 0.7, groups=groups, topk_groups=topk_groups)
        return c
    if op == "round_trip":
        return dict(op=op, B=rng.randint(1, 4), R=_log(rng, 1, 8192), C=_step(rng, 32, 8192, 32))
    if op in ("linear", "linear_grad"):
        lo = 1 if op == "linear" else 16
        return dict(op=op, M=_log(rng, lo, 8191), N=_step(rng, 64, 8192, 8), K=_step(rng, 64, 8192, 32),
                    out=rng.choice(("bf16", "fp32")))
    E = rng.choice((4, 8, 31, 64))
    c = dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, min(8, E)), E=E, N=256 * rng.randint(1, 8),
             K=_step(rng, 64, 6144, 32))
    if op == "experts_up":
        c["out"] = rng.choice(("bf16", "fp32"))
    return c


# ------------------------------------------------------------------- work --

def _popularity(E):
    """Expected share of the router's choices that go to each expert (the recipe of _expert_ids)."""
    p = np.arange(1, E + 1, dtype=np.float64) ** -1.1
    return p / p.sum()


def _active(T, k, E):
    """About how many of E experts get a row."""
    return float(np.sum(1.0 - (1.0 - np.minimum(1.0, k * _popularity(E))) ** T))


def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        item = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * E * item + T * k * 8, "flops": 4.0 * T * E}
        dense = case["score"] == "softmax" and not case["renorm"]
        return {"bytes": T * E * item + T * k * 8 + T * (E if dense else k) * item, "flops": 4.0 * T * (E if dense else k)}
    if op == "round_trip":
        n = case["B"] * case["R"] * case["C"]
        return {"bytes": n * (2 + 0.53125 + 0.53125 + 2), "flops": 4.0 * n}
    N, K = case["N"], case["K"]
    if op in ("linear", "linear_grad"):
        M = case["M"]
        item = 2 if case["out"] == "bf16" else 4
        moved = 2 * M * K + item * M * N if op == "linear" else 2 * M * N + item * M * K
        return {"bytes": moved + 0.53125 * N * K, "flops": 2.0 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    weights = _active(T, k, E) * N * K * 0.53125
    if op == "experts_up":
        return {"bytes": 2 * T * K + T * k * (8 + N * (2 if case["out"] == "bf16" else 4)) + weights,
                "flops": 2.0 * T * k * N * K}
    return {"bytes": 2 * T * k * K + 8 * T * k + 2 * T * N + weights, "flops": 2.0 * T * k * N * K}


# --------------------------------------------------------------- MXFP4 form --

def _pow2(byte):
    """2^(byte - 127) in fp32 (255: NaN)."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23)
    return torch.where(b == 255, torch.full_like(b, 0x7FC00000), bits).view(torch.float32)


def _encode(x):
    """bf16 [..., C] -> (codes 0..15 [..., C], scale bytes [..., C/32])."""
    f = x.float()
    f = f.reshape(*f.shape[:-1], f.shape[-1] // 32, 32)
    amax = f.abs().amax(-1)
    exponent = amax.view(torch.int32) >> 23
    bad = (f != f).any(-1) | (exponent == 255)
    byte = torch.where(bad, torch.full_like(exponent, 255), (exponent - 2).clamp_min(0))
    # 2^(127 - byte) with its exponent field 254 - byte; byte 253 and above never come from finite values
    inverse = ((254 - byte.clamp_max(252)) << 23).view(torch.float32)
    v = f.abs() * inverse[..., None]
    m = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int() + (v > 2.5).int()
         + (v >= 3.5).int() + (v > 5.0).int())
    code = torch.where(bad[..., None], torch.zeros_like(m), m + 8 * torch.signbit(f).int())
    return code.reshape(x.shape), byte.to(torch.uint8)


def _values(code, byte):
    """fp32 values of codes [..., C] and scale bytes [..., C/32]."""
    mag = torch.tensor(_E2M1, dtype=torch.float32, device=code.device)[(code & 7).long()]
    v = torch.where(code >= 8, -mag, mag)
    v = v.reshape(*byte.shape, 32) * _pow2(byte)[..., None]
    return v.reshape(code.shape)


def _pack(x):
    """bf16 [..., C] -> packed codes [..., C/2] (even element in the low nibble), scale bytes [..., C/32]."""
    code, byte = _encode(x)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), byte


def _unpack(codes, byte):
    return _values(torch.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1).int(), byte)


def _swizzle(byte):
    """Scale bytes [R, S] in 128 x 4 atoms: the order that the tensor cores take them in."""
    R, S = byte.shape
    pad = torch.zeros((R + 127) // 128 * 128, (S + 3) // 4 * 4, dtype=torch.uint8, device=byte.device)
    pad[:R, :S] = byte
    return pad.reshape(pad.shape[0] // 128, 4, 32, pad.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


# ----------------------------------------------------------------- prepare --

def _normal(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def _activations(gen, rows, cols):
    """Unit-variance activations, one in a hundred an outlier."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x = torch.where(torch.rand(rows, cols, generator=gen, device=DEV) < 0.01, x * 20, x)
    return x.to(torch.bfloat16)


def _expert_ids(gen, T, k, E):
    """Skewed routing: top-k of normal scores plus a bias of -1.1 ln(rank), ranks shuffled."""
    rank = torch.randperm(E, generator=gen, device=DEV) + 1
    score = torch.randn(T, E, generator=gen, device=DEV) - 1.1 * rank.float().log()
    return torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()


def _expert_weights(gen, E, N, K):
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    byte = torch.empty(E, N, K // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        codes[e], byte[e] = _pack(_normal(gen, N, K, scale=0.02))
    return codes, byte


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op in ("route", "route_grad"):
        T, E, k = case["T"], case["E"], case["k"]
        skew = -0.5 * (torch.randperm(E, generator=gen, device=DEV) + 1).float().log()
        s["logits"] = (torch.randn(T, E, generator=gen, device=DEV) + skew).to(_DTYPE[case["dtype"]])
        if op == "route":
            s["b"] = torch.randn(E, generator=gen, device=DEV) * 0.05 if case["bias"] else None
        else:
            s["ids"] = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :k]
            s["ids"] = s["ids"].to(torch.int32).contiguous()
            s["grad"] = torch.randn(T, k, generator=gen, device=DEV) * 1e-2
    elif op == "round_trip":
        s["x"] = _normal(gen, case["B"], case["R"], case["C"], scale=0.02)
        s["x"] = torch.where(torch.rand(s["x"].shape, generator=gen, device=DEV) < 0.001, s["x"] * 50, s["x"])
    elif op in ("linear", "linear_grad"):
        s["codes"], s["byte"] = _pack(_normal(gen, case["N"], case["K"], scale=0.02))
        s["sf"] = _swizzle(s["byte"])
        s["x"] = (_activations(gen, case["M"], case["K"]) if op == "linear"
                  else _normal(gen, case["M"], case["N"], scale=1e-2))
    else:
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        s["codes"], s["byte"] = _expert_weights(gen, E, N, K)
        s["sf"] = _swizzle(s["byte"].reshape(E * N, K // 32))
        s["ids"] = _expert_ids(gen, T, k, E)
        if op == "experts_up":
            s["x"] = _activations(gen, T, K)
        else:
            # the expert-grouped order of the up-projection: rows of one expert together, by pair index
            s["x"] = _activations(gen, T * k, K)
            flat = s["ids"].reshape(-1).long()
            s["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32)
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
            s["offsets"][1:] = torch.bincount(flat, minlength=E).cumsum(0).to(torch.int32)
            w = torch.rand(T, k, generator=gen, device=DEV) + 0.05
            s["w"] = w / w.sum(1, keepdim=True)
    if own:
        _plan(s)
    return s


def _plan(s):
    """The package's prepared call of this state: its output buffers and workspace."""
    import nvfp4_block_scaled_06_gb300 as nv
    op = s["op"]
    if op == "route":
        s["call"], s["y"] = nv.prepare_route_topk(
            s["logits"], s["k"], bias=s["b"], score=s["score"], num_groups=s["groups"],
            topk_groups=s["topk_groups"], group_top=2 if s["score"] == "sigmoid" else 1, renormalize=s["renorm"],
            scale=s["scale"])
    elif op == "route_grad":
        s["call"], s["y"] = nv.prepare_route_topk_backward(
            s["logits"], s["ids"], s["grad"], score=s["score"], renormalize=s["renorm"], scale=s["scale"])
    elif op == "round_trip":
        quantize, q = nv.prepare_mxfp4_quantize(s["x"], sf_layout="linear")
        dequantize, s["y"] = nv.prepare_mxfp4_dequantize(q["codes"], q["sf"], sf_layout="linear")
        s["call"] = lambda: (quantize(), dequantize())
    elif op == "linear":
        s["call"], s["y"] = nv.prepare_mxfp4_gemm(s["codes"], s["sf"], s["N"], s["K"], a_bf16=s["x"],
                                                  out_dtype=_DTYPE[s["out"]])
    elif op == "linear_grad":
        s["call"], s["y"] = nv.prepare_mxfp4_dgrad(s["x"], s["codes"], s["sf"], s["N"], s["K"],
                                                   out_dtype=_DTYPE[s["out"]])
    elif op == "experts_up":
        s["call"], s["y"] = nv.prepare_mxfp4_grouped(s["ids"], s["x"], s["codes"], s["sf"], s["N"], s["K"], s["E"],
                                                     out_dtype=_DTYPE[s["out"]])
    else:
        s["call"], s["y"] = nv.prepare_mxfp4_moe_down(s["x"], s["perm"], s["offsets"], s["w"], s["codes"], s["sf"],
                                                      s["N"], s["K"], s["E"])


# --------------------------------------------------------------------- run --

def run(state):
    if own:
        state["call"]()
        return state["y"]
    return globals()["_plain_" + state["op"]](state)


def _first(keys, k):
    """Indices of the k largest of each row, ties to the lowest index."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k]


def _scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _select(x, s):
    """(scores, chosen experts): keys are the scores plus the bias, without one the logits.  Groups are
    ranked by the sum of their two largest scores (plus bias) for sigmoid, by their largest key for softmax."""
    T, E = x.shape
    p = _scores(x, s["score"])
    biased = p if s["b"] is None else p + s["b"]
    key = x if s["b"] is None else biased
    if s["groups"] > 1:
        g = key.reshape(T, s["groups"], E // s["groups"])
        if s["score"] == "sigmoid" and g.shape[2] > 1:
            top = torch.sort(biased.reshape(g.shape), dim=2, descending=True).values[:, :, :2]
            rank = top[:, :, 0] + top[:, :, 1]
        else:
            rank = g.amax(2)
        keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=x.device)
        keep.scatter_(1, _first(rank, s["topk_groups"]), True)
        key = torch.where(keep[:, :, None], g, torch.full_like(g, -math.inf)).reshape(T, E)
    return p, _first(key, s["k"])


def _plain_route(s):
    p, ids = _select(s["logits"].float(), s)
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"expert_ids": ids.to(torch.int32), "weights": w * s["scale"]}


def _plain_route_grad(s):
    x, ids = s["logits"].float(), s["ids"].long()
    p = _scores(x, s["score"])
    sel = p.gather(1, ids)
    d = s["grad"] * s["scale"]
    if s["renorm"]:
        total = sel.sum(1, keepdim=True)
        d = (d - (d * sel).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_(1, ids, d)
    if s["score"] == "sigmoid":
        g = ds * p * (1.0 - p)
    else:
        g = p * (ds - (ds * p).sum(1, keepdim=True))
        if s["renorm"]:      # the other experts' part cancels: the weights depend on the chosen logits alone
            g = torch.zeros_like(p).scatter_(1, ids, g.gather(1, ids))
    return g.to(s["logits"].dtype)


def _plain_round_trip(s):
    return _values(*_encode(s["x"])).to(torch.bfloat16)


def _plain_linear(s):
    x = _values(*_encode(s["x"]))
    return (x @ _unpack(s["codes"], s["byte"]).t()).to(_DTYPE[s["out"]])


def _plain_linear_grad(s):
    return (s["x"].float() @ _unpack(s["codes"], s["byte"])).to(_DTYPE[s["out"]])


def _expert_products(rows, s, offsets):
    """Rows of each expert (offsets on the host) times its weights, fp32."""
    d = torch.empty(rows.shape[0], s["N"], dtype=torch.float32, device=rows.device)
    for e in range(s["E"]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            d[a:b] = rows[a:b] @ _unpack(s["codes"][e], s["byte"][e]).t()
    return d


def _plain_experts_up(s):
    flat = s["ids"].reshape(-1).long()
    perm = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(s["E"] + 1, dtype=torch.int32, device=flat.device)
    offsets[1:] = torch.bincount(flat, minlength=s["E"]).cumsum(0).to(torch.int32)
    x = _values(*_encode(s["x"]))
    d = _expert_products(x[perm // s["k"]], s, offsets.tolist())
    return d.to(_DTYPE[s["out"]]), perm.to(torch.int32), offsets


def _plain_experts_down(s):
    d = _expert_products(_values(*_encode(s["x"])), s, s["offsets"].tolist())
    pairs = torch.empty_like(d)
    pairs[s["perm"].long()] = d
    y = (pairs.reshape(s["T"], s["k"], s["N"]) * s["w"][:, :, None]).sum(1)
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------- exact --
# From the definitions in 64 bits, apart from the plain forms: scales by frexp,
# codes by rounding to the spacing of the E2M1 grid, softmax by log-sum-exp.

def _exact_mx(x):
    f = x.double().reshape(*x.shape[:-1], -1, 32)
    _, exponent = torch.frexp(f.abs().amax(-1, keepdim=True))          # amax = m 2^exponent, 0.5 <= m < 1
    scale = torch.exp2((exponent - 3).clamp_min(-127).double())        # 2^(floor(log2 amax) - 2)
    v = f / scale
    spacing = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    return ((v / spacing).round() * spacing).clamp(-6, 6).mul(scale).reshape(x.shape)


def _exact_packed(codes, byte):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=codes.device)
    v = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    v[..., 0::2] = table[(codes & 15).long()]
    v[..., 1::2] = table[(codes >> 4).long()]
    return (v.reshape(*byte.shape, 32) * torch.exp2(byte.double() - 127)[..., None]).reshape(v.shape)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return globals()["_exact_" + case["op"]](s)


def _exact_route(s):
    # the choice is by fp32 keys; the weights are a function of the logits of the chosen
    _, ids = _select(s["logits"].float(), s)
    x = s["logits"].double()
    log_p = -torch.log1p(torch.exp(-x)) if s["score"] == "sigmoid" else x - torch.logsumexp(x, 1, keepdim=True)
    log_w = log_p.gather(1, ids)
    if s["renorm"]:
        log_w = log_w - torch.logsumexp(log_w, 1, keepdim=True)
    return {"expert_ids": None, "weights": log_w.exp() * s["scale"]}


def _exact_route_grad(s):
    # the derivative of sum(grad * weights) by torch's reverse mode in 64 bits
    x = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
        w = p.gather(1, s["ids"].long())
        if s["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (w * s["grad"].double() * s["scale"]).sum().backward()
    return x.grad


def _exact_round_trip(s):
    return torch.stack([_exact_mx(m) for m in s["x"]])


def _exact_linear(s):
    return _exact_mx(s["x"]) @ _exact_packed(s["codes"], s["byte"]).t()


def _exact_linear_grad(s):
    return s["x"].double() @ _exact_packed(s["codes"], s["byte"])


def _exact_products(x, ids, s):
    """x: one row per pair; its product with its expert's weights."""
    d = torch.empty(x.shape[0], s["N"], dtype=torch.float64, device=x.device)
    for e in range(s["E"]):
        at = torch.nonzero(ids == e).squeeze(1)
        if at.numel():
            d[at] = _exact_mx(x[at]) @ _exact_packed(s["codes"][e], s["byte"][e]).t()
    return d


def _exact_experts_up(s):
    ids = s["ids"].reshape(-1).long()
    d = _exact_products(s["x"].repeat_interleave(s["k"], 0), ids, s)
    order = torch.argsort(ids * ids.numel() + torch.arange(ids.numel(), device=ids.device))
    return d[order], None, None


def _exact_experts_down(s):
    ids = s["ids"].reshape(-1).long()
    x = torch.empty_like(s["x"])
    x[s["perm"].long()] = s["x"]
    d = _exact_products(x, ids, s).reshape(s["T"], s["k"], s["N"])
    return torch.einsum("tk,tkn->tn", s["w"].double(), d)
