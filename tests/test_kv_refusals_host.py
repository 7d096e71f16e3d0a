"""What the calls on the key-value cache refuse before any device work, beyond test_kv_host.py: scales whose
form for the kernels overflows, strides that let rows overlap."""

import numpy as np
import pytest

from nvfp4_block_scaled_06_gb300 import _binding as B
from test_kv_host import REFUSED, attend, clib, read, write  # noqa: F401


@pytest.mark.parametrize("scale", [2.3e38, 2.0 ** 100, 1e-38])
def test_scales_that_the_kernels_can_hold(clib, scale):  # noqa: F811
    assert attend(clib, scale=scale) not in REFUSED


@pytest.mark.parametrize("scale", [2.4e38, 3.0e38, float(np.finfo(np.float32).max)])
def test_scales_whose_base_2_form_overflows(clib, scale):  # noqa: F811
    """The kernels multiply by scale * log2(e): infinite, it would make NaN of every score of 0."""
    assert scale * 1.4426950408889634 > float(np.finfo(np.float32).max)
    assert attend(clib, scale=scale) == B.ERR_INVALID_ARG


# (tokens, heads, row stride, head stride) at head_dim 64, and whether rows are apart
STRIDES = [
    (5, 4, 256, 64, True), (5, 4, 320, 80, True), (5, 4, 248, 64, False), (5, 4, 256, 56, False),
    (5, 4, 64, 320, True), (5, 4, 72, 352, True), (5, 4, 64, 312, False), (5, 4, 56, 320, False),
    (5, 4, 128, 128, False), (5, 4, 0, 320, False), (5, 4, 256, 0, False), (5, 4, -64, 320, False),
    (1, 4, 8, 64, True), (1, 4, 256, 64, True), (1, 4, 0, 56, False), (5, 4, 1 << 62, 1 << 62, False),
    (5, 4, 64, 1 << 62, True), (5, 4, 1 << 62, 64, True), (5, 4, 1 << 61, 1 << 62, False),
]


@pytest.mark.parametrize("tokens,heads,ld,head_ld,apart", STRIDES)
def test_strides_of_tokens_and_heads(clib, tokens, heads, ld, head_ld, apart):  # noqa: F811
    """Heads within a token's row, or tokens within a head's matrix; no two rows share an element."""
    cache = dict(num_kv_heads=heads, codes_page_stride=heads * 16 * 32, sf_page_stride=heads * 16 * 4)
    for name in ("k", "v"):
        form = {f"{m}_ld": 64 * heads for m in "kv"} | {f"{m}_head_ld": 64 for m in "kv"}
        form |= {f"{name}_ld": ld, f"{name}_head_ld": head_ld, "num_tokens": tokens}
        for call in (write, read):
            got = call(clib, cache, **form)
            assert (got not in REFUSED) if apart else got == B.ERR_INVALID_ARG, (call.__name__, name)
    for name in ("q", "out"):
        got = attend(clib, total_q=tokens, num_seqs=tokens, num_heads=heads, **{f"{name}_ld": ld, f"{name}_head_ld": head_ld})
        assert (got not in REFUSED) if apart else got == B.ERR_INVALID_ARG, name
