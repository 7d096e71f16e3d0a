"""The key-value cache's entry points on a machine without a GPU: the argument
structs against the header, what the calls refuse before any device work, and
the workspace query."""
import ctypes as C
import os
import re
import shutil
import subprocess

import pytest
import torch

from nvfp4_block_scaled_06_gb300 import _binding as B
from nvfp4_block_scaled_06_gb300 import build as builder

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096                     # an aligned stand-in pointer, never dereferenced


@pytest.fixture(scope="module")
def clib():
    builder.build()
    return B.load()


MIRRORS = {"nvfp4_kv_pages": B.KvPages, "nvfp4_kv_write_args": B.KvWriteArgs, "nvfp4_kv_read_args": B.KvReadArgs,
           "nvfp4_kv_attention_args": B.KvAttentionArgs}


def test_structs_mirror_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    header = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "nvfp4.h")).read(), flags=re.S)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "nvfp4.h"', "int main(void) {"]
    for name, cls in MIRRORS.items():
        body = re.search(r"typedef struct\s*\{([^{}]*)\}\s*" + name + r"\s*;", header).group(1)
        fields = [re.findall(r"\w+", part)[-1] for decl in body.split(";") if decl.strip() for part in decl.split(",")]
        assert fields == [f for f, _ in cls._fields_], name
        lines.append(f'  printf("%zu\\n", sizeof({name}));')
        lines += [f'  printf("%zu\\n", offsetof({name}, {f}));' for f in fields]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in MIRRORS.values():
        want += [C.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def pages(**kw):
    base = dict(k_codes=P, k_sf=P, v_codes=P, v_sf=P, num_pages=10, num_kv_heads=2, page_size=16, head_dim=64,
                codes_page_stride=2 * 16 * 32, sf_page_stride=2 * 16 * 4)
    base.update(kw)
    return B.KvPages(**base)


def write(clib, cache=None, **kw):
    base = dict(k_global_scale=P, v_global_scale=P, num_tokens=3, k=P, v=P, k_ld=128, k_head_ld=64, v_ld=128,
                v_head_ld=64, slots=P)
    base.update(kw)
    return clib.nvfp4_kv_write(C.byref(B.KvWriteArgs(cache=pages(**(cache or {})), **base)), None)


def read(clib, cache=None, **kw):
    base = dict(k_global_scale=P, v_global_scale=P, num_tokens=3, k=P, v=P, k_ld=128, k_head_ld=64, v_ld=128,
                v_head_ld=64, slots=P, out_dtype=B.OUT_BF16)
    base.update(kw)
    return clib.nvfp4_kv_read(C.byref(B.KvReadArgs(cache=pages(**(cache or {})), **base)), None)


def attend_args(cache=None, **kw):
    base = dict(k_global_scale=P, v_global_scale=P, total_q=4, num_heads=4, num_seqs=4, q=P, q_ld=256, q_head_ld=64,
                max_q_len=1, page_table=P, table_ld=8, max_pages=8, kv_lens=P, scale=0.125, causal=1, out=P,
                out_ld=256, out_head_ld=64, workspace=P, workspace_bytes=1 << 40)
    base.update(kw)
    return B.KvAttentionArgs(cache=pages(**(cache or {})), **base)


def attend(clib, cache=None, **kw):
    return clib.nvfp4_kv_attention(C.byref(attend_args(cache, **kw)), None)


REFUSED = (B.ERR_INVALID_ARG, B.ERR_UNSUPPORTED_SHAPE, B.ERR_ALIGNMENT, B.ERR_WORKSPACE)

CACHE_FAULTS = [
    (dict(k_codes=0), B.ERR_INVALID_ARG), (dict(v_sf=0), B.ERR_INVALID_ARG), (dict(num_pages=0), B.ERR_INVALID_ARG),
    (dict(num_kv_heads=0), B.ERR_INVALID_ARG), (dict(page_size=0), B.ERR_INVALID_ARG),
    (dict(head_dim=0), B.ERR_INVALID_ARG), (dict(head_dim=96), B.ERR_UNSUPPORTED_SHAPE),
    (dict(head_dim=256), B.ERR_UNSUPPORTED_SHAPE), (dict(page_size=8), B.ERR_UNSUPPORTED_SHAPE),
    (dict(page_size=24), B.ERR_UNSUPPORTED_SHAPE), (dict(page_size=2048), B.ERR_UNSUPPORTED_SHAPE),
    (dict(num_pages=1 << 31), B.ERR_UNSUPPORTED_SHAPE), (dict(codes_page_stride=1008), B.ERR_INVALID_ARG),
    (dict(sf_page_stride=112), B.ERR_INVALID_ARG), (dict(codes_page_stride=1032), B.ERR_ALIGNMENT),
    (dict(sf_page_stride=136), B.ERR_ALIGNMENT), (dict(k_codes=P + 8), B.ERR_ALIGNMENT),
    (dict(v_sf=P + 4), B.ERR_ALIGNMENT),
]


@pytest.mark.parametrize("fault,status", CACHE_FAULTS)
def test_bad_caches(clib, fault, status):
    for call in (write, read, attend):
        assert call(clib) not in REFUSED                     # (then no device)
        assert call(clib, fault) == status, call.__name__


@pytest.mark.parametrize("call", [write, read])
def test_bad_copies(clib, call):
    fn = {write: clib.nvfp4_kv_write, read: clib.nvfp4_kv_read}[call]
    cls = {write: B.KvWriteArgs, read: B.KvReadArgs}[call]
    assert fn(C.cast(None, C.POINTER(cls)), None) == B.ERR_INVALID_ARG
    for name in ("k", "v", "slots", "k_global_scale", "v_global_scale"):
        assert call(clib, **{name: 0}) == B.ERR_INVALID_ARG, name
    assert call(clib, num_tokens=0) == B.ERR_INVALID_ARG
    assert call(clib, num_tokens=-1) == B.ERR_INVALID_ARG
    assert call(clib, num_tokens=1 << 31) == B.ERR_UNSUPPORTED_SHAPE
    assert call(clib, k_ld=127) == B.ERR_INVALID_ARG          # rows overlap
    assert call(clib, v_head_ld=32) == B.ERR_INVALID_ARG
    assert call(clib, k_ld=132) == B.ERR_ALIGNMENT
    assert call(clib, v_ld=140, v_head_ld=68) == B.ERR_ALIGNMENT
    assert call(clib, k=P + 8) == B.ERR_ALIGNMENT
    assert call(clib, slots=P + 4) == B.ERR_ALIGNMENT
    if call is read:
        assert call(clib, out_dtype=2) == B.ERR_INVALID_ARG
        assert call(clib, out_dtype=B.OUT_FP32, k_ld=132) not in REFUSED     # 16-byte rows of fp32


def test_bad_attention(clib):
    assert clib.nvfp4_kv_attention(C.cast(None, C.POINTER(B.KvAttentionArgs)), None) == B.ERR_INVALID_ARG
    for name in ("q", "out", "page_table", "kv_lens", "k_global_scale", "v_global_scale", "total_q", "num_heads",
                 "num_seqs", "max_pages", "max_q_len"):
        assert attend(clib, **{name: 0}) == B.ERR_INVALID_ARG, name
    assert attend(clib, total_q=5) == B.ERR_INVALID_ARG       # without offsets: a query per sequence
    assert attend(clib, total_q=5, q_offsets=P, max_q_len=2) not in REFUSED
    assert attend(clib, table_ld=7) == B.ERR_INVALID_ARG
    assert attend(clib, window=-1) == B.ERR_INVALID_ARG
    assert attend(clib, window=4, causal=0) == B.ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attend(clib, scale=scale) == B.ERR_INVALID_ARG, scale
    assert attend(clib, q_ld=192) == B.ERR_INVALID_ARG        # rows overlap
    assert attend(clib, out_head_ld=0) == B.ERR_INVALID_ARG
    assert attend(clib, num_heads=3, q_ld=192, out_ld=192) == B.ERR_UNSUPPORTED_SHAPE   # not a multiple of kv heads
    assert attend(clib, total_q=1 << 31, num_seqs=1 << 31) == B.ERR_UNSUPPORTED_SHAPE
    assert attend(clib, max_pages=1 << 31, table_ld=1 << 31) == B.ERR_UNSUPPORTED_SHAPE
    for name, value in (("q", P + 8), ("out", P + 2), ("q_ld", 260), ("out_ld", 260), ("page_table", P + 2),
                        ("kv_lens", P + 1), ("lse", P + 2), ("k_global_scale", P + 2)):
        assert attend(clib, **{name: value}) == B.ERR_ALIGNMENT, name
    assert attend(clib, workspace=0) == B.ERR_WORKSPACE
    assert attend(clib, workspace=P + 128) == B.ERR_WORKSPACE
    need = clib.nvfp4_kv_attention_workspace_size(C.byref(attend_args()))
    assert need > 0 and attend(clib, workspace_bytes=need) not in REFUSED
    assert attend(clib, workspace_bytes=need - 1) == B.ERR_WORKSPACE


def test_workspace_query(clib):
    q = clib.nvfp4_kv_attention_workspace_size
    assert q(C.cast(None, C.POINTER(B.KvAttentionArgs))) == 0
    for name in ("total_q", "num_heads", "num_seqs", "max_q_len"):
        for v in (0, -5):
            assert q(C.byref(attend_args(**{name: v}))) == 0, name
    for name in ("num_kv_heads", "head_dim"):
        assert q(C.byref(attend_args({name: 0}))) == 0
    assert q(C.byref(attend_args(dict(num_kv_heads=8)))) > 0   # (fewer query heads: the call refuses)
    # it does not depend on the lengths of the contexts
    assert q(C.byref(attend_args())) == q(C.byref(attend_args(max_pages=1 << 20, table_ld=1 << 20)))


def test_binding_takes_cuda_tensors_only():
    import nvfp4_block_scaled_06_gb300 as nv
    cache = nv.nvfp4_kv_cache(2, 1, 16, 64, device="cpu")
    assert cache["k_codes"].shape == (2, 1, 16, 32) and cache["v_sf"].shape == (2, 1, 16, 4)
    g, x = torch.ones(1), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_write(x, x, torch.zeros(1, dtype=torch.int64), cache, g, g)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_read(torch.zeros(1, dtype=torch.int64), cache, g, g)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_attention(x, cache, g, g, torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
