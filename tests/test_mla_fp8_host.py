"""Host-side checks of the 8-bit latent cache's calls: what the library and the binding refuse
before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

from fp8_block_scaled_biased_b200 import binding as B
from fp8_block_scaled_biased_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


P = ctypes.c_void_p(256)          # never dereferenced: every call below is refused first
ODD = ctypes.c_void_p(8)          # not 16-byte aligned


def _call(lib, name, base, **over):
    args = dict(base)
    for k, v in over.items():
        assert k in args
        args[k] = v
    return getattr(lib, name)(*args.values()), lib.fp8moe_last_error().decode()


APPEND = dict(kv_new=P, ld=576, append_indptr=P, cache=P, scale=P, indptr=P, indices=P, last=P, batch=2, tokens=3,
              pages=4, page_size=16, n_idx=4, stream=None)
GATHER = dict(cache=P, scale=P, indptr=P, indices=P, last=P, out_indptr=P, out=P, ld=576, batch=2, rows=3, pages=4,
              page_size=16, n_idx=4, stream=None)
DECODE = dict(q=P, cache=P, scale=P, o=P, indptr=P, indices=P, last=P, lse=None, batch=2, heads=16, pages=4,
              page_size=16, n_idx=4, sm_scale=0.04, cap=0.0, ws=P, ws_bytes=1 << 40, stream=None)
EXTEND = dict(q=P, qo_indptr=P, cache=P, scale=P, o=P, indptr=P, indices=P, last=P, lse=None, batch=2, rows=3, heads=16,
              pages=4, page_size=16, n_idx=4, sm_scale=0.04, cap=0.0, ws=P, ws_bytes=1 << 40, stream=None)
ALL = [("mla_kv_append_fp8", APPEND), ("mla_kv_gather_fp8", GATHER), ("mla_decode_fp8_fwd", DECODE),
       ("mla_extend_fp8_fwd", EXTEND)]


@pytest.mark.parametrize("name,base", ALL, ids=[n for n, _ in ALL])
def test_table_and_cache_arguments(lib, name, base):
    for over, code in ((dict(batch=-1), 1), (dict(pages=-1), 1), (dict(n_idx=-1), 1), (dict(page_size=0), 1),
                       (dict(indptr=None), 1), (dict(last=None), 1), (dict(indices=None), 1), (dict(cache=None), 1),
                       (dict(scale=None), 1), (dict(pages=0), 1), (dict(cache=ODD), 1),
                       (dict(batch=(1 << 20) + 1), 2), (dict(pages=1 << 27), 2), (dict(n_idx=1 << 27), 2)):
        rc, msg = _call(lib, name, base, **over)
        assert rc == code, (over, rc, msg)
        assert name in msg
    assert _call(lib, name, base, batch=0)[0] == 0                       # nothing to do


@pytest.mark.parametrize("name,base,x,rows,ld,indptr", [
    ("mla_kv_append_fp8", APPEND, "kv_new", "tokens", "ld", "append_indptr"),
    ("mla_kv_gather_fp8", GATHER, "out", "rows", "ld", "out_indptr")])
def test_rows_of_append_and_gather(lib, name, base, x, rows, ld, indptr):
    for over, code in (({rows: -1}, 1), ({rows: (1 << 30) + 1}, 2), ({ld: 575}, 1), ({ld: 580}, 1), ({x: None}, 1),
                       ({x: ODD}, 1), ({indptr: None}, 1)):
        assert _call(lib, name, base, **over)[0] == code, over
    assert _call(lib, name, base, **{rows: 0})[0] == 0


@pytest.mark.parametrize("name,base", ALL[2:], ids=[n for n, _ in ALL[2:]])
def test_attention_arguments(lib, name, base):
    for over, code in ((dict(heads=0), 2), (dict(heads=129), 2), (dict(q=None), 1), (dict(o=None), 1), (dict(q=ODD), 1),
                       (dict(o=ODD), 1), (dict(sm_scale=0.0), 1), (dict(sm_scale=float("nan")), 1),
                       (dict(sm_scale=float("inf")), 1), (dict(cap=-1.0), 1), (dict(cap=float("inf")), 1)):
        rc, msg = _call(lib, name, base, **over)
        assert rc == code, (over, rc, msg)
    if lib.mla_fp8_workspace(16, 2):
        assert _call(lib, name, base, ws=None)[0] == 3
        assert _call(lib, name, base, ws=ODD)[0] == 3
        assert _call(lib, name, base, ws_bytes=lib.mla_fp8_workspace(16, 2) - 1)[0] == 3
    if name == "mla_extend_fp8_fwd":
        assert _call(lib, name, base, qo_indptr=None)[0] == 1
        assert _call(lib, name, base, rows=-1)[0] == 1
        assert _call(lib, name, base, rows=(1 << 22) + 1)[0] == 2
        assert _call(lib, name, base, rows=0)[0] == 0


def test_binding_refuses_host_tensors():
    cache = torch.zeros(2, 4, 1, 576, dtype=torch.float8_e4m3fn)
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(1, 576, dtype=torch.bfloat16)
    q, o = torch.zeros(1, 16, 576, dtype=torch.bfloat16), torch.zeros(1, 16, 512, dtype=torch.bfloat16)
    for call in (lambda: B.mla_kv_append_fp8(x, i, cache, torch.zeros(2, 1), i, i, i[:1]),
                 lambda: B.mla_kv_gather_fp8(cache, torch.zeros(2, 1), i, i, i[:1], i, x),
                 lambda: B.mla_decode_fp8_fwd(q, cache, torch.zeros(2, 1), o, i, i, i[:1]),
                 lambda: B.mla_extend_fp8_fwd(q, i, cache, torch.zeros(2, 1), o, i, i, i[:1])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("file", ["mla_fp8_cache.cuh", "mla_fp8_attn.cuh"])
def test_kernels_launched_early_do_not_read_through_the_read_only_path(file):
    """They are resident while the work before them still writes what they read, so memory is not
    read-only for as long as they live: no load may say that it is."""
    with open(os.path.join(build.PKG_DIR, "csrc", file)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert "griddepcontrol.wait" in code
    for words in ("__ldg", "ld.global.nc", "__ldlu", "ldg(", "__restrict__"):
        assert words not in code, words
