"""Argument rules of the paged-cache entry points, without a GPU: the C ABI returns before any
launch, the binding raises before any call."""
import ctypes

import pytest
import torch

from sink_aware_sliding_head_b200 import build as build_mod
from sink_aware_sliding_head_b200 import flint_attn as fa

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return fa.load_library()


def cache(**kw):
    d = dict(num_pages=8, page_size=16, max_pages=4, num_kv_heads=4, head_dim=128,
             cache_dtype=fa.CACHE_BF16, page_stride=0, head_stride=0, token_stride=0,
             table_stride=0)
    d.update(kw)
    return fa.PagedCacheDesc(*d.values())


def decode_params(c=None, **kw):
    d = dict(batch=2, num_q_heads=32, window=0, use_rope=1, rope_theta=1e6, rms_eps=1e-6,
             softmax_scale=0.0, dtype=fa.FLINT_BF16, fp32_out=0, reserved=0, q_stride=0,
             k_stride=0, v_stride=0)
    d.update(kw)
    return fa.DecodePagedParams(c or cache(), *d.values())


def append_params(c=None, **kw):
    d = dict(num_seqs=2, total_tokens=5, use_rope=1, rope_theta=1e6, rms_eps=1e-6,
             dtype=fa.FLINT_BF16, k_stride=0, v_stride=0)
    d.update(kw)
    return fa.PagedAppendParams(c or cache(), *d.values())


def call_decode(lib, p, ws=0x100000, ws_bytes=0, scales=(None, None), **ptr):
    a = dict(q=0x1000, k=0x1000, v=0x1000, wq=0x1000, wk=0x1000, sink=0x1000, lens=0x1000,
             table=0x1000, kp=0x1000, vp=0x1000)
    o = dict(out=0x1000, lse=0x1000)
    a.update({k: v for k, v in ptr.items() if k in a})
    o.update({k: v for k, v in ptr.items() if k in o})
    return lib.flint_attn_decode_paged(ctypes.byref(p), *a.values(), *scales, *o.values(), ws,
                                       ws_bytes, None)


def call_append(lib, p, scales=(None, None), status=0x100000, **ptr):
    a = dict(k=0x1000, v=0x1000, wk=0x1000, cu=0x1000, lens=0x1000, table=0x1000, kp=0x1000,
             vp=0x1000)
    a.update(ptr)
    return lib.flint_attn_paged_append(ctypes.byref(p), *a.values(), *scales, status, None)


BAD_CACHES = [
    (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=17), UNSUPPORTED),
    (dict(max_pages=0), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=64), UNSUPPORTED),
    (dict(cache_dtype=2), INVALID), (dict(max_pages=1 << 27), INVALID),
    (dict(page_stride=8192, head_stride=2048, token_stride=64), INVALID),
    (dict(page_stride=8192, head_stride=2048), INVALID),                # token stride 0
    (dict(page_stride=8196, head_stride=2048, token_stride=128), INVALID),
    (dict(page_stride=8200, head_stride=2048, token_stride=128, cache_dtype=1), INVALID),
    (dict(page_stride=-8192, head_stride=2048, token_stride=128), INVALID),
    (dict(page_stride=1 << 38, head_stride=2048, token_stride=128), INVALID),
    (dict(table_stride=3), INVALID), (dict(table_stride=-4), INVALID),
]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_cache_descriptors(lib, kw, code):
    c = cache(**kw)
    assert lib.flint_attn_decode_paged_workspace_bytes(ctypes.byref(decode_params(c))) == 0
    assert call_decode(lib, decode_params(c), ws_bytes=1 << 40) == code
    assert call_append(lib, append_params(c)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_q_heads=30), INVALID),
    (dict(num_q_heads=68), UNSUPPORTED),                                # G = 17
    (dict(dtype=fa.FLINT_FP32), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(rope_theta=0.0), INVALID), (dict(rope_theta=float("inf")), INVALID),
    (dict(rms_eps=-1.0), INVALID), (dict(rms_eps=float("nan")), INVALID),
    (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("inf")), INVALID),
    (dict(reserved=1), INVALID), (dict(q_stride=4095), INVALID), (dict(q_stride=4092), INVALID),
    (dict(k_stride=516), INVALID), (dict(v_stride=-512), INVALID),
    (dict(batch=1 << 25), INVALID),
])
def test_bad_decode_params(lib, kw, code):
    p = decode_params(**kw)
    assert lib.flint_attn_decode_paged_workspace_bytes(ctypes.byref(p)) == 0
    assert call_decode(lib, p, ws_bytes=1 << 40) == code


def test_bad_decode_pointers(lib):
    p = decode_params()
    n = lib.flint_attn_decode_paged_workspace_bytes(ctypes.byref(p))
    assert n > 0 and n % 256 == 0
    for name in ("q", "k", "v", "wq", "wk", "kp", "vp", "out"):
        assert call_decode(lib, p, ws_bytes=n, **{name: None}) == INVALID
        assert call_decode(lib, p, ws_bytes=n, **{name: 0x1008}) == INVALID
    for name in ("sink", "lens", "table", "lse"):
        assert call_decode(lib, p, ws_bytes=n, **{name: None}) == INVALID
        assert call_decode(lib, p, ws_bytes=n, **{name: 0x1002}) == INVALID
    assert call_decode(lib, p, ws_bytes=n, scales=(0x1000, None)) == INVALID   # bf16 cache
    e = decode_params(cache(cache_dtype=fa.CACHE_E4M3))
    assert call_decode(lib, e, ws_bytes=n, scales=(0x1002, 0x1000)) == INVALID
    assert call_decode(lib, p, ws=None, ws_bytes=n) == INVALID
    assert call_decode(lib, p, ws=0x100010, ws_bytes=n) == INVALID
    assert call_decode(lib, p, ws_bytes=n - 1) == WORKSPACE
    assert lib.flint_attn_decode_paged(None, *([None] * 15), 0, None) == INVALID


def test_workspace_serves_smaller_batches(lib):
    size = [lib.flint_attn_decode_paged_workspace_bytes(ctypes.byref(decode_params(batch=b)))
            for b in (1, 2, 100, 4000)]
    assert size == sorted(size)


@pytest.mark.parametrize("kw,code", [
    (dict(num_seqs=0), INVALID), (dict(total_tokens=-1), INVALID),
    (dict(dtype=fa.FLINT_FP32), UNSUPPORTED), (dict(dtype=-1), INVALID),
    (dict(rope_theta=-1.0), INVALID), (dict(rms_eps=float("inf")), INVALID),
    (dict(k_stride=504), INVALID), (dict(v_stride=513), INVALID),
])
def test_bad_append_params(lib, kw, code):
    assert call_append(lib, append_params(**kw)) == code


def test_bad_append_pointers(lib):
    p = append_params()
    for name in ("k", "v", "wk", "kp", "vp"):
        assert call_append(lib, p, **{name: None}) == INVALID
        assert call_append(lib, p, **{name: 0x1008}) == INVALID
    for name in ("cu", "lens", "table"):
        assert call_append(lib, p, **{name: None}) == INVALID
        assert call_append(lib, p, **{name: 0x1001}) == INVALID
    assert call_append(lib, p, status=None) == INVALID
    assert call_append(lib, p, status=0x100004) == INVALID
    assert call_append(lib, p, scales=(None, 0x1000)) == INVALID
    assert lib.flint_attn_paged_append(None, *([None] * 12)) == INVALID
    # no tokens: k and v may be null, the rest stays required, nothing is launched
    none = append_params(total_tokens=0)
    assert call_append(lib, none, k=None, v=None) == 0
    assert call_append(lib, none, k=None, v=None, kp=None) == INVALID


def test_packed_params_match_the_structures():
    """The bytes that a call packs are the ctypes structures' (and so the header's)."""
    desc = (8, 16, 4, 2, 128, 1, 8192, 4096, 256, 5)
    assert fa._PACK_APPEND(*desc, 3, 7, 1, 1e6, 1e-6, 0, 512, 520) == \
        bytes(fa.PagedAppendParams(fa.PagedCacheDesc(*desc), 3, 7, 1, 1e6, 1e-6, 0, 512, 520))
    assert fa._PACK_DECODE(*desc, 3, 32, 9, 1, 1e6, 1e-6, 0.5, 0, 1, 0, 4096, 512, 520) == \
        bytes(fa.DecodePagedParams(fa.PagedCacheDesc(*desc), 3, 32, 9, 1, 1e6, 1e-6, 0.5, 0, 1, 0,
                                   4096, 512, 520))


def test_structures_match_the_header(lib, tmp_path):
    """Sizes and offsets of the paged structures as a C compiler sees them."""
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    fields = [("flint_paged_cache_t", fa.PagedCacheDesc),
              ("flint_paged_append_params_t", fa.PagedAppendParams),
              ("flint_decode_paged_params_t", fa.DecodePagedParams)]
    body = "".join(f'printf("%zu ", offsetof({c}, {n}));' for c, s in fields for n, _ in s._fields_)
    body += "".join(f'printf("%zu ", sizeof({c}));' for c, _ in fields)
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"flint_attn.h\"\n"
                   "int main(void) {" + body + "return 0; }\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([gcc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True).stdout
    want = [getattr(s, n).offset for _, s in fields for n, _ in s._fields_]
    want += [ctypes.sizeof(s) for _, s in fields]
    assert list(map(int, got.split())) == want


def tensors(**kw):
    bf = torch.bfloat16
    t = dict(q=torch.zeros(2, 32, 128, dtype=bf), k=torch.zeros(2, 4, 128, dtype=bf),
             v=torch.zeros(2, 4, 128, dtype=bf), wq=torch.zeros(128, dtype=bf),
             wk=torch.zeros(128, dtype=bf), sink=torch.zeros(32),
             lens=torch.zeros(2, dtype=torch.int32), table=torch.zeros(2, 3, dtype=torch.int32),
             kp=torch.zeros(6, 4, 16, 128, dtype=bf), vp=torch.zeros(6, 4, 16, 128, dtype=bf),
             cu=torch.zeros(3, dtype=torch.int32))
    t.update(kw)
    return t


def decode(t, **kw):
    return fa.decode_paged(t["q"], t["k"], t["v"], t["wq"], t["wk"], t["sink"], t["lens"],
                           t["table"], t["kp"], t["vp"], 0, True, 1e6, **kw)


def append(t, **kw):
    return fa.paged_append(t["k"], t["v"], t["wk"], t["cu"], t["lens"], t["table"], t["kp"],
                           t["vp"], True, 1e6, **kw)


def test_binding_refuses_cpu_tensors(lib):
    with pytest.raises(ValueError, match="CUDA"):
        decode(tensors())
    with pytest.raises(ValueError, match="CUDA"):
        append(tensors())


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(2, 4, 128)), dict(k=torch.zeros(2, 3, 128, dtype=torch.bfloat16)),
    dict(k=torch.zeros(1, 4, 128, dtype=torch.bfloat16).expand(2, 4, 128)),
    dict(k=torch.zeros(2, 128, 4, dtype=torch.bfloat16).transpose(1, 2)),
    dict(v=torch.zeros(2, 4, 64, dtype=torch.bfloat16)),
    dict(wk=torch.zeros(128)), dict(lens=torch.zeros(2, dtype=torch.int64)),
    dict(table=torch.zeros(2, 3, dtype=torch.int64)), dict(table=torch.zeros(3, 3, dtype=torch.int32)),
    dict(table=torch.zeros(1, 3, dtype=torch.int32).expand(2, 3)),
    dict(table=torch.zeros(3, 2, dtype=torch.int32).t()),
    dict(kp=torch.zeros(6, 4, 16, 128)), dict(kp=torch.zeros(5, 4, 16, 128, dtype=torch.bfloat16)),
    dict(vp=torch.zeros(6, 16, 4, 128, dtype=torch.bfloat16).transpose(1, 2)),
    dict(kp=torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16).expand(6, 4, 16, 128),
         vp=torch.zeros(1, 1, 1, 128, dtype=torch.bfloat16).expand(6, 4, 16, 128)),
    dict(kp=torch.zeros(6, 4, 128, 16, dtype=torch.bfloat16).transpose(2, 3),
         vp=torch.zeros(6, 4, 128, 16, dtype=torch.bfloat16).transpose(2, 3)),
])
def test_binding_refuses_shapes_types_and_strides(lib, kw):
    with pytest.raises((ValueError, TypeError)):
        decode(tensors(**kw))
    with pytest.raises((ValueError, TypeError)):
        append(tensors(**kw))


def test_binding_refuses_the_rest(lib):
    for kw in (dict(q=torch.zeros(2, 32, 128)), dict(q=torch.zeros(3, 32, 128, dtype=torch.bfloat16)),
               dict(q=torch.zeros(2, 4096, dtype=torch.bfloat16)), dict(sink=torch.zeros(31)),
               dict(wq=torch.zeros(64, dtype=torch.bfloat16))):
        with pytest.raises((ValueError, TypeError)):
            decode(tensors(**kw))
    for kw in (dict(out=torch.zeros(2, 32, 128)), dict(lse=torch.zeros(32, 2)),
               dict(workspace=torch.zeros(4096)), dict(k_scale=torch.ones(4))):
        with pytest.raises((ValueError, TypeError)):
            decode(tensors(), **kw)
    for kw in (dict(cu=torch.zeros(2, dtype=torch.int32)), dict(cu=torch.zeros(3))):
        with pytest.raises((ValueError, TypeError)):
            append(tensors(**kw))
    with pytest.raises(ValueError):
        append(tensors(), status=torch.zeros(1, dtype=torch.int32))
