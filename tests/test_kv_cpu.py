"""The paged cache's boundary on a machine without a GPU: what include/cccl_kv.h
declares is exported, its structures are the binding's, and arguments are
refused before anything is enqueued."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cccl_kv.h")


@pytest.fixture(scope="module")
def cc():
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    return m


def test_header_and_library_agree(cc):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(cccl_kv_[a-z_]+)\s*\(", text))
    assert names == {"cccl_kv_clear_status", "cccl_kv_workspace_bytes", "cccl_kv_write", "cccl_kv_read",
                     "cccl_kv_attention"}
    lib = ctypes.CDLL(cc.LIB_PATH)
    for name in names:
        assert hasattr(lib, name) and hasattr(cc, name), name


def test_structures_match_the_header(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is missing")
    from compression_coupled_collectives_gb300 import kv

    lines = []
    for c_name, cls in (("cccl_kv_cache", kv._Cache), ("cccl_kv_batch", kv._Batch)):
        lines.append('std::printf("%%zu\\n", sizeof(%s));' % c_name)
        lines += ['std::printf("%%zu\\n", offsetof(%s, %s));' % (c_name, f) for f, _ in cls._fields_]
    src = tmp_path / "layout.cpp"
    src.write_text('#include <cstddef>\n#include <cstdio>\n#include "cccl_kv.h"\nint main() {\n%s\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.check_call([gxx, "-std=c++17", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for cls in (kv._Cache, kv._Batch):
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def _good(kv, **over):
    c = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, dtype=1, format=0, kv_heads=8, head_dim=128,
             page_tokens=16, reserved=0, pages=100, page_stride=16 * 1024, token_stride=1024, head_stride=128,
             scale_page_stride=0, scale_token_stride=0, scale_head_stride=0)
    b = dict(page_table=0x30000, cu_tokens=0x40000, kv_lens=0x50000, table_stride=10, n_tokens=4, batch=2,
             table_pages=10, max_new=2, max_len=160)
    for k, v in over.items():
        (c if k in c else b)[k] = v
    return kv._Cache(**c), kv._Batch(**b)


BAD = [dict(dtype=3), dict(dtype=0), dict(format=3), dict(kv_heads=0), dict(kv_heads=4097), dict(head_dim=24),
       dict(head_dim=144), dict(head_dim=0), dict(page_tokens=0), dict(pages=0), dict(reserved=1), dict(batch=-1),
       dict(batch=1025), dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(table_pages=0), dict(table_stride=9),
       dict(max_new=0), dict(max_len=0)]
# found after the sizes: a workspace size is still given
BAD_MEMORY = [dict(k=None), dict(v=0x20008), dict(page_stride=-8), dict(token_stride=1020), dict(head_stride=4),
              dict(page_stride=1 << 50), dict(format=1), dict(page_table=None), dict(page_table=0x30002),
              dict(cu_tokens=0x40001), dict(kv_lens=None), {}]  # {}: addresses without an allocation behind them


@pytest.mark.parametrize("over", BAD + BAD_MEMORY)
def test_refusals(cc, over):
    from compression_coupled_collectives_gb300 import kv

    lib = cc._lib
    c, b = _good(kv, **over)
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)
    need = lib.cccl_kv_workspace_bytes(pc, pb, 32)
    assert (need == 0) == (over in BAD)
    X, W, big = 0x60000, 0x80000, 1 << 40
    for f in (lib.cccl_kv_write, lib.cccl_kv_read):
        assert f(pc, pb, X, 1024, 128, X, 1024, 128, W, big, None) == cc.CCCL_ERR_INVALID_ARG
    assert lib.cccl_kv_attention(pc, pb, X, 32, 4096, 128, 0.1, 1, 0, X, 4096, 128, None, W, big, None) == \
        cc.CCCL_ERR_INVALID_ARG


def test_attention_refusals(cc):
    from compression_coupled_collectives_gb300 import kv

    lib = cc._lib
    c, b = _good(kv)
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)
    X, W, big = 0x60000, 0x80000, 1 << 40
    nan, inf = float("nan"), float("inf")

    def call(heads=32, scale=0.1, causal=1, window=0, cache=pc, batch=pb):
        return lib.cccl_kv_attention(cache, batch, X, heads, 4096, 128, scale, causal, window, X, 4096, 128, None, W,
                                     big, None)

    for kw in (dict(heads=0), dict(heads=12), dict(heads=8192), dict(scale=nan), dict(scale=inf), dict(causal=2),
               dict(window=-1), dict(cache=None), dict(batch=None)):
        assert call(**kw) == cc.CCCL_ERR_INVALID_ARG
    assert lib.cccl_kv_workspace_bytes(pc, pb, 12) == 0
    assert lib.cccl_kv_workspace_bytes(pc, pb, -1) == 0
    assert lib.cccl_kv_workspace_bytes(pc, pb, 0) == 16
    assert lib.cccl_kv_clear_status(None, 16, None) == cc.CCCL_ERR_INVALID_ARG
    assert lib.cccl_kv_clear_status(W + 8, 16, None) == cc.CCCL_ERR_INVALID_ARG
    assert lib.cccl_kv_clear_status(W, 8, None) == cc.CCCL_ERR_INVALID_ARG


def test_empty_batches_are_no_ops(cc):
    from compression_coupled_collectives_gb300 import kv

    for over in (dict(n_tokens=0), dict(batch=0)):
        c, b = _good(kv, **over)
        pc, pb = ctypes.addressof(c), ctypes.addressof(b)
        assert cc._lib.cccl_kv_write(pc, pb, None, 0, 0, None, 0, 0, None, 0, None) == cc.CCCL_OK
        assert cc._lib.cccl_kv_attention(pc, pb, None, 32, 0, 0, 0.1, 1, 0, None, 0, 0, None, None, 0, None) == cc.CCCL_OK


def test_binding_refusals(cc):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 16, 2)
    cc.KvCache(k, k.clone())
    cc.KvCache(codes, codes.clone(), scales, scales.clone(), dtype=torch.float16, fmt=cc.CCCL_KV_INT8)
    with pytest.raises(TypeError):
        cc.KvCache(k.float(), k.float())
    with pytest.raises(TypeError):
        cc.KvCache(k, k.half())
    with pytest.raises(ValueError):
        cc.KvCache(k, k.clone(), scales, scales)
    with pytest.raises(ValueError):
        cc.KvCache(k, torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16).transpose(1, 2))
    with pytest.raises(ValueError):
        cc.KvCache(k.transpose(2, 3), k.transpose(2, 3))
    with pytest.raises(ValueError):
        cc.KvCache(codes, codes, scales, None, dtype=torch.float16, fmt=cc.CCCL_KV_INT8)
    with pytest.raises(ValueError):
        cc.KvCache(codes, codes, scales, scales[:, :8], dtype=torch.float16, fmt=cc.CCCL_KV_E4M3)
    with pytest.raises(TypeError):
        cc.KvCache(k, k, scales, scales, fmt=cc.CCCL_KV_INT8)
    with pytest.raises(ValueError):
        cc.KvCache(codes, codes, dtype=torch.float16, fmt=7)
    table, cu, lens = (torch.zeros(s, dtype=torch.int32) for s in ((2, 5), 3, 2))
    batch = cc.KvBatch(table, cu, lens, n_tokens=3, max_new=2, max_len=80)
    with pytest.raises(TypeError):
        cc.KvBatch(table.long(), cu, lens, n_tokens=3, max_new=2, max_len=80)
    with pytest.raises(TypeError):
        cc.KvBatch(table.t().contiguous().t(), cu, lens, n_tokens=3, max_new=2, max_len=80)
    with pytest.raises(ValueError):
        cc.KvBatch(table, cu[:2], lens, n_tokens=3, max_new=2, max_len=80)
    cache = cc.KvCache(k, k.clone())
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(TypeError):
        cc.cccl_kv_write(cache, batch, x.half(), x, ws)
    with pytest.raises(ValueError):
        cc.cccl_kv_write(cache, batch, x, x[:2], ws)
    with pytest.raises(ValueError):
        cc.cccl_kv_read(cache, batch, x[:, :1], x, ws)
    with pytest.raises(ValueError):
        cc.cccl_kv_attention(cache, batch, x, x[:, :1], ws)
    with pytest.raises(ValueError):
        cc.cccl_kv_attention(cache, batch, x, x, ws, lse=torch.zeros(3, 2, dtype=torch.float64))
