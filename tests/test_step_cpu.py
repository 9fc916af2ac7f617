"""A step with drafted tokens on a machine without a GPU: what include/cccl_step.h
declares is exported, its structures are the binding's, frequencies are the
formula's, and arguments are refused before anything is enqueued."""

import ctypes
import math
import os
import re
import shutil
import subprocess

import pytest
import torch

import step_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "cccl_step.h")


@pytest.fixture(scope="module")
def cc():
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    return m


def test_header_and_library_agree(cc):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(cccl_step_[a-z_]+)\s*\(", text))
    assert names == {"cccl_step_plan", "cccl_step_rotary_turns", "cccl_step_write", "cccl_step_attention",
                     "cccl_step_verify", "cccl_step_keep"}
    lib = ctypes.CDLL(cc.LIB_PATH)
    for name in names:
        assert hasattr(lib, name)
        assert name == "cccl_step_rotary_turns" or hasattr(cc, name)


def test_structures_match_the_header(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is missing")
    from compression_coupled_collectives_gb300 import step

    classes = {"cccl_step_tables": step._Tables, "cccl_step_out": step._Out, "cccl_step_rotary": step._Rotary,
               "cccl_step_draft": step._Draft}
    lines = []
    for c_name, cls in classes.items():
        lines.append('std::printf("%%zu\\n", sizeof(%s));' % c_name)
        lines += ['std::printf("%%zu\\n", offsetof(%s, %s));' % (c_name, f) for f, _ in cls._fields_]
    src = tmp_path / "layout.cpp"
    src.write_text('#include <cstddef>\n#include <cstdio>\n#include "cccl_step.h"\nint main() {\n%s\n}\n' % "\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.check_call([gxx, "-std=c++17", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    want = []
    for cls in classes.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_packed_structures_are_the_declared_ones(cc):
    from compression_coupled_collectives_gb300 import step

    for pack, cls in ((step._pack_out, step._Out), (step._pack_draft, step._Draft)):
        values = list(range(1, len(cls._fields_) + 1))
        assert pack(*values) == bytes(cls(*values))


@pytest.mark.parametrize("rot,base,factor,length,few,many", [
    (128, 1e4, 1.0, 0, 1, 32), (64, 5e5, 8.0, 8192, 1, 4), (16, 1e6, 4.0, 0, 1, 32), (96, 1e4, 16.0, 4096, 1, 32),
    (48, 0.5, 1.0, 0, 1, 32)])
def test_frequencies(cc, rot, base, factor, length, few, many):
    turns = cc.StepRotary(rot, base=base, factor=factor, original_length=length, few=few, many=many, device="cpu").turns
    for i, got in enumerate(turns.tolist()):
        f = base ** (-2.0 * i / rot)
        g = min(1.0, max(0.0, (length * f / (2 * math.pi) - few) / (many - few))) if length else 0.0
        want = (g * f + (1 - g) * f / factor) / (2 * math.pi)
        # a few roundings of binary64 in either
        off = ((got & (1 << 64) - 1) / 2.0 ** 64 - want + 0.5) % 1.0 - 0.5
        assert abs(off) <= 8 * 2.0 ** -53 * max(want, want % 1.0)


@pytest.mark.parametrize("over", [dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=-16), dict(base=0.0),
                                  dict(base=-2.0), dict(base=math.nan), dict(base=math.inf), dict(factor=0.0),
                                  dict(factor=math.inf), dict(original_length=-1.0), dict(original_length=math.nan),
                                  dict(original_length=10, few=4.0, many=4.0), dict(original_length=10, many=math.inf)])
def test_frequencies_refused(cc, over):
    kw = dict(rot_dim=64, device="cpu")
    kw.update(over)
    with pytest.raises(cc.CcclError):
        cc.StepRotary(kw.pop("rot_dim"), **kw)


def test_magnitude_refused(cc):
    with pytest.raises(ValueError):
        cc.StepRotary(64, magnitude=math.nan, device="cpu")


A, W, BIG = 0x10000, 0x80000, 1 << 40  # addresses without an allocation behind them are refused last


def refused(cc, status):
    assert status == cc.CCCL_ERR_INVALID_ARG


def test_plan_refusals(cc):
    from compression_coupled_collectives_gb300 import step

    def call(lens=A, new=A, parents=None, ws=W, size=BIG, tables=True, out=True, **over):
        t = dict(page_table=A, held=A, free_pages=A, free_count=A, table_stride=8, free_capacity=9, batch=2, table_pages=8,
                 page_tokens=16, t_reserved=0)
        o = dict(cu_tokens=A, kv_lens=A, out_held=A, out_count=A, slots=A, positions=A, mask=A, mask_stride=2, rows=10,
                 mask_words=2, o_reserved=0)
        for k, v in over.items():
            (t if k in t else o)[k] = v
        t = step._Tables(*t.values())
        o = step._Out(*o.values())
        return cc._lib.cccl_step_plan(ctypes.addressof(t) if tables else None, lens, new, parents,
                                      ctypes.addressof(o) if out else None, ws, size, None)

    for kw in (dict(tables=False), dict(out=False), dict(batch=-1), dict(batch=1025), dict(table_pages=0),
               dict(table_stride=7), dict(page_tokens=0), dict(free_capacity=0), dict(free_capacity=1 << 31),
               dict(t_reserved=1), dict(o_reserved=1), dict(rows=-1), dict(rows=1 << 31), dict(mask_words=0),
               dict(mask_words=33, mask_stride=40), dict(mask_stride=1), dict(mask=None), dict(ws=None), dict(ws=W + 8),
               dict(size=15), dict(lens=None), dict(new=A + 2), dict(page_table=A + 1), dict(cu_tokens=None),
               dict(slots=A + 4), dict(parents=A + 2), {}):
        refused(cc, call(**kw))
    assert call(batch=0) == cc.CCCL_OK


def _good(kv, **over):
    c = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, dtype=1, format=0, kv_heads=8, head_dim=128,
             page_tokens=16, reserved=0, pages=100, page_stride=16 * 1024, token_stride=1024, head_stride=128,
             scale_page_stride=0, scale_token_stride=0, scale_head_stride=0)
    b = dict(page_table=0x30000, cu_tokens=0x40000, kv_lens=0x50000, table_stride=10, n_tokens=4, batch=2,
             table_pages=10, max_new=2, max_len=160)
    for k, v in over.items():
        (c if k in c else b)[k] = v
    return kv._Cache(**c), kv._Batch(**b)


CACHES = [dict(dtype=3), dict(format=3), dict(head_dim=24), dict(batch=1025), dict(n_tokens=-1), dict(max_new=0), dict(k=None),
          dict(page_table=None), dict(kv_lens=0x50001), {}]


@pytest.mark.parametrize("over", CACHES)
def test_cache_and_batch_refusals(cc, over):
    from compression_coupled_collectives_gb300 import kv, step

    c, b = _good(kv, **over)
    r = step._Rotary(A, 1.0, 64, 0, 0)
    pc, pb, pr = ctypes.addressof(c), ctypes.addressof(b), ctypes.addressof(r)
    refused(cc, cc._lib.cccl_step_write(pc, pb, pr, None, A, 32, 4096, 128, A, 4096, 128, A, 1024, 128, A, 1024, 128, W, BIG,
                                        None))
    refused(cc, cc._lib.cccl_step_attention(pc, pb, A, 32, 4096, 128, 0.1, A, 1, 1, 0, A, 4096, 128, None, W, BIG, None))
    refused(cc, cc._lib.cccl_step_keep(pc, pb, A, A, A, W, BIG, None))


def test_write_refusals(cc):
    from compression_coupled_collectives_gb300 import kv, step

    c, b = _good(kv)
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)

    def call(turns=A, magnitude=1.0, rot_dim=64, interleaved=0, reserved=0, heads=32, rotary=True):
        r = step._Rotary(turns, magnitude, rot_dim, interleaved, reserved)
        return cc._lib.cccl_step_write(pc, pb, ctypes.addressof(r) if rotary else None, None, A, heads, 4096, 128, A, 4096,
                                       128, A, 1024, 128, A, 1024, 128, W, BIG, None)

    for kw in (dict(rotary=False), dict(magnitude=math.nan), dict(rot_dim=0), dict(rot_dim=24), dict(rot_dim=144),
               dict(interleaved=2), dict(reserved=1), dict(heads=-1), dict(heads=4097), dict(turns=None)):
        refused(cc, call(**kw))
    b.n_tokens = 0
    assert call() == cc.CCCL_OK and call(rot_dim=24) == cc.CCCL_ERR_INVALID_ARG


def test_attention_refusals(cc):
    from compression_coupled_collectives_gb300 import kv

    c, b = _good(kv)
    pc, pb = ctypes.addressof(c), ctypes.addressof(b)

    def call(heads=32, scale=0.1, mask=A, stride=2, words=2, window=0):
        return cc._lib.cccl_step_attention(pc, pb, A, heads, 4096, 128, scale, mask, stride, words, window, A, 4096, 128, None,
                                           W, BIG, None)

    for kw in (dict(heads=0), dict(heads=12), dict(scale=math.inf), dict(words=0), dict(words=3), dict(stride=1),
               dict(window=-1), dict(mask=None), dict(words=(1 << 20) + 1, stride=1 << 30)):
        refused(cc, call(**kw))
    b.n_tokens = 0
    assert call() == cc.CCCL_OK


def test_verify_refusals(cc):
    from compression_coupled_collectives_gb300 import step

    def call(path=A, kept=A, following=A, ws=W, size=BIG, draft=True, **over):
        d = dict(p=A, q=None, p_stride=100, q_stride=0, tokens=A, parents=None, uniform=A, cu_tokens=A, rows=4, batch=2,
                 vocab=100)
        d.update(over)
        d = step._Draft(*d.values())
        return cc._lib.cccl_step_verify(ctypes.addressof(d) if draft else None, path, kept, following, ws, size, None)

    for kw in (dict(draft=False), dict(batch=-1), dict(batch=1025), dict(rows=-1), dict(rows=1 << 31), dict(vocab=0),
               dict(vocab=(1 << 20) + 1, p_stride=1 << 21), dict(p_stride=99), dict(q=A, q_stride=99), dict(p=None),
               dict(tokens=None), dict(uniform=A + 2), dict(cu_tokens=None), dict(path=None), dict(kept=None),
               dict(following=A + 1), dict(ws=W + 4), dict(size=8), {}):
        refused(cc, call(**kw))
    assert call(batch=0) == cc.CCCL_OK


def test_binding_refusals(cc):
    """What a tensor is says what the call gets; the rest is refused with its name."""
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    tables = cc.StepTables(i(2, 5), i(2), i(9), i(1), page_tokens=16)
    assert (tables._c.table_stride, tables._c.table_pages, tables._c.batch, tables._c.free_capacity) == (5, 5, 2, 9)
    wide = cc.StepTables(i(4, 10)[::2, 1:4], i(2), i(9), i(1), page_tokens=16)
    assert (wide._c.table_stride, wide._c.table_pages) == (20, 3)
    with pytest.raises(ValueError):
        cc.StepTables(i(1, 5).expand(2, 5), i(2), i(9), i(1), page_tokens=16)
    for bad in ((i(2, 5).long(), i(2), i(9), i(1)), (i(2, 5), i(3), i(9), i(1)), (i(2, 5), i(2), i(9, 1), i(1)),
                (i(2, 5), i(2), i(9), i(2)), (i(2, 5), i(4)[::2], i(9), i(1))):
        with pytest.raises(TypeError):
            cc.StepTables(*bad, page_tokens=16)
    with pytest.raises(ValueError, match="rows"):
        cc.cccl_step_plan(tables, i(2), i(2), i(4), cu_tokens=i(3), kv_lens=i(2))
    with pytest.raises(TypeError, match="mask"):
        cc.cccl_step_plan(tables, i(2), i(2), i(4), cu_tokens=i(3), kv_lens=i(2), mask=i(7), rows=7)
    with pytest.raises(TypeError, match="slots"):
        cc.cccl_step_plan(tables, i(2), i(2), i(4), cu_tokens=i(3), kv_lens=i(2), slots=i(7))
    with pytest.raises(TypeError, match="p:"):
        cc.cccl_step_verify(torch.zeros(4, 9).double(), None, i(4), None, torch.zeros(4), i(3), i(4), i(2), i(2), i(4))
    with pytest.raises(TypeError, match="q:"):
        cc.cccl_step_verify(torch.zeros(4, 9), torch.zeros(4, 8), i(4), None, torch.zeros(4), i(3), i(4), i(2), i(2), i(4))
    with pytest.raises(TypeError, match="cu_tokens"):
        cc.cccl_step_verify(torch.zeros(4, 9), None, i(4), None, torch.zeros(4), i(4), i(4), i(2), i(2), i(4))
    with pytest.raises(ValueError, match="CUDA"):
        cc.cccl_step_verify(torch.zeros(4, 9), None, i(4), None, torch.zeros(4), i(3), i(4), i(2), i(2), i(4))


# ------------------------------------------------------------------ the reference itself
def test_reference_of_verification_keeps_what_the_target_would_say():
    """Against the definition for a chain: u q < p keeps, the residual max(p - q, 0) is drawn from after a refusal."""
    p, q = [[0.5, 0.25, 0.25], [0.125, 0.375, 0.5]], [[0.25, 0.5, 0.25], [0.5, 0.25, 0.25]]
    got = ref.verify(p, q, [9, 1], [-1, 0], [0.3, 0.49], [0, 2])  # 0.49 * 0.5 < 0.25: kept
    assert got == ([0, 1], [2], [1])  # 0.125 <= 0.3 < 0.5 of row 1
    got = ref.verify(p, q, [9, 1], [-1, 0], [0.3, 0.51], [0, 2])
    assert got == ([0, -1], [1], [0])  # only token 0 has more of p than of q
    got = ref.verify(p, None, [9, 0, 2], [-1, 0, 0], [0.7, 0.6, 0.9], [0, 3][:1] + [3])
    # 0.6 >= 0.5: refused; 0.9 (1 - 0.5) >= 0.25: refused; what is left of the root's row is token 1
    assert got == ([0, -1, -1], [1], [1])


def test_reference_of_masks_and_plans():
    assert ref.ancestors([-1, 0, 0, 1]) == [1, 3, 5, 11] and ref.depths([-1, 0, 0, 1]) == [0, 1, 1, 2]
    got = ref.plan([3, 0], [2, 4], [1, 0], [[8, 0], [0, 0]], [4, 5, 6], 3, 4, None, 6, 2, 1)
    assert got["table"] == [[8, 6], [5, 0]] and got["free_count"] == [1] and got["slots"] == [35, 24, 20, 21, 22, 23]
