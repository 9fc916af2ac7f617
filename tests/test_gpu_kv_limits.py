"""The chunk kernel's bounded waits.  A build whose limit is zero gives up at the
first wait that is not over when it begins, in every role: the call then reports
a timeout and nothing else, with no write outside the results, whatever the
workspace held, and the device stays usable.  A build whose limit is 2 ms, some
twenty times what any wait takes, works out rows of NaN that take far longer:
nothing waits for them."""

import ctypes
import math
import os
import subprocess

import pytest
import torch

from kv_reference import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    torch.cuda.set_device(0)
    return m


def with_limit(cc, out, limit_ns):
    """The library with the chunk kernel's source compiled for another limit."""
    from compression_coupled_collectives_gb300 import build as b

    objects = [os.path.join(b.HERE, "_build", s.replace(".cu", ".o")) for s in b.SOURCES if s != "cccl_kv_chunk.cu"]
    if not all(os.path.exists(o) for o in objects):
        b.build(force=True)
    obj, lib = str(out / "chunk.o"), str(out / "libcccl_limit.so")
    subprocess.check_call([b._nvcc(), *b.ARCH, *b.FLAGS, "-DCCCL_WAIT_LIMIT_NS=%dull" % limit_ns, "-c",
                           os.path.join(b.CSRC, "cccl_kv_chunk.cu"), "-o", obj])
    subprocess.check_call([b._nvcc(), *b.ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-Bsymbolic", "-o", lib, obj,
                           *objects])
    handle = ctypes.CDLL(lib)
    handle.cccl_kv_attention.argtypes = cc._lib.cccl_kv_attention.argtypes
    handle.cccl_kv_attention.restype = ctypes.c_int
    return handle


@pytest.fixture(scope="module")
def impatient(cc, tmp_path_factory):
    return with_limit(cc, tmp_path_factory.mktemp("zero"), 0)


@pytest.fixture(scope="module")
def brisk(cc, tmp_path_factory):
    return with_limit(cc, tmp_path_factory.mktemp("brisk"), 2000000)


def attend(lib, cache, batch, q, out, lse, ws, scale):
    _, heads, dim = q.shape
    return lib.cccl_kv_attention(cache._ref, batch._ref, q.data_ptr(), heads, heads * dim, dim, scale, 1, 0, out.data_ptr(),
                                 heads * dim, dim, lse.data_ptr(), ws.data_ptr(), ws.nbytes,
                                 torch.cuda.current_stream().cuda_stream)


CALLS = {
    # lens, new, what the program says: several pieces a block with cut items, whole ones, clusters
    "cut": ([300 + 7 * b for b in range(200)], 64, dict(max_len=1 << 20)),
    "whole": ([300 + 7 * b for b in range(100)], 64, {}),
    "clusters": ([1500], 64, {}),
}


@pytest.mark.parametrize("page", [16, 24])  # by TMA boxes, by asynchronous copies
@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("how", sorted(CALLS))
def test_giving_up_is_an_error_and_no_more(cc, impatient, how, fmt, page):
    lens, new, over = CALLS[how]
    c = Case(lens, [new] * len(lens), heads=8, group=4, dim=128, page=page, fmt=fmt, seed=70)
    cache, batch = c.objects(cc, **over)
    heads = c.heads * c.group
    ws = cc.empty_kv_workspace(cache, batch, heads)
    guard = 64
    for junk in (0xFF, 0x7F):
        ws[16:] = junk
        cc.cccl_kv_clear_status(ws)
        frame = torch.full((c.T + 2 * guard, heads, c.dim), 3.0, dtype=c.dtype, device="cuda")
        lse = torch.full((c.T + 2 * guard, heads), 3.0, device="cuda")
        out = frame[guard:-guard]
        status = attend(impatient, cache, batch, c.q, out, lse[guard:-guard], ws, 0.1)
        assert status == cc.CCCL_OK
        torch.cuda.synchronize()
        assert cc.cccl_get_result(ws)[1] == 4  # CCCL_ERR_TIMEOUT
        for t in (frame, lse):
            assert (t[:guard] == 3.0).all() and (t[-guard:] == 3.0).all()
    cc.cccl_kv_clear_status(ws)
    out = torch.empty_like(c.q)
    cc.cccl_kv_attention(cache, batch, c.q, out, ws)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK
    assert torch.equal(out, cc.kv_attention(cache, batch, c.q)[0])


@pytest.mark.parametrize("how,length,count", [("whole", 2500, 6), ("cut", 6000, 2), ("clusters", 3000, 1)])
@pytest.mark.parametrize("fmt,value", [("int8", math.nan), ("16bit", math.inf)])
def test_no_wait_spans_rows_that_are_not_finite(cc, brisk, fmt, value, how, length, count):
    """One vector of head 0 is not finite: rows that see it say so, all others are as if it were not there."""
    new = 640 if how != "clusters" else 64
    c = Case([length] * count, [new] * count, heads=8, group=4, dim=128, page=16, fmt=fmt, seed=71)
    ref, ref_lse, tol, ltol = c.attention()
    bad = length - new + new // 2  # seen by the second half of the rows
    for b in range(count):
        at = (int(c.table[b, bad // 16]), bad % 16)
        if fmt == "16bit":
            c.v[at][0, 7] = value
        else:
            c.vs[at][0] = value
    cache, batch = c.objects(cc, **(dict(max_len=1 << 20) if how == "cut" else {}))
    ws = cc.empty_kv_workspace(cache, batch, 32)
    out, lse = torch.full_like(c.q, 9.0), torch.full((c.T, 32), 9.0, device="cuda")
    assert attend(brisk, cache, batch, c.q, out, lse, ws, 128 ** -0.5) == cc.CCCL_OK
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK
    sees = (torch.arange(c.T, device="cuda") % new >= new // 2)[:, None, None].expand(-1, 32, 128).clone()
    sees[:, 4:] = False
    if fmt == "16bit":
        sees[..., :7] = sees[..., 8:] = False
        assert (out[sees] == math.inf).all()
    else:
        assert out[sees].isnan().all()
    assert ((out.double() - ref).abs() <= tol)[~sees].all()
    assert ((lse.double() - ref_lse).abs() <= ltol).all()  # the values have no part in it
