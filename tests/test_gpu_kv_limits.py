"""The chunk kernel's bounded waits: a build whose limit is zero gives up at
the first wait that is not over when it begins, in every role.  The call then reports a timeout and
nothing else: no write outside the results, whatever the workspace held, and
the device stays usable."""

import ctypes
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


@pytest.fixture(scope="module")
def impatient(cc, tmp_path_factory):
    """The library with the chunk kernel's source compiled for a limit of zero."""
    from compression_coupled_collectives_gb300 import build as b

    objects = [os.path.join(b.HERE, "_build", s.replace(".cu", ".o")) for s in b.SOURCES if s != "cccl_kv_chunk.cu"]
    if not all(os.path.exists(o) for o in objects):
        b.build(force=True)
    out = tmp_path_factory.mktemp("impatient")
    obj, lib = str(out / "chunk.o"), str(out / "libcccl_impatient.so")
    subprocess.check_call([b._nvcc(), *b.ARCH, *b.FLAGS, "-DCCCL_WAIT_LIMIT_NS=0ull", "-c",
                           os.path.join(b.CSRC, "cccl_kv_chunk.cu"), "-o", obj])
    subprocess.check_call([b._nvcc(), *b.ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-Bsymbolic", "-o", lib, obj,
                           *objects])
    handle = ctypes.CDLL(lib)
    handle.cccl_kv_attention.argtypes = cc._lib.cccl_kv_attention.argtypes
    handle.cccl_kv_attention.restype = ctypes.c_int
    return handle


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
        status = impatient.cccl_kv_attention(cache._ref, batch._ref, c.q.data_ptr(), heads, heads * c.dim, c.dim, 0.1, 1, 0,
                                             out.data_ptr(), heads * c.dim, c.dim, lse[guard:-guard].data_ptr(),
                                             ws.data_ptr(), ws.nbytes, torch.cuda.current_stream().cuda_stream)
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
