"""The binding of a step with drafted tokens on a machine without a GPU: what is
refused before the library is called, and how exact the frequencies are."""

from decimal import Decimal, getcontext

import pytest
import torch


@pytest.fixture(scope="module")
def cc():
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    return m


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


def test_a_workspace_on_another_device_is_refused(cc):
    """In every call: a report into it would go through another device's address."""
    ws = torch.zeros(64, dtype=torch.uint8).as_subclass(Elsewhere)
    tables = cc.StepTables(ints(2, 5), ints(2), ints(9), ints(1), page_tokens=16)
    cache = cc.KvCache.empty(4, 16, 2, 64, device="cpu")
    batch = cc.KvBatch(ints(2, 5), ints(3), ints(2), n_tokens=4, max_new=2, max_len=9)
    rotary = cc.StepRotary(64, device="cpu")
    q, kv = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    p = torch.zeros(4, 9)
    for call in (lambda: cc.cccl_step_plan(tables, ints(2), ints(2), ws, cu_tokens=ints(3), kv_lens=ints(2), rows=4),
                 lambda: cc.cccl_step_write(cache, batch, rotary, q, kv, kv, q, ws),
                 lambda: cc.cccl_step_attention(cache, batch, q, ints(4, 1), q, ws),
                 lambda: cc.cccl_step_verify(p, None, ints(4), None, torch.zeros(4), ints(3), ints(4), ints(2), ints(2), ws),
                 lambda: cc.cccl_step_keep(cache, batch, ints(4), ints(2), None, ws)):
        with pytest.raises(ValueError, match="ws is on another device|on the cache's device"):
            call()


def exact_turns(rot, base, factor, length, few, many):
    """Turns a position of every pair, to 60 digits, modulo whole ones."""
    getcontext().prec = 70
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")
    d = lambda x: Decimal(x)  # noqa: E731  (a float's value, exactly)
    out = []
    for i in range(rot // 2):
        f = (d(base).ln() * Decimal(-2 * i) / Decimal(rot)).exp()
        stay = Decimal(0)
        if length:
            stay = min(Decimal(1), max(Decimal(0), (d(length) * f / two_pi - d(few)) / (d(many) - d(few))))
        out.append((stay * f + (1 - stay) * f / d(factor)) / two_pi % 1)
    return out


@pytest.mark.parametrize("rot,base,factor,length,few,many", [
    (128, 1e4, 1.0, 0, 1, 32), (128, 5e5, 1.0, 0, 1, 32), (64, 5e5, 8.0, 8192, 1, 4), (96, 1e6, 4.0, 4096, 1, 32),
    (128, 1e4, 40.0, 4096, 1, 32), (48, 12345.678, 1.7, 0, 1, 32), (128, 1e300, 1.0, 0, 1, 32), (112, 1.0, 3.0, 0, 1, 32)])
def test_how_exact_frequencies_are(cc, rot, base, factor, length, few, many):
    """Against arithmetic of 70 digits.  In binary64, with e = 2^-53 and f = exp(-y): the exponent's rounding enters as
    f y e, at most 0.37 e; the power is off by 2 e f; a mixing weight by 4 e many / (many - few) + 2 e, at most 8 e with
    many >= 4/3 few; the products, the quotient, the difference, the sum and the division by a rounded 2 pi by 7 e f.
    So a turn, f / (2 pi), is off by less than 17.4 e / (2 pi) < 2^-51.  (Few of these errors meet: the usual bases
    keep to 2^-55, which is what is documented for them.)"""
    turns = cc.StepRotary(rot, base=base, factor=factor, original_length=length, few=few, many=many, device="cpu").turns
    worst = Decimal(0)
    for got, want in zip(turns.tolist(), exact_turns(rot, base, factor, length, few, many)):
        off = abs(Decimal(got & (1 << 64) - 1) / Decimal(1 << 64) - want)
        worst = max(worst, min(off, 1 - off))
    assert worst < Decimal(2) ** (-55 if base <= 1e6 else -51)
