"""The table of a rotation against frequencies of fifty digits that share nothing with
it: roots taken by repeated square roots, and pi by Machin's formula."""
from decimal import Decimal, localcontext

import pytest
import torch


@pytest.fixture(scope="module")
def cake():
    import __graft_entry__
    __graft_entry__.build()
    import bwd_dw_column_gb300 as cake
    return cake


def two_pi():
    """16 arctan(1/5) - 4 arctan(1/239) is pi; in whole numbers of 10^-70."""
    one = 10 ** 70

    def arctan_of_inverse(n):
        total, term, k = 0, one // n, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return Decimal(2 * (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239))) / Decimal(one)


def ladder(base, n):
    """base^(-i / n), n a power of two."""
    step = 1 / Decimal(base)
    for _ in range(n.bit_length() - 1):
        step = step.sqrt()
    return [step ** i for i in range(n)]


def off(turns, freqs):
    """How far each entry is from the frequency's share of a turn, in units of 2^-64 turn."""
    out = []
    for t, f in zip(turns.tolist(), freqs):
        d = (f / two_pi() * 2 ** 64 - t) % 2 ** 64
        out.append(float(min(d, 2 ** 64 - d)))
    return out


@pytest.mark.parametrize("sections,base", [((64,), 10000.0), ((128,), 500000.0), ((8, 16, 32), 100.0), ((1,), 10000.0),
                                           ((2, 256), 1e6), ((16,), 0.5)])
def test_entries_are_good_to_half_a_unit(cake, sections, base):
    with localcontext() as c:
        c.prec = 60
        turns, axes = cake.cake_rotary_table(sections, base, device="cpu")
        freqs = [f for n in sections for f in ladder(base, n)]
        assert turns.dtype == torch.int64 and axes.tolist() == [a for a, n in enumerate(sections) for _ in range(n)]
        assert max(off(turns, freqs)) <= 0.5 + 1e-9
        # far positions: the product takes nothing away, so the angle is off by the position times half a unit at most
        far = 2 ** 40
        for t, f in zip(turns.tolist(), freqs):
            d = (f / two_pi() * far - Decimal(t * far % 2 ** 64) / 2 ** 64) % 1
            assert min(d, 1 - d) <= Decimal(far) / 2 ** 65 * (1 + Decimal("1e-9"))


def test_a_shared_ladder_and_given_frequencies(cake):
    with localcontext() as c:
        c.prec = 60
        turns, _ = cake.cake_rotary_table((24, 20, 20), 10000.0, shared=True, device="cpu")
        assert max(off(turns, ladder(10000.0, 64))) <= 0.5 + 1e-9
        given = [1.0, 0.1, -0.25, 1e-8, 7.5, 1e9 + 0.5, -1e25, -0.0]
        turns, _ = cake.cake_rotary_table((8,), freqs=given, device="cpu")
        assert max(off(turns, [Decimal(f) for f in given])) <= 0.5 + 1e-9
        tensor = torch.tensor(given, dtype=torch.float64)
        assert torch.equal(turns, cake.cake_rotary_table((8,), freqs=tensor, device="cpu")[0])


def test_refusals(cake):
    for kw in ({"freqs": [1.0]}, {"freqs": [1.0, float("nan")]}, {"freqs": [float("inf"), 1.0]}, {"base": 0.0},
               {"base": -2.0}, {"base": float("nan")}):
        with pytest.raises(ValueError):
            cake.cake_rotary_table((2,), device="cpu", **kw)
    for base, want in ((float("inf"), [1, 0]), (1.0, [1, 1]), (1e-300, [1, 10 ** 150])):
        turns, _ = cake.cake_rotary_table((2,), base, device="cpu")
        same, _ = cake.cake_rotary_table((1,), freqs=[1.0], device="cpu")
        assert int(turns[0]) == int(same[0]) and (want[1] > 1 or int(turns[1]) == want[1] * int(same[0]))
    turns, axes = cake.cake_rotary_table((), device="cpu")
    assert turns.numel() == axes.numel() == 0
    turns, _ = cake.cake_rotary_table((0, 8), shared=True, device="cpu")
    assert turns.numel() == 8


def test_the_callers_context_and_an_unused_base(cake):
    import decimal
    want = cake.cake_rotary_table((16,), device="cpu")[0]
    given = cake.cake_rotary_table((2,), freqs=[0.5, 0.25], device="cpu")[0]
    with localcontext() as c:
        c.prec, c.rounding, c.Emax = 5, decimal.ROUND_DOWN, 20
        c.traps[decimal.Inexact] = True
        assert torch.equal(cake.cake_rotary_table((16,), device="cpu")[0], want)
        assert torch.equal(cake.cake_rotary_table((2,), None, freqs=[0.5, 0.25], device="cpu")[0], given)
