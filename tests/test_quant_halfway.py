"""float32 values whose quotient x qmax / max |x| lies halfway between two float32 numbers, the larger or smaller of which
is a tie of the 8-bit type: the quotient as a rounded float32 is then the even one, and which 8-bit value follows depends on
it.  They need a largest value whose odd part is small (3 or 5 for e4m3, up to 127 for int8), and are found here in whole
numbers.  q is equal to what float64's quotient gives: x qmax is exact there, and the quotient, off every halfway point by
2^-49 or more where it is not on one, is rounded once to float64 and then to float32 as the exact one is."""
from fractions import Fraction

import pytest
import torch

from memory_bound_row_rmsnorm_gb300 import binding as qb
from test_add_rmsnorm import DEV, QT, cuda, lib  # noqa: F401
from test_quant import check

gpu = pytest.mark.gpu


def ties(qname):
    """Numbers halfway between two neighbours of the type, below its largest."""
    if qname == "int8":
        return [Fraction(2 * n + 1, 2) for n in range(127)]
    normal = [Fraction(m, 16) * Fraction(2) ** e for e in range(-6, 9) for m in range(17, 32, 2)]
    return [Fraction(2 * n + 1, 1024) for n in range(8)] + [t for t in normal if t < 448]


def halfway(qname, odd):
    """All x for the largest value `odd` whose quotient is halfway between a tie and one of its float32 neighbours."""
    qmax, found = int(QT[qname][2]), []
    for t in ties(qname):
        e = 0
        while Fraction(2) ** (e + 1) <= t:
            e += 1
        while Fraction(2) ** e > t:
            e -= 1
        step = Fraction(2) ** (e - 23)
        for q in (t - step / 2, t + step / 2):
            x = q * odd / qmax
            n = x.numerator
            while n % 2 == 0:
                n //= 2
            if n < 2 ** 24 and x.denominator & (x.denominator - 1) == 0 and x < odd:
                found.append(float(x))
    return found


ODD = {"e4m3": [1, 3, 5], "int8": list(range(1, 128, 2))}


def test_there_are_such_values():
    assert all(torch.tensor(x).item() == x for q in ODD for o in ODD[q] for x in halfway(q, o))
    assert float.fromhex("0x1.3b6db6p0") in halfway("e4m3", 3)


@gpu
@pytest.mark.parametrize("qname", ["e4m3", "int8"])
@pytest.mark.parametrize("exponent", [0, -50, -54, -90, -99, 100, 120])
def test_quotients_halfway_between_two_floats(cuda, qname, exponent):
    for odd in ODD[qname]:
        xs = halfway(qname, odd)
        if not xs:
            continue
        xs = xs + [-x for x in xs]
        values = torch.tensor([v for i in range(0, len(xs), 127) for v in ([float(odd)] + xs[i:i + 127] + [0.0] * 127)[:128]])
        x = (values.view(-1, 128) * 2.0 ** exponent).to(DEV)  # a row a group, its first value the largest
        for rows in (1, 128):
            q, scale, qt, scale_t = qb.quant_fwd(x, block_rows=rows, qdtype=QT[qname][1], want_t=True)
            check(q, scale, x, rows, qname, f"{qname} {odd}")
            check(qt, scale_t, x.T.contiguous(), rows, qname, f"turned {qname} {odd}")
        y = x.T.contiguous()  # and down the columns
        q, scale, qt, scale_t = qb.quant_fwd(y, qdtype=QT[qname][1], want_t=True)
        check(qt, scale_t, x, 1, qname, f"columns {qname} {odd}")
