"""How exact the turns of a rotary plan are: they come from a double, so a
position's angle is off by up to 2^-55 of a turn for each position (the power's
and the quotient's roundings, 2^-53 of at most 0.16 turns each, and 2 pi's)."""
from decimal import Decimal, getcontext

import pytest

from backward_tcgen05_tma_gemms_gb300 import api
from test_abi_host import lib  # noqa: F401  (fixture)

pytestmark = pytest.mark.usefixtures("lib")
getcontext().prec = 50
TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937511")


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 3.0), ("linear", 8.0), ("ntk", 4.0), ("ntk", 31.7)])
@pytest.mark.parametrize("base", [10.0, 10000.0, 500000.0, 1234.567])
@pytest.mark.parametrize("rot", [4, 64, 96, 128, 512])
def test_turns_are_good_to_2_to_the_minus_55(rot, base, scaling, factor):
    plan = api.rope_plan(rot, base=base, scaling=scaling, factor=factor)
    b, s = Decimal(base), Decimal(factor)
    if scaling == "ntk":
        b *= s ** (Decimal(rot) / Decimal(rot - 2))
    for i in range(rot // 2):
        want = b ** (Decimal(-2 * i) / Decimal(rot)) / TWO_PI / (s if scaling == "linear" else 1)
        assert abs(Decimal(int(plan.turns[i])) / Decimal(2) ** 64 - want) <= Decimal(2) ** -55


def test_plans_whose_numbers_are_not_finite_are_refused():
    for kw in (dict(attention_factor=float("inf")), dict(attention_factor=float("nan")),
               dict(scaling="ntk", factor=1e300, base=1e20)):
        with pytest.raises(api.TpsError) as e:
            api.rope_plan(64, **kw)
        assert e.value.code == api.ERR_ARG
    assert api.rope_plan(64, attention_factor=0.5).amplitude == 0.5
