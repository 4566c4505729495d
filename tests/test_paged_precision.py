"""The fp32 bound of paged_precision.py on the host: an fp32 evaluation keeps it, and evaluations with inputs,
weights or values of fewer bits do not."""
import pytest

import paged_precision as pp


@pytest.mark.parametrize("case", pp.CASES, ids=str)
def test_fewer_bits_exceed_the_bound(case):
    data = pp.inputs(case)
    ref = pp.reference(case, data)
    assert pp.worst(case, data, pp.evaluate(case, data), ref) <= 1.0
    for kept in (dict(qk=10), dict(v=10), dict(p=10), dict(qk=10, v=10), dict(p=7), dict(qk=7, p=7, v=7)):
        assert pp.worst(case, data, pp.evaluate(case, data, **kept), ref) > 4.0, kept
