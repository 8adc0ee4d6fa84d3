"""Which kernel the calls of tests/_tiles.py take on a card of 256 compute units, by the
library's own rules: each case runs the kernel that it is there for, with more tiles than
the launch has workgroups, and with reductions that go round the ring of stages."""

import pytest

from tests import _tiles as r

CUS = 256


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return r.load_rules(str(tmp_path_factory.mktemp("rules")))


@pytest.mark.parametrize("c", r.CASES, ids=[r.name(c) for c in r.CASES])
def test_case(rules, c):
    assert r.shape_taken(rules, c, CUS) == c["shape"]
    if c["shape"] == r.VECTORS:
        # 8 workgroups of 256 threads a compute unit at most
        assert r.vector_groups(c) > 8 * CUS or max(c["sizes"]) > 4
        return
    resident = 2 if c["shape"] == r.MIDDLE else 1
    assert r.tiles(c) > resident * CUS
    ring = 4 if c["shape"] in (r.DEEP, r.SMALL) else 2
    assert r.stages(c) > ring


def test_stages_of_the_cases():
    """Odd and even numbers of stages, whole and ragged last ones, in both directions."""
    for shape in (r.LARGE, r.MIDDLE):
        for op in ("fwd", "bwd", "i8"):
            n = {r.stages(c) % 2 for c in r.CASES if c["shape"] == shape and c["op"] == op}
            assert n == {0, 1}, (shape, op, n)
    assert any(c["depth"] * 2 % r.STAGE == 0 for c in r.CASES if c["op"] == "fwd")
    assert any(c["depth"] % r.STAGE == 0 for c in r.CASES if c["op"] == "i8")


def test_small_calls_and_long_sums(rules):
    """Where the vectors end: sums of the longest reduction run on both kernels."""
    K = 131056
    assert rules.vec(2, 1, 8, 0, K, CUS)
    for rows in (5, 130):
        assert not rules.vec(rows, 1, 8, 0, K, CUS)
