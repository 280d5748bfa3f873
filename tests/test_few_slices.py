"""Who writes a column tile of moe_layer_few's out when K is cut into slices (host check, no
GPU): the kernel's own rules (csrc/few_rules.hpp) are compiled for the host and played
through orders of arrival, with slices that gave their wait up, and with a clear of the
arrivals by another call on the same workspace.

  * all slices waited, workspace of the call's own: one store, of the sum of all slices;
  * a slice gave up: the tile ends as NaN, whatever the order;
  * a slice gave up and the arrivals are cleared at any point: the tile is written all the
    same (with what is undefined; it does not keep what stood there before).
"""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_mixture_experts_05_amd", "csrc")
STORE, HAND_OVER, GIVE_UP = range(3)
NAN = "nan"


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("few") / "slices_host.so")
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}",
                        os.path.join(ROOT, "tests", "slices_host.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(out)
    L.few_adds_up.argtypes = [ctypes.c_uint, ctypes.c_int]
    return (lambda waited, D: L.few_slice_step(int(waited), D),
            lambda before, D: bool(L.few_adds_up(before, D)))


def play(rules, waited, order, clear_at=None):
    """What the slices store in turn: NAN, or the slices that a sum has. A slice's partial
    sum is NaN where it gave up."""
    step, adds_up = rules
    D, arrived, parts, stores = len(waited), 0, {}, []
    for n, d in enumerate(order):
        if n == clear_at:
            arrived = 0
        what = step(waited[d], D)
        if what == GIVE_UP:
            stores.append(NAN)
            continue
        value = frozenset([d]) if waited[d] else NAN
        if what == STORE:
            stores.append(value)
            continue
        assert what == HAND_OVER
        parts[d] = value
        before, arrived = arrived, arrived + 1
        if adds_up(before, D):
            had = [parts.get(i, frozenset()) for i in range(D)]
            stores.append(NAN if NAN in had else frozenset().union(*had))
    return stores


def orders(D):
    if D <= 4:
        return list(itertools.permutations(range(D)))
    rng = random.Random(D)
    return [rng.sample(range(D), D) for _ in range(60)]


def check(rules):
    for D in (1, 2, 4, 8):
        for order in orders(D):
            assert play(rules, [True] * D, order) == [frozenset(range(D))]
            for gave_up in range(1, 1 << D):
                waited = [not gave_up >> d & 1 for d in range(D)]
                stores = play(rules, waited, order)
                assert stores and set(stores) == {NAN}, (D, order, waited)
                for clear_at in range(D):
                    assert play(rules, waited, order, clear_at), (D, order, waited, clear_at)


def test_tile_of_a_slice_that_gave_up_is_written(rules):
    check(rules)


def test_check_finds_a_give_up_that_only_arrives(rules):
    """The check is not blind: slices that hand NaN over, and leave its store to the last
    arrival, leave the tile as it was after a clear."""
    handing = (lambda waited, D: HAND_OVER if D > 1 else STORE, rules[1])
    assert play(handing, [False, True], (0, 1)) == [NAN]
    with pytest.raises(AssertionError):
        check(handing)
