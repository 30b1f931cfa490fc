"""Which waits the products make before a CTA that gave up ends (csrc/ring.cuh): over
random schedules of a ring's loaders, its consumer and the moment of giving up, every load
still in flight is covered by one of them."""

import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mini_ema_means_b200", "csrc")


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    at = tmp_path_factory.mktemp("ring")
    (at / "r.cpp").write_text('#include "ring.cuh"\n' + "".join(
        f'extern "C" uint32_t {n}(uint32_t a, uint32_t b) {{ return em::ring_{n}(a, b); }}\n'
        for n in ("first", "stage", "parity")))
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-I", CSRC, "-o", str(at / "r.so"), str(at / "r.cpp")], check=True)
    lib = ctypes.CDLL(str(at / "r.so"))
    for n in ("first", "stage", "parity"):
        getattr(lib, n).argtypes, getattr(lib, n).restype = [ctypes.c_uint32] * 2, ctypes.c_uint32
    return lib


def _run(rng, stages, loaders, total):
    """(fills begun by each loader, loads in flight as (fill, loader), completed phases of
    each stage's barrier) when every role of a CTA has ended after one gave up."""
    begun, consumed = [0] * loaders, 0
    flight, landed, phases = set(), {}, [0] * stages
    stops = [False] * loaders
    gives_up = rng.randrange(4 * total)
    for step in range(10 ** 6):
        if step >= gives_up:  # each loader sees it when it next waits, or gets through some waits before
            stops = [s or rng.random() < 0.5 for s in stops]
            if all(s or b == total for s, b in zip(stops, begun)):
                break
        move = rng.random()
        who = rng.randrange(loaders)
        if move < 0.5 and not stops[who] and begun[who] < total and begun[who] < consumed + stages:
            flight.add((begun[who], who))
            begun[who] += 1
        elif move < 0.8 and flight:
            fill, at = rng.choice(sorted(flight))
            flight.remove((fill, at))
            landed[fill] = landed.get(fill, 0) + 1
            if landed[fill] == loaders:
                assert phases[fill % stages] == fill // stages
                phases[fill % stages] += 1
        elif step < gives_up and landed.get(consumed, 0) == loaders:
            consumed += 1
        if step >= gives_up and min(begun) == total:
            break
    return begun, flight, phases


@pytest.mark.parametrize("stages,loaders", [(3, 2), (4, 2), (5, 2), (6, 1), (6, 2), (6, 4)])
def test_every_load_in_flight_is_waited_for(ring, stages, loaders):
    rng = random.Random(stages * 10 + loaders)
    apart = in_flight = 0
    for _ in range(3000):
        begun, flight, phases = _run(rng, stages, loaders, total=rng.choice([1, stages, 3 * stages + 1, 40]))
        lead = max(begun)
        waits = {i: (ring.stage(i, stages), ring.parity(i, stages)) for i in range(ring.first(lead, stages), lead)}
        assert len({s for s, _ in waits.values()}) == len(waits)  # one wait a stage
        for fill, _ in flight:
            stage, parity = waits[fill]
            # the wait holds on: the phase that this load belongs to is not complete
            assert stage == fill % stages and phases[stage] % 2 == parity and phases[stage] == fill // stages
        for fill, (stage, _) in waits.items():  # and returns where the phase is complete
            assert phases[stage] in (fill // stages, fill // stages + 1)
        apart += any(b != lead for b in begun) and any(i >= min(begun) for i, _ in flight)
        in_flight += bool(flight)
    assert in_flight > 300 and (loaders == 1 or apart > 100)
