"""The ring of K/V tiles of the tensor-core chunk attention, as a model that tries
every order in which its steps can come, with the rule for waits that the kernel
is compiled with."""

import os
import shutil
import subprocess

import pytest

from self_speculative_verification_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))

# steps, heads' streams, steps of tile A, of tile B, steps whose values every row sees
LAYOUTS = {
    "both tiles throughout": "4,1,4,4,3 3,1,3,3,2",
    "tile B absent, then there": "4,1,4,0,4 3,1,3,3,2",
    "tile A a step short": "5,1,4,5,4 3,1,3,3,3",
    "tile A through, then there": "3,1,0,3,0 4,1,4,4,3",
    "two heads": "2,2,2,2,1 2,2,2,2,1",
    "short ones of all kinds": "3,1,3,0,2 2,2,2,2,1 1,1,1,0,0 1,1,1,1,0",
    "single steps": "1,1,1,0,0 1,1,1,0,0 3,1,3,3,0 1,1,0,1,0 2,2,2,2,0",
}


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    gxx = shutil.which("g++") or shutil.which("c++")
    if not gxx:
        pytest.skip("no C++ compiler")
    exe = tmp_path_factory.mktemp("ring") / "ring_model"
    subprocess.run([gxx, "-O2", "-std=c++17", "-Wall", "-Werror", "-I", _build.CSRC,
                    os.path.join(HERE, "chunk_ring_model.cpp"), "-o", str(exe)], check=True)

    def run(slots, in_order, rule, parts):
        r = subprocess.run([str(exe), str(slots), str(int(in_order)), str(rule), *parts.split()],
                           capture_output=True, text=True, timeout=600, check=True)
        return r.stdout.strip()

    return run


@pytest.mark.parametrize("slots,in_order", [(5, False), (8, False), (3, True), (8, True)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_no_tile_takes_another_fill(model, slots, in_order, layout):
    assert model(slots, in_order, 0, LAYOUTS[layout]).startswith("ok")


@pytest.mark.parametrize("slots", [5, 8])
@pytest.mark.parametrize("rule,layout", [
    (1, "tile B absent, then there"), (1, "tile A a step short"), (1, "tile A through, then there"),
    (2, "tile B absent, then there"), (2, "short ones of all kinds")])
def test_fewer_questions_are_not_enough(model, slots, rule, layout):
    """The model tells: asked only where a part begins (and in units of two heads),
    a wait is met by the fill before."""
    assert "takes another fill" in model(slots, False, rule, LAYOUTS[layout])
