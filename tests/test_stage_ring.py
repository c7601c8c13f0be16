"""The ring that the wide attention kernel's loading warp fills (csrc/stage_ring.h), run by host threads whose waits
run out in every order that a late copy brings about: no copy is issued over one under way, none outlives the ring."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "quantized_linear_layer_gb300", "csrc")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    out = str(tmp_path_factory.mktemp("ring") / "stage_ring")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I" + CSRC, os.path.join(HERE, "stage_ring.cpp"), "-o", out],
                   check=True)
    return out


@pytest.mark.parametrize("late", [0, 5, 39])
@pytest.mark.parametrize("delay,reader,filler", [
    (0, 5000, 5000),       # nothing runs out
    (30, 5000, 5000),      # a copy takes long, every wait is patient
    (60, 8, 5000),         # the readers give up first
    (60, 5000, 8),         # the filling role gives up first
    (60, 8, 8), (60, 10, 8), (60, 8, 10)])
def test_waits_that_run_out(program, late, delay, reader, filler):
    r = subprocess.run([program, "40", str(late), str(delay), str(reader), str(filler)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, "%d: %s" % (r.returncode, r.stdout)


@pytest.mark.parametrize("stages,takers", [(8, 5), (6, 6), (8, 7), (12, 7), (16, 7)])
@pytest.mark.parametrize("late", [0, 1, 9])
def test_taking_turns(program, stages, takers, late):
    """Each reader finds its own fill, as many stages and readers as the kernels have."""
    r = subprocess.run([program, "turns", str(stages), str(takers), str(late), "40"], timeout=60)
    assert r.returncode == 0


def test_more_readers_than_stages(program):
    """Seven readers at six stages: one is a whole round ahead when a copy is late, which the kernels' geometry excludes."""
    r = subprocess.run([program, "turns", "6", "7", "1", "300"], timeout=60)
    assert r.returncode == 1
