"""Host checks of the gated recurrence's launches on several devices: tests/scan_devices.cu, the calls' own source with
stand-ins for CUDA, compiled here without device code."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LONG, SHORT, OK = 16384, 10, 0


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("needs nvcc")
    out = str(tmp_path_factory.mktemp("launches") / "scan_devices")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=compute_103a", "-std=c++17", "-O0", "-Xcicc", "-O0",
                    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "diagonal_state_space_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "scan_devices.cu"), "-o", out], check=True, timeout=600)
    return out


def run(program, *calls):
    """Status and cluster forward, status backward, of each call (device, length)."""
    text = subprocess.run([program, *(str(v) for c in calls for v in c)], check=True, capture_output=True, text=True).stdout
    return [tuple(int(v) for v in line.split()) for line in text.splitlines()]


def test_a_long_sequence_takes_the_largest_cluster(program):
    assert run(program, (0, LONG)) == [(OK, 16, OK)]


@pytest.mark.parametrize("order", [[(0, LONG), (1, SHORT), (1, LONG)], [(0, SHORT), (1, LONG), (0, LONG)], [(70, LONG), (71, SHORT), (71, LONG)]])
def test_what_another_device_ran_first_does_not_matter(program, order):
    assert run(program, *order) == [(OK, 16 if n == LONG else 1, OK) for _, n in order]


def test_each_device_has_its_own_room(program):
    """Device 2 has no room for more than eight blocks of a cluster at once."""
    assert run(program, (0, LONG), (2, LONG), (0, LONG)) == [(OK, 16, OK), (OK, 8, OK), (OK, 16, OK)]
    assert run(program, (2, LONG), (0, LONG)) == [(OK, 8, OK), (OK, 16, OK)]
