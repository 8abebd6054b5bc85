"""The hand-over protocol of the attention tiles (csrc/m2_tile_meet.h) in a host
model: every warp comes to its end, also when bounded waits run out."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path_factory.mktemp("tile_meet") / "model")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-pthread", "-I",
                        os.path.join(ROOT, "full_duplex_speech_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "tile_meet", "model.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_every_warp_comes_to_its_end(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_model_sees_a_protocol_that_gets_stuck(model):
    """Softmax warps that arrive without waiting are counted for one meeting
    twice once a wait of theirs has run out."""
    r = subprocess.run([model, "arrive"], capture_output=True, text=True, timeout=120)
    assert r.returncode == 2 and "stuck" in r.stdout, r.stdout + r.stderr


def test_the_kernel_hands_over_by_this_protocol_alone():
    """The tiles' barriers are used through the protocol: no arrival without a
    wait, and every role by the functions that the model runs."""
    src = open(os.path.join(ROOT, "full_duplex_speech_gb300", "csrc", "m2_attn_paged_tile.cu")).read()
    assert "barrier.arrive" not in src
    assert src.count("tile_rows_meet(") == 1 and src.count("tile_turns_meet(") == 2
