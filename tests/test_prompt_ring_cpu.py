"""The ring of shared memory of the prompts' tiles (csrc/m2_prompt_ring.h) in a
host model: no wait passes before its piece's turn, and every warp comes to its
end, whoever is slow."""
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
    exe = str(tmp_path_factory.mktemp("prompt_ring") / "model")
    r = subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-pthread", "-I",
                        os.path.join(ROOT, "full_duplex_speech_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "prompt_ring", "model.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


def test_every_wait_has_its_turn(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_the_model_sees_a_wait_that_passes_early(model):
    """With room for the outputs of refused pairs, a tile without rows in the pair before comes to
    such a piece while its stage's turn before is still under way."""
    r = subprocess.run([model, "pieces"], capture_output=True, text=True, timeout=200)
    assert r.returncode == 2 and "early" in r.stdout, r.stdout + r.stderr


def test_the_model_sees_a_run_that_gets_stuck(model):
    """A warp that looks at an output's room only when the stage's next piece has landed waits for its own answer."""
    r = subprocess.run([model, "full"], capture_output=True, text=True, timeout=200)
    assert r.returncode == 2 and "stuck" in r.stdout, r.stdout + r.stderr


def test_the_kernel_uses_its_ring_by_these_rules():
    src = open(os.path.join(ROOT, "full_duplex_speech_gb300", "csrc", "m2_attn_prompt_tile.cu")).read()
    for rule in ("ring_pieces(", "ring_fill(", "ring_look(", "ring_room("):
        assert src.count(rule) == 1, rule
