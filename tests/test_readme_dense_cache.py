"""The README's example of the bounded dense caches: on host tensors through all
of the argument checks, and as it stands on a GPU."""
import pytest

from test_abi_cpu import NO_GPU
from test_readme_paged import _examples


def _example():
    code = [c for c in _examples() if "mamba2_kv_evict(" in c]
    assert len(code) == 1
    return compile(code[0], "README.md", "exec")


@pytest.mark.skipif(not NO_GPU, reason="host tensors would reach a launch where a GPU is present")
def test_example_passes_the_host_checks():
    torch = pytest.importorskip("torch")
    from full_duplex_speech_gb300 import build
    build.build()
    import full_duplex_speech_gb300 as m2
    rcs = {}

    class Checked:
        def __getattr__(self, name):
            f = getattr(m2, name)
            if name.endswith("_workspace_bytes"):
                return f
            return lambda *a: rcs.setdefault(name, set()).add(f(*a, stream=0, check=False))

    exec(_example(), {"torch": torch, "m2": Checked(), "dev": "cpu", "bf": torch.bfloat16})
    want = {5}  # M2_ECUDA: no device here
    assert rcs == {n: want for n in ("mamba2_attn_prompt", "mamba2_attn_prompt_weights", "mamba2_attn_decode_weights",
                                     "mamba2_kv_evict")}


@pytest.mark.gpu
def test_example_runs():
    """The sessions after an eviction and some frames; the last frame against fp64."""
    import numpy as np
    import torch

    import full_duplex_speech_gb300 as m2
    from dense_cache_lib import check_rows
    names = {"torch": torch, "m2": m2, "dev": "cuda", "bf": torch.bfloat16}
    exec(_example(), names)
    torch.cuda.synchronize()
    assert m2.mamba2_device_error() == 0
    # 196 frames to 4096 positions, then 54 behind the 2048 that stay
    assert names["have"].tolist() == [2048 + 54, 300 + 250]
    for s, L in enumerate(names["have"].tolist()):
        k, v, q, out = (names[x][s].double().cpu().numpy() for x in ("k_cache", "v_cache", "q1", "frame_out"))
        check_rows(out[None], None, q[None], k[:, :L], v[:, :L], names["scale"], L - 1, "bf16")
        weight = names["weight"][s, :, :L].double().cpu().numpy()
        # each of a kv head's five queries hands out a weight of one: the last 32 rows of the prompt's and the frames'
        if s == 1:
            assert np.all(np.abs(weight.sum(-1) - 5 * (32 + 250)) < 1e-3 * 5 * 282)
        assert np.all(weight >= 0)
