"""The README's example of the paged cache: on host tensors through all of the
argument checks, and as it stands on a GPU."""
import os
import re

import pytest

from test_abi_cpu import NO_GPU, ROOT


def _examples():
    src = open(os.path.join(ROOT, "README.md")).read()
    return re.findall(r"```python\n(.*?)```", src, re.S)


@pytest.mark.skipif(not NO_GPU, reason="host tensors would reach a launch where a GPU is present")
def test_paged_example_passes_the_host_checks():
    torch = pytest.importorskip("torch")
    from full_duplex_speech_gb300 import build
    build.build()
    import full_duplex_speech_gb300 as m2
    rcs = []

    class Checked:
        def __getattr__(self, name):
            f = getattr(m2, name)
            if not name.startswith("mamba2_"):
                return f
            return lambda *a: rcs.append((name, f(*a, stream=0, check=False)))

    code = [c for c in _examples() if "kv_cache(" in c]
    assert len(code) == 1
    exec(compile(code[0], "README.md", "exec"), {"torch": torch, "m2": Checked(), "dev": "cpu", "bf": torch.bfloat16})
    assert [n for n, _ in rcs] == ["mamba2_kv_append", "mamba2_attn_paged"] * 2
    assert all(rc == 5 for _, rc in rcs), rcs  # M2_ECUDA: no device here


@pytest.mark.gpu
def test_paged_example_runs():
    """Both examples in order; the paged one's last frame against fp64."""
    import torch

    from test_gpu_kv_paged import Cache
    from test_gpu_kv_paged_forms import check
    names = {}
    for code in _examples():
        exec(compile(code, "README.md", "exec"), names)
    torch.cuda.synchronize()
    m2 = names["m2"]
    assert m2.mamba2_device_error() == 0
    S, Hq, D, T = names["S"], names["Hq"], names["D"], names["T"]
    assert names["lengths"].tolist() == [301, 42] and T == 1
    held = Cache.__new__(Cache)
    held.d_table, held.ps = names["table"], names["page"]
    held.kp, held.vp, held.ks, held.vs = (names[n] for n in ("kp", "vp", "ks", "vs"))
    q = names["q"].reshape(S, T, Hq, D)
    check(held, q, names["out"].view(S, T, Hq, D), [300, 41], [1, 1], True, D ** -0.5, "bf16")
