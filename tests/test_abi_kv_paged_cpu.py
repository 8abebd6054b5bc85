"""CPU-side checks of the paged 8-bit cache's entry points: bad arguments are
rejected before the GPU is touched (these run without a GPU)."""
import pytest

from test_abi_cpu import NO_GPU, _fake_ptrs, _past_host_checks


@pytest.fixture(scope="module")
def m2():
    from full_duplex_speech_gb300 import build
    build.build()
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


def test_kv_paged_validation_without_gpu(m2):
    """mamba2_kv_append and mamba2_attn_paged check sizes, pointers, strides and
    alignment on the host, before any device call."""
    a = _fake_ptrs(18)
    table, kp, vp, ks, vs, kt, vt, lens, new, k, v, q, qo, cos, sin, out = a[:16]

    def cache(S=2, Hkv=8, ps=64, pages=100, cols=10, D=128, act="bf16", **p):
        f = dict(page_table=table, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, k_tail=kt, v_tail=vt) | p
        return m2.kv_cache(S, Hkv, ps, pages, cols, act=act, head_dim=D, **f)

    def app(c=None, T=4, lens=lens, new=new, k=k, v=v, ks_=1024, rope=None, H=0, q=None, qs=0, o=None, os_=0):
        return m2.mamba2_kv_append(c or cache(), T, lens, new, k, v, ks_, rope, H, q, qs, o, os_, stream=0, check=False)

    def att(c=None, T=4, H=40, causal=True, lens=lens, new=new, q=q, qs=5120, scale=0.1, o=out, os_=5120, ws=1 << 30,
            wsb=1 << 40):
        return m2.mamba2_attn_paged(c or cache(), T, H, causal, lens, new, q, qs, scale, o, os_, ws, workspace_bytes=wsb,
                                    stream=0, check=False)

    for f in (app, att):
        for bad in (dict(S=-1), dict(Hkv=0), dict(ps=0), dict(pages=0), dict(cols=0), dict(D=0)):
            assert f(cache(**bad)) == 1, bad
        assert f(T=-1) == 1
        # head_dim, page sizes, grid limits, 2^30 positions, 2^31 rows
        for bad in (dict(D=64), dict(ps=48), dict(ps=8), dict(ps=256), dict(S=65536), dict(Hkv=65536),
                    dict(cols=(1 << 24) + 1), dict(pages=1 << 22)):
            assert f(cache(**bad)) == 2, bad
        assert f(T=(1 << 24) + 1) == 2
        for n in ("page_table", "k_pages", "v_pages", "k_scales", "v_scales"):
            assert f(cache(**{n: None})) == 1, n
            assert f(cache(**{n: a[17] + 2})) == 3, n
        assert f(lens=None) == 1 and f(lens=lens + 2) == 3 and f(new=new + 1) == 3
    bad_act = cache()
    bad_act.act = 7
    assert app(bad_act) == 1 and att(bad_act) == 1
    for n in ("k_tail", "v_tail"):
        assert app(cache(**{n: None})) == 1 and app(cache(**{n: a[17] + 8})) == 3
        assert app(cache(**{n + "_out": a[17] + 4})) == 3
    assert app(k=None) == 1 and app(v=None) == 1 and app(k=k + 8) == 3 and app(v=v + 2) == 3
    assert app(ks_=1023) == 1 and app(ks_=1028) == 3        # rows overlap; pitch not a multiple of 16 bytes
    full = dict(H=40, q=q, qs=5120, o=qo, os_=5120)
    assert app(**full | dict(q=None)) == 1 and app(**full | dict(o=None)) == 1
    assert app(**full | dict(H=41)) == 2 and app(**full | dict(H=0)) == 1 and app(H=-1) == 1
    assert app(**full | dict(qs=5119)) == 1 and app(**full | dict(os_=5124)) == 3 and app(**full | dict(o=qo + 4)) == 3
    assert app(**full | dict(o=q, os_=5248)) == 1 and att(o=q) == 1  # rotated in place at two strides; out over q
    rope = lambda rot=64, n=10, c=cos, s=sin: m2.rope(rot, n, c, s)  # noqa: E731
    assert app(rope=rope(rot=-16)) == 1 and app(rope=rope(n=0)) == 1 and app(rope=rope(c=None)) == 1
    assert app(rope=rope(rot=24)) == 2 and app(rope=rope(rot=144)) == 2 and app(rope=rope(s=sin + 4)) == 3
    assert att(H=0) == 1 and att(H=44) == 2 and att(scale=float("nan")) == 1 and att(scale=float("inf")) == 1
    assert att(q=None) == 1 and att(o=None) == 1 and att(q=q + 2) == 3 and att(o=out + 8) == 3
    assert att(qs=5119) == 1 and att(os_=5119) == 1 and att(qs=5124) == 3
    assert m2.mamba2_attn_paged_workspace_bytes(cache(), 4, 40) == 0  # merges in shared memory
    assert att(ws=(1 << 30) + 8) == 3 and _past_host_checks(att(cache(S=0), ws=None, wsb=0))
    for S in (0, 2) if NO_GPU else (0,):
        c = cache(S=S)
        assert _past_host_checks(app(c)) and _past_host_checks(app(c, **full, rope=rope())) and _past_host_checks(att(c))
        assert _past_host_checks(app(c, new=None)) and _past_host_checks(att(c, new=None, causal=False))
    assert _past_host_checks(att(T=0))


def test_the_plan_of_a_call_is_refused_like_the_call(m2):
    """m2_attn_paged_plan, which the tests of each form ask, checks sizes as
    mamba2_attn_paged does and returns the negative status."""
    import ctypes
    plan = m2.load().m2_attn_paged_plan

    def ask(T=4, H=40, D=128, ps=64):
        c = m2.kv_cache(2, 8, ps, 100, 10, *(None,) * 5, head_dim=D)
        return plan(ctypes.byref(c), T, H)

    assert plan(None, 1, 1) == -1
    assert ask(T=-1) == -1 and ask(H=0) == -1
    assert ask(H=41) == -2 and ask(D=64) == -2 and ask(ps=48) == -2
    if NO_GPU:
        assert ask() == -5
