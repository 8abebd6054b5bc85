"""CPU-side checks of the bounded dense caches' entry points: bad arguments are
rejected before the GPU is touched (these run without a GPU)."""
import pytest

from test_abi_cpu import NO_GPU, _past_host_checks

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def m2():
    from full_duplex_speech_gb300 import build
    build.build()
    import full_duplex_speech_gb300 as m2
    m2.load()
    return m2


def _caller(f, order, good):
    def call(**change):
        return f(*[{**good, **change}[n] for n in order], stream=0, check=False)
    return call


# distinct addresses far enough apart that arrays of the sizes below do not meet
PTR = [(1 << 40) + (i << 32) for i in range(16)]
SIZES = ["S", "rows", "Hq", "Hkv", "D", "max_len", "act"]
GOOD = dict(S=2, rows=10, Hq=40, Hkv=8, D=128, max_len=100, act="bf16", row_start=PTR[0], lengths=PTR[1], q=PTR[2], qs=7168,
            k=PTR[3], v=PTR[4], kvs=7168, kc=PTR[5], vc=PTR[6], scale=0.1, out=PTR[7], outs=5120, lse=PTR[8], window=4,
            acc=PTR[9], acc_out=PTR[10])


def _sizes_are_checked(call, rows):
    for bad in (dict(S=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(max_len=0)) + ((dict(rows=-1),) if rows else ()):
        assert call(**bad) == 1, bad
    for bad in (dict(D=64), dict(Hq=44), dict(Hq=72), dict(S=65536)):
        assert call(**bad) == 2, bad


def _scale_is_checked(call):
    assert call(scale=NAN) == 1 and call(scale=INF) == 1


def test_attn_prompt_validation_without_gpu(m2):
    call = _caller(m2.mamba2_attn_prompt, SIZES + ["row_start", "lengths", "q", "qs", "k", "v", "kvs", "kc", "vc", "scale",
                                                   "out", "outs", "lse"], GOOD)
    _sizes_are_checked(call, True)
    _scale_is_checked(call)
    assert call(rows=(1 << 30) // 8 + 1) == 2 and call(max_len=(1 << 30) + 1) == 2
    for n in ("row_start", "q", "k", "v", "kc", "vc", "out"):
        assert call(**{n: None}) == 1, n
    for n in ("q", "k", "v", "kc", "vc", "out"):
        assert call(**{n: GOOD[n] + 8}) == 3, n
    for n in ("row_start", "lengths", "lse"):
        assert call(**{n: GOOD[n] + 2}) == 3, n
    assert call(qs=5119) == 1 and call(kvs=1023) == 1 and call(outs=5119) == 1  # rows overlap
    assert call(qs=5124) == 3 and call(kvs=1028) == 3 and call(outs=5124) == 3  # pitch not a multiple of 16 bytes
    assert call(out=GOOD["q"]) == 1 and call(out=GOOD["k"]) == 1 and call(out=GOOD["v"]) == 1 and call(kc=GOOD["vc"]) == 1
    for zero in (dict(S=0), dict(rows=0)):
        assert _past_host_checks(call(**zero))
    if NO_GPU:
        assert _past_host_checks(call()) and _past_host_checks(call(lengths=None, lse=None)) and _past_host_checks(call(act="f32"))


def test_attn_prompt_weights_validation_without_gpu(m2):
    call = _caller(m2.mamba2_attn_prompt_weights, SIZES + ["row_start", "lengths", "q", "qs", "kc", "scale", "lse", "window",
                                                           "acc", "acc_out"], GOOD)
    _sizes_are_checked(call, True)
    _scale_is_checked(call)
    for n in ("row_start", "q", "kc", "lse", "acc", "acc_out"):
        assert call(**{n: None}) == 1, n
    for n in ("q", "kc", "acc", "acc_out"):
        assert call(**{n: GOOD[n] + 8}) == 3, n
    for n in ("row_start", "lengths", "lse"):
        assert call(**{n: GOOD[n] + 2}) == 3, n
    assert call(window=-1) == 1 and call(qs=5119) == 1 and call(qs=5124) == 3
    assert call(acc_out=GOOD["acc"] + 16) == 1 and call(acc_out=GOOD["acc"] + 2 * 8 * 100 * 4 - 16) == 1  # it overlaps acc
    assert _past_host_checks(call(S=0))
    if NO_GPU:
        for ok in (dict(), dict(acc_out=GOOD["acc"]), dict(acc_out=GOOD["acc"] + 2 * 8 * 100 * 4), dict(window=0), dict(rows=0)):
            assert _past_host_checks(call(**ok)), ok


def test_attn_decode_weights_validation_without_gpu(m2):
    need = m2.mamba2_attn_decode_weights_workspace_bytes(2, 40, 8, 128, 100)
    assert need >= 2 * 40 * 100 * 4
    assert m2.mamba2_attn_decode_weights_workspace_bytes(2, 40, 8, 128, 100, "f32") > need
    assert m2.mamba2_attn_decode_weights_workspace_bytes(0, 40, 8, 128, 100) == 0
    assert m2.mamba2_attn_decode_weights_workspace_bytes(2, 40, 8, 64, 100) == 0
    good = dict(GOOD, ws=PTR[11], wsb=need)
    call = _caller(m2.mamba2_attn_decode_weights, ["S", "Hq", "Hkv", "D", "max_len", "act", "lengths", "q", "k", "v", "kc", "vc",
                                                   "scale", "out", "acc", "acc_out", "ws", "wsb"], good)
    _sizes_are_checked(call, False)
    _scale_is_checked(call)
    for n in ("lengths", "q", "k", "v", "kc", "vc", "out", "acc", "acc_out"):
        assert call(**{n: None}) == 1, n
    for n in ("q", "k", "v", "kc", "vc", "out", "acc", "acc_out", "ws"):
        assert call(**{n: good[n] + 8}) == 3, n
    assert call(lengths=good["lengths"] + 2) == 3 and call(acc_out=good["acc"] + 32) == 1
    assert call(ws=None) == 6 and call(wsb=need - 1) == 6
    assert _past_host_checks(call(S=0, ws=None, wsb=0))
    if NO_GPU:
        assert _past_host_checks(call()) and _past_host_checks(call(acc_out=good["acc"]))


def test_caches_past_the_limit_are_refused_by_every_call(m2):
    """max_len at most 2^30: by the frames and the query of their scratch too."""
    assert m2.mamba2_attn_decode_weights_workspace_bytes(1, 1, 1, 128, 1 << 30) >= (1 << 30) * 4
    for longest in ((1 << 30) + 1, (1 << 31) - 1):
        for act in ("bf16", "f32"):
            assert m2.mamba2_attn_decode_weights_workspace_bytes(1, 1, 1, 128, longest, act) == 0
    good = dict(GOOD, S=1, Hq=8, Hkv=1, ws=PTR[11], wsb=1 << 62, keep=50, recent=10, out_max=60, ko=PTR[12], vo=PTR[13],
                kept=PTR[14])
    for f, order in ((m2.mamba2_attn_prompt, SIZES + ["row_start", "lengths", "q", "qs", "k", "v", "kvs", "kc", "vc", "scale",
                                                      "out", "outs", "lse"]),
                     (m2.mamba2_attn_prompt_weights, SIZES + ["row_start", "lengths", "q", "qs", "kc", "scale", "lse", "window",
                                                              "acc", "acc_out"]),
                     (m2.mamba2_attn_decode_weights, ["S", "Hq", "Hkv", "D", "max_len", "act", "lengths", "q", "k", "v", "kc",
                                                      "vc", "scale", "out", "acc", "acc_out", "ws", "wsb"]),
                     (m2.mamba2_kv_evict, ["S", "Hkv", "D", "max_len", "act", "lengths", "kc", "vc", "acc", "keep", "recent",
                                           "out_max", "ko", "vo", "acc_out", "kept"])):
        for longest in ((1 << 30) + 1, (1 << 31) - 1):
            assert _caller(f, order, good)(max_len=longest, acc_out=GOOD["acc"]) == 2, f.__name__


def test_kv_evict_validation_without_gpu(m2):
    good = dict(GOOD, keep=50, recent=10, out_max=60, ko=PTR[11], vo=PTR[12], kept=PTR[13])
    call = _caller(m2.mamba2_kv_evict, ["S", "Hkv", "D", "max_len", "act", "lengths", "kc", "vc", "acc", "keep", "recent",
                                        "out_max", "ko", "vo", "acc_out", "kept"], good)
    for bad in (dict(S=-1), dict(Hkv=0), dict(D=0), dict(max_len=0), dict(keep=0), dict(recent=-1), dict(recent=51),
                dict(out_max=0)):
        assert call(**bad) == 1, bad
    for bad in (dict(D=64), dict(S=65536), dict(Hkv=65536), dict(keep=61), dict(max_len=(1 << 30) + 1)):
        assert call(**bad) == 2, bad
    for n in ("lengths", "kc", "vc", "acc", "ko", "vo", "acc_out"):
        assert call(**{n: None}) == 1, n
    for n in ("kc", "vc", "acc", "ko", "vo", "acc_out"):
        assert call(**{n: good[n] + 8}) == 3, n
    assert call(lengths=good["lengths"] + 2) == 3 and call(kept=good["kept"] + 2) == 3
    kc, vc, acc = good["kc"], good["vc"], good["acc"]
    place = dict(ko=kc, vo=vc, acc_out=acc, out_max=100)
    # one of the two in place, in place into another pitch, partly over an input or over one another
    for bad in (dict(ko=kc), dict(vo=vc), dict(place, out_max=99), dict(acc_out=acc), dict(ko=kc + 256), dict(vo=vc + 1024),
                dict(acc_out=acc + 64), dict(ko=vc + 256), dict(vo=kc + 256), dict(ko=good["vo"]), dict(place, ko=vc, vo=kc)):
        assert call(**bad) == 1, bad
    assert _past_host_checks(call(S=0))
    if NO_GPU:
        for ok in (dict(), place, dict(place, acc_out=good["acc_out"]), dict(kept=None), dict(acc_out=acc, out_max=100),
                   dict(keep=60, recent=60), dict(act="f32")):
            assert _past_host_checks(call(**ok)), ok


def test_kv_evict_outputs_lie_over_nothing_else(m2):
    """k_out, v_out, acc_out and kept over an input that is not theirs in place, or over one another."""
    good = dict(GOOD, keep=50, recent=10, out_max=60, ko=PTR[11], vo=PTR[12], kept=PTR[13])
    call = _caller(m2.mamba2_kv_evict, ["S", "Hkv", "D", "max_len", "act", "lengths", "kc", "vc", "acc", "keep", "recent",
                                        "out_max", "ko", "vo", "acc_out", "kept"], good)
    kc, vc, acc, lengths = good["kc"], good["vc"], good["acc"], good["lengths"]
    place = dict(ko=kc, vo=vc, acc_out=acc, out_max=100)
    cache, rows, sums = 2 * 8 * 100 * 256, 2 * 8 * 60 * 256, 2 * 8 * 60 * 4
    for bad in [dict(ko=acc), dict(vo=acc + 16), dict(ko=lengths), dict(vo=lengths - rows + 16), dict(acc_out=kc),
                dict(acc_out=vc + cache - 16), dict(acc_out=lengths), dict(acc_out=good["ko"]), dict(acc_out=good["vo"] - sums + 16),
                dict(place, acc_out=kc), dict(place, acc_out=vc + 64)] + \
               [dict(more, kept=at + 4) for more in (dict(), place)
                for at in (kc, vc, acc, lengths, {**good, **more}["ko"], {**good, **more}["vo"], {**good, **more}["acc_out"])]:
        assert call(**bad) == 1, bad
    if NO_GPU:
        for ok in (dict(kept=kc + cache), dict(kept=acc - 2 * 8 * 50 * 4), dict(ko=acc + 2 * 8 * 100 * 4), dict(acc_out=good["ko"] + rows),
                   dict(place, kept=vc + cache), dict(S=0, ko=acc)):
            assert _past_host_checks(call(**ok)), ok


def test_row_strides_past_the_limit_are_refused(m2):
    """2^40 bytes, which the copies' descriptors have room for, and what would wrap when multiplied out."""
    prompt = _caller(m2.mamba2_attn_prompt, SIZES + ["row_start", "lengths", "q", "qs", "k", "v", "kvs", "kc", "vc", "scale",
                                                     "out", "outs", "lse"], GOOD)
    weights = _caller(m2.mamba2_attn_prompt_weights, SIZES + ["row_start", "lengths", "q", "qs", "kc", "scale", "lse", "window",
                                                              "acc", "acc_out"], GOOD)
    for act, size in (("bf16", 2), ("f32", 4)):
        for stride in ((1 << 40) // size, (1 << 62), (1 << 63) - 8):
            for n in ("qs", "kvs", "outs"):
                assert prompt(rows=1, act=act, **{n: stride}) == 2, (n, stride)
            assert weights(rows=1, act=act, qs=stride) == 2
        if NO_GPU:
            assert _past_host_checks(prompt(rows=1, act=act, qs=(1 << 40) // size - 8))
