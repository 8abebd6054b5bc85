"""GPU parity of eviction by accumulated weight (mamba2_kv_evict): what stays is
chosen as the plain reference chooses (oracle/dense_cache.py) and moved bit for
bit, in place or into other caches; and prompts, frames and evictions together."""
import math

import numpy as np
import pytest

from dense_cache_lib import D, Caches, Packed, check_rows, check_sums, dtype
from oracle import dense_cache as dc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m2():
    import full_duplex_speech_gb300 as m2
    m2.load()
    m2.mamba2_device_error()
    return m2


def _done(m2, code=0):
    import torch
    torch.cuda.synchronize()
    assert m2.mamba2_device_error() == code


def _bits(t):
    import torch
    return t.contiguous().view(torch.uint8)


def _numbered(S, Hkv, max_len, act, seed=0):
    """Random caches and sums; NaN bits among them are fine."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randint(-2 ** 31, 2 ** 31, (S, Hkv, max_len, D * (2 if act == "bf16" else 4) // 4), generator=g,
                          device="cuda", dtype=torch.int32) for _ in "kv")
    acc = torch.rand(S, Hkv, max_len, generator=g, device="cuda") ** 4
    return k.view(dtype(act)), v.view(dtype(act)), acc


def _evict(m2, k, v, acc, lengths, keep, recent, out, kept, act, stream=None):
    S, Hkv, max_len = acc.shape
    ko, vo, ao = out
    m2.mamba2_kv_evict(S, Hkv, D, max_len, act, lengths, k, v, acc, keep, recent, ao.shape[2], ko, vo, ao, kept, stream=stream)


def _check(m2, k, v, acc, lens, keep, recent, act, out_max=None):
    """Out of place, then in place."""
    import torch
    S, Hkv, max_len = acc.shape
    lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out_max = out_max or keep
    ko, vo = (torch.full((S, Hkv, out_max, D), -7.0, dtype=dtype(act), device="cuda") for _ in "kv")
    ao, kept = torch.full((S, Hkv, out_max), -7.0, device="cuda"), torch.full((S, Hkv, keep), -7, dtype=torch.int32, device="cuda")
    held = k.clone(), v.clone(), acc.clone()
    _evict(m2, k, v, acc, lengths, keep, recent, (ko, vo, ao), kept, act)
    _done(m2)
    for now, was in zip((k, v, acc), held):
        assert torch.equal(_bits(now), _bits(was))
    place = [t.clone() for t in (k, v, acc)]
    _evict(m2, *place, lengths, keep, recent, place, None, act)
    _done(m2)
    host = acc.cpu().numpy()
    for s, n in enumerate(lens):
        for g in range(Hkv):
            stay = dc.kept(host[s, g, :n].tolist(), keep, recent)
            at = torch.tensor(stay, dtype=torch.long, device="cuda")
            m = len(stay)
            assert kept[s, g, :m].tolist() == stay and torch.all(kept[s, g, m:] == -7)
            for src, moved, own in ((k, ko, place[0]), (v, vo, place[1]), (acc, ao, place[2])):
                assert torch.equal(_bits(moved[s, g, :m]), _bits(src[s, g, at]))
                assert torch.all(moved[s, g, m:] == -7)
                assert torch.equal(_bits(own[s, g, :m]), _bits(src[s, g, at]))
                assert torch.equal(_bits(own[s, g, n if m < n else m:]), _bits(src[s, g, n if m < n else m:]))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("max_len,lens,keep,recent", [
    (1, [1, 0], 1, 0), (5, [5, 4, 3, 0], 3, 1), (64, [64, 33, 1], 63, 63), (300, [300, 299, 151, 150], 150, 0),
    (1025, [1025, 1024, 513], 512, 512), (1500, [1500], 1499, 7), (2500, [2500, 1700], 1, 1), (2500, [2500, 1024], 1, 0),
    (3001, [3001, 2999, 2050, 5], 2049, 750), (7500, [7500], 4096, 750),
])
def test_sizes(m2, act, max_len, lens, keep, recent):
    """Nothing to the last position evicted, none recent, all of them, around the blocks' edges."""
    k, v, acc = _numbered(len(lens), 3, max_len, act, seed=max_len)
    _check(m2, k, v, acc, lens, keep, recent, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("S,Hkv", [(1, 1), (1, 8), (3, 8), (7, 8), (20, 8), (40, 8)])
def test_shares_of_a_row(m2, act, S, Hkv):
    """One to eight CTAs a kv head, by the number of them; a wider cache out than what is kept."""
    rng = np.random.default_rng(S)
    k, v, acc = _numbered(S, Hkv, 400, act, seed=S)
    _check(m2, k, v, acc, rng.integers(0, 401, S).tolist(), 177, 20, act, out_max=190)


@pytest.mark.parametrize("act", ["bf16"])
def test_ties_zeros_and_what_is_not_finite(m2, act):
    import torch
    rng = np.random.default_rng(3)
    lens = [900, 900, 900, 900, 900, 900]
    k, v, acc = _numbered(6, 2, 1000, act, seed=4)
    acc[0] = 0.25                                                          # all alike
    acc[1] = torch.from_numpy(rng.integers(0, 3, (2, 1000))).float().cuda()  # three sizes
    acc[2, :, ::2] = -0.0                                                  # of zeros of both signs
    acc[2, :, 1::2] = 0.0
    acc[3, :, 100:140] = math.nan
    acc[3, :, 200:240] = math.inf
    acc[3, :, 300:340] = -math.inf
    acc[4] = -acc[4]
    acc[5] = torch.from_numpy(rng.integers(1, 4000, (2, 1000)).astype(np.int32)).cuda().view(torch.float32)  # subnormal
    for keep, recent in ((450, 100), (60, 30), (899, 0), (20, 0)):
        _check(m2, k, v, acc, lens, keep, recent, act)


def test_lengths_past_the_cache_are_recorded(m2):
    import torch
    k, v, acc = _numbered(3, 2, 100, "bf16", seed=5)
    held = [t.clone() for t in (k, v, acc)]
    lengths = torch.tensor([101, 80, -1], dtype=torch.int32, device="cuda")
    _evict(m2, k, v, acc, lengths, 40, 10, (k, v, acc), None, "bf16")
    _done(m2, 0x104)
    for now, was in zip((k, v, acc), held):
        assert torch.equal(_bits(now[::2]), _bits(was[::2]))
        assert torch.equal(_bits(now[1, :, 80:]), _bits(was[1, :, 80:]))


def test_sums_in_place_beside_caches_out_of_place(m2):
    """acc_out may be acc by itself where the pitches are alike."""
    import torch
    k, v, acc = _numbered(1, 8, 3000, "bf16", seed=6)
    was = acc.clone()
    ko, vo = (torch.empty_like(k) for _ in "kv")
    lengths = torch.tensor([3000], dtype=torch.int32, device="cuda")
    for _ in range(3):
        acc.copy_(was)
        _evict(m2, k, v, acc, lengths, 1000, 100, (ko, vo, acc), None, "bf16")
        _done(m2)
        for g in range(8):
            stay = torch.tensor(dc.kept(was[0, g].tolist(), 1000, 100), device="cuda")
            assert torch.equal(acc[0, g, :1000], was[0, g, stay])
            assert torch.equal(_bits(ko[0, g, :1000]), _bits(k[0, g, stay]))


def test_another_stream_and_a_replayed_graph(m2):
    import torch
    k, v, acc = _numbered(2, 8, 2000, "bf16", seed=7)
    lengths = torch.tensor([2000, 1500], dtype=torch.int32, device="cuda")
    out = [torch.full((2, 8, 700, D), -7.0, dtype=dtype("bf16"), device="cuda") for _ in "kv"] + \
        [torch.full((2, 8, 700), -7.0, device="cuda")]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _evict(m2, k, v, acc, lengths, 700, 70, out, None, "bf16", stream=side)
    _done(m2)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _evict(m2, k, v, acc, lengths, 700, 70, out, None, "bf16")
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        _done(m2)
        for t, x in zip(out, want):
            assert torch.equal(_bits(t), _bits(x))


def test_offsets_past_32_bits(m2):
    """Caches of more than 2^31 elements, in place: the last head of the last session."""
    import torch
    S, Hkv, max_len = 36, 8, 60000
    k, v = (torch.zeros(S, Hkv, max_len, D, dtype=dtype("bf16"), device="cuda") for _ in "kv")
    acc = torch.zeros(S, Hkv, max_len, device="cuda")
    for t in (k, v):
        t[-1, -1] = torch.randn(max_len, D, device="cuda").to(t.dtype)
    acc[-1, -1] = torch.rand(max_len, device="cuda")
    was = k[-1, -1].clone(), v[-1, -1].clone(), acc[-1, -1].clone()
    lengths = torch.tensor([0] * (S - 1) + [max_len], dtype=torch.int32, device="cuda")
    _evict(m2, k, v, acc, lengths, 20000, 1000, (k, v, acc), None, "bf16")
    _done(m2)
    stay = torch.tensor(dc.kept(was[2].tolist(), 20000, 1000), device="cuda")
    for now, old in zip((k, v, acc), was):
        assert torch.equal(now[-1, -1, :20000], old[stay])
        assert torch.equal(now[-1, -1, 20000:], old[20000:])
    assert not k[:-1].any() and not k[-1, :-1].any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_a_session_from_prompt_to_eviction(m2, act):
    """Prompts of different lengths, their weights, frames that add theirs, an
    eviction in place whenever a session has more than `keep` positions, further
    prompts behind it: each step against fp64 on what the caches hold."""
    import torch
    keep, recent, max_len = 120, 30, 260
    c = Caches(m2, [0, 0, 0], 10, 2, act, max_len, seed=40)
    acc = torch.full((3, 2, max_len), math.nan, device="cuda")
    at = [0, 0, 0]

    def lengths():
        c.before, c.lengths = list(at), torch.tensor(at, dtype=torch.int32, device="cuda")

    def prompt(new, window):
        lengths()
        p = Packed(c, new)
        held = acc.clone()
        p.attend()
        p.weigh(acc, acc, window)
        _done(m2)
        for s, n in enumerate(new):
            b = at[s]
            if n:
                k, v = c.host(s, b + n)
                q = p.q[p.mine(s)].double().cpu().numpy().reshape(n, 10, D)
                lse = p.lse[p.mine(s)].double().cpu().numpy()
                check_rows(p.out[p.mine(s), :10 * D].double().cpu().numpy().reshape(n, 10, D), lse, q, k, v, p.scale, b, act)
                check_sums(acc[s, :, :b + n].double().cpu().numpy(), held[s].double().cpu().numpy(), q, k, p.scale, b, lse,
                           window)
            at[s] += n

    def frames(count):
        need = m2.mamba2_attn_decode_weights_workspace_bytes(3, 10, 2, D, max_len, act)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        for _ in range(count):
            lengths()
            q, k, v = c.values(3, 10, D), c.values(3, 2, D), c.values(3, 2, D)
            out, held = torch.empty(3, 10, D, dtype=dtype(act), device="cuda"), acc.clone()
            m2.mamba2_attn_decode_weights(3, 10, 2, D, max_len, act, c.lengths, q, k, v, c.kc, c.vc, 0.1, out, acc, acc, ws)
            _done(m2)
            for s in range(3):
                kk, vv = c.host(s, at[s] + 1)
                qq = q[s:s + 1].double().cpu().numpy()
                check_rows(out[s:s + 1].double().cpu().numpy(), None, qq, kk, vv, 0.1, at[s], act)
                lse = dc.attend(qq, kk, vv, 0.1, at[s])[1]
                check_sums(acc[s, :, :at[s] + 1].double().cpu().numpy(), held[s].double().cpu().numpy(), qq, kk, 0.1, at[s], lse,
                           1)
                at[s] += 1

    def evict():
        lengths()
        held = [t.clone() for t in (c.kc, c.vc, acc)]
        _evict(m2, c.kc, c.vc, acc, c.lengths, keep, recent, (c.kc, c.vc, acc), None, act)
        _done(m2)
        for s in range(3):
            for g in range(2):
                stay = torch.tensor(dc.kept(held[2][s, g, :at[s]].tolist(), keep, recent), device="cuda", dtype=torch.long)
                for now, was in zip((c.kc, c.vc, acc), held):
                    assert torch.equal(_bits(now[s, g, :len(stay)]), _bits(was[s, g, stay]))
            at[s] = min(at[s], keep)

    prompt([130, 57, 0], 1000)
    frames(2)
    evict()
    prompt([20, 70, 125], 16)
    evict()
    frames(3)
    evict()
    assert at == [120, 120, 120]
