"""GPU parity of the weights that cached positions receive, over packed prompts
(mamba2_attn_prompt_weights) and over single frames (mamba2_attn_decode_weights),
against the plain reference (oracle/dense_cache.py). The bounds stand in
tests/dense_cache_lib.py."""
import math

import numpy as np
import pytest

from dense_cache_lib import D, Caches, Packed, check_rows, check_sums, dtype

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


def _acc(c, seed=0):
    """Sums so far, NaN past each session's positions."""
    import torch
    acc = torch.rand(c.S, c.Hkv, c.max_len, generator=torch.Generator().manual_seed(seed)).cuda() * 3
    for s, b in enumerate(c.before):
        acc[s, :, max(0, b):] = math.nan
    return acc


def _check_prompt(c, p, acc, out, window, sessions=None):
    import torch
    for s in range(c.S) if sessions is None else sessions:
        b, n = c.before[s], p.new[s]
        k, _ = c.host(s, b + n)
        q = p.q[p.mine(s)].double().cpu().numpy().reshape(n, c.Hq, D)
        lse = p.lse[p.mine(s)].double().cpu().numpy()
        check_sums(out[s, :, :b + n].double().cpu().numpy(), acc[s].double().cpu().numpy(), q, k, p.scale, b, lse, window)
        assert torch.all(out[s, :, b + n:] == -7)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(40, 8), (4, 4), (8, 1), (14, 2), (12, 2), (9, 3), (6, 3), (4, 1)])
def test_prompt_head_layouts(m2, act, Hq, Hkv):
    import torch
    c = Caches(m2, [0, 37, 130, 5], Hq, Hkv, act, 300, seed=Hq)
    p = Packed(c, [70, 1, 61, 0], lead=2, tail=3, pad=8)
    p.attend()
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, p.n_rows)
    _done(m2)
    _check_prompt(c, p, acc, out, p.n_rows)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 2, 25, 64, 129, 10000])
def test_prompt_windows(m2, act, window):
    """No rows, one, some, all; sessions shorter than the window, at chunks' edges."""
    import torch
    c = Caches(m2, [0, 0, 127, 128, 300, 64, 7], 10, 2, act, 450, seed=window % 97)
    p = Packed(c, [300, 128, 1, 129, 26, 64, 0])
    p.attend()
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, window)
    _done(m2)
    _check_prompt(c, p, acc, out, window)
    again = acc.clone()
    p.weigh(again, again, window)  # in place: the same bits
    _done(m2)
    for s in range(c.S):
        n = c.before[s] + p.new[s]
        assert torch.equal(again[s, :, :n], out[s, :, :n]) and torch.isnan(again[s, :, n:]).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_rows_and_keys_that_are_not_finite(m2, act):
    """A query that is not finite reaches what it sees, a key its own position."""
    import torch
    c = Caches(m2, [10], 10, 2, act, 200, seed=20)
    p = Packed(c, [150])
    p.attend()
    acc = _acc(c)
    clean, out = torch.full_like(acc, -7.0), torch.full_like(acc, -7.0)
    p.weigh(acc, clean, 1000)
    p.q[30, 2] = math.nan        # head 0, position 40
    c.kc[0, 1, 90, 5] = math.nan
    p.weigh(acc, out, 1000)
    _done(m2)
    assert torch.isnan(out[0, 0, :41]).all() and torch.equal(out[0, 0, 41:], clean[0, 0, 41:])
    other = torch.arange(200, device="cuda") != 90
    assert torch.isnan(out[0, 1, 90]) and torch.equal(out[0, 1, other], clean[0, 1, other])


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_refused_sessions(m2, act):
    import torch
    c = Caches(m2, [10, 95, -3, 60], 10, 2, act, 100, seed=21)
    p = Packed(c, [30, 10, 4, 40])
    p.attend()
    _done(m2, 0x104)
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 100)
    _done(m2, 0x104)
    _check_prompt(c, p, acc, out, 100, sessions=[0, 3])
    assert torch.all(out[1:3] == -7)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_prompt_row_starts_outside_the_rows(m2, act):
    import torch
    c = Caches(m2, [10, 0, 5], 10, 2, act, 100, seed=22)
    p = Packed(c, [30, 10, 20])
    p.attend()
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 100, row_start=torch.tensor([0, 30, 40, 61], dtype=torch.int32, device="cuda"))
    _done(m2, 0x106)
    _check_prompt(c, p, acc, out, 100, sessions=[0, 1])
    assert torch.all(out[2] == -7)


def _frame(m2, c, seed=0):
    import torch
    q, k, v = c.values(c.S, c.Hq, D), c.values(c.S, c.Hkv, D), c.values(c.S, c.Hkv, D)
    out = torch.full((c.S, c.Hq, D), -7.0, dtype=dtype(c.act), device="cuda")
    need = m2.mamba2_attn_decode_weights_workspace_bytes(c.S, c.Hq, c.Hkv, D, c.max_len, c.act)
    ws = torch.full((need + 256,), 0x7F, dtype=torch.uint8, device="cuda")
    return dict(q=q, k=k, v=v, out=out, ws=ws, need=need)


def _decode(m2, c, f, acc, acc_out, scale=D ** -0.5, stream=None):
    m2.mamba2_attn_decode_weights(c.S, c.Hq, c.Hkv, D, c.max_len, c.act, c.lengths, f["q"], f["k"], f["v"], c.kc, c.vc, scale,
                                  f["out"], acc, acc_out, f["ws"], f["need"], stream=stream)


@pytest.mark.parametrize("act,Hq,Hkv,max_len,before", [
    ("bf16", 40, 8, 300, [0, 1, 63, 64, 65, 127, 128, 299]),
    ("f32", 40, 8, 300, [0, 31, 32, 33, 200, 299]),
    ("bf16", 40, 8, 7500, [7499]),          # a cluster of 16 walkers
    ("bf16", 16, 2, 2000, [1999]),          # every walker owns a head
    ("bf16", 40, 8, 1500, [700]),           # walkers without positions
    ("bf16", 4, 4, 160, [40, 130, 0]), ("bf16", 14, 2, 160, [40, 130, 0]), ("bf16", 9, 3, 160, [40, 130, 0]),
    ("f32", 4, 4, 160, [40, 130, 0]), ("f32", 14, 2, 160, [40, 130, 0]), ("f32", 8, 1, 600, [599]),
    ("bf16", 5, 1, 1, [0]), ("f32", 5, 1, 1, [0]),
])
def test_frames(m2, act, Hq, Hkv, max_len, before):
    import torch
    c = Caches(m2, before, Hq, Hkv, act, max_len, seed=30)
    f = _frame(m2, c)
    # the same frame without the weights: the same bits
    kc, vc, plain = c.kc.clone(), c.vc.clone(), torch.empty_like(f["out"])
    need = m2.mamba2_attn_decode_workspace_bytes(c.S, Hq, Hkv, D, max_len, act)
    ws = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    m2.mamba2_attn_decode(c.S, Hq, Hkv, D, max_len, act, c.lengths, f["q"], f["k"], f["v"], kc, vc, D ** -0.5, plain, ws)
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    _decode(m2, c, f, acc, out)
    _done(m2)
    assert torch.equal(f["out"], plain)
    for now, want in ((c.kc, kc), (c.vc, vc)):
        assert torch.equal(now.view(torch.uint8), want.view(torch.uint8))
    assert torch.all(f["ws"][f["need"]:] == 0x7F)
    for s, b in enumerate(before):
        k, v = c.host(s, b + 1)
        q = f["q"][s:s + 1].double().cpu().numpy()
        from oracle import dense_cache as dc
        _, lse, _, _ = dc.attend(q, k, v, D ** -0.5, b)
        check_rows(f["out"][s:s + 1].double().cpu().numpy(), None, q, k, v, D ** -0.5, b, act)
        check_sums(out[s, :, :b + 1].double().cpu().numpy(), acc[s].double().cpu().numpy(), q, k, D ** -0.5, b, lse, 1)
        assert torch.all(out[s, :, b + 1:] == -7)
    again = acc.clone()
    _decode(m2, c, f, again, again)
    _done(m2)
    for s, b in enumerate(before):
        assert torch.equal(again[s, :, :b + 1], out[s, :, :b + 1]) and torch.isnan(again[s, :, b + 1:]).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_frame_of_many_sessions(m2, act):
    """64 sessions of all ages: one walker a session and kv head."""
    import torch
    rng = np.random.default_rng(31)
    before = rng.integers(0, 750, 64).tolist()
    c = Caches(m2, before, 40, 8, act, 750, seed=31)
    f = _frame(m2, c)
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    _decode(m2, c, f, acc, out)
    _done(m2)
    for s in range(0, 64, 7):
        b = before[s]
        gained = out[s, :, :b + 1].double()
        gained[:, :b] -= acc[s, :, :b].double()
        # the weights of a head sum to one: five heads a kv head
        assert torch.all((gained.sum(-1) - 5).abs() < 1e-3)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_frames_refuse_a_length_past_the_cache(m2, act):
    import torch
    c = Caches(m2, [10, 300, -1], 10, 2, act, 300, seed=32)
    f = _frame(m2, c)
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    held = c.kc.clone()
    _decode(m2, c, f, acc, out)
    _done(m2, 0x104)
    assert torch.all(out[1:] == -7) and torch.all(f["out"][1:] == 0)
    assert torch.equal(c.kc[1:].view(torch.uint8), held[1:].view(torch.uint8))
    assert torch.isfinite(out[0, :, :11]).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_two_graphs_share_a_workspace(m2, act):
    """Captured frames of two layers with one workspace, replayed in turn."""
    import torch
    c = [Caches(m2, [200, 31], 10, 2, act, 210, seed=33 + i) for i in range(2)]
    f = [_frame(m2, x) for x in c]
    f[1]["ws"] = f[0]["ws"]
    acc = [_acc(x, i) for i, x in enumerate(c)]
    want, out = [], [torch.full_like(a, -7.0) for a in acc]
    for i in range(2):
        _decode(m2, c[i], f[i], acc[i], out[i])
        torch.cuda.synchronize()
        want.append((f[i]["out"].clone(), out[i].clone()))
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _decode(m2, c[i], f[i], acc[i], out[i])
        graphs.append(g)
    for i in (0, 1, 1, 0):
        f[i]["out"].fill_(-7.0), out[i].fill_(-7.0)
        graphs[i].replay()
    _done(m2)
    for i in range(2):
        assert torch.equal(f[i]["out"], want[i][0]) and torch.equal(out[i], want[i][1])


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0, 2.0 ** -50])
def test_prompt_scales(m2, act, scale):
    import torch
    c = Caches(m2, [20, 0], 10, 2, act, 200, seed=23, spread=0.5)
    p = Packed(c, [150, 60])
    p.attend(scale=scale)
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, 1000)
    _done(m2)
    _check_prompt(c, p, acc, out, 1000)


@pytest.mark.parametrize("before,new,window", [(0, 700, 10000), (500, 40, 33), (0, 1, 1), (3, 530, 64)])
def test_many_sessions_and_long_caches(m2, before, new, window):
    """More (session, kv head)s than CTAs: a CTA takes several tiles of positions, of sessions that end anywhere."""
    import torch
    rng = np.random.default_rng(new)
    S = 90
    b = rng.integers(0, before + 1, S).tolist()
    n = rng.integers(0, new + 1, S).tolist()
    b[0], n[0], b[1], n[2] = before, new, 0, 0
    c = Caches(m2, b, 8, 8, "bf16", 1300, seed=24)
    p = Packed(c, n, lead=1)
    p.attend()
    acc = _acc(c)
    out = torch.full_like(acc, -7.0)
    p.weigh(acc, out, window)
    _done(m2)
    _check_prompt(c, p, acc, out, window, sessions=list(range(0, S, 7)) + [1, 2])
    for s in range(S):
        assert torch.all(out[s, :, b[s] + n[s]:] == -7)
