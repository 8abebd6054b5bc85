"""Dense attention caches that stay bounded over a long session, as cases to
measure and to compare: the attention of whole prompts, packed, with their
append to the caches; the weight that a cached position has received, added up
over a prompt and over single frames; and the eviction of the positions that
received least.

The caches are those of the cached decode: keys and values
[sessions, kv_heads, max_len, 128] in the activation dtype, and beside them
the accumulated weights [sessions, kv_heads, max_len] in fp32. Query head h
reads kv head h // (heads // kv_heads); a new position t of a session with
`before` positions cached sees the positions up to before + t.

`run` computes a case in elementary torch operations where `own` is false,
and through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

D = 128  # head width


def listed():
    common = {"heads": 40, "kv_heads": 8, "act": "bf16"}
    return [
        # One prompt of 24 s of frames in a fresh cache: latency counts.
        dict(common, name="prompt_300", op="prompt", sessions=1, tokens=300, longest=0, ragged=False),
        # Prompts of different lengths packed into one call, some behind a cache, one without new positions.
        dict(common, name="prompt_packed", op="prompt", sessions=9, tokens=750, longest=750, ragged=True),
        # Several sessions catching up by different numbers of positions behind long caches.
        dict(common, name="prompt_catch_up", op="prompt", sessions=6, tokens=75, longest=3001, ragged=True),
        # The prefill of four long histories.
        dict(common, name="prompt_long", op="prompt", sessions=4, tokens=4096, longest=0, ragged=False),
        # Few heads, fp32 activations.
        dict(common, name="prompt_f32", op="prompt", sessions=5, tokens=301, longest=77, ragged=True, heads=12, kv_heads=2,
             act="f32"),
        # What the last positions of prompts look at, before the first eviction.
        dict(common, name="weights_window", op="weights", sessions=6, tokens=2048, longest=0, ragged=True, window=32),
        # What all the positions of long prompts look at.
        dict(common, name="weights_all", op="weights", sessions=4, tokens=4096, longest=0, ragged=False, window=4096),
        # One frame of the longest session, and of 64 sessions of all ages.
        dict(common, name="frame_7500", op="frame", sessions=1, longest=7499, ragged=False),
        dict(common, name="frame_64", op="frame", sessions=64, longest=7499, ragged=True),
        # The same in fp32, few heads.
        dict(common, name="frame_f32", op="frame", sessions=9, longest=2047, ragged=True, heads=12, kv_heads=2, act="f32"),
        # The longest session's cache cut back, and those of 64 sessions of all ages (some short enough to stay whole).
        dict(common, name="evict_7500", op="evict", sessions=1, longest=7500, ragged=False, keep=4096, recent=750),
        dict(common, name="evict_64", op="evict", sessions=64, longest=7500, ragged=True, keep=2048, recent=301),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, kv_heads = rng.choice([(40, 8), (40, 8), (32, 4), (16, 2), (12, 2), (5, 1), (4, 4), (64, 8), (9, 3), (14, 2)])
    case = {"heads": heads, "kv_heads": kv_heads, "act": rng.choice(["bf16", "bf16", "bf16", "f32"]),
            "ragged": rng.random() < 0.7, "op": rng.choice(["prompt", "prompt", "weights", "frame", "evict"])}
    sessions, tokens = spread(1, 64), rng.choice([spread(1, 48), spread(2, 4096)])
    longest = rng.choice([0, spread(1, 7500), spread(250, 7500)])
    if case["op"] in ("frame", "evict"):
        longest = max(longest, 1)
        while sessions * kv_heads * longest * (2 if case["act"] == "f32" else 1) > 64 * 8 * 7500:
            sessions, longest = max(1, sessions * 2 // 3), longest * 9 // 10
        if case["op"] == "evict":
            case["keep"] = spread(1, longest + 1)
            case["recent"] = rng.choice([0, case["keep"], rng.randint(0, case["keep"])])
    else:
        f32 = case["act"] == "f32"
        if f32:  # fp32 is for checks of a few positions
            tokens = min(tokens, 600)
        while (sessions * tokens * heads * (longest + tokens) * (16 if f32 else 1) > 4 * 4096 * 40 * 4096
               or sessions * kv_heads * (longest + tokens) > 64 * 8 * 7500):
            if tokens > 16:
                tokens = tokens * 2 // 3
            else:
                sessions, longest = max(1, sessions * 2 // 3), longest * 9 // 10
        case["tokens"] = tokens
        if case["op"] == "weights":
            case["window"] = rng.choice([tokens, spread(1, tokens)])
    case.update(sessions=sessions, longest=longest)
    return case


def _lengths(case):
    """(positions cached before, new positions) of each session; ragged ones
    differ, with an empty cache and a session without new positions among
    them where there are enough sessions."""
    S, T, L = case["sessions"], case.get("tokens", 1), case["longest"]
    if not case["ragged"]:
        return [L] * S, [T] * S
    rng = random.Random("%d %d %d" % (S, T, L))
    before = [L] + [rng.randint(0, L) for _ in range(S - 1)]
    new = [T] + [rng.randint(1, T) for _ in range(S - 1)]
    if S >= 4:
        before[1] = 0
        if T > 1:
            new[2] = 0
    return before, new


def _generator(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + stream)
    return g


def _values(g, *shape):
    """Keys, queries or values as a model makes them: a few wide channels, and
    positions of different size."""
    x = torch.randn(*shape, generator=g, device="cuda")
    channel = torch.randn(shape[-1], generator=g, device="cuda").mul_(0.5).exp_()
    place = torch.randn(*shape[:-1], 1, generator=g, device="cuda").mul_(0.3).exp_()
    return x.mul_(channel).mul_(place)


def _received(g, *shape):
    """Accumulated weights: most positions little, some far more."""
    return torch.randn(*shape, generator=g, device="cuda").mul_(2.0).exp_().mul_(0.05)


def prepare(case, seed):
    S, Hq, Hkv, op = (case[k] for k in ("sessions", "heads", "kv_heads", "op"))
    act = torch.bfloat16 if case["act"] == "bf16" else torch.float32
    before, new = _lengths(case)
    reach = max(b + (n if op in ("prompt", "weights", "frame") else 0) for b, n in zip(before, new))
    g = _generator(seed, 1)
    st = {"case": dict(case), "max_len": max(1, reach), "before": before, "new": new,
          "lengths": torch.tensor(before, dtype=torch.int32).cuda()}
    M = st["max_len"]
    for name in ("k_cache", "v_cache"):
        x = torch.empty(S, Hkv, M, D, dtype=act, device="cuda")
        for s in range(S):
            x[s] = _values(g, Hkv, M, D).to(act)
        st[name] = x
    if op != "prompt":
        st["acc"] = _received(g, S, Hkv, M)
        st["acc_out"] = torch.zeros(S, Hkv, M, device="cuda")
    if op in ("prompt", "weights"):
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["row_start"] = torch.tensor(starts, dtype=torch.int32).cuda()
        N = st["n_rows"] = starts[-1]
        # the rows of the q | k | v projection, as the layer's matrix product leaves them
        rows = _values(g, N, (Hq + 2 * Hkv) * D).to(act)
        st["rows"] = rows
        st["q"], st["k"], st["v"] = rows[:, :Hq * D], rows[:, Hq * D:(Hq + Hkv) * D], rows[:, (Hq + Hkv) * D:]
        if op == "prompt":
            st["out"] = torch.zeros(N, Hq * D, dtype=act, device="cuda")
            st["lse"] = torch.zeros(N, Hq, device="cuda")
        else:
            # the caches hold the prompts, and the attention left its lse
            _append_plain(st)
            st["lse"] = torch.zeros(N, Hq, device="cuda")
            for s, score, _ in _scores_plain(st, max(new)):
                n = score.shape[2]
                st["lse"][starts[s]:starts[s] + n] = torch.logsumexp(score, -1).permute(2, 0, 1).reshape(n, Hq)
    elif op == "frame":
        st["q"] = _values(g, S, Hq, D).to(act)
        st["k"], st["v"] = _values(g, S, Hkv, D).to(act), _values(g, S, Hkv, D).to(act)
        st["out"] = torch.zeros(S, Hq, D, dtype=act, device="cuda")
    else:
        # compacted into caches of the size that is kept
        keep = case["keep"]
        st["acc_out"] = torch.zeros(S, Hkv, keep, device="cuda")
        st["k_out"], st["v_out"] = (torch.zeros(S, Hkv, keep, D, dtype=act, device="cuda") for _ in "kv")
        st["kept"] = torch.full((S, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    if own:
        import full_duplex_speech_gb300 as m2
        st["m2"] = m2
        if op == "frame":
            need = m2.mamba2_attn_decode_weights_workspace_bytes(S, Hq, Hkv, D, M, case["act"])
            st["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return st


def _append_plain(st):
    """The packed rows' keys and values into the caches behind each session's positions."""
    Hkv, at = st["case"]["kv_heads"], 0
    for s, (b, n) in enumerate(zip(st["before"], st["new"])):
        for cache, rows in (("k_cache", "k"), ("v_cache", "v")):
            st[cache][s, :, b:b + n] = st[rows][at:at + n].view(n, Hkv, D).transpose(0, 1)
        at += n


def _scores_plain(st, window):
    """(session, masked scores [kv heads, heads a kv head, rows, positions] of its last `window` rows, first row)."""
    case = st["case"]
    Hq, Hkv, at = case["heads"], case["kv_heads"], 0
    for s, (b, n) in enumerate(zip(st["before"], st["new"])):
        take = min(n, window)
        if take:
            first = n - take
            q = st["q"][at + first:at + n].float().view(take, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
            k = st["k_cache"][s, :, :b + n].float()
            score = torch.matmul(q.reshape(Hkv, -1, D), k.transpose(1, 2)).mul_(D ** -0.5).view(Hkv, Hq // Hkv, take, b + n)
            hidden = torch.arange(b + n, device="cuda") > (b + first + torch.arange(take, device="cuda"))[:, None]
            yield s, score.masked_fill_(hidden, -math.inf), first
        at += n


def _prompt_plain(st):
    _append_plain(st)
    Hq, starts = st["case"]["heads"], [0]
    for n in st["new"]:
        starts.append(starts[-1] + n)
    for s, score, _ in _scores_plain(st, max(st["new"])):
        n = score.shape[2]
        top = score.amax(-1, keepdim=True)
        weight = score.sub_(top).exp_()
        total = weight.sum(-1, keepdim=True)
        v = st["v_cache"][s, :, :weight.shape[-1]].float()
        o = torch.matmul(weight.view(weight.shape[0], -1, weight.shape[-1]), v).view(*weight.shape[:3], D) / total
        mine = slice(starts[s], starts[s] + n)
        st["out"][mine] = o.permute(2, 0, 1, 3).reshape(n, Hq * D).to(st["out"].dtype)
        st["lse"][mine] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(n, Hq)
    return {k: st[k] for k in ("out", "lse", "k_cache", "v_cache")}


def _weights_plain(st):
    case = st["case"]
    Hq, Hkv, starts = case["heads"], case["kv_heads"], [0]
    for n in st["new"]:
        starts.append(starts[-1] + n)
    for s, (b, n) in enumerate(zip(st["before"], st["new"])):  # a session without new positions keeps its sums
        st["acc_out"][s, :, :b] = st["acc"][s, :, :b]
        st["acc_out"][s, :, b:b + n] = 0
    for s, score, first in _scores_plain(st, case["window"]):
        n = score.shape[2]
        lse = st["lse"][starts[s] + first:starts[s] + first + n].view(n, Hkv, Hq // Hkv).permute(1, 2, 0)[..., None]
        st["acc_out"][s, :, :score.shape[-1]] += score.sub_(lse).exp_().sum((1, 2))
    return st["acc_out"]


def _frame_plain(st):
    case = st["case"]
    S, Hq, Hkv, M = case["sessions"], case["heads"], case["kv_heads"], st["max_len"]
    at = st["lengths"].long()
    every = torch.arange(S, device="cuda")
    st["k_cache"][every, :, at] = st["k"]
    st["v_cache"][every, :, at] = st["v"]
    q = st["q"].float().view(S, Hkv, Hq // Hkv, D)
    score = torch.matmul(q, st["k_cache"].float().transpose(2, 3)).mul_(D ** -0.5)  # [S, Hkv, R, M]
    place = torch.arange(M, device="cuda")
    hidden = (place > at[:, None])[:, None]
    score.masked_fill_(hidden[:, :, None], -math.inf)
    weight = score.sub_(score.amax(-1, keepdim=True)).exp_()
    weight /= weight.sum(-1, keepdim=True)
    values = st["v_cache"].float().masked_fill(hidden[..., None], 0)
    st["out"].copy_(torch.matmul(weight, values).view(S, Hq, D))
    held = (place < at[:, None])[:, None]
    sums = torch.where(held, st["acc"], torch.zeros_like(st["acc"])) + weight.sum(2)
    st["acc_out"].copy_(torch.where(hidden, st["acc_out"], sums))
    return {k: st[k] for k in ("out", "acc_out", "k_cache", "v_cache")}


def _evict_plain(st):
    case = st["case"]
    keep, recent, Hkv = case["keep"], case["recent"], case["kv_heads"]
    for s, n in enumerate(st["before"]):
        if n <= keep:
            which = torch.arange(n, device="cuda").expand(Hkv, n)
        else:
            old = st["acc"][s, :, :n - recent]
            order = torch.sort(old, dim=-1, descending=True, stable=True)[1][:, :keep - recent]
            late = torch.arange(n - recent, n, device="cuda").expand(Hkv, recent)
            which = torch.cat((torch.sort(order, dim=-1)[0], late), -1)
        m = which.shape[1]
        st["kept"][s, :, :m] = which.int()
        st["acc_out"][s, :, :m] = st["acc"][s].gather(1, which)
        for out, cache in (("k_out", "k_cache"), ("v_out", "v_cache")):
            st[out][s, :, :m] = st[cache][s].gather(1, which[..., None].expand(Hkv, m, D))
    return {k: st[k] for k in ("k_out", "v_out", "acc_out", "kept")}


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"prompt": _prompt_plain, "weights": _weights_plain, "frame": _frame_plain, "evict": _evict_plain}[op](st)
    m2, S, Hq, Hkv, M, act = st["m2"], case["sessions"], case["heads"], case["kv_heads"], st["max_len"], case["act"]
    width = (Hq + 2 * Hkv) * D
    if op == "prompt":
        m2.mamba2_attn_prompt(S, st["n_rows"], Hq, Hkv, D, M, act, st["row_start"], st["lengths"], st["q"], width, st["k"],
                              st["v"], width, st["k_cache"], st["v_cache"], D ** -0.5, st["out"], Hq * D, st["lse"])
        return {k: st[k] for k in ("out", "lse", "k_cache", "v_cache")}
    if op == "weights":
        m2.mamba2_attn_prompt_weights(S, st["n_rows"], Hq, Hkv, D, M, act, st["row_start"], st["lengths"], st["q"], width,
                                      st["k_cache"], D ** -0.5, st["lse"], case["window"], st["acc"], st["acc_out"])
        return st["acc_out"]
    if op == "frame":
        m2.mamba2_attn_decode_weights(S, Hq, Hkv, D, M, act, st["lengths"], st["q"], st["k"], st["v"], st["k_cache"],
                                      st["v_cache"], D ** -0.5, st["out"], st["acc"], st["acc_out"], st["workspace"])
        return {k: st[k] for k in ("out", "acc_out", "k_cache", "v_cache")}
    m2.mamba2_kv_evict(S, Hkv, D, M, act, st["lengths"], st["k_cache"], st["v_cache"], st["acc"], case["keep"],
                       case["recent"], case["keep"], st["k_out"], st["v_out"], st["acc_out"], st["kept"])
    return {k: st[k] for k in ("k_out", "v_out", "acc_out", "kept")}


def work(case):
    Hq, Hkv, op = case["heads"], case["kv_heads"], case["op"]
    e = 2 if case["act"] == "bf16" else 4
    total, flops = 4 * case["sessions"], 0
    for before, new in zip(*_lengths(case)):
        reach = before + new
        if op == "prompt" and new:
            total += new * (2 * Hq + 2 * Hkv) * D * e            # rows in, outputs
            total += 2 * new * Hkv * D * e + new * Hq * 4        # the append, lse
            total += 2 * before * Hkv * D * e                    # the cache
            flops += 4 * D * Hq * sum(before + i + 1 for i in range(new))
        elif op == "weights":
            take = min(new, case["window"])
            total += take * Hq * (D * e + 4) + (before + reach) * Hkv * 4
            total += reach * Hkv * D * e if take else 0
            flops += 2 * D * Hq * sum(reach - i for i in range(take))
        elif op == "frame":
            total += 2 * Hq * D * e + 4 * Hkv * D * e            # q, out, the new key and value in and into the cache
            total += 2 * before * Hkv * D * e + (2 * before + 1) * Hkv * 4
            flops += 4 * D * Hq * (before + 1)
        elif op == "evict":
            m = min(before, case["keep"])
            total += Hkv * ((before if before > m else m) * 4 + m * (4 * D * e + 8))
            flops += Hkv * before
    return {"bytes": total, "flops": flops}


def exact(case, seed):
    """The operators' definition in 64 bits, session by session and head by head."""
    st = prepare(case, seed)
    S, Hq, Hkv, op = (case[k] for k in ("sessions", "heads", "kv_heads", "op"))
    R = Hq // Hkv
    before, new = _lengths(case)
    k_all, v_all = st["k_cache"].double(), st["v_cache"].double()
    if op == "evict":
        found = {k: st[k].double() for k in ("k_out", "v_out", "acc_out")}
        found["kept"] = st["kept"].clone()
        for s in range(S):
            n, keep, recent = before[s], case["keep"], case["recent"]
            sums = st["acc"][s, :, :n].tolist()
            for g in range(Hkv):
                stay = list(range(n))
                if n > keep:
                    old = sorted(range(n - recent), key=lambda p: (-sums[g][p], p))[:keep - recent]
                    stay = sorted(old) + stay[n - recent:]
                at = torch.tensor(stay, dtype=torch.long, device="cuda")
                m = len(stay)
                found["kept"][s, g, :m] = at.int()
                found["acc_out"][s, g, :m] = st["acc"][s, g, at].double()
                found["k_out"][s, g, :m], found["v_out"][s, g, :m] = k_all[s, g, at], v_all[s, g, at]
        return found
    if op == "frame":
        out, sums = st["out"].double(), st["acc_out"].double()
        for s in range(S):
            n = before[s]
            k_all[s, :, n], v_all[s, :, n] = st["k"][s].double(), st["v"][s].double()
            for g in range(Hkv):
                a = st["q"][s, g * R:(g + 1) * R].double() @ k_all[s, g, :n + 1].T / math.sqrt(D)
                w = torch.softmax(a, -1)
                out[s, g * R:(g + 1) * R] = w @ v_all[s, g, :n + 1]
                sums[s, g, :n + 1] = w.sum(0)
                sums[s, g, :n] += st["acc"][s, g, :n].double()
        return {"out": out, "acc_out": sums, "k_cache": k_all, "v_cache": v_all}
    if op == "prompt":
        out, lse, at = st["out"].double(), st["lse"].double(), 0
        for s in range(S):
            b, n = before[s], new[s]
            if n == 0:
                continue
            k_all[s, :, b:b + n] = st["k"][at:at + n].double().view(n, Hkv, D).permute(1, 0, 2)
            v_all[s, :, b:b + n] = st["v"][at:at + n].double().view(n, Hkv, D).permute(1, 0, 2)
            q = st["q"][at:at + n].double().view(n, Hq, D)
            late = torch.arange(b + n, device="cuda") > b + torch.arange(n, device="cuda")[:, None]
            for h in range(Hq):
                a = q[:, h] @ k_all[s, h // R, :b + n].T / math.sqrt(D)
                a[late] = -math.inf
                out[at:at + n, h * D:(h + 1) * D] = torch.softmax(a, -1) @ v_all[s, h // R, :b + n]
                lse[at:at + n, h] = torch.logsumexp(a, -1)
            at += n
        return {"out": out, "lse": lse, "k_cache": k_all, "v_cache": v_all}
    sums, at = st["acc_out"].double(), 0
    for s in range(S):
        b, n = before[s], new[s]
        sums[s, :, :b] = st["acc"][s, :, :b].double()
        sums[s, :, b:b + n] = 0
        first = max(0, n - case["window"])
        if n:
            q = st["q"][at + first:at + n].double().view(n - first, Hq, D)
            late = torch.arange(b + n, device="cuda") > b + torch.arange(first, n, device="cuda")[:, None]
            for h in range(Hq):
                a = q[:, h] @ k_all[s, h // R, :b + n].T / math.sqrt(D)
                a -= st["lse"][at + first:at + n, h].double()[:, None]
                a[late] = -math.inf
                sums[s, h // R, :b + n] += a.exp().sum(0)
        at += n
    return sums
