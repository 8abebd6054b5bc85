"""The paged 8-bit key/value cache of the hybrid model's attention layers: the
append of new positions (with the rotation of keys and queries) and the
attention that reads the cache, as cases to measure and to compare.

A session's positions live in pages of `page` positions, listed by its row of
a page table. Keys and values are held in e4m3, with one fp32 scale for each
block of 16 positions and kv head:

    scale = max |block| / 448,   code = e4m3(value * (448 / max |block|)).

The positions of the block that is still open are also held in fp32 (the
tail), so the block is always quantised from its exact values and the cache
does not depend on how the positions were split over calls.

`run` computes a case in elementary torch operations where `own` is false,
and through the package's entry points where it is true.
"""
import math
import random

import torch

own = False

D = 128          # head width
BLOCK = 16       # positions that share a scale
TINY = 2.0 ** -100  # the least block maximum a scale is made of
E4M3_MAX = 448.0


def listed():
    common = {"heads": 40, "kv_heads": 8, "act": "bf16"}
    return [
        # One frame of one session early in a conversation: latency alone counts.
        dict(common, name="append_frame", op="append", sessions=1, tokens=1, longest=300, ragged=False, page=64,
             rot=128, interleaved=False, queries=True),
        # One frame for 64 sessions of all ages; the layers of the model itself rotate nothing.
        dict(common, name="append_frame_64", op="append", sessions=64, tokens=1, longest=7500, ragged=True, page=64,
             rot=0, interleaved=False, queries=False),
        # Prompts of different lengths appended in fp32 behind open blocks, small pages, half the width rotated.
        dict(common, name="append_prompts_f32", op="append", sessions=5, tokens=301, longest=77, ragged=True, page=16,
             rot=64, interleaved=True, queries=True, act="f32"),
        # The prefill of four long histories.
        dict(common, name="append_long", op="append", sessions=4, tokens=4096, longest=0, ragged=False, page=64,
             rot=128, interleaved=False, queries=True),
        # One frame of one session over a short cache, and over the longest one a session reaches.
        dict(common, name="attend_frame", op="attend", causal=True, sessions=1, tokens=1, longest=300, ragged=False,
             page=64),
        dict(common, name="attend_frame_7500", op="attend", causal=True, sessions=1, tokens=1, longest=7499,
             ragged=False, page=64),
        # One frame for 64 sessions of all ages.
        dict(common, name="attend_frame_64", op="attend", causal=True, sessions=64, tokens=1, longest=7499,
             ragged=True, page=64),
        # Few heads, fp32 activations, small pages.
        dict(common, name="attend_frame_f32", op="attend", causal=True, sessions=9, tokens=1, longest=2047,
             ragged=True, page=16, heads=12, kv_heads=2, act="f32"),
        # Several sessions catching up by different numbers of positions.
        dict(common, name="attend_catch_up", op="attend", causal=True, sessions=6, tokens=75, longest=3001,
             ragged=True, page=32),
        # The prefill of four long histories.
        dict(common, name="attend_prefill", op="attend", causal=True, sessions=4, tokens=4096, longest=0,
             ragged=False, page=64),
        # Cross attention to an encoder's states of another length: many rows, and one row for each session.
        dict(common, name="cross_300_to_1500", op="attend", causal=False, sessions=2, tokens=300, longest=1500,
             ragged=True, page=128),
        dict(common, name="cross_frame_64", op="attend", causal=False, sessions=64, tokens=1, longest=251,
             ragged=True, page=16, heads=32, kv_heads=4),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    heads, kv_heads = rng.choice([(40, 8), (40, 8), (32, 4), (16, 2), (12, 2), (5, 1), (4, 4), (64, 8)])
    case = {"heads": heads, "kv_heads": kv_heads, "act": rng.choice(["bf16", "bf16", "bf16", "f32"]),
            "page": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.7}
    case["op"] = rng.choice(["append", "attend", "attend"])
    sessions, tokens = spread(1, 64), rng.choice([1, spread(2, 4096)])
    longest = rng.choice([0, spread(1, 7500), spread(250, 7500)])
    if case["op"] == "append":
        rot = rng.choice([0, 32, 64, 128])
        case.update(rot=rot, interleaved=rng.random() < 0.5, queries=rot > 0 and rng.random() < 0.7)
        most = 4 * 4096 * 56  # rows of heads that the largest listed append takes
        while sessions * tokens * (heads + 2 * kv_heads) * (2 if case["act"] == "f32" else 1) > most:
            sessions, tokens = max(1, sessions // 2), max(1, tokens * 2 // 3)
    else:
        case["causal"] = rng.random() < 0.7
        if not case["causal"]:
            longest = max(longest, 1)
        f32 = case["act"] == "f32"
        if f32:  # fp32 is for checks of a few positions
            tokens = min(tokens, 48)
        while (sessions * tokens * heads * (longest + tokens) * (8 if f32 else 1) > 4 * 4096 * 40 * 4096
               or sessions * kv_heads * (longest + tokens) > 64 * 8 * 7500):
            if tokens > 16:
                tokens = tokens * 2 // 3
            else:
                sessions, longest = max(1, sessions * 2 // 3), longest * 9 // 10
    case.update(sessions=sessions, tokens=tokens, longest=longest)
    return case


def _lengths(case):
    """(positions cached before, new positions) of each session; ragged ones
    differ, with an empty cache and a session without new positions among
    them where there are enough sessions."""
    S, T, L = case["sessions"], case["tokens"], case["longest"]
    if not case["ragged"]:
        return [L] * S, [T] * S
    rng = random.Random("%d %d %d" % (S, T, L))
    before = [L] + [rng.randint(0, L) for _ in range(S - 1)]
    new = [T] + [rng.randint(1, T) for _ in range(S - 1)]
    if S >= 4:
        before[1], new[2] = 0, 0
    return before, new


def _generator(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 16 + stream)
    return g


def _values(g, *shape):
    """Keys or values as a model makes them: a few wide channels, and
    positions of different size."""
    x = torch.randn(*shape, generator=g, device="cuda")
    channel = torch.randn(shape[-1], generator=g, device="cuda").mul_(0.5).exp_()
    place = torch.randn(*shape[:-1], 1, generator=g, device="cuda").mul_(0.3).exp_()
    return x.mul_(channel).mul_(place)


def _dtype(case):
    return torch.bfloat16 if case["act"] == "bf16" else torch.float32


def prepare(case, seed):
    S, T, Hq, Hkv, ps = (case[k] for k in ("sessions", "tokens", "heads", "kv_heads", "page"))
    act = _dtype(case)
    before, new = _lengths(case)
    reach = max(b + n for b, n in zip(before, new))
    columns = max(1, -(-reach // ps))
    used = [-(-(b + n) // ps) for b, n in zip(before, new)]
    pages = max(1, sum(used))
    order = list(range(pages))
    random.Random(int(seed)).shuffle(order)
    table = torch.full((S, columns), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    st = {"case": dict(case), "pages": pages, "columns": columns, "table": table.cuda(),
          "lengths": torch.tensor(before, dtype=torch.int32).cuda(), "n_new": torch.tensor(new, dtype=torch.int32).cuda()}
    g = _generator(seed, 1)
    if case["op"] == "append":
        # one page more than the table lists: the plain form's place for rows that are not there
        for name in ("k", "v"):
            st[name + "_pages"] = torch.zeros(pages + 1, Hkv, ps, D, dtype=torch.uint8, device="cuda")
            st[name + "_scales"] = torch.ones(pages + 1, Hkv, ps // BLOCK, device="cuda")
            st[name + "_tail"] = _values(g, S, Hkv, BLOCK, D)
            st[name + "_tail_out"] = torch.zeros(S, Hkv, BLOCK, D, device="cuda")
        # the rows of the q | k | v projection, as the layer's matrix product leaves them
        rows = _values(g, S * T, (Hq + 2 * Hkv) * D).to(act)
        st["rows"] = rows
        st["q"], st["k"], st["v"] = rows[:, :Hq * D], rows[:, Hq * D:(Hq + Hkv) * D], rows[:, (Hq + Hkv) * D:]
        if case["rot"]:
            half = case["rot"] // 2
            angle = torch.arange(max(1, reach), dtype=torch.float64)[:, None] * \
                10000.0 ** -(torch.arange(half, dtype=torch.float64) / half)
            st["cos"], st["sin"] = angle.cos().float().cuda(), angle.sin().float().cuda()
        if case["queries"]:
            st["q_out"] = torch.zeros(S * T, Hq * D, dtype=act, device="cuda")
    else:
        for name in ("k", "v"):
            x = _values(g, pages, Hkv, ps // BLOCK, BLOCK * D)
            top = x.abs().amax(-1, keepdim=True).clamp_min(TINY)
            st[name + "_scales"] = (top / E4M3_MAX)[..., 0]
            st[name + "_pages"] = x.mul_(E4M3_MAX / top).to(torch.float8_e4m3fn).view(torch.uint8).view(pages, Hkv, ps, D)
            del x
        st["q"] = _values(g, S * T, Hq * D).to(act)
        st["out"] = torch.zeros(S * T, Hq * D, dtype=act, device="cuda")
    if own:
        import full_duplex_speech_gb300 as m2
        st["m2"] = m2
        st["cache"] = m2.kv_cache(S, Hkv, ps, pages, columns, st["table"], st["k_pages"], st["v_pages"], st["k_scales"],
                                  st["v_scales"], st.get("k_tail"), st.get("v_tail"), st.get("k_tail_out"),
                                  st.get("v_tail_out"), act=case["act"])
        if case["op"] == "append":
            st["rope"] = m2.rope(case["rot"], max(1, reach), st["cos"], st["sin"], case["interleaved"]) if case["rot"] else None
        else:
            need = m2.mamba2_attn_paged_workspace_bytes(st["cache"], T, Hq)
            st["workspace"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    return st


def _rotated(x, cos, sin, interleaved):
    """x [..., D] in fp32 with its first 2 x cos.shape[-1] dims rotated."""
    half = cos.shape[-1]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    u, w = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., 2 * half:]), -1)


def _append_outputs(st):
    out = {k: st[k] for k in ("k_tail_out", "v_tail_out")}
    for name in ("k", "v"):
        out[name + "_pages"] = st[name + "_pages"][:-1].view(torch.float8_e4m3fn)
        out[name + "_scales"] = st[name + "_scales"][:-1]
    if st["case"]["queries"]:
        out["q_out"] = st["q_out"]
    return out


def _append_plain(st):
    case = st["case"]
    S, T, Hq, Hkv, ps = (case[k] for k in ("sessions", "tokens", "heads", "kv_heads", "page"))
    before, new = st["lengths"].long(), st["n_new"].long()
    step = torch.arange(T, device="cuda")
    place = before[:, None] + step  # [S, T]
    k, v = st["k"].float().view(S, T, Hkv, D), st["v"].float().view(S, T, Hkv, D)
    if case["rot"]:
        at = place.clamp_max(st["cos"].shape[0] - 1)
        cos, sin = st["cos"][at][:, :, None], st["sin"][at][:, :, None]
        k = _rotated(k, cos, sin, case["interleaved"])
        if case["queries"]:
            q = _rotated(st["q"].float().view(S, T, Hq, D), cos, sin, case["interleaved"]).to(st["q"].dtype)
            there = (step < new[:, None])[:, :, None, None]
            st["q_out"].copy_(torch.where(there, q, st["q_out"].view(S, T, Hq, D)).view(S * T, Hq * D))
    # the blocks that the new positions touch, from the start of the open one
    open_rows = before % BLOCK
    blocks = -(-(BLOCK - 1 + T) // BLOCK)
    row = torch.arange(blocks * BLOCK, device="cuda")
    end = open_rows + new
    written = (row < end[:, None]) & (new > 0)[:, None]  # [S, rows]
    from_new = (row - open_rows[:, None]).clamp(0, T - 1)
    is_old = (row < open_rows[:, None])[:, :, None, None]
    position = (before - open_rows)[:, None] + row
    column = (position // ps).clamp_max(st["columns"] - 1)
    page = torch.where(written, st["table"].gather(1, column).long(), st["pages"])
    first = row[::BLOCK]
    for name, x in (("k", k), ("v", v)):
        tail = st[name + "_tail"].transpose(1, 2)  # [S, BLOCK, Hkv, D]
        fresh = x.gather(1, from_new[:, :, None, None].expand(S, row.numel(), Hkv, D))
        kept = tail[:, row.clamp_max(BLOCK - 1)]
        w = torch.where(is_old, kept, fresh) * (row < end[:, None])[:, :, None, None]
        w = w.view(S, blocks, BLOCK, Hkv, D)
        top = w.abs().amax((2, 4)).clamp_min(TINY)  # [S, blocks, Hkv]
        codes = (w * (E4M3_MAX / top)[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st[name + "_pages"][page, :, position % ps] = codes.view(S, row.numel(), Hkv, D)
        st[name + "_scales"][page[:, first], :, (position % ps)[:, first] // BLOCK] = top / E4M3_MAX
        last = (end // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
        rows = w.view(S, row.numel(), Hkv, D).gather(
            1, last.clamp_max(row.numel() - 1)[:, :, None, None].expand(S, BLOCK, Hkv, D)).transpose(1, 2)
        stays = (torch.arange(BLOCK, device="cuda") < (end % BLOCK)[:, None])[:, None, :, None]
        st[name + "_tail_out"].copy_(torch.where(stays, rows, st[name + "_tail_out"]))
    return _append_outputs(st)


def _attend_plain(st):
    case = st["case"]
    S, T, Hq, Hkv, ps = (case[k] for k in ("sessions", "tokens", "heads", "kv_heads", "page"))
    R, L = Hq // Hkv, st["columns"] * ps
    before, new = st["lengths"].long(), st["n_new"].long()
    table = st["table"].long().clamp_min(0)

    def cached(name):
        codes = st[name + "_pages"][table].view(torch.float8_e4m3fn).float()  # [S, columns, Hkv, ps, D]
        codes = codes.view(S, -1, Hkv, ps // BLOCK, BLOCK, D) * st[name + "_scales"][table][..., None, None]
        return codes.view(S, -1, Hkv, ps, D).transpose(1, 2).reshape(S, Hkv, L, D)

    q = st["q"].float().view(S, T, Hkv, R, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, T * R, D)
    score = torch.matmul(q, cached("k").transpose(2, 3)).mul_(D ** -0.5).view(S, Hkv, T, R, L)
    key = torch.arange(L, device="cuda")
    if case["causal"]:
        seen = key <= (before[:, None] + torch.arange(T, device="cuda"))[:, :, None]  # [S, T, L]
    else:
        seen = (key < before[:, None, None]).expand(S, T, L)
    hidden = ~seen[:, None, :, None]
    score.masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)  # a row that sees nothing gets zeros
    weight = score.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(weight.view(S, Hkv, T * R, L), cached("v")).view(S, Hkv, T, R, D) / total
    o = o.permute(0, 2, 1, 3, 4).reshape(S, T, Hq * D).to(st["out"].dtype)
    there = (torch.arange(T, device="cuda") < new[:, None])[:, :, None]
    return torch.where(there, o, st["out"].view(S, T, Hq * D)).view(S * T, Hq * D)


def run(st):
    case = st["case"]
    if not own:
        return _append_plain(st) if case["op"] == "append" else _attend_plain(st)
    m2, T, Hq, Hkv = st["m2"], case["tokens"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        width = (Hq + 2 * Hkv) * D
        if case["queries"]:
            m2.mamba2_kv_append(st["cache"], T, st["lengths"], st["n_new"], st["k"], st["v"], width, st["rope"], Hq, st["q"],
                                width, st["q_out"], Hq * D)
        else:
            m2.mamba2_kv_append(st["cache"], T, st["lengths"], st["n_new"], st["k"], st["v"], width, st["rope"])
        return _append_outputs(st)
    m2.mamba2_attn_paged(st["cache"], T, Hq, case["causal"], st["lengths"], st["n_new"], st["q"], Hq * D, D ** -0.5,
                         st["out"], Hq * D, st["workspace"])
    return st["out"]


def work(case):
    Hq, Hkv, ps = case["heads"], case["kv_heads"], case["page"]
    e = 2 if case["act"] == "bf16" else 4
    total, flops = 0, 0
    for before, new in zip(*_lengths(case)):
        if case["op"] == "append":
            if not new:
                total += before % BLOCK * Hkv * 2 * D * 4 * 2  # the tail, in and out
                continue
            opened, end = before % BLOCK, before % BLOCK + new
            total += opened * Hkv * 2 * D * 4 + end % BLOCK * Hkv * 2 * D * 4  # the tail in, the tail out
            total += new * Hkv * 2 * D * e + end * Hkv * 2 * D                 # the new rows, the codes
            total += -(-end // BLOCK) * Hkv * 2 * 4 + -(-end // ps) * 4        # scales, page numbers
            total += new * case["rot"] * 4 + (2 * new * Hq * D * e if case["queries"] else 0)
            flops += 6 * new * D * (Hq * case["queries"] + 2 * Hkv)
        elif new:
            reach = before + new if case["causal"] else before
            pairs = sum(before + i + 1 for i in range(new)) if case["causal"] else new * before
            total += 2 * new * Hq * D * e + reach * Hkv * 2 * D + -(-reach // BLOCK) * Hkv * 2 * 4 + -(-reach // ps) * 4
            flops += 4 * D * Hq * pairs
    return {"bytes": total + 8 * case["sessions"], "flops": flops}


def exact(case, seed):
    """The operators' definition in 64 bits, session by session."""
    st = prepare(case, seed)
    T, Hq, Hkv, ps = (case[k] for k in ("tokens", "heads", "kv_heads", "page"))
    S, R = case["sessions"], Hq // Hkv
    before, new = _lengths(case)
    table = st["table"].tolist()
    if case["op"] == "append":
        found = {n: st[n].double() for n in ("k_tail_out", "v_tail_out")}
        for n in ("k", "v"):
            found[n + "_pages"] = st[n + "_pages"][:-1].view(torch.float8_e4m3fn).double()
            found[n + "_scales"] = st[n + "_scales"][:-1].double()
        if case["queries"]:
            found["q_out"] = st["q_out"].double()

        def turned(x, places):  # [T', heads, D]
            half = case["rot"] // 2
            z = x.clone()
            c, s = st["cos"][places].double()[:, None], st["sin"][places].double()[:, None]
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
                z[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
                z[..., b] = x[..., a] * s[..., i] + x[..., b] * c[..., i]
            return z

        for s in range(S):
            b, n = before[s], new[s]
            lo = b // BLOCK * BLOCK
            places = torch.arange(b, b + n, device="cuda")
            mine = slice(s * T, s * T + n)
            if case["queries"] and n:
                found["q_out"][mine] = turned(st["q"][mine].double().view(n, Hq, D), places).view(n, Hq * D)
            for name in ("k", "v"):
                x = st[name][mine].double().view(n, Hkv, D)
                if name == "k" and case["rot"] and n:
                    x = turned(x, places)
                x = torch.cat((st[name + "_tail"][s, :, :b - lo].double().transpose(0, 1), x))  # from position lo on
                left = (b + n) % BLOCK
                if left:
                    found[name + "_tail_out"][s, :, :left] = x[-left:].transpose(0, 1)
                for p in range(0, x.shape[0] if n else 0, BLOCK):
                    block = x[p:p + BLOCK]  # [rows, Hkv, D]
                    size = block.abs().amax((0, 2)).clamp_min(TINY)
                    page, slot = table[s][(lo + p) // ps], (lo + p) % ps
                    found[name + "_scales"][page, :, slot // BLOCK] = size / E4M3_MAX
                    codes = (block / size[None, :, None] * E4M3_MAX).float().to(torch.float8_e4m3fn).double()
                    found[name + "_pages"][page, :, slot:slot + block.shape[0]] = codes.transpose(0, 1)
        return found
    out = st["out"].double().view(S, T, Hq, D)
    for s in range(S):
        n = new[s]
        reach = before[s] + n if case["causal"] else before[s]
        if not n or not reach:
            continue
        use = table[s][:-(-reach // ps)]

        def whole(name):
            z = st[name + "_pages"][use].view(torch.float8_e4m3fn).double()
            z = z * st[name + "_scales"][use].double().repeat_interleave(BLOCK, -1)[..., None]
            return z.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :reach]

        k, v = whole("k"), whole("v")
        q = st["q"].view(S, T, Hq, D)[s, :n].double()
        late = torch.arange(reach, device="cuda") > before[s] + torch.arange(n, device="cuda")[:, None]
        for h in range(Hq):
            a = q[:, h] @ k[h // R].T / math.sqrt(D)
            if case["causal"]:
                a[late] = -math.inf
            out[s, :n, h] = torch.softmax(a, -1) @ v[h // R]
    return out.view(S * T, Hq * D)
