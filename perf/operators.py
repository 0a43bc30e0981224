"""The frame cache's operators as cases to be timed: writing K/V rows into a cache held in 4 or 8
bits and reading them back, and attention of a few query rows, or of whole frames, over it.

A cached number is code * s with one scale s per 16 channels of a token.  The scale is a byte b,
s = (8 + b % 8) / 8 * 2^(b // 8 - 16).
  4 bits  s is the smallest scale with 7.5 s >= max|x|, code = clamp(round(x / s), -7, 7)
  8 bits  s is the smallest power of two with 127.5 s >= max|x|, code = clamp(round(x / s), -127, 127)
(round half to even).  Pool: uint8 [pages][heads][page bytes]; a page holds the K codes, the K scales,
the V codes and the V scales of `page` tokens of one head, d = 64.  Codes sit in 16-bit units, four
4-bit codes (code + 8, lowest nibble first) or two 8-bit codes (a: magnitude in bits 0-6, sign in bit
15; b: magnitude in bits 8-14, sign in bit 7), and units in pairs (little endian):
  K   [token][...]         a pair's first unit holds even channels, its second the odd ones after them
  V   [token pair][...]    a pair's first unit holds the even token's channels, its second the odd one's
  K scales [token][4 blocks], V scales [token pair][4 blocks][even, odd token]
"""
import torch

own = False

HD = 64


def listed():
    return [
        # one new frame of the 1 374-token workload joins 16 cached ones (streaming, once a layer)
        dict(name="write_frame_4bit", op="write", bits=4, dtype="bf16", scenes=1, heads=16, page=128, tokens=23358,
             new=1374, ragged=False),
        # three f32 scenes grow by different odd amounts, one of them by nothing
        dict(name="write_ragged_8bit_f32", op="write", bits=8, dtype="f32", scenes=3, heads=6, page=32, tokens=3001,
             new=333, ragged=True),
        # a 128-frame scene is cached at once
        dict(name="write_128_frames_4bit", op="write", bits=4, dtype="bf16", scenes=1, heads=16, page=128,
             tokens=175872, new=175872, ragged=False),
        # 64 cached frames handed back in bf16 to a layer that wants plain rows
        dict(name="read_64_frames_4bit", op="read", bits=4, dtype="bf16", scenes=1, heads=16, page=128, tokens=90000,
             new=87936, ragged=False),
        # ragged odd ranges in f32 from small pages
        dict(name="read_ragged_8bit_f32", op="read", bits=8, dtype="f32", scenes=5, heads=4, page=16, tokens=4099,
             new=2047, ragged=True),
        # one camera token against two frames: the smallest call, where latency counts
        dict(name="attend_1_row_2_frames_4bit", op="attend", bits=4, scenes=1, heads=16, group=1, page=128,
             tokens=2748, rows=1, frame=0, ragged=False),
        # the five special tokens of a new frame against 1 024 cached frames: the longest cache
        dict(name="attend_5_rows_1024_frames_4bit", op="attend", bits=4, scenes=1, heads=16, group=1, page=128,
             tokens=1406976, rows=5, frame=0, ragged=False),
        # a server's batch: scenes of every length (an empty one, one of a single token), grouped heads
        dict(name="attend_ragged_scenes_8bit", op="attend", bits=8, scenes=13, heads=4, group=4, page=64, tokens=40001,
             rows=3, frame=0, ragged=True),
        # a few dozen query points, token-causal among themselves
        dict(name="attend_45_rows_4bit", op="attend", bits=4, scenes=2, heads=8, group=1, page=32, tokens=30011,
             rows=45, frame=1, ragged=True),
        # a whole new frame against 64 cached frames (itself among them)
        dict(name="attend_frame_64_frames_4bit", op="attend", bits=4, scenes=1, heads=16, group=1, page=128,
             tokens=87936, rows=1374, frame=1374, ragged=False),
        # a whole new frame, 8 bits, two scenes of different ages
        dict(name="attend_frame_ragged_8bit", op="attend", bits=8, scenes=3, heads=8, group=1, page=128,
             tokens=21984, rows=1374, frame=1374, ragged=True),
        # eight frames at once, each sees itself and the earlier ones
        dict(name="attend_8_frames_causal_4bit", op="attend", bits=4, scenes=1, heads=16, group=1, page=128,
             tokens=10992, rows=10992, frame=1374, ragged=False),
    ]


def _log(rng, lo, hi):
    import math
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    bits = rng.choice([4, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    scenes = rng.choice([1, 1, 2, 3, 7])
    ragged = scenes > 1
    if op != "attend":
        new = _log(rng, 1, 60000)
        return dict(op=op, bits=bits, dtype=rng.choice(["bf16", "f32"]), scenes=scenes, heads=rng.randint(1, 16),
                    page=page, tokens=new + _log(rng, 1, 20000), new=new, ragged=ragged)
    heads, group = rng.choice([(16, 1), (3, 1), (8, 2), (2, 5)])
    rows = _log(rng, 1, 1600)
    top = min(400000, int(1.2e8 / (rows * scenes)))
    tokens = max(rows, _log(rng, 64, max(65, top)))
    return dict(op=op, bits=bits, scenes=scenes, heads=heads, group=group, page=page, tokens=tokens, rows=rows,
                frame=rng.choice([0, 0, 1, 77, 1374]), ragged=ragged)


# ------------------------------------------------------------------------------ the inputs


def _lens(case):
    """Tokens of every scene, the new ones included: the first has them all, then an empty scene, one of one token, and others."""
    some = [case["tokens"], 0, 1] + [1 + (case["tokens"] * (37 * i % 101)) // 101 for i in range(3, case["scenes"])]
    return some[:case["scenes"]] if case["ragged"] else [case["tokens"]] * case["scenes"]


def _news(case):
    """New tokens (query rows) of every scene, never more than it has where they are written or read."""
    most = case["rows"] if case["op"] == "attend" else case["new"]
    if not case["ragged"]:
        return [most] * case["scenes"]
    some = [most] + [1 + (most * (53 * i % 89)) // 89 for i in range(1, case["scenes"])]
    some = [min(a, most) for a in some]
    return some if case["op"] == "attend" else [min(a, b) for a, b in zip(some, _lens(case))]


def _page_bytes(page, bits):
    return page * 2 * (HD * bits // 8 + 4)


def _rows(gen, shape, dtype, spread):
    """Rows as a projection makes them: Gaussian, each channel with a width of its own, a few rows large."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    x *= torch.exp(spread * torch.randn(shape[-1], generator=gen, device="cuda"))
    x *= 1 + 3 * (torch.rand(shape[:-1] + (1,), generator=gen, device="cuda") < 0.01)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    scenes, heads, page, bits = case["scenes"], case["heads"], case["page"], case["bits"]
    lens, news = _lens(case), _news(case)
    need = [-(-n // page) for n in lens]
    cols = max(1, max(need)) + 1
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((scenes, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    # pages hold whatever was in them before
    pool = torch.randint(0, 256, (pages, heads, _page_bytes(page, bits)), generator=gen, device="cuda",
                         dtype=torch.uint8)
    state = dict(case=case, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 news=torch.tensor(news, dtype=torch.int32, device="cuda"))
    if case["op"] == "write":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        for name, spread in (("k", 0.6), ("v", 0.3)):
            state[name] = _rows(gen, (scenes * heads, case["new"], HD), dt, spread)
        return state
    # fill the cache, 2^17 tokens at a time
    for i, n in enumerate(lens):
        for lo in range(0, n, 1 << 17):
            m = min(1 << 17, n - lo)
            k = _rows(gen, (heads, m, HD), torch.bfloat16, 0.6)
            v = _rows(gen, (heads, m, HD), torch.bfloat16, 0.3)
            t = torch.arange(lo, lo + m, device="cuda")
            _store(pool, table[i, t // page].long(), t % page, k.transpose(0, 1), v.transpose(0, 1), page, bits)
    if case["op"] == "attend":
        state["q"] = _rows(gen, (scenes * heads * case["group"], case["rows"], HD), torch.bfloat16, 0.2)
    else:
        state["start"] = (state["lens"] - state["news"]) // 2
    return state


# ------------------------------------------------------------------------------ plain form: the cache


def _scale_values(device):
    b = torch.arange(256, device=device)
    return (8 + b % 8).double() / 8 * torch.exp2((b // 8 - 16).double())


def _quantise(x, bits):
    """Codes [..., 64] (int32) and scale bytes [..., 4] of rows x [..., 64]."""
    s = _scale_values(x.device)
    y = x.double().unflatten(-1, (4, 16))
    most = y.abs().amax(-1)
    if bits == 4:
        byte = torch.searchsorted(7.5 * s, most).clamp(max=255)
        top = 7
    else:
        byte = 8 * torch.searchsorted(127.5 * s[::8].contiguous(), most).clamp(max=31)
        top = 127
    code = (y / s[byte][..., None]).round().clamp(-top, top)
    return code.to(torch.int32).flatten(-2), byte.to(torch.uint8)


def _units(code, bits):
    """16-bit units (as int32) of codes [..., n]: four 4-bit codes or two 8-bit ones each."""
    if bits == 4:
        c = (code + 8).unflatten(-1, (-1, 4))
        return c[..., 0] | c[..., 1] << 4 | c[..., 2] << 8 | c[..., 3] << 12
    c = code.unflatten(-1, (-1, 2))
    m, g = c.abs(), (c < 0).int()
    return m[..., 0] | g[..., 0] << 15 | m[..., 1] << 8 | g[..., 1] << 7


def _codes(unit, bits):
    """Codes (f32) of 16-bit units, the inverse of _units."""
    if bits == 4:
        return torch.stack([(unit >> 4 * j & 15) - 8 for j in range(4)], -1).flatten(-2).float()
    a = (unit & 127) * (1 - 2 * (unit >> 15 & 1))
    b = (unit >> 8 & 127) * (1 - 2 * (unit >> 7 & 1))
    return torch.stack([a, b], -1).flatten(-2).float()


def _parts(pool, page, bits):
    """The four parts of every page, viewed as [pages][heads][...]."""
    db = HD * bits // 8
    p, h, _ = pool.shape
    kc, ks, vc, vs = pool.split([page * db, page * 4, page * db, page * 4], -1)
    return (kc.unflatten(-1, (page, db)), ks.unflatten(-1, (page, 4)),
            vc.unflatten(-1, (page // 2, db // 2, 2, 2)), vs.unflatten(-1, (page // 2, 4, 2)))


def _bytes(unit):
    return torch.stack([unit & 255, unit >> 8 & 255], -1).to(torch.uint8)


def _store(pool, pid, slot, k, v, page, bits):
    """Quantise rows k, v [tokens][heads][64] into page pid[t], slot slot[t]."""
    kc, ks, vc, vs = _parts(pool, page, bits)
    per = 16 // bits  # codes of one unit
    code, byte = _quantise(k, bits)
    # a pair of units: even channels, then odd channels, of 2 * per consecutive ones
    u = _units(code.unflatten(-1, (-1, per, 2)).transpose(-1, -2).flatten(-3), bits)
    kc[pid, :, slot] = _bytes(u).flatten(-2)
    ks[pid, :, slot] = byte
    code, byte = _quantise(v, bits)
    u = _bytes(_units(code, bits))
    vc[pid, :, slot // 2, :, slot % 2] = u
    vs[pid, :, slot // 2, :, slot % 2] = byte


def _load(pool, pid, slot, page, bits):
    """Rows k, v [...][heads][64] in f32 of page pid[...], slot slot[...]."""
    kc, ks, vc, vs = _parts(pool, page, bits)
    per = 16 // bits
    s = _scale_values(pool.device).float()

    def rows(unit_bytes, byte, pairs):
        u = unit_bytes[..., 0].int() | unit_bytes[..., 1].int() << 8
        c = _codes(u, bits)
        if pairs:
            c = c.unflatten(-1, (-1, 2, per)).transpose(-1, -2).flatten(-3)
        return (c.unflatten(-1, (4, 16)) * s[byte.long()][..., None]).flatten(-2)

    k = rows(kc[pid, :, slot].unflatten(-1, (-1, 2)), ks[pid, :, slot], True)
    v = rows(vc[pid, :, slot // 2, :, slot % 2], vs[pid, :, slot // 2, :, slot % 2], False)
    return k, v


def _positions(state, first, n):
    """Positions first[s] + 0..n, their pages and slots, and whether row r of scene s is one of its news[s]."""
    page = state["case"]["page"]
    r = torch.arange(n, device="cuda")
    pos = first[:, None] + r
    live = r < state["news"][:, None]
    pos = torch.where(live, pos, 0).long()
    pid = torch.gather(state["table"], 1, pos // page).clamp(min=0).long()
    return pid, pos % page, live


def _read_plain(state, first, n, dtype):
    case = state["case"]
    pid, slot, live = _positions(state, first, n)
    out = []
    for x in _load(state["pool"], pid, slot, case["page"], case["bits"]):
        x = torch.where(live[..., None, None], x, 0.0).transpose(1, 2)
        out.append(x.reshape(case["scenes"] * case["heads"], n, HD).to(dtype))
    return out


def _attend_plain(state):
    case = state["case"]
    scenes, heads, group, rows = case["scenes"], case["heads"], case["group"], case["rows"]
    n = max(_lens(case))
    t = torch.arange(n, device="cuda")
    pid = torch.gather(state["table"], 1, (t // case["page"]).expand(scenes, n)).clamp(min=0).long()
    k, v = _load(state["pool"], pid, (t % case["page"]).expand(scenes, n), case["page"], case["bits"])
    q = state["q"].float().view(scenes, heads, group, rows, HD)
    lens, news = state["lens"].long(), state["news"].long()
    r = torch.arange(rows, device="cuda")
    pos = lens[:, None] - news[:, None] + r
    seen = lens[:, None].expand(scenes, rows)
    if case["frame"]:
        seen = torch.minimum(seen, (pos // case["frame"] + 1) * case["frame"])
        seen = torch.where(pos < 0, 0, seen)
    hidden = (t >= seen[..., None])[:, None, None]
    s = torch.matmul(q.flatten(2, 3), k.permute(0, 2, 3, 1)).view(scenes, heads, group, rows, n)
    s *= HD ** -0.5
    s.masked_fill_(hidden, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1)
    o = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(scenes, heads, group, rows, HD)
    o = o / torch.where(total > 0, total, 1.0)[..., None]
    lse = m[..., 0] + total.log()
    live = (r < news[:, None])[:, None, None]
    o = torch.where(live[..., None], o, 0.0).to(torch.bfloat16)
    lse = torch.where(live, lse, 0.0)
    return o.view(-1, rows, HD), lse.view(-1, rows)


# ------------------------------------------------------------------------------ one pass


def _own_cache(state):
    """The handle that a user's program keeps beside its pool, page table and lengths."""
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    case = state["case"]
    cache = FrameCache.wrap(state["pool"], state["table"], state["lens"], page=case["page"], bits=case["bits"])
    state["cache"] = cache
    if case["op"] == "attend":
        state["layer"] = CachedGlobalAttention(cache, case["rows"], q_heads=case["heads"] * case["group"],
                                               frame=case["frame"])
    else:
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        shape = (case["scenes"] * case["heads"], case["new"], HD)
        state["k_out"] = torch.zeros(shape, dtype=dt, device="cuda")
        state["v_out"] = torch.zeros(shape, dtype=dt, device="cuda")


def run(state):
    case = state["case"]
    if own:
        if "cache" not in state:
            _own_cache(state)
        if case["op"] == "attend":
            return state["layer"].forward(state["q"], q_len=state["news"])
        cache = state["cache"]
        if case["op"] == "write":
            # the last news[s] tokens of scene s; read back from where they went
            cache.append(state["k"], state["v"], new_len=state["news"])
            return cache.read(state["k_out"], state["v_out"], n_len=state["news"])
        return cache.read(state["k_out"], state["v_out"], start=state["start"], n_len=state["news"])
    if case["op"] == "attend":
        return _attend_plain(state)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "write":
        scenes, heads, n = case["scenes"], case["heads"], case["new"]
        first = state["lens"] - state["news"]
        pid, slot, live = _positions(state, first, n)
        if not case["ragged"]:
            pid, slot, live = pid.flatten(), slot.flatten(), slice(None)
            rows = [state[x].view(scenes, heads, n, HD).transpose(1, 2).flatten(0, 1) for x in "kv"]
        else:
            pid, slot = pid[live], slot[live]
            rows = [state[x].view(scenes, heads, n, HD).transpose(1, 2)[live] for x in "kv"]
        _store(state["pool"], pid, slot, rows[0], rows[1], case["page"], case["bits"])
        return tuple(_read_plain(state, first, n, dt))
    return tuple(_read_plain(state, state["start"], case["new"], dt))


def work(case):
    row = 2 * (HD * case["bits"] // 8 + 4)
    lens, news = _lens(case), _news(case)
    if case["op"] != "attend":
        plain = 2 * HD * (2 if case["dtype"] == "bf16" else 4)
        n = sum(news) * case["heads"]
        if case["op"] == "read":
            return {"bytes": n * (row + plain), "flops": 0}
        return {"bytes": n * (2 * plain + 2 * row), "flops": 0}
    heads = case["heads"] * case["group"]
    pairs = 0
    for n, m in zip(lens, news):
        if not case["frame"]:
            pairs += n * m
            continue
        f = case["frame"]
        for p in range(max(0, n - m), n):
            pairs += min(n, (p // f + 1) * f)
    return {"bytes": sum(lens) * case["heads"] * row + sum(news) * heads * (2 * HD * 2 + 4),
            "flops": 4 * HD * pairs * heads}


# ------------------------------------------------------------------------------ the definition in 64 bits


def _exact_numbers(x, bits):
    """What a cache of this many bits holds for rows x, in 64 bits."""
    y = x.double().reshape(*x.shape[:-1], 4, 16)
    most = y.abs().max(-1, keepdim=True).values
    lim = 7 if bits == 4 else 127
    m, e = torch.frexp(most / (lim + 0.5))
    if bits == 4:
        s = torch.ceil(16 * m) * torch.exp2(e.double() - 4)
        s = s.clamp(2.0 ** -16, 15 * 2.0 ** 12)
    else:
        s = torch.exp2(torch.where(m > 0.5, e, e - 1).double())
        s = torch.where(most == 0, 2.0 ** -16, s).clamp(2.0 ** -16, 2.0 ** 15)
    return ((y / s).round().clamp(-lim, lim) * s).reshape(x.shape)


def _exact_cache(state, scene):
    """K and V [heads][tokens][64] of one scene in 64 bits, taken byte by byte from its pages."""
    case = state["case"]
    page, bits, heads = case["page"], case["bits"], case["heads"]
    n = _lens(case)[scene]
    db = HD * bits // 8
    pages = -(-n // page)
    blob = state["pool"][state["table"][scene, :pages].long()].transpose(0, 1)  # [heads][pages][bytes]
    out = []
    ch = torch.arange(HD, device="cuda")
    for part in (0, 1):
        base = part * page * (db + 4)
        if part == 0:
            grain = 32 // bits  # channels of two units
            inner = ch % grain
            unit, within = 2 * (ch // grain) + inner % 2, inner // 2
            t = torch.arange(page, device="cuda")[:, None]
            at = base + t * db + 2 * unit
            at_s = base + page * db + t * 4 + ch // 16
        else:
            per = 16 // bits
            t = torch.arange(page, device="cuda")[:, None]
            within = ch % per
            at = base + (t // 2) * 2 * db + (ch // per) * 4 + (t % 2) * 2
            at_s = base + page * db + (t // 2) * 8 + (ch // 16) * 2 + t % 2
        lo, hi = blob[..., at].int(), blob[..., at + 1].int()
        if bits == 4:
            byte = torch.where(within < 2, lo, hi)
            code = torch.where(within % 2 == 0, byte % 16, byte // 16) - 8
        else:
            first = within == 0
            code = torch.where(first, lo % 128, hi % 128)
            neg = torch.where(first, hi // 128, lo // 128)
            code = torch.where(neg == 1, -code, code)
        b = blob[..., at_s].int()
        x = code.double() * (1 + (b % 8).double() / 8) * torch.exp2((b // 8).double() - 16)
        out.append(x.flatten(1, 2)[:, :n])
    return out


def exact(case, seed):
    state = prepare(case, seed)
    scenes, heads = case["scenes"], case["heads"]
    lens, news = _lens(case), _news(case)
    if case["op"] == "write":
        got = []
        for name in "kv":
            x = _exact_numbers(state[name], case["bits"]).view(scenes, heads, case["new"], HD)
            for i, n in enumerate(news):
                x[i, :, n:] = 0
            got.append(x.flatten(0, 1))
        return tuple(got)
    if case["op"] == "read":
        got = [torch.zeros(scenes, heads, case["new"], HD, dtype=torch.float64, device="cuda") for _ in "kv"]
        for i in range(scenes):
            lo = int(state["start"][i])
            for x, y in zip(got, _exact_cache(state, i)):
                x[i, :, :news[i]] = y[:, lo:lo + news[i]]
        return tuple(x.flatten(0, 1) for x in got)
    group, rows, frame = case["group"], case["rows"], case["frame"]
    o = torch.zeros(scenes, heads, group, rows, HD, dtype=torch.float64, device="cuda")
    lse = torch.zeros(scenes, heads, group, rows, dtype=torch.float64, device="cuda")
    q = state["q"].double().view(scenes, heads, group, rows, HD)
    for i in range(scenes):
        k, v = _exact_cache(state, i)
        step = max(1, int(4e8 / max(1, lens[i] * group)))
        for lo in range(0, news[i], step):
            hi = min(news[i], lo + step)
            at = lens[i] - news[i] + torch.arange(lo, hi, device="cuda")
            seen = torch.full_like(at, lens[i])
            if frame:
                seen = torch.clamp((torch.div(at, frame, rounding_mode="floor") + 1) * frame, max=lens[i])
                seen[at < 0] = 0
            mask = torch.arange(lens[i], device="cuda") < seen[:, None]
            for h in range(heads):
                z = q[i, h, :, lo:hi] @ k[h].T / 8
                z = torch.where(mask, z, -torch.inf)
                top = torch.logsumexp(z, -1) if lens[i] else torch.full(z.shape[:-1], -torch.inf, device="cuda").double()
                w = torch.exp(z - torch.where(top == -torch.inf, 0.0, top)[..., None])
                o[i, h, :, lo:hi] = w @ v[h]
                lse[i, h, :, lo:hi] = top
    return o.view(-1, rows, HD), lse.view(-1, rows)
