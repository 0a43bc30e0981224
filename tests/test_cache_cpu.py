"""The frame cache without a GPU: its numbers and page layout as the oracle has them, host checks
(refused before any launch), and the pages' bookkeeping."""
import ctypes

import numpy as np
import pytest

from oracle import oracle as orc


@pytest.fixture(scope="module")
def lib():
    from view_recon_b200 import _build, sa
    _build.build()
    return sa.load()


def _bf16(x):
    b = np.asarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


@pytest.mark.parametrize("bits", [4, 8])
def test_stored_numbers_are_bf16_numbers_within_half_a_step(bits):
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((200, 64)) * np.exp(2 * rng.standard_normal((200, 1)))
    y = orc.cache_numbers(x, bits)
    assert np.array_equal(orc.to_f64(_bf16(y)), y)
    most = np.abs(x).reshape(200, 4, 16).max(-1)
    err = np.abs(y - x).reshape(200, 4, 16).max(-1)
    # half a step: s / 2, and s < most / 7.5 * 9/8 (the next smaller scale is 8/9 or more of it), or
    # twice most / 127.5 for powers of two
    assert (err <= (most / 7.5 * 9 / 8 if bits == 4 else 2 * most / 127.5) / 2).all()
    # reading back and writing again changes nothing
    assert np.array_equal(orc.cache_numbers(y, bits), y) or bits == 4
    assert np.array_equal(orc.cache_numbers(np.zeros((1, 64)), bits), np.zeros((1, 64)))


def test_scale_range_and_saturation():
    assert orc.cache_scale(0) == 2.0 ** -16 and orc.cache_scale(255) == 1.875 * 2.0 ** 15
    x = np.zeros((1, 64))
    x[0, 0], x[0, 1] = 1e9, 1.0
    assert orc.cache_numbers(x, 4)[0, 0] == 7 * 1.875 * 2.0 ** 15
    assert orc.cache_numbers(x, 8)[0, 0] == 127 * 2.0 ** 15
    x[0, 0] = 0.0
    assert abs(orc.cache_numbers(x, 4)[0, 1] - 1.0) <= 1 / 7.5 * 9 / 16


@pytest.mark.parametrize("bits", [4, 8])
def test_unpack_knows_every_code_and_place(bits):
    """Bytes written one code at a time, by the layout's own words, come back in their places."""
    page, db = 16, 8 * bits
    rng = np.random.default_rng(3)
    top = 8 if bits == 4 else 128
    code = rng.integers(-top + 1, top, (2, page, 64))
    byte = rng.integers(0, 256, (2, page, 4))
    raw = np.zeros(page * 2 * (db + 4), np.uint8)
    per = 16 // bits
    for part in range(2):
        base = part * page * (db + 4)
        for t in range(page):
            for ch in range(64):
                if part == 0:
                    group, r = divmod(ch, 2 * per)
                    at, j = base + t * db + (2 * group + r % 2) * 2, r // 2
                else:
                    group, j = divmod(ch, per)
                    at = base + (t // 2) * 2 * db + (2 * group + t % 2) * 2
                c = int(code[part, t, ch])
                if bits == 4:
                    u = (c + 8) << (4 * j)
                elif j == 0:
                    u = abs(c) | (c < 0) << 15
                else:
                    u = abs(c) << 8 | (c < 0) << 7
                raw[at] |= u & 255
                raw[at + 1] |= u >> 8
            for b in range(4):
                at = t * 4 + b if part == 0 else (t // 2) * 8 + 2 * b + t % 2
                raw[base + page * db + at] = byte[part, t, b]
    got = orc.cache_unpack(raw, page, bits)
    for part in range(2):
        assert np.array_equal(got[part], code[part] * np.repeat(orc.cache_scale(byte[part]), 16, -1))


def test_cache_attend_is_softmax_attention():
    rng = np.random.default_rng(1)
    q, K, V = (rng.standard_normal(s) for s in ((4, 5, 64), (2, 9, 64), (2, 9, 64)))
    O, lse, _, _ = orc.cache_attend(q, K, V, 0.125, frame=4)
    for h in range(4):
        for r in range(5):
            n = min(9, ((9 - 5 + r) // 4 + 1) * 4)
            s = 0.125 * K[h // 2, :n] @ q[h, r]
            w = np.exp(s) / np.exp(s).sum()
            assert np.allclose(O[h, r], w @ V[h // 2, :n], rtol=0, atol=1e-14)
            assert abs(lse[h, r] - np.log(np.exp(s).sum())) < 1e-13
    O, lse, _, _ = orc.cache_attend(q, K[:, :3], V[:, :3], 0.125, frame=1)  # two rows before token 0
    assert (O[:, :2] == 0).all() and np.isneginf(lse[:, :2]).all() and np.isfinite(lse[:, 2:]).all()


def test_host_checks(lib):
    from view_recon_b200 import sa
    P = ctypes.c_void_p
    fake, odd, odd2 = P(0x10000), P(0x10008), P(0x10002)
    ok = sa.kv_cache(2, 4, 10, 5, 64, 4)
    R = ctypes.byref
    inv, uns, wsp = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_WORKSPACE
    assert sa.sa_kv_pool_size(ok) == 10 * 4 * 64 * 72
    assert sa.sa_kv_pool_size(sa.kv_cache(2, 4, 10, 5, 16, 8)) == 10 * 4 * 16 * 136
    # 1 024 frames x 1 374 tokens x 16 heads in 4 bits: 10 992 pages of 128
    assert sa.sa_kv_pool_size(sa.kv_cache(1, 16, 10992, 10992)) == 16 * 10992 * 128 * 72
    bad = [sa.kv_cache(0, 4, 10, 5), sa.kv_cache(2, 0, 10, 5), sa.kv_cache(2, 4, 0, 5), sa.kv_cache(2, 4, 10, 0),
           sa.kv_cache(2, 4, 10, 5, page=48), sa.kv_cache(2, 4, 10, 5, page=256), sa.kv_cache(2, 4, 10, 5, bits=5),
           sa.kv_cache(2, 4, 10, 5, head_dim=32), sa.kv_cache(2, 4, 10, 1 << 24), sa.kv_cache(1 << 16, 1 << 16, 10, 5)]
    for c in bad:
        want = uns if c.head_dim == 32 or c.max_pages == 1 << 24 or c.scenes == 1 << 16 else inv
        assert sa.sa_kv_pool_size(c) == 0
        assert lib.sa_kv_append(R(c), 1, fake, fake, 1, None, fake, fake, fake, None) == want
        assert lib.sa_kv_read(R(c), 1, 1, None, None, fake, fake, fake, fake, fake, None) == want
        assert sa.sa_kv_attn_workspace_size(c, 4, 1) == 0
        assert lib.sa_kv_attn_fwd(R(c), fake, 4, 1, None, 0, 0.0, fake, fake, fake, fake, 1 << 40, fake, None,
                                  None) == want
    args = dict(dtype=1, k=fake, v=fake, n=3, n_len=None, lens=fake, table=fake, pool=fake)
    for change in (dict(dtype=2), dict(k=None), dict(v=None), dict(n=0), dict(lens=None), dict(table=None),
                   dict(pool=None), dict(k=odd), dict(v=odd), dict(pool=odd), dict(n_len=odd2), dict(lens=odd2),
                   dict(table=odd2)):
        a = {**args, **change}
        assert lib.sa_kv_append(R(ok), a["dtype"], a["k"], a["v"], a["n"], a["n_len"], a["lens"], a["table"],
                                a["pool"], None) == inv, change
    args = dict(dtype=1, n=3, n_len=None, start=None, lens=fake, table=fake, pool=fake, k=fake, v=fake)
    for change in (dict(dtype=-1), dict(n=0), dict(start=odd2), dict(n_len=odd2), dict(lens=None), dict(table=None),
                   dict(pool=None), dict(k=None, v=None), dict(k=odd), dict(v=odd), dict(pool=odd)):
        a = {**args, **change}
        assert lib.sa_kv_read(R(ok), a["dtype"], a["n"], a["n_len"], a["start"], a["lens"], a["table"], a["pool"],
                              a["k"], a["v"], None) == inv, change
    args = dict(q=fake, heads=8, rows=3, q_len=None, frame=0, scale=0.0, lens=fake, table=fake, pool=fake, ws=fake,
                nb=1 << 40, o=fake, lse=None)
    for change, want in ((dict(q=None), inv), (dict(q=odd), inv), (dict(heads=6), inv), (dict(heads=0), inv),
                         (dict(rows=0), inv), (dict(q_len=odd2), inv), (dict(frame=-1), inv), (dict(scale=-1.0), inv),
                         (dict(scale=float("inf")), inv), (dict(scale=float("nan")), inv), (dict(lens=None), inv),
                         (dict(table=None), inv), (dict(pool=None), inv), (dict(o=None), inv), (dict(o=odd), inv),
                         (dict(lse=odd2), inv), (dict(ws=None), wsp), (dict(ws=odd), inv),
                         (dict(nb=sa.sa_kv_attn_workspace_size(ok, 8, 3) - 1), wsp), (dict(rows=1 << 30), uns)):
        a = {**args, **change}
        assert lib.sa_kv_attn_fwd(R(ok), a["q"], a["heads"], a["rows"], a["q_len"], a["frame"], a["scale"], a["lens"],
                                  a["table"], a["pool"], a["ws"], a["nb"], a["o"], a["lse"], None) == want, change
    assert sa.status_string(sa.SA_ERR_NONFINITE) == "infinities or NaN cannot be stored"


def test_binding_refuses_cpu_and_strided_tensors(lib):
    import torch
    from view_recon_b200 import sa
    c = sa.kv_cache(1, 1, 4, 4)
    x = torch.zeros(1, 3, 64)
    with pytest.raises(ValueError):
        sa.sa_kv_append(c, x, x, 3, None, x, x, x)
    with pytest.raises(ValueError):
        sa.sa_kv_append(c, x.half(), x.half(), 3, None, x, x, x)
    with pytest.raises(ValueError):
        sa.sa_kv_append(c, x, x.bfloat16(), 3, None, x, x, x)
    with pytest.raises(ValueError):
        sa.sa_kv_read(c, 3, None, None, x, x, x, None, None)


def test_pages_bookkeeping(lib):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(3, 2, tokens=100, n_pages=8, page=16, device="cpu")
    assert c.max_pages == 7 and c.pool.numel() == 8 * 2 * 16 * 72
    c.grow([17, 0, 1])
    assert c.lens.tolist() == [17, 0, 1]
    used = c.page_table[c.page_table >= 0].tolist()
    assert len(used) == len(set(used)) == 3 and (c.page_table[1] == -1).all()
    before = c.page_table.clone()
    c.grow([15, 0, 0])                                   # still the scene's second page
    assert c.page_table.equal(before) and c.lens.tolist() == [32, 0, 1]
    with pytest.raises(MemoryError):                       # 6 pages wanted, 5 free
        c.grow([0, 96, 0])
    assert c.page_table.equal(before) and c.lens.tolist() == [32, 0, 1]
    with pytest.raises(ValueError):                        # longer than the table's row
        c.grow([81, 0, 0])
    with pytest.raises(ValueError):
        c.grow([1, 2])
    with pytest.raises(ValueError):
        c.grow(-1)
    c.release(0)
    assert c.lens.tolist() == [0, 0, 1] and (c.page_table[0] == -1).all()
    c.grow([0, 96, 0])
    used = c.page_table[c.page_table >= 0].tolist()
    assert len(used) == len(set(used)) == 7
    other = FrameCache(3, 5, tokens=100, page=16, bits=8, like=c)
    assert other.lens is c.lens and other.page_table is c.page_table and other.n_pages == 8
    with pytest.raises(ValueError):
        other.grow(1)
    for kw in (dict(page=48), dict(bits=3), dict(head_dim=32)):
        with pytest.raises(ValueError):
            FrameCache(1, 1, 10, device="cpu", **kw)
    with pytest.raises(ValueError):
        FrameCache(2, 5, tokens=100, page=16, like=c)


def test_wrap_and_layer_refusals(lib):
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    pool = torch.zeros(4, 2, 16 * 72, dtype=torch.uint8)
    table = torch.zeros(1, 3, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    c = FrameCache.wrap(pool, table, lens, page=16)
    assert (c.scenes, c.heads, c.n_pages, c.max_pages) == (1, 2, 4, 3)
    with pytest.raises(ValueError):
        FrameCache.wrap(pool, table, lens, page=32)
    with pytest.raises(ValueError):
        FrameCache.wrap(pool, table.long(), lens, page=16)
    with pytest.raises(ValueError):
        FrameCache.wrap(pool, table, lens[:0], page=16)
    with pytest.raises(ValueError):
        c.grow(1)
    x = torch.zeros(2, 5, 64)
    for k, v in ((x[:1], x), (x, x.bfloat16()), (x.half(), x.half()), (x[:, :, :32], x), (x.transpose(0, 1), x),
                 (x[0], x)):
        with pytest.raises(ValueError):
            c.append(k, v)
    with pytest.raises(ValueError):
        c.append(x, x, new_len=torch.zeros(1))
    with pytest.raises(ValueError):
        c.read()
    with pytest.raises(ValueError, match="CUDA"):    # bookkeeping works on the host, calls do not
        c.append(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        c.read(x, x)
    for rows, heads in ((0, 2), (3, 3), (3, 0)):
        with pytest.raises(ValueError):
            CachedGlobalAttention(c, rows, q_heads=heads)
    layer = CachedGlobalAttention(c, 3, q_heads=4)
    assert layer.o.shape == (4, 3, 64)
    with pytest.raises(ValueError, match="CUDA"):
        layer.forward(torch.zeros(4, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(4, 3, 64))
    with pytest.raises(ValueError):
        layer.forward(torch.zeros(4, 2, 64, dtype=torch.bfloat16))


def test_grow_takes_any_integer(lib):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(2, 1, tokens=64, page=16, device="cpu")
    c.grow(np.int64(3))
    c.grow(np.array([1, 14], dtype=np.int32))
    assert c.lens.tolist() == [4, 17]


def test_single_lanes_rejoin_their_warp_before_warp_wide_instructions():
    """Register splits and tensor-memory accesses (.sync.aligned) want a warp that stands together; where one lane
    walked alone, or lanes took a branch of their own, a __syncwarp() is what brings it together again.  (Read in
    the source: no run can be relied on to show the absence.)"""
    import os
    import re
    from view_recon_b200 import _build
    src = {}
    for name in ("k_kv_attn.cuh", "k_kv_attn_tc.cuh"):
        with open(os.path.join(os.path.dirname(_build.__file__), "csrc", name)) as f:
            src[name] = re.sub(r"//[^\n]*", "", f.read())
        notes = [m.end() for m in re.finditer(r"if \(threadIdx\.x == \d+\) note_parts\([^;]*;", src[name])]
        assert len(notes) == 1
        for at in notes:
            assert re.match(r"\s*__syncwarp\(\);", src[name][at:]), name
    softmax = src["k_kv_attn_tc.cuh"]
    raised = softmax.index("if (mx > m_run + 8.0f)")
    close = softmax.index("}", raised)
    assert re.match(r"\s*__syncwarp\(\);", softmax[close + 1:])
    assert re.search(r"__syncwarp\(\);\s*named_bar_sync\(", src["k_kv_attn.cuh"])


def test_pools_past_64_bit_sizes_are_refused(lib):
    """A pool's size that does not fit 64 bits wrapped round to a small number, and calls took that pool."""
    from view_recon_b200 import sa
    top = 2 ** 31 - 1
    fake = ctypes.c_void_p(0x10000)
    most = (2 ** 63 - 1) // (128 * 136 * 2 ** 20)        # pages of 2^20 heads that still fit
    assert sa.sa_kv_pool_size(sa.kv_cache(1, 2 ** 20, most, 5, 128, 8)) == most * 2 ** 20 * 128 * 136
    for c in (sa.kv_cache(1, top, top, 5, 128, 8), sa.kv_cache(1, 2 ** 20 + 1, most, 5, 128, 8),
              sa.kv_cache(1, 2 ** 27 + 3, 2 ** 27 + 1, 5, 128, 4)):
        assert c.n_pages * c.heads * c.page * 2 * (8 * c.bits + 4) >= 2 ** 63
        assert sa.sa_kv_pool_size(c) == 0
        assert lib.sa_kv_append(ctypes.byref(c), 1, fake, fake, 0, None, fake, fake, fake, None) == sa.SA_ERR_UNSUPPORTED
        assert sa.sa_kv_attn_workspace_size(c, c.heads, 1) == 0


def test_a_cache_off_the_gpu_has_no_streams(lib):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(1, 1, tokens=64, page=16, device="cpu")
    for call in (lambda: c.grow(1, stream=object()), lambda: c.release(0, stream=object())):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert c.lens.tolist() == [0] and c._len == [0]


def test_rows_that_grow_did_not_count_in_are_refused(lib):
    """Without new_len every scene's last n tokens are written: n has to be what grow counted into each of them.
    (Off the GPU a call that passes this check ends at the next one.)"""
    import torch
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(2, 1, tokens=200, page=16, device="cpu")
    layers = [c, FrameCache(2, 1, tokens=200, page=16, bits=8, like=c)]

    def check(n, good, **kw):
        x = torch.zeros(2, n, 64)
        for layer in layers:
            with pytest.raises(ValueError, match="CUDA" if good else "grow counted"):
                layer.append(x, x, **kw)

    check(3, False)                                       # nothing counted in
    c.grow(5)
    check(4, False)
    check(6, False)
    check(5, True)
    check(5, True)                                        # the same rows once more
    c.grow([3, 0])
    check(3, False)                                       # the second scene's last rows are old ones
    check(5, False)
    check(3, True, new_len=torch.tensor([3, 0], dtype=torch.int32))
    c.grow(2)
    check(2, True)
    c.grow(4)
    c.grow(3)                                             # two frames, written at once or the second alone
    check(7, True)
    check(3, True)
    check(4, False)
    c.grow(3)
    check(3, True)
    check(10, False)                                      # the seven were written
    c.release(1)
    check(3, False)
    c.grow([0, 3])
    check(3, False)
    c.grow([6, 3])
    check(6, True)                                        # nothing written since: 6 and 6
    layers[1].append(torch.empty(2, 0, 64), torch.empty(2, 0, 64))


def test_binding_refuses_other_types(lib):
    """An LSE of a smaller type would be written past its end, lengths of another would be read as nonsense."""
    import torch
    from view_recon_b200 import sa
    c = sa.kv_cache(1, 1, 4, 4)
    x, i = torch.zeros(1, 3, 64), torch.zeros(4, dtype=torch.int32)
    h = x.bfloat16()
    for n_len, lens, table in ((None, x, i), (None, i, i.long()), (i.long(), i, i)):
        with pytest.raises(ValueError, match="int32"):
            sa.sa_kv_append(c, x, x, 3, n_len, lens, table, x)
        with pytest.raises(ValueError, match="int32"):
            sa.sa_kv_read(c, 3, n_len, None, lens, table, x, x, x)
        with pytest.raises(ValueError, match="int32"):
            sa.sa_kv_attn_fwd(c, h, 1, 3, n_len, 0, 0.0, lens, table, x, x, h)
    with pytest.raises(ValueError, match="int32"):
        sa.sa_kv_read(c, 3, None, x, i, i, x, x, x)
    for q, o, lse in ((x, h, None), (h, x, None), (h, h, h), (h.half(), h, x)):
        with pytest.raises(ValueError, match="bf16"):
            sa.sa_kv_attn_fwd(c, q, 1, 3, None, 0, 0.0, i, i, x, x, o, lse)
    with pytest.raises(ValueError, match="CUDA"):
        sa.sa_kv_attn_fwd(c, h, 1, 3, None, 0, 0.0, i, i, x, x, h, x)


def test_sizes_past_32_bits_are_refused(lib):
    """ctypes cuts an integer to the low bits of its argument: 2^32 + 1 scenes were one, a frame of 2^32 + 7 tokens
    seven."""
    import torch
    from view_recon_b200 import sa
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    big = 2 ** 32
    for args in ((big + 1, 1, 4, 4), (1, big + 1, 4, 4), (1, 1, big + 4, 4), (1, 1, 4, big + 4), (2 ** 31, 1, 4, 4)):
        with pytest.raises(ValueError, match="32 bits"):
            sa.kv_cache(*args)
    with pytest.raises(ValueError, match="32 bits"):
        sa.kv_cache(1, 1, 4, 4, bits=big + 4)
    c = sa.kv_cache(1, 1, 4, 4)
    for heads, rows in ((1, big + 5), (big + 1, 5)):
        with pytest.raises(ValueError, match="32 bits"):
            sa.sa_kv_attn_workspace_size(c, heads, rows)
    i, x = torch.zeros(4, dtype=torch.int32), torch.zeros(1, 3, 64)
    with pytest.raises(ValueError, match="32 bits"):
        sa.sa_kv_attn_fwd(c, x.bfloat16(), 1, 3, None, big + 7, 0.0, i, i, x, x, x.bfloat16())
    for kw in (dict(scenes=big + 1), dict(heads=big + 1), dict(tokens=128 * (big + 1)), dict(n_pages=big + 1)):
        with pytest.raises(ValueError):
            FrameCache(**{**dict(scenes=1, heads=1, tokens=128, device="cpu"), **kw})
    cache = FrameCache(1, 1, tokens=128, device="cpu")
    for frame in (-1, 2 ** 31, big + 7):
        with pytest.raises(ValueError, match="frame"):
            CachedGlobalAttention(cache, 2, frame=frame)
    with pytest.raises(ValueError, match="32 bits"):
        CachedGlobalAttention(cache, big + 2)
    assert CachedGlobalAttention(cache, 2, frame=2 ** 31 - 1).frame == 2 ** 31 - 1


def test_a_failed_send_leaves_the_books_as_they_were(lib, monkeypatch):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(2, 1, tokens=64, n_pages=6, page=16, device="cpu")
    c.grow([20, 3])
    books = lambda: (c._len[:], [p[:] for p in c._pages], c._free[:], c.lens.tolist(), list(c._news.last))  # noqa: E731
    before, send = books(), c._send
    for failing in (1, 2):                                 # the pages' copy, or the lengths'
        calls = []

        def fail(values, dtype):
            calls.append(0)
            if len(calls) == failing:
                raise RuntimeError("no memory")
            return send(values, dtype)

        monkeypatch.setattr(c, "_send", fail)
        with pytest.raises(RuntimeError, match="no memory"):
            c.grow([20, 0])
        assert books() == before
    table, calls, failing = c.page_table.clone(), [], 1
    monkeypatch.setattr(c, "_send", fail)
    with pytest.raises(RuntimeError, match="no memory"):
        c.release(0)
    assert books() == before and c.page_table.equal(table)
    monkeypatch.setattr(c, "_send", send)
    c.grow([44, 29])                                       # all six pages, each once
    used = [p for pages in c._pages for p in pages]
    assert sorted(used) == list(range(6)) and c._free == [] and c.lens.tolist() == [64, 32]
    assert [x for x in c.page_table.flatten().tolist() if x >= 0] == used
    c.release(0)
    assert sorted(c._free) == sorted(set(range(6)) - set(c._pages[1])) and c.lens.tolist() == [0, 32]


def test_grow_refuses_parts_of_tokens(lib):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(2, 1, tokens=64, page=16, device="cpu")
    for n in ([1.5, 0], np.array([0.0, 0.5])):
        with pytest.raises(ValueError):
            c.grow(n)
    assert c.lens.tolist() == [0, 0]
    c.grow([2.0, np.float32(3)])
    assert c.lens.tolist() == [2, 3] and c._len == [2, 3]


def test_a_cache_like_another_is_on_its_device(lib):
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(1, 1, tokens=64, page=16, device="cpu")
    for device in ("cuda", "cuda:1", "meta"):
        with pytest.raises(ValueError, match="device"):
            FrameCache(1, 1, tokens=64, page=16, like=c, device=device)
    assert FrameCache(1, 1, tokens=64, page=16, like=c, device="cpu").device == c.device


@pytest.mark.parametrize("bits", [4, 8])
def test_writing_what_was_read(bits):
    """8 bits: the same numbers again.  4 bits: not always (once the largest code is 7 a smaller scale may do: 14/15
    of s reaches 7 s), but each within half a step of what was read, and a block's largest stays its largest."""
    rng = np.random.default_rng(40 + bits)
    x = rng.standard_normal((400, 64)) * np.exp(2 * rng.standard_normal((400, 1)))
    y = orc.cache_numbers(x, bits)
    z = orc.cache_numbers(y, bits)
    if bits == 8:
        assert np.array_equal(z, y)
        return
    blocks = [a.reshape(400, 4, 16) for a in (y, z)]
    most = np.abs(blocks[0]).max(-1, keepdims=True)
    # the smallest scale with 7.5 s >= most is below most / 7.5 * 9/8
    assert (np.abs(blocks[1] - blocks[0]) <= most / 7.5 * 9 / 16).all()
    assert (z != y).any()
    at = np.abs(blocks[0]).argmax(-1)[..., None]
    assert (np.take_along_axis(np.abs(blocks[1]), at, -1) == np.abs(blocks[1]).max(-1, keepdims=True)).all()
