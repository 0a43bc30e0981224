"""The frame cache on the GPU: written numbers, read-back and attention against the fp64 oracle.

Bars.  Written and read numbers equal the oracle's bit for bit (they are exact by definition, in bf16
and in f32).  Attention: a bf16 rounding is off by at most 2^-8 of the value; probabilities are
rounded once before they meet V and O once at the end, so
  |O - O_ref| <= 2^-8 |O_ref| + (2^-8 + 2^-14) A,   A = sum_j w_j |v_j|
(2^-14 A: f32 sums of scores, exponentials and O), plus 2^-100 max|v|: a weight below 2^-126 of the
row's largest is below f32's smallest normal number and drops out, with at most 2^-126 |v_j| for each of fewer
than 2^26 keys (it shows where the keys that count hold a zero in a channel).  LSE: f32 sums of 64 exact products, each addition off
by at most 2^-24 of the largest partial sum, and an exponential of 2^-22:
  |LSE - ref| <= 2^-18 B + 2^-20 (1 + |ref|),       B = scale max_j sum_e |q_e k_je|.
"""
import numpy as np
import pytest

from oracle import oracle as orc
from tests import helpers as H

pytestmark = pytest.mark.gpu


def _rows(rng, shape, dtype, spread=0.5):
    """Rows that the type holds exactly, as a float64 array and a CUDA tensor."""
    import torch
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t.float().numpy().astype(np.float64), t.cuda()


class Pool:
    """A cache over tensors of its own: pages in random order among spare ones, every byte random at first."""

    def __init__(self, rng, lens, heads, page, bits, spare=3, extra_cols=1):
        import torch
        from view_recon_b200.pipeline import FrameCache
        self.lens, self.heads, self.page, self.bits = list(lens), heads, page, bits
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + spare
        self.bytes = rng.integers(0, 256, (n_pages, heads, page * 2 * (8 * bits + 4)), dtype=np.uint8)
        if bits == 8:
            # scales of 8-bit codes are powers of two: a 7-bit code times one is a bf16 number, times
            # a 4-bit significand (11 bits) it is not, and no append writes such a byte
            for lo in (page * 64, page * 132):
                self.bytes[:, :, lo:lo + page * 4] &= 0xF8
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), max(1, max(need)) + extra_cols), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.t_pool = torch.from_numpy(self.bytes).cuda()
        self.t_table = torch.from_numpy(self.table).cuda()
        self.t_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.cache = FrameCache.wrap(self.t_pool, self.t_table, self.t_lens, page=page, bits=bits)

    def rows(self, s):
        """K, V [heads][len][64] of scene s as the pool's bytes have them now."""
        raw = self.t_pool.cpu().numpy()
        n = self.lens[s]
        k, v = orc.cache_unpack(raw[self.table[s, :-(-n // self.page)]], self.page, self.bits)
        join = lambda x: np.moveaxis(x, 1, 0).reshape(self.heads, -1, 64)[:, :n]  # noqa: E731
        return join(k), join(v)


def _bar(ref, A):
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -14) * A + 2.0 ** -100 * A.max(initial=0.0)


def _counts(xs):
    import torch
    return torch.tensor(xs, dtype=torch.int32, device="cuda")


def _ok(want=0):
    import torch
    from view_recon_b200 import sa
    torch.cuda.synchronize()
    assert sa.sa_check_device_error() == want


# ------------------------------------------------------------------------------ writing and reading

WRITES = [
    # lens, rows per scene given, rows per scene taken (None: all)
    ([1], 1, None), ([2], 1, None), ([33], 1, None), ([200], 200, None), ([301], 45, None), ([17, 64, 5], 5, None),
    ([0, 1, 130, 77], 9, [0, 1, 9, 4]), ([129, 257, 16], 130, [129, 130, 7]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits,page", [(4, 16), (4, 128), (8, 32), (8, 64)])
@pytest.mark.parametrize("lens,n,taken", WRITES)
def test_append_writes_the_oracles_numbers_and_nothing_else(bits, page, dtype, lens, n, taken):
    rng = np.random.default_rng(hash((bits, page, n)) % 1000)
    heads = 3
    p = Pool(rng, lens, heads, page, bits)
    before = [p.rows(s) for s in range(len(lens))]
    spare = sorted(set(range(len(p.bytes))) - set(p.table[p.table >= 0]))
    k, tk = _rows(rng, (len(lens) * heads, n, 64), dtype)
    v, tv = _rows(rng, (len(lens) * heads, n, 64), dtype)
    p.cache.append(tk, tv, new_len=None if taken is None else _counts(taken))
    _ok()
    for s, L in enumerate(lens):
        m = n if taken is None else taken[s]
        for got, old, new in zip(p.rows(s), before[s], (k, v)):
            assert np.array_equal(got[:, :L - m], old[:, :L - m])
            assert np.array_equal(got[:, L - m:], orc.cache_numbers(new[s * heads:(s + 1) * heads, :m], bits))
    raw = p.t_pool.cpu().numpy()
    assert np.array_equal(raw[spare], p.bytes[spare])
    for s, L in enumerate(lens):  # the last page's bytes behind the scene's end
        if L % page:
            full = orc.cache_unpack(raw[p.table[s, L // page]], page, bits)
            old = orc.cache_unpack(p.bytes[p.table[s, L // page]], page, bits)
            for a, b in zip(full, old):
                assert np.array_equal(a[:, L % page:], b[:, L % page:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits,page", [(4, 16), (4, 128), (8, 32), (8, 128)])
def test_read_returns_every_byte_pattern_exactly(bits, page, dtype):
    """Random bytes: every scale byte that an append can write and every code among them."""
    import torch
    rng = np.random.default_rng(bits + page)
    lens, n = [700, 0, 1, 339], 301
    p = Pool(rng, lens, 2, page, bits)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    want = [p.rows(s) for s in range(4)]
    for start, taken in (([399, 0, 0, 20], None), ([5, 0, 0, 301], [301, 0, 1, 38]), (None, [301, 0, 1, 200])):
        k = torch.full((8, n, 64), -7.0, dtype=dt, device="cuda")
        v = torch.full((8, n, 64), -7.0, dtype=dt, device="cuda")
        out = p.cache.read(k, v, start=None if start is None else _counts(start),
                           n_len=None if taken is None else _counts(taken))
        _ok()
        assert out[0] is k and out[1] is v
        for s, L in enumerate(lens):
            m = n if taken is None else taken[s]
            lo = L - m if start is None else start[s]
            m = min(m, L - lo)
            for got, ref in zip((k, v), want[s]):
                got = H.from_device(got)[2 * s:2 * s + 2]
                assert np.array_equal(got[:, :m], ref[:, lo:lo + m])
                assert (got[:, m:] == -7).all()
    # one of the two alone; a start before token 0 leaves the rows before it
    k = torch.full((8, 4, 64), -7.0, dtype=dt, device="cuda")
    p.cache.read(k=k, start=_counts([-2, -9, -1, 338]))
    v = torch.full((8, 4, 64), -7.0, dtype=dt, device="cuda")
    p.cache.read(v=v, start=_counts([-2, -9, -1, 338]))
    _ok()
    for x, i in ((H.from_device(k), 0), (H.from_device(v), 1)):
        assert np.array_equal(x[:2, 2:], want[0][i][:, :2]) and (x[:2, :2] == -7).all()
        assert (x[2:4] == -7).all()
        assert np.array_equal(x[4:6, 1:2], want[2][i]) and (x[4:6, 2:] == -7).all()
        assert np.array_equal(x[6:, :1], want[3][i][:, 338:]) and (x[6:, 1:] == -7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_borders_between_codes_and_scales(bits, dtype):
    """Values on, and one step of the type beside, every border: ties of codes for many scales, block
    maxima at which the scale changes, zeros, the smallest and largest numbers of the type."""
    import torch
    rng = np.random.default_rng(5)
    top = 7 if bits == 4 else 127
    scales = orc.cache_scale(np.arange(0, 256, 1 if bits == 4 else 8))
    blocks = []
    for s in scales[rng.permutation(len(scales))[:96 if bits == 4 else 32]]:
        ties = (rng.integers(0, top, 15) + 0.5) * s * rng.choice([-1, 1], 15)
        blocks.append(np.concatenate([[(top + 0.5) * s], ties]))
        blocks.append(np.concatenate([[top * s], ties]))
    x = np.array(blocks).reshape(-1, 64)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    t = torch.from_numpy(x.astype(np.float32)).to(dt)
    if dtype == "bf16":
        i = t.view(torch.int16)
        t = torch.cat([t, (i + 1).view(dt), (i - 1).view(dt)])
    else:
        i = t.view(torch.int32)
        t = torch.cat([t, (i + 1).view(dt), (i - 1).view(dt), (i + 300).view(dt)])
    big = torch.finfo(dt).max
    more = torch.zeros((4, 64), dtype=dt)
    more[1] = 1e-30
    more[2, ::5] = big
    more[3, 3::16] = -1e-4
    t = torch.cat([t, more])
    n = t.shape[0]
    p = Pool(rng, [n + 3], 1, 16, bits)
    p.cache.append(t[None].cuda().contiguous(), t[None].flip(1).cuda().contiguous())
    _ok()
    k, v = p.rows(0)
    ref = orc.cache_numbers(t.double().numpy(), bits)
    assert np.array_equal(k[0, 3:], ref)
    assert np.array_equal(v[0, 3:], ref[::-1])


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (8, "f32")])
def test_nonfinite_rows_are_reported(bits, dtype):
    import torch
    from view_recon_b200 import sa
    rng = np.random.default_rng(6)
    p = Pool(rng, [40], 2, 32, bits)
    x, t = _rows(rng, (2, 40, 64), dtype)
    t[0, 3, 5], t[1, 7, 20], t[1, 7, 21] = float("nan"), float("inf"), -float("inf")
    p.cache.append(t, t)
    _ok(sa.SA_ERR_NONFINITE)
    top = 7 * 1.875 * 2.0 ** 15 if bits == 4 else 127 * 2.0 ** 15
    x[0, 3, 5], x[1, 7, 20], x[1, 7, 21] = 0.0, 1e30, -1e30
    ref = orc.cache_numbers(x, bits)
    assert ref[1, 7, 20] == top and ref[1, 7, 21] == -top
    for got in p.rows(0):
        assert np.array_equal(got, ref)
    p.cache.append(t.nan_to_num(0.0, 0.0, 0.0), t.nan_to_num(0.0, 0.0, 0.0))
    _ok()


# ------------------------------------------------------------------------------ attention

def _check(p, q, o, lse, q_heads, frame, taken, scale=0.125, fill=None):
    group = q_heads // p.heads
    for s in range(len(p.lens)):
        m = taken[s]
        K, V = p.rows(s)
        got_o, got_l = o[s * q_heads:(s + 1) * q_heads], lse[s * q_heads:(s + 1) * q_heads]
        ref, ref_l, A, B = orc.cache_attend(q[s * q_heads:(s + 1) * q_heads, :m], K, V, scale, frame)
        err, bar = np.abs(got_o[:, :m] - ref), _bar(ref, A)
        assert (err <= bar).all(), "scene %d: O off by %.3g of its bar" % (s, (err / np.maximum(bar, 1e-300)).max())
        dead = np.isneginf(ref_l)
        assert (np.isneginf(got_l[:, :m]) == dead).all()
        assert (got_o[:, :m][dead] == 0).all()
        e, b = np.abs(got_l[:, :m][~dead] - ref_l[~dead]), (2.0 ** -18 * B + 2.0 ** -20 * (1 + np.abs(ref_l)))[~dead]
        assert (e <= b).all(), "scene %d: LSE off by %.3g of its bar" % (s, (e / b).max())
        if fill is not None:
            assert (got_o[:, m:] == fill).all() and (got_l[:, m:] == fill).all()
    assert group >= 1


def _fill(p, rng, dtype="bf16"):
    n = max(p.lens)
    if n:
        _, k = _rows(rng, (len(p.lens) * p.heads, n, 64), dtype)
        _, v = _rows(rng, (len(p.lens) * p.heads, n, 64), dtype)
        p.cache.append(k, v, new_len=p.t_lens)


def _attend(p, rng, rows, q_heads, frame=0, taken=None, scale=0.0, q_spread=0.5):
    from view_recon_b200.pipeline import CachedGlobalAttention
    q, tq = _rows(rng, (len(p.lens) * q_heads, rows, 64), "bf16", q_spread)
    layer = CachedGlobalAttention(p.cache, rows, q_heads=q_heads, frame=frame, softmax_scale=scale)
    layer.o.fill_(-3.0)
    layer.lse.fill_(-3.0)
    layer.forward(tq, q_len=None if taken is None else _counts(taken))
    _ok()
    _check(p, q, H.from_device(layer.o), H.from_device(layer.lse), q_heads, frame,
           [rows] * len(p.lens) if taken is None else taken, scale or 0.125, fill=-3.0)
    return q, tq, layer


LENS = [[1], [2], [31], [127], [128], [129], [1000], [0, 1, 300, 64], [513, 5, 0, 0, 2]]


@pytest.mark.parametrize("bits,page", [(4, 16), (4, 128), (8, 32), (8, 64)])
@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("rows", [1, 9, 33, 131])
def test_attention_lengths(bits, page, lens, rows):
    rng = np.random.default_rng(rows + sum(lens))
    p = Pool(rng, lens, 2, page, bits)
    _fill(p, rng)
    _attend(p, rng, rows, 2)


@pytest.mark.parametrize("bits,page", [(4, 32), (8, 128)])
@pytest.mark.parametrize("heads,q_heads,rows", [(1, 1, 5), (2, 6, 3), (1, 8, 1), (1, 8, 2), (2, 10, 3), (1, 4, 8),
                                                (1, 3, 40), (1, 2, 128), (1, 5, 150)])
@pytest.mark.parametrize("frame", [0, 1, 50])
def test_attention_grouped_heads_and_frame_masks(bits, page, heads, q_heads, rows, frame):
    rng = np.random.default_rng(rows * 7 + frame)
    p = Pool(rng, [420, rows, max(1, rows - 3), 1, 0], heads, page, bits)
    _fill(p, rng)
    _attend(p, rng, rows, q_heads, frame)
    _attend(p, rng, rows, q_heads, frame, taken=[rows, max(0, rows - 1), 1, 0, rows])


@pytest.mark.parametrize("rows", [3, 20, 200])
def test_attention_many_short_scenes_and_long_ones(rows):
    """More problems than thread blocks, and problems that many of them share."""
    rng = np.random.default_rng(rows)
    lens = [int(x) for x in rng.integers(0, 200, 150)] + [9000, 1, 4000]
    p = Pool(rng, lens, 4 if rows < 100 else 2, 16, 4)
    _fill(p, rng)
    _attend(p, rng, rows, p.heads, taken=[int(x) for x in rng.integers(0, rows + 1, len(lens))])


@pytest.mark.parametrize("rows", [8, 16, 17, 24, 25, 32, 34, 48, 49, 64, 127, 128, 129, 255, 256, 257, 400])
@pytest.mark.parametrize("bits", [4, 8])
def test_attention_every_row_tile_and_its_borders(rows, bits):
    """Row counts on both sides of every tile and kernel border, over scenes that one block takes alone
    and scenes that many share."""
    rng = np.random.default_rng(rows + bits)
    p = Pool(rng, [5000, 140, 0, rows], 1, 64, bits)
    _fill(p, rng)
    _attend(p, rng, rows, 1)
    _attend(p, rng, rows, 1, frame=33, taken=[rows, rows // 2, rows, max(0, rows - 1)])


@pytest.mark.parametrize("rows", [1, 20, 60, 300])
def test_attention_more_problems_than_blocks_all_cut(rows):
    """Many heads of a length that leaves nearly every block with an end and a beginning."""
    rng = np.random.default_rng(rows)
    p = Pool(rng, [1700], 61, 128, 8)
    _fill(p, rng)
    _attend(p, rng, rows, 61 * 2 if rows < 50 else 61)


@pytest.mark.parametrize("rows", [3, 150])
def test_a_wait_that_runs_out_is_reported_and_the_context_survives(rows):
    from view_recon_b200 import sa
    import time
    rng = np.random.default_rng(17)
    p = Pool(rng, [2000, 7], 3, 64, 4)
    _fill(p, rng)
    _, tq, layer = _attend(p, rng, rows, 3)
    layer.ws.random_(0, 256)   # notes of an earlier call would name parts that this one has not made
    try:
        sa.sa_set_wait_limit_ns(50_000_000)
        sa.sa_test_withhold_query_load(True)
        t0 = time.time()
        layer.forward(tq)
        status = sa.sa_check_device_error()
        elapsed = time.time() - t0
    finally:
        sa.sa_test_withhold_query_load(False)
        sa.sa_set_wait_limit_ns(2_000_000_000)
    assert status == sa.SA_ERR_TIMEOUT and elapsed < 20.0
    _ok()
    _attend(p, rng, rows, 3)


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (8, "f32")])
def test_rows_on_sixteen_byte_boundaries(bits, dtype):
    """Rows that start 16 bytes past a 32-byte boundary, and the refusal of less."""
    import torch
    rng = np.random.default_rng(18)
    p = Pool(rng, [77], 2, 32, bits)
    k, tk = _rows(rng, (2, 77, 64), dtype)
    off = 16 // tk.element_size()

    def shifted(t):
        buf = torch.zeros(t.numel() + off, dtype=t.dtype, device="cuda")
        out = buf[off:].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % 32 == 16
        return out

    p.cache.append(shifted(tk), shifted(tk))
    a, b = p.cache.read(shifted(torch.zeros_like(tk)), shifted(torch.zeros_like(tk)))
    _ok()
    ref = orc.cache_numbers(k, bits)
    assert np.array_equal(H.from_device(a), ref) and np.array_equal(H.from_device(b), ref)
    bad = torch.zeros(tk.numel() + 1, dtype=tk.dtype, device="cuda")[1:].view(tk.shape)
    with pytest.raises(ValueError):
        p.cache.append(bad, tk)
    with pytest.raises(ValueError):
        p.cache.append(tk.cpu(), tk.cpu())


@pytest.mark.parametrize("rows", [2, 150])
@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_attention_scales_and_peaked_rows(rows, scale):
    rng = np.random.default_rng(8)
    p = Pool(rng, [3000], 2, 64, 4)
    _fill(p, rng)
    _attend(p, rng, rows, 2, scale=scale, q_spread=1.5)


@pytest.mark.parametrize("rows", [4, 140])
def test_scores_rising_along_the_cache(rows):
    """Every later tile raises the running maximum, by a lot or by a little."""
    import torch
    rng = np.random.default_rng(9)
    for step in (0.5, 0.004):
        p = Pool(rng, [1500], 1, 128, 8)
        k = np.ones((1, 1500, 64)) * (step * np.arange(1500))[None, :, None]
        t = torch.from_numpy(k.astype(np.float32)).cuda()
        _, v = _rows(rng, (1, 1500, 64), "f32")
        p.cache.append(t, v)
        from view_recon_b200.pipeline import CachedGlobalAttention
        q = np.broadcast_to(np.where(np.arange(rows) % 2, -1.0, 1.0)[None, :, None], (1, rows, 64)).copy()
        layer = CachedGlobalAttention(p.cache, rows)
        layer.forward(torch.from_numpy(q).to(torch.bfloat16).cuda())
        _ok()
        _check(p, q, H.from_device(layer.o), H.from_device(layer.lse), 1, 0, [rows])


@pytest.mark.parametrize("rows", [1, 40, 140])
def test_nan_in_one_query_row_stays_there(rows):
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention
    rng = np.random.default_rng(10)
    p = Pool(rng, [260], 2, 32, 4)
    _fill(p, rng)
    q, tq = _rows(rng, (2, rows, 64), "bf16")
    tq[1, rows - 1, 3] = float("nan")
    layer = CachedGlobalAttention(p.cache, rows)
    o, lse = layer.forward(tq)
    _ok()
    assert o[1, rows - 1].isnan().all() and lse[1, rows - 1].isnan()
    o[1, rows - 1], lse[1, rows - 1] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    q[1, rows - 1] = 0
    ref, ref_l, A, B = orc.cache_attend(q, *p.rows(0), 0.125)
    ref[1, rows - 1], ref_l[1, rows - 1] = 0, 0
    err = np.abs(H.from_device(o) - ref)
    assert (err <= _bar(ref, A)).all()
    assert (np.abs(H.from_device(lse) - ref_l) <= 2.0 ** -18 * B + 2.0 ** -20 * (1 + np.abs(ref_l))).all()


@pytest.mark.parametrize("rows", [2, 140])
def test_bad_pages_and_lengths_are_reported_and_left_out(rows):
    import torch
    from view_recon_b200 import sa
    from view_recon_b200.pipeline import CachedGlobalAttention
    rng = np.random.default_rng(11)
    p = Pool(rng, [300], 2, 32, 4)
    _fill(p, rng)
    K, V = p.rows(0)
    q, tq = _rows(rng, (2, rows, 64), "bf16")
    layer = CachedGlobalAttention(p.cache, rows)
    good = p.t_table.clone()
    for bad in (-1, p.cache.n_pages, 2 ** 31 - 1, -2 ** 31):
        p.t_table[0, 3] = bad          # tokens 96..127
        layer.forward(tq)
        _ok(sa.SA_ERR_BAD_LIST)
        keep = np.r_[0:96, 128:300]
        ref, ref_l, A, B = orc.cache_attend(q, K[:, keep], V[:, keep], 0.125)
        err = np.abs(H.from_device(layer.o) - ref)
        assert (err <= _bar(ref, A)).all()
        out = torch.full((2, 300, 64), -7.0, device="cuda")
        p.cache.read(k=out)
        _ok(sa.SA_ERR_BAD_LIST)
        assert (out[:, 96:128] == -7).all() and np.array_equal(H.from_device(out)[:, keep], K[:, keep])
        raw = p.t_pool.clone()
        p.cache.append(out, out)
        _ok(sa.SA_ERR_BAD_LIST)
        assert torch.equal(p.t_pool[good[0, 3].item()], raw[good[0, 3].item()])
        p.t_pool.copy_(raw)
    p.t_table[:] = -1                  # no page at all: rows that see nothing
    layer.forward(tq)
    _ok(sa.SA_ERR_BAD_LIST)
    assert (layer.o == 0).all() and torch.isneginf(layer.lse).all()
    p.t_table.copy_(good)
    # lengths and counts out of range are clamped
    p.t_lens.fill_(-5)
    layer.forward(tq)
    _ok(sa.SA_ERR_INVALID_ARG)
    assert (layer.o == 0).all() and torch.isneginf(layer.lse).all()
    p.t_lens.fill_(300)
    layer.forward(tq, q_len=_counts([rows + 1]))
    _ok(sa.SA_ERR_INVALID_ARG)
    _check(p, q, H.from_device(layer.o), H.from_device(layer.lse), 2, 0, [rows])
    layer.o.fill_(-3.0)
    layer.forward(tq, q_len=_counts([-1]))
    _ok(sa.SA_ERR_INVALID_ARG)
    assert (layer.o == -3).all()
    p.t_lens.fill_(2 ** 30)           # more than the table's columns hold
    p.t_table.copy_(torch.where(p.t_table < 0, 0, p.t_table))
    layer.forward(tq)
    _ok(sa.SA_ERR_INVALID_ARG)
    p.t_lens.fill_(3)                  # more rows than the scene has tokens: the last three are stored
    x, t = _rows(rng, (2, 10, 64), "f32")
    p.cache.append(t, t)
    _ok(sa.SA_ERR_INVALID_ARG)
    p.lens = [3]
    assert np.array_equal(p.rows(0)[0], orc.cache_numbers(x[:, 7:], 4))


def test_pages_beyond_four_gigabytes():
    """A pool whose last pages lie past 2^32 bytes (and past 2^31 of them for one head)."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(12)
    page, heads, bits = 128, 2, 8
    n_pages = (5 << 30) // (heads * page * 136)
    pool = torch.empty((n_pages, heads, page * 136), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2, n_pages // 2]], dtype=torch.int32, device="cuda")
    c = FrameCache.wrap(pool, table, _counts([500]), page=page, bits=bits)
    k, tk = _rows(rng, (heads, 500, 64), "f32")
    v, tv = _rows(rng, (heads, 500, 64), "f32")
    c.append(tk, tv)
    out = c.read(torch.empty_like(tk), torch.empty_like(tv))
    _ok()
    K, V = orc.cache_numbers(k, bits), orc.cache_numbers(v, bits)
    assert np.array_equal(H.from_device(out[0]), K) and np.array_equal(H.from_device(out[1]), V)
    for rows in (1, 130):
        q, tq = _rows(rng, (heads, rows, 64), "bf16")
        layer = CachedGlobalAttention(c, rows)
        layer.forward(tq)
        _ok()
        ref, _, A, _ = orc.cache_attend(q, K, V, 0.125)
        assert (np.abs(H.from_device(layer.o) - ref) <= _bar(ref, A)).all()


@pytest.mark.parametrize("rows", [3, 30, 300])
def test_attention_repeats_bit_for_bit(rows):
    import torch
    rng = np.random.default_rng(13)
    p = Pool(rng, [20000, 3, 700], 2, 128, 4)
    _fill(p, rng)
    _, tq, layer = _attend(p, rng, rows, 2)
    first = layer.o.clone(), layer.lse.clone()
    for _ in range(3):
        layer.o.zero_()
        layer.ws.random_(0, 256)
        layer.forward(tq)
        assert torch.equal(layer.o, first[0]) and torch.equal(layer.lse, first[1])


@pytest.mark.parametrize("rows", [2, 140])
def test_graph_follows_lengths_and_pages(rows):
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(14)
    c = FrameCache(2, 2, tokens=900, page=32, bits=4)
    other = FrameCache(2, 2, tokens=900, page=32, bits=8, like=c)
    lay = [CachedGlobalAttention(c, rows), CachedGlobalAttention(other, rows, frame=100)]
    K, V = [[np.zeros((2, 0, 64))] * 2 for _ in range(2)], [[np.zeros((2, 0, 64))] * 2 for _ in range(2)]
    tq = torch.zeros((4, rows, 64), dtype=torch.bfloat16, device="cuda")
    graphs = [x.capture(tq) for x in lay]
    for ns in ([300, 1], [1, 0], [150, 333]):
        c.grow(ns)
        for i, x in enumerate((c, other)):
            k, tk = _rows(rng, (4, 333, 64), "bf16")
            v, tv = _rows(rng, (4, 333, 64), "bf16")
            x.append(tk, tv, new_len=_counts(ns))
            for s in range(2):
                K[i][s] = np.concatenate([K[i][s], orc.cache_numbers(k[2 * s:2 * s + 2, :ns[s]], x.bits)], 1)
                V[i][s] = np.concatenate([V[i][s], orc.cache_numbers(v[2 * s:2 * s + 2, :ns[s]], x.bits)], 1)
        q, new = _rows(rng, (4, rows, 64), "bf16")
        tq.copy_(new)
        for i in range(2):
            graphs[i].replay()
        _ok()
        for i in range(2):
            o, lse = H.from_device(lay[i].o), H.from_device(lay[i].lse)
            for s in range(2):
                ref, ref_l, A, B = orc.cache_attend(q[2 * s:2 * s + 2], K[i][s], V[i][s], 0.125, 100 * i)
                err = np.abs(o[2 * s:2 * s + 2] - ref)
                assert (err <= _bar(ref, A)).all()
                live = ~np.isneginf(ref_l)
                assert (np.isneginf(lse[2 * s:2 * s + 2]) == ~live).all()


def test_two_layers_on_two_streams():
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention
    rng = np.random.default_rng(15)
    p = Pool(rng, [30000], 4, 128, 4)
    _fill(p, rng)
    torch.cuda.synchronize()
    for rows in (2, 200):
        q, tq = _rows(rng, (4, rows, 64), "bf16")
        q2, tq2 = _rows(rng, (4, rows, 64), "bf16")
        a, b = CachedGlobalAttention(p.cache, rows), CachedGlobalAttention(p.cache, rows)
        a.forward(tq)
        b.forward(tq2)
        torch.cuda.synchronize()
        want = [x.clone() for x in (a.o, a.lse, b.o, b.lse)]
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for _ in range(10):
            a.forward(tq, stream=s1)
            b.forward(tq2, stream=s2)
        torch.cuda.synchronize()
        for x, y in zip((a.o, a.lse, b.o, b.lse), want):
            assert torch.equal(x, y)


def test_streaming_frames_as_they_would_be_used():
    """Three layers, two scenes: frames arrive, are stored and attended to, one scene is dropped and
    another takes its pages; and the dense attention over the rows read back agrees."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache, dense_attention
    rng = np.random.default_rng(16)
    N, heads = 137, 3
    caches = [FrameCache(2, heads, tokens=6 * N, n_pages=90, page=16, bits=4)]
    caches += [FrameCache(2, heads, tokens=6 * N, page=16, bits=b, like=caches[0]) for b in (8, 4)]
    frame_layers = [CachedGlobalAttention(c, N, frame=N) for c in caches]
    token_layers = [CachedGlobalAttention(c, 5) for c in caches]
    K, V = [[[], []] for _ in caches], [[[], []] for _ in caches]
    for step in range(7):
        if step == 4:
            caches[0].release(1)
            for i in range(3):
                K[i][1], V[i][1] = [], []
        caches[0].grow([N if step < 5 else 0, N])
        new = _counts([N if step < 5 else 0, N])
        for i, c in enumerate(caches):
            k, tk = _rows(rng, (2 * heads, N, 64), "bf16")
            v, tv = _rows(rng, (2 * heads, N, 64), "bf16")
            c.append(tk, tv, new_len=new)
            for s in range(2):
                if step < 5 or s == 1:
                    K[i][s].append(orc.cache_numbers(k[s * heads:(s + 1) * heads], c.bits))
                    V[i][s].append(orc.cache_numbers(v[s * heads:(s + 1) * heads], c.bits))
            for layer, rows in ((frame_layers[i], N), (token_layers[i], 5)):
                q, tq = _rows(rng, (2 * heads, rows, 64), "bf16")
                layer.forward(tq)
                _ok()
                o = H.from_device(layer.o)
                for s in range(2):
                    ref, _, A, _ = orc.cache_attend(q[s * heads:(s + 1) * heads], np.concatenate(K[i][s], 1),
                                                    np.concatenate(V[i][s], 1), 0.125, layer.frame)
                    err = np.abs(o[s * heads:(s + 1) * heads] - ref)
                    assert (err <= _bar(ref, A)).all()
    # the framework's dense attention over the rows read back: scene 0 has five frames, all of them queries
    c = caches[0]
    L = 5 * N
    k, v = (torch.zeros((2 * heads, L, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c.read(k, v, start=_counts([0, 0]))
    _, tq = _rows(rng, (heads, L, 64), "bf16")
    od, ld = dense_attention(tq, k[:heads].contiguous(), v[:heads].contiguous(), 5, N)
    whole = CachedGlobalAttention(c, L)
    o, lse = whole.forward(torch.cat([tq, tq]), q_len=_counts([L, 0]))
    _ok()
    # each is within 2^-8 (|O| + A) of the exact value, |O| <= A <= max |v|
    assert (o[:heads].float() - od.float()).abs().max().item() <= 4 * 2.0 ** -8 * v.abs().max().item()
    assert (lse[:heads] - ld).abs().max().item() <= 1e-3


def test_pages_and_lengths_stay_out_of_graphs():
    import torch
    from view_recon_b200.pipeline import FrameCache
    c = FrameCache(2, 2, tokens=200, page=16)
    c.grow([20, 5])
    x = torch.zeros(8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.add_(1)
        with pytest.raises(RuntimeError):
            c.grow(1)
        with pytest.raises(RuntimeError):
            c.release(0)
    g.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1.0] * 8 and c.lens.tolist() == [20, 5] and c._len == [20, 5]
    assert (c.page_table >= 0).sum().item() == 3


def test_growing_in_step_with_queued_work():
    """Lengths and pages sent while earlier calls are still queued arrive in their turn: every call sees its own."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(21)
    N, steps, heads = 37, 24, 2
    rows = [_rows(rng, (heads, N, 64), "bf16") for _ in range(2 * steps)]
    q, tq = _rows(rng, (heads, 4, 64), "bf16")
    c = FrameCache(1, heads, tokens=N * steps, page=16)
    layer = CachedGlobalAttention(c, 4)
    busy = torch.randn((6000, 6000), device="cuda")
    torch.cuda.synchronize()
    for _ in range(8):
        busy = busy @ busy * 1e-3                  # some milliseconds of work ahead of the first copy
    outs = []
    for i in range(steps):
        c.grow(N)
        c.append(rows[2 * i][1], rows[2 * i + 1][1])
        outs.append(layer.forward(tq)[0].clone())
    _ok()
    for i in (0, 1, 7, steps - 1):
        k = np.concatenate([orc.cache_numbers(rows[2 * j][0], 4) for j in range(i + 1)], 1)
        v = np.concatenate([orc.cache_numbers(rows[2 * j + 1][0], 4) for j in range(i + 1)], 1)
        ref, _, A, _ = orc.cache_attend(q, k, v, 0.125, 0)
        assert (np.abs(H.from_device(outs[i]) - ref) <= _bar(ref, A)).all()


@pytest.mark.parametrize("scenes", [14, 66])
@pytest.mark.parametrize("rows,bits", [(2, 8), (20, 4), (100, 8), (300, 4)])
def test_attention_long_runs_of_problems(rows, bits, scenes):
    """So much work that a problem's beginning counts in the cut; short problems beside long ones."""
    rng = np.random.default_rng(rows + scenes)
    heads = 14 if scenes == 14 else 4
    lens = [1900 + int(x) for x in rng.integers(0, 200, scenes)]
    lens[3:6] = [0, 1, 130]
    p = Pool(rng, lens, heads, 128, bits)
    _fill(p, rng)
    taken = [rows] * scenes
    taken[1], taken[6] = 0, max(1, rows // 3)
    _attend(p, rng, rows, heads, taken=taken)
    if rows in (20, 300):
        _attend(p, rng, rows, heads, frame=7, taken=taken)


def test_rows_without_keys_past_two_to_the_31_pieces():
    """Empty scenes of so many heads that a row tile's 16-byte pieces of O are more than 2^31: every row gets its
    zeros.  (Queries and O are one tensor, which rows without keys allow, to hold half the memory.)"""
    import torch
    from view_recon_b200 import sa
    heads, rows = 1 << 20, 256
    c = sa.kv_cache(1, heads, 1, 1, 16, 4)
    pool = torch.empty((sa.sa_kv_pool_size(c),), dtype=torch.uint8, device="cuda")
    o = torch.empty((heads, rows, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((heads, rows), device="cuda")
    o.fill_(1.0)
    lse.fill_(1.0)
    ws = torch.empty((sa.sa_kv_attn_workspace_size(c, heads, rows),), dtype=torch.uint8, device="cuda")
    table, lens = torch.full((1, 1), -1, dtype=torch.int32, device="cuda"), _counts([0])
    sa.sa_kv_attn_fwd(c, o, heads, rows, None, 0, 0.0, lens, table, pool, ws, o, lse)
    _ok()
    assert all((part == 0).all().item() for part in o.split(1 << 16))
    assert all(torch.isneginf(part).all().item() for part in lse.split(1 << 18))


def _same(got, ref):
    """O and LSE of a call within their bars of the oracle's (O, LSE, A, B)."""
    o, lse = (H.from_device(t) for t in got)
    ref_o, ref_l, A, B = ref
    dead = np.isneginf(ref_l)
    assert (np.abs(o - ref_o) <= _bar(ref_o, A)).all()
    assert (np.isneginf(lse) == dead).all() and (o[dead] == 0).all()
    assert (np.abs(lse - ref_l)[~dead] <= (2.0 ** -18 * B + 2.0 ** -20 * (1 + np.abs(ref_l)))[~dead]).all()


def test_lengths_and_pages_change_on_the_stream_of_the_calls():
    """Frames counted in, written and attended to on a side stream, while the current one is far behind."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(22)
    N, heads, steps = 45, 2, 4
    s = torch.cuda.Stream()
    rows = [_rows(rng, (heads, N, 64), "bf16") for _ in range(2 * steps)]
    q, tq = _rows(rng, (heads, 3, 64), "bf16")
    c = FrameCache(1, heads, tokens=N * steps, page=16)
    layer = CachedGlobalAttention(c, 3)
    outs = []
    torch.cuda.synchronize()
    for i in range(steps):
        torch.cuda._sleep(20_000_000)
        c.grow(N, stream=s)
        c.append(rows[2 * i][1], rows[2 * i + 1][1], stream=s)
        layer.forward(tq, stream=s)
        with torch.cuda.stream(s):
            outs.append((layer.o.clone(), layer.lse.clone()))
    c.release(0, stream=s)
    layer.forward(tq, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()      # the current stream is still asleep
    assert (layer.o == 0).all() and torch.isneginf(layer.lse).all()
    _ok()
    for i in range(steps):
        k = np.concatenate([orc.cache_numbers(rows[2 * j][0], 4) for j in range(i + 1)], 1)
        v = np.concatenate([orc.cache_numbers(rows[2 * j + 1][0], 4) for j in range(i + 1)], 1)
        _same(outs[i], orc.cache_attend(q, k, v, 0.125))
    assert c.lens.tolist() == [0] and (c.page_table == -1).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):                 # recorded on the stream that is named
        with pytest.raises(RuntimeError):
            c.grow(1, stream=s)
        torch.zeros(1, device="cuda")
    assert c._len == [0]


@pytest.mark.parametrize("rows", [3, 200])
def test_tensors_of_calls_on_a_side_stream_live_until_they_have_run(rows):
    """Rows, queries, counts and a layer's workspace dropped right after a call that is still queued on another
    stream: their memory is not handed out again before it has run."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention
    rng = np.random.default_rng(23)
    p = Pool(rng, [20000], 2, 64, 4)
    _fill(p, rng)
    k, tk = _rows(rng, (2, 300, 64), "bf16")
    v, tv = _rows(rng, (2, 300, 64), "bf16")
    q, tq = _rows(rng, (2, rows, 64), "bf16")
    tn, tm = _counts([300]), _counts([rows])
    s = torch.cuda.Stream()
    for cycles in (1000, 200_000_000):   # once to have memory and kernels loaded: getting those waits for the device
        a, b, n, x, m = (t.clone() for t in (tk, tv, tn, tq, tm))
        layer = CachedGlobalAttention(p.cache, rows)
        o, lse, size = layer.o, layer.lse, layer.ws.numel()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(cycles)
        p.cache.append(a, b, new_len=n, stream=s)
        layer.forward(x, q_len=m, stream=s)
        del a, b, n, x, m, layer
        junk = [torch.full_like(t, 7) for _ in range(8) for t in (tk, tq, tn)]
        junk += [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]
        torch.cuda.current_stream().synchronize()
        ahead = not s.query()
        _ok()
        K, V = p.rows(0)
        assert np.array_equal(K[:, 19700:], orc.cache_numbers(k, 4))
        assert np.array_equal(V[:, 19700:], orc.cache_numbers(v, 4))
        _same((o, lse), orc.cache_attend(q, K, V, 0.125))
        del junk
    assert ahead                         # all of that came before the calls


@pytest.mark.parametrize("rows", [2, 60])
def test_recorded_writes_and_calls_follow_the_cache(rows):
    """One graph that writes a frame, attends to the cache and reads the frame back, replayed as frames come, a
    scene is dropped and its pages are used again: O, LSE and the rows at every step."""
    import torch
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(24)
    N, heads = 70, 2
    c = FrameCache(2, heads, tokens=5 * N, n_pages=34, page=16, bits=8)
    layer = CachedGlobalAttention(c, rows, q_heads=2 * heads)
    tk, tv, out = (torch.zeros((2 * heads, N, 64), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    tq = torch.zeros((4 * heads, rows, 64), dtype=torch.bfloat16, device="cuda")
    c.grow(N)
    c.append(tk, tv)
    layer.forward(tq)
    c.read(v=out)
    c.release(0)
    c.release(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(tk, tv)
        layer.forward(tq)
        c.read(v=out)
    K, V = ([np.zeros((heads, 0, 64))] * 2 for _ in range(2))
    for step in range(7):
        if step in (3, 5):
            s = step // 2 - 1
            c.release(s)
            K[s] = V[s] = np.zeros((heads, 0, 64))
        c.grow(N)
        k, new_k = _rows(rng, tuple(tk.shape), "bf16")
        v, new_v = _rows(rng, tuple(tv.shape), "bf16")
        q, new_q = _rows(rng, tuple(tq.shape), "bf16")
        for a, b in ((tk, new_k), (tv, new_v), (tq, new_q)):
            a.copy_(b)
        g.replay()
        _ok()
        assert np.array_equal(H.from_device(out), orc.cache_numbers(v, 8))
        for s in range(2):
            mine = slice(s * heads, (s + 1) * heads)
            K[s] = np.concatenate([K[s], orc.cache_numbers(k[mine], 8)], 1)
            V[s] = np.concatenate([V[s], orc.cache_numbers(v[mine], 8)], 1)
            mine = slice(2 * s * heads, 2 * (s + 1) * heads)
            _same((layer.o[mine], layer.lse[mine]), orc.cache_attend(q[mine], K[s], V[s], 0.125))


@pytest.mark.parametrize("rows", [4, 100])
def test_binding_calls_and_layer_objects_agree(rows):
    """The thin binding's three calls, with scenes that share their first pages, and no LSE asked for."""
    import torch
    from view_recon_b200 import sa
    from view_recon_b200.pipeline import CachedGlobalAttention, FrameCache
    rng = np.random.default_rng(25)
    page, heads = 32, 2
    table = torch.tensor([[4, 0, 2], [4, 0, 3]], dtype=torch.int32, device="cuda")
    lens = _counts([90, 70])
    pools = [torch.zeros((5, heads, page * 72), dtype=torch.uint8, device="cuda") for _ in range(2)]
    caches = [FrameCache.wrap(p, table, lens, page=page) for p in pools]
    desc = caches[0].desc
    first, first_k = _rows(rng, (2 * heads, 64, 64), "f32")
    k, tk = _rows(rng, (2 * heads, 26, 64), "f32")
    shared = _counts([64, 64])
    own = _counts([26, 6])
    sa.sa_kv_append(desc, first_k, first_k, 64, _counts([64, 0]), shared, table, pools[0])   # the shared pages, once
    sa.sa_kv_append(desc, tk, tk, 26, own, lens, table, pools[0])
    whole = FrameCache.wrap(pools[1], table, shared, page=page)
    whole.append(first_k, first_k, new_len=_counts([64, 0]))
    caches[1].append(tk, tk, new_len=own)
    _ok()
    assert torch.equal(*pools)
    a, b = (torch.zeros((2 * heads, 26, 64), device="cuda") for _ in range(2))
    sa.sa_kv_read(desc, 26, own, None, lens, table, pools[0], None, a)
    caches[1].read(v=b, n_len=own)
    q, tq = _rows(rng, (2 * heads, rows, 64), "bf16")
    ws = torch.empty((sa.sa_kv_attn_workspace_size(desc, heads, rows),), dtype=torch.uint8, device="cuda")
    o = torch.zeros((2 * heads, rows, 64), dtype=torch.bfloat16, device="cuda")
    sa.sa_kv_attn_fwd(desc, tq, heads, rows, None, 0, 0.0, lens, table, pools[0], ws, o)
    plain = CachedGlobalAttention(caches[1], rows, with_lse=False)
    got, none = plain.forward(tq)
    layer = CachedGlobalAttention(caches[1], rows)
    layer.forward(tq)
    _ok()
    assert none is None and torch.equal(a, b) and torch.equal(o, got) and torch.equal(o, layer.o)
    for s, m in ((0, 26), (1, 6)):
        K = np.concatenate([orc.cache_numbers(first[:heads], 4),
                            orc.cache_numbers(k[s * heads:(s + 1) * heads, :m], 4)], 1)
        mine = slice(s * heads, (s + 1) * heads)
        _same((layer.o[mine], layer.lse[mine]), orc.cache_attend(q[mine], K, K, 0.125))


def test_recording_a_write_is_not_a_write():
    """A graph recorded between two grows: the tokens of both are still to be written, together or by the replay."""
    import torch
    from view_recon_b200.pipeline import FrameCache
    rng = np.random.default_rng(26)
    c = FrameCache(1, 2, tokens=64, page=16)
    k, tk = _rows(rng, (2, 9, 64), "bf16")
    part = tk[:, :5].contiguous()
    c.grow(5)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.append(tk, tk)                 # nine rows, of which five have been counted in by now
    c.grow(4)
    c.append(tk, tk)
    out, _ = c.read(torch.empty_like(tk), torch.empty_like(tk))
    _ok()
    assert np.array_equal(H.from_device(out), orc.cache_numbers(k, 4))
    with pytest.raises(ValueError):
        c.append(part, part)
    c.release(0)
    c.grow(9)
    g.replay()
    out, _ = c.read(torch.empty_like(tk), torch.empty_like(tk))
    _ok()
    assert np.array_equal(H.from_device(out), orc.cache_numbers(k, 4))
