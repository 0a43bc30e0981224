"""One sparse global-attention layer call: the four C-ABI steps on caller-visible buffers.

`SparseGlobalAttention` owns the intermediate device buffers (tile means,
scores or the streamed-selection block, kept lists, landmark workspace) as
torch tensors and runs

    sa_tile_pool -> sa_tile_scores (materialised mode only) -> sa_select_topk
                 -> sa_sparse_attn_fwd

on the current CUDA stream.  torch provides device memory and streams only;
every step runs in libsa's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import numbers

from . import sa


@dataclasses.dataclass
class Buffers:
    q_pool: object
    k_pool: object
    v_pool: object
    k_cnt: object
    sink_k: object
    sink_v: object
    scores: object
    sel_ws: object
    kept_idx: object
    kept_cnt: object
    attn_ws: object
    o: object
    lse: object


@dataclasses.dataclass
class GradBuffers:
    ws: object
    dq: object
    dk: object
    dv: object


class SparseGlobalAttention:
    """Dynamic tile-sparse global attention for bh heads of S frames x N tokens (d = 64).

    k          key tiles chosen per query tile beyond its own frame's tiles: one budget for every
               head, or a sequence of bh per-head budgets (a budget at or above the candidate
               count makes that head dense)
    adaptive   None, or a dict(temperature=, beta=, k_lo=) that sets every head's budget on the
               device from the spread of its own pooled scores (sa_head_budgets) before each
               selection; k is then the largest budget (k_hi); temperature defaults to tile/sqrt(d)
    landmark   fold every unselected tile into one mean-K/mean-V token (+ln count bias)
    streamed   select without materialising the [bh][nt][nt] score matrix
    """

    def __init__(self, bh: int, frames: int, tokens: int, k: int, tile: int = 128, n_sink: int = 5,
                 dtype: str = "bf16", landmark: bool = False, streamed: bool = False, head_dim: int = 64,
                 device=None, with_lse: bool = True, adaptive=None):
        import torch
        self.shape = sa.shape(bh, frames, tokens, head_dim, tile, n_sink, dtype)
        self.adaptive = None
        if adaptive is not None:
            if not (isinstance(k, int) or getattr(k, "ndim", None) == 0):
                raise ValueError("with adaptive budgets k is the single largest budget")
            ad = dict(adaptive)
            self.adaptive = (float(ad.get("temperature", tile / head_dim ** 0.5)), float(ad.get("beta", 1.0)),
                             int(ad.get("k_lo", 0)), int(k))
        if isinstance(k, (int,)) or getattr(k, "ndim", None) == 0:
            self.k, self.k_per_head = int(k), None
        else:
            ks = [int(x) for x in k]
            if len(ks) != bh or min(ks) < 0:
                raise ValueError("k needs one non-negative budget per head")
            self.k, self.k_per_head = max(ks), ks
        self.landmark = bool(landmark)
        self.streamed = bool(streamed)
        self.nt = sa.sa_num_tiles(self.shape)
        if self.nt < 0:
            raise ValueError("invalid shape")
        self.max_kept = sa.sa_max_kept(self.shape, self.k)
        self.bh, self.frames, self.tokens, self.d = bh, frames, tokens, head_dim
        self.L = frames * tokens
        dev = torch.device(device if device is not None else "cuda")
        self.device = dev
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype = tdt
        f32, i32 = torch.float32, torch.int32
        nt = self.nt
        sel_bytes = sa.sa_select_workspace_size(self.shape, self.streamed)
        attn_bytes = sa.sa_sparse_attn_workspace_size(self.shape, self.landmark)
        self.k_head = (torch.tensor(self.k_per_head, dtype=torch.int32, device=dev)
                       if self.k_per_head is not None else None)
        self.perplexity = None
        self.budget_ws = None
        if self.adaptive is not None:
            self.k_head = torch.zeros((bh,), dtype=torch.int32, device=dev)
            self.perplexity = torch.zeros((bh,), dtype=torch.float32, device=dev)
            self.budget_ws = torch.empty((sa.sa_head_budget_workspace_size(self.shape),), dtype=torch.uint8,
                                         device=dev)
        self.buf = Buffers(
            q_pool=torch.empty((bh, nt, head_dim), dtype=f32, device=dev),
            k_pool=torch.empty((bh, nt, head_dim), dtype=f32, device=dev),
            v_pool=torch.empty((bh, nt, head_dim), dtype=f32, device=dev) if self.landmark else None,
            k_cnt=torch.empty((nt,), dtype=i32, device=dev),
            sink_k=torch.empty((bh, max(1, frames * n_sink), head_dim), dtype=tdt, device=dev),
            sink_v=torch.empty((bh, max(1, frames * n_sink), head_dim), dtype=tdt, device=dev),
            scores=None if self.streamed else torch.empty((bh, nt, nt), dtype=f32, device=dev),
            sel_ws=torch.empty((max(1, sel_bytes),), dtype=torch.uint8, device=dev) if sel_bytes else None,
            kept_idx=torch.empty((bh, nt, self.max_kept), dtype=i32, device=dev),
            kept_cnt=torch.empty((bh, nt), dtype=i32, device=dev),
            attn_ws=torch.empty((attn_bytes,), dtype=torch.uint8, device=dev) if attn_bytes else None,
            o=torch.empty((bh, self.L, head_dim), dtype=tdt, device=dev),
            lse=torch.empty((bh, self.L), dtype=f32, device=dev) if with_lse else None,
        )
        self.grad = None  # backward buffers, allocated by the first backward call

    # individual steps (each one C call) ---------------------------------------------------------
    def pool(self, q, k, v, stream=None):
        b = self.buf
        sa.sa_tile_pool(self.shape, q, k, v, b.q_pool, b.k_pool, b.v_pool, b.k_cnt, b.sink_k, b.sink_v, stream)

    def score(self, stream=None):
        if not self.streamed:
            sa.sa_tile_scores(self.shape, self.buf.q_pool, self.buf.k_pool, self.buf.scores, stream)

    def budgets(self, stream=None):
        """Adaptive mode: every head's budget from its own pooled scores (one C call)."""
        if self.adaptive is not None:
            tau, beta, k_lo, k_hi = self.adaptive
            sa.sa_head_budgets(self.shape, self.buf.q_pool, self.buf.k_pool, tau, beta, k_lo, k_hi, self.k_head,
                               self.perplexity, self.budget_ws, stream)

    def select(self, stream=None):
        b = self.buf
        self.budgets(stream)
        if self.k_head is None:
            sa.sa_select_topk(self.shape, b.scores, b.q_pool, b.k_pool, self.k, b.kept_idx, b.kept_cnt,
                              self.max_kept, b.sel_ws, stream)
        else:
            sa.sa_select_topk_per_head(self.shape, b.scores, b.q_pool, b.k_pool, self.k_head, self.k, b.kept_idx,
                                       b.kept_cnt, self.max_kept, b.sel_ws, stream)

    def attend(self, q, k, v, stream=None):
        b = self.buf
        sa.sa_sparse_attn_fwd(self.shape, q, k, v, b.kept_idx, b.kept_cnt, self.max_kept, b.sink_k, b.sink_v,
                              self.landmark, b.k_pool, b.v_pool, b.k_cnt, b.attn_ws, b.o, b.lse, stream)

    def forward(self, q, k, v, stream=None):
        """Run the whole layer call on device tensors [bh][S*N][d]; returns (O, LSE) buffers."""
        self.pool(q, k, v, stream)
        self.score(stream)
        self.select(stream)
        self.attend(q, k, v, stream)
        return self.buf.o, self.buf.lse

    __call__ = forward

    def capture(self, q, k, v):
        """Record one whole layer call on these input tensors as a CUDA graph and return it.

        `g.replay()` then re-runs every launch of the call (pooling, scoring, selection -- a few
        hundred launches in streamed mode -- and attention) from one host call, on the current
        stream; new inputs are written into q, k, v in place before a replay, and the results
        land in `self.buf.o` / `self.buf.lse` as with `forward`.  The library allocates nothing
        and every step is stream-ordered, so the call is captured as it runs.  One eager call
        comes first so that no kernel attribute is set inside the capture."""
        import torch
        self.forward(q, k, v)
        torch.cuda.current_stream(self.device).synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.forward(q, k, v)
        return g

    def backward(self, q, k, v, d_o, stream=None):
        """Gradients (dq, dk, dv) of sum(d_o * O) for the last forward on these q, k, v, with its
        kept lists held fixed; d_o is [bh][S*N][d] like O.  Needs the forward's LSE."""
        import torch
        b = self.buf
        if b.lse is None:
            raise ValueError("the backward needs the forward's LSE (with_lse=True)")
        if self.grad is None:
            nbytes = sa.sa_sparse_attn_bwd_workspace_size(self.shape, self.max_kept, self.landmark)
            if nbytes == 0:
                raise ValueError("no backward for this shape (bf16, tile 128, d 64 only)")
            dev = self.device
            self.grad = GradBuffers(
                ws=torch.empty((nbytes,), dtype=torch.uint8, device=dev),
                dq=torch.empty((self.bh, self.L, self.d), dtype=self.dtype, device=dev),
                dk=torch.empty((self.bh, self.L, self.d), dtype=self.dtype, device=dev),
                dv=torch.empty((self.bh, self.L, self.d), dtype=self.dtype, device=dev),
            )
        gr = self.grad
        sa.sa_sparse_attn_bwd(self.shape, q, k, v, b.o, b.lse, d_o, b.kept_idx, b.kept_cnt, self.max_kept,
                              b.sink_k, b.sink_v, self.landmark, b.k_pool, b.v_pool, b.k_cnt, gr.ws, gr.dq, gr.dk,
                              gr.dv, stream)
        return gr.dq, gr.dk, gr.dv

    def backward_launches(self) -> int:
        """Kernel launches libsa makes for one backward (memsets not counted)."""
        n = 1 + 3 + 3 + 3  # row terms; Q, dO, K transposes; list scan, plan, fill; dQ, dK/dV, finalize
        if self.frames * self.shape.n_sink > 0:
            n += 1  # transposed sink K tiles
        if self.landmark:
            n += 3  # landmark K and V tables, transposed landmark K chunks
        return n

    def launches_per_call(self) -> int:
        """Kernel launches libsa makes for one forward (for launch accounting)."""
        n = 1  # pooling
        if self.streamed:
            rows = sa.sa_select_workspace_size(self.shape, True) // (4 * self.nt)
            n += 2 * self.bh * (-(-self.nt // rows))  # score block + select block
        else:
            n += 2  # scores + select
        if self.adaptive is not None:
            n += 2  # per-head statistic + budgets
        n += 1  # attention
        if sa.sa_sparse_attn_workspace_size(self.shape, self.landmark) > 0:
            n += 1  # transposed V tiles
            if self.frames * self.shape.n_sink > 0:
                n += 1  # transposed sink V tiles
            if self.landmark:
                n += 1  # landmark tables
        return n


class HostPipeline:
    """Layer calls on host-resident (pinned) Q/K/V with the transfers overlapped.

    Two layer objects and two sets of device inputs alternate between calls; three streams
    carry the host-to-device copies, the four C-ABI steps and the device-to-host copy of O, so
    that the copy-in of call i+1 and the copy-out of call i-1 run while call i computes.
    `make_layer` builds one `SparseGlobalAttention`; inputs are [bh][L][d] host tensors.
    """

    def __init__(self, make_layer):
        import torch
        self.layers = [make_layer(), make_layer()]
        lay = self.layers[0]
        shape = (lay.bh, lay.L, lay.d)
        self.dev_in = [[torch.empty(shape, dtype=lay.dtype, device=lay.device) for _ in range(3)] for _ in range(2)]
        self.s_in = torch.cuda.Stream(lay.device)
        self.s_comp = torch.cuda.Stream(lay.device)
        self.s_out = torch.cuda.Stream(lay.device)
        self.ev_in = [torch.cuda.Event() for _ in range(2)]    # inputs of buffer set s are on the device
        self.ev_comp = [torch.cuda.Event() for _ in range(2)]  # the layer of set s has finished
        self.ev_out = [torch.cuda.Event() for _ in range(2)]   # O of set s has left the device
        self.calls = 0

    def submit(self, hq, hk, hv, ho):
        """Queue one call: hq, hk, hv pinned host inputs, ho the pinned host output."""
        import torch
        s = self.calls % 2
        self.calls += 1
        dq, dk, dv = self.dev_in[s]
        self.s_in.wait_event(self.ev_comp[s])  # the call two back has consumed these buffers
        with torch.cuda.stream(self.s_in):
            dq.copy_(hq, non_blocking=True)
            dk.copy_(hk, non_blocking=True)
            dv.copy_(hv, non_blocking=True)
        self.ev_in[s].record(self.s_in)
        self.s_comp.wait_event(self.ev_in[s])
        self.s_comp.wait_event(self.ev_out[s])  # O of the call two back has been copied out
        o, _ = self.layers[s].forward(dq, dk, dv, stream=self.s_comp)
        self.ev_comp[s].record(self.s_comp)
        self.s_out.wait_event(self.ev_comp[s])
        with torch.cuda.stream(self.s_out):
            ho.copy_(o, non_blocking=True)
        self.ev_out[s].record(self.s_out)

    def synchronize(self):
        self.s_out.synchronize()
        self.s_comp.synchronize()
        self.s_in.synchronize()


class SubsampledGlobalAttention:
    """Subsampled global attention (AVGGT SGA) for bh heads of S frames x N tokens, N = n_special +
    grid_h * grid_w: keys/values kept on a stride_h x stride_w grid of each frame's patches plus
    every special token, each token's own key, and one mean pair for the other discarded tokens.
    One C call (sa_sga_fwd); the workspace is allocated once."""

    def __init__(self, bh: int, frames: int, tokens: int, grid=(37, 37), stride=(3, 3), n_special: int = 5,
                 dtype: str = "bf16", head_dim: int = 64, device=None, with_lse: bool = True):
        import torch
        self.shape = sa.shape(bh, frames, tokens, head_dim, 128, n_special, dtype)
        self.grid = (int(grid[0]), int(grid[1]))
        self.stride = (int(stride[0]), int(stride[1]))
        nbytes = sa.sa_sga_workspace_size(self.shape, *self.grid, *self.stride)
        if nbytes == 0:
            raise ValueError("unsupported shape or grid for subsampled global attention")
        dev = torch.device(device if device is not None else "cuda")
        self.bh, self.frames, self.tokens, self.d = bh, frames, tokens, head_dim
        self.L = frames * tokens
        self.device = dev
        self.ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype = tdt
        kh = -(-self.grid[0] // self.stride[0])
        kw = -(-self.grid[1] // self.stride[1])
        self.kept_keys = frames * (n_special + kh * kw)  # compacted key sequence per head
        self.o = torch.empty((bh, self.L, head_dim), dtype=tdt, device=dev)
        self.lse = torch.empty((bh, self.L), dtype=torch.float32, device=dev) if with_lse else None

    def forward(self, q, k, v, stream=None):
        sa.sa_sga_fwd(self.shape, *self.grid, *self.stride, q, k, v, self.ws, self.o, self.lse, stream)
        return self.o, self.lse

    __call__ = forward


def dense_attention(q, k, v, frames: int, tokens: int, dtype: str = "bf16", with_lse: bool = True, stream=None):
    """Dense control on device tensors [bh][S*N][64]; returns (O, LSE)."""
    import torch
    bh = q.shape[0]
    shp = sa.shape(bh, frames, tokens, q.shape[2], 128, 0, dtype)
    o = torch.empty_like(q)
    lse = torch.empty((bh, frames * tokens), dtype=torch.float32, device=q.device) if with_lse else None
    nbytes = sa.sa_dense_attn_workspace_size(shp)
    ws = torch.empty((nbytes,), dtype=torch.uint8, device=q.device) if nbytes else None
    sa.sa_dense_attn_fwd(shp, q, k, v, ws, o, lse, stream)
    return o, lse


class DenseAttention:
    """Dense control with its workspace allocated once (for repeated calls at one shape)."""

    def __init__(self, bh: int, frames: int, tokens: int, dtype: str = "bf16", head_dim: int = 64, device=None):
        import torch
        self.shape = sa.shape(bh, frames, tokens, head_dim, 128, 0, dtype)
        dev = torch.device(device if device is not None else "cuda")
        nbytes = sa.sa_dense_attn_workspace_size(self.shape)
        self.ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.o = torch.empty((bh, frames * tokens, head_dim), dtype=tdt, device=dev)
        self.lse = torch.empty((bh, frames * tokens), dtype=torch.float32, device=dev)

    def __call__(self, q, k, v, stream=None):
        sa.sa_dense_attn_fwd(self.shape, q, k, v, self.ws, self.o, self.lse, stream)
        return self.o, self.lse


def _want(name, t, shape, dtypes, device, align=16):
    """Refuse a tensor that is not of this shape, one of these types, contiguous, aligned and on this device;
    returns its address.  (Calls of a few microseconds: the common case is one line of cheap tests.)"""
    if t.shape == shape and t.dtype in dtypes and t.device == device and t.is_contiguous() and t.data_ptr() % align == 0:
        return t.data_ptr()
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s has type %s, expected %s" % (name, t.dtype, " or ".join(str(d) for d in dtypes)))
    if t.device != device:
        raise ValueError("%s is on %s, the cache is on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % name)
    raise ValueError("%s does not start on a %d-byte boundary" % (name, align))


class _Counted:
    """What grow has counted into the scenes, shared by the caches of a model's layers: the last grow's counts, and
    those of all grows since the last append."""

    def __init__(self, scenes):
        self.last, self.open, self.appended, self.fits = [0] * scenes, [0] * scenes, False, ()

    def grow(self, ns):
        self.open = [m if self.appended else o + m for o, m in zip(self.open, ns)]
        self.last, self.appended = list(ns), False
        self._settle()

    def release(self, scene):
        self.last[scene] = self.open[scene] = 0
        self._settle()

    def _settle(self):
        self.fits = tuple(x[0] for x in (self.last, self.open) if min(x) == max(x))  # counts that suit every scene


class FrameCache:
    """K and V of the frames seen so far, of one layer, held in 4 or 8 bits in pages.

    scenes     independent scenes of any lengths
    heads      key/value heads
    tokens     the longest scene, in tokens
    n_pages    pages of the pool, shared by the scenes (default: enough for every scene at its longest)
    page       tokens per page (16, 32, 64 or 128)
    bits       4 (72 bytes per token and head for K and V) or 8 (136 bytes)

    `grow(n)` counts new tokens in and gives them pages; `append(k, v)` then writes their rows;
    `read` hands rows back; `CachedGlobalAttention` attends over them.  Lengths (`lens`) and page
    table (`page_table`) are device tensors read by the kernels when they run, so recorded graphs
    follow them.  The layers of a model see the same tokens: give the second and later layers'
    caches `like=` the first one and they share its lengths, its table and its pages' numbering
    (and only the first one's grow and release are called).  `wrap` adopts tensors that the caller
    manages.  Calls on one cache, grow and release among them, are ordered by the caller: one stream (each
    takes `stream=`; without it the device's current one), or events.
    """

    def __init__(self, scenes: int, heads: int, tokens: int, n_pages: int | None = None, page: int = 128, bits: int = 4,
                 head_dim: int = 64, device=None, like: "FrameCache | None" = None):
        import torch
        if page not in (16, 32, 64, 128):
            raise ValueError("page is 16, 32, 64 or 128 tokens")
        max_pages = -(-int(tokens) // page)
        if like is not None:
            if (like.scenes, like.page, like.max_pages) != (scenes, page, max_pages) or n_pages not in (None, like.n_pages):
                raise ValueError("a cache like another has its scenes, page size, length and pages")
            if device is not None and torch.device(device) not in (like.device, torch.device(like.device.type)):
                raise ValueError("a cache like another is on its device, %s" % like.device)
            n_pages, device = like.n_pages, like.device
        n_pages = scenes * max_pages if n_pages is None else int(n_pages)
        dev = torch.device(device if device is not None else "cuda")
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self._describe(scenes, heads, n_pages, max_pages, page, bits, head_dim, dev)
        self.pool = torch.empty((self.pool_bytes,), dtype=torch.uint8, device=dev)
        self._owner = like is None
        if like is not None:
            self.page_table, self.lens, self._news = like.page_table, like.lens, like._news
            return
        self.page_table = torch.full((scenes, max_pages), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros((scenes,), dtype=torch.int32, device=dev)
        self._len = [0] * scenes              # host copies: the pages' bookkeeping is the host's
        self._pages = [[] for _ in range(scenes)]
        self._free = list(range(n_pages - 1, -1, -1))
        self._news = _Counted(scenes)

    def _describe(self, scenes, heads, n_pages, max_pages, page, bits, head_dim, device):
        self.desc = sa.kv_cache(scenes, heads, n_pages, max_pages, page, bits, head_dim)
        self.pool_bytes = sa.sa_kv_pool_size(self.desc)
        if self.pool_bytes == 0:
            raise ValueError("unsupported cache (head_dim 64, 4 or 8 bits, at least one scene, head and page)")
        self.scenes, self.heads, self.n_pages, self.max_pages = scenes, heads, n_pages, max_pages
        self.page, self.bits, self.d, self.device = page, bits, head_dim, device
        import torch
        self._ref = ctypes.byref(self.desc)
        self._types = (torch.bfloat16, torch.float32)
        self._count = (torch.int32,)

    @classmethod
    def wrap(cls, pool, page_table, lens, page: int = 128, bits: int = 4, head_dim: int = 64) -> "FrameCache":
        """A cache over the caller's own tensors: pool uint8 [n_pages][heads][bytes of a page], page_table int32
        [scenes][max_pages], lens int32 [scenes].  The caller assigns pages and sets lengths."""
        import torch
        if pool.dim() != 3 or page_table.dim() != 2:
            raise ValueError("pool is [n_pages][heads][bytes], page_table [scenes][max_pages]")
        c = cls.__new__(cls)
        c._describe(page_table.shape[0], pool.shape[1], pool.shape[0], page_table.shape[1], page, bits, head_dim,
                    pool.device)
        per_page = c.pool_bytes // (c.n_pages * c.heads)
        _want("pool", pool, (c.n_pages, c.heads, per_page), (torch.uint8,), pool.device)
        _want("page_table", page_table, (c.scenes, c.max_pages), (torch.int32,), pool.device, 4)
        _want("lens", lens, (c.scenes,), (torch.int32,), pool.device, 4)
        c.pool, c.page_table, c.lens, c._owner, c._news = pool, page_table, lens, False, None
        return c

    # ---- pages and lengths (host bookkeeping, device tables)
    def _owned(self, stream):
        """Refuse what is not this cache's to change now; returns the context in which its tables are written."""
        if not self._owner:
            raise ValueError("pages and lengths of this cache are managed elsewhere")
        if self.device.type != "cuda":
            if stream is not None:
                raise ValueError("the cache is not on a CUDA device")
            return contextlib.nullcontext()
        import torch
        if stream is not None and stream.device != self.device:
            raise ValueError("the stream is on %s, the cache is on %s" % (stream.device, self.device))
        if self._recording(stream):
            raise RuntimeError("pages and lengths are the host's: change them outside a recorded graph")
        return torch.cuda.stream(torch.cuda.current_stream(self.device) if stream is None else stream)

    def _send(self, values, dtype):
        """Host numbers on the device.  From pinned memory, so that the host does not wait for the work that is
        queued before the copy (torch keeps the pinned block until the copy has run)."""
        import torch
        pin = self.device.type == "cuda"
        return torch.tensor(values, dtype=dtype, pin_memory=pin).to(self.device, non_blocking=pin)

    def _send_lengths(self, lens):
        import torch
        self.lens.copy_(self._send(lens, torch.int32))

    def grow(self, n, stream=None):
        """Count n more tokens (one number, or one per scene) into the cache and give them pages.  Call it once
        before the layers' appends.  Lengths and table change on `stream` (default: the device's current one),
        in order with the calls there.  Raises MemoryError, changing nothing, when pages run out."""
        there = self._owned(stream)
        ns = [n] * self.scenes if isinstance(n, numbers.Integral) else list(n)
        if len(ns) != self.scenes or any(int(x) != x for x in ns) or min(ns) < 0:
            raise ValueError("grow needs one non-negative count, or one per scene")
        lens = [have + int(x) for have, x in zip(self._len, ns)]
        if max(lens) > self.max_pages * self.page:
            raise ValueError("a scene is longer than its row of the page table")
        more = [-(-new // self.page) - len(have) for new, have in zip(lens, self._pages)]
        free = len(self._free) - sum(more)
        if free < 0:
            raise MemoryError("%d more pages needed, %d free" % (sum(more), len(self._free)))
        ids = self._free[:free - 1 if free else None:-1]  # from the end
        rows = [s for s in range(self.scenes) for _ in range(more[s])]
        cols = [len(self._pages[s]) + i for s in range(self.scenes) for i in range(more[s])]
        with there:
            if ids:
                import torch
                at = self._send([rows, cols, ids], torch.int64)
                self.page_table.index_put_((at[0], at[1]), at[2].to(torch.int32))
            self._send_lengths(lens)
        # the host's books last: what fails above (memory, the device) has changed nothing that a call reads
        del self._free[free:]
        for s, page in zip(rows, ids):
            self._pages[s].append(page)
        self._len = lens
        self._news.grow([int(x) for x in ns])
        if stream is not None:
            self._hold(stream)

    def release(self, scene: int, stream=None):
        """Drop a scene: its pages are free again and its length is 0, for what follows on `stream` (default:
        the device's current one)."""
        there = self._owned(stream)
        lens = list(self._len)
        lens[scene] = 0
        with there:
            self._send_lengths(lens)   # (first: should it fail, the table is as it was)
            self.page_table[scene].fill_(-1)
        self._free.extend(reversed(self._pages[scene]))
        self._pages[scene] = []
        self._len = lens
        self._news.release(scene)
        if stream is not None:
            self._hold(stream)

    # ---- rows (each one C call)
    def _counts(self, name, t):
        return None if t is None else _want(name, t, (self.scenes,), self._count, self.device, 4)

    def _call(self, fn, *args, stream):
        """One C call on the cache's device, on `stream` or the device's current one."""
        import torch
        index = self.device.index
        if index is None:
            raise ValueError("the cache is not on a CUDA device")
        if torch.cuda.current_device() == index:
            st = fn(self._ref, *args, sa.raw_stream(index, stream))
        else:
            with torch.cuda.device(index):
                st = fn(self._ref, *args, sa.raw_stream(index, stream))
        if st != sa.SA_OK:
            raise sa.SaError(fn.__name__, st, sa.status_string(st))

    def _recording(self, stream):
        import torch
        if self.device.type != "cuda":
            return False
        with torch.cuda.device(self.device), torch.cuda.stream(stream):
            return torch.cuda.is_current_stream_capturing()

    def _hold(self, stream, *tensors):
        """Tensors of a call that is queued on a stream that is named: their memory is not handed out again before
        the stream has come past it, whoever drops them."""
        for t in (*tensors, self.pool, self.page_table, self.lens):
            if t is not None and t.is_cuda:
                t.record_stream(stream)

    def append(self, k, v, new_len=None, stream=None):
        """Write rows k, v [scenes * heads][n][64] (bf16 or f32) as the last n tokens of every scene; with
        new_len (int32 device tensor [scenes]) only the first new_len[s] rows, as the last new_len[s] tokens.
        Without new_len, n has to be what the last grow counted into every scene, or what the grows since the last
        append did together: other rows would go over tokens that were there before, or leave new ones unwritten.
        (Not asked of caches that the caller manages, nor while a graph is recorded, whose replays have their own
        grows.)"""
        n = k.shape[1] if k.dim() == 3 else -1
        shape = (self.scenes * self.heads, n, self.d)
        pk = _want("k", k, shape, self._types, self.device)
        pv = _want("v", v, shape, (k.dtype,), self.device)
        if n == 0:
            return
        news = self._news
        if news is not None:
            if new_len is not None or n in news.fits:
                news.appended = True
            elif not self._recording(stream):  # (a recorded call writes when it is replayed)
                raise ValueError("%d rows for every scene, but the last grow counted in %s: rows of other counts "
                                 "need new_len" % (n, news.last))
        self._call(sa.load().sa_kv_append, sa.SA_BF16 if k.dtype is self._types[0] else sa.SA_F32, pk, pv, n,
                   self._counts("new_len", new_len), self.lens.data_ptr(), self.page_table.data_ptr(),
                   self.pool.data_ptr(), stream=stream)
        if stream is not None:
            self._hold(stream, k, v, new_len)

    def read(self, k=None, v=None, start=None, n_len=None, stream=None):
        """Fill k and v [scenes * heads][n][64] (bf16 or f32, either may be None) with the tokens from start[s]
        (default: the last n, or n_len[s], of each scene); returns (k, v)."""
        ref = k if k is not None else v
        if ref is None:
            raise ValueError("nothing to read into")
        n = ref.shape[1] if ref.dim() == 3 else -1
        shape = (self.scenes * self.heads, n, self.d)
        pk = None if k is None else _want("k", k, shape, self._types, self.device)
        pv = None if v is None else _want("v", v, shape, self._types if k is None else (k.dtype,), self.device)
        if n:
            self._call(sa.load().sa_kv_read, sa.SA_BF16 if ref.dtype is self._types[0] else sa.SA_F32, n,
                       self._counts("n_len", n_len), self._counts("start", start), self.lens.data_ptr(),
                       self.page_table.data_ptr(), self.pool.data_ptr(), pk, pv, stream=stream)
            if stream is not None:
                self._hold(stream, k, v, start, n_len)
        return k, v


class CachedGlobalAttention:
    """Attention of up to `rows` query rows per scene over a FrameCache.

    q_heads    query heads (default: the cache's heads; a multiple of them for grouped heads)
    frame      0: every row sees every cached token; n > 0: the rows are the scene's last tokens and see
               their own and earlier frames of n tokens (1: causal by token)

    Workspace and outputs are allocated once: an object's calls (and graphs recorded from it) run one
    after another; calls that overlap need an object each.  For inference: the outputs carry no gradient
    (the stored numbers are rounded)."""

    def __init__(self, cache: FrameCache, rows: int, q_heads: int | None = None, frame: int = 0,
                 softmax_scale: float = 0.0, with_lse: bool = True):
        import torch
        self.cache, self.rows, self.frame = cache, int(rows), int(frame)
        self.q_heads = cache.heads if q_heads is None else int(q_heads)
        self.softmax_scale = float(softmax_scale)
        nbytes = sa.sa_kv_attn_workspace_size(cache.desc, self.q_heads, self.rows)
        if nbytes == 0:
            raise ValueError("q_heads is a multiple of the cache's heads and rows is positive")
        if not 0 <= self.frame < 2 ** 31:
            raise ValueError("frame is 0 or a frame's tokens, below 2^31")
        bh, dev = cache.scenes * self.q_heads, cache.device
        self._q_shape = (bh, self.rows, cache.d)
        self.ws = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
        self.o = torch.zeros((bh, self.rows, cache.d), dtype=torch.bfloat16, device=dev)
        self.lse = torch.zeros((bh, self.rows), dtype=torch.float32, device=dev) if with_lse else None

    def forward(self, q, q_len=None, stream=None):
        """q [scenes * q_heads][rows][64] bf16; with q_len (int32 device tensor [scenes]) only the first q_len[s]
        rows of scene s.  Returns the (O, LSE) buffers; rows past q_len[s] keep what they held."""
        c = self.cache
        pq = _want("q", q, self._q_shape, c._types[:1], c.device)
        c._call(sa.load().sa_kv_attn_fwd, pq, self.q_heads, self.rows, c._counts("q_len", q_len), self.frame,
                self.softmax_scale, c.lens.data_ptr(), c.page_table.data_ptr(), c.pool.data_ptr(), self.ws.data_ptr(),
                self.ws.numel(), self.o.data_ptr(), None if self.lse is None else self.lse.data_ptr(), stream=stream)
        if stream is not None:
            c._hold(stream, q, q_len, self.ws, self.o, self.lse)
        return self.o, self.lse

    __call__ = forward

    def capture(self, q, q_len=None):
        """Record one call on these tensors as a CUDA graph.  A replay follows the cache's lengths and page
        table as they are then (frames appended in between are seen) and new queries written into q.  Keep this
        object, the cache, q and q_len for as long as the graph."""
        import torch
        dev = self.cache.device
        self.forward(q, q_len)
        with torch.cuda.device(dev):
            torch.cuda.current_stream(dev).synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=torch.cuda.Stream(dev)):
                self.forward(q, q_len)
        return g
