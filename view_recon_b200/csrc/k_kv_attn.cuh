// Attention of query rows over the frame cache (k_kv_cache.cuh): O = softmax(scale q K^T) V over the
// cached tokens of each scene, every key or those of a row's own and earlier frames.
//
// Work is a list of (scene, tile of query rows, head) problems, each a run of 128-key tiles; their
// number is known on the device only (lengths are device memory, so that a captured call follows
// them).  The concatenated list of key tiles, each with its cost, is cut into runs of equal cost,
// one per CTA, whatever the lengths; a CTA that holds all tiles of a problem writes its rows,
// otherwise it leaves (O, max, sum) of its part in the workspace and kv_merge_kernel joins the
// parts in a fixed order (no atomics: results do not depend on timing).
#pragma once
#include "k_attn_tc.cuh"
#include "k_kv_cache.cuh"

namespace kv {

struct AttnArgs {
    const uint8_t* pool;
    const int32_t* table;  // [scenes][max_pages]
    const int32_t* lens;   // [scenes]
    const int32_t* q_len;  // [scenes] or null
    const __nv_bfloat16* q;
    __nv_bfloat16* o;
    float* lse;            // or null
    float* part_o;         // [2 * ctas][tile_rows][64]
    float* part_ml;        // [2 * ctas][2][tile_rows]: running max (base 2), sum
    int4* part_rec;        // [ctas][2]: notes of the problems that several CTAs share
    int32_t scenes, kv_heads, group, rows;
    int32_t tile_rows, row_tiles;  // query rows per problem, problems per (scene, head)
    int32_t page_log2, n_pages, max_pages, frame;
    int32_t ctas;             // grid of the attention kernel
    int32_t tile_cost, solo_cost, start_cost;  // of a key tile and of beginning a problem (kv_costs)
    int64_t page_bytes, page_stride;  // of one page of one head, of a page of every head
    float scale_log2;
};

// One scene's share: cached tokens and query rows.
struct Scene {
    int32_t len, n;
};
__device__ __forceinline__ Scene scene_of(const AttnArgs& a, int s) {
    return Scene{scene_len(a.lens, s, a.max_pages, a.page_log2), scene_rows(a.q_len, s, a.rows)};
}
// Keys that query row r of a scene sees: positions below this.  Row r is position len - n + r.
__device__ __forceinline__ int32_t key_limit(const AttnArgs& a, const Scene& sc, int32_t r) {
    if (a.frame == 0) return sc.len;
    const int32_t pos = sc.len - sc.n + r;
    if (pos < 0) return 0;
    return (int32_t)min(((int64_t)(pos / a.frame) + 1) * a.frame, (int64_t)sc.len);
}
// x / y where y is mostly 1: an integer division is a hundred dependent cycles, and the start of every
// block would make a handful of them.
__device__ __forceinline__ int32_t over(int32_t x, int32_t y) { return y == 1 ? x : x / y; }
// A problem's rows are numbered row-major, the query heads of one key head innermost: row x of the
// (scene, key head) is query row x / group of query head x % group.  Limits ascend with x.
__device__ __forceinline__ int32_t valid_rows(const AttnArgs& a, const Scene& sc, int32_t rt) {
    return max(0, min(a.tile_rows, sc.n * a.group - rt * a.tile_rows));
}
__device__ __forceinline__ int32_t key_tiles(const AttnArgs& a, const Scene& sc, int32_t rt) {
    const int32_t nv = valid_rows(a, sc, rt);
    if (nv == 0) return 0;
    if (a.frame == 0) return (sc.len + 127) / 128;
    return (key_limit(a, sc, over(rt * a.tile_rows + nv - 1, a.group)) + 127) / 128;
}
// (rows * group, scenes * row_tiles and the rows of all heads are below 2^31: checked on the host)
__device__ __forceinline__ int64_t out_row(const AttnArgs& a, int s, int h, int32_t x) {
    const int32_t r = over(x, a.group);
    return (int64_t)((s * a.kv_heads + h) * a.group + (x - r * a.group)) * a.rows + r;
}

// Named barrier over `nthreads` threads that tells each of them whether all came with true.
__device__ __forceinline__ bool all_agree(uint32_t id, uint32_t nthreads, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(nthreads), "r"((uint32_t)mine)
        : "memory");
    return r != 0;
}
// A bounded wait whose first tries take no clock: reading the timer and the limit costs more than most
// of these waits last.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    bool ok = false;
#pragma unroll 1
    for (int i = 0; i < 200 && !ok; ++i) ok = mbar_test(bar, parity);
    if (!ok) ok = mbar_wait(bar, parity, abort_flag);
    return __all_sync(0xffffffffu, ok);
}
// Waits until the kernel before this one in the stream, whose end this one was launched ahead of, is
// done and its writes are seen.  Every thread of such a kernel comes through here before it ends, so
// that what follows in the stream follows both.
__device__ __forceinline__ void wait_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The tensor-core kernel takes 256 rows a problem, 128 in each half of a block.  One that has at most
// 128 of them is done by both halves together, every other key tile each ("solo").
constexpr int kPairRows = 256;
__device__ __forceinline__ bool is_solo(const AttnArgs& a, int32_t nv) { return a.tile_rows == kPairRows && nv <= 128; }
__device__ __forceinline__ int32_t tile_cost(const AttnArgs& a, int32_t nv) {
    return is_solo(a, nv) ? a.solo_cost : a.tile_cost;
}

// The list of problems, entry e = (scene e / row_tiles, row tile e % row_tiles), heads within.
struct Cut {
    int64_t per;    // cost of one CTA's run
    int32_t start;  // of beginning a problem: its first tile costs this much more
};
__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
// Cost of an entry's key tiles; `empty`: it has rows, but no key for any of them.
__device__ __forceinline__ int64_t entry_cost(const AttnArgs& a, int32_t e, bool* empty) {
    const int s = over(e, a.row_tiles), rt = e - s * a.row_tiles;
    const Scene sc = scene_of(a, s);
    const int32_t nv = valid_rows(a, sc, rt), tiles = key_tiles(a, sc, rt);
    *empty = nv > 0 && tiles == 0;
    return (int64_t)tiles * tile_cost(a, nv) * a.kv_heads;
}
__device__ __forceinline__ int64_t warp_scan(int64_t c) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, c, d);
        if (lane >= d) c += y;
    }
    return c;
}
// Small dividends take the short division.
__device__ __forceinline__ int64_t quotient(int64_t x, int64_t y) {
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
// Rows of the problems that have no keys at all: O = 0, LSE = -inf.  Every thread of every block.
__device__ __forceinline__ void write_empty_rows(const AttnArgs& a) {
    const int32_t n = a.scenes * a.row_tiles;
    for (int32_t e = blockIdx.x; e < n; e += a.ctas) {
        const int s = over(e, a.row_tiles), rt = e - s * a.row_tiles;
        const Scene sc = scene_of(a, s);
        const int32_t nv = valid_rows(a, sc, rt);
        if (nv == 0 || key_tiles(a, sc, rt) > 0) continue;
        const int64_t pieces = (int64_t)nv * a.kv_heads * 8;  // of 16 bytes (rows are below 2^31, these are not)
        for (int64_t i = threadIdx.x; i < pieces; i += blockDim.x) {
            const int32_t y = (int32_t)(i / 8), h = y / nv, x = y - h * nv;
            const int64_t row = out_row(a, s, h, rt * a.tile_rows + x);
            reinterpret_cast<uint4*>(a.o + row * 64)[i % 8] = make_uint4(0, 0, 0, 0);
            if (a.lse && i % 8 == 0) a.lse[row] = -INFINITY;
        }
    }
}

// The CTA's run: the cut of the list, and the entry in which the run begins and the place within it
// (entry < 0: nothing to do).
struct Start {
    Cut cut;
    int64_t left, within;
    int32_t entry, any_empty;  // any_empty: rows without keys have to be written
};
// Up to 32 entries are one scan in the registers of the warp that calls this; for more every thread of the
// block calls it, and `red` is shared memory of two int64 per warp.
__device__ __forceinline__ Start find_start(const AttnArgs& a, int64_t* red) {
    const int lane = threadIdx.x & 31;
    const int32_t n = a.scenes * a.row_tiles;
    Start s;
    int64_t scan = 0, cost = 0, total = 0;
    int32_t busy = 0;  // entries with key tiles
    if (n <= 32) {
        bool empty = false;
        cost = lane < n ? entry_cost(a, lane, &empty) : 0;
        scan = warp_scan(cost);
        total = __shfl_sync(0xffffffffu, scan, 31);
        busy = __popc(__ballot_sync(0xffffffffu, cost > 0));
        s.any_empty = __any_sync(0xffffffffu, empty);
    } else {
        int64_t sum = 0;
        bool empty;
        for (int32_t e = threadIdx.x; e < n; e += blockDim.x) {
            cost = entry_cost(a, e, &empty);
            sum += cost;
            busy += cost > 0;
        }
        s.any_empty = 1;
        sum = warp_sum(sum);
        busy = __reduce_add_sync(0xffffffffu, busy);
        const int warps = blockDim.x >> 5;
        if (lane == 0) red[threadIdx.x >> 5] = sum, red[warps + (threadIdx.x >> 5)] = busy;
        __syncthreads();
        busy = 0;
        for (int w = 0; w < warps; ++w) total += red[w], busy += (int32_t)red[warps + w];
    }
    // Where runs are longer than a problem's first tile, its beginning counts; shorter runs are best cut
    // as finely as the tiles are.  Either way a run is as long as any tile, and so, within a problem, holds
    // a tile's beginning.
    const int64_t least = a.tile_cost + a.start_cost;
    s.cut.start = total >= a.ctas * least ? a.start_cost : 0;
    const int64_t extra = (int64_t)s.cut.start * a.kv_heads;  // of an entry that is busy
    total += busy * extra;
    s.cut.per = max(quotient(total + a.ctas - 1, a.ctas), (int64_t)a.tile_cost);
    const int64_t x = blockIdx.x * s.cut.per;
    s.left = min(s.cut.per, total - x);
    s.entry = -1;
    s.within = 0;
    if (s.left <= 0) return s;
    int64_t before = 0;
    for (int32_t e0 = 0; e0 < n; e0 += 32) {
        bool empty;
        if (n > 32) cost = e0 + lane < n ? entry_cost(a, e0 + lane, &empty) : 0;
        if (n > 32 || extra != 0) scan = warp_scan(cost + (cost > 0 ? extra : 0));
        const uint32_t past = __ballot_sync(0xffffffffu, before + scan > x);
        if (past) {
            const int first = __ffs(past) - 1;
            const int64_t prev = __shfl_sync(0xffffffffu, scan, max(first - 1, 0));
            s.within = x - before - (first > 0 ? prev : 0);
            s.entry = e0 + first;
            break;
        }
        before += __shfl_sync(0xffffffffu, scan, 31);
    }
    return s;
}

// The whole block's start.  One warp's work reaches the others through shared memory, so that nothing of
// it stays in the registers of the loops to come (inlined into each of them, the same code cost the
// tensor-core kernel 5 % of every tile).
__device__ __forceinline__ Start block_start(const AttnArgs& a, Start* box, int64_t* red) {
    if (a.scenes * a.row_tiles > 32 || threadIdx.x / 32 == 2) {  // (warps 0 and 1 have the barriers and tensor memory)
        const Start s = find_start(a, red);
        if (threadIdx.x == 64) *box = s;
    }
    __syncthreads();
    Start s;
    const uint32_t at = smem_u32(box);
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(s.cut.per) : "r"(at + (uint32_t)offsetof(Start, cut.per)) : "memory");
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(s.cut.start) : "r"(at + (uint32_t)offsetof(Start, cut.start)) : "memory");
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(s.left) : "r"(at + (uint32_t)offsetof(Start, left)) : "memory");
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(s.within) : "r"(at + (uint32_t)offsetof(Start, within)) : "memory");
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(s.entry) : "r"(at + (uint32_t)offsetof(Start, entry)) : "memory");
    if (box->any_empty) write_empty_rows(a);
    return s;
}

// One problem's share of a CTA's run of key tiles.
struct Segment {
    int32_t s, rt, h;
    int32_t t0, t1, tiles;  // key tiles [t0, t1) of the problem's `tiles`
    int32_t nv;             // its rows
    int32_t last;           // the CTA that has its last tile, when this one has its first and not all
    Scene sc;
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
    // Workspace slot of a part: a CTA leaves at most two, one of a problem that began before its run
    // and one of a problem that goes on after it.
    __device__ __forceinline__ int slot() const { return 2 * (int)blockIdx.x + (t0 > 0 ? 0 : 1); }
};
// Walks the CTA's run; every role of the CTA makes the same walk.  A tile belongs to the run in which
// its place in the list (cost by cost) begins.
// Tiles of a problem that begin before place u: the first at 0, tile t at start + t * cost.
__device__ __forceinline__ int32_t tiles_before(int64_t u, int32_t start, int32_t cost) {
    const int64_t x = max(u - start, (int64_t)0);
    return u <= 0 ? 0 : (int32_t)max(cost == 1 ? x : quotient(x + cost - 1, cost), (int64_t)1);
}
struct Walk {
    int64_t left, u;  // cost still to come, place within the problem at hand
    int32_t e, h;
    __device__ __forceinline__ Walk(const AttnArgs& a, const Start& s) : left(s.left), u(0), e(s.entry), h(0) {
        if (e < 0) return;
        const int sc = over(e, a.row_tiles), rt = e - sc * a.row_tiles;
        const Scene scene = scene_of(a, sc);
        const int64_t one =
            s.cut.start + (int64_t)key_tiles(a, scene, rt) * tile_cost(a, valid_rows(a, scene, rt));
        h = s.within < one ? 0 : (int32_t)quotient(s.within, one);
        u = s.within - h * one;
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, const Cut& cut, Segment* g) {
        const int32_t n = a.scenes * a.row_tiles;
        while (left > 0 && e < n) {
            g->s = over(e, a.row_tiles);
            g->rt = e - g->s * a.row_tiles;
            g->sc = scene_of(a, g->s);
            g->nv = valid_rows(a, g->sc, g->rt);
            g->tiles = key_tiles(a, g->sc, g->rt);
            if (g->tiles == 0 || h >= a.kv_heads) {
                ++e;
                h = 0;
                u = 0;
                continue;
            }
            const int32_t cost = tile_cost(a, g->nv);
            const int64_t u1 = min(cut.start + (int64_t)g->tiles * cost, u + left);
            g->h = h;
            g->t0 = tiles_before(u, cut.start, cost);
            g->t1 = tiles_before(u1, cut.start, cost);
            // the problem's first tile is at this CTA's end - left, and its last one begins so much behind the end
            const int64_t behind = (g->tiles > 1 ? cut.start + (int64_t)(g->tiles - 1) * cost : 0) - left;
            g->last = u == 0 && behind >= 0 ? (int32_t)(blockIdx.x + 1 + quotient(behind, cut.per)) : -1;
            left -= u1 - u;
            u = 0;
            ++h;
            if (g->t0 < g->t1) return true;
        }
        return false;
    }
};

// Leaves the merge kernel notes of the problems that begin in this CTA's run and go on after it.  With
// no more problems than CTAs a note belongs to a problem, which leaves the merge few blocks, and says
// "none" for a problem that needs no merge; otherwise it belongs to a CTA, which has one at most.  One
// thread writes them all before anything can fail: whatever a wait that runs out leaves undone, the
// merge kernel reads notes of this launch.
__device__ __forceinline__ bool notes_by_problem(const AttnArgs& a) {
    return (int64_t)a.scenes * a.row_tiles * a.kv_heads <= a.ctas;
}
__device__ __forceinline__ void note_parts(const AttnArgs& a, const Cut& cut, Walk walk) {
    const bool by_problem = notes_by_problem(a);
    bool none = !by_problem;
    if (by_problem && (int)blockIdx.x < a.scenes * a.row_tiles * a.kv_heads) {
        const int32_t e = over(blockIdx.x, a.kv_heads), s = over(e, a.row_tiles);
        none = key_tiles(a, scene_of(a, s), e - s * a.row_tiles) == 0;
    }
    if (none) a.part_rec[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
    Segment g;
    while (walk.next(a, cut, &g)) {
        if (!(by_problem ? g.t0 == 0 : g.last >= 0)) continue;
        int4* rec = a.part_rec + 2 * (by_problem ? (g.s * a.row_tiles + g.rt) * a.kv_heads + g.h : (int)blockIdx.x);
        rec[1] = make_int4(g.h, g.nv, blockIdx.x, 0);
        rec[0] = make_int4(g.last, g.s, g.rt, 0);
    }
}

// ------------------------------------------------------------------------------ few rows
//
// Up to 32 query rows a problem (33 to 48 in two of 24, each decoding every key): every page is read and decoded for few products, so the
// rows ride on the narrow side of mma.sync (m16n8k16, keys on m, rows on n): S^T = K Q^T with 16 keys x
// 8 rows, O^T += V^T P^T with 16 channels x 8 rows (tcgen05 would take 128 rows, mostly padding, and
// operands through shared memory).  A lane's decoded words are its operand registers as they stand (the
// page layout is made for it): no shuffle and no shared-memory round trip between a page's bytes and
// the tensor cores; P^T is transposed by one movmatrix per 8 x 8.
// Four warps take 32 keys each of every 128-key tile; a fifth keeps a ring of tiles in flight with
// bulk copies of whole pages (K, V and scales of a page and head are one run of bytes).
// Measured in a recorded graph, 16 heads over 351 744 tokens: in 4 bits 5 rows 100 us, 4.05 TB/s, 12 rows 131,
// 24 rows 178, 32 rows 226 us; in 8 bits 5 rows 124 us, 6.2 TB/s, 12 rows 147 us, 5.2 TB/s, 32 rows 244 us.
// 4 bits are bound by the decoding's instructions (65 % of the issue slots, the ALU pipe 57 %; 1483 warp
// instructions a tile; the same ring with nothing done to the tiles takes 73 us, everything but the decoding
// 76 us) and, with 20 warps an SM, by what latency the other third of the slots waits for.
// Blocks an SM, by groups of 8 rows: 4, 3, 2, 2.  One group with 5 blocks and 3 stages: 111 us against 104;
// two groups with 4: 174 against 133; four groups with 3: 324 against 241.  Registers a thread 96, 128, 168,
// 168: one and two groups do not spill.  Two blocks of five warps put three warps on one quarter of an SM,
// which leaves each 168, and there three groups spill 20 bytes (8 in 8 bits) and four groups 228 (loaded again:
// 364, 360).  What one block an SM, with registers enough, would take has not been measured.

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int BITS, int NT>  // NT: groups of 8 query rows
struct FewLayout {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kRows = 8 * NT;
    static constexpr int kStageBytes = 128 * Fmt<BITS>::kTokenBytes;
    static constexpr int kStages = BITS == 4 ? 4 : 3;
    static constexpr int kRing = 0;
    static constexpr int kMergeO = kRing + kStages * kStageBytes;       // [warp][row][64 + 4] f32
    static constexpr int kMergeRow = 68;
    static constexpr int kMergeMl = kMergeO + kWarps * kRows * kMergeRow * 4;  // [warp][2][row]
    static constexpr int kBars = kMergeMl + kWarps * 2 * kRows * 4;     // full[], empty[]
    static constexpr int kMeta = kBars + 16 * kStages;                  // per stage: bad sub-pages
    static constexpr int kMisc = kMeta + 4 * kStages + (kStages & 1 ? 4 : 0);  // abort flag, reduction[10]
    static constexpr int kStart = kMisc + 96;
    static constexpr int kEnd = kStart + sizeof(Start);
    static constexpr int smem_bytes() { return kEnd; }
    static_assert(kStageBytes % 16 == 0 && kMergeO % 16 == 0 && kBars % 8 == 0 && kMisc % 8 == 0 && kStart % 8 == 0, "alignment");
};

template <int BITS, int NT>
__global__ void __launch_bounds__(160, NT == 1 ? 4 : (NT == 2 ? 3 : 2)) kv_few_rows_kernel(const AttnArgs a) {
    using L = FewLayout<BITS, NT>;
    using F = Fmt<BITS>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* empty = full + L::kStages;
    volatile uint32_t* meta = reinterpret_cast<volatile uint32_t*>(smem + L::kMeta);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
    int64_t* red = reinterpret_cast<int64_t*>(smem + L::kMisc + 8);  // two per warp
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], L::kWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    const Start start = block_start(a, reinterpret_cast<Start*>(smem + L::kStart), red);
    const Cut cut = start.cut;
    Walk walk(a, start);

    const int page = 1 << a.page_log2, sub_pages = 128 >> a.page_log2;
    Segment g;
    int it = 0;  // tiles so far: ring stage it % kStages
    if (warp == L::kWarps) {
        // ---------------------------------------------------------------- loads
        bool ok = !(g_sa_test_withhold != 0 && blockIdx.x == 0);
        while (ok && walk.next(a, cut, &g)) {
            const int32_t* row = a.table + (int64_t)g.s * a.max_pages;
            const int32_t lim = (int32_t)min((int64_t)g.tiles * 128, (int64_t)g.sc.len);
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int st = it % L::kStages;
                const int key = t * 128 + lane * page;
                const bool mine = lane < sub_pages && key < lim;
                const int32_t pid = mine ? __ldg(row + (key >> a.page_log2)) : 0;
                const bool good = mine && pid >= 0 && pid < a.n_pages;
                const uint32_t bad = __ballot_sync(0xffffffffu, mine && !good);
                const int n = __popc(__ballot_sync(0xffffffffu, good));
                if (!wait_warp(&empty[st], ((it / L::kStages) & 1) ^ 1, abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (bad) sa_flag_error(SA_ERR_BAD_LIST);
                    meta[st] = bad;
                    mbar_arrive_expect_tx(&full[st], (uint32_t)(n * a.page_bytes));
                }
                __syncwarp();
                if (good)
                    bulk_load(smem + L::kRing + st * L::kStageBytes + lane * a.page_bytes,
                              a.pool + ((int64_t)pid * a.kv_heads + g.h) * a.page_bytes, (uint32_t)a.page_bytes,
                              &full[st]);
            }
        }
        // every copy has landed before the CTA exits
        for (int i = max(0, it - L::kStages); i < it; ++i) tc::drain_wait(&full[i % L::kStages], (i / L::kStages) & 1);
    } else {
        // ---------------------------------------------------------------- products
        const int qg = lane >> 2, qc = lane & 3;
        if (threadIdx.x == 0) note_parts(a, cut, walk);  // while the first tile is on its way
        __syncwarp();
        // where this lane's codes and scales of its 32 keys are within a stage, 16 keys at a time (a page
        // holds 16 keys at least)
        int k_at[2], ks_at[2], v_at[2], vs_at[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kk = 32 * warp + 16 * u, slot = kk & (page - 1);
            const int base = L::kRing + (kk >> a.page_log2) * (int)a.page_bytes;
            k_at[u] = base + (slot + qg) * F::kDB + qc * (F::kDB / 4);
            ks_at[u] = base + page * F::kDB + (slot + qg) * 4 + qc;
            v_at[u] = base + page * (F::kDB + 4) + (slot / 2 + qc) * (2 * F::kDB) + qg * (F::kDB / 4);
            vs_at[u] = base + page * (2 * F::kDB + 4) + (slot / 2 + qc) * 8 + (qg & ~1);
        }
        bool ok = true;
        while (ok && walk.next(a, cut, &g)) {
            const int32_t nv = g.nv;
            const int32_t r0 = g.rt * a.tile_rows;
            // Q^T operand: row 8 i + qg, channels 16 qc .. 16 qc + 15
            uint32_t qb[NT][8];
            int32_t lim[NT][2];  // key limits of this lane's columns, rows 8 i + 2 qc and the next
            int32_t least = 0x7FFFFFFF;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (8 * i + qg < nv) {
                    const uint4* src =
                        reinterpret_cast<const uint4*>(a.q + out_row(a, g.s, g.h, r0 + 8 * i + qg) * 64 + 16 * qc);
                    u[0] = __ldg(src);
                    u[1] = __ldg(src + 1);
                }
                const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
                for (int j = 0; j < 8; ++j) qb[i][j] = w[j];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int32_t x = 8 * i + 2 * qc + j;
                    lim[i][j] = x < nv ? key_limit(a, g.sc, over(r0 + x, a.group)) : 0x7FFFFFFF;
                    least = min(least, lim[i][j]);
                }
            }
            least = min(least, g.sc.len);
            least = __reduce_min_sync(0xffffffffu, least);
            float o[NT][4][4], m[NT][2];
            float2 l[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][j][c] = 0.0f;
                m[i][0] = m[i][1] = -INFINITY;
                l[i] = make_float2(0.0f, 0.0f);
            }
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                const int st = it % L::kStages;
                if (!wait_warp(&full[st], (it / L::kStages) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint8_t* ring = smem + st * L::kStageBytes;
                const int key0 = t * 128 + 32 * warp;  // this warp's keys of the tile
                if (key0 < g.sc.len) {
                    float sc[NT][2][4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t ka[2][8];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t w[F::kWords];
                            const uint2* src = reinterpret_cast<const uint2*>(ring + k_at[u] + 8 * e * F::kDB);
#pragma unroll
                            for (int i = 0; i < F::kWords; i += 2) {
                                const uint2 v = src[i / 2];
                                w[i] = v.x;
                                w[i + 1] = v.y;
                            }
                            const uint32_t s2 = scale_both(ring[ks_at[u] + 32 * e]);
                            decode<BITS>(w, s2, offset_pair<BITS>(s2), ka[e]);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) sc[i][u][c] = 0.0f;
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_16816(sc[i][u], ka[0][2 * ks], ka[1][2 * ks], ka[0][2 * ks + 1], ka[1][2 * ks + 1],
                                          qb[i][2 * ks], qb[i][2 * ks + 1]);
                        }
                    }
                    const uint32_t bad = meta[st];
                    if (key0 + 32 > least || bad) {
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int kk = 32 * warp + 16 * u + 8 * e + qg, key = t * 128 + kk;
                                const bool gone = (bad >> (kk >> a.page_log2)) & 1;
#pragma unroll
                                for (int i = 0; i < NT; ++i)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        if (gone || key >= min(lim[i][c], g.sc.len)) sc[i][u][2 * e + c] = -INFINITY;
                            }
                    }
                    // running maximum, raised only when a score is over it by more than 2^8
                    float mx[NT][2];
                    bool up = false;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            mx[i][c] = a.scale_log2 * fmaxf(fmaxf(sc[i][0][c], sc[i][0][2 + c]),
                                                            fmaxf(sc[i][1][c], sc[i][1][2 + c]));
                            up |= mx[i][c] > m[i][c] + 8.0f;
                        }
                    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
#pragma unroll
                                for (int d = 4; d < 32; d <<= 1)
                                    mx[i][c] = fmaxf(mx[i][c], __shfl_xor_sync(0xffffffffu, mx[i][c], d));
                                const float mn = fmaxf(m[i][c], mx[i][c]);
                                const float alpha = mn == -INFINITY ? 1.0f : ex2_approx(m[i][c] - mn);
                                m[i][c] = mn;
                                if (c == 0) l[i].x *= alpha;
                                else l[i].y *= alpha;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    o[i][j][c] *= alpha;
                                    o[i][j][2 + c] *= alpha;
                                }
                            }
                    }
                    uint32_t pb[NT][2][2];
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float2 neg = make_float2(m[i][0] == -INFINITY ? 0.0f : -m[i][0],
                                                       m[i][1] == -INFINITY ? 0.0f : -m[i][1]);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 x = __ffma2_rn(make_float2(sc[i][u][2 * e], sc[i][u][2 * e + 1]),
                                                            make_float2(a.scale_log2, a.scale_log2), neg);
                                const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                                l[i] = __fadd2_rn(l[i], p);
                                // P enters its product rounded to bf16, as in the other attention
                                // kernels; the sum takes it unrounded
                                pb[i][u][e] = transpose_8x8(pack_bf16x2(p.x, p.y));
                            }
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t va[2][8];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t w[F::kWords];
                            const uint2* src = reinterpret_cast<const uint2*>(ring + v_at[u] + 8 * e * F::kDB);
#pragma unroll
                            for (int i = 0; i < F::kWords; i += 2) {
                                const uint2 v = src[i / 2];
                                w[i] = v.x;
                                w[i + 1] = v.y;
                            }
                            const uint32_t s2 =
                                scale_halves(*reinterpret_cast<const uint16_t*>(ring + vs_at[u] + 32 * e));
                            decode<BITS>(w, s2, offset_pair<BITS>(s2), va[e]);
                        }
#pragma unroll
                        for (int i = 0; i < NT; ++i)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_16816(o[i][j], va[0][2 * j], va[0][2 * j + 1], va[1][2 * j], va[1][2 * j + 1],
                                          pb[i][u][0], pb[i][u][1]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            // ---- join the four warps' parts
            float* mo = reinterpret_cast<float*>(smem + L::kMergeO) + warp * L::kRows * L::kMergeRow;
            float* ml = reinterpret_cast<float*>(smem + L::kMergeMl) + warp * 2 * L::kRows;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float sum = c == 0 ? l[i].x : l[i].y;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                    const int x = 8 * i + 2 * qc + c;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<float2*>(mo + x * L::kMergeRow + 8 * qg + 2 * j) =
                            make_float2(o[i][j][c], o[i][j][2 + c]);
                    if (qg == 0) {
                        ml[x] = m[i][c];
                        ml[L::kRows + x] = sum;
                    }
                }
            ok = all_agree(1, 32 * L::kWarps, ok);  // a wait that ran out ends all four warps here
            const bool whole = g.whole();
            const float* all_ml = reinterpret_cast<const float*>(smem + L::kMergeMl);
            const float* all_o = reinterpret_cast<const float*>(smem + L::kMergeO);
            const int slot = g.slot();
            if (ok)
                for (int x = threadIdx.x / 16; x < nv; x += 8) {
                    const int c4 = threadIdx.x % 16;
                    float mm = -INFINITY;
#pragma unroll
                    for (int w = 0; w < L::kWarps; ++w) mm = fmaxf(mm, all_ml[w * 2 * L::kRows + x]);
                    const float mu = mm == -INFINITY ? 0.0f : mm;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < L::kWarps; ++w) {
                        const float f = ex2_approx(all_ml[w * 2 * L::kRows + x] - mu);
                        const float4 v =
                            *reinterpret_cast<const float4*>(all_o + (w * L::kRows + x) * L::kMergeRow + 4 * c4);
                        acc.x += f * v.x;
                        acc.y += f * v.y;
                        acc.z += f * v.z;
                        acc.w += f * v.w;
                        sum += f * all_ml[w * 2 * L::kRows + L::kRows + x];
                    }
                    if (whole) {
                        const int64_t row = out_row(a, g.s, g.h, r0 + x);
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                        *reinterpret_cast<uint2*>(a.o + row * 64 + 4 * c4) =
                            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                        if (a.lse && c4 == 0)
                            a.lse[row] = sum == 0.0f ? -INFINITY : (mu + log2f(sum)) * 0.69314718055994530942f;
                    } else {
                        *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * a.tile_rows + x) * 64 + 4 * c4) = acc;
                        if (c4 == 0) {
                            a.part_ml[(int64_t)slot * 2 * a.tile_rows + x] = mm;
                            a.part_ml[((int64_t)slot * 2 + 1) * a.tile_rows + x] = sum;
                        }
                    }
                }
            __syncwarp();  // (the halves of a warp took different rows)
            named_bar_sync(1, 32 * L::kWarps);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------------------ joining the parts
//
// One block per note and 32 rows (or the whole tile of rows): a problem that begins in one CTA's run and
// ends in another's.  O = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over its parts i.  A thread sums
// four channels of a row over the parts, in order; for short tiles of rows groups of threads take every
// second or fourth part, and the groups are summed in order.  A chain of a few loads, not bandwidth, is
// its time: launched early, with six parts in flight and no block for a problem without parts, a call of
// 1 row over 2 748 tokens and 16 heads came down from 12.4 to 9.8 us in a recorded graph.
constexpr int kMergeThreads = 512;

__global__ void __launch_bounds__(kMergeThreads, 2) kv_merge_kernel(const AttnArgs a) {
    __shared__ float4 acc_smem[32][16];
    __shared__ float ml_smem[2][32];
    wait_previous_kernel();
    const int4 r0 = __ldcg(a.part_rec + 2 * blockIdx.x), r1 = __ldcg(a.part_rec + 2 * blockIdx.x + 1);
    const int32_t c0 = r1.z, c1 = min(r0.x, a.ctas - 1);
    if (c1 < 0) return;
    const int32_t nv = r1.y, rows = min(a.tile_rows, 32), groups = 32 / rows;
    const int y = threadIdx.x / 16, c4 = threadIdx.x % 16, grp = y / rows;
    if (grp >= groups) return;  // 24 rows leave a quarter of the threads over
    for (int x = rows * blockIdx.y + y % rows; x - y % rows < nv; x += rows * gridDim.y) {
        float m = -INFINITY, l = 0.0f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < nv) {
            constexpr int kBatch = 6;  // parts whose loads are in flight together: the kernel is all latency
            for (int c = c0 + grp; c <= c1; c += groups * kBatch) {
                float pm[kBatch], pl[kBatch];
                float4 v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int ci = c + i * groups;
                    pm[i] = -INFINITY;
                    pl[i] = 0.0f;
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (ci > c1) continue;
                    const int64_t slot = 2 * (int64_t)ci + (ci == c0 ? 1 : 0);
                    pm[i] = __ldcg(a.part_ml + slot * 2 * a.tile_rows + x);
                    pl[i] = __ldcg(a.part_ml + (slot * 2 + 1) * a.tile_rows + x);
                    v[i] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (slot * a.tile_rows + x) * 64 + 4 * c4));
                }
                float mn = m;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) mn = fmaxf(mn, pm[i]);
                const float mu = mn == -INFINITY ? 0.0f : mn, f = ex2_approx(m - mu);
                acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
                l *= f;
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const float w = ex2_approx(pm[i] - mu);
                    acc.x += v[i].x * w;
                    acc.y += v[i].y * w;
                    acc.z += v[i].z * w;
                    acc.w += v[i].w * w;
                    l += pl[i] * w;
                }
                m = mn;
            }
        }
        if (groups > 1) {
            acc_smem[y][c4] = acc;
            if (c4 == 0) ml_smem[0][y] = m, ml_smem[1][y] = l;
            __syncthreads();
            if (grp != 0) return;  // (shorter tiles are one round)
            for (int i = 1; i < groups; ++i) m = fmaxf(m, ml_smem[0][i * rows + y]);
            const float mu = m == -INFINITY ? 0.0f : m;
            acc = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.0f;
            for (int i = 0; i < groups; ++i) {
                const float w = ex2_approx(ml_smem[0][i * rows + y] - mu);
                const float4 v = acc_smem[i * rows + y][c4];
                acc.x += v.x * w;
                acc.y += v.y * w;
                acc.z += v.z * w;
                acc.w += v.w * w;
                l += ml_smem[1][i * rows + y] * w;
            }
        }
        if (x >= nv) continue;
        const float mu = m == -INFINITY ? 0.0f : m;
        const int64_t row = out_row(a, r0.y, r1.x, r0.z * a.tile_rows + x);
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(a.o + row * 64 + 4 * c4) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (a.lse && c4 == 0) a.lse[row] = l == 0.0f ? -INFINITY : (mu + log2f(l)) * 0.69314718055994530942f;
    }
}

}  // namespace kv
