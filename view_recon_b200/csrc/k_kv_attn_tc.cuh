// Attention over the frame cache for more than 48 query rows a problem (whole frames): the
// products on the 5th-generation tensor cores, 128 keys a step, scores and O in tensor memory.
// One block per SM, two halves: each takes 128 of a problem's 256 query rows through the same decoded
// keys, so that a page is decoded once for both and one half's exponentials fill the other's waits.  A
// problem of at most 128 rows is done "solo": both halves hold the same rows, take every other tile
// and join their results through shared memory.
// Roles (512 threads):
//   warps 0, 1   tensor-core issue of half 0, 1: S = Q K^T of the next tile before O += P V of this one
//   warps 4-7    decode: a thread takes one key's K (4 blocks of 16 channels) and one 8 channel x 8 key
//                patch of V straight from the pages into registers, a tile ahead, and writes bf16
//                operands: K [128 keys][64], V^T [64][128 keys], both K-major with the 128-byte
//                swizzle (eight lanes write the eight 16-byte chunks of a row: no bank conflicts)
//   warps 8-15   softmax of half 0, 1: thread r owns row r.  The running maximum is raised (and O
//                rescaled) only when a score is over it by more than 2^8; P goes to tensor memory as bf16
// TMEM (512 columns), per half: S 128 (f32), P 64 (bf16 pairs), O 64 (f32).
// Measured, 16 heads: 1 374 rows over 87 936 tokens in 4 bits 831 us, 596 TFLOP/s (4 * 64 FLOP a row
// and key).  No one unit is full: exponentials 59 % of the XU pipe, tensor pipe 30 %, issue 51 %, DRAM 5 %; each
// half's chain (scores, maximum, exponentials, P, product) waits on its own hand-offs, and the other half
// fills only part of them.  Without any exponential 250 us of 382 (1 280 rows over 43 968 tokens).
// The sparse layer's kernel does 396 kFLOP a cycle where this one does 349: part of the difference is the last
// row tile of a frame, 94 rows of 1 374 that cost 6/8 of a tile of 256.
// Problems of at most 128 rows: 49, 64, 96 and 128 rows over 175 872 tokens all take 220 us in 4 bits and 264 us
// in 8 bits (48 rows in the few-rows kernel: 177 and 189 us).  The time is the decoding's, not the rows': one
// warpgroup reads pages from global memory a tile ahead, and padded rows take part in softmax and products.
// The split leaves 100 bytes of spills a thread (272 loaded again).
// Other shapes of the same work were slower: 2 blocks an SM of 128 rows with a decode of their own 1039 us,
// three slots with 64-key steps 1131, two threads a row 976, the halves taking turns at the exponentials
// 1004, exponentials of 1 to 4 of 8 pairs on the FMA pipe +8 to +15 %.
#pragma once
#include "k_kv_attn.cuh"

namespace kv {

struct TcLayoutKv {
    static constexpr int kThreads = 512;
    // registers per thread after the split (launched with 128 each; the sum is the launch's own): the softmax
    // holds 128 scores and 32 pairs of P at once; 8 registers either way are within 1 %
    static constexpr uint32_t kRegsIssue = 40, kRegsDecode = 88, kRegsSoftmax = 192;
    static constexpr uint32_t kRegsNeeded = 128 * (kRegsIssue + kRegsDecode + 2 * kRegsSoftmax);
    static constexpr int kStages = 4;
    static constexpr int kTile = 128 * 128;  // bytes of a 128 x 64 bf16 operand
    static constexpr int kQ = 0;                            // [half]
    static constexpr int kKV = kQ + 2 * kTile;              // [stage] K, V^T
    static constexpr int kBars = kKV + 2 * kStages * kTile;
    // kv_full[stage], kv_empty[stage]; per half: q_full, s_full, s_free, p_full, pv_done, drain,
    // q_seen; solo: x_full, x_empty
    static constexpr int kNumBars = 2 * kStages + 2 * 7 + 2;
    static constexpr int kBad = kBars + 8 * kNumBars;      // [stage][8 sub-pages] bytes
    static constexpr int kSeg = kBad + 8 * kStages;        // per half: tiles of the problem at hand, solo flag
    static constexpr int kMisc = kSeg + 16;                // abort flag, tmem base, reduction[32]
    static constexpr int kJoin = kMisc + 8 + 256;     // solo: half 1's O [64][128 rows], max, sum (f32)
    static constexpr int kStart = kJoin + 66 * 128 * 4;
    static constexpr int kEnd = kStart + sizeof(Start);
    static constexpr uint32_t kTmemCols = 512;
    static constexpr uint32_t colS(int x) { return 256 * x; }
    static constexpr uint32_t colP(int x) { return 256 * x + 128; }
    static constexpr uint32_t colO(int x) { return 256 * x + 192; }
    static constexpr int smem_bytes() { return 1024 + kEnd; }
    static_assert(kBars % 8 == 0 && kMisc % 8 == 0 && kStart % 8 == 0, "alignment");
};

// Where the pages of a problem are: its row of the page table, its head's page 0, and the tokens that
// any of its rows sees.
struct PageRun {
    const int32_t* row;
    const uint8_t* head;
    int32_t lim;
    __device__ __forceinline__ PageRun(const AttnArgs& a, const Segment& g) {
        row = a.table + (int64_t)g.s * a.max_pages;
        head = a.pool + g.h * a.page_bytes;
        lim = (int32_t)min((int64_t)g.tiles * 128, (int64_t)g.sc.len);
    }
    // The table's entry for token `key` (-1 past the limit); nothing here waits for it.
    __device__ __forceinline__ int32_t entry(const AttnArgs& a, int32_t key) const {
        return key < lim ? __ldg(row + (key >> a.page_log2)) : -1;
    }
};
// The page that an entry names, of the problem's head, or null.
__device__ __forceinline__ const uint8_t* page_at(const AttnArgs& a, const uint8_t* head, int32_t entry) {
    return (uint32_t)entry < (uint32_t)a.n_pages ? head + (int64_t)entry * a.page_stride : nullptr;
}

__device__ __forceinline__ uint2 ld_shared_v2(const void* p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)) : "memory");
    return v;
}

template <int BITS>
struct KeyRegs {  // one key's K
    uint32_t w[4][Fmt<BITS>::kWords], scales;
    __device__ __forceinline__ void load(const AttnArgs& a, const uint8_t* base, int tid) {
        using F = Fmt<BITS>;
        const int page = 1 << a.page_log2, slot = tid & (page - 1);
        if (!base) {
            scales = 0;
#pragma unroll
            for (int i = 0; i < 4 * F::kWords; ++i) w[i / F::kWords][i % F::kWords] = 0;
            return;
        }
        const uint4* src = reinterpret_cast<const uint4*>(base + slot * F::kDB);
#pragma unroll
        for (int i = 0; i < F::kWords; ++i) {
            const uint4 q = __ldg(src + i);
            w[(4 * i) / F::kWords][(4 * i) % F::kWords] = q.x;
            w[(4 * i + 1) / F::kWords][(4 * i + 1) % F::kWords] = q.y;
            w[(4 * i + 2) / F::kWords][(4 * i + 2) % F::kWords] = q.z;
            w[(4 * i + 3) / F::kWords][(4 * i + 3) % F::kWords] = q.w;
        }
        scales = __ldg(reinterpret_cast<const uint32_t*>(base + page * F::kDB + slot * 4));
    }
    __device__ __forceinline__ void store(uint8_t* tile, int tid) const {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t out[8];
            const uint32_t s2 = scale_both((scales >> (8 * c)) & 0xFFu);
            decode<BITS>(w[c], s2, offset_pair<BITS>(s2), out);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<uint4*>(tile + tid * 128 + (((2 * c + j) ^ (tid & 7)) << 4)) =
                    make_uint4(out[4 * j], out[4 * j + 1], out[4 * j + 2], out[4 * j + 3]);
        }
    }
};

template <int BITS>
struct ValueRegs {  // channels 8 ch8 .. + 7 of keys 8 oct .. + 7
    uint32_t w[4][Fmt<BITS>::kWords], scales[4];
    // lane l of decode warp y: octet (l & 7) + 8 (y & 1), channels 8 ((l >> 3) + 4 (y >> 1))
    static __device__ __forceinline__ int oct(int tid) { return (tid & 7) + ((tid >> 5) & 1) * 8; }
    static __device__ __forceinline__ int ch8(int tid) { return ((tid >> 3) & 3) + (tid >> 6) * 4; }
    __device__ __forceinline__ void load(const AttnArgs& a, const uint8_t* base, int tid) {
        using F = Fmt<BITS>;
        const int page = 1 << a.page_log2, slot = (8 * oct(tid)) & (page - 1);
        if (!base) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                scales[i] = 0;
#pragma unroll
                for (int j = 0; j < F::kWords; ++j) w[i][j] = 0;
            }
            return;
        }
        const uint8_t* codes = base + page * (F::kDB + 4) + (slot / 2) * (2 * F::kDB) + ch8(tid) * (F::kDB / 4);
        const uint8_t* sc = base + page * (2 * F::kDB + 4) + (slot / 2) * 8 + (ch8(tid) & ~1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < F::kWords; j += 2) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes + i * 2 * F::kDB + 4 * j));
                w[i][j] = q.x;
                w[i][j + 1] = q.y;
            }
            scales[i] = __ldg(reinterpret_cast<const uint16_t*>(sc + 8 * i));
        }
    }
    __device__ __forceinline__ void store(uint8_t* tile, int tid) const {
        uint32_t s2[4], c2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s2[i] = scale_halves(scales[i]);
            c2[i] = offset_pair<BITS>(s2[i]);
        }
        // V^T is two 64-key halves of 8 KB; row = channel, 16-byte chunk = key octet
        uint8_t* half = tile + (oct(tid) >> 3) * 8192 + ch8(tid) * 8 * 128;
        constexpr int kPer = 16 / BITS;  // channels of a word
#pragma unroll
        for (int j = 0; j < Fmt<BITS>::kWords; ++j) {
            uint32_t out[4][kPer];  // [token pair][channel] (even, odd token)
#pragma unroll
            for (int i = 0; i < 4; ++i) decode_word<BITS>(w[i][j], s2[i], c2[i], out[i]);
#pragma unroll
            for (int p = 0; p < kPer; ++p)
                *reinterpret_cast<uint4*>(half + (j * kPer + p) * 128 + (((oct(tid) & 7) ^ (j * kPer + p)) << 4)) =
                    make_uint4(out[0][p], out[1][p], out[2][p], out[3][p]);
        }
    }
};

template <int BITS>
__global__ void __launch_bounds__(512, 1) kv_tc_kernel(const AttnArgs a) {
    using L = TcLayoutKv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* kv_empty = kv_full + L::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int half = warp >= 8 ? (warp - 8) >> 2 : warp & 1;
    uint64_t* bars = kv_empty + L::kStages + 7 * half;
    uint64_t *q_full = bars, *s_full = bars + 1, *s_free = bars + 2, *p_full = bars + 3, *pv_done = bars + 4,
             *drain_bar = bars + 5, *q_seen = bars + 6;
    uint64_t *x_full = kv_empty + L::kStages + 14, *x_empty = x_full + 1;
    volatile uint8_t* bad_pages = smem + L::kBad;
    volatile int* seg = reinterpret_cast<volatile int*>(smem + L::kSeg) + 2 * half;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(smem + L::kMisc + 4);
    int64_t* red = reinterpret_cast<int64_t*>(smem + L::kMisc + 8);

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&kv_full[i], 4);
            mbar_init(&kv_empty[i], 2);
        }
        for (int y = 0; y < 2; ++y) {
            uint64_t* b = kv_empty + L::kStages + 7 * y;
            mbar_init(&b[0], 4);  // q_full
            mbar_init(&b[1], 2);  // s_full: the products' completion, and the issuing thread's release of bad_pages
            mbar_init(&b[2], 4);  // s_free
            mbar_init(&b[3], 4);  // p_full
            mbar_init(&b[4], 1);  // pv_done
            mbar_init(&b[5], 1);  // drain
            mbar_init(&b[6], 1);  // q_seen
        }
        mbar_init(x_full, 4);
        mbar_init(x_empty, 4);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_base_smem, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const Start start = block_start(a, reinterpret_cast<Start*>(smem + L::kStart), red);
    tc_fence_after();
    const Cut cut = start.cut;
    Walk walk(a, start);
    const uint32_t tmem = *tmem_base_smem;
    if (threadIdx.x == 64) note_parts(a, cut, walk);  // (of a warp without other work)
    __syncwarp();  // the register split below wants whole warps
    if (start.entry < 0) {  // the whole block: nothing to do
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if (warp == 1) tmem_dealloc(tmem, L::kTmemCols);
        return;
    }

    if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------------ decode
        setmaxnreg_dec<L::kRegsDecode>();
        const int tid = threadIdx.x - 128;
        const bool withhold = g_sa_test_withhold != 0 && blockIdx.x == 0;
        // The registers hold the tile that is written next; its page pointers were looked up a tile
        // before it was loaded, and it was loaded a tile before it is written.
        Segment g;
        bool more = walk.next(a, cut, &g);  // tile t of the problem at hand, up to t1
        if (more) {
            PageRun run(a, g);
            int32_t t = g.t0, t1 = g.t1;
            KeyRegs<BITS> kr;
            ValueRegs<BITS> vr;
            int32_t ek, ev;
            bool seen;
            const uint8_t* head = run.head;
            auto look_up = [&]() {
                seen = t * 128 + tid < run.lim;
                ek = run.entry(a, t * 128 + tid);
                ev = run.entry(a, t * 128 + 8 * ValueRegs<BITS>::oct(tid));
                head = run.head;
            };
            auto advance = [&]() {
                if (++t == t1 && (more = walk.next(a, cut, &g))) {
                    run = PageRun(a, g);
                    t = g.t0;
                    t1 = g.t1;
                }
                if (more) look_up();
            };
            look_up();
            bool bad = seen && !page_at(a, head, ek);
            kr.load(a, page_at(a, head, ek), tid);
            vr.load(a, page_at(a, head, ev), tid);
            advance();
            for (int it = 0;; ++it) {
                const int st = it % L::kStages;
                if (!wait_warp(&kv_empty[st], ((it / L::kStages) & 1) ^ 1, abort_flag)) break;
                uint8_t* tile = smem + L::kKV + st * 2 * L::kTile;
                const bool last = !more;
                kr.store(tile, tid);
                if (!last) kr.load(a, page_at(a, head, ek), tid);
                vr.store(tile + L::kTile, tid);
                if ((tid & ((1 << a.page_log2) - 1)) == 0) {
                    bad_pages[st * 8 + (tid >> a.page_log2)] = bad;
                    if (bad) sa_flag_error(SA_ERR_BAD_LIST);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !(withhold && it == 0)) mbar_arrive(&kv_full[st]);
                if (last) break;
                vr.load(a, page_at(a, head, ev), tid);
                bad = seen && !page_at(a, head, ek);
                advance();
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------------ tensor-core issue
        setmaxnreg_dec<L::kRegsIssue>();
        if (warp < 2) {
            constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0), kIdescPV = idesc_bf16_f32(128, 64, 0);
            const bool leader = tc::elect_one();
            const uint64_t dq = smem_desc_sw128(smem_u32(smem + L::kQ + half * L::kTile), 16, 1024);
            const uint64_t dk0 = smem_desc_sw128(smem_u32(smem + L::kKV), 16, 1024);
            constexpr uint64_t kStep = (2 * L::kTile) >> 4;
            const uint32_t tS = tmem + L::colS(half), tP = tmem + L::colP(half), tO = tmem + L::colO(half);
            int it = 0, own = 0, problem = 0;  // tiles, this half's tiles, problems so far
            bool ok = true, any_mma = false;
            for (;;) {
                // the softmax warps say with each Q how many tiles follow, and with none that all is done
                if (!wait_warp(q_full, problem & 1, abort_flag)) break;
                const int n_tiles = seg[0], solo = seg[1];
                if (n_tiles == 0) break;
                __syncwarp();
                if (leader) mbar_arrive(q_seen);
                ++problem;
                int last = -1;  // stage of this half's last tile, whose P V is still to come
                const int first_own = own;
                for (int n = 0; n <= n_tiles; ++n) {
                    const bool mine = n < n_tiles && (!solo || (n & 1) == half);
                    const int st = (it + n) % L::kStages;
                    if (n < n_tiles && !wait_warp(&kv_full[st], ((it + n) / L::kStages) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (n < n_tiles && !mine) {  // the other half's tile
                        if (leader) mbar_arrive(&kv_empty[st]);
                        __syncwarp();
                        continue;
                    }
                    if (mine) {
                        if (own > 0 && !wait_warp(s_free, (own - 1) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_ss(tS, dq + 2 * kk, dk0 + st * kStep + 2 * kk, kIdescS, kk > 0);
                            umma_commit(s_full);
                            mbar_arrive(s_full);
                        }
                        __syncwarp();
                        any_mma = true;
                    }
                    if (last >= 0) {
                        const int i = own - 1;
                        if (!wait_warp(p_full, i & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
                            const uint64_t dv = dk0 + last * kStep + (L::kTile >> 4);
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk)
                                umma_ts(tO, tP + 8 * kk, dv + (uint64_t)((kk >> 2) * (8192 >> 4) + (kk & 3) * 2),
                                        kIdescPV, i > first_own || kk > 0);
                            umma_commit(&kv_empty[last]);
                            umma_commit(pv_done);
                        }
                        __syncwarp();
                    }
                    if (mine) {
                        last = st;
                        ++own;
                    }
                }
                if (!ok) break;
                it += n_tiles;
            }
            // every product (and its commits) is finished before TMEM is released
            if (any_mma) {
                if (leader) umma_commit(drain_bar);
                __syncwarp();
                tc::drain_wait(drain_bar, 0);
            }
        }
    } else {
        // ------------------------------------------------------------------ softmax
        setmaxnreg_inc<L::kRegsSoftmax>();
        const int quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        const uint32_t tS = tmem + L::colS(half) + lane_off, tP = tmem + L::colP(half) + lane_off,
                       tO = tmem + L::colO(half) + lane_off;
        uint8_t* rows_smem = smem + L::kQ + half * L::kTile + quad * 4096;  // this warp's rows of Q, later of O
        const float mul = a.scale_log2;
        Segment g;
        int it = 0, own = 0, joins = 0, problem = 0;
        bool ok = true;
        while (ok && walk.next(a, cut, &g)) {
            const bool solo = is_solo(a, g.nv);
            const int in = solo ? r : 128 * half + r;  // row within the problem
            const bool valid = in < g.nv;
            const int32_t x = g.rt * a.tile_rows + in;
            const int64_t row = valid ? out_row(a, g.s, g.h, x) : -1;
            // the products that read the last Q are done: their scores have been read (and a half without
            // tiles of the last problem waits until that has been noticed)
            if (problem > 0 && !wait_warp(q_seen, (problem - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            ++problem;
            // a warp's 32 rows, four whole rows an access (a row a lane would touch 32 lines with each)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = 4 * j + (lane >> 3);
                const int64_t from = __shfl_sync(0xffffffffu, row, i);
                const uint4 v = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + from * 64) + (lane & 7))
                                          : make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(rows_smem + i * 128 + (((lane & 7) ^ (i & 7)) << 4)) = v;
            }
            fence_proxy_async_smem();
            const int n_tiles = g.t1 - g.t0;
            if (r == 0) {
                seg[0] = n_tiles;
                seg[1] = solo;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            const int32_t lim = valid ? key_limit(a, g.sc, over(x, a.group)) : g.sc.len;
            const int32_t least = __reduce_min_sync(0xffffffffu, lim);
            float m_run = -INFINITY, l_run = 0.0f;
            const int first = solo ? half : 0, step = solo ? 2 : 1, first_own = own;
            for (int n = first; n < n_tiles; n += step, ++own) {
                const int t = g.t0 + n, st = (it + n) % L::kStages;
                if (!wait_warp(s_full, own & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t sv[128];
                uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 0);
                uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 32);
                uint32_t(&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 64);
                uint32_t(&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 96);
                tmem_ld_32x32b_x32(tS, s0);
                tmem_ld_32x32b_x32(tS + 32, s1);
                tmem_ld_32x32b_x32(tS + 64, s2);
                tmem_ld_32x32b_x32(tS + 96, s3);
                // one byte per sub-page; those of this tile's sub-pages were written
                const uint2 bad8 = ld_shared_v2(smem + L::kBad + st * 8);
                const int subs = 128 >> a.page_log2;
                const bool bad = (bad8.x & (subs >= 4 ? ~0u : (1u << (8 * subs)) - 1u)) != 0 || (subs == 8 && bad8.y != 0);
                tmem_ld_wait(s0);
                reg_fence(s1);
                reg_fence(s2);
                reg_fence(s3);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
                if ((int64_t)t * 128 + 128 > least || bad) {
                    const int32_t keys = min(max(lim - t * 128, 0), 128);
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const int k0 = min(max(keys - 16 * c, 0), 16);
                        uint32_t seen = (1u << k0) - 1u;
                        if (bad && bad_pages[st * 8 + ((16 * c) >> a.page_log2)]) seen = 0;
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (!((seen >> u) & 1u)) sv[16 * c + u] = __float_as_uint(-INFINITY);
                    }
                }
                float m8[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) m8[u] = __uint_as_float(sv[u]);
#pragma unroll
                for (int c = 8; c < 120; c += 16)
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        m8[u] = fmax3(m8[u], __uint_as_float(sv[c + u]), __uint_as_float(sv[c + 8 + u]));
#pragma unroll
                for (int u = 0; u < 8; ++u) m8[u] = fmaxf(m8[u], __uint_as_float(sv[120 + u]));
                const float mx = mul * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                float alpha = 1.0f;
                if (mx > m_run + 8.0f) {
                    alpha = ex2_approx(m_run - mx);
                    m_run = mx;
                    l_run *= alpha;
                }
                __syncwarp();  // the accesses to tensor memory below want whole warps
                const float m_use = m_run == -INFINITY ? 0.0f : m_run;
                const float2 mul2 = make_float2(mul, mul), neg2 = make_float2(-m_use, -m_use);
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pk[32];
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        const float2 xv = __ffma2_rn(make_float2(__uint_as_float(sv[64 * c + 2 * u]),
                                                                 __uint_as_float(sv[64 * c + 2 * u + 1])),
                                                     mul2, neg2);
                        float2 p;
                        p.x = ex2_approx(xv.x);
                        p.y = ex2_approx(xv.y);
                        acc[u & 1] = __fadd2_rn(acc[u & 1], p);
                        pk[u] = pack_bf16x2(p.x, p.y);
                    }
                    if (c == 0 && own > first_own) {
                        // O may be rescaled, and P's place is free, once the last tile's product is done
                        if (!wait_warp(pv_done, (own - 1) & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
                            for (int d = 0; d < 64; d += 16) {
                                uint32_t ov[16];
                                tmem_ld_32x32b_x16(tO + d, ov);
                                tmem_ld_wait16(ov);
#pragma unroll
                                for (int u = 0; u < 16; ++u) ov[u] = __float_as_uint(__uint_as_float(ov[u]) * alpha);
                                tmem_st_32x32b_x16(tO + d, ov);
                            }
                        }
                    }
                    tmem_st_32x32b_x32(tP + 32 * c, pk);
                }
                if (!ok) break;
                const float2 sum = __fadd2_rn(acc[0], acc[1]);
                l_run += sum.x + sum.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            it += n_tiles;
            const bool any = own > first_own;  // a solo half may have none of a single tile
            if (!ok || (any && !wait_warp(pv_done, (own - 1) & 1, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            float* join = reinterpret_cast<float*>(smem + L::kJoin) + r;
            float f0 = 1.0f, f1 = 0.0f;
            if (solo) {
                // half 1 hands its part to half 0
                if (half == 1) {
                    if (!wait_warp(x_empty, (joins & 1) ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
#pragma unroll 1
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t ov[16];
                        tmem_ld_32x32b_x16(tO + c, ov);
                        tmem_ld_wait16(ov);
#pragma unroll
                        for (int u = 0; u < 16; ++u) join[128 * (c + u)] = any ? __uint_as_float(ov[u]) : 0.0f;
                    }
                    join[128 * 64] = m_run;
                    join[128 * 65] = l_run;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(x_full);
                    ++joins;
                    continue;
                }
                if (!wait_warp(x_full, joins & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const float m1 = join[128 * 64], l1 = join[128 * 65];
                const float mm = fmaxf(m_run, m1), mu = mm == -INFINITY ? 0.0f : mm;
                f0 = ex2_approx(m_run - mu);
                f1 = ex2_approx(m1 - mu);
                l_run = l_run * f0 + l1 * f1;
                m_run = mm;
            }
            const bool whole = g.whole();
            const int64_t part = (int64_t)g.slot() * a.tile_rows + in - lane;  // this warp's first row
            const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
            // rows go out through the place of Q, 128 bytes a row at a time: all of O in bf16, or a part's
            // 32 f32 columns
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t ov[32];
                tmem_ld_32x32b_x32(tO + c, ov);
                tmem_ld_wait(ov);
                if (solo) {
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        ov[u] = __float_as_uint(__uint_as_float(ov[u]) * f0 + join[128 * (c + u)] * f1);
                }
                if (whole) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            w[u] = pack_bf16x2(__uint_as_float(ov[8 * j + 2 * u]) * inv,
                                               __uint_as_float(ov[8 * j + 2 * u + 1]) * inv);
                        *reinterpret_cast<uint4*>(rows_smem + lane * 128 + (((c / 8 + j) ^ (lane & 7)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (c == 0) continue;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(rows_smem + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_uint4(ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 4 * j + (lane >> 3);
                    const int64_t to = __shfl_sync(0xffffffffu, row, i);
                    const uint4 v = *reinterpret_cast<const uint4*>(rows_smem + i * 128 + (((lane & 7) ^ (i & 7)) << 4));
                    if (to < 0) continue;
                    if (whole) *(reinterpret_cast<uint4*>(a.o + to * 64) + (lane & 7)) = v;
                    else *(reinterpret_cast<uint4*>(a.part_o + (part + i) * 64 + c) + (lane & 7)) = v;
                }
                __syncwarp();
            }
            if (valid) {
                if (!whole) {
                    float* ml = a.part_ml + (int64_t)g.slot() * 2 * a.tile_rows + in;
                    ml[0] = m_run;
                    ml[a.tile_rows] = l_run;
                } else if (a.lse) {
                    const float m_fin = m_run == -INFINITY ? 0.0f : m_run;
                    a.lse[row] = l_run == 0.0f ? -INFINITY : (m_fin + log2f(l_run)) * 0.69314718055994530942f;
                }
            }
            if (solo) {
                __syncwarp();
                if (lane == 0) mbar_arrive(x_empty);
                ++joins;
            }
        }
        if (ok && (problem == 0 || wait_warp(q_seen, (problem - 1) & 1, abort_flag))) {
            if (r == 0) seg[0] = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
    }

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

}  // namespace kv
