// Attention over the frame cache for more than 32 query rows a problem (whole frames): the
// products on the 5th-generation tensor cores, 128 query rows against 128 keys at a time, O and the
// scores in tensor memory.  The decoding of the pages and the exponentials share the SM with them, so
// two thread blocks stay resident per SM and fill each other's waits.
// Roles (384 threads):
//   warps 0-3  softmax: thread r owns query row r and takes a tile's scores in halves of 64.  The
//              running maximum is raised (and O rescaled) only when a score is over it by more
//              than 2^8, once or twice per problem.  P goes to tensor memory as bf16, a half at a
//              time, each with barriers of its own: a half waits for no product but the one of the
//              same half a tile before.
//   warps 4-7  decode: a thread takes one key's K (4 blocks of 16 channels) and one 8 channel x 8 key
//              patch of V straight from the pages into registers, a tile ahead, and writes bf16
//              operands: K [128 keys][64], V^T [64][128 keys], both K-major with the 128-byte
//              swizzle (eight lanes write the eight 16-byte chunks of a row: no bank conflicts).
//   warp 8     (of a third warpgroup, whose registers go to the other two) tensor-core issue: per tile
//              the first half of P V, then S = Q K^T of the next tile, then the second half.
// TMEM (256 columns a block): S 128 (f32), P 64 (bf16 pairs), O 64 (f32).
#pragma once
#include "k_kv_attn.cuh"

namespace kv {

struct TcLayoutKv {
    static constexpr int kThreads = 384;
    // registers per thread after the split (launched with 80 each; the sum is the launch's own)
    static constexpr uint32_t kRegsSoftmax = 112, kRegsDecode = 80, kRegsIssue = 48;
    static constexpr uint32_t kRegsNeeded = 128 * (kRegsSoftmax + kRegsDecode + kRegsIssue);
    static constexpr int kStages = 2;
    static constexpr int kTile = 128 * 128;  // bytes of a 128 x 64 bf16 operand
    static constexpr int kQ = 0;
    static constexpr int kK = kQ + kTile;
    static constexpr int kV = kK + kStages * kTile;
    static constexpr int kBars = kV + kStages * kTile;
    // k_full[2], k_empty[2], v_full[2], v_empty[2], q_full, s_full, s_free, p_full[2], pv_done[2], drain
    static constexpr int kNumBars = 4 * kStages + 8;
    static constexpr int kBad = kBars + 8 * kNumBars;  // [4 tiles][8 sub-pages] bytes
    static constexpr int kSeg = kBad + 32;             // tiles of the problem whose Q has come
    static constexpr int kMisc = kSeg + 8;             // abort flag, tmem base, walk[2], reduction[12]
    static constexpr int kEnd = kMisc + 8 + 16 + 96;
    static constexpr uint32_t kTmemCols = 256, kColS = 0, kColP = 128, kColO = 192;
    static constexpr int smem_bytes() { return 1024 + kEnd; }
    static_assert(kBars % 8 == 0 && kMisc % 8 == 0, "alignment");
};

// The tiles of a CTA's run one after the other, across its problems.
struct TileCursor {
    Walk walk;
    Segment g;
    int32_t t;
    bool live;
    __device__ __forceinline__ TileCursor(const AttnArgs& a, const Walk& w) : walk(w) {
        live = walk.next(a, &g);
        t = live ? g.t0 : 0;
    }
    __device__ __forceinline__ void next(const AttnArgs& a) {
        if (++t < g.t1) return;
        live = walk.next(a, &g);
        t = live ? g.t0 : 0;
    }
};

// Page base (of head h) that holds token `key` of the segment's scene, or null: past the keys that
// any row sees, or a bad page.
__device__ __forceinline__ const uint8_t* page_of(const AttnArgs& a, const Segment& g, int32_t key, bool* bad) {
    *bad = false;
    if (key >= (int32_t)min((int64_t)g.tiles * 128, (int64_t)g.sc.len)) return nullptr;
    const int32_t pid = __ldg(a.table + (int64_t)g.s * a.max_pages + (key >> a.page_log2));
    if (pid < 0 || pid >= a.n_pages) {
        *bad = true;
        return nullptr;
    }
    return a.pool + ((int64_t)pid * a.kv_heads + g.h) * a.page_bytes;
}

__device__ __forceinline__ uint2 ld_shared_v2(const void* p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(smem_u32(p)) : "memory");
    return v;
}

template <int BITS>
struct KeyRegs {  // one key's K
    uint32_t w[4][Fmt<BITS>::kWords], scales;
    bool bad;
    __device__ __forceinline__ void load(const AttnArgs& a, const Segment& g, int32_t t, int tid) {
        using F = Fmt<BITS>;
        const int page = 1 << a.page_log2, slot = tid & (page - 1);
        const uint8_t* base = page_of(a, g, t * 128 + tid, &bad);
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
            const uint32_t s2 = scale_pair(((scales >> (8 * c)) & 0xFFu) * 0x00010001u);
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
    __device__ __forceinline__ void load(const AttnArgs& a, const Segment& g, int32_t t, int tid) {
        using F = Fmt<BITS>;
        const int page = 1 << a.page_log2, slot = (8 * oct(tid)) & (page - 1);
        bool bad;
        const uint8_t* base = page_of(a, g, t * 128 + 8 * oct(tid), &bad);
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
            s2[i] = scale_pair((scales[i] & 0xFFu) | (scales[i] & 0xFF00u) << 8);
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
__global__ void __launch_bounds__(384, 2) kv_tc_kernel(const AttnArgs a) {
    using L = TcLayoutKv;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t *k_full = bars, *k_empty = bars + 2, *v_full = bars + 4, *v_empty = bars + 6;
    uint64_t *q_full = bars + 8, *s_full = bars + 9, *s_free = bars + 10, *p_full = bars + 11, *pv_done = bars + 13,
             *drain_bar = bars + 15;
    volatile uint8_t* bad_pages = smem + L::kBad;
    volatile int* seg_tiles = reinterpret_cast<volatile int*>(smem + L::kSeg);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
    uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(smem + L::kMisc + 4);
    int64_t* walk_smem = reinterpret_cast<int64_t*>(smem + L::kMisc + 8);
    int64_t* red = reinterpret_cast<int64_t*>(smem + L::kMisc + 24);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&k_full[i], 4);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 4);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(q_full, 4);
        mbar_init(s_full, 2);  // the products' completion, and the issuing thread's release of bad_pages
        mbar_init(s_free, 4);
        for (int i = 0; i < 2; ++i) {  // of a tile's two 64-key halves
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    const Cut cut = cut_of(a, red);
    const int64_t x0 = blockIdx.x * cut.per;
    Walk walk;
    walk.left = min(cut.per, cut.total - x0);
    if (walk.left <= 0) {  // the whole block: nothing to do
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        return;
    }
    if (warp == 0) {
        int64_t within;
        const int32_t e = find_entry(a, x0, &within);
        if (lane == 0) walk_smem[0] = e, walk_smem[1] = within;
    }
    if (warp == 8) {
        tmem_alloc(tmem_base_smem, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_base_smem;
    walk.start(a, (int32_t)walk_smem[0], walk_smem[1]);

    if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------------ decode
        setmaxnreg_dec<L::kRegsDecode>();
        const int tid = threadIdx.x - 128;
        const bool withhold = g_sa_test_withhold != 0 && blockIdx.x == 0;
        TileCursor c(a, walk);
        KeyRegs<BITS> kr;
        ValueRegs<BITS> vr;
        if (c.live) {
            kr.load(a, c.g, c.t, tid);
            vr.load(a, c.g, c.t, tid);
        }
        for (int it = 0; c.live; ++it) {
            const int st = it & 1, ph = (it >> 1) & 1;
            if (!mbar_wait_warp(&k_empty[st], ph ^ 1, abort_flag)) break;
            kr.store(smem + L::kK + st * L::kTile, tid);
            if ((tid & ((1 << a.page_log2) - 1)) == 0) {
                bad_pages[(it & 3) * 8 + (tid >> a.page_log2)] = kr.bad;
                if (kr.bad) sa_flag_error(SA_ERR_BAD_LIST);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && !(withhold && it == 0)) mbar_arrive(&k_full[st]);
            c.next(a);
            if (c.live) kr.load(a, c.g, c.t, tid);
            if (!mbar_wait_warp(&v_empty[st], ph ^ 1, abort_flag)) break;
            vr.store(smem + L::kV + st * L::kTile, tid);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[st]);
            if (c.live) vr.load(a, c.g, c.t, tid);
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------------ tensor-core issue
        setmaxnreg_dec<L::kRegsIssue>();
        if (warp == 8) {
        constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0), kIdescPV = idesc_bf16_f32(128, 64, 0);
        const bool leader = tc::elect_one();
        const uint64_t dq = smem_desc_sw128(smem_u32(smem + L::kQ), 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(smem_u32(smem + L::kK), 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(smem_u32(smem + L::kV), 16, 1024);
        constexpr uint64_t kStep = L::kTile >> 4;
        int it = 0, seg = 0;
        bool ok = true, any_mma = false;
        for (;;) {
            // the softmax warps say with each Q how many tiles follow, and with none that all is done
            if (!mbar_wait_warp(q_full, seg & 1, abort_flag)) break;
            const int n_tiles = *seg_tiles;
            if (n_tiles == 0) break;
            // S of tile n goes out between the two halves of P V of tile n - 1
            for (int n = 0; n <= n_tiles && ok; ++n) {
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    if (part == 1) {
                        if (n == n_tiles) continue;
                        const int i = it + n, st = i & 1;
                        if (!mbar_wait_warp(&k_full[st], (i >> 1) & 1, abort_flag) ||
                            (i > 0 && !mbar_wait_warp(s_free, (i - 1) & 1, abort_flag))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_ss(tmem + L::kColS, dq + 2 * kk, dk0 + st * kStep + 2 * kk, kIdescS, kk > 0);
                            umma_commit(&k_empty[st]);
                            umma_commit(s_full);
                            mbar_arrive(s_full);
                        }
                        __syncwarp();
                        any_mma = true;
                    } else {
                        if (n == 0) continue;
                        const int i = it + n - 1, st = i & 1, half = part / 2;
                        if ((half == 0 && !mbar_wait_warp(&v_full[st], (i >> 1) & 1, abort_flag)) ||
                            !mbar_wait_warp(&p_full[half], i & 1, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_ts(tmem + L::kColO, tmem + L::kColP + 32 * half + 8 * kk,
                                        dv0 + st * kStep + (uint64_t)(half * (8192 >> 4) + kk * 2), kIdescPV,
                                        n > 1 || half > 0 || kk > 0);
                            if (half == 1) umma_commit(&v_empty[st]);
                            umma_commit(&pv_done[half]);
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok) break;
            it += n_tiles;
            ++seg;
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
        const int r = threadIdx.x;
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        const uint32_t tS = tmem + L::kColS + lane_off, tP = tmem + L::kColP + lane_off, tO = tmem + L::kColO + lane_off;
        const float mul = a.scale_log2;
        Segment g;
        int it = 0;
        bool ok = true, first_seg = true;
        while (ok && walk.next(a, &g)) {
            const int32_t nv = valid_rows(a, g.sc, g.rt);
            const int32_t x = g.rt * a.tile_rows + r;
            const int64_t row = out_row(a, g.s, g.h, x);
            // the products that read the last Q are done: their scores have been read
            {
                uint8_t* dst = smem + L::kQ + r * 128;
                const uint4* src = reinterpret_cast<const uint4*>(a.q + row * 64);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 v = r < nv ? __ldg(src + j) : make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(dst + ((j ^ (r & 7)) << 4)) = v;
                }
            }
            fence_proxy_async_smem();
            if (r == 0) *seg_tiles = g.t1 - g.t0;
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            const int32_t lim = r < nv ? key_limit(a, g.sc, x / a.group) : g.sc.len;
            const int32_t least = __reduce_min_sync(0xffffffffu, lim);
            float m_run = -INFINITY, l_run = 0.0f;
            for (int t = g.t0; t < g.t1; ++t, ++it) {
                if (!mbar_wait_warp(s_full, it & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // one byte per sub-page; those of this tile's sub-pages were written
                const uint2 bad8 = ld_shared_v2(smem + L::kBad + (it & 3) * 8);
                const int subs = 128 >> a.page_log2;
                const bool bad = (bad8.x & (subs >= 4 ? ~0u : (1u << (8 * subs)) - 1u)) != 0 || (subs == 8 && bad8.y != 0);
                const bool masked = (int64_t)t * 128 + 128 > least || bad;
                const int32_t keys = min(max(lim - t * 128, 0), 128);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t tSh = tS + 64 * half;
                    uint32_t sv[64];
                    uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv);
                    uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 32);
                    tmem_ld_32x32b_x32(tSh, s0);
                    tmem_ld_32x32b_x32(tSh + 32, s1);
                    tmem_ld_wait(s0);
                    reg_fence(s1);
                    if (half == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_free);
                    }
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int col = 64 * half + 16 * c, k0 = min(max(keys - col, 0), 16);
                            uint32_t seen = (1u << k0) - 1u;
                            if (bad && bad_pages[(it & 3) * 8 + (col >> a.page_log2)]) seen = 0;
#pragma unroll
                            for (int u = 0; u < 16; ++u)
                                if (!((seen >> u) & 1u)) sv[16 * c + u] = __float_as_uint(-INFINITY);
                        }
                    }
                    float m8[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) m8[u] = __uint_as_float(sv[u]);
#pragma unroll
                    for (int c = 8; c < 56; c += 16)
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            m8[u] = fmax3(m8[u], __uint_as_float(sv[c + u]), __uint_as_float(sv[c + 8 + u]));
#pragma unroll
                    for (int u = 0; u < 8; ++u) m8[u] = fmaxf(m8[u], __uint_as_float(sv[56 + u]));
                    const float mx = mul * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
                    if (__any_sync(0xffffffffu, mx > m_run + 8.0f)) {
                        // raise the maximum of the rows that need it and rescale what was summed, once every
                        // product so far is done
                        const float m_new = mx > m_run + 8.0f ? mx : m_run;
                        const float alpha = m_new == m_run ? 1.0f : ex2_approx(m_run - m_new);
                        m_run = m_new;
                        l_run *= alpha;
                        if (t > g.t0 || half > 0) {
                            // the half before: of this tile, or the second one of the tile before
                            if (!mbar_wait_warp(&pv_done[half ^ 1], (half ? it : it - 1) & 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < 64; c += 8) {
                                uint32_t ov[8];
                                tmem_ld_32x32b_x8(tO + c, ov);
                                tmem_ld_wait8(ov);
#pragma unroll
                                for (int u = 0; u < 8; ++u) ov[u] = __float_as_uint(__uint_as_float(ov[u]) * alpha);
                                tmem_st_32x32b_x8(tO + c, ov);
                            }
                        }
                    }
                    const float m_use = m_run == -INFINITY ? 0.0f : m_run;
                    const float2 mul2 = make_float2(mul, mul), neg2 = make_float2(-m_use, -m_use);
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int u = 0; u < 16; ++u) {
                            const float2 xv = __ffma2_rn(make_float2(__uint_as_float(sv[32 * c + 2 * u]),
                                                                     __uint_as_float(sv[32 * c + 2 * u + 1])),
                                                         mul2, neg2);
                            float2 p;
                            p.x = ex2_approx(xv.x);
                            p.y = ex2_approx(xv.y);
                            acc = __fadd2_rn(acc, p);
                            pk[u] = pack_bf16x2(p.x, p.y);
                        }
                        // this half's place for P is free once its product of the tile before is done
                        if (c == 0 && t > g.t0) {
                            if (!mbar_wait_warp(&pv_done[half], (it - 1) & 1, abort_flag)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        tmem_st_32x32b_x16(tP + 32 * half + 16 * c, pk);
                    }
                    if (!ok) break;
                    l_run += acc.x + acc.y;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[half]);
                }
                if (!ok) break;
            }
            if (!ok || !mbar_wait_warp(&pv_done[1], (it - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const bool whole = g.t0 == 0 && g.t1 == g.tiles;
            const int slot = part_slot(first_seg);
            const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t ov[32];
                tmem_ld_32x32b_x32(tO + 32 * c, ov);
                tmem_ld_wait(ov);
                if (r < nv) {
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(a.o + row * 64 + 32 * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t w[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                w[u] = pack_bf16x2(__uint_as_float(ov[8 * j + 2 * u]) * inv,
                                                   __uint_as_float(ov[8 * j + 2 * u + 1]) * inv);
                            dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(a.part_o + ((int64_t)slot * a.tile_rows + r) * 64 + 32 * c);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            dst[j] = make_uint4(ov[4 * j], ov[4 * j + 1], ov[4 * j + 2], ov[4 * j + 3]);
                    }
                }
            }
            if (r < nv) {
                if (!whole) {
                    a.part_ml[(int64_t)slot * 2 * a.tile_rows + r] = m_run;
                    a.part_ml[((int64_t)slot * 2 + 1) * a.tile_rows + r] = l_run;
                } else if (a.lse) {
                    const float m_fin = m_run == -INFINITY ? 0.0f : m_run;
                    a.lse[row] = l_run == 0.0f ? -INFINITY : (m_fin + log2f(l_run)) * 0.69314718055994530942f;
                }
            }
            first_seg = false;
        }
        if (ok) {
            if (r == 0) *seg_tiles = 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
    }

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

}  // namespace kv
