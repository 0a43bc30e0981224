// The frame cache: K and V rows of the frames seen so far, held in 4 or 8 bits in pages.
//
// A stored number is code * s, one scale s per 16 channels of one token:
//   s = (8 + b % 8) / 8 * 2^(b / 8 - 16)   for the scale byte b
//   4 bits: s = smallest scale with 7.5 s >= max|x|,            code = clamp(rne(x / s), -7, 7)
//   8 bits: s = smallest power of two with 127.5 s >= max|x|,   code = clamp(rne(x / s), -127, 127)
// 7.5 s (127.5 s) is the largest magnitude that still rounds to within half a step of the top code, so
// no finite value within the scales' range is off by more than s / 2.  Every stored number is exactly
// a bf16 number (4-bit code times 4-bit significand; 7-bit code times a power of two): reading back in
// bf16 and bf16 tensor-core operands built from a page add no rounding.  Every bit pattern of a page
// decodes to a finite number, so a masked key's bytes, whatever they are, times a zero probability
// give zero.
//
// Page of one head (64 channels, DB = 32 or 64 bytes of codes per vector):
//   [K codes  page x DB][K scales page x 4][V codes page x DB][V scales page x 4]
// Codes come in 16-bit units: four 4-bit codes (code + 8; code j in bits 4j..4j+3), or two 8-bit codes
// (a: magnitude in bits 0-6, sign in bit 15; b: magnitude in bits 8-14, sign in bit 7).  The two
// units of a 32-bit word become the two halves of bf16x2 registers:
//   K word of a token:       low unit even channels, high unit odd channels of 8 (4) consecutive ones
//   V word of a token pair:  low unit the even token, high unit the odd token, 4 (2) channels
// so that one word gives register pairs in the operand order of both products (K: pairs along the
// channels, V: pairs along the keys), and one token of a pair can be written without reading the other.
//   K scales [token][4 blocks], V scales [token pair][4 blocks][even, odd token]
#pragma once
#include "sa_device.cuh"

namespace kv {

constexpr int kScaleBias = 16;
constexpr uint32_t kScaleF32Bits = (uint32_t)(127 - kScaleBias) << 23;   // float bits of s for b = 0
constexpr uint32_t kScaleBf16Pair = (uint32_t)((127 - kScaleBias) << 7) * 0x00010001u;

template <int BITS>
struct Fmt {
    static constexpr int kDB = 64 * BITS / 8;        // bytes of codes per 64-channel vector
    static constexpr int kWords = BITS / 2;          // 32-bit words per 16 codes
    static constexpr int kTokenBytes = 2 * (kDB + 4);  // K and V of one token and head
};

__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (a & b) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// (a & b) ^ c in one instruction
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// bf16x2 scales of two scale bytes in bits 0-7 (low half) and 16-23 (high half).
__device__ __forceinline__ uint32_t scale_pair(uint32_t bytes) { return (bytes << 4) + kScaleBf16Pair; }
// One scale byte for both halves (a multiply-add), and two bytes of bits 0-15 for the halves.
__device__ __forceinline__ uint32_t scale_both(uint32_t b) { return b * 0x00100010u + kScaleBf16Pair; }
__device__ __forceinline__ uint32_t scale_halves(uint32_t b01) { return scale_pair(__byte_perm(b01, 0, 0x4140)); }

// The offset that goes with a scale pair: a code enters the product as 128 + (code + 8) (4 bits)
// or +-(128 + magnitude) (8 bits), the bf16 numbers whose low mantissa bits are the stored ones;
// -136 s (17 * 8 times a 4-bit significand: 8 bits) and -128 s are bf16 numbers as well.
template <int BITS>
__device__ __forceinline__ uint32_t offset_pair(uint32_t s2) {
    return hmul2_bf16(s2, BITS == 4 ? 0xC308C308u : 0xC300C300u);  // -136, -128
}

// Decodes one word: out[p] holds (low unit's code p, high unit's code p) times their scales.  One
// mask and one FMA a pair (plus a shift, or a byte swap and the sign).
template <int BITS>
__device__ __forceinline__ void decode_word(uint32_t x, uint32_t s2, uint32_t c2, uint32_t* out) {
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = hfma2_bf16(and_or(x >> (4 * j), 0x000F000Fu, 0x43004300u), s2, c2);
    } else {
        const uint32_t y = __byte_perm(x, 0, 0x2301);
        out[0] = hfma2_bf16(and_or(x, 0x807F807Fu, 0x43004300u), s2, and_xor(x, 0x80008000u, c2));
        out[1] = hfma2_bf16(and_or(y, 0x807F807Fu, 0x43004300u), s2, and_xor(y, 0x80008000u, c2));
    }
}
// The words of 16 codes (a K block, or 8 channels of a V pair), in order.
template <int BITS>
__device__ __forceinline__ void decode(const uint32_t (&w)[Fmt<BITS>::kWords], uint32_t s2, uint32_t c2,
                                       uint32_t (&out)[8]) {
#pragma unroll
    for (int i = 0; i < Fmt<BITS>::kWords; ++i) decode_word<BITS>(w[i], s2, c2, out + i * (16 / BITS));
}

struct CacheArgs {
    uint8_t* pool;
    const int32_t* table;   // [scenes][max_pages]
    const int32_t* lens;    // [scenes]
    const int32_t* n_len;   // [scenes] or null: rows of each scene, <= n
    const int32_t* start;   // read: [scenes] or null
    void *k, *v;            // rows [scenes * heads][n][64]
    int32_t scenes, heads, n;
    int32_t page_log2, n_pages, max_pages;
    int64_t page_bytes;     // bytes of one page of one head
    int32_t wide;           // k and v start on 32-byte boundaries: whole sectors a lane and access
};

// Tokens of a scene, clamped to what its row of the page table can hold (reported when it is not).
__device__ __forceinline__ int32_t scene_len(const int32_t* lens, int s, int32_t max_pages, int32_t page_log2) {
    const int32_t len = __ldg(lens + s);
    const int64_t top = (int64_t)max_pages << page_log2;
    if (len < 0 || len > top) {
        sa_flag_error(SA_ERR_INVALID_ARG);
        return len < 0 ? 0 : (int32_t)top;
    }
    return len;
}
// Rows of a scene, clamped into [0, n] (reported when they were not).
__device__ __forceinline__ int32_t scene_rows(const int32_t* n_len, int s, int32_t n) {
    if (!n_len) return n;
    const int32_t m = __ldg(n_len + s);
    if (m < 0 || m > n) {
        sa_flag_error(SA_ERR_INVALID_ARG);
        return m < 0 ? 0 : n;
    }
    return m;
}

// 32 bytes of a row, as one access where the address allows it: with two of 16 bytes every lane's
// sector is touched twice (half a sector a store cost the reading kernel a quarter of its rate).
__device__ __forceinline__ void load32(const void* p, int wide, uint32_t* w) {
    if (wide) {
        asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldcs(static_cast<const uint4*>(p)), b = __ldcs(static_cast<const uint4*>(p) + 1);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* p, int wide, const uint32_t* w) {
    if (wide) {
        asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        __stcs(static_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        __stcs(static_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
    }
}

// --------------------------------------------------------------------------- writing

// 16 channels of one row as they lie in memory.
template <typename T>
struct Raw {
    static constexpr int kWords = 4 * sizeof(T);
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* src, int wide) {
#pragma unroll
        for (int i = 0; i < kWords; i += 8) load32(reinterpret_cast<const uint32_t*>(src) + i, wide, w + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};

// max(|a|, |b|, |c|), NaN if one of them is
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// x limited to [-top, top] in one instruction: the smaller magnitude with x's sign
__device__ __forceinline__ float limit_abs(float x, float top) {
    float d;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(top));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float c) { return __fadd2_rn(a, make_float2(c, c)); }

// Scale byte of 16 channels; replaces what cannot be stored (infinities become the largest stored
// magnitude, NaN zero) and reports it.
template <int BITS, typename T>
__device__ __forceinline__ int32_t scale_byte(float (&x)[16]) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) most = max_abs3(most, x[i], x[i + 1]);
    if (!(most <= 3.402823466e38f)) {
        sa_flag_error(SA_ERR_NONFINITE);
        most = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = x[i] != x[i] ? 0.0f : fminf(fmaxf(x[i], -3.0e38f), 3.0e38f);
            most = fmaxf(most, fabsf(x[i]));
        }
    }
    if constexpr (BITS == 4) {
        // truncated to 4 significant bits, most / 7.5 is the scale sought or the one below it (or, when an
        // f32 quotient rounded down across a scale, the second below)
        int32_t b = (int32_t)(__float_as_uint(most * (1.0f / 7.5f)) >> 20);
        b += 7.5f * __uint_as_float((uint32_t)b << 20) < most;
        if (sizeof(T) == 4) b += 7.5f * __uint_as_float((uint32_t)b << 20) < most;
        return min(max(b - (int32_t)(kScaleF32Bits >> 20), 0), 255);
    } else {
        int32_t e = (int32_t)(__float_as_uint(most * (1.0f / 127.5f)) >> 23);
        e += 127.5f * __uint_as_float((uint32_t)e << 23) < most;
        e += 127.5f * __uint_as_float((uint32_t)e << 23) < most;
        return 8 * min(max(e - (127 - kScaleBias), 0), 31);
    }
}

// Codes (as whole floats) of pairs of channels: n.x of a channel with scale s.x, n.y of one with s.y.
// x / s is decided exactly.  A product with the reciprocal of s is within 2^-21 of it; what rounding can
// get wrong is a value on, or next to, the border m + 1/2 between two codes.
//   8 bits: s is a power of two, the product is exact.
//   bf16 x: x / s is a border exactly or at least 1e-3 off it (8-bit x, 4-bit s), so rounding the
//     product to a multiple of 2^-14 first (adding and subtracting 1.5 * 2^9) restores the tie.
//   f32 x: the remainder x - n s is exact (one FMA; it has at most the bits of x).  Where none of a
//     thread's 16 reaches s / 2, which is nearly always, all are right; otherwise n moves where the
//     remainder is over s / 2, or is s / 2 and n is odd.
struct PairScale {
    float2 s, inv;
};
template <int BITS>
__device__ __forceinline__ PairScale pair_scale(int32_t bx, int32_t by) {
    PairScale p;
    p.s = make_float2(__uint_as_float(((uint32_t)bx << 20) + kScaleF32Bits),
                      __uint_as_float(((uint32_t)by << 20) + kScaleF32Bits));
    if constexpr (BITS == 4) {
        p.inv = make_float2(__frcp_rn(p.s.x), __frcp_rn(p.s.y));
    } else {
        p.inv = make_float2(__uint_as_float((254u << 23) - __float_as_uint(p.s.x)),
                            __uint_as_float((254u << 23) - __float_as_uint(p.s.y)));
    }
    return p;
}
template <int BITS, typename T, int N>
__device__ __forceinline__ void round_codes(const float2 (&x)[N], const PairScale& p, float2 (&n)[N]) {
    constexpr float kTop = BITS == 4 ? 7.0f : 127.0f;
    float worst = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float2 u = __fmul2_rn(x[i], p.inv);
        u.x = limit_abs(u.x, kTop);
        u.y = limit_abs(u.y, kTop);
        if (BITS == 4 && sizeof(T) == 2) u = add2(add2(u, 768.0f), -768.0f);
        // adding and subtracting 1.5 * 2^23 rounds to the nearest integer, ties to even
        n[i] = add2(add2(u, 12582912.0f), -12582912.0f);
        if (BITS == 4 && sizeof(T) == 4) {
            const float2 d = __ffma2_rn(make_float2(-n[i].x, -n[i].y), p.s, x[i]);
            worst = max_abs3(worst, d.x * p.inv.x, d.y * p.inv.y);
        }
    }
    if (BITS == 4 && sizeof(T) == 4 && worst >= 0.49999f) {
        auto settle = [&](float x1, float s1, float& n1) {
            const float d = fmaf(-n1, s1, x1), over = fabsf(d) - 0.5f * s1;
            if (over > 0.0f || (over == 0.0f && ((int)n1 & 1))) n1 += d > 0.0f ? 1.0f : -1.0f;
            n1 = fminf(fmaxf(n1, -kTop), kTop);
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            settle(x[i].x, p.s.x, n[i].x);
            settle(x[i].y, p.s.y, n[i].y);
        }
    }
}
// The two units of a word from 16 / BITS code pairs (pair.x for the low unit, pair.y for the high one):
// 4 bits: sum of (code + 8) 16^j in f32, exact below 2^16; 2^23 more leaves it in the low bits
template <int BITS>
__device__ __forceinline__ uint32_t pack_word(const float2* n) {
    if constexpr (BITS == 4) {
        float2 v = add2(n[0], 8388608.0f + 8.0f * 4369.0f);
        v = __ffma2_rn(n[1], make_float2(16.0f, 16.0f), v);
        v = __ffma2_rn(n[2], make_float2(256.0f, 256.0f), v);
        v = __ffma2_rn(n[3], make_float2(4096.0f, 4096.0f), v);
        return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x5410);
    } else {
        const float2 v = __ffma2_rn(make_float2(fabsf(n[1].x), fabsf(n[1].y)), make_float2(256.0f, 256.0f),
                                    make_float2(fabsf(n[0].x) + 8388608.0f, fabsf(n[0].y) + 8388608.0f));
        const uint32_t mag = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x5410);
        // signs: bytes 3 of n[1].x, n[0].x, n[1].y, n[0].y in bytes 0 to 3
        const uint32_t lo = __byte_perm(__float_as_uint(n[1].x), __float_as_uint(n[0].x), 0x0073);
        const uint32_t hi = __byte_perm(__float_as_uint(n[1].y), __float_as_uint(n[0].y), 0x0073);
        return and_or(__byte_perm(lo, hi, 0x5410), 0x80808080u, mag);
    }
}

// One thread: 16 channels of a token pair, K and V: the maximum of a scale's 16 channels is a thread's
// own, and no thread shares a word with another.  Bound by its arithmetic at first (17 instructions an
// element, 3.0 TB/s of bf16 into 4 bits); packed f32 pairs, three-input maxima and packing by
// multiply-add leave about 8.  65 536 tokens x 16 heads in a recorded graph (bytes read and written):
// bf16 into 4 bits 61 us, 5.6 TB/s (issue 75 %, DRAM 62 % of its peak), into 8 bits 70 us, 5.9 TB/s; f32 into
// 4 bits 109 us, 5.6 TB/s, 8 bits 99 us, 6.9 TB/s.  Four blocks an SM for bf16 into 4
// bits (three for the others) make it spill 48 bytes a thread, three make f32 into 4 bits spill 152; 8 bits have none.
template <int BITS, typename T>
__global__ void __launch_bounds__(256, BITS == 4 && sizeof(T) == 2 ? 4 : 3) append_kernel(const CacheArgs a) {
    using F = Fmt<BITS>;
    constexpr int kPer = 16 / BITS;  // codes of one unit
    const int h = blockIdx.x % a.heads, s = blockIdx.x / a.heads;
    const int32_t n = scene_rows(a.n_len, s, a.n);
    const int32_t len = scene_len(a.lens, s, a.max_pages, a.page_log2);
    const int32_t p0 = len - n;  // position of the scene's first new row
    if (p0 < 0) sa_flag_error(SA_ERR_INVALID_ARG);  // rows before position 0 have no place
    const int32_t lo = max(p0, 0);
    if (lo >= len) return;  // nothing new: below, a pair that is visited has a new token
    const int32_t page = 1 << a.page_log2;
    const int blk = threadIdx.x & 3;
    for (int64_t pair = lo / 2 + (int64_t)(blockIdx.y * 64 + threadIdx.x / 4); 2 * pair < len;
         pair += (int64_t)gridDim.y * 64) {
        const int32_t t = (int32_t)(2 * pair);
        const int32_t pid = __ldg(a.table + (int64_t)s * a.max_pages + (t >> a.page_log2));
        if (pid < 0 || pid >= a.n_pages) {
            sa_flag_error(SA_ERR_BAD_LIST);
            continue;
        }
        const bool live[2] = {t >= lo, t + 1 < len};
        const int64_t at = ((int64_t)blockIdx.x * a.n + (t - p0)) * 64 + 16 * blk;
        Raw<T> raw[2][2];  // [K, V][token]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            raw[0][e].zero();
            raw[1][e].zero();
            if (live[e]) {
                raw[0][e].load(static_cast<const T*>(a.k) + at + 64 * e, a.wide);
                raw[1][e].load(static_cast<const T*>(a.v) + at + 64 * e, a.wide);
            }
        }
        const int32_t slot = t & (page - 1);
        uint8_t* base = a.pool + ((int64_t)pid * a.heads + h) * a.page_bytes;
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // K: pairs along the channels
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = raw[0][e].get(i);
            const int32_t b = scale_byte<BITS, T>(x);
            float2 xp[8], np[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) xp[i] = make_float2(x[2 * i], x[2 * i + 1]);
            round_codes<BITS, T>(xp, pair_scale<BITS>(b, b), np);
            if (!live[e]) continue;
            uint8_t* kc = base + (slot + e) * F::kDB + blk * (F::kDB / 4);
            uint32_t w[F::kWords];
#pragma unroll
            for (int i = 0; i < F::kWords; ++i) w[i] = pack_word<BITS>(np + i * kPer);
            if constexpr (BITS == 4) *reinterpret_cast<uint2*>(kc) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint4*>(kc) = make_uint4(w[0], w[1], w[2], w[3]);
            base[page * F::kDB + (slot + e) * 4 + blk] = (uint8_t)b;
        }
        // V: pairs along the tokens
        float x[2][16];
        int32_t b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[e][i] = raw[1][e].get(i);
            b[e] = scale_byte<BITS, T>(x[e]);
        }
        float2 xp[16], np[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) xp[i] = make_float2(x[0][i], x[1][i]);
        round_codes<BITS, T>(xp, pair_scale<BITS>(b[0], b[1]), np);
        uint8_t* vc = base + page * (F::kDB + 4) + (slot / 2) * (2 * F::kDB) + blk * (F::kDB / 2);
        uint8_t* vs = base + page * (2 * F::kDB + 4) + (slot / 2) * 8 + 2 * blk;
        uint32_t w[2 * F::kWords];
#pragma unroll
        for (int i = 0; i < 2 * F::kWords; ++i) w[i] = pack_word<BITS>(np + i * kPer);
        if (live[0] && live[1]) {
#pragma unroll
            for (int i = 0; i < 2 * F::kWords; i += 4)
                *reinterpret_cast<uint4*>(vc + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            *reinterpret_cast<uint16_t*>(vs) = (uint16_t)(b[0] | b[1] << 8);
        } else {
            const int e = live[1] ? 1 : 0;
#pragma unroll
            for (int i = 0; i < 2 * F::kWords; ++i)
                *reinterpret_cast<uint16_t*>(vc + 4 * i + 2 * e) = (uint16_t)(e ? w[i] >> 16 : w[i]);
            vs[e] = (uint8_t)(e ? b[1] : b[0]);
        }
    }
}

// --------------------------------------------------------------------------- reading back

// 16 channels as bf16x2 words, in the row's type
template <typename T>
__device__ __forceinline__ void store16(T* dst, int wide, const uint32_t (&w)[8]) {
    if constexpr (sizeof(T) == 2) {
        store32(dst, wide, w);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = w[4 * j + i] << 16;
                f[2 * i + 1] = w[4 * j + i] & 0xFFFF0000u;
            }
            store32(dst + 8 * j, wide, f);
        }
    }
}

// One thread: 16 channels of a token pair, K and V (the writing kernel's mapping).  Bound by its writes:
// 65 536 tokens x 16 heads in a recorded graph, from 4 bits to bf16 56 us, 6.1 TB/s, from 8 bits 66 us, 6.3 TB/s;
// to f32 95 and 104 us, 6.4 and 6.5 TB/s.
template <int BITS, typename T>
__global__ void __launch_bounds__(256) read_kernel(const CacheArgs a) {
    using F = Fmt<BITS>;
    const int h = blockIdx.x % a.heads, s = blockIdx.x / a.heads;
    const int32_t n = scene_rows(a.n_len, s, a.n);
    const int32_t len = scene_len(a.lens, s, a.max_pages, a.page_log2);
    const int64_t p0 = a.start ? (int64_t)__ldg(a.start + s) : (int64_t)len - n;
    const int32_t lo = (int32_t)max(p0, (int64_t)0), hi = (int32_t)min(p0 + n, (int64_t)len);
    const int32_t page = 1 << a.page_log2;
    const int blk = threadIdx.x & 3;
    for (int64_t pair = lo / 2 + (int64_t)(blockIdx.y * 64 + threadIdx.x / 4); 2 * pair < hi;
         pair += (int64_t)gridDim.y * 64) {
        const int32_t t = (int32_t)(2 * pair);
        const int32_t pid = __ldg(a.table + (int64_t)s * a.max_pages + (t >> a.page_log2));
        if (pid < 0 || pid >= a.n_pages) {
            sa_flag_error(SA_ERR_BAD_LIST);
            continue;
        }
        const bool live[2] = {t >= lo, t + 1 < hi};
        const int32_t slot = t & (page - 1);
        const uint8_t* base = a.pool + ((int64_t)pid * a.heads + h) * a.page_bytes;
        const int64_t row = ((int64_t)blockIdx.x * a.n + (t - p0)) * 64 + 16 * blk;
        if (a.k) {
            const uint8_t* kc = base + slot * F::kDB + blk * (F::kDB / 4);
            const uint8_t* ks = base + page * F::kDB + slot * 4 + blk;
            uint32_t w[2][F::kWords], sb[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int i = 0; i < F::kWords; i += 2) {
                    const uint2 q = __ldg(reinterpret_cast<const uint2*>(kc + e * F::kDB + 4 * i));
                    w[e][i] = q.x;
                    w[e][i + 1] = q.y;
                }
                sb[e] = __ldg(ks + 4 * e);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t out[8];
                const uint32_t s2 = scale_both(sb[e]);
                decode<BITS>(w[e], s2, offset_pair<BITS>(s2), out);
                if (live[e]) store16<T>(static_cast<T*>(a.k) + row + 64 * e, a.wide, out);
            }
        }
        if (a.v) {
            const uint8_t* vc = base + page * (F::kDB + 4) + (slot / 2) * (2 * F::kDB) + blk * (F::kDB / 2);
            const uint8_t* vs = base + page * (2 * F::kDB + 4) + (slot / 2) * 8 + 2 * blk;
            uint32_t w[2][F::kWords];  // channels 0-7 and 8-15 of the block, both tokens
#pragma unroll
            for (int i = 0; i < 2 * F::kWords; i += 4) {
                const uint4 q = __ldg(reinterpret_cast<const uint4*>(vc + 4 * i));
                w[i / F::kWords][i % F::kWords] = q.x;
                w[i / F::kWords][(i + 1) % F::kWords] = q.y;
                w[(i + 2) / F::kWords][(i + 2) % F::kWords] = q.z;
                w[(i + 2) / F::kWords][(i + 3) % F::kWords] = q.w;
            }
            const uint32_t sb = __ldg(reinterpret_cast<const uint16_t*>(vs));
            const uint32_t s2 = scale_halves(sb), c2 = offset_pair<BITS>(s2);
            uint32_t even[8], odd[8];  // channel pairs of each token
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t out[8];
                decode<BITS>(w[i], s2, c2, out);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    even[4 * i + j] = __byte_perm(out[2 * j], out[2 * j + 1], 0x5410);
                    odd[4 * i + j] = __byte_perm(out[2 * j], out[2 * j + 1], 0x7632);
                }
            }
            if (live[0]) store16<T>(static_cast<T*>(a.v) + row, a.wide, even);
            if (live[1]) store16<T>(static_cast<T*>(a.v) + row + 64, a.wide, odd);
        }
    }
}

}  // namespace kv
