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

// --------------------------------------------------------------------------- writing

template <typename T>
__device__ __forceinline__ void load16(const T* src, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* src, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 q = __ldcs(reinterpret_cast<const float4*>(src) + i);
        x[4 * i] = q.x;
        x[4 * i + 1] = q.y;
        x[4 * i + 2] = q.z;
        x[4 * i + 3] = q.w;
    }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* src, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 q = __ldcs(reinterpret_cast<const uint4*>(src) + i);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

// Quantises 16 channels: integer codes (4 bits: code + 8; 8 bits: signed) and the scale byte.
// x / s is decided exactly.  A product with the rounded reciprocal of s is within 2^-22 of it; what
// rounding can get wrong is a value on, or next to, the border m + 1/2 between two codes.
//   8 bits: s is a power of two, the product is exact.
//   bf16 x: x / s is a border exactly or at least 1e-3 off it (8-bit x, 4-bit s), so rounding the
//     product to a multiple of 2^-14 first (adding and subtracting 1.5 * 2^9) restores the tie.
//   f32 x: the remainder x - m s is exact (one FMA; it has at most the bits of x) and moves m where
//     it is over s / 2, or a tie that rounded to odd.
template <int BITS, typename T>
__device__ __forceinline__ uint32_t quantise16(float (&x)[16], int32_t (&code)[16]) {
    constexpr bool kBf16 = sizeof(T) == 2;
    constexpr float kTop = BITS == 4 ? 7.0f : 127.0f;
    float most = 0.0f, bad = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        most = fmaxf(most, fabsf(x[i]));
        bad = fmaf(x[i], 0.0f, bad);  // NaN once any x is infinite or NaN
    }
    if (!(bad == 0.0f)) {
        // no code stands for them: infinities become the largest stored magnitude, NaN zero
        sa_flag_error(SA_ERR_NONFINITE);
        most = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = x[i] != x[i] ? 0.0f : fminf(fmaxf(x[i], -3.0e38f), 3.0e38f);
            most = fmaxf(most, fabsf(x[i]));
        }
    }
    int32_t b;
    if constexpr (BITS == 4) {
        // truncated to 4 significant bits it is the scale sought or the one or two below it
        b = (int32_t)(__float_as_uint(most * (1.0f / 7.5f)) >> 20);
        b += 7.5f * __uint_as_float((uint32_t)b << 20) < most;
        b += 7.5f * __uint_as_float((uint32_t)b << 20) < most;
        b = min(max(b - (int32_t)(kScaleF32Bits >> 20), 0), 255);
    } else {
        int32_t e = (int32_t)(__float_as_uint(most * (1.0f / 127.5f)) >> 23);
        e += 127.5f * __uint_as_float((uint32_t)e << 23) < most;
        e += 127.5f * __uint_as_float((uint32_t)e << 23) < most;
        b = 8 * min(max(e - (127 - kScaleBias), 0), 31);
    }
    const float s = __uint_as_float(((uint32_t)b << 20) + kScaleF32Bits);
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float u = fminf(fmaxf(x[i] * inv, -kTop), kTop);
        float m;
        if constexpr (BITS == 4 && kBf16) {
            u = __fadd_rn(__fadd_rn(u, 768.0f), -768.0f);
            m = u;
        } else if constexpr (BITS == 4) {
            float n = rintf(u);
            const float d = fmaf(-n, s, x[i]);
            const float over = fabsf(d) - 0.5f * s;
            if (over > 0.0f || (over == 0.0f && ((int)n & 1))) n += d > 0.0f ? 1.0f : -1.0f;
            m = fminf(fmaxf(n, -kTop), kTop);
        } else {
            m = u;
        }
        // adding 1.5 * 2^23 rounds to the nearest integer, ties to even
        code[i] = (int32_t)__float_as_uint(__fadd_rn(m, 12582912.0f)) - (BITS == 4 ? 0x4B400000 - 8 : 0x4B400000);
    }
    return (uint32_t)b;
}

__device__ __forceinline__ uint32_t unit4(int32_t a, int32_t b, int32_t c, int32_t d) {
    return (uint32_t)a | (uint32_t)b << 4 | (uint32_t)c << 8 | (uint32_t)d << 12;
}
__device__ __forceinline__ uint32_t unit8(int32_t a, int32_t b) {
    return (uint32_t)abs(a) | (a < 0 ? 0x8000u : 0u) | (uint32_t)abs(b) << 8 | (b < 0 ? 0x80u : 0u);
}

// One thread: 16 channels of a token pair, K and V.  Whole 16-byte loads (eight in flight a
// thread for bf16), no shuffles: the maximum of a scale's 16 channels is a thread's own.
template <int BITS, typename T>
__global__ void __launch_bounds__(256) append_kernel(const CacheArgs a) {
    using F = Fmt<BITS>;
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
        const T* k = static_cast<const T*>(a.k) + ((int64_t)blockIdx.x * a.n + (t - p0)) * 64 + 16 * blk;
        const T* v = static_cast<const T*>(a.v) + ((int64_t)blockIdx.x * a.n + (t - p0)) * 64 + 16 * blk;
        float x[4][16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (live[e]) {
                load16<T>(k + 64 * e, x[e]);
                load16<T>(v + 64 * e, x[2 + e]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[e][i] = x[2 + e][i] = 0.0f;
            }
        }
        const int32_t slot = t & (page - 1);
        uint8_t* base = a.pool + ((int64_t)pid * a.heads + h) * a.page_bytes;
        uint8_t* kc = base + slot * F::kDB + blk * (F::kDB / 4);
        uint8_t* ks = base + page * F::kDB + slot * 4 + blk;
        uint8_t* vc = base + page * (F::kDB + 4) + (slot / 2) * (2 * F::kDB) + blk * (F::kDB / 2);
        uint8_t* vs = base + page * (2 * F::kDB + 4) + (slot / 2) * 8 + 2 * blk;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            int32_t c[16];
            const uint32_t b = quantise16<BITS, T>(x[e], c);
            if (!live[e]) continue;
            if constexpr (BITS == 4) {
                uint2 w;
                w.x = unit4(c[0], c[2], c[4], c[6]) | unit4(c[1], c[3], c[5], c[7]) << 16;
                w.y = unit4(c[8], c[10], c[12], c[14]) | unit4(c[9], c[11], c[13], c[15]) << 16;
                *reinterpret_cast<uint2*>(kc + e * F::kDB) = w;
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = unit8(c[4 * i], c[4 * i + 2]) | unit8(c[4 * i + 1], c[4 * i + 3]) << 16;
                *reinterpret_cast<uint4*>(kc + e * F::kDB) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            ks[4 * e] = (uint8_t)b;
        }
        {
            constexpr int kUnits = 16 * BITS / 16;  // units of one token's 16 channels
            uint32_t unit[2][kUnits], b[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                int32_t c[16];
                b[e] = quantise16<BITS, T>(x[2 + e], c);
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    unit[e][i] = BITS == 4 ? unit4(c[4 * i % 16], c[(4 * i + 1) % 16], c[(4 * i + 2) % 16], c[(4 * i + 3) % 16])
                                           : unit8(c[2 * i], c[2 * i + 1]);
            }
            if (live[0] && live[1]) {
#pragma unroll
                for (int i = 0; i < kUnits; i += 4)
                    *reinterpret_cast<uint4*>(vc + 4 * i) =
                        make_uint4(unit[0][i] | unit[1][i] << 16, unit[0][i + 1] | unit[1][i + 1] << 16,
                                   unit[0][i + 2] | unit[1][i + 2] << 16, unit[0][i + 3] | unit[1][i + 3] << 16);
                *reinterpret_cast<uint16_t*>(vs) = (uint16_t)(b[0] | b[1] << 8);
            } else {
                const int e = live[1] ? 1 : 0;
#pragma unroll
                for (int i = 0; i < kUnits; ++i)
                    *reinterpret_cast<uint16_t*>(vc + 4 * i + 2 * e) = (uint16_t)(e ? unit[1][i] : unit[0][i]);
                vs[e] = (uint8_t)(e ? b[1] : b[0]);
            }
        }
    }
}

// --------------------------------------------------------------------------- reading back

template <typename T>
__device__ __forceinline__ void store16(T* dst, const uint32_t (&w)[8]);  // w: bf16x2 of 16 channels
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* dst, const uint32_t (&w)[8]) {
    __stcs(reinterpret_cast<uint4*>(dst), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(dst) + 1, make_uint4(w[4], w[5], w[6], w[7]));
}
template <>
__device__ __forceinline__ void store16<float>(float* dst, const uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        __stcs(reinterpret_cast<uint4*>(dst) + i, make_uint4(w[2 * i] << 16, w[2 * i] & 0xFFFF0000u, w[2 * i + 1] << 16,
                                                             w[2 * i + 1] & 0xFFFF0000u));
}

// One thread: 16 channels of a token pair, K and V (the writing kernel's mapping).
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
                const uint32_t s2 = scale_pair(sb[e] * 0x00010001u);
                decode<BITS>(w[e], s2, offset_pair<BITS>(s2), out);
                if (live[e]) store16<T>(static_cast<T*>(a.k) + row + 64 * e, out);
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
            const uint32_t s2 = scale_pair((sb & 0xFFu) | (sb & 0xFF00u) << 8), c2 = offset_pair<BITS>(s2);
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
            if (live[0]) store16<T>(static_cast<T*>(a.v) + row, even);
            if (live[1]) store16<T>(static_cast<T*>(a.v) + row + 64, odd);
        }
    }
}

}  // namespace kv
