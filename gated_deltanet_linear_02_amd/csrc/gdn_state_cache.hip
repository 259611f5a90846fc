// gdn_state_cache.hip -- states kept in a cache at 8 bits (gfx950).
//
// A row x of dk values of a state is kept as codes c and one fp32 scale:
//     scale = max|x| / M,   c = x / scale rounded to the nearest code
//     (ties to even),       read back: c * scale
// with M = 127 (int8: the codes -127 .. 127) or 448 (e4m3, the largest value).
// A row that holds a NaN or an infinity gets the scale NaN and codes 0, so
// that it reads back as NaN; a row of zeros gets the scale 0.
//
// The codes are those of the exact quotient. A quotient rounded to fp32 first
// could land on the middle between two codes, and bf16 states have many exact
// ties. So it is rounded to odd: cut off towards zero, the last bit set if that
// lost anything. No middle between codes has that bit, so that rounding to a
// code from there gives what rounding the quotient itself gives. x - q s is
// exact in one fused multiply-add and tells whether q is the quotient, or past
// it. Rows of tiny values are lifted (exactly) by 2^64 first, so that reciprocal
// and remainder are ordinary numbers.
//
// Bound by memory: 4 bytes (2 for bf16 states) and 1 byte per value, each
// touched once. A lane takes one 16-byte piece of a state row and its 4 (8)
// codes, LPR = dk / EPL lanes a row, so that every load and store of a wave is
// contiguous; NR rows per lane group keep several loads in flight. 64 states of
// 32 heads, 128 x 128, int8 or e4m3: fp32 written in 31.4 us (5.4 TB/s), read back
// in 24.5 (6.9); bf16 22.5 (4.5) and 15.4 (6.6). NR = 1, 2, 4, 8: fp32 written in
// 34.3, 32.9, 31.4, 32.0, bf16 read in 18.9, 15.6, 15.4, 15.7. A write does some
// 19 operations a value beside its memory; deciding near-ties apart, with both
// neighbouring codes formed, took fp32 states 30.6 us and bf16 states 25.4.
#include "gdn_linattn.hpp"
#include "gdn_rows.hpp"

namespace gdn {

template <typename SE, int DK> struct CacheRows {
    static constexpr int EPL = 16 / (int)sizeof(SE);  // state elements per lane
    static constexpr int LPR = DK / EPL;              // lanes per row
    static constexpr int THREADS = 256;
    static constexpr int RPP = THREADS / LPR;         // rows per pass of the workgroup
    static constexpr int NR = 4;                      // passes
    static constexpr int ROWS = RPP * NR;
};

// Largest x over the LPR lanes of a row (2 .. 32).
template <int LPR> __device__ __forceinline__ uint32_t row_umax(uint32_t x) {
    auto step = [&](uint32_t y) { x = max(x, y); };
    step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xf, 0xf, false));                         // lane ^ 1
    if constexpr (LPR >= 4) step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xf, 0xf, false));   // lane ^ 2
    if constexpr (LPR >= 8) step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xf, 0xf, false));  // 7 - i of 8
    if constexpr (LPR >= 16) step((uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xf, 0xf, false)); // 15 - i of 16
    if constexpr (LPR >= 32) step((uint32_t)__shfl_xor((int)x, 16));
    return x;
}

// Where a workgroup's item lies in the state pool and in the cache (first row
// of each), and which of the item's workgroups it is; find() is false where
// the item names no slot or no entry.
struct CacheWhere {
    const int32_t *slots, *entries;
    int32_t num_slots, num_entries;
    int32_t rows;    // of one state: hv * dv
    int32_t blocks;  // workgroups per item
    __device__ __forceinline__ bool find(size_t &slot_row, size_t &entry_row, int &block) const {
        const int i = blockIdx.x / blocks;
        block = blockIdx.x - i * blocks;
        const int s = slots ? slots[i] : i, e = entries ? entries[i] : i;
        slot_row = (size_t)s * rows;
        entry_row = (size_t)e * rows;
        return s >= 0 && s < num_slots && e >= 0 && e < num_entries;
    }
};

constexpr float kInt8Top = 127.f, kE4m3Top = 448.f;

// x / s, rounded to odd; inv is 1 / s to a step or so.
__device__ __forceinline__ float quotient_odd(float x, float s, float inv) {
    const float t = x * inv;                                  // within three steps
    const float q = __builtin_fmaf(__builtin_fmaf(-t, s, x), inv, t);  // within one
    const float rest = __builtin_fmaf(-q, s, x);
    uint32_t b = __builtin_bit_cast(uint32_t, q);
    const uint32_t past = (__builtin_bit_cast(uint32_t, rest) ^ __builtin_bit_cast(uint32_t, x)) >> 31;
    b = rest == 0.f ? b : (b - past) | 1u;
    return __builtin_bit_cast(float, b);
}

// Four quotients to four code bytes, to nearest, ties to even. int8: adding
// 1.5 2^23 rounds to a whole number and leaves it in the low bits.
template <bool kE4m3> __device__ __forceinline__ uint32_t pack_codes(const float (&t)[4]) {
    if constexpr (kE4m3) {
        int w = 0;
        w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], w, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
        return (uint32_t)w;
    } else {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __builtin_bit_cast(uint32_t, t[e] + 12582912.f);
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0c);
        return lo | hi;
    }
}

template <bool kE4m3> __device__ __forceinline__ void unpack_codes(uint32_t w, float (&c)[4]) {
    if constexpr (kE4m3) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        c[0] = lo[0]; c[1] = lo[1]; c[2] = hi[0]; c[3] = hi[1];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = (float)(int8_t)(w >> (8 * e));
    }
}

template <typename SE, int DK, bool kE4m3>
__global__ __launch_bounds__(256) void gdn_state_cache_write_kernel(const SE *__restrict__ state,
                                                                    uint8_t *__restrict__ cache,
                                                                    float *__restrict__ scales, CacheWhere where)
{
    typedef CacheRows<SE, DK> SH;
    constexpr int EPL = SH::EPL, LPR = SH::LPR, NR = SH::NR;
    constexpr float kTop = kE4m3 ? kE4m3Top : kInt8Top;
    size_t from, to;
    int block;
    if (!where.find(from, to, block)) return;
    const int lr = threadIdx.x % LPR;
    const int r0 = block * SH::ROWS + threadIdx.x / LPR;

    float x[NR][EPL];
#pragma unroll
    for (int p = 0; p < NR; ++p) {
        const int r = min(r0 + p * SH::RPP, where.rows - 1);
        const SE *src = state + (from + r) * DK + EPL * lr;
        if constexpr (EPL == 4) {
            const f32x4 w = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(src));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[p][e] = w[e];
        } else {
            const bf16x8 w = __builtin_nontemporal_load(reinterpret_cast<const bf16x8 *>(src));
#pragma unroll
            for (int e = 0; e < 8; ++e) x[p][e] = static_cast<float>(w[e]);
        }
    }
#pragma unroll
    for (int p = 0; p < NR; ++p) {
        const int r = r0 + p * SH::RPP;
        uint32_t top = 0;  // bits of |x| order as the values do, NaN above infinity
#pragma unroll
        for (int e = 0; e < EPL; ++e) top = max(top, __builtin_bit_cast(uint32_t, x[p][e]) & 0x7fffffffu);
        top = row_umax<LPR>(top);
        const bool finite = top < 0x7f800000u;
        const float amax = __builtin_bit_cast(float, top);
        float scale = finite ? amax / kTop : __builtin_nanf("");
        // Rounded up, the scale of the largest values would read back as infinity.
        if (scale * kTop == __builtin_inff())
            scale = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, scale) - 1u);
        const bool some = finite && scale > 0.f;
        float s = scale;
        if (amax < 0x1p-60f) {
            s *= 0x1p64f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) x[p][e] *= 0x1p64f;
        }
        const float inv = some ? __builtin_amdgcn_rcpf(s) : 0.f;
        uint32_t w[EPL / 4];
#pragma unroll
        for (int m = 0; m < EPL / 4; ++m) {
            float t[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                // (a scale that underflowed may be too small for its row)
                t[e] = __builtin_amdgcn_fmed3f(quotient_odd(x[p][4 * m + e], s, inv), -kTop, kTop);
            w[m] = pack_codes<kE4m3>(t);
            if (!some) w[m] = 0;
        }
        if (r < where.rows) {
            uint8_t *dst = cache + (to + r) * DK + EPL * lr;
            if constexpr (EPL == 4) {
                *reinterpret_cast<uint32_t *>(dst) = w[0];
            } else {
                *reinterpret_cast<uint64_t *>(dst) = (uint64_t)w[0] | (uint64_t)w[1] << 32;
            }
            if (lr == 0) scales[to + r] = scale;
        }
    }
}

template <typename SE, int DK, bool kE4m3>
__global__ __launch_bounds__(256) void gdn_state_cache_read_kernel(const uint8_t *__restrict__ cache,
                                                                   const float *__restrict__ scales,
                                                                   SE *__restrict__ state, CacheWhere where)
{
    typedef CacheRows<SE, DK> SH;
    constexpr int EPL = SH::EPL, LPR = SH::LPR, NR = SH::NR;
    size_t to, from;
    int block;
    if (!where.find(to, from, block)) return;
    const int lr = threadIdx.x % LPR;
    const int r0 = block * SH::ROWS + threadIdx.x / LPR;
    uint32_t w[NR][EPL / 4];
    float s[NR];
#pragma unroll
    for (int p = 0; p < NR; ++p) {
        const int r = min(r0 + p * SH::RPP, where.rows - 1);
        const uint32_t *src = reinterpret_cast<const uint32_t *>(cache + (from + r) * DK + EPL * lr);
        if constexpr (EPL == 4) {
            w[p][0] = src[0];
        } else {
            const uint64_t d = *reinterpret_cast<const uint64_t *>(src);
            w[p][0] = (uint32_t)d;
            w[p][1] = (uint32_t)(d >> 32);
        }
        s[p] = scales[from + r];
    }
#pragma unroll
    for (int p = 0; p < NR; ++p) {
        const int r = r0 + p * SH::RPP;
        if (r >= where.rows) break;
        SE *dst = state + (to + r) * DK + EPL * lr;
        float c[4];
        if constexpr (EPL == 4) {
            unpack_codes<kE4m3>(w[p][0], c);
            const f32x4 x = {c[0] * s[p], c[1] * s[p], c[2] * s[p], c[3] * s[p]};
            __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(dst));
        } else {
            bf16x8 x;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                unpack_codes<kE4m3>(w[p][m], c);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * m + e] = static_cast<bf16>(c[e] * s[p]);
            }
            __builtin_nontemporal_store(x, reinterpret_cast<bf16x8 *>(dst));
        }
    }
}

// Calls f(SE, DK, e4m3) for the call's types and row length.
template <typename F> static hipError_t with_cache(const StateCacheArgs &A, F f) {
    auto sized = [&](auto se) {
        auto coded = [&](auto dk) {
            return A.e4m3 ? f(se, dk, std::true_type()) : f(se, dk, std::false_type());
        };
        switch (A.dk) {
        case 16: return coded(std::integral_constant<int, 16>());
        case 32: return coded(std::integral_constant<int, 32>());
        case 64: return coded(std::integral_constant<int, 64>());
        case 128: return coded(std::integral_constant<int, 128>());
        default: return hipErrorInvalidValue;
        }
    };
    return A.state_bf16 ? sized(bf16()) : sized(float());
}

static CacheWhere cache_where(const StateCacheArgs &A, int rows_per_block) {
    const int32_t rows = A.hv * A.dv;
    return CacheWhere{A.slots, A.entries, A.num_slots, A.num_entries, rows,
                      (rows + rows_per_block - 1) / rows_per_block};
}

hipError_t launch_state_cache_write(const StateCacheArgs &A, hipStream_t st) {
    return with_cache(A, [&](auto se, auto dk, auto e4m3) {
        typedef decltype(se) SE;
        typedef CacheRows<SE, dk()> SH;
        const CacheWhere where = cache_where(A, SH::ROWS);
        const dim3 grid((unsigned)where.blocks * (unsigned)A.n), block(SH::THREADS);
        return launch_kernel(kCacheWrite, gdn_state_cache_write_kernel<SE, dk(), e4m3()>, grid, block, 0, st,
                             (const SE *)A.state, (uint8_t *)A.cache, A.scales, where);
    });
}

hipError_t launch_state_cache_read(const StateCacheArgs &A, hipStream_t st) {
    return with_cache(A, [&](auto se, auto dk, auto e4m3) {
        typedef decltype(se) SE;
        typedef CacheRows<SE, dk()> SH;
        const CacheWhere where = cache_where(A, SH::ROWS);
        const dim3 grid((unsigned)where.blocks * (unsigned)A.n), block(SH::THREADS);
        return launch_kernel(kCacheRead, gdn_state_cache_read_kernel<SE, dk(), e4m3()>, grid, block, 0, st,
                             (const uint8_t *)A.cache, (const float *)A.scales, (SE *)A.state, where);
    });
}

}  // namespace gdn
