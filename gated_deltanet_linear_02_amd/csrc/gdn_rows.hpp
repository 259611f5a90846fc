// gdn_rows.hpp -- state rows spread over the lanes of a wave: the kernels that
// step or stream whole states (gdn_decode.hip, gdn_linattn.hip) share these.
#pragma once

#include "gdn_device.hpp"

namespace gdn {

template <typename E> __device__ __forceinline__ void load4(const E *p, float *dst);
template <> __device__ __forceinline__ void load4<float>(const float *p, float *dst) {
    const f32x4 x = *reinterpret_cast<const f32x4 *>(p);
    dst[0] = x[0]; dst[1] = x[1]; dst[2] = x[2]; dst[3] = x[3];
}
template <> __device__ __forceinline__ void load4<bf16>(const bf16 *p, float *dst) {
    const bf16x4 x = *reinterpret_cast<const bf16x4 *>(p);
    dst[0] = static_cast<float>(x[0]); dst[1] = static_cast<float>(x[1]);
    dst[2] = static_cast<float>(x[2]); dst[3] = static_cast<float>(x[3]);
}

// A lane's share of one state row: 8 elements, held as floats whatever the
// storage type SE. fp32 storage: two 16-byte pieces at columns 4 lr and
// 4 lr + 4 LPR, so that the LPR lanes of a row read 16 LPR contiguous bytes
// per load; bf16 storage: one 16-byte piece at columns 8 lr .. 8 lr + 7.
// Element j of the lane sits at column col(lr, j); columns 4m .. 4m + 3 of
// the lane are consecutive in both layouts. States are read and written
// once per step, so the stores are nontemporal, and so are the fp32 loads;
// bf16 rows load faster with the default policy (see kDecodeThreads).
template <typename SE, int LPR> struct StateLane;
template <int LPR> struct StateLane<float, LPR> {
    static __device__ __forceinline__ int col(int lr, int j) { return 4 * lr + 4 * LPR * (j >> 2) + (j & 3); }
    static __device__ __forceinline__ void load(const float *row, int lr, float (&s)[8]) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(row + col(lr, 4 * m)));
#pragma unroll
            for (int e = 0; e < 4; ++e) s[4 * m + e] = x[e];
        }
    }
    static __device__ __forceinline__ void store(float *row, int lr, const float (&w)[8]) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const f32x4 x = {w[4 * m], w[4 * m + 1], w[4 * m + 2], w[4 * m + 3]};
            __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(row + col(lr, 4 * m)));
        }
    }
};
template <int LPR> struct StateLane<bf16, LPR> {
    static __device__ __forceinline__ int col(int lr, int j) { return 8 * lr + j; }
    static __device__ __forceinline__ void load(const bf16 *row, int lr, float (&s)[8]) {
        const bf16x8 x = *reinterpret_cast<const bf16x8 *>(row + 8 * lr);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = static_cast<float>(x[j]);
    }
    static __device__ __forceinline__ void store(bf16 *row, int lr, const float (&w)[8]) {
        bf16x8 x;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = static_cast<bf16>(w[j]);  // round to nearest even
        __builtin_nontemporal_store(x, reinterpret_cast<bf16x8 *>(row + 8 * lr));
    }
};

// Sum of x over the LPR consecutive lanes of a row (LPR = 2, 4, 8 or 16; rows
// aligned to LPR), on DPP lane moves (no trip through the LDS crossbar, as
// a shuffle takes). Each step adds the value of a partner lane from a group
// whose lanes all hold the same partial sum: quads by xor 1 and xor 2, then
// half-rows by mirroring within 8 lanes, then rows by mirroring within 16.
template <int Ctrl> __device__ __forceinline__ float dpp_mov(float y) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, y), Ctrl, 0xf, 0xf, false));
}
template <int LPR> __device__ __forceinline__ float row_sum(float x) {
    static_assert(LPR == 2 || LPR == 4 || LPR == 8 || LPR == 16, "row width");
    x += dpp_mov<0xB1>(x);                         // quad_perm [1, 0, 3, 2]: lane ^ 1
    if constexpr (LPR >= 4) x += dpp_mov<0x4E>(x);   // quad_perm [2, 3, 0, 1]: lane ^ 2
    if constexpr (LPR >= 8) x += dpp_mov<0x141>(x);  // row_half_mirror: lane i <- 7 - i
    if constexpr (LPR >= 16) x += dpp_mov<0x140>(x); // row_mirror: lane i <- 15 - i
    return x;
}

}  // namespace gdn
