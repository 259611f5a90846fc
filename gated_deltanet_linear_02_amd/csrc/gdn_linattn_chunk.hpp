// gdn_linattn_chunk.hpp -- linear attention with a decay per head, chunk by
// chunk (gfx950).
//
// A chunk of C tokens starts from the state S0 (dv x dk). With c_t the sum of
// the gates from the chunk's first token to t, gamma_t = exp(c_t) and
// delta_t = exp(c_C - c_t):
//     o_i = scale ( gamma_i S0 q_i + sum_{j <= i} exp(c_i - c_j) (q_i . k_j) v_j )
//     S  <- gamma_C S0 + sum_t (delta_t v_t) k_t^T
// All sums are matrix products. Sums of gates are kept in fp64 (in units of
// log 2) and every factor is formed from a difference of them, so that a decay
// to nothing inside the chunk costs its neighbours no accuracy.
//
// A workgroup owns one (sequence or segment, value head) state for its whole
// run: the fp32 state stays in the accumulators of its waves, S^T in 16 x 16
// tiles (rows over dk), each wave holding all dk of 16 NT dv columns (NT = 2 for
// 128 rows, so that a fragment of q or k feeds two products). An accumulator
// tile is an operand of the next product as it stands, so the state never leaves
// the registers:
//     O^T[dv][i]  = S0 Q^T          state tiles (bf16) x Q rows from LDS
//                 + V^T P^T         V columns x the scores P from LDS
//     S^T[dk][dv] += K^T (delta V)  K columns from LDS x V columns
// Columns (operands that run over tokens) are read from row-major LDS with the
// transposing LDS read.
//
// With bf16 I/O the products are bf16 MFMAs with fp32 sums. Rounded on the way
// are the operand copy of S0 and the scores P, each once to bf16, as the output
// itself is. The state is fp32 and must not lose what it sums over
// thousands of tokens: delta_t v_t is split in three bf16 parts that hold all
// its 24 bits, and their products with k_t (bf16 already) are exact.
//
// What bounds it. A chunk of a 128 x 128 state is 64 KB of q, k, v and out
// and 8.4 MFLOP of products (outputs), so that a long call is bound by
// memory: 8 sequences of 62,064 tokens, 32 heads, move 2.15 GB in the output
// pass in 408 us (5.3 TB/s, some of it from the last-level cache; a large copy
// reaches 4.95) and 1.04 GB in the state pass in 209 us. A short call is bound by the chain of chunks, 3.1 us each (two
// workgroups on a compute unit 5.1 us each) and by two launches: 4,096 tokens
// take 20 + 36 us, 29 us of memory. Chunks of 64: with 32 a step took as long
// and did half as much. Four waves, two workgroups on a compute unit: eight waves
// in two roles, products and staging, were slower.
#pragma once

#include <type_traits>

#include "gdn_device.hpp"
#include "gdn_linattn.hpp"

// Keeps LDS reads of one phase out of the phase before it, where they would
// hold registers that the kernel does not have.
#define GDN_SCHED_BARRIER() __builtin_amdgcn_sched_barrier(0)

namespace gdn {

// ------------------------------------------------------------- operands

// A contraction of length K: bf16 MFMAs 32 (or, for K = 16, 16) deep, or fp32,
// where four 4-deep MFMAs make one 16-deep step. A lane (m = lane % 16, g =
// lane / 16) holds the KPL contraction indices of acc_k: 4 g .. 4 g + 3 of
// each 16.
template <typename E, int K> struct LinOp;
template <int K> struct LinOp<bf16, K> : Mma<bf16, K> {};
template <int K> struct LinOp<float, K> {
    static constexpr int KW = 16, KPL = 4;
    typedef f32x4 Frag;
    static __device__ __forceinline__ f32x4 mma(Frag a, Frag b, f32x4 c) {
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
        return c;
    }
};

// Where index k (a multiple of 4) of a contraction over tokens stands in an LDS
// row, so that a lane's KPL indices are contiguous.
template <typename OP> __device__ __forceinline__ constexpr int frag_pos(int k) {
    if constexpr (OP::KPL == 8) return (k & ~31) | ((k & 12) << 1) | ((k & 16) >> 2);
    else return k;
}
// Contractions over dk take their indices in natural order: lane group g has
// KPL side by side. So that state tiles are operands of it as they stand,
// rows 4 g + r of tiles 2 b and 2 b + 1 are (KPL = 8) dk 32 b + 8 g + r and
// 32 b + 8 g + 4 + r; with KPL = 4 tile t is dk 16 t .. 16 t + 15.
template <typename OP> __device__ __forceinline__ constexpr int tile_base(int t) {
    return OP::KPL == 8 ? 32 * (t >> 1) + 4 * (t & 1) : 16 * t;
}
// Fragment kb of row (r0 + lane % 16).
template <typename OP, typename E>
__device__ __forceinline__ typename OP::Frag row_frag(const E *base, int ld, int r0, int kb, int lane) {
    return *reinterpret_cast<const typename OP::Frag *>(base + (r0 + (lane & 15)) * ld + kb * OP::KW +
                                                        OP::KPL * (lane >> 4));
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 LdsQuad;

// Four tokens of one column. Lane (m, g) gets rows t0 + 4 g .. + 3 of column
// col(m), where col(m) = c0 + stride (m / 4) + m % 4 and `stride` is the
// distance of the column groups: 4 (16 columns side by side) or 8.
// bf16: the transposing read takes, from each 16 lanes, four rows of four
// 8-byte pieces (lane i: row i / 4, piece i % 4) and hands lane i column i.
template <typename E>
__device__ __forceinline__ auto col_quad(const E *base, int ld, int t0, int c0, int stride, int lane) {
    const int m = lane & 15, g = lane >> 4;
    if constexpr (std::is_same<E, bf16>::value) {
        const E *p = base + (t0 + 4 * g + (m >> 2)) * ld + c0 + stride * (m & 3);
        return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsQuad *)p));
    } else {
        const E *p = base + (t0 + 4 * g) * ld + c0 + stride * (m >> 2) + (m & 3);
        return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]};
    }
}
// Fragment kb of a contraction over tokens, for 16 columns.
template <typename OP, typename E>
__device__ __forceinline__ typename OP::Frag col_frag(const E *base, int ld, int kb, int c0, int stride, int lane) {
    if constexpr (OP::KPL == 8) {
        const bf16x4 lo = col_quad(base, ld, kb * 32, c0, stride, lane),
                     hi = col_quad(base, ld, kb * 32 + 16, c0, stride, lane);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
        return col_quad(base, ld, kb * 16, c0, stride, lane);
    }
}
// Fragment kb of a contraction over the rows of accumulator tiles t[16-row tile].
template <typename OP, typename E> __device__ __forceinline__ typename OP::Frag acc_frag(const f32x4 *t, int kb) {
    if constexpr (std::is_same<E, float>::value) {
        return t[kb];
    } else {
        typename OP::Frag f;
#pragma unroll
        for (int e = 0; e < OP::KPL; ++e) f[e] = static_cast<bf16>(t[kb * (OP::KPL / 4) + e / 4][e & 3]);
        return f;
    }
}

// ------------------------------------------------------------- work split

// The work of one launch. Unsplit (seg_shift < 0): item i is sequence i.
// Otherwise sequences are cut into segments of L = 2^seg_shift tokens; sequence
// n's segments are items floor(start_n / L) + n and following (start_n its
// first token), which leaves room for all of them whatever the lengths,
// needs no table, and is less than floor(T / L) + N in all.
struct LinWork {
    const int32_t *cu;
    bool sorted;         // cu is in order already (kLinListed)
    int32_t num_seqs, total_tokens, seg_shift;
    uint32_t hk, group;  // query/key heads, value heads on each
    uint32_t units;      // items x hk
};
struct LinItem {
    int seq, seg;  // seg: which segment of the sequence
    int segs;      // how many it has (an empty sequence has one, empty)
    int lo, hi;    // the item's tokens
    bool none;
};

// Moves across the wave on DPP; lanes that have no source keep x.
template <int Ctrl, int RowMask> __device__ __forceinline__ int dpp_keep(int x) {
    return __builtin_amdgcn_update_dpp(x, x, Ctrl, RowMask, 0xf, false);
}
// Running maximum over the lanes: within rows of 16, then rows 1 and 3 take
// row 0's and 2's last, then lanes 32 .. 63 lane 31's.
__device__ __forceinline__ int wave_scan_max(int x) {
    x = max(x, dpp_keep<0x111, 0xf>(x));  // row_shr 1
    x = max(x, dpp_keep<0x112, 0xf>(x));
    x = max(x, dpp_keep<0x114, 0xf>(x));
    x = max(x, dpp_keep<0x118, 0xf>(x));
    x = max(x, dpp_keep<0x142, 0xa>(x));  // row_bcast 15
    x = max(x, dpp_keep<0x143, 0xc>(x));  // row_bcast 31
    return x;
}

// The sequence of an item where the offsets are in order: the last n whose
// first item, floor(start / L) + n, is not behind it. 64 candidates at a time.
__device__ __forceinline__ int lin_search(const LinWork &w, int item, int lane) {
    if (w.seg_shift < 0) return item;
    int from = 0, len = w.num_seqs;
    for (;;) {
        const int step = (len + 63) >> 6, n = from + lane * step;
        const uint64_t at = __ballot(lane * step < len && (w.cu[min(n, w.num_seqs)] >> w.seg_shift) + n <= item);
        if (!at) return -1;  // (in the first turn only)
        const int l = 63 - __builtin_clzll(at);
        from += l * step;
        len = min(step, len - l * step);
        if (step == 1) return from;
    }
}

// Each wave finds its workgroup's item. Offsets are clamped into [0, T] and
// made non-decreasing (a running maximum), 64 sequences at a time; many
// sequences have it done before (gdn_linattn_offsets_kernel).
__device__ __forceinline__ LinItem lin_item(const LinWork &w, int item, int lane) {
    auto clampT = [&](int x) { return min(max(x, 0), w.total_tokens); };
    int carry = clampT(w.cu[0]);  // where sequence `base` starts
    int lo = 0, hi = 0, seq = -1;
    if (w.sorted) {
        seq = __builtin_amdgcn_readfirstlane(lin_search(w, item, lane));
        lo = w.cu[max(seq, 0)];
        hi = w.cu[max(seq, 0) + 1];
    } else for (int base = 0; base < w.num_seqs; base += 64) {
        const int n = base + lane;
        int e = n < w.num_seqs ? clampT(w.cu[n + 1]) : 0;
        e = wave_scan_max(max(e, carry));        // where sequence n ends
        // and starts (the move stands alone: every lane has to take part in it)
        const int before = __builtin_amdgcn_update_dpp(carry, e, 0x138, 0xf, 0xf, false);  // wave_shr 1
        const int s = lane == 0 ? carry : before;
        const int first = w.seg_shift < 0 ? n : (s >> w.seg_shift) + n;
        const uint64_t at = __ballot(n < w.num_seqs && first <= item);
        if (at) {
            const int l = 63 - __builtin_clzll(at);
            seq = base + l;
            lo = __builtin_amdgcn_readlane(s, l);
            hi = __builtin_amdgcn_readlane(e, l);
        }
        carry = __builtin_amdgcn_readlane(e, 63);
        if (at != ~0ull) break;
    }
    LinItem r;
    r.seq = seq;
    r.none = seq < 0;
    r.seg = 0;
    r.segs = 1;
    r.lo = lo;
    r.hi = hi;
    if (w.seg_shift >= 0) {
        const int len = hi - lo, L = 1 << w.seg_shift;
        r.seg = item - ((lo >> w.seg_shift) + seq);
        r.segs = max(1, (int)(((uint32_t)len + (uint32_t)L - 1u) >> w.seg_shift));
        r.none = r.none || r.seg >= r.segs;
        const int off = r.none ? 0 : r.seg << w.seg_shift;
        r.lo = lo + off;
        r.hi = lo + off + min(len - off, L);
    }
    return r;
}

// Workgroups go to the XCDs in turn. The heads that share a key head's
// items sit eight apart, on one XCD, whose L2 then reads their q and k once.
__device__ __forceinline__ bool lin_place(const LinWork &w, uint32_t &item, uint32_t &kh, uint32_t &h) {
    const uint32_t x = blockIdx.x & 7, m = blockIdx.x >> 3;
    const uint32_t r = m / w.group, u = x + 8 * r;
    item = u / w.hk;
    kh = u - item * w.hk;
    h = kh * w.group + (m - r * w.group);
    return u < w.units;
}
inline int64_t lin_grid(int64_t units, int64_t group) { return (units + 7) / 8 * 8 * group; }

// Offsets in order for calls of more sequences than kLinListed, where each
// workgroup would read many. One workgroup, a chain of turns of 4,096 sequences:
// 4 us for the first, 38 us for 65,536.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void gdn_linattn_offsets_kernel(const int32_t *__restrict__ cu, int num_seqs,
                                                                      int total_tokens, int32_t *__restrict__ sorted)
{
    __shared__ int s_top[2][THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto clampT = [&](int x) { return min(max(x, 0), total_tokens); };
    int carry = clampT(cu[0]), turn = 0;
    if (tid == 0) sorted[0] = carry;
    for (int base = 0; base < num_seqs; base += 4 * THREADS, turn ^= 1) {
        const int n = base + 4 * tid;
        int e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = n + j < num_seqs ? clampT(cu[n + j + 1]) : 0;
#pragma unroll
        for (int j = 1; j < 4; ++j) e[j] = max(e[j], e[j - 1]);
        const int upto = wave_scan_max(e[3]);
        const int before = __builtin_amdgcn_update_dpp(0, upto, 0x138, 0xf, 0xf, false);  // wave_shr 1
        if (lane == 63) s_top[turn][wave] = upto;
        __syncthreads();
        int start = max(carry, lane == 0 ? 0 : before);
        for (int i = 0; i < THREADS / 64; ++i) {
            const int top = s_top[turn][i];
            if (i < wave) start = max(start, top);
            carry = max(carry, top);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n + j < num_seqs) sorted[n + j + 1] = max(e[j], start);
    }
}

// ------------------------------------------------------------- the kernel

struct LinIo {
    const void *q, *k, *v, *g;
    int64_t gate_ld;     // elements of g from a token to the next
    int32_t gate_shift;  // value head h of the launch has gate h >> gate_shift
    const void *s0;
    void *s_final;
    void *out;
    float *seg_state;  // [item][hv] states of segments, accumulator order
    float *seg_decay;  // [item][hv]
    float scale;
    bool gate_bf16, state_bf16;
    bool joined;  // the join kernel has run: seg_state holds the states at the ends of the segments
};

template <typename E, int DK, int DV> struct LinShape {
    static constexpr int C = std::is_same<E, bf16>::value ? 64 : 32;  // tokens per chunk
    static constexpr int NW = DV >= 64 ? 4 : DV / 16, THREADS = 64 * NW;
    static constexpr int NT = DV / 16 / NW;                           // 16-column tiles of dv per wave
    static constexpr int WPS = NW == 4 ? 2 : 1;                       // waves per SIMD to fit
    static constexpr int MT = DK / 16;                                // 16-row tiles of dk
    typedef LinOp<E, DK> OK;                                          // contractions over dk
    typedef LinOp<E, C> OT;                                           // contractions over tokens
    static constexpr int KB = DK / OK::KW, TB = C / OT::KW;           // steps of each
    // LDS rows, elements. With rows 32 bytes off a multiple of 256 fragment
    // reads (16 bytes from each of 16 rows) and transposing reads (32 bytes
    // from each of 16) are free of bank conflicts: 213 and 167 bytes a clock,
    // 120 and 123 with rows 16 bytes off.
    static constexpr int PAD = 32 / (int)sizeof(E);
    static constexpr int LDK = DK + PAD, LDV = DV + PAD, LDP = C + PAD;
};

// A chunk's rows of one head in global memory, as a buffer: rows from `rows`
// on lie past its end, so that they read as zeros and are not written, by the
// hardware's range check. Row distances fit 32 bits (64 rows of at most 2^22
// elements, checked on the host).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const void *first, uint32_t row_bytes, int rows,
                                                             uint32_t used_bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(first), 0,
                                             (int)((uint32_t)(rows - 1) * row_bytes + used_bytes), 0x00027000);
}

// Rows of a chunk between global memory, registers and LDS, 16-byte pieces:
// thread tid takes the same piece of every STEP-th row.
template <typename E, int D, int C, int THREADS> struct LinStage {
    static constexpr int PIECE = 16 / (int)sizeof(E), PPR = D / PIECE, STEP = THREADS / PPR, N = C > STEP ? C / STEP : 1;
    static_assert(THREADS % PPR == 0 && (C % STEP == 0 || STEP > C), "whole rows per step");
    u32x4 r[N];
    __device__ __forceinline__ void load(const E *first, uint32_t row_bytes, int rows, int tid) {
        const __amdgpu_buffer_rsrc_t rsrc = chunk_rows(first, row_bytes, min(rows, C), D * (uint32_t)sizeof(E));
        asm volatile("" : "+v"(tid));  // addresses formed here, not kept in registers over the loop
        const uint32_t at = (uint32_t)(tid / PPR) * row_bytes + (uint32_t)(tid % PPR) * 16u;
#pragma unroll
        for (int i = 0; i < N; ++i)
            r[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)(at + (uint32_t)(i * STEP) * row_bytes), 0, 0);
    }
    __device__ __forceinline__ void store(E *dst, int ld, int tid) {
        asm volatile("" : "+v"(tid));
        const int row = tid / PPR;
        if (STEP > C && row >= C) return;
        E *d = dst + row * ld + tid % PPR * PIECE;
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(d + i * STEP * ld) = r[i];
    }
};

// Inclusive sums over the wave's lanes on DPP moves: within rows of 16, then
// rows 1 and 3 take row 0's and 2's last, then lanes 32 .. 63 lane 31's.
template <int Ctrl, int RowMask> __device__ __forceinline__ double dpp_add_f64(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, Ctrl, RowMask, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), Ctrl, RowMask, 0xf, false);
    return x + __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}
__device__ __forceinline__ double wave_scan_f64(double x) {
    x = dpp_add_f64<0x111, 0xf>(x);  // row_shr 1
    x = dpp_add_f64<0x112, 0xf>(x);
    x = dpp_add_f64<0x114, 0xf>(x);
    x = dpp_add_f64<0x118, 0xf>(x);
    x = dpp_add_f64<0x142, 0xa>(x);  // row_bcast 15
    x = dpp_add_f64<0x143, 0xc>(x);  // row_bcast 31
    return x;
}
__device__ __forceinline__ double lane_f64(double x, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)lo | (uint64_t)hi << 32);
}

__device__ __forceinline__ float gate_value(uint32_t bits, bool is_bf16) {
    return __builtin_bit_cast(float, is_bf16 ? bits << 16 : bits);
}
// A gate in units of log 2, at least -1024: exp of anything lower is 0 in fp32
// as well, and a difference of two sums stays a number after exp(g) = 0.
__device__ __forceinline__ double gate_log2(float g) { return fmax((double)g * 1.4426950408889634, -1024.0); }

// Two numbers as sums of N bf16 pairs, largest first.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int N> struct SplitPair { bf16x2 part[N]; };
template <int N> __device__ __forceinline__ SplitPair<N> split_pair(float a, float b) {
    SplitPair<N> s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s.part[i] = __builtin_convertvector((f32x2){a, b}, bf16x2);
        const uint32_t w = __builtin_bit_cast(uint32_t, s.part[i]);
        a -= __builtin_bit_cast(float, w << 16);
        b -= __builtin_bit_cast(float, w & 0xffff0000u);
    }
    return s;
}

// What a launch computes. kLinWhole: outputs and final states of whole
// sequences. Split: kLinSegState, the state at the end of each segment as if
// it began from zero (the first one from the initial state), and its decay;
// then kLinSegOut, the outputs from the states before each segment (joined by
// the kernel below, or summed by each workgroup), and the final states. The state
// that kLinSegOut carries from chunk to chunk only goes into outputs, so two parts
// of delta v, 16 bits, are enough there.
enum LinMode { kLinWhole, kLinSegState, kLinSegOut };

// A chunk goes in two steps with a barrier after each, each with as much
// independent work as there is, for the waves of a CU wait on latencies far
// more than on any unit:
//   1. scores of the wave's tiles, to LDS; S0 q; the new state
//   2. P v and the stores; the next chunk, on its way since step 1, to LDS
// (step 2 reads the scores only: v's columns are in registers by then).
template <typename E, int DK, int DV, LinMode kMode>
__global__ __launch_bounds__((LinShape<E, DK, DV>::THREADS), (LinShape<E, DK, DV>::WPS)) void gdn_linattn_chunk_kernel(
    LinWork w, LinIo io)
{
    typedef LinShape<E, DK, DV> SH;
    typedef typename SH::OK OK;
    typedef typename SH::OT OT;
    constexpr int C = SH::C, TT = C / 16, MT = SH::MT, KB = SH::KB, TB = SH::TB, THREADS = SH::THREADS, NW = SH::NW,
                  NT = SH::NT, LDK = SH::LDK, LDV = SH::LDV, LDP = SH::LDP;
    constexpr bool kBf16 = std::is_same<E, bf16>::value;
    constexpr bool kOut = kMode != kLinSegState;
    constexpr int kParts = !kBf16 ? 1 : kMode == kLinSegOut ? 2 : 3;  // parts of delta v
    constexpr int kColStride = OK::KPL == 8 ? 8 : 4;                  // of k's columns in a tile, see tile_base

    __shared__ __attribute__((aligned(16))) E s_q[kOut ? C * LDK : 8];
    __shared__ __attribute__((aligned(16))) E s_k[C * LDK];
    __shared__ __attribute__((aligned(16))) E s_v[C * LDV];
    __shared__ __attribute__((aligned(16))) E s_p[kOut ? C * LDP : 8];
    __shared__ __attribute__((aligned(16))) float s_chi[C], s_clo[C], s_gamma[C], s_delta[C];
    __shared__ float s_total;

    const int tid = threadIdx.x, lane0 = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = lane0, m = lane & 15, g = lane >> 4;

    uint32_t item, kh, h;
    if (!lin_place(w, item, kh, h)) return;
    const LinItem it = lin_item(w, (int)item, lane);
    if (it.none) return;
    const int hv = (int)(w.hk * w.group);

    const E *q = (const E *)io.q + (size_t)kh * DK, *k = (const E *)io.k + (size_t)kh * DK,
            *v = (const E *)io.v + (size_t)h * DV;
    const size_t ldk = (size_t)w.hk * DK, ldv = (size_t)hv * DV;
    LinStage<E, DK, C, THREADS> rq, rk;
    LinStage<E, DV, C, THREADS> rv;
    const uint32_t k_bytes = (uint32_t)(ldk * sizeof(E)), v_bytes = (uint32_t)(ldv * sizeof(E));
    uint32_t rg = 0;  // the gate's bits: converting them here would wait for the load
    auto load_q = [&](int t0) {
        if constexpr (kOut) rq.load(q + (size_t)t0 * ldk, k_bytes, it.hi - t0, tid);
    };
    auto load_k = [&](int t0) { rk.load(k + (size_t)t0 * ldk, k_bytes, it.hi - t0, tid); };
    auto load_v = [&](int t0) {
        rv.load(v + (size_t)t0 * ldv, v_bytes, it.hi - t0, tid);
        if (wave == NW - 1) {
            const int rows = min(it.hi - t0, C);
            const size_t ga = (size_t)(t0 + min(lane, rows - 1)) * io.gate_ld + (h >> io.gate_shift);
            rg = io.gate_bf16 ? ((const uint16_t *)io.g)[ga] : ((const uint32_t *)io.g)[ga];
        }
    };
    double decay = 0.0;  // of the chunks staged so far, log 2 (last wave)
    auto stage = [&](int t0) {
        const int rows = min(it.hi - t0, C);
        if (wave == NW - 1) {
            const double c = wave_scan_f64(lane < rows ? gate_log2(gate_value(rg, io.gate_bf16)) : 0.0);
            const double total = lane_f64(c, C - 1);
            if (lane < C) {
                if constexpr (kOut) {
                    const float hi = (float)c;
                    s_chi[lane] = hi;
                    s_clo[lane] = (float)(c - (double)hi);
                    s_gamma[lane] = io.scale * __builtin_amdgcn_exp2f((float)c);
                    s_delta[lane] = __builtin_amdgcn_exp2f((float)(total - c));
                } else {
                    s_delta[lane] = __builtin_amdgcn_exp2f((float)(decay + (total - c)));
                }
            }
            if (kOut && lane == 0) s_total = __builtin_amdgcn_exp2f((float)total);
            decay += total;
        }
        if constexpr (kOut) rq.store(s_q, LDK, tid);
        rk.store(s_k, LDK, tid);
        rv.store(s_v, LDV, tid);
    };
    // kLinSegState needs no state on its way, only the one at the end: it goes
    // from the last chunk to the first, so that every token's decay to the end of
    // the segment is known when the token comes, and the sum is never scaled.
    constexpr int step = kOut ? C : -C;
    const int first = kOut ? it.lo : it.lo + ((it.hi - it.lo + C - 1) / C - 1) * C;
    // The first chunk's loads go out before the state's: they are waited for first.
    if (it.lo < it.hi) {
        load_q(first);
        load_k(first);
        load_v(first);
    }

    // This lane's part of the state: tile (mt, nt) holds dk dk_of(mt) .. + 3 of
    // column dv_of(nt). Two tiles' columns alternate in fours, so that a
    // lane's outputs of one token are 4 NT consecutive dv.
    constexpr int kTiles = MT * NT, kVStride = 4 * NT;
    const int dv0 = 16 * NT * wave;
    auto dk_of = [&](int t) { return tile_base<OK>(t / NT) + OK::KPL * g; };
    auto dv_of = [&](int t) { return dv0 + kVStride * (m >> 2) + 4 * (t % NT) + (m & 3); };
    f32x4 S[kTiles];
    const size_t state_at = ((size_t)it.seq * hv + h) * (DK * DV);
    auto load_initial = [&](int t) {
        const size_t at = state_at + (size_t)dv_of(t) * DK + dk_of(t);
        return io.state_bf16 ? load4f<bf16>((const bf16 *)io.s0 + at) : load4f<float>((const float *)io.s0 + at);
    };
    const size_t seg_at = ((size_t)item * hv + h) * (DK * DV) + tid * 4;
    // The state at the end of segment seg + n - 1, from the states of the
    // segments (not joined: a chain over all of them).
    auto load_segments = [&](int n) {
        const size_t ld = (size_t)hv * (DK * DV);
        const float *src = io.seg_state + seg_at + (ptrdiff_t)(io.joined ? n - 1 : -it.seg) * (ptrdiff_t)ld;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) S[t] = *reinterpret_cast<const f32x4 *>(src + t * THREADS * 4);
        if (io.joined) return;
        const float *dec = io.seg_decay + (size_t)item * hv + h - (ptrdiff_t)it.seg * hv;
        // (four segments' loads at once, where there are registers for them)
#pragma clang loop unroll_count(NT == 1 ? 4 : 1)
        for (int s = 1; s < it.seg + n; ++s) {
            src += ld;
            dec += hv;
            const float d = *dec;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(src + t * THREADS * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][e] = __builtin_fmaf(d, S[t][e], x[e]);
            }
        }
    };
    if (kMode == kLinSegOut && it.seg > 0) {
        load_segments(0);
    } else if (kOut && io.s0 && it.seg == 0) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) S[t] = load_initial(t);
    } else {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    if (it.lo < it.hi) stage(first);
    for (int t0 = first; kOut ? t0 < it.hi : t0 >= it.lo; t0 += step) {
        const bool more = kOut ? t0 + C < it.hi : t0 > it.lo;
        // The next chunk's loads are spread over the step, so that no wave
        // stands in the way of its own products with all of them at once.
        if (!kOut && more) {
            load_k(t0 + step);
            load_v(t0 + step);
        }
        __syncthreads();
        if (kOut && more) load_q(t0 + step);

        // ---- step 1
        int lane_ = lane0;
        asm volatile("" : "+v"(lane_));
        const int lane = lane_, m = lane & 15, g = lane >> 4, g4 = 4 * g;
        typename OT::Frag fv[TB * NT];
#pragma unroll
        for (int t = 0; t < TB * NT; ++t)
            fv[t] = col_frag<OT>(s_v, LDV, t / NT, dv0 + 4 * (t % NT), kVStride, lane);

        f32x4 o[kOut ? TT * NT : 1];
        float gam[TT];  // of the tokens of this lane's output columns
        if constexpr (kOut) {
            // Scores P^T = K Q^T, tiles (tokens j, tokens i). A product's
            // contraction steps reach kStep tiles, past the diagonal too:
            // row I has the tiles of its last step, (I / kStep + 1) kStep,
            // those above the diagonal zero. Tile number u of the list
            // (0,0), .. goes to wave u % NW.
            constexpr int kStep = OT::KW / 16, kScores = TT * (TT + kStep) / 2, kMine = (kScores + NW - 1) / NW,
                          kSide = kMine < 3 ? kMine : 3;
#pragma unroll
            for (int r = 0; r < kMine; r += kSide) {
                f32x4 p[kSide];
                int I[kSide], J[kSide];
#pragma unroll
                for (int s = 0; s < kSide; ++s) {
                    // (a wave past the list's end repeats the last tile)
                    const int u = min((r + s) * NW + wave, kScores - 1);
                    if constexpr (kStep == 2) {  // rows of 2, 2, 4, 4 tiles
                        I[s] = u < 4 ? u >> 1 : 2 + ((u - 4) >> 2);
                        J[s] = u < 4 ? u & 1 : (u - 4) & 3;
                    } else {                     // rows of 1, 2 tiles
                        I[s] = u > 0;
                        J[s] = u >> 1;
                    }
                    p[s] = f32x4{0.f, 0.f, 0.f, 0.f};
                }
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int s = 0; s < kSide; ++s)
                        p[s] = OK::mma(row_frag<OK>(s_k, LDK, 16 * J[s], kb, lane),
                                       row_frag<OK>(s_q, LDK, 16 * I[s], kb, lane), p[s]);
#pragma unroll
                for (int s = 0; s < kSide; ++s) {
                    const int i = 16 * I[s] + m, j0 = 16 * J[s] + g4;
                    const float hi = s_chi[i], lo = s_clo[i];
                    const f32x4 jhi = *reinterpret_cast<const f32x4 *>(s_chi + j0),
                                jlo = *reinterpret_cast<const f32x4 *>(s_clo + j0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // (exp2 of -16384 is 0)
                        const float x = j0 + e <= i ? (hi - jhi[e]) + (lo - jlo[e]) : -16384.f;
                        p[s][e] *= io.scale * __builtin_amdgcn_exp2f(x);
                    }
                    store4<E>(s_p + i * LDP + frag_pos<OT>(j0), p[s]);
                }
            }
#pragma unroll
            for (int I = 0; I < TT; ++I) gam[I] = s_gamma[16 * I + m];
            GDN_SCHED_BARRIER();
        }
        if (kOut && more) load_k(t0 + step);
        // delta V of contraction step tb, for the state
        typename OT::Frag vd[2][NT][kParts];
        auto weigh = [&](int tb, typename OT::Frag (&x)[NT][kParts]) {
#pragma unroll
            for (int u = 0; u < OT::KPL / 4; ++u) {
                const f32x4 d = *reinterpret_cast<const f32x4 *>(s_delta + tb * OT::KW + 16 * u + g4);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float x0 = d[e] * to_f32(fv[tb * NT + nt][4 * u + e]),
                                    x1 = d[e + 1] * to_f32(fv[tb * NT + nt][4 * u + e + 1]);
                        if constexpr (kBf16) {
                            const SplitPair<kParts> s = split_pair<kParts>(x0, x1);
#pragma unroll
                            for (int i = 0; i < kParts; ++i) {
                                x[nt][i][4 * u + e] = s.part[i][0];
                                x[nt][i][4 * u + e + 1] = s.part[i][1];
                            }
                        } else {
                            x[nt][0][4 * u + e] = x0;
                            x[nt][0][4 * u + e + 1] = x1;
                        }
                    }
            }
        };
        const bool carry = kMode != kLinSegOut || more;
        if constexpr (kOut) {
            typename OK::Frag fs[NT * KB];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                f32x4 col[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) col[mt] = S[mt * NT + nt];
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) fs[nt * KB + kb] = acc_frag<OK, E>(col, kb);
            }
#pragma unroll
            for (int t = 0; t < TT * NT; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int I = 0; I < TT; ++I) {
                    const typename OK::Frag fq = row_frag<OK>(s_q, LDK, 16 * I, kb, lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) o[I * NT + nt] = OK::mma(fs[nt * KB + kb], fq, o[I * NT + nt]);
                }
        }
        weigh(0, vd[0]);
        if constexpr (kOut) {
            const float total = s_total;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) S[t] *= total;
        }
        GDN_SCHED_BARRIER();

        if (kOut && more) load_v(t0 + step);
        if (carry) {
            // S^T <- gamma_C S^T + K^T (delta V)
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                // Two tiles of dk at a time, so that a product does not follow
                // on the one it adds to.
                constexpr int kSide = MT < 2 ? 1 : 2;
#pragma unroll
                for (int mt = 0; mt < MT; mt += kSide) {
                    typename OT::Frag fk[kSide];
#pragma unroll
                    for (int s = 0; s < kSide; ++s)
                        fk[s] = col_frag<OT>(s_k, LDK, tb, tile_base<OK>(mt + s), kColStride, lane);
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int s = 0; s < kSide; ++s)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                S[(mt + s) * NT + nt] = OT::mma(fk[s], vd[tb & 1][nt][part], S[(mt + s) * NT + nt]);
                }
                if (tb + 1 < TB) weigh(tb + 1, vd[(tb + 1) & 1]);
                GDN_SCHED_BARRIER();
            }
        }
        __syncthreads();

        // ---- step 2
        if constexpr (kOut) {
            constexpr int kStep = OT::KW / 16;
#pragma unroll
            for (int I = 0; I < TT; ++I) {
                const float gamma = gam[I];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) o[I * NT + nt] *= gamma;
            }
#pragma unroll
            for (int b = 0; b < TB; ++b)
#pragma unroll
                for (int I = b * kStep; I < TT; ++I) {
                    const typename OT::Frag fp = row_frag<OT>(s_p, LDP, 16 * I, b, lane);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) o[I * NT + nt] = OT::mma(fv[b * NT + nt], fp, o[I * NT + nt]);
                }
        }
        GDN_SCHED_BARRIER();
        if (more) stage(t0 + step);
        GDN_SCHED_BARRIER();
        if constexpr (kOut) {
            const __amdgpu_buffer_rsrc_t rsrc = chunk_rows((E *)io.out + (size_t)t0 * ldv + (size_t)h * DV, v_bytes,
                                                           min(it.hi - t0, C), DV * (uint32_t)sizeof(E));
            const uint32_t at = (uint32_t)m * v_bytes + (uint32_t)((dv0 + kVStride * g) * (int)sizeof(E));
#pragma unroll
            for (int I = 0; I < TT; ++I) {
                const int off = (int)(at + (uint32_t)(16 * I) * v_bytes);
                if constexpr (kBf16) {
                    bf16x4 x[NT];
#pragma unroll
                    for (int e = 0; e < 4 * NT; ++e) x[e / 4][e & 3] = static_cast<bf16>(o[I * NT + e / 4][e & 3]);
                    if constexpr (NT == 2)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7)),
                            rsrc, off, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x[0]), rsrc, off, 0, 0);
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[I * NT + nt]), rsrc,
                                                               off + 16 * nt, 0, 0);
                }
            }
        }
    }

    if constexpr (kMode == kLinSegState) {
        if (io.s0 && it.seg == 0) {
            if (tid == THREADS - 64) s_total = __builtin_amdgcn_exp2f((float)decay);
            __syncthreads();
            const float total = s_total;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const f32x4 x = load_initial(t);
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][e] = __builtin_fmaf(total, x[e], S[t][e]);
            }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) *reinterpret_cast<f32x4 *>(io.seg_state + seg_at + t * THREADS * 4) = S[t];
        if (tid == THREADS - 64) io.seg_decay[(size_t)item * hv + h] = __builtin_amdgcn_exp2f((float)decay);
    } else if (io.s_final && it.seg == 0) {
        // Split: the state at the end of the last segment, stored by the
        // workgroup that has read the initial state, which may be the same
        // buffer.
        if constexpr (kMode == kLinSegOut) load_segments(it.segs);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            const size_t at = state_at + (size_t)dv_of(t) * DK + dk_of(t);
            if (io.state_bf16) store4<bf16>((bf16 *)io.s_final + at, S[t]);
            else store4<float>((float *)io.s_final + at, S[t]);
        }
    }
}

// Joins the segments of a sequence: each segment's state becomes the state at
// its end, S_s = decay_s S_{s-1} + local_s. One lane per four elements; the
// chain over segments is a multiply-add each, the loads run ahead of it. Bound by
// memory, the states read and written once: 34 segments of 32 heads of 128 x 128,
// 71 MB, take 22 us (6.5 TB/s, some of it from the last-level cache). Few states
// leave compute units idle; they go in workgroups of 64 lanes with more loads
// ahead: 63 segments of 4 heads 10.6 us with 256 and 8, 8.9 with 64 and 16; 118 of
// 2 heads of 64 x 64 13.9 and 11.1; but 16 of 32 heads 11.9 and 14.9.
template <int DK, int DV, int THREADS, int kAhead>
__global__ __launch_bounds__(THREADS) void gdn_linattn_join_kernel(LinWork w, LinIo io)
{
    constexpr int kQuads = DK * DV / 4, kBlocks = (kQuads + THREADS - 1) / THREADS;
    const int lane = threadIdx.x & 63;
    const int hv = (int)(w.hk * w.group);
    const int block = blockIdx.x % kBlocks, nh = blockIdx.x / kBlocks;
    const int n = nh / hv, h = nh - n * hv;
    // the sequence's bounds, as lin_item finds them
    auto clampT = [&](int x) { return min(max(x, 0), w.total_tokens); };
    int lo = clampT(w.cu[w.sorted ? n : 0]), hi = lo;
    for (int j = w.sorted ? n : lane; j <= n; j += 64) {
        const int e = clampT(w.cu[j + 1]);
        hi = max(hi, e);
        if (j < n) lo = max(lo, e);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        hi = max(hi, __shfl_xor(hi, off));
        lo = max(lo, __shfl_xor(lo, off));
    }
    const int segs = (int)(((uint32_t)(hi - lo) + (1u << w.seg_shift) - 1u) >> w.seg_shift);
    const int item0 = (lo >> w.seg_shift) + n;
    const int quad = block * THREADS + threadIdx.x;
    if (quad >= kQuads) return;
    float *at = io.seg_state + ((size_t)item0 * hv + h) * (DK * DV) + (size_t)quad * 4;
    const float *dec = io.seg_decay + (size_t)item0 * hv + h;
    const size_t ld = (size_t)hv * (DK * DV);
    f32x4 S = *reinterpret_cast<const f32x4 *>(at);
    for (int s0 = 1; s0 < segs; s0 += kAhead) {
        f32x4 x[kAhead];
        float d[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int s = min(s0 + u, segs - 1);
            x[u] = *reinterpret_cast<const f32x4 *>(at + s * ld);
            d[u] = dec[(size_t)s * hv];
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s0 + u >= segs) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) S[e] = __builtin_fmaf(d[u], S[e], x[u][e]);
            *reinterpret_cast<f32x4 *>(at + (s0 + u) * ld) = S;
        }
    }
}

}  // namespace gdn
