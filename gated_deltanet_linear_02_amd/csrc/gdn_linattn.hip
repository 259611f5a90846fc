// gdn_linattn.hip -- linear attention with a decay per head (gfx950): the
// decode step, and how a prefill is split and dispatched.
//
// Per (sequence, value head), with a = exp(g):
//     S <- a S + v k^T,   o = scale S q
// The delta rule without its correction: nothing of the old state is
// subtracted along k, so every row of S is scaled and added to, and the
// output of the new state is scale (a (S q) + v (k.q)) over the old one.
#include "gdn_linattn.hpp"

#include <cmath>

#include "gdn_rows.hpp"

namespace gdn {

// ---------------------------------------------------------------------------
// Decode: one token per sequence
// ---------------------------------------------------------------------------
//
// Bound by the bytes of the states, read once and written once (64 sequences
// at 32 heads, d = 128, fp32: 268 MB). Rows of a state are independent: a row
// is spread over LPR = DK / 8 lanes (StateLane), every lane group takes
// NRL rows of its workgroup, and q.S, k.q are summed over the lanes of a row
// by DPP moves. Loads and stores of fp32 states are nontemporal (nothing reads
// them again before the next step). 64 sequences, 32 heads, d = 128: fp32 states
// 42.7 us (6.3 TB/s), bf16 states 22.8 us (5.9 TB/s); one sequence 4.3 us.
// Threads and rows per lane group, same sizes: fp32 256 and 1 42.7 us, 1,024 and
// 2 44.0; bf16 256 and 1 26.9, 512 and 2 24.8, 1,024 and 2 22.8.
template <typename SE> constexpr int kLinDecodeThreads = 256;
template <> constexpr int kLinDecodeThreads<bf16> = 1024;
template <typename SE> constexpr int kLinDecodeRowsPerLane = 1;
template <> constexpr int kLinDecodeRowsPerLane<bf16> = 2;

template <typename SE, int DK, int DV> struct LinDecodeShape {
    static constexpr int LPR = DK / 8;  // lanes per state row
    static constexpr int TMAX = DV * LPR / kLinDecodeRowsPerLane<SE>;
    static constexpr int THREADS = kLinDecodeThreads<SE> < TMAX ? kLinDecodeThreads<SE> : (TMAX < 64 ? 64 : TMAX);
    static constexpr int RPP = THREADS / LPR;  // rows per pass of the workgroup
    static constexpr int NRL =
        RPP >= DV ? 1 : (kLinDecodeRowsPerLane<SE> < DV / RPP ? kLinDecodeRowsPerLane<SE> : DV / RPP);
    static constexpr int ROWS = RPP * NRL;  // rows per workgroup
    static constexpr int SLICES = (DV + ROWS - 1) / ROWS;
};

template <typename E, typename G, typename SE, int DK, int DV, bool kSlots>
__global__ __launch_bounds__((LinDecodeShape<SE, DK, DV>::THREADS)) void gdn_linattn_decode_kernel(
    const E *__restrict__ q, const E *__restrict__ k, const E *__restrict__ v, const G *__restrict__ gate_g,
    int32_t gate_ld,  // elements of g from one sequence to the next: hv, or 0 (one gate per head)
    const SE *state, SE *state_out,  // may be the same pool
    const int32_t *__restrict__ slots, int32_t num_slots, E *__restrict__ out, int32_t hk, int32_t hv, float scale)
{
    typedef LinDecodeShape<SE, DK, DV> SH;
    typedef StateLane<SE, SH::LPR> SL;
    constexpr int LPR = SH::LPR, RPP = SH::RPP, NRL = SH::NRL, ROWS = SH::ROWS, SLICES = SH::SLICES;

    const int bhs = blockIdx.x;
    const int bh = bhs / SLICES;
    const int row0 = (bhs - bh * SLICES) * ROWS;
    const int b = bh / hv;
    const int h = bh - b * hv;
    const int kh = h / (hv / hk);
    const int tid = threadIdx.x;
    const int lr = tid % LPR;
    const int r0 = row0 + tid / LPR;  // this lane group's rows: r0 + p RPP, p < NRL

    const int slot = kSlots ? slots[b] : b;
    E *o_row = out + ((size_t)b * hv + h) * DV;
    if (kSlots && (slot < 0 || slot >= num_slots)) {
#pragma unroll
        for (int p = 0; p < NRL; ++p)
            if (r0 + p * RPP < DV && lr == 0) o_row[r0 + p * RPP] = from_f32<E>(0.0f);
        return;
    }
    const size_t base = ((size_t)slot * hv + h) * (size_t)(DV * DK);

    float s[NRL][8];
#pragma unroll
    for (int p = 0; p < NRL; ++p) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[p][j] = 0.f;
        if (r0 + p * RPP < DV) SL::load(state + base + (size_t)(r0 + p * RPP) * DK, lr, s[p]);
    }
    float kk[8], qq[8];
    const size_t kq0 = ((size_t)b * hk + kh) * DK;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        load4<E>(k + kq0 + SL::col(lr, 4 * m), kk + 4 * m);
        load4<E>(q + kq0 + SL::col(lr, 4 * m), qq + 4 * m);
    }
    const float a = expf(static_cast<float>(gate_g[(size_t)b * gate_ld + h]));
    float vv[NRL];
#pragma unroll
    for (int p = 0; p < NRL; ++p)
        vv[p] = r0 + p * RPP < DV ? static_cast<float>(v[((size_t)b * hv + h) * DV + r0 + p * RPP]) : 0.f;

    float kq = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) kq = __builtin_fmaf(kk[j], qq[j], kq);
    kq = row_sum<LPR>(kq);
#pragma unroll
    for (int p = 0; p < NRL; ++p) {
        float sq = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sq = __builtin_fmaf(s[p][j], qq[j], sq);
        sq = row_sum<LPR>(sq);
        const int row = r0 + p * RPP;
        if (row < DV) {
            if (lr == 0) o_row[row] = from_f32<E>(scale * __builtin_fmaf(a, sq, kq * vv[p]));
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __builtin_fmaf(a, s[p][j], vv[p] * kk[j]);
            SL::store(state_out + base + (size_t)row * DK, lr, w);
        }
    }
}

// ---------------------------------------------------------------------------
// Launchers
// ---------------------------------------------------------------------------

// Calls f(DK, DV) as integral constants for the built head sizes.
template <typename F> static hipError_t with_heads(int dk, int dv, F f) {
    auto inner = [&](auto kc) {
        switch (dv) {
        case 16: return f(kc, std::integral_constant<int, 16>());
        case 32: return f(kc, std::integral_constant<int, 32>());
        case 64: return f(kc, std::integral_constant<int, 64>());
        case 128: return f(kc, std::integral_constant<int, 128>());
        default: return hipErrorInvalidValue;
        }
    };
    switch (dk) {
    case 16: return inner(std::integral_constant<int, 16>());
    case 32: return inner(std::integral_constant<int, 32>());
    case 64: return inner(std::integral_constant<int, 64>());
    case 128: return inner(std::integral_constant<int, 128>());
    default: return hipErrorInvalidValue;
    }
}

// Calls f(E, G, SE) as values of the built element, gate and state types
// (bf16 states with bf16 I/O only).
template <typename F> static hipError_t with_types(bool io_bf16, bool gate_bf16, bool state_bf16, F f) {
    if (io_bf16) {
        if (state_bf16) return gate_bf16 ? f(bf16(), bf16(), bf16()) : f(bf16(), float(), bf16());
        return gate_bf16 ? f(bf16(), bf16(), float()) : f(bf16(), float(), float());
    }
    if (state_bf16) return hipErrorInvalidValue;
    return gate_bf16 ? f(float(), bf16(), float()) : f(float(), float(), float());
}

int32_t linattn_decode_lanes(int32_t dk, int32_t dv, bool state_bf16) {
    int32_t n = 0;
    (void)with_heads(dk, dv, [&](auto kc, auto vc) {
        typedef LinDecodeShape<bf16, kc(), vc()> B;
        typedef LinDecodeShape<float, kc(), vc()> F;
        n = state_bf16 ? B::SLICES * B::THREADS : F::SLICES * F::THREADS;
        return hipSuccess;
    });
    return n;
}

hipError_t launch_linattn_decode(const LinDecodeArgs &A, hipStream_t st) {
    return with_types(A.io_bf16, A.gate_bf16, A.state_bf16, [&](auto e, auto g, auto se) {
        typedef decltype(e) E;
        typedef decltype(g) G;
        typedef decltype(se) SE;
        return with_heads(A.dk, A.dv, [&](auto kc, auto vc) {
            constexpr int DK = kc(), DV = vc();
            typedef LinDecodeShape<SE, DK, DV> SH;
            const dim3 grid((unsigned)A.batch * (unsigned)A.hv * (unsigned)SH::SLICES), block(SH::THREADS);
            const auto kernel = A.slots ? gdn_linattn_decode_kernel<E, G, SE, DK, DV, true>
                                        : gdn_linattn_decode_kernel<E, G, SE, DK, DV, false>;
            return launch_kernel(kLinDecode, kernel, grid, block, 0, st, (const E *)A.q, (const E *)A.k,
                                 (const E *)A.v, (const G *)A.g, A.gate_per_head ? 0 : A.hv, (const SE *)A.state,
                                 (SE *)A.state_out, A.slots, A.num_slots, (E *)A.out, A.hk, A.hv, A.scale);
        });
    });
}

// ---------------------------------------------------------------------------
// Prefill
// ---------------------------------------------------------------------------

// How a prefill is split, by an estimate of its time (us). Workgroups run in
// rounds of two per compute unit; one takes a fixed time and one per chunk of
// its segment, less with a unit to itself. States of 128 rows may go as two of
// 64: half the work per workgroup, but the scores are formed twice. Segments cost
// a pass for their states, and their states one of two ways: summed by every
// workgroup for itself, a chain over the segments before it, which is less for
// few segments; or by the join kernel, a launch and one pass over the states.
// Fitted at HK = 16, HV = 32, d = 128 to 1 x 512 .. 16,384 and to eight sequences
// of 62,064 tokens in all; measured there (all kernels, us; "+" with the join):
//   1 x 256     two of 64 rows: whole 15.9; segments of 128: 17.9
//   1 x 512     two of 64: of 128 20.1, 26.4+; whole 26.0; one: of 128 26.3
//   1 x 1,024   two of 64: of 128 26.5, 30.3+, of 256 29.1, 32.7+
//   1 x 2,048   two of 64: of 256 35.1, 41.4+; one: of 256 42.6, 43.9+
//   1 x 4,096   two of 64: of 512 56.2, 61.4+; one: of 256 60.0, of 512 59.8
//   1 x 16,384  one: of 1,024 163, 161+, of 512 179+; two of 64: of 1,024 193+
//   8: 62,064   one: of 2,048 606, 603+, of 1,024 629, 625+, of 4,096 665
//   8 x 512     one: whole 39.6, of 256 62.2; two of 64: whole 41.4
// and at HK = 2, HV = 4, 16,001 tokens: two of 64: of 256 62.8, 44.6+.
LinPlan linattn_plan(int64_t num_seqs, int64_t total_tokens, int64_t max_seqlen, int64_t hk, int64_t hv, int64_t dk,
                     int64_t dv, bool io_bf16) {
    const double chunk = io_bf16 ? 64 : 32, xcds = 8, cus = 32;  // compute units of an XCD
    const double N = (double)num_seqs, T = (double)total_tokens;
    // Without a hint the longest sequence may be all there is.
    const double longest = max_seqlen ? (double)max_seqlen : T;
    LinPlan best;
    double best_t = 0;
    auto consider = [&](int32_t dv_shift, int32_t seg_shift) {
        const bool wide = (dv >> dv_shift) == 128;
        const double heads = (double)(hv << dv_shift);
        const bool split = seg_shift >= 0;
        const double L = split ? (double)((int64_t)1 << seg_shift) : 0;
        // The grids (launch_linattn_chunk): items x heads, rounded up to whole
        // turns over the XCDs, and up to 16 workgroups of the join per head.
        const double most_items = (split ? (double)(total_tokens >> seg_shift) : 0) + N;
        if (!launchable((most_items * hk + 7) * (heads / hk) * 256) || (split && !launchable(N * hv * 16 * 256)))
            return;
        // Sequences end inside their last segment: half a segment more each on
        // average, one at most.
        const double items = split ? std::max(N, T / L + (num_seqs > 1 ? 0.5 * N : 0)) : N;
        const double bound = split ? T / L + (num_seqs > 1 ? N : 0) : N;
        // An XCD takes whole groups of heads that share a key head (lin_place).
        auto per_xcd = [&](double n) { return std::ceil(n * hk / xcds) * (heads / hk); };
        const bool shared = per_xcd(bound) > cus;  // units with two
        auto pass = [&](double fixed, double one, double two, double most) {
            const double step = shared ? two : one;
            auto rounds = [&](double n, double tokens) {
                const double r = per_xcd(n) / (2 * cus);
                return (r > 1 ? r + 0.1 : 1.0) * (fixed + std::max(1.0, tokens / chunk) * step);
            };
            // between even segments and as many full ones as there may be
            double t = rounds(items, std::min(most, T / items));
            if (split) t = 0.5 * (t + rounds(bound, most));
            // the longest workgroup may outlast the rounds of the others (whole
            // sequences: in company at first, then alone)
            return std::max(t, fixed + std::ceil(most / chunk) * (split ? one : 0.5 * (one + step)));
        };
        double t;
        bool join = false;
        if (split) {
            const double segs = std::ceil(longest / L), tile = (double)(dk * (dv >> dv_shift) * 4);
            const double states = items * heads * tile;
            const double chain = std::max(segs * (wide ? tile * 13e-6 : 0.08 + tile * 4.5e-6),
                                          states * (0.5 * items / N + 1) / 28e6);
            const double joined = 3.7 + states / 3.9e6 + 0.055 * segs;
            join = joined < chain;
            t = wide ? pass(7, 2.0, 3.35, std::min(L, longest)) + pass(8, 3.1, 5.1, std::min(L, longest))
                     : pass(6.5, 1.15, 1.8, std::min(L, longest)) + pass(6.2, 2.35, 3.5, std::min(L, longest));
            t += std::min(joined, chain) + 1;
        } else {
            t = wide ? pass(8, 4.0, 6.5, longest) : pass(6.2, 2.45, 4.4, longest);
        }
        if (best_t == 0 || t < best_t) {
            best_t = t;
            best.dv_shift = dv_shift;
            best.seg_shift = seg_shift;
            best.join = join;
        }
    };
    for (int32_t f = 0; f <= (dv == 128 ? 1 : 0); ++f) {
        consider(f, -1);
        for (int32_t s = 6; ((int64_t)1 << s) < total_tokens && s < 31; ++s) consider(f, s);
    }
    LinPlan P = best;
    P.items = best_t > 0 ? num_seqs : 0;
    if (num_seqs > kLinListed) {
        P.sorted = true;
        P.off_cu = 0;
        P.total = align256(sizeof(int32_t) * ((size_t)num_seqs + 1));
    }
    if (P.seg_shift >= 0) {
        P.items = (total_tokens >> P.seg_shift) + num_seqs;
        P.off_state = P.total;
        P.off_decay = align256(P.off_state + (size_t)P.items * hv * dk * dv * sizeof(float));
        P.total = align256(P.off_decay + (size_t)P.items * (hv << P.dv_shift) * sizeof(float));
    }
    return P;
}

hipError_t launch_linattn_prefill(const LinPrefillArgs &A, hipStream_t st) {
    switch (A.dk + A.io_bf16) {
    case 16: return launch_linattn_chunk_k<0, 16>(A, st);
    case 17: return launch_linattn_chunk_k<1, 16>(A, st);
    case 32: return launch_linattn_chunk_k<0, 32>(A, st);
    case 33: return launch_linattn_chunk_k<1, 32>(A, st);
    case 64: return launch_linattn_chunk_k<0, 64>(A, st);
    case 65: return launch_linattn_chunk_k<1, 64>(A, st);
    case 128: return launch_linattn_chunk_k<0, 128>(A, st);
    case 129: return launch_linattn_chunk_k<1, 128>(A, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn
