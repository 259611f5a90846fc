// gdn_linattn_inst.hip -- one (element type, dk) instantiation of the chunked
// linear attention (gdn_linattn_chunk.hpp), for every dv. The build compiles
// this file once per pair, with GDN_INST_BF16 (1: bf16 I/O, 0: fp32 I/O) and
// GDN_INST_DK defined, so that they compile in parallel.
#include "gdn_linattn_chunk.hpp"

// Compiled without the two macros the file is empty.
#if defined(GDN_INST_BF16) && defined(GDN_INST_DK)

namespace gdn {

#if GDN_INST_BF16
typedef bf16 InstElem;
#else
typedef float InstElem;
#endif

template <typename E, int DK, int DV> hipError_t launch_linattn_chunk(const LinPrefillArgs &A, hipStream_t st) {
    typedef LinShape<E, DK, DV> SH;
    // The rows of a state are independent, so that one of dv rows is also
    // 2^dv_shift heads of DV rows with the same gates, whose v, out and states
    // lie as they do.
    const int32_t hv = A.hv << A.plan.dv_shift;
    const uint32_t hk = (uint32_t)A.hk, group = (uint32_t)(hv / A.hk);
    LinWork w{A.cu, A.plan.sorted, A.num_seqs, (int32_t)A.total_tokens, A.plan.seg_shift, hk, group,
              (uint32_t)A.plan.items * hk};
    hipError_t e = hipSuccess;
    if (w.sorted) {
        int32_t *cu = reinterpret_cast<int32_t *>(A.ws + A.plan.off_cu);
        e = launch_kernel(kSchedule, gdn_linattn_offsets_kernel<1024>, dim3(1), dim3(1024), 0, st, A.cu, A.num_seqs,
                          (int32_t)A.total_tokens, cu);
        if (e != hipSuccess) return e;
        w.cu = cu;
    }
    LinIo io;
    io.q = A.q; io.k = A.k; io.v = A.v; io.g = A.g;
    io.gate_ld = A.gate_per_head ? 0 : A.hv; io.gate_shift = A.plan.dv_shift;
    io.s0 = A.s0; io.s_final = A.s_final; io.out = A.out; io.scale = A.scale;
    io.gate_bf16 = A.gate_bf16; io.state_bf16 = A.state_bf16;
    io.seg_state = reinterpret_cast<float *>(A.ws + A.plan.off_state);
    io.seg_decay = reinterpret_cast<float *>(A.ws + A.plan.off_decay);
    io.joined = A.plan.join;
    const dim3 grid((unsigned)lin_grid(w.units, group)), block(SH::THREADS);
    auto launch = [&](KernelKind kind, auto mode) {
        return launch_kernel(kind, gdn_linattn_chunk_kernel<E, DK, DV, mode()>, grid, block, 0, st, w, io);
    };
    if (w.seg_shift < 0) return launch(kLinOut, std::integral_constant<LinMode, kLinWhole>());
    e = launch(kLinState, std::integral_constant<LinMode, kLinSegState>());
    if (e != hipSuccess) return e;
    if (io.joined) {
        const unsigned heads = (unsigned)A.num_seqs * (unsigned)hv, quads = DK * DV / 4;
        const unsigned wide = heads * ((quads + 255) / 256);
        const dim3 few(heads * (quads / 64));
        e = wide >= 256
                ? launch_kernel(kLinJoin, gdn_linattn_join_kernel<DK, DV, 256, 8>, dim3(wide), dim3(256), 0, st, w, io)
                : launch_kernel(kLinJoin, gdn_linattn_join_kernel<DK, DV, 64, 16>, few, dim3(64), 0, st, w, io);
        if (e != hipSuccess) return e;
    }
    return launch(kLinOut, std::integral_constant<LinMode, kLinSegOut>());
}

template <> hipError_t launch_linattn_chunk_k<GDN_INST_BF16, GDN_INST_DK>(const LinPrefillArgs &A, hipStream_t st) {
    switch (A.dv >> A.plan.dv_shift) {
    case 16: return launch_linattn_chunk<InstElem, GDN_INST_DK, 16>(A, st);
    case 32: return launch_linattn_chunk<InstElem, GDN_INST_DK, 32>(A, st);
    case 64: return launch_linattn_chunk<InstElem, GDN_INST_DK, 64>(A, st);
    case 128: return launch_linattn_chunk<InstElem, GDN_INST_DK, 128>(A, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace gdn

#endif
