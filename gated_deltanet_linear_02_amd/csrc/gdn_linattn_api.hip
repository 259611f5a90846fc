// gdn_linattn_api.hip -- the C ABI of the linear attention with decay and of
// the 8-bit state cache: argument checks (all before any HIP call) and
// dispatch.
#include "gdn.h"
#include "gdn_checks.hpp"
#include "gdn_linattn.hpp"

#include <algorithm>

using namespace gdn;

// Sizes and types that both linear-attention calls share.
static int32_t check_linattn(int32_t hk, int32_t hv, int32_t dk, int32_t dv, int32_t io_dtype, int32_t gate_dtype,
                             int32_t gate_per_head, int32_t state_dtype) {
    if (hk < 1 || hv < 1 || hv % hk != 0) return GDN_ERR_BAD_SHAPE;
    if (!valid_head(dk) || !valid_head(dv) || !valid_dtype(io_dtype) || !valid_dtype(gate_dtype) ||
        !valid_dtype(state_dtype) || (state_dtype == GDN_BF16 && io_dtype != GDN_BF16))
        return GDN_ERR_UNSUPPORTED;
    if (gate_per_head != 0 && gate_per_head != 1) return GDN_ERR_BAD_VALUE;
    return GDN_OK;
}

static int32_t check_linattn_prefill(int32_t num_seqs, int64_t total_tokens, int64_t max_seqlen, int32_t hk,
                                     int32_t hv, int32_t dk, int32_t dv, int32_t io_dtype, int32_t gate_dtype,
                                     int32_t gate_per_head, int32_t state_dtype) {
    if (num_seqs < 1 || total_tokens < 0 || total_tokens > INT32_MAX) return GDN_ERR_BAD_SHAPE;
    const int32_t sc = check_linattn(hk, hv, dk, dv, io_dtype, gate_dtype, gate_per_head, state_dtype);
    if (sc != GDN_OK) return sc;
    if (max_seqlen != 0 &&
        (max_seqlen < 0 || max_seqlen > total_tokens || max_seqlen * (int64_t)num_seqs < total_tokens))
        return GDN_ERR_BAD_VALUE;
    // A chunk's rows lie within 32 bits of each other (LinStage), and no sum
    // of a token's number and a chunk passes an int.
    if ((int64_t)hv * dv > (int64_t)1 << 22 || (int64_t)hk * dk > (int64_t)1 << 22 || total_tokens > INT32_MAX - 64)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

extern "C" {

size_t gdn_linattn_prefill_workspace_size(int32_t num_seqs, int64_t total_tokens, int64_t max_seqlen, int32_t hk,
                                          int32_t hv, int32_t dk, int32_t dv, int32_t io_dtype) {
    if (check_linattn_prefill(num_seqs, total_tokens, max_seqlen, hk, hv, dk, dv, io_dtype, GDN_F32, 0, GDN_F32) !=
        GDN_OK)
        return 0;
    const LinPlan plan = linattn_plan(num_seqs, total_tokens, max_seqlen, hk, hv, dk, dv, io_dtype == GDN_BF16);
    return plan.items ? std::max<size_t>(256, plan.total) : 0;
}

int32_t gdn_linattn_prefill(const void *q, const void *k, const void *v, const void *g, const int32_t *cu_seqlens,
                            int32_t num_seqs, int64_t total_tokens, int64_t max_seqlen, int32_t hk, int32_t hv,
                            int32_t dk, int32_t dv, float scale, int32_t io_dtype, int32_t gate_dtype,
                            int32_t gate_per_head, const void *initial_state, void *final_state,
                            int32_t state_dtype, void *out, void *workspace, size_t workspace_bytes, void *stream) {
    const int32_t sc = check_linattn_prefill(num_seqs, total_tokens, max_seqlen, hk, hv, dk, dv, io_dtype,
                                             gate_dtype, gate_per_head, state_dtype);
    if (sc != GDN_OK) return sc;
    const LinPlan plan = linattn_plan(num_seqs, total_tokens, max_seqlen, hk, hv, dk, dv, io_dtype == GDN_BF16);
    if (plan.items == 0) return GDN_ERR_UNSUPPORTED;
    if (!cu_seqlens) return GDN_ERR_NULL_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !g || !out)) return GDN_ERR_NULL_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(initial_state) ||
        !aligned16(final_state))
        return GDN_ERR_MISALIGNED;
    const size_t used = plan.total;
    if (used && (!workspace || workspace_bytes < used || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return GDN_ERR_WORKSPACE;

    const size_t T = (size_t)total_tokens, eb = dtype_bytes(io_dtype), gb = dtype_bytes(gate_dtype);
    const size_t state_bytes = (size_t)num_seqs * hv * dv * dk * dtype_bytes(state_dtype);
    const Range r_out = span(out, T * hv * dv * eb), r_fin = span(final_state, state_bytes),
                r_init = span(initial_state, state_bytes), r_ws = span(workspace, used);
    const Range inputs[] = {span(q, T * hk * dk * eb), span(k, T * hk * dk * eb), span(v, T * hv * dv * eb),
                            span(g, (gate_per_head ? 1 : T) * hv * gb),
                            span(cu_seqlens, sizeof(int32_t) * ((size_t)num_seqs + 1))};
    for (const Range &r : inputs)
        if (overlaps(r_out, r) || overlaps(r_fin, r) || overlaps(r_ws, r)) return GDN_ERR_ALIAS;
    if (overlaps(r_out, r_fin) || overlaps(r_out, r_init) || overlaps(r_out, r_ws) || overlaps(r_ws, r_fin) ||
        overlaps(r_ws, r_init) || (initial_state != final_state && overlaps(r_init, r_fin)))
        return GDN_ERR_ALIAS;

    LinPrefillArgs A;
    A.q = q; A.k = k; A.v = v; A.g = g; A.cu = cu_seqlens;
    A.num_seqs = num_seqs; A.total_tokens = total_tokens;
    A.hk = hk; A.hv = hv; A.dk = dk; A.dv = dv; A.scale = scale;
    A.io_bf16 = io_dtype == GDN_BF16; A.gate_bf16 = gate_dtype == GDN_BF16; A.state_bf16 = state_dtype == GDN_BF16;
    A.gate_per_head = gate_per_head != 0;
    A.s0 = initial_state; A.s_final = final_state; A.out = out; A.ws = static_cast<char *>(workspace);
    A.plan = plan;
    try {
        return launch_linattn_prefill(A, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    } catch (...) {
        return GDN_ERR_HIP;
    }
}

int32_t gdn_linattn_decode_step(const void *q, const void *k, const void *v, const void *g, int32_t batch,
                                int32_t hk, int32_t hv, int32_t dk, int32_t dv, float scale, int32_t io_dtype,
                                int32_t gate_dtype, int32_t gate_per_head, void *state, void *state_out,
                                int32_t state_dtype, const int32_t *state_slots, int32_t num_slots, void *out,
                                void *stream) {
    if (batch < 0 || num_slots < 0) return GDN_ERR_BAD_SHAPE;
    const int32_t sc = check_linattn(hk, hv, dk, dv, io_dtype, gate_dtype, gate_per_head, state_dtype);
    if (sc != GDN_OK) return sc;
    if (batch == 0) return GDN_OK;
    if (!state_slots && num_slots < batch) return GDN_ERR_BAD_SHAPE;
    if (!launchable((double)batch * hv * linattn_decode_lanes(dk, dv, state_dtype == GDN_BF16)))
        return GDN_ERR_UNSUPPORTED;
    if (!q || !k || !v || !g || !state || !out) return GDN_ERR_NULL_ARG;
    if (!state_out) state_out = state;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(state) ||
        !aligned16(state_out))
        return GDN_ERR_MISALIGNED;

    const size_t eb = dtype_bytes(io_dtype), gb = dtype_bytes(gate_dtype), B = (size_t)batch;
    const size_t state_bytes = (size_t)num_slots * hv * dv * dk * dtype_bytes(state_dtype);
    const Range r_out = span(out, B * hv * dv * eb), r_in = span(state, state_bytes),
                r_new = span(state_out, state_bytes);
    const Range inputs[] = {span(q, B * hk * dk * eb), span(k, B * hk * dk * eb), span(v, B * hv * dv * eb),
                            span(g, (gate_per_head ? 1 : B) * hv * gb), span(state_slots, B * sizeof(int32_t))};
    for (const Range &r : inputs)
        if (overlaps(r_out, r) || overlaps(r_new, r)) return GDN_ERR_ALIAS;
    if (overlaps(r_out, r_in) || overlaps(r_out, r_new) || (state_out != state && overlaps(r_in, r_new)))
        return GDN_ERR_ALIAS;

    LinDecodeArgs A;
    A.q = q; A.k = k; A.v = v; A.g = g;
    A.state = state; A.state_out = state_out; A.slots = state_slots; A.num_slots = num_slots; A.out = out;
    A.batch = batch; A.hk = hk; A.hv = hv; A.dk = dk; A.dv = dv; A.scale = scale;
    A.io_bf16 = io_dtype == GDN_BF16; A.gate_bf16 = gate_dtype == GDN_BF16; A.state_bf16 = state_dtype == GDN_BF16;
    A.gate_per_head = gate_per_head != 0;
    try {
        return launch_linattn_decode(A, static_cast<hipStream_t>(stream)) == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    } catch (...) {
        return GDN_ERR_HIP;
    }
}

}  // extern "C"

// gdn_state_cache_write and gdn_state_cache_read: `to_cache` tells which side is written.
static int32_t state_cache_impl(bool to_cache, void *state, int32_t state_dtype, const int32_t *slots,
                                int32_t num_slots, void *cache, int32_t cache_dtype, float *scales,
                                const int32_t *entries, int32_t num_entries, int32_t n, int32_t hv, int32_t dk,
                                int32_t dv, void *stream) {
    if (n < 0 || num_slots < 0 || num_entries < 0 || hv < 1) return GDN_ERR_BAD_SHAPE;
    if (!valid_head(dk) || !valid_head(dv) || !valid_dtype(state_dtype) ||
        (cache_dtype != GDN_I8 && cache_dtype != GDN_E4M3))
        return GDN_ERR_UNSUPPORTED;
    if (n == 0) return GDN_OK;
    if ((!slots && num_slots < n) || (!entries && num_entries < n)) return GDN_ERR_BAD_SHAPE;
    // A workgroup takes at least 32 rows.
    const int64_t rows = (int64_t)hv * dv;
    if (rows > INT32_MAX || !launchable((double)((rows + 31) / 32) * n * 256)) return GDN_ERR_UNSUPPORTED;
    if (!state || !cache || !scales) return GDN_ERR_NULL_ARG;
    if (!aligned16(state) || !aligned16(cache)) return GDN_ERR_MISALIGNED;
    const Range r_state = span(state, (size_t)num_slots * rows * dk * dtype_bytes(state_dtype)),
                r_cache = span(cache, (size_t)num_entries * rows * dk),
                r_scales = span(scales, (size_t)num_entries * rows * sizeof(float)),
                r_slots = span(slots, (size_t)n * sizeof(int32_t)),
                r_entries = span(entries, (size_t)n * sizeof(int32_t));
    if (overlaps(r_state, r_cache) || overlaps(r_state, r_scales) || overlaps(r_cache, r_scales))
        return GDN_ERR_ALIAS;
    for (const Range &r : {r_slots, r_entries})
        if (to_cache ? overlaps(r_cache, r) || overlaps(r_scales, r) : overlaps(r_state, r)) return GDN_ERR_ALIAS;

    StateCacheArgs A;
    A.state = state; A.slots = slots; A.num_slots = num_slots;
    A.cache = cache; A.scales = scales; A.entries = entries; A.num_entries = num_entries;
    A.n = n; A.hv = hv; A.dk = dk; A.dv = dv;
    A.state_bf16 = state_dtype == GDN_BF16; A.e4m3 = cache_dtype == GDN_E4M3;
    try {
        const hipStream_t st = static_cast<hipStream_t>(stream);
        const hipError_t e = to_cache ? launch_state_cache_write(A, st) : launch_state_cache_read(A, st);
        return e == hipSuccess ? GDN_OK : GDN_ERR_HIP;
    } catch (...) {
        return GDN_ERR_HIP;
    }
}

extern "C" {

int32_t gdn_state_cache_write(const void *state, int32_t state_dtype, const int32_t *slots, int32_t num_slots,
                              void *cache, int32_t cache_dtype, float *scales, const int32_t *entries,
                              int32_t num_entries, int32_t n, int32_t hv, int32_t dk, int32_t dv, void *stream) {
    return state_cache_impl(true, const_cast<void *>(state), state_dtype, slots, num_slots, cache, cache_dtype,
                            scales, entries, num_entries, n, hv, dk, dv, stream);
}

int32_t gdn_state_cache_read(const void *cache, int32_t cache_dtype, const float *scales, const int32_t *entries,
                             int32_t num_entries, void *state, int32_t state_dtype, const int32_t *slots,
                             int32_t num_slots, int32_t n, int32_t hv, int32_t dk, int32_t dv, void *stream) {
    return state_cache_impl(false, state, state_dtype, slots, num_slots, const_cast<void *>(cache), cache_dtype,
                            const_cast<float *>(scales), entries, num_entries, n, hv, dk, dv, stream);
}

}  // extern "C"
