// gdn_linattn.hpp -- internal host-side interface of the linear attention
// with decay (gdn_linattn_api.hip to the kernel launchers). Not part of the
// ABI.
#pragma once

#include "gdn_launch.hpp"

namespace gdn {

// A launch has fewer than 2^32 lanes.
inline bool launchable(double lanes) { return lanes <= (double)UINT32_MAX; }

// How a prefill is split: whole sequences (seg_shift < 0), or segments of
// 2^seg_shift tokens whose states go through the workspace.
struct LinPlan {
    int32_t seg_shift = -1;
    int32_t dv_shift = 0;       // a state of dv rows goes as 2^dv_shift states of fewer
    bool join = false;          // segments are joined by a kernel, not by each workgroup for itself
    int64_t items = 0;          // sequences, or the bound on segments; 0: too many to launch
    bool sorted = false;        // the offsets are put in order first
    size_t off_cu = 0;          // int32 [num_seqs + 1]
    size_t off_state = 0;       // float [items][hv][dv * dk], accumulator order
    size_t off_decay = 0;       // float [items][hv << dv_shift]
    size_t total = 0;           // bytes of workspace
};
// From how many sequences on the offsets are put in order by a kernel of its
// own, 4 us up to 4,096 of them. Without and with it, all kernels (us), one
// token each, d = 64, 4 or 8 heads: 257 sequences 22.4 and 26.4, 512 42.4 and
// 37.5, 4,096 358 and 137, 16,384 3,630 and 578.
constexpr int32_t kLinListed = 400;
LinPlan linattn_plan(int64_t num_seqs, int64_t total_tokens, int64_t max_seqlen, int64_t hk, int64_t hv, int64_t dk,
                     int64_t dv, bool io_bf16);

struct LinPrefillArgs {
    const void *q, *k, *v, *g;
    const int32_t *cu;
    int32_t num_seqs;
    int64_t total_tokens;
    int32_t hk, hv, dk, dv;
    float scale;
    bool io_bf16, gate_bf16, state_bf16;
    bool gate_per_head;  // g is [hv], not [T][hv]
    const void *s0;
    void *s_final;
    void *out;
    char *ws;
    LinPlan plan;
};
// Chunk by chunk, one instantiation per I/O type and dk (gdn_linattn_inst.hip).
template <int kIoBf16, int DK> hipError_t launch_linattn_chunk_k(const LinPrefillArgs &a, hipStream_t st);
hipError_t launch_linattn_prefill(const LinPrefillArgs &a, hipStream_t st);

struct LinDecodeArgs {
    const void *q, *k, *v, *g;
    const void *state;
    void *state_out;  // may be `state`
    const int32_t *slots;
    int32_t num_slots;
    void *out;
    int32_t batch, hk, hv, dk, dv;
    float scale;
    bool io_bf16, gate_bf16, state_bf16, gate_per_head;
};
hipError_t launch_linattn_decode(const LinDecodeArgs &a, hipStream_t st);

// Lanes per (sequence, value head) that launch_linattn_decode takes.
int32_t linattn_decode_lanes(int32_t dk, int32_t dv, bool state_bf16);

struct StateCacheArgs {
    void *state;            // written by a read, read by a write
    const int32_t *slots;   // NULL: the identity
    int32_t num_slots;
    void *cache;
    float *scales;
    const int32_t *entries;
    int32_t num_entries;
    int32_t n, hv, dk, dv;
    bool state_bf16, e4m3;
};
hipError_t launch_state_cache_write(const StateCacheArgs &a, hipStream_t st);
hipError_t launch_state_cache_read(const StateCacheArgs &a, hipStream_t st);

}  // namespace gdn
