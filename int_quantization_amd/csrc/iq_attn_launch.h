// Internal interface between the attention entry points (iq_attn_api.cpp) and
// their kernel launchers (iq_cache.hip, iq_attend.hip).  Not part of the
// public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

namespace iqk {

struct RotaryArgs {
    int dtype, interleaved;
    int tokens, heads, dim, rot;
    int64_t ld_token, ld_head, ld_token_out, ld_head_out;
    float amplitude, way;        // way: 1, or -1 for the transposed rotation
    const void* x;
    const int32_t* positions;
    const double* table;
    void* y;
};

// The paged cache as kernels see it: blocks of 32 tokens, 1 << shift of them a page.
struct CacheArgs {
    int fmt, heads, dim, shift, batch, width;
    int64_t pages;
    uint8_t* codes;
    float* scales;
    const int32_t* page_table;
    const int32_t* lengths;
    const int32_t* starts;       // may be null: one token a sequence
    int tokens;
};

struct AppendArgs {
    CacheArgs c;
    int dtype, interleaved, q_heads, rot;
    int64_t ld_k_token, ld_k_head, ld_v_token, ld_v_head, ld_q_token, ld_q_head;
    float amplitude;
    const void* k;
    const void* v;
    const void* q;               // may be null
    void* q_out;
    const double* table;
};

struct ReadArgs {
    CacheArgs c;
    int dtype;
    void* k;                     // may be null
    void* v;                     // may be null
};

struct AttendArgs {
    CacheArgs c;
    int q_heads, group;          // group: query heads of a key head
    int causal;
    int64_t ld_token, ld_head;
    int window;                  // 1 to 2^30; the latter is as good as none, since no table has entries for more
    float scale;
    const void* q;
    void* o;
    void* workspace;
};

// Each returns hipSuccess or the launch error.
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);
hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream);
hipError_t launch_cache_read(const ReadArgs& a, hipStream_t stream);
hipError_t launch_attend(const AttendArgs& a, hipStream_t stream);
// Workspace of launch_attend: the parts of rows whose sum is split.
size_t attend_workspace_bytes(const AttendArgs& a);

}  // namespace iqk
