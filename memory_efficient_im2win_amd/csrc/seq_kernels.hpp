// Parameters and launchers of the sequence operators, shared by their C
// entry points. Launchers return 0, or -3 if a launch failed; arguments are
// checked by the entry points first.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "im2win_seq.h"
#include "kernels.hpp"

namespace im2win {
namespace seq {

struct Tensor {
    unsigned char* p;
    int64_t sb, sl, sh;  // strides in bytes
};

// Window attention. Rows are flattened: row r of key head hk is query r / G of
// query head hk * G + r % G, so the heads that share keys share a tile.
struct AttnParams {
    Tensor q, k, v, out, dout, dq, dk, dv;
    float* lse;
    const int32_t *q_lens, *kv_lens, *table;
    int64_t table_stride;
    int B, Lq, Lk, Hq, Hkv, D, G, rows;  // rows = Lq * G
    int pages, window, sinks;
    float scale;
    FastDiv by_group, by_page;
    // Forward: key tiles split over nsplit workgroups, partial results in ws.
    int nsplit, tiles;
    float* part;
    // Backward: row statistics (lse in log2 units, sum of dout * out), padded
    // to stat_rows for each (sequence, key head); partial sums of the keys in
    // sink tiles.
    float *stat_lse, *stat_delta;
    int stat_rows, key_tiles, sink_tiles, chunks, chunk_len;
};

// How a forward call is laid out.
struct AttnPlan {
    int tile_rows, tiles, nsplit;
    size_t ws_bytes;
};
AttnPlan attn_plan(const AttnParams& a);
int launch_attn_fwd(AttnParams a, const AttnPlan& plan, bool bf, hipStream_t st);

struct AttnBwdPlan {
    int stat_rows, group_keys, key_tiles, sink_tiles, chunks, chunk_len;
    size_t stat_bytes, ws_bytes;
};
AttnBwdPlan attn_bwd_plan(const AttnParams& a);
int launch_attn_bwd(AttnParams a, const AttnBwdPlan& plan, void* ws, bool bf, hipStream_t st);

// Linear attention, as a recurrence over tokens in either direction:
//     T_(t+1) = a (T_t + ...) , see seq_linear.hip. One job is one recurrence.
struct LinJob {
    Tensor q, k, v, out;
    const float* s_in;         // (B, H) blocks of Dk x Dv floats with the strides below, or NULL
    float* s_out;              // the same, or NULL
    int sk, sv;                // strides of a state's rows (dk) and columns (dv)
    int dk, dv;                // head sizes of q and k, of v and out
    int reverse;               // tokens from the last to the first
    int lead;                  // 1: out_t sees a S_t-1 (forward); 0: the state given counts undecayed
    float w_in, w_state, w_new;  // factors of q k^T, of q S, and of k v^T in the state
    float* seg;                // workspace: states before each segment
};
struct LinParams {
    LinJob job[2];
    const float* log_decay;
    const int32_t* lens;
    int jobs, B, L, H, nseg, seg_len;
};
// Segments of a call of `jobs` recurrences, and the workspace of one job.
struct LinPlan {
    int nseg, seg_len;
};
LinPlan lin_plan(int jobs, int B, int L, int H);
size_t lin_seg_bytes(const LinPlan& p, int B, int H, int dk, int dv);
// Jobs of one launch have the same head sizes. pair: two jobs over the same
// tensors, see seq_linear.hip; both head sizes pad to the same one.
int launch_linear(const LinParams& a, bool pair, bool bf, hipStream_t st);
int padded_head(int d);

struct LinStep {
    Tensor q, k, v, out;
    const float* log_decay;
    float* state;
    int B, H, dk, dv;
    float scale;
};
int launch_linear_step(const LinStep& a, bool bf, hipStream_t st);

// Calls f with the padded head size as a constant: 64, 96 or 128.
template <typename F>
int with_head(int D, F f)
{
    if (D <= 64) return f(std::integral_constant<int, 64>());
    if (D <= 96) return f(std::integral_constant<int, 96>());
    return f(std::integral_constant<int, 128>());
}

}  // namespace seq
}  // namespace im2win
