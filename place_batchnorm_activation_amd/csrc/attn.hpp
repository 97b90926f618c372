// Host launchers and arguments of the attention operators and of the rotary positions
// (attn_fwd.hip, attn_bwd.hip, rotary.hip).  They enqueue on `s` and return; arguments
// are validated by the C ABI layer (api_attn.cpp) before any of these is called.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "block.hpp"
#include "plan.hpp"

namespace iabn {

constexpr int64_t kAttnMaxD = 128;                 // of a head
constexpr int64_t kAttnMaxLen = int64_t(1) << 29;  // of a sequence, and of its rows

// A tensor of heads: element (b, row, head, d) at b*batch + row*row_ + head*head_ + d.
struct Heads {
    char* p;
    int64_t batch, row, head;
};

// One attention problem.  A "row" is a query of one head of a key head's group: row r of
// key head h is token r / G of query head h * G + r % G.  All rows of a key head stand
// beside the same keys, so a tile of rows serves grouped heads and single tokens alike.
struct AttnArgs {
    Heads q, k, v, out;
    float* lse;                                    // [B, H, Sq], packed: [H, q_rows]
    int B, KV, G, D, Sq, Sk;                       // Sq, Sk: the most of a sequence
    int64_t q_rows, k_rows;                        // rows of packed tensors
    const int32_t *q_starts, *k_starts, *q_lens, *k_lens;
    int left, right;                               // kAttnMaxLen: unbounded
    float scale, c;                                // c = scale * log2(e)
    FastDiv group;                                 // by G
};

struct AttnGrads {
    Heads dout, dq, dk, dv;
};

// The most keys that some of n neighbouring queries see (of queries that n neighbouring keys are
// seen by).
inline int64_t seen_most(const AttnArgs& a, int64_t n, int64_t most)
{
    return min64(most, int64_t(a.left) + a.right + n);
}

size_t attn_fwd_workspace_bytes(const AttnArgs& a, int dtype, int64_t cus);
size_t attn_bwd_workspace_bytes(const AttnArgs& a, int64_t cus);
void launch_attn_forward(const AttnArgs& a, int dtype, int64_t cus, void* ws, hipStream_t s);
void launch_attn_backward(const AttnArgs& a, const AttnGrads& g, int dtype, int64_t cus, void* ws,
                          hipStream_t s);

// rotary.hip
enum PosType { kPosI32 = 0, kPosI64 = 1, kPosF32 = 2 };
struct RotaryArgs {
    Heads x[2], y[2];                              // the second with heads[1] == 0: none
    int heads[2];
    int64_t B, S;
    int D, pairs, axes, interleaved, pos_type;
    const double* inv_freq;
    const int32_t* axis;                           // or NULL
    const void* positions;
    int64_t pos_batch, pos_row;                    // elements
    float sign;                                    // -1: the inverse
};
void launch_rotary(const RotaryArgs& a, int dtype, int64_t cus, hipStream_t s);

}  // namespace iabn
