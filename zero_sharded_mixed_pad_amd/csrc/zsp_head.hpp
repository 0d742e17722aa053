// zsp_head.hpp -- what the entry points of the head's losses (zsp_head.cpp)
// and their kernels (zsp_head.hip) share: one call's arguments, sizes and
// workspace.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zsp.h"

namespace zsp {

constexpr int32_t kHeadTile = 256;       // columns of P, and rows of more than 64 tokens, are
                                         // padded to it
constexpr int32_t kHeadBlock = 64;       // vocabulary columns per partial of a softmax
constexpr int32_t kHeadDepth = 64;       // d is padded to it
constexpr int32_t kHeadMaxTop = 1024;    // teacher's entries per token
constexpr int32_t kHeadFew = 128;        // tokens whose gradient of the head has a way of its own
constexpr int32_t kHeadThin = 64;        // tokens whose tiles hold so many at most; they read an
                                         // fp32 head in place
constexpr int32_t kHeadRawColumns = 8192;   // logits of a token that a workgroup keeps in LDS
constexpr int32_t kHeadRawSmall = 4096;     // ... of 256 threads

// How a product is cut: columns and rows of a tile, how many the card runs at
// once (log2), which form, and the most of a call that the device may make of
// them once it knows the tokens that count.
struct HeadTiles {
    uint32_t ba = 0, bb = 0, slot_bits = 0;
    int32_t form = 0;
    uint32_t segs = 1;            // stages of a step of 64 k's
    uint64_t items = 0;           // tiles times the parts of their sums
    uint64_t split_rows = 0;      // rows times parts, where sums are split
};

// Sizes of a call, and the byte offsets of its parts of the workspace.
struct HeadShape {
    int64_t n = 0, v = 0, d = 0;
    int32_t top = 1;              // entries per token (a target is one)
    bool f32 = false, teacher = false;
    bool grad_hidden = false, grad_head = false;
    bool in_place = false;        // an fp32 head may be read in place
    bool thin = false;            // and is, by few tokens
    bool pack_head = false;       // the head is copied: fp32, d or its address not aligned
    bool raw = false;             // logits summed in parts, in the workspace
    int32_t planes = 1;           // bf16 planes of an operand: 3 hold an fp32 value
    int32_t top_pad = 1;          // entries per row in the workspace
    int64_t rows = 0;             // n padded to the tokens of a tile
    int64_t vp = 0, dp = 0;       // v padded to kHeadTile, d to kHeadDepth
    int64_t chunk = 0;            // tokens whose softmax is kept at a time
    int64_t chunk_most = 0;       // ... of a call with any number of tokens
    int64_t nchunk = 0;
    int64_t xt_tokens = 0;        // columns of the copy of X^T, for few tokens
    HeadTiles raw_tiles;          // of the logits in parts
    HeadTiles hidden_tiles[2], head_tiles[2];   // the gradients' of a chunk, and of the last one
    int64_t split_bytes = 0;      // for the parts of the sums that are split
    // offsets
    int64_t o_count = 0, o_rows = 0, o_coef = 0, o_entry = 0, o_pick = 0, o_teach = 0, o_start = 0,
            o_flag = 0, o_x = 0, o_xt = 0, o_w = 0, o_part = 0, o_p = 0, o_g = 0, o_split = 0, o_acc = 0;
    int64_t bytes = 0;
};

struct HeadCall {
    const void* hidden;
    const void* head;
    const int64_t* index;         // target [n], or the teacher's [n, top]
    const float* logit;           // the teacher's [n, top], else NULL
    const float* token_weight;    // [n] or NULL
    float scale, temperature;
    float* loss;                  // [n]
    float* lse;                   // [n] or NULL
    void* grad_hidden;
    void* grad_head;
    char* ws;
};

// Whether its rows can be set up in one launch.
bool head_fits_launch(const HeadShape& s);
// How its products are cut, whether its logits are summed in parts, and the
// bytes for parts of sums.
void head_products(HeadShape* s);
// No fewer bytes for parts of sums than any call with up to s.n tokens needs.
int64_t head_split_most(const HeadShape& s);
// Every launch of a call, in order, on `stream`.
hipError_t launch_head(const HeadShape& s, const HeadCall& c, hipStream_t stream);

}  // namespace zsp
