// What the attention kernels and their launcher share.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mmq.h"

namespace mmq {

// One call's work.  A row is one (token, head of the kv head's group) pair,
// row r of kv head h being token r / group, head h * group + r % group.  Each
// part (a range of prefix keys, or a range of a token's own suffix) leaves
// per (token, head) its unnormalised sum of weights x values, f32
// [part][token][head][dim], and (m, l): a reference near its largest score, in
// units of log2, and its sum of weights 2^(score - m); (-inf, 0) and no values
// for no keys.
struct AttnArgs {
    mmq_shared_prefix_attention_t p;
    float* part_o;
    float2* part_ml;
    int* status;
    int64_t tokens;       // batch * q_len
    int group;            // heads per kv head
    int prefix_tiles;     // the prefix kernel's 128-row tiles per CTA
    int prefix_parts;     // parts 0 .. prefix_parts - 1
    int64_t part_keys;    // prefix keys per part, a multiple of the kernel's key tile
    int suffix_parts;     // the parts after them
    int inject;           // test hook: the prefix kernel's first CTA withholds one key tile
    bool beside;          // the suffix kernel follows a prefix kernel, which it does not depend on
    int page_shift;
    float scale_log2;     // scale * log2(e)
};

// The prefix's parts on the tensor cores (attention_tc.cu); cfg: stream and attributes.
cudaError_t launch_attention_prefix(const AttnArgs& a, int nsm, const cudaLaunchConfig_t& cfg);

}  // namespace mmq
