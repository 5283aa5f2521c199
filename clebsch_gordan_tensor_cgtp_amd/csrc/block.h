// A block plan: the row norm at a block's entry and the join at its end, for one irreps row and
// one configuration.  Its kernels (block_kernels.h) are compiled per plan, as the convolution's are.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "cgtp.h"
#include "plan.h"

namespace cgtp {

struct Block {
    struct Segment {
        int col, ch, k, mul;  // first column, first channel, 2l+1, channels
    };
    std::vector<Segment> segs;  // neighbouring irreps of equal degree are one
    int d = 0, c = 0;           // columns, channels
    bool flat = false;          // lanes are dealt columns, not channels
    cgtp_block_config cfg{};
    int elem = 4, real = 4;     // bytes of an element; of a statistic, weight or sum
    int vec = 4;                        // elements of 16 bytes
    int lanes = 64, cv = 1, elems = 1;  // lanes of a row, channels of a slot, elements of a lane
    int block = 256;                    // threads of a workgroup
    std::string source;
    std::vector<char> code;

    std::mutex mu;  // guards the per-device modules
    struct Fns {
        hipModule_t module = nullptr;
        hipFunction_t norm_fwd = nullptr, norm_bwd = nullptr, join_fwd = nullptr, join_bwd = nullptr, reduce = nullptr;
    };
    std::map<int, Fns> loaded;

    int rows_per_group() const { return block / lanes; }  // rows of a workgroup at a time
    // what lanes are dealt: the channels of the irreps, or the row's columns
    std::vector<Segment> slots_over() const { return flat ? std::vector<Segment>{{0, 0, 1, d}} : segs; }
    int gate_width() const { return cfg.gate == CGTP_GATE_CHANNEL ? c : cfg.gate == CGTP_GATE_ROW ? 1 : 0; }
};

void build_block(Block &b, const std::string &irreps);
const Block::Fns &block_for_current_device(Block &b);
void unload_block(Block &b);
// workgroups of a pass over N rows; a backward's write one partial of the weight gradients each
int64_t block_groups(const Block &b, int64_t N, int waves_per_simd = 2);

}  // namespace cgtp
