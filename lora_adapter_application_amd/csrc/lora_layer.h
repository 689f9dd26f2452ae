// lora_layer.h -- launch interface between the host side (lora_layer.cpp) and
// the kernels of a layer's frozen part: the 4-bit base product and its gated
// form (lora_base.hip), and rotary positions (lora_rotary.hip).  Not installed;
// not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora_internal.h"

namespace lora {

// ---------------------------------------------------------------------------
// 4-bit base weights
//
// A weight block is 16 output columns x 128 inputs, 1 KB: lane l = 16 g + n of
// the wave that reads it holds column n, inputs 32 j + 8 g .. + 7 in its word
// j = 0..3, the order in which v_mfma_f32_16x16x32_bf16 takes its right operand.
// A word holds the even inputs in nibbles 0..3 and the odd ones in nibbles 4..7,
// so that one mask gives a pair of neighbours in the halves of a register.
// Blocks are stored column block by column block, their K blocks in order.
// Beside each block stand the scales of its columns, `spb` per block and column
// (a group of 32 or 64 inputs has 4 or 2, every longer one 1): in a bf16 ctx one
// 32-bit word, the scale's upper 24 bits (16 significant bits, exact for scales
// that came from 16-bit floats) over the byte 16 + zero; in an fp32 ctx two
// floats, the scale and 16 + zero.  Columns past d_out and groups past d_in have
// scale 0.
constexpr int kBaseCols = 16;
constexpr int kBaseK = 128;
// Largest d_in of a base weight: a workgroup's rows of x (64 of 4 bytes an input) and
// a column block's weights are addressed by 31-bit offsets.
constexpr int kBaseMaxIn = 1 << 22;

struct BasePack {
    uint32_t *q = nullptr;       // [col blocks][K blocks][64][4]
    void *scales[3] = {};        // for 1, 2 and 4 scales a block: [col blocks][K blocks][16][spb] words
                                 // (fp32: pairs of floats); each stays where it is, so that a graph
                                 // captured on it finds the scales of every later load of its kind
    void *bias = nullptr;        // [d_out], ctx dtype
    int32_t spb = 0;             // 0: no weight loaded
    bool has_bias = false;
    void *&sc(int of) { return scales[of >> 1]; }
    void *sc() const { return scales[spb >> 1]; }
    bool zero = false;           // loaded with zero points (else all are 8), and the same
    uint32_t *has_zero = nullptr;   // in a device word behind q, for captured launches
};

struct BasePackArgs {
    const uint8_t *q;            // rows x d_in / 2
    const float *scale;          // rows x groups
    const uint8_t *zero;         // rows x groups, or null (8)
    uint32_t *q_out;             // the first of the rows' column blocks
    void *sc_out;
    uint32_t *has_zero;          // set to whether there are zero points
    int32_t rows;                // rows given; the rest of the last column block is padding
    int32_t d_in, group, groups, spb;
};
hipError_t launch_base_pack(bool bf16, const BasePackArgs &a, hipStream_t st);

struct BaseMember {
    const uint32_t *q;
    const void *sc;
    const void *bias;            // or null
    const void *x;               // [T][d_in]
    const void *add;             // [T][d_out] or null
    void *y;                     // [T][d_out]
    int32_t d_in, d_out;
    int32_t kb;                  // K blocks
    const uint32_t *has_zero;    // device word: 1 if loaded with zero points, else all are 8
};

// Where every zero point is 8 the products leave a multiplication per sum out.  A launch
// into a graph may be replayed after a reload that brings zero points: it asks the device
// word, a dependent load at its start (calls in a graph, without zero points: 64 tokens of
// 4096 -> 4096 9.4 us against 9.0, from 128 tokens on the same).
enum Zeros : int32_t { kZerosNone, kZerosSome, kZerosAsk };

struct BaseArgs {
    BaseMember m[kMaxGroup];     // gated: m[0] gate, m[1] up, y in m[0]
    int32_t tile_start[kMaxGroup + 1];  // column tiles of the members before member i, and
    int32_t items;                      // work items (both set by the launch)
    int32_t n;
    int32_t T;
    int32_t act;                 // gated: LORA_ACT_*
    Zeros zeros;
};
// All members share spb.
hipError_t launch_base(bool bf16, bool gated, int spb, const BaseArgs &a, hipStream_t st);

// ---------------------------------------------------------------------------
// rotary positions

struct RotaryMember {
    const void *x;
    void *y;
    int32_t heads;
    int32_t width;               // heads * head_dim
};

struct RotaryArgs {
    lora_rotary rot;
    RotaryMember m[kMaxGroup];
    int32_t n;
    int32_t T;
    int32_t total_heads;
    const int32_t *positions;
};
hipError_t launch_rotary(bool bf16, bool vec, const RotaryArgs &a, hipStream_t st);

}  // namespace lora
