// Internal interface of the W8A8 kernels (fp8_skinny.hip, fp8_gemm.hip, fp8_ffn.hip).
#pragma once

#include "kernels.h"

namespace moe {

// y [M][N] = (a . sa) (w . sw)^T; leading dimensions in elements.
struct Fp8Dense {
    const uint8_t* a;   // [M][K], row stride lda
    const float* sa;    // [M][ceil(K/128)]
    const uint8_t* w;   // [N][K], row stride ldw
    const float* sw;    // [ceil(N/128)][ceil(K/128)]
    int M, N, K;
    int64_t lda, ldw, ldy;
    void* y;
    int out_f32;
    int vec;            // 1: y's base and stride allow 16-byte stores (and those of four neighbouring outputs)
};

// Grouped SwiGLU experts on quantised rows.
struct Fp8Ffn {
    int T, k, H, F, E, P;
    const int32_t* offsets;      // [E+1] or nullptr (identity: E == 1)
    const int32_t* sorted_pair;  // [P] or nullptr
    const int32_t* tiles;        // tiles[0] = count, then (expert, first row, end row) triples
    const uint8_t *gate, *up, *down;
    const float *sgate, *sup, *sdown;
    const uint8_t* xq;           // [T][H]
    const float* xs;             // [T][H/128]
    uint8_t* hq;                 // [P][F]
    float* hs;                   // [P][F/128]
    void* rows;                  // [P][H]
    int out_f32;
};

hipError_t launch_fp8_skinny(const Fp8Dense& p, hipStream_t s);
long fp8_skinny_workgroups(int M, int N);

// Tiles of bt rows (256, 128 or 64; fp32 outputs 128 or 64) x 256 outputs.
hipError_t launch_fp8_gemm(const Fp8Dense& d, int bt, hipStream_t s);
hipError_t launch_fp8_gemm_gateup(const Fp8Ffn& p, int bt, long max_tiles, hipStream_t s);
// The most workgroups of a pass that takes one a tile (0: both passes take runs of tiles).
long fp8_grouped_workgroups(int H, int F, long max_tiles);
hipError_t launch_fp8_gemm_down(const Fp8Ffn& p, int bt, long max_tiles, hipStream_t s);

}  // namespace moe
