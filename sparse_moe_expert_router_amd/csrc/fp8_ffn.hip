// Dispatch of the W8A8 products: dense (moe_fp8_matmul) and grouped experts
// (moe_grouped_ffn_a8).
#include "ffn_internal.h"
#include "fp8.h"
#include "fp8_internal.h"

namespace moe {

hipError_t launch_fp8_matmul(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int M, int N, int K,
                             int64_t lda, int64_t ldw, int out_f32, void* y, int64_t ldy, hipStream_t s) {
    Fp8Dense p{a, sa, w, sw, M, N, K, lda, ldw, ldy, y, out_f32, 0};
    const int v = out_f32 ? 16 : 8;
    p.vec = (uintptr_t)y % v == 0 && ldy % 4 == 0;
    return launch_fp8_skinny(p, s);
}

// Workspace of a grouped call, in order: tile table, quantised rows and
// scales, quantised SwiGLU products and scales; every region 256-byte aligned.
static size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Row tiles of BM rows over E experts: at most one partial tile per expert.
static size_t a8_max_tiles(long P, int E, int BM) { return (size_t)(P / BM + (P < E ? P : E)); }

constexpr int kA8Rows = 16;  // rows of a tile

size_t ffn_a8_ws_bytes(int T, int k, int E, int H, int F) {
    const long P = (long)T * k;
    return up256((1 + 2 * a8_max_tiles(P, E, kA8Rows)) * sizeof(int32_t)) + up256((size_t)T * H) +
           up256((size_t)T * fp8_blocks(H) * 4) + up256((size_t)P * F) + up256((size_t)P * fp8_blocks(F) * 4);
}

hipError_t launch_ffn_a8(const FfnArgs& f, void* ws, hipStream_t s) {
    Fp8Ffn p{};
    p.T = f.T; p.k = f.k; p.H = f.H; p.F = f.F; p.P = f.T * f.k;
    p.E = f.offsets ? f.E : 1;
    p.offsets = f.offsets;
    p.sorted_pair = f.sorted_pair;
    p.gate = f.ex->gate.codes; p.up = f.ex->up.codes; p.down = f.ex->down.codes;
    p.sgate = f.ex->gate.block_scales; p.sup = f.ex->up.block_scales; p.sdown = f.ex->down.block_scales;
    p.rows = f.rows;
    p.out_f32 = f.out_f32;
    const size_t mt = a8_max_tiles(p.P, p.E, kA8Rows);
    char* w = static_cast<char*>(ws);
    int32_t* tiles = reinterpret_cast<int32_t*>(w);
    w += up256((1 + 2 * mt) * sizeof(int32_t));
    uint8_t* xq = reinterpret_cast<uint8_t*>(w);
    w += up256((size_t)p.T * p.H);
    float* xs = reinterpret_cast<float*>(w);
    w += up256((size_t)p.T * (p.H / 128) * 4);
    p.hq = reinterpret_cast<uint8_t*>(w);
    w += up256((size_t)p.P * p.F);
    p.hs = reinterpret_cast<float*>(w);
    p.tiles = tiles; p.xq = xq; p.xs = xs;
    launch_tile_table(p.offsets, p.E, p.P, kA8Rows, tiles, s);
    hipError_t err = launch_fp8_quantize(f.x, 0, p.T, p.H, p.H, xq, xs, s);
    if (err != hipSuccess) return err;
    return launch_fp8_skinny_ffn(p, (int)mt, s);
}

}  // namespace moe
