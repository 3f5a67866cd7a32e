// Dispatch of the W8A8 products: dense (moe_fp8_matmul) and grouped experts
// (moe_grouped_ffn_a8).
#include <limits.h>

#include "ffn_internal.h"
#include "fp8.h"
#include "fp8_internal.h"

namespace moe {

// Workgroups of 512 threads that a launch holds: fewer than 2^32 threads, and
// tiles come in whole eighths (one an XCD).
constexpr long kMaxWorkgroups = (1l << 23) - 8;

// Whether a dense product streams the weights (fp8_skinny.hip): while all of its
// workgroups, 16 outputs x 32 rows each, are resident at once (two a compute
// unit); beyond that they read rows and weights too often.  With very few rows
// there is nothing but the weights to read.  Measured, streaming / 64-row tiles,
// us: 96 x 2560 x 2560 (480 workgroups) 11.7 / 15.6, 128 rows (640) 16.4 / 15.6;
// 32 x 8192 x 8192 (512) 31 / 38, 64 rows (1024) 59 / 38; 512 x 512 x 2560 (512)
// 11.8 / 15.6; 16384 x 8192 (1024), one row 26 / 38, 16 rows 40 / 38.  With fp32
// outputs the tiles take nearly twice as long, streaming the same: 64 x 8192 x
// 8192 (1024) 61 / 71, 96 rows (1536) 89 / 72; 256 x 2560 x 2560 (1280) 26.7 / 27.0.
static bool dense_streams(int M, int N, int out_f32) {
    const long wgs = fp8_skinny_workgroups(M, N);
    return (M <= 8 && wgs <= kMaxWorkgroups) || wgs <= (out_f32 ? 1024 : 512);
}

// Rows of a dense tile.  256 tiles run at once, and such a round takes times as
// 10 : 16 : 24 for tiles of 64, 128 and 256 rows (8192 x 8192: 512 rows 46 us,
// 1024 77, 2048 117); the fewest of these units wins.  (4096 x 2560 x 2560: 3
// rounds of 64 rows 48.6 us, 2 of 128 50.5, 1 of 256 41.4; 1024 x 2560 x 2560, one
// round of any: 17.7, 24.5, 36.4.)  fp32 outputs have the first two: 1024 x 8192 x
// 8192 in 2 rounds of 64 rows 156 us, one of 128 124; 512 rows 83, 113.
static int dense_bt(int M, int N, int out_f32) {
    const long nt = ((long)N + 255) / 256;
    auto cost = [&](long rows, long round) { return ((M + rows - 1) / rows * nt + 255) / 256 * round; };
    const long c64 = cost(64, 10), c128 = cost(128, 16), c256 = out_f32 ? LONG_MAX : cost(256, 24);
    return c64 <= c128 && c64 <= c256 ? 64 : c128 <= c256 ? 128 : 256;
}

bool fp8_matmul_fits(int M, int N, int out_f32) {
    if (dense_streams(M, N, out_f32)) return true;
    const long bt = dense_bt(M, N, out_f32);
    return ((long)M + bt - 1) / bt * (((long)N + 255) / 256) <= kMaxWorkgroups;
}

hipError_t launch_fp8_matmul(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int M, int N, int K,
                             int64_t lda, int64_t ldw, int out_f32, void* y, int64_t ldy, hipStream_t s) {
    Fp8Dense p{a, sa, w, sw, M, N, K, lda, ldw, ldy, y, out_f32, 0};
    p.vec = (uintptr_t)y % 16 == 0 && ldy % (out_f32 ? 4 : 8) == 0;
    if (dense_streams(M, N, out_f32)) return launch_fp8_skinny(p, s);
    return launch_fp8_gemm(p, dense_bt(M, N, out_f32), s);
}

// Workspace of a grouped call, in order: tile table, quantised rows and
// scales, quantised SwiGLU products and scales; every region 256-byte aligned.
static size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Row tiles of at most bt rows over E experts: at most one partial tile per expert.
static size_t a8_max_tiles(long P, int E, int bt) { return (size_t)(P / bt + (P < E ? P : E)); }

// Rows of a tile.  64 while an expert with rows has fewer on average, and also
// while all tiles run at once; 256 from 160 rows on average, where that still
// makes four rounds of 256 tiles, so that the last one's unevenness counts little.
// Measured with hidden 2560, inter 640, tiles of 64 / 128 / 256 rows, us.  Rows on
// average over 64 experts: 8 79 / 91 / 128, 48 92 / 101 / 136, 80 112 / 109 / 142, 128
// 140 / 119 / 150, 320 234 / 202 / 226; over 256: 64 330 / 295 / 380, 128 446 / 397 /
// 412, 192 583 / 491 / 442, 256 702 / 601 / 617, 384 1008 / 827 / 807, 640 1507 / 1251
// / 1199, 1280 2863 / 2332 / 2160.  Hidden 4096, inter 1152, over 8 experts: 128 rows
// 56 / 61 / 83, 512 131 / 122 / 114, 1024 217 / 193 / 203.  (How a tile's size divides
// an expert's rows matters as much as it: at 256 rows over 256 experts the rule is 3 %
// off the best, at 512 over 8 experts 7 %.)  One row per expert, where the bytes of
// the touched experts' weights need less than the steps of a tile: 1 token of ten
// experts 31 / 40 / 58, its bytes 10; 16 tokens 136 / 150 / 219, its bytes 137.  fp32
// rows (exact products) have the first two, us: over 512 experts 5 rows on average
// 496 / 688, 80 932 / 790; over 256 128 605 / 582, 1280 4497 / 3757.
static int a8_bt(long P, int E, int F, int out_f32) {
    const long active = P < E ? P : E, avg = P / active, cols = F / 128;
    auto tiles = [&](long rows) { return (P / rows + active / 2) * cols; };
    if (avg < 64 || tiles(64) <= 256) return 64;
    return !out_f32 && avg >= 160 && tiles(256) >= 1024 ? 256 : 128;
}

static size_t a8_tiles_bytes(long P, int E, int bt) { return up256((1 + 3 * a8_max_tiles(P, E, bt)) * sizeof(int32_t)); }

constexpr int kPrepThreads = 1024;  // at least the most experts

// Tile table: tiles[0] = number of tiles, then (expert, first row, end row).
// An expert with n rows gets ceil(n / bt) tiles of equal size, rounded up to
// 16 rows (the last one shorter).  Offsets that do not ascend from 0 to P may
// ask for more tiles than the table holds; those are left out.
__device__ __forceinline__ void a8_tile_table(const int32_t* __restrict__ offsets, int E, int P, int bt, int most,
                                              int32_t* __restrict__ tiles) {
    __shared__ int scan[kPrepThreads];
    const int e = threadIdx.x;
    int cnt = 0, r0 = 0;
    if (offsets) {
        if (e < E) {
            r0 = min(max(offsets[e], 0), P);
            cnt = min(max(offsets[e + 1], r0), P) - r0;
        }
    } else if (e == 0) {
        cnt = P;
    }
    const int nt = (cnt + bt - 1) / bt;
    const int sz = nt ? ((cnt + nt - 1) / nt + 15) / 16 * 16 : 0;
    scan[e] = nt;
    __syncthreads();
    for (int off = 1; off < kPrepThreads; off <<= 1) {
        const int v = e >= off ? scan[e - off] : 0;
        __syncthreads();
        scan[e] += v;
        __syncthreads();
    }
    const int start = scan[e] - nt;
    for (int i = 0; i < nt && start + i < most; ++i) {
        tiles[1 + 3 * (start + i)] = e;
        tiles[2 + 3 * (start + i)] = r0 + i * sz;
        tiles[3 + 3 * (start + i)] = min(r0 + (i + 1) * sz, r0 + cnt);
    }
    if (e == kPrepThreads - 1) tiles[0] = min(scan[kPrepThreads - 1], most);
}

// What the products need first, in one launch: workgroup 0 writes the tile table,
// the others quantise x.  (Against two launches, 16 tokens of 512 experts: 137.2
// -> 134.3 us, 4096 tokens 580 -> 577, 32768 tokens of 256 no difference: between
// the experts' passes the quantiser takes 58 us in either launch.)
__global__ __launch_bounds__(kPrepThreads) void a8_prepare_kernel(const Fp8Ffn p, const uint16_t* __restrict__ x, int bt, int most,
                                                                  int32_t* __restrict__ tiles, uint8_t* __restrict__ xq,
                                                                  float* __restrict__ xs) {
    if (blockIdx.x == 0) {
        a8_tile_table(p.offsets, p.E, p.P, bt, most, tiles);
    } else {
        const int nb = p.H / 128;
        fp8_quantize_piece<false>((blockIdx.x - 1) * (uint32_t)kPrepThreads + threadIdx.x, x, (uint32_t)p.T * 8u * (uint32_t)nb, p.H,
                                  nb, p.H, xq, xs);
    }
}

// Grows with T: the tile table is sized for 64-row tiles throughout.
size_t ffn_a8_ws_bytes(int T, int k, int E, int H, int F) {
    const long P = (long)T * k;
    return a8_tiles_bytes(P, E, 64) + up256((size_t)T * H) + up256((size_t)T * fp8_blocks(H) * 4) +
           up256((size_t)P * F) + up256((size_t)P * fp8_blocks(F) * 4);
}

bool ffn_a8_fits(const FfnArgs& f) {
    const long P = (long)f.T * f.k;
    const int E = f.offsets ? f.E : 1;
    return fp8_grouped_workgroups(f.H, f.F, (long)a8_max_tiles(P, E, a8_bt(P, E, f.F, f.out_f32))) <= kMaxWorkgroups;
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
    const int bt = a8_bt(p.P, p.E, p.F, p.out_f32);
    const long mt = (long)a8_max_tiles(p.P, p.E, bt);
    char* w = static_cast<char*>(ws);
    int32_t* tiles = reinterpret_cast<int32_t*>(w);
    w += a8_tiles_bytes(p.P, p.E, bt);
    uint8_t* xq = reinterpret_cast<uint8_t*>(w);
    w += up256((size_t)p.T * p.H);
    float* xs = reinterpret_cast<float*>(w);
    w += up256((size_t)p.T * (p.H / 128) * 4);
    p.hq = reinterpret_cast<uint8_t*>(w);
    w += up256((size_t)p.P * p.F);
    p.hs = reinterpret_cast<float*>(w);
    p.tiles = tiles; p.xq = xq; p.xs = xs;
    const uint32_t pieces = (uint32_t)p.T * (uint32_t)(p.H / 16);
    hipLaunchKernelGGL(a8_prepare_kernel, dim3(1 + (pieces + kPrepThreads - 1) / kPrepThreads), dim3(kPrepThreads), 0, s, p, f.x,
                       bt, (int)mt, tiles, xq, xs);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    err = launch_fp8_gemm_gateup(p, bt, mt, s);
    if (err != hipSuccess) return err;
    return launch_fp8_gemm_down(p, bt, mt, s);
}

}  // namespace moe
