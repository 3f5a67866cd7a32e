// Dispatch of the W8A8 products: dense (moe_fp8_matmul) and grouped experts
// (moe_grouped_ffn_a8).
#include "ffn_internal.h"
#include "fp8.h"
#include "fp8_internal.h"

namespace moe {

// Dense products up to this many rows stream the weights (fp8_skinny.hip).
constexpr int kSkinnyRows = 128;

// Rows of a dense tile: the largest that still gives every compute unit one.
static int dense_bt(int M, int N) {
    const long nt = (N + 255) / 256;
    if ((M + 255) / 256 * nt >= 256) return 256;
    if ((M + 127) / 128 * nt >= 128) return 128;
    return 64;
}

hipError_t launch_fp8_matmul(const uint8_t* a, const float* sa, const uint8_t* w, const float* sw, int M, int N, int K,
                             int64_t lda, int64_t ldw, int out_f32, void* y, int64_t ldy, hipStream_t s) {
    Fp8Dense p{a, sa, w, sw, M, N, K, lda, ldw, ldy, y, out_f32, 0};
    p.vec = (uintptr_t)y % 16 == 0 && ldy % (out_f32 ? 4 : 8) == 0;
    if (M <= kSkinnyRows) return launch_fp8_skinny(p, s);
    return launch_fp8_gemm(p, dense_bt(M, N), s);
}

// Workspace of a grouped call, in order: tile table, quantised rows and
// scales, quantised SwiGLU products and scales; every region 256-byte aligned.
static size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Row tiles of at most bt rows over E experts: at most one partial tile per expert.
static size_t a8_max_tiles(long P, int E, int bt) { return (size_t)(P / bt + (P < E ? P : E)); }

// Rows of a tile by the average rows of an expert that has any: 16 (the
// streaming kernels) to 256.
static int a8_bt(long P, int E) {
    const long avg = P / (P < E ? P : E);
    return avg >= 160 ? 256 : avg >= 80 ? 128 : avg >= 24 ? 64 : 16;
}

static size_t a8_tiles_bytes(long P, int E, int bt) { return up256((1 + 3 * a8_max_tiles(P, E, bt)) * sizeof(int32_t)); }

// Tile table: tiles[0] = number of tiles, then (expert, first row, end row).
// An expert with n rows gets ceil(n / bt) tiles of equal size, rounded up to
// 16 rows (the last one shorter).  Offsets that do not ascend from 0 to P may
// ask for more tiles than the table holds; those are left out.
__global__ __launch_bounds__(1024) void a8_tile_table_kernel(const int32_t* __restrict__ offsets, int E, int P, int bt,
                                                             int most, int32_t* __restrict__ tiles) {
    __shared__ int scan[1024];
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
    for (int off = 1; off < 1024; off <<= 1) {
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
    if (e == 1023) tiles[0] = min(scan[1023], most);
}

// Grows with T: the tile table is sized for 16-row tiles throughout.
size_t ffn_a8_ws_bytes(int T, int k, int E, int H, int F) {
    const long P = (long)T * k;
    return a8_tiles_bytes(P, E, 16) + up256((size_t)T * H) + up256((size_t)T * fp8_blocks(H) * 4) +
           up256((size_t)P * F) + up256((size_t)P * fp8_blocks(F) * 4);
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
    const int bt = a8_bt(p.P, p.E);
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
    hipLaunchKernelGGL(a8_tile_table_kernel, dim3(1), dim3(1024), 0, s, p.offsets, p.E, p.P, bt, (int)mt, tiles);
    hipError_t err = launch_fp8_quantize(f.x, 0, p.T, p.H, p.H, xq, xs, s);
    if (err != hipSuccess) return err;
    if (bt == 16) return launch_fp8_skinny_ffn(p, (int)mt, s);
    err = launch_fp8_gemm_gateup(p, bt, mt, s);
    if (err != hipSuccess) return err;
    return launch_fp8_gemm_down(p, bt, mt, s);
}

}  // namespace moe
