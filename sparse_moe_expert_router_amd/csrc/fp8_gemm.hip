// W8A8 products for many rows: tiles of 32 TF rows x 256 outputs on gfx950's
// 16 x 16 x 128 FP8 MFMA (fp32 outputs: the bf16 MFMA on widened codes, see
// mfma_fp8), scales per 128 inputs applied in fp32 after every block:
//   acc[n][m] += (sa[m][kb] * sw[n / 128][kb]) * sum_{i in kb} w[n][i] a[m][i].
// Three uses: a dense product, the gate/up pass of the grouped experts (a
// tile holds 128 gate and the same 128 up columns; SwiGLU and quantisation in
// the epilogue) and their down pass.
//
// A workgroup is 8 waves, 4 along the outputs x 2 along the rows; a wave owns
// 64 outputs x 16 TF rows.  One step is one block of 128 inputs.  Rows and
// weights both go from memory straight into LDS (16-byte buffer loads to LDS),
// 128 bytes a row, 16-byte pieces XOR-swizzled, and from there into MFMA
// operands; the row scales are staged in LDS eight steps at a time.  (Weights
// loaded straight into operand registers measured slower: neighbouring lanes
// then read different rows, 64 cache accesses an instruction, and the cache's
// one access a cycle bounded the kernel: 8192^3 in 676 us.)
// The weights are the MFMA's row operand, so a lane ends up with outputs of one
// row and one row scale covers them.  A product gives a lane 4 neighbouring
// operand rows; the weights are laid into LDS in an order (g_order) that makes
// two products of a lane 8 neighbouring outputs, 16 bytes of bf16.
//
// Pipeline: one barrier M_j in the middle of each step j.  A wave holds step
// j's weights in registers (read at the end of step j - 1), so M_j ends the
// use of their LDS stage, of the first half of step j's rows and of the second
// half of step j - 1's.  After M_j the wave issues the loads that refill these,
// of S steps later (S stages); they are waited for at M_{j + S - 1}, so every
// load has S - 1 whole steps to land and nothing stops at the step's border.
//
// Measured: 8192 x 8192 x 8192 in 477 to 505 us by the card, 2.18 to 2.30 PFLOP/s;
// 32768 tokens to 10 of 256 experts (hidden 2560, inter 640): gate/up 1260 us, 1.70
// PFLOP/s, down 820 us, of which its 1.7 GB of rows need 340.  The MFMA is busy 54,
// 44 and 34 % of the cycles, other vector instructions 35, 40 and 27 % (1.93 GHz
// under this load): every 128 products of an output need an fp32 multiply-add
// outside it.  Gate/up spends about 35 us on SwiGLU and 48 on the quantisation, and
// both passes compute the rows that pad each expert's last tile.  In down, with
// five steps a tile, the matrix cores also stand still while all waves convert and
// store a tile together.
#include "fp8.h"
#include "ffn_internal.h"
#include "fp8_internal.h"

namespace moe {

enum { G_DENSE = 0, G_GATEUP = 1, G_DOWN = 2 };

constexpr int kGThreads = 512;
constexpr int kGN = 256;       // outputs of a tile (gate/up: 128 of each)
// LDS of a tile of BT rows, in bytes.
template <int TF>
struct GemmLds {
    static constexpr int BT = 32 * TF;
    static constexpr int S = TF >= 8 ? 2 : 3;            // stages
    static constexpr int A = BT * 128;                   // one stage of rows
    static constexpr int B = kGN * 128;                  // one stage of weights
    static constexpr int W = S * A;                      // weights [S][256][128]
    static constexpr int SA = W + S * B;                 // row scales [2][8][BT]
    static constexpr int SW = SA + 2 * 8 * BT * 4;       // weight scales [2][2][8]
    static constexpr int ROW = SW + 2 * 2 * 8 * 4;       // byte offsets of the rows' scales [BT]
    static constexpr int AMAX = ROW + BT * 4;            // gate/up: group maxima [4][BT]
    static constexpr int TOTAL = AMAX + 4 * BT * 4;
    static_assert(TOTAL <= 160 * 1024, "LDS of a compute unit");
};

// 16-byte piece c of row r sits at piece c ^ g_swz(r).  A 16-byte LDS read
// serves 16 lanes at a time, not always neighbouring ones; this swizzle keeps
// rows 0..15 of one piece on different banks, and also rows 0-3, 12-15 of one
// piece beside rows 4-11 of the next.
__device__ __forceinline__ int g_swz(int r) { return (r >> 1) & 7; }

// Weight row (of a group of 32) at LDS row r: product (r / 16) of the pair,
// operand row i = r % 16 = 4 g + j, holds output 8 g + 4 (r / 16) + j.
__device__ __forceinline__ int g_order(int r) {
    const int i = r & 15;
    return (r & ~31) + 8 * (i >> 2) + 4 * ((r >> 4) & 1) + (i & 3);
}

typedef __attribute__((address_space(3))) void lds_void;

// A load of 16 (4) bytes a lane from memory to LDS: lane i's land at lds + 16 i (4 i).
__device__ __forceinline__ void load16_lds(const void* base, uint32_t bytes, uint8_t* lds, uint32_t voff, int soff) {
    const __amdgpu_buffer_rsrc_t r = fp8_rsrc(base, bytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, (int)voff, soff, 0, 0);
}
__device__ __forceinline__ void load4_lds(const void* base, uint32_t bytes, void* lds, uint32_t voff, int soff) {
    const __amdgpu_buffer_rsrc_t r = fp8_rsrc(base, bytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 4, (int)voff, soff, 0, 0);
}

// Waits until at most n of the wave's memory loads are under way, and for its
// LDS reads; then for the other waves.
template <int n>
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(n) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Eight neighbouring outputs of a row, rounded once, in 16-byte stores.
__device__ __forceinline__ void store8(void* row, int out_f32, int n, f32x4_t a, f32x4_t b) {
    if (out_f32) {
        f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(row) + n);
        o[0] = a;
        o[1] = b;
    } else {
        const u32x4_t o = {pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(row) + n) = o;
    }
}

// The sums of the first n groups of rows are final here.  Without it the compiler
// moves additions, with all their operands, past the branches that follow, which
// costs 40 registers a lane.
template <int TF>
__device__ __forceinline__ void hold(f32x4_t (&acc)[4][TF], int n) {
#pragma unroll
    for (int t = 0; t < n; ++t)
#pragma unroll
        for (int f = 0; f < 4; ++f) asm volatile("" : "+v"(acc[f][t]));
}

template <int TF, int MODE, bool kExact>
__global__ __launch_bounds__(kGThreads, 2) void fp8_gemm_kernel(const Fp8Dense d, const Fp8Ffn p) {
    using L = GemmLds<TF>;
    constexpr int BT = L::BT;
    constexpr int S = L::S;
    constexpr int NA = BT / 64;   // row loads of a wave per step; 4 weight loads
    constexpr int NL = NA + 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv & 3, wt = wv >> 2, g = lane >> 4, l16 = lane & 15;

    // ---- the tile: rows [m0, m1), outputs from n0
    int e = 0, m0, m1, n0;
    if (MODE == G_DENSE) {
        const int mt = (d.M + BT - 1) / BT, nt = (d.N + kGN - 1) / kGN;
        const int l = xcd_remap(blockIdx.x, mt * nt);
        if (l < 0) return;
        // groups of 4 row tiles, all output tiles of a group in turn
        const int grp = l / (4 * nt), rem = l - grp * 4 * nt, gm = min(4, mt - 4 * grp);
        m0 = (4 * grp + rem % gm) * BT;
        n0 = rem / gm * kGN;
        m1 = min(m0 + BT, d.M);
    } else {
        const int nt = MODE == G_GATEUP ? p.F / 128 : (p.H + kGN - 1) / kGN;
        const int l = xcd_remap(blockIdx.x, p.tiles[0] * nt);
        if (l < 0) return;
        const int i = l / nt;
        n0 = (l - i * nt) * (MODE == G_GATEUP ? 128 : kGN);
        e = p.tiles[1 + 3 * i];
        m0 = p.tiles[2 + 3 * i];
        m1 = min(p.tiles[3 + 3 * i], p.P);
        if (m0 < 0 || m0 >= m1) return;
    }
    const int K = MODE == G_DENSE ? d.K : MODE == G_GATEUP ? p.H : p.F;
    const int KB = (K + 127) / 128;
    const int N = MODE == G_DENSE ? d.N : MODE == G_GATEUP ? p.F : p.H;
    const int mr = m1 - m0;
    const bool tail = MODE == G_DENSE && K % 128 != 0;  // the last block is shorter

    // ---- buffers
    const uint32_t lda = MODE == G_DENSE ? (uint32_t)d.lda : (uint32_t)K;
    const uint32_t ldw = MODE == G_DENSE ? (uint32_t)d.ldw : (uint32_t)K;
    const __amdgpu_buffer_rsrc_t ra =
        MODE == G_DENSE    ? fp8_rsrc(d.a + (size_t)m0 * lda, (uint32_t)(min(mr, BT) - 1) * lda + (uint32_t)K)
        : MODE == G_GATEUP ? fp8_rsrc(p.xq, (uint32_t)p.T * (uint32_t)K)
                           : fp8_rsrc(p.hq + (size_t)m0 * K, (uint32_t)mr * (uint32_t)K);
    const __amdgpu_buffer_rsrc_t rs =
        MODE == G_DENSE    ? fp8_rsrc(d.sa + (size_t)m0 * KB, (uint32_t)min(mr, BT) * (uint32_t)KB * 4u)
        : MODE == G_GATEUP ? fp8_rsrc(p.xs, (uint32_t)p.T * (uint32_t)KB * 4u)
                           : fp8_rsrc(p.hs + (size_t)m0 * KB, (uint32_t)mr * (uint32_t)KB * 4u);
    const uint32_t wrows = MODE == G_GATEUP ? 128u : (uint32_t)min(N - n0, kGN);
    const uint32_t wbytes = (wrows - 1) * ldw + (uint32_t)K;
    const size_t wbase = MODE == G_DENSE ? (size_t)n0 * ldw : ((size_t)e * N + n0) * K;
    const __amdgpu_buffer_rsrc_t rw0 = fp8_rsrc((MODE == G_DENSE ? d.w : MODE == G_GATEUP ? p.gate : p.down) + wbase, wbytes);
    const __amdgpu_buffer_rsrc_t rw1 = MODE == G_GATEUP ? fp8_rsrc(p.up + wbase, wbytes) : rw0;
    // two rows of weight scales: the gate's and the up's, or those of the tile's two blocks of 128 outputs
    const int NB = (N + 127) / 128;
    const size_t sbase = ((size_t)e * NB + n0 / 128) * KB;
    const uint32_t sbytes = (uint32_t)KB * 4u;
    const __amdgpu_buffer_rsrc_t rsw0 =
        fp8_rsrc((MODE == G_DENSE ? d.sw : MODE == G_GATEUP ? p.sgate : p.sdown) + sbase, sbytes);
    const __amdgpu_buffer_rsrc_t rsw1 =
        MODE == G_GATEUP ? fp8_rsrc(p.sup + sbase, sbytes)
                         : fp8_rsrc((MODE == G_DENSE ? d.sw : p.sdown) + sbase + (n0 / 128 + 1 < NB ? KB : 0), sbytes);

    // ---- loads: load i of wave wv fills rows 8 (8 i + wv) .. +7 of a stage,
    // lane = 8 (row % 8) + piece position; the piece read is position ^ g_swz(row)
    const int lr = 8 * wv + (lane >> 3), piece = (lane & 7) ^ g_swz(lr);  // g_swz: the same for rows 64 apart
    auto source_row = [&](int r) {  // row of the source matrix (relative to its base) behind row r of the tile
        if (MODE == G_DENSE) return (uint32_t)r;
        const int q = min(r, mr - 1);
        if (MODE == G_DOWN) return (uint32_t)q;
        return (uint32_t)(p.sorted_pair ? min(max(p.sorted_pair[m0 + q] / p.k, 0), p.T - 1) : m0 + q);
    };
    uint32_t aoff[NA];
#pragma unroll
    for (int i = 0; i < NA; ++i) aoff[i] = source_row(64 * i + lr) * lda + 16u * (uint32_t)piece;
    // weight rows 64 i + lr; gate/up: 0..127 the gate's, 128..255 the up's
    const uint32_t woff = (uint32_t)g_order(lr) * ldw + 16u * (uint32_t)piece;
    uint32_t* rowoff = reinterpret_cast<uint32_t*>(smem + L::ROW);
    for (int r = tid; r < BT; r += kGThreads)
        rowoff[r] = (MODE == G_DENSE && r >= mr) ? kOob : source_row(r) * (uint32_t)KB * 4u;
    const bool cut = tail && 16 * piece >= K - (KB - 1) * 128;  // nothing of the lane's piece in the last block

    auto load_w = [&](int i, int j) {
        uint8_t* st = smem + L::W + (j % S) * L::B;
        j = min(j, KB - 1);
        uint32_t off = woff + (uint32_t)(MODE == G_GATEUP ? i & 1 : i) * 64u * ldw;
        if (tail && j == KB - 1) off = cut ? kOob : off;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(MODE == G_GATEUP && i >= 2 ? rw1 : rw0,
                                                 (lds_void*)(st + (8 * i + wv) * 1024), 16, (int)off, j * 128, 0, 0);
    };
    auto load_a = [&](int i, int j) {
        uint8_t* st = smem + (j % S) * L::A;
        j = min(j, KB - 1);
        uint32_t off = aoff[i];
        if (tail && j == KB - 1) off = cut ? kOob : off;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void*)(st + (8 * i + wv) * 1024), 16, (int)off, j * 128, 0, 0);
    };
    // load n of the group issued after M_j: 4 of the weights of step j + S, then
    // the rows: first halves (of each row wave's rows) of step j + S, second
    // halves of step j + S - 1.  The first group of all has no second halves.
    auto load_group = [&](int n, int j) {
        if (n < 4) {
            load_w(n, j + S);
        } else {
            const int second = ((64 * (n - 4) + 8 * wv) / (8 * TF)) & 1;
            load_a(n - 4, max(j + S - second, 0));
        }
    };
    // scales of blocks 8 c .. 8 c + 7: wave v loads block 8 c + v of every row
    auto load_s = [&](int c) {
        const int kb = min(8 * c + wv, KB - 1);
        float* sa = reinterpret_cast<float*>(smem + L::SA) + (c & 1) * 8 * BT + wv * BT;
#pragma unroll
        for (int t = 0; t < NA; ++t)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void*)(sa + 64 * t), 4, (int)rowoff[64 * t + lane], kb * 4,
                                                     0, 0);
        if (wv < 2 && lane < 8) {
            float* sw = reinterpret_cast<float*>(smem + L::SW) + (c & 1) * 16 + wv * 8;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(wv ? rsw1 : rsw0, (lds_void*)sw, 4, min(8 * c + lane, KB - 1) * 4, 0,
                                                     0, 0);
        }
    };

    f32x4_t acc[4][TF];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int t = 0; t < TF; ++t) acc[f][t] = f32x4_t{};

    __syncthreads();  // rowoff
    load_s(0);
#pragma unroll
    for (int j = -S; j < 0; ++j)
#pragma unroll
        for (int n = 0; n < NL; ++n) load_group(n, j);

    // LDS offsets of the lane's two pieces of row l16 of the wave's rows, of
    // weight row l16 of its outputs, and of its scales
    const int x0 = 16 * (g ^ g_swz(l16)), x1 = 16 * ((g + 4) ^ g_swz(l16));
    const int ar = (wt * 16 * TF + l16) * 128;
    const int br = L::W + ((MODE == G_GATEUP ? 32 * wn : 64 * wn) + l16) * 128;
    const int sr0 = L::SA + (wt * 16 * TF + l16) * 4;
    const int sw0 = L::SW + (MODE != G_GATEUP && wn >= 2 ? 32 : 0);
    auto read_a = [&](int j, int t) {  // rows 16 t + l16 of step j
        const uint8_t* st = smem + (j % S) * L::A + ar + t * 2048;
        return join8(*reinterpret_cast<const i32x4_t*>(st + x0), *reinterpret_cast<const i32x4_t*>(st + x1));
    };
    auto read_w = [&](int j, int f) {
        const uint8_t* st = smem + (j % S) * L::B + br + (MODE == G_GATEUP && f >= 2 ? 128 + 16 * (f - 2) : 16 * f) * 128;
        return join8(*reinterpret_cast<const i32x4_t*>(st + x0), *reinterpret_cast<const i32x4_t*>(st + x1));
    };
    auto read_sa = [&](int j, int t) {
        return *reinterpret_cast<const float*>(smem + sr0 + (((j >> 3) & 1) * 8 + (j & 7)) * BT * 4 + t * 64);
    };
    auto read_sw = [&](int j, int half) {
        return *reinterpret_cast<const float*>(smem + sw0 + ((j >> 3) & 1) * 64 + (j & 7) * 4 + half * 32);
    };

    i32x8_t w[4], an;
    float sn, swn0, swn1 = 0.0f;
    auto read_first = [&](int j) {
        an = read_a(j, 0);
        sn = read_sa(j, 0);
        swn0 = read_sw(j, 0);
        if (MODE == G_GATEUP) swn1 = read_sw(j, 1);
    };
    wait_and_meet<(S - 1) * NL>();
#pragma unroll
    for (int f = 0; f < 4; ++f) w[f] = read_w(0, f);
    read_first(0);

    // One step: 4 TF products q = 4 t + f.  The order is fixed: product q is
    // issued, then product q - 2 (its MFMA done by then) is scaled and added,
    // so that the matrix cores and the vector units overlap within the wave.
    // Rows are read one group of 16 ahead, the next step's weights into each
    // register block after its last use.
    constexpr int kMeet = TF / 2 - 1;  // the group of rows before which the waves meet
    for (int j = 0; j < KB; ++j) {
        i32x8_t a;
        f32x4_t v[3];
        float c0[2], c1[2];   // scales of rows t in slot t & 1
        const float s0 = swn0, s1 = swn1;
        auto add = [&](int q) {
            const int t = q / 4, f = q % 4;
            const float c = MODE == G_GATEUP && f >= 2 ? c1[t & 1] : c0[t & 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[f][t][i] = fmaf(c, v[q % 3][i], acc[f][t][i]);
        };
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            if (t == kMeet) {
                hold(acc, kMeet);
                wait_and_meet<(S - 2) * NL>();
                if ((j & 7) == 0 && j + 8 < KB) load_s(j / 8 + 1);
            }
            a = an;
            c0[t & 1] = sn * s0;
            if (MODE == G_GATEUP) c1[t & 1] = sn * s1;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int q = 4 * t + f;
                v[q % 3] = mfma_fp8<kExact>(w[f], a);
                if (t + 1 == TF) w[f] = read_w(j + 1, f);
                if (f == 0) {
                    if (t + 1 < TF) {
                        an = read_a(j, t + 1);
                        sn = read_sa(j, t + 1);
                    } else {
                        read_first(j + 1);
                    }
                }
                if (q >= 4 * kMeet && q - 4 * kMeet < NL) load_group(q - 4 * kMeet, j);
                if (q >= 2) add(q - 2);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        add(4 * TF - 2);
        add(4 * TF - 1);
        hold(acc, TF);
    }
    wait_and_meet<0>();  // no load still writes LDS, no wave still reads it

    if constexpr (MODE == G_GATEUP) {
        // h = silu(gate) up in fp32; its largest magnitude per row over the
        // group's 128 columns: lanes of a row, then the 4 waves
        uint32_t* amax = reinterpret_cast<uint32_t*>(smem + L::AMAX);
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            uint32_t m = 0;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float h = silu(acc[f][t][i]) * acc[f + 2][t][i];
                    acc[f][t][i] = h;
                    m = max(m, abs_bits(h));
                }
            m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
            m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
            if (g == 0) amax[wn * BT + wt * 16 * TF + 16 * t + l16] = m;
        }
        __syncthreads();
        // codes [BT][128] through LDS (rows padded to 144 bytes), then 16 bytes a lane
        constexpr int LD = 144;
        static_assert(BT * LD <= L::SA, "codes fit the stages");
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            const int r = wt * 16 * TF + 16 * t + l16;
            const uint32_t m = max(max(amax[r], amax[BT + r]), max(amax[2 * BT + r], amax[3 * BT + r]));
            const float s = fp8_scale(m);
            const Fp8Div by = fp8_div(s);
            *reinterpret_cast<uint2*>(smem + r * LD + 32 * wn + 8 * g) =
                make_uint2(fp8_pack4(acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3], by),
                           fp8_pack4(acc[1][t][0], acc[1][t][1], acc[1][t][2], acc[1][t][3], by));
            if (wn == 0 && g == 0 && r < mr) p.hs[(size_t)(m0 + r) * NB + n0 / 128] = s;
        }
        __syncthreads();
        for (int q = tid; q < mr * 8; q += kGThreads) {
            const int r = q >> 3, c = q & 7;
            *reinterpret_cast<uint4*>(p.hq + (size_t)(m0 + r) * p.F + n0 + 16 * c) =
                *reinterpret_cast<const uint4*>(smem + r * LD + 16 * c);
        }
    } else {
        const int out_f32 = MODE == G_DENSE ? d.out_f32 : p.out_f32;
        const bool vec = MODE == G_DENSE ? d.vec : true;
        char* y = static_cast<char*>(MODE == G_DENSE ? d.y : p.rows);
        const int64_t ldy = MODE == G_DENSE ? d.ldy : (int64_t)p.H;
#pragma unroll
        for (int t = 0; t < TF; ++t) {
            const int r = wt * 16 * TF + 16 * t + l16;
            if (r >= mr) continue;
            char* row = y + (m0 + r) * ldy * (out_f32 ? 4 : 2);
#pragma unroll
            for (int f = 0; f < 4; f += 2) {
                const int n = n0 + 64 * wn + 16 * f + 8 * g;
                if (n >= N) continue;
                if (vec && n + 7 < N) {
                    store8(row, out_f32, n, acc[f][t], acc[f + 1][t]);
                } else {
                    fp8_store4(row, out_f32, n, N, false, acc[f][t]);
                    fp8_store4(row, out_f32, n + 4, N, false, acc[f + 1][t]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// The grouped passes on a run of tiles per workgroup, one workgroup a compute
// unit: the steps of its tiles are one sequence, u = tile * KB + j, and the
// pipeline above runs across tile borders, so the first loads of a tile are
// under way while the tile before is computed and stored.  (One workgroup per
// tile left 10 us of its 20 to 47 us without an MFMA; no second one fits the
// LDS.)  Needs KB >= kRunMinKB, so that what the next tile needs can be
// prepared within the present one:
//   step 0     gate/up: the next tile's (token, slot) pairs are loaded
//   step 2     and turned into token rows, seen after the barrier of step 3
//   last steps the first scales and, S steps before the end, rows and weights
// Scales come in chunks of 4 to 8 steps, two LDS buffers.
template <int TF>
struct RunLds {
    using G = GemmLds<TF>;
    static constexpr int BT = G::BT, S = G::S, A = G::A, B = G::B, W = G::W, SA = G::SA, SW = G::SW;
    static constexpr int TOK = G::ROW;                // gate/up: token rows [2][BT]
    static constexpr int RAW = TOK + 2 * BT * 4;      // and the pairs they come from [BT]
    static constexpr int AMAX = RAW + BT * 4;         // group maxima [4][BT]
    static constexpr int TOTAL = AMAX + 4 * BT * 4;
    static_assert(TOTAL <= 160 * 1024, "LDS of a compute unit");
};

constexpr int kRunMinKB = 8, kRunMinKBDown = 4;

struct RunTile {
    int e, m0, mr, n0;
};

typedef const __attribute__((address_space(4))) int32_t const_int;

// A value that no kernel writes meanwhile, at a uniform address: a scalar load.
__device__ __forceinline__ int const_load(const int32_t* p) { return *(const_int*)p; }

template <int TF, int MODE, bool kExact>
__global__ __launch_bounds__(kGThreads, 2) void fp8_run_kernel(const Fp8Ffn p) {
    using L = RunLds<TF>;
    constexpr int BT = L::BT, S = L::S, NA = BT / 64, NL = NA + 4;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wv & 3, wt = wv >> 2, g = lane >> 4, l16 = lane & 15;

    // ---- the run: XCD x takes a contiguous eighth of the tiles, its workgroups every (grid / 8)-th of it
    const int K = MODE == G_GATEUP ? p.H : p.F, N = MODE == G_GATEUP ? p.F : p.H;
    const int KB = K / 128, NB = N / 128;
    const int nt = MODE == G_GATEUP ? p.F / 128 : (p.H + kGN - 1) / kGN;
    const int total = const_load(p.tiles) * nt, q = (total + kXcd - 1) / kXcd, stride = (int)gridDim.x / kXcd;
    const int l0 = (int)blockIdx.x % kXcd * q + (int)blockIdx.x / kXcd, lend = min(((int)blockIdx.x % kXcd + 1) * q, total);
    if (l0 >= lend) return;
    const int count = (lend - l0 + stride - 1) / stride;
    auto tile_at = [&](int i) {  // tile i of the run
        const int l = l0 + i * stride, t = l / nt;
        RunTile r;
        r.n0 = (l - t * nt) * (MODE == G_GATEUP ? 128 : kGN);
        r.e = const_load(p.tiles + 1 + 3 * t);
        r.m0 = const_load(p.tiles + 2 + 3 * t);
        r.mr = min(const_load(p.tiles + 3 + 3 * t), p.P) - r.m0;
        return r;
    };
    const int chunks = (KB + 7) / 8;
    auto chunk_first = [&](int c) { return c * KB / chunks; };  // 4 to 8 steps each

    // ---- loads, as in fp8_gemm_kernel
    const int lr = 8 * wv + (lane >> 3), piece = (lane & 7) ^ g_swz(lr);
    const uint32_t woff = (uint32_t)g_order(lr) * (uint32_t)K + 16u * (uint32_t)piece;
    const uint32_t aoff = (uint32_t)lr * (uint32_t)K + 16u * (uint32_t)piece;  // down: rows of a tile are neighbours
    uint32_t* tok = reinterpret_cast<uint32_t*>(smem + L::TOK);
    const int32_t* raw = reinterpret_cast<const int32_t*>(smem + L::RAW);

    // gate/up: where the rows of the wave's loads begin, kept for the length of a
    // tile (read from LDS before each load, their waits cost a tenth of the pass)
    uint32_t rowoff[NA] = {};

    // where loads stand: tile i of the run, step j, and where its weights and (down) rows begin
    struct At {
        uint64_t w, a;
        uint32_t wb, ab;   // bytes of them
        int i, j;
    };
    auto at_tile = [&](const RunTile& t, int i) {
        At r;
        r.w = ((uint64_t)t.e * N + t.n0) * K;
        r.wb = (MODE == G_GATEUP ? 128u : (uint32_t)min(N - t.n0, kGN)) * (uint32_t)K;
        r.a = (uint64_t)t.m0 * K;
        r.ab = (uint32_t)t.mr * (uint32_t)K;
        r.i = i;
        r.j = 0;
        return r;
    };
    auto load_w = [&](int n, const At& at, int st) {
        const uint8_t* src = MODE == G_GATEUP ? (n >= 2 ? p.up : p.gate) : p.down;
        const uint32_t off = woff + (uint32_t)(MODE == G_GATEUP ? n & 1 : n) * 64u * (uint32_t)K;
        load16_lds(src + at.w, at.wb, smem + L::W + st * L::B + (8 * n + wv) * 1024, off, at.j * 128);
    };
    // whether the wave's row load n belongs to the second half of the rows
    auto second_half = [&](int n) { return (((64 * n + 8 * wv) / (8 * TF)) & 1) != 0; };
    // load n of a group: weights and first halves of the rows at `a`, second
    // halves at `b`, one step behind.  Rows past the tile's end: gate/up repeats
    // some token, down reads zeros; their results are dropped.
    auto load_group = [&](int n, const At& a, const At& b, int st) {
        if (n < 4) {
            load_w(n, a, st);
            return;
        }
        n -= 4;
        const bool second = second_half(n);
        const int stage = second ? (st == 0 ? S - 1 : st - 1) : st, j = second ? b.j : a.j;
        const uint8_t* src = MODE == G_GATEUP ? p.xq : p.hq + (second ? b.a : a.a);
        const uint32_t bytes = MODE == G_GATEUP ? (uint32_t)p.T * (uint32_t)K : second ? b.ab : a.ab;
        const uint32_t off = MODE == G_GATEUP ? rowoff[n] : aoff + (uint32_t)n * 64u * (uint32_t)K;
        load16_lds(src, bytes, smem + stage * L::A + (8 * n + wv) * 1024, off, j * 128);
    };
    auto row_offsets = [&](bool second, int i) {  // of tile i, of one half of the rows
        if (MODE != G_GATEUP) return;
#pragma unroll
        for (int n = 0; n < NA; ++n)
            if (second_half(n) == second) rowoff[n] = tok[(i & 1) * BT + 64 * n + lr] * (uint32_t)K + 16u * (uint32_t)piece;
    };
    // scales of steps c0 .. c0 + 7 of a tile into buffer `par`: wave v loads step c0 + v
    auto load_s = [&](const RunTile& t, int i, int c0, int par) {
        const int kb = min(c0 + wv, KB - 1);
        const float* rs = MODE == G_GATEUP ? p.xs : p.hs + (size_t)t.m0 * KB;
        const uint32_t bytes = (uint32_t)(MODE == G_GATEUP ? p.T : t.mr) * (uint32_t)KB * 4u;
        float* sa = reinterpret_cast<float*>(smem + L::SA) + par * 8 * BT + wv * BT;
#pragma unroll
        for (int n = 0; n < NA; ++n) {
            const uint32_t row = MODE == G_GATEUP ? tok[(i & 1) * BT + 64 * n + lane] : (uint32_t)(64 * n + lane);
            load4_lds(rs, bytes, sa + 64 * n, row * (uint32_t)KB * 4u, kb * 4);
        }
        if (wv < 2 && lane < 8) {
            // the gate's and the up's, or those of the tile's two blocks of 128 outputs
            const size_t at = ((size_t)t.e * NB + min(t.n0 / 128 + (MODE == G_GATEUP ? 0 : wv), NB - 1)) * KB;
            const float* src = MODE == G_GATEUP ? (wv ? p.sup : p.sgate) : p.sdown;
            float* sw = reinterpret_cast<float*>(smem + L::SW) + par * 16 + wv * 8;
            load4_lds(src + at, (uint32_t)KB * 4u, sw, (uint32_t)min(c0 + lane, KB - 1) * 4u, 0);
        }
    };
    auto token_row = [&](int r, const RunTile& t, int pair) {
        if (r >= t.mr) return 0u;
        return (uint32_t)(p.sorted_pair ? min(max(pair / p.k, 0), p.T - 1) : t.m0 + r);
    };

    const RunTile first = tile_at(0);
    RunTile cur = first, nx = count > 1 ? tile_at(1) : first;  // the tile computed, the one after it
    if (MODE == G_GATEUP) {
        for (int r = tid; r < BT; r += kGThreads)
            tok[r] = token_row(r, first, p.sorted_pair && r < first.mr ? p.sorted_pair[first.m0 + r] : 0);
        __syncthreads();
    }
    load_s(first, 0, 0, 0);
    // (b before the first step: the first step's rows, where the loads of step S - 1 will overwrite them)
    At a = at_tile(first, 0), b = a;
    int st = 0;  // stage of `a`
    row_offsets(false, 0);
    row_offsets(true, 0);
    auto advance = [&] {
        if (MODE == G_GATEUP && a.i != b.i) row_offsets(true, a.i);
        b = a;
        if (++a.j == KB) {
            if (a.i + 1 < count) {
                a = at_tile(nx, a.i + 1);  // (while the tile before is computed)
                row_offsets(false, a.i);
            } else {
                a.j = KB - 1;  // past the run's end: the last step again
            }
        }
        st = st + 1 == S ? 0 : st + 1;
    };
#pragma unroll
    for (int u = 0; u < S; ++u) {
#pragma unroll
        for (int n = 0; n < NL; ++n) load_group(n, a, b, st);
        advance();
    }

    const int x0 = 16 * (g ^ g_swz(l16)), x1 = 16 * ((g + 4) ^ g_swz(l16));
    const int ar = (wt * 16 * TF + l16) * 128;
    const int br = L::W + ((MODE == G_GATEUP ? 32 * wn : 64 * wn) + l16) * 128;
    const int sr0 = L::SA + (wt * 16 * TF + l16) * 4;
    const int sw0 = L::SW + (MODE != G_GATEUP && wn >= 2 ? 32 : 0);
    auto read16 = [&](int at) {
        return join8(*reinterpret_cast<const i32x4_t*>(smem + at + x0), *reinterpret_cast<const i32x4_t*>(smem + at + x1));
    };
    auto read_a = [&](int stage, int t) { return read16(stage * L::A + ar + t * 2048); };
    auto read_w = [&](int stage, int f) {
        return read16(stage * L::B + br + (MODE == G_GATEUP && f >= 2 ? 128 + 16 * (f - 2) : 16 * f) * 128);
    };
    auto read_sa = [&](int par, int pos, int t) {
        return *reinterpret_cast<const float*>(smem + sr0 + (par * 8 + pos) * BT * 4 + t * 64);
    };
    auto read_sw = [&](int par, int pos, int half) {
        return *reinterpret_cast<const float*>(smem + sw0 + par * 64 + pos * 4 + half * 32);
    };
    i32x8_t w[4], an;
    float sn, swn0, swn1 = 0.0f;
    auto read_first = [&](int stage, int par, int pos) {
        an = read_a(stage, 0);
        sn = read_sa(par, pos, 0);
        swn0 = read_sw(par, pos, 0);
        if (MODE == G_GATEUP) swn1 = read_sw(par, pos, 1);
    };
    wait_and_meet<(S - 1) * NL>();
#pragma unroll
    for (int f = 0; f < 4; ++f) w[f] = read_w(0, f);
    read_first(0, 0, 0);

    constexpr int kMeet = TF / 2 - 1;
    // Memory operations complete in order, and a tile's stores are the last before
    // the next tile: the loads that its first S - 1 steps wait for are older, so
    // those steps leave the stores under way.  Every wave issues at least this many.
    constexpr int NST = 2 * TF;
    // position: tile i, step j, step `pos` of a chunk of `len` in scale buffer `par`; `st` is also the
    // stage of the present step (that of S steps later)
    int par = 0;
    for (int i = 0; i < count; ++i) {
        f32x4_t acc[4][TF];
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int t = 0; t < TF; ++t) acc[f][t] = f32x4_t{};
        int pos = 0, chunk = 0, len = chunk_first(1);
#pragma unroll 1
        for (int j = 0; j < KB; ++j) {
            const int cs = st;                                 // this step's stage
            const int ns = st + 1 == S ? 0 : st + 1;           // the next step's
            const bool turn = pos + 1 == len;
            const int npos = turn ? 0 : pos + 1, npar = turn ? par ^ 1 : par;
            f32x4_t v[3];
            float c0[2], c1[2];
            const float s0 = swn0, s1 = swn1;
            auto add = [&](int x) {
                const int t = x / 4, f = x % 4;
                const float c = MODE == G_GATEUP && f >= 2 ? c1[t & 1] : c0[t & 1];
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[f][t][y] = fmaf(c, v[x % 3][y], acc[f][t][y]);
            };
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                if (t == kMeet) {
                    hold(acc, kMeet);
                    if (i > 0 && j < S - 1) wait_and_meet<(S - 2) * NL + NST>();
                    else wait_and_meet<(S - 2) * NL>();
                    if (MODE == G_GATEUP && i + 1 < count) {
                        if (j == 0 && p.sorted_pair && wv < NA) {
                            load4_lds(p.sorted_pair + nx.m0, (uint32_t)max(nx.mr, 0) * 4u, smem + L::RAW + wv * 256,
                                      (uint32_t)(64 * wv + lane) * 4u, 0);
                        }
                        if (j == S && tid < BT) tok[((i + 1) & 1) * BT + tid] = token_row(tid, nx, raw[tid]);
                    }
                    if (pos == len - S - 1) {
                        const int c = j - pos + len;  // the next chunk's first step
                        if (c < KB) load_s(cur, i, c, par ^ 1);
                        else if (i + 1 < count) load_s(nx, i + 1, 0, par ^ 1);
                    }
                }
                const i32x8_t ac = an;
                c0[t & 1] = sn * s0;
                if (MODE == G_GATEUP) c1[t & 1] = sn * s1;
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int x = 4 * t + f;
                    v[x % 3] = mfma_fp8<kExact>(w[f], ac);
                    if (t + 1 == TF) w[f] = read_w(ns, f);
                    if (f == 0) {
                        if (t + 1 < TF) {
                            an = read_a(cs, t + 1);
                            sn = read_sa(par, pos, t + 1);
                        } else {
                            read_first(ns, npar, npos);
                        }
                    }
                    if (x >= 4 * kMeet && x - 4 * kMeet < NL) load_group(x - 4 * kMeet, a, b, cs);
                    if (x >= 2) add(x - 2);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            add(4 * TF - 2);
            add(4 * TF - 1);
            hold(acc, TF);
            advance();
            if (turn) {
                ++chunk;
                len = chunk_first(chunk + 1) - chunk_first(chunk);
            }
            pos = npos;
            par = npar;
        }

        // ---- the tile is done.  (Row and column come from a value the compiler
        // cannot see through, or it would keep every row's address in registers
        // across the loop.)
        int le = lane;
        asm volatile("" : "+v"(le));
        const int re = wt * 16 * TF + (le & 15), ge = le >> 4;
        if constexpr (MODE == G_GATEUP) {
            uint32_t* amax = reinterpret_cast<uint32_t*>(smem + L::AMAX);
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                uint32_t m = 0;
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const float h = silu(acc[f][t][y]) * acc[f + 2][t][y];
                        acc[f][t][y] = h;
                        m = max(m, abs_bits(h));
                    }
                m = max(m, (uint32_t)__shfl_xor((int)m, 16, kWave));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
                if (ge == 0) amax[wn * BT + re + 16 * t] = m;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            // (the stores of rows past the tile's end, and all but one lane's of a
            // scale, fall outside their buffers: each is issued all the same)
            const __amdgpu_buffer_rsrc_t rq = fp8_rsrc(p.hq + (size_t)cur.m0 * p.F, (uint32_t)cur.mr * (uint32_t)p.F);
            const __amdgpu_buffer_rsrc_t rs = fp8_rsrc(p.hs + (size_t)cur.m0 * NB, (uint32_t)(cur.mr * NB) * 4u);
#pragma unroll
            for (int t = 0; t < TF; ++t) {
                const int r = re + 16 * t;
                const uint32_t m = max(max(amax[r], amax[BT + r]), max(amax[2 * BT + r], amax[3 * BT + r]));
                const float s = fp8_scale(m);
                const Fp8Div by = fp8_div(s);
                const u32x2_t q = {fp8_pack4(acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3], by),
                                   fp8_pack4(acc[1][t][0], acc[1][t][1], acc[1][t][2], acc[1][t][3], by)};
                __builtin_amdgcn_raw_buffer_store_b64(q, rq, r * p.F + cur.n0 + 32 * wn + 8 * ge, 0, 0);
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s), rs,
                                                      wn == 0 && ge == 0 ? (r * NB + cur.n0 / 128) * 4 : (int)kOob, 0, 0);
            }
        } else {
            const uint32_t rowb = (uint32_t)p.H * (p.out_f32 ? 4u : 2u);
            const __amdgpu_buffer_rsrc_t rr = fp8_rsrc(static_cast<char*>(p.rows) + (size_t)cur.m0 * rowb, (uint32_t)cur.mr * rowb);
#pragma unroll
            for (int t = 0; t < TF; ++t)
#pragma unroll
                for (int f = 0; f < 4; f += 2) {
                    const int n = cur.n0 + 64 * wn + 16 * f + 8 * ge;
                    const f32x4_t u = acc[f][t], v = acc[f + 1][t];
                    const uint32_t at = n < N ? (uint32_t)(re + 16 * t) * rowb + (uint32_t)n * (p.out_f32 ? 4u : 2u) : kOob;
                    if (p.out_f32) {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, u), rr, (int)at, 0, 0);
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), rr, (int)(at + 16u), 0, 0);
                    } else {
                        const u32x4_t o = {pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(v[0], v[1]),
                                           pack_bf16x2(v[2], v[3])};
                        __builtin_amdgcn_raw_buffer_store_b128(o, rr, (int)at, 0, 0);
                    }
                }
        }
        cur = nx;
        if (i + 2 < count) nx = tile_at(i + 2);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load still writes LDS when the workgroup ends
}

template <int TF, int MODE, bool kExact>
static hipError_t launch_one(const Fp8Dense& d, const Fp8Ffn& p, long tiles, hipStream_t s) {
    const long grid = (tiles + kXcd - 1) / kXcd * kXcd;
    const void* fn = reinterpret_cast<const void*>(fp8_gemm_kernel<TF, MODE, kExact>);
    const hipError_t err = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, GemmLds<TF>::TOTAL);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((fp8_gemm_kernel<TF, MODE, kExact>), dim3((unsigned)grid), dim3(kGThreads),
                       GemmLds<TF>::TOTAL, s, d, p);
    return hipGetLastError();
}

hipError_t launch_fp8_gemm(const Fp8Dense& d, int bt, hipStream_t s) {
    const Fp8Ffn p{};
    auto tiles = [&](int rows) { return ((long)d.M + rows - 1) / rows * (((long)d.N + kGN - 1) / kGN); };
    if (d.out_f32)
        return bt == 64 ? launch_one<2, G_DENSE, true>(d, p, tiles(64), s) : launch_one<4, G_DENSE, true>(d, p, tiles(128), s);
    if (bt == 256) return launch_one<8, G_DENSE, false>(d, p, tiles(256), s);
    if (bt == 128) return launch_one<4, G_DENSE, false>(d, p, tiles(128), s);
    return launch_one<2, G_DENSE, false>(d, p, tiles(64), s);
}

template <int TF, int MODE, bool kExact>
static hipError_t launch_run(const Fp8Ffn& p, long tiles, hipStream_t s) {
    const long grid = tiles < 256 ? (tiles + kXcd - 1) / kXcd * kXcd : 256;
    const void* fn = reinterpret_cast<const void*>(fp8_run_kernel<TF, MODE, kExact>);
    const hipError_t err = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, RunLds<TF>::TOTAL);
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((fp8_run_kernel<TF, MODE, kExact>), dim3((unsigned)grid), dim3(kGThreads), RunLds<TF>::TOTAL, s, p);
    return hipGetLastError();
}

long fp8_grouped_workgroups(int H, int F, long max_tiles) {
    const long up = H / 128 >= kRunMinKB ? 0 : max_tiles * (F / 128);
    const long down = F / 128 >= kRunMinKBDown ? 0 : max_tiles * ((H + kGN - 1) / kGN);
    return up > down ? up : down;
}

template <int TF, int MODE, bool kExact>
static hipError_t launch_grouped(const Fp8Ffn& p, long tiles, hipStream_t s) {
    const int KB = (MODE == G_GATEUP ? p.H : p.F) / 128;
    if (KB >= (MODE == G_GATEUP ? kRunMinKB : kRunMinKBDown)) return launch_run<TF, MODE, kExact>(p, tiles, s);
    const Fp8Dense d{};
    return launch_one<TF, MODE, kExact>(d, p, tiles, s);
}

template <int MODE>
static hipError_t launch_pass(const Fp8Ffn& p, int bt, long tiles, hipStream_t s) {
    if (p.out_f32) return bt == 64 ? launch_grouped<2, MODE, true>(p, tiles, s) : launch_grouped<4, MODE, true>(p, tiles, s);
    if (bt == 256) return launch_grouped<8, MODE, false>(p, tiles, s);
    if (bt == 128) return launch_grouped<4, MODE, false>(p, tiles, s);
    return launch_grouped<2, MODE, false>(p, tiles, s);
}

hipError_t launch_fp8_gemm_gateup(const Fp8Ffn& p, int bt, long max_tiles, hipStream_t s) {
    return launch_pass<G_GATEUP>(p, bt, max_tiles * (p.F / 128), s);
}

hipError_t launch_fp8_gemm_down(const Fp8Ffn& p, int bt, long max_tiles, hipStream_t s) {
    return launch_pass<G_DOWN>(p, bt, max_tiles * ((p.H + kGN - 1) / kGN), s);
}

}  // namespace moe
