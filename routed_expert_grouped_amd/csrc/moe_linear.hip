// moe_linear.hip -- one dense projection with FP8 operands in 128-blocks: y = x W^T.
//
//     y[m][n] = bf16( sum_b s[n / 128][b] * 2^e[m][b] * sum_{k in block b} a[m][k] w[n][k] )
//
// a: E4M3FN codes with one power-of-two scale per row and 128 values (moe_quantize_act, or the
// norm before the projection); w: E4M3FN codes with one fp32 scale per 128 x 128 block ("native FP8
// GEMV", Figures 9-10 of the OSDI'26 hybrid-inference article).  The scaled matrix instruction multiplies
// the codes and applies 2^e per row itself; a block's sum (exact products, fp32) is then multiplied by s
// and added in fp32, one fused multiply-add a value, so that every finite s means what it says
// (zeros and subnormals too).
//
// Two shapes:
//   stream  few rows: the weights' bytes bound it.  A workgroup owns 16, 32 or 64 columns, its eight waves a
//           part of K each, streamed through a ring of register stages (as in moe_few.hip); every
//           weight stage meets 1, 2 or 4 tiles of 16 rows.  One 16x16x128 instruction is a whole 128-block.
//   tile    many rows: the matrix cores bound it (8192^3: 2.34 PFLOP/s).  256 x 256 tiles (eight waves of 128 x
//           64), or 128 x 128 (four waves of 64 x 64) where the large ones would leave CUs idle.
//           A K step is one 128-block, loaded directly to LDS two or four steps deep, one barrier a step.
// Measured, N = K = 7168: 1 row 11 us, 16 rows 12 us, 64 rows 20 us, 512 rows 43 us, 1024 rows 63 us, 4096 rows 195
// to 234 us (1.8 to 2.15 PFLOP/s: 448 tiles are 1.75 rounds of the CUs).
// Rows and columns past the end read the last one's codes and are not stored, so every size takes the
// same path.
#include "libmoe.h"
#include "moe_device.h"
#include "moe_host.h"
#include "moe_lds.h"
#include "moe_ring.h"

#include <algorithm>
#include <type_traits>

namespace moe {

typedef int i32x8 __attribute__((__vector_size__(8 * sizeof(int))));

constexpr int kLinE8M0One = 127;  // E8M0 encoding of 1.0
constexpr int kLinMaxBlocks = MOE_LINEAR_MAX_K / 128;

struct LinArgs {
    const uint8_t* a;    // [M][K]
    const int8_t* e;     // [M][pitch]
    int pitch, M, N, K;
    const uint8_t* w;    // [N][K]
    const float* s;      // [ceil(N/128)][K/128]
    uint16_t* y;         // [M][N]
    int m_tiles, n_tiles;
};

__device__ __forceinline__ i32x8 lin_join(u32x4 lo, u32x4 hi) {
    i32x8 r = {(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    return r;
}

// The workgroup's tile: consecutive workgroups go to the 8 XCDs in turn, so XCD i takes the contiguous
// range i of logical tiles; logical tiles go in groups of up to kM row tiles, the row tile fastest, so
// that neighbours share the weight rows in one L2.
template <int kM>
__device__ __forceinline__ bool lin_tile(const LinArgs& a, int& mt, int& nt) {
    const int R = a.m_tiles * a.n_tiles, R8 = (R + 7) >> 3;
    const int L = ((int)blockIdx.x & 7) * R8 + ((int)blockIdx.x >> 3);
    if (L >= R || ((int)blockIdx.x >> 3) >= R8) return false;
    const int b = L / (kM * a.n_tiles), r = L - b * kM * a.n_tiles;
    const int gm = min(kM, a.m_tiles - b * kM);
    nt = r / gm;
    mt = b * kM + r - nt * gm;
    return true;
}

constexpr int kLinWaves = 8;
constexpr int kLinLD = 128 + 16;  // LDS row stride of a wave's 16 weight rows

// MT row tiles of 16, kG groups of 16 columns: a weight stage meets MT row tiles and an activation stage kG
// column groups, so a wave reads MT + kG tiles' bytes for MT kG tiles' products.
template <int MT, int kG>
__global__ __launch_bounds__(kLinWaves * 64) void linear_stream_kernel(LinArgs a) {
    constexpr int D = MT + kG <= 4 ? 4 : MT + kG == 5 ? 3 : 2;  // stages in flight, within the registers
    __shared__ __attribute__((aligned(16))) uint8_t sW[kLinWaves][16 * kLinLD];
    __shared__ int8_t sE[MT * 16][kLinMaxBlocks + 4];  // (padded: 16 rows' bytes of a block in as many banks)
    __shared__ f32x4 red[kLinWaves][kG][kWave];
    int mt, nt;
    if (!lin_tile<16>(a, mt, nt)) return;
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int m = lane & 15, q = lane >> 4;
    const int K = a.K, kb_all = K / 128, m0 = mt * MT * 16, n0 = nt * 16 * kG;
    const int st0 = kb_all * wave / kLinWaves, ns = kb_all * (wave + 1) / kLinWaves - st0;
    uint8_t* lds = sW[wave];

    // Instruction i of a 16-row tile of either operand loads rows 8 i + lane / 8, 16-byte chunk lane % 8: whole
    // 128-byte lines, 16 cache accesses.  (Straight to the operand layout, a row a lane, it would be 64:
    // the cache's tags then bounded 64 x 2048 x 7168 at 22 us.)  Both operands change layout through the
    // wave's LDS rows; lane quarter q takes chunks q and q + 4 (which K a chunk holds does not matter as
    // long as both operands agree).  Offsets from the tile's first row and the wave's first block.
    const gbytes W = held(a.w + (size_t)n0 * K + (size_t)st0 * 128), A = held(a.a + (size_t)m0 * K + (size_t)st0 * 128);
    uint32_t wo[kG][2], xo[MT][2];
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            wo[g][i] = __umul24(min(16 * g + 8 * i + (lane >> 3), a.N - 1 - n0), K) + (lane & 7) * 16;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            xo[t][i] = __umul24(min(16 * t + 8 * i + (lane >> 3), a.M - 1 - m0), K) + (lane & 7) * 16;
    // (16 kG divides 128: one scale row for all groups)
    const gbytes sp = held(a.s + (size_t)(n0 / 128) * kb_all + st0);
    u32x4 bw[D][kG][2], ax[D][MT][2];
    float sc[D];
    int is = 0;
    auto issue = [&](auto tag) {  // past the wave's part its last block is loaded again (not used)
        constexpr int d = decltype(tag)::value;
        const size_t at = (size_t)is * 128;
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i) bw[d][g][i] = __builtin_nontemporal_load((gvec<u32x4>)(W + at + wo[g][i]));
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) ax[d][t][i] = *(gvec<u32x4>)(A + at + xo[t][i]);
        sc[d] = *(gvec<float>)(sp + 4 * (size_t)is);
        is = min(is + 1, ns - 1);
    };
    // the first stages (in slot order, as the loop has them: the waits count on it), then the block
    // exponents of the workgroup's rows, all of K, eight loads in flight a thread
    if (ns > 0)
        each_slot<D>([&](auto tag) {
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
        });
    const int n_e = MT * 16 * kb_all;
    for (int i0 = tid; i0 < n_e; i0 += 8 * kLinWaves * 64) {
        int8_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = min(i0 + j * kLinWaves * 64, n_e - 1), r = i / kb_all;
            v[j] = a.e[(size_t)min(m0 + r, a.M - 1) * a.pitch + (i - r * kb_all)];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = i0 + j * kLinWaves * 64, r = i / kb_all;
            if (i < n_e) sE[r][i - r * kb_all] = v[j];
        }
    }
    __syncthreads();
    f32x4 acc[MT][kG];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int g = 0; g < kG; ++g) acc[t][g] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (ns > 0) {
        int kb = st0;
        ring_loop<D>(ns, [&](auto tag) {
            constexpr int d = decltype(tag)::value;
            auto turn = [&](const u32x4* v) {  // all through the same rows: a wave's LDS operations complete in order
#pragma unroll
                for (int i = 0; i < 2; ++i) *(u32x4*)&lds[(8 * i + (lane >> 3)) * kLinLD + (lane & 7) * 16] = v[i];
                __builtin_amdgcn_wave_barrier();
                const i32x8 f = lin_join(*(const u32x4*)&lds[m * kLinLD + q * 16], *(const u32x4*)&lds[m * kLinLD + 64 + q * 16]);
                __builtin_amdgcn_wave_barrier();
                return f;
            };
            i32x8 fb[kG];
#pragma unroll
            for (int g = 0; g < kG; ++g) fb[g] = turn(bw[d][g]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const i32x8 fa = turn(ax[d][t]);
                const int e = (int)sE[16 * t + m][kb] + 127;
#pragma unroll
                for (int g = 0; g < kG; ++g) {
                    const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fa, fb[g], f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, e, 0, kLinE8M0One);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[t][g][r] = fmaf(p[r], sc[d], acc[t][g][r]);
                }
            }
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int g = 0; g < kG; ++g) asm volatile("" : "+v"(acc[t][g]));  // (taken before the slot is loaded again)
            __builtin_amdgcn_sched_barrier(0);
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
            ++kb;
        });
    }
    // the waves' sums, in wave order, a row tile at a time: wave g finishes column group g
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int g = 0; g < kG; ++g) red[wave][g][lane] = acc[t][g];
        __syncthreads();
        if (wave < kG) {
            f32x4 v = red[0][wave][lane];
#pragma unroll
            for (int w = 1; w < kLinWaves; ++w) v += red[w][wave][lane];
            const int n = n0 + 16 * wave + m;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = m0 + 16 * t + 4 * q + r;
                if (row < a.M && n < a.N) a.y[(size_t)row * a.N + n] = f32_to_bf16(v[r]);
            }
        }
    }
}

// kMI x 2 subtiles of 32 x 32 a wave, kWM x kWN waves, kD steps (128 K each) in LDS.
//
// LDS rows are 128 bytes (one block's codes), eight 16-byte chunks, chunk c at slot c ^ ((row >> 1) & 7):
// 16 consecutive rows' reads of one chunk fall in distinct banks.  32x32x64 operands: lane l holds row
// l % 32, chunks 4 j + l / 32 and 4 j + 2 + l / 32 of half j of the block (both operands alike).
//
// A block's sum must leave the matrix cores to be scaled (16 fused multiply-adds a subtile, half the matrix
// cores' time if they waited for each other), and its operands come from LDS.  So every wave runs three
// things at once: subtile t's two products, subtile t - 1's multiply-adds between them, and the LDS reads
// of later subtiles.  The last row of subtiles of a step reads the next step's first operands: the step's
// barrier stands before it, when all of this step's operands are in registers and the next step's have landed.
// The loads of the step after next go to the buffer that it frees, over the four subtiles after the
// barrier (two where a step has but four).
template <int kMI, int kWM, int kWN, int kD>
__global__ __launch_bounds__(kWM * kWN * 64) void linear_tile_kernel(LinArgs a) {
    constexpr int kNI = 2, kWaves = kWM * kWN, BM = 32 * kMI * kWM, BN = 32 * kNI * kWN;
    constexpr int kIA = BM / 8 / kWaves, kIB = BN / 8 / kWaves;  // direct loads a wave a step (8 rows each)
    constexpr int kT = kMI * kNI;  // subtiles a step: even, so that subtile -1 is kT - 1 of the step before
    static_assert(kT % 2 == 0, "p alternates over steps too");
    static_assert(kMI == 2 || kMI == 4, "the last row of subtiles follows the barrier");
    __shared__ __attribute__((aligned(1024))) uint8_t sA[kD][BM * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t sB[kD][BN * 128];
    __shared__ uint8_t sE[2][BM * 16];
    __shared__ float sS[2][BN / 128 * 16];
    int mt, nt;
    if (!lin_tile<8>(a, mt, nt)) return;
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    const int wm = wave / kWN, wn = wave % kWN, fr = lane & 31, half = lane >> 5;
    const int K = a.K, kb_all = K / 128, m0 = uniform(mt * BM), n0 = uniform(nt * BN);

    // direct loads, eight rows each: from their first row (the group of the last row for those past the
    // end, whose products are not stored) at a byte offset per lane
    constexpr int kLoads = kIA + kIB, kSlots = kT == 8 ? 4 : 2, kPart = kLoads / kSlots;
    static_assert(kLoads == 8 && kIA % 2 == 0, "parts of whole loads; a load's parity is its row group's");
    const uint8_t *ab = a.a + (size_t)m0 * K, *bb = a.w + (size_t)n0 * K;
    const uint32_t la = lds_address(sA) + 8 * kIA * wave * 128, lb = lds_address(sB) + 8 * kIB * wave * 128;
    const uint32_t lr = lane >> 3, lc = ((lane & 7) ^ (lane >> 4)) << 4;
    auto issue = [&](int kb, auto tag) {  // loads part * kPart ... of step kb (past the end: of the last)
        const uint32_t buf = kb & (kD - 1);
        const int at = min(kb, kb_all - 1) * 128;
#pragma unroll
        for (int l = decltype(tag)::value * kPart; l < decltype(tag)::value * kPart + kPart; ++l) {
            const bool of_a = l < kIA;
            const int i = of_a ? l : l - kIA, last = of_a ? a.M - 1 - m0 : a.N - 1 - n0;
            const int row = min(8 * ((of_a ? kIA : kIB) * wave + i), last & ~7);
            const uint32_t offset = __umul24(min(lr, (uint32_t)(last - row)), (uint32_t)K) + (lc ^ (64 * (i & 1)));
            lds_dma16_from((of_a ? ab : bb) + (uint32_t)uniform(at + row * K), offset,
                           (of_a ? la + buf * (BM * 128) : lb + buf * (BN * 128)) + i * 1024);
        }
    };
    // the tile's scales, 16 blocks at a time in two buffers: E8M0 bytes of the rows, fp32 of the 128-column
    // groups (registers hold none of them over a step)
    auto window = [&](int w) {
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));  // (nothing of this is kept in registers from one window to the next)
#pragma unroll 1
        for (int i = tid; i < BM * 16; i += kWaves * 64)
            sE[w & 1][i] = (uint8_t)(a.e[(size_t)min(m0 + (i >> 4), a.M - 1) * a.pitch + min(16 * w + (i & 15), kb_all - 1)] + 127);
        if (tid < BN / 128 * 16)
            sS[w & 1][tid] = a.s[(size_t)(min(n0 + 128 * (tid >> 4), a.N - 1) / 128) * kb_all + min(16 * w + (tid & 15), kb_all - 1)];
    };
    // this lane's LDS chunks: rows 32 apart have the same swizzle; half j's chunks 4 j + half, 4 j + 2 + half
    const uint32_t c0 = fr * 128 + ((half ^ ((fr >> 1) & 7)) << 4);
    auto frag = [&](const uint8_t* t, int j) {
        return lin_join(*(const u32x4*)&t[c0 ^ (64 * j)], *(const u32x4*)&t[c0 ^ (64 * j + 32)]);
    };
    i32x8 fa[2], fb[kNI][2];  // halves of the current subtile row of A, and of B
    int ea[2];                // block scales of subtile rows i and i + 1
    auto read_e = [&](auto tag, int kb) {
        constexpr int i = decltype(tag)::value;
        ea[i & 1] = sE[(kb >> 4) & 1][((wm * kMI + i) * 32 + fr) * 16 + (kb & 15)];
    };
    auto read_a = [&](auto tag, int j, int kb) {
        constexpr int i = decltype(tag)::value;
        fa[j] = frag(sA[kb & (kD - 1)] + (wm * kMI + i) * 32 * 128, j);
    };
    auto read_b = [&](auto tag, int kb) {
        constexpr int i = decltype(tag)::value;
#pragma unroll
        for (int j = 0; j < 2; ++j) fb[i][j] = frag(sB[kb & (kD - 1)] + (wn * kNI + i) * 32 * 128, j);
    };
    auto scale_of = [&](int kb) { return sS[(kb >> 4) & 1][(wn * 32 * kNI / 128) * 16 + (kb & 15)]; };
    f32x16 acc[kMI][kNI], p[2];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const f32x16 zero = {};
    p[1] = zero;
    float s = 0.0f, sl = 0.0f;  // the step's weight scale, and the scale of the subtile before
    auto take = [&](auto tag, int v0, float scale) {  // half of subtile t's multiply-adds
        constexpr int t = decltype(tag)::value;
#pragma unroll
        for (int v = 0; v < 8; ++v)
            acc[t / kNI][t % kNI][v0 + v] = fmaf(p[t & 1][v0 + v], scale, acc[t / kNI][t % kNI][v0 + v]);
        // (taken here: the compiler would otherwise move products and sums past the barrier to their next
        // use, and hold every operand of the step in registers until then)
        asm volatile("" : "+v"(acc[t / kNI][t % kNI]));
    };
    auto subtile = [&](auto tag, int kb) {
        constexpr int t = decltype(tag)::value, i = t / kNI, j = t % kNI;
        using prev = std::integral_constant<int, (t + kT - 1) % kT>;
        // a half of A is read for the next subtile row (the last row: of the next step; after the last step
        // nothing uses it) when its last product is issued, one product before its first use
        using next = std::integral_constant<int, (i + 1) % kMI>;
        const int kn = i + 1 == kMI ? kb + 1 : kb;
        const float scale = t == 0 ? sl : s;
        p[t & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[0], fb[j][0], zero, 0, 0, 0, ea[i & 1], 0, kLinE8M0One);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (j == 0) read_e(next{}, kn);
        if constexpr (j == kNI - 1) read_a(next{}, 0, kn);
        constexpr int slot = (t + kNI) % kT;  // subtiles since the barrier
        if constexpr (slot < kSlots) issue(kb + kD - (t < kT - kNI), std::integral_constant<int, slot>{});
        take(prev{}, 0, scale);
        __builtin_amdgcn_sched_barrier(0);
        p[t & 1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[1], fb[j][1], p[t & 1], 0, 0, 0, ea[i & 1], 0, kLinE8M0One);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (j == kNI - 1) read_a(next{}, 1, kn);
        if constexpr (i + 1 == kMI) read_b(std::integral_constant<int, j>{}, kb + 1);
        take(prev{}, 8, scale);
        __builtin_amdgcn_sched_barrier(0);
    };
    window(0);
#pragma unroll
    for (int i = 0; i < kD - 1; ++i) each_slot<kSlots>([&](auto tag) { issue(i, tag); });
    each_slot<2>([&](auto tag) { issue(kD - 1, tag); });  // (the other parts: in step 0)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads * (kD - 2) + 2 * kPart));
    __syncthreads();
    read_e(std::integral_constant<int, 0>{}, 0);
    read_a(std::integral_constant<int, 0>{}, 0, 0);
    read_a(std::integral_constant<int, 0>{}, 1, 0);
    read_b(std::integral_constant<int, 0>{}, 0);
    read_b(std::integral_constant<int, 1>{}, 0);
    s = scale_of(0);
    for (int kb = 0; kb < kb_all; ++kb) {
        if ((kb & 15) == 8 && (kb | 15) + 1 < kb_all) window(kb / 16 + 1);
        each_slot<kT - kNI>([&](auto tag) { subtile(tag, kb); });
        // every wave has this step's operands in registers, and the next step's codes are in LDS (the kD - 2
        // steps after it may be in flight)
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(kLoads * (kD - 2)));
        __syncthreads();
        const float next = scale_of(kb + 1);
        subtile(std::integral_constant<int, kT - 2>{}, kb);
        subtile(std::integral_constant<int, kT - 1>{}, kb);
        sl = s;
        s = next;
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // (no load may land after the workgroup's LDS is another's)
    take(std::integral_constant<int, kT - 1>{}, 0, sl);
    take(std::integral_constant<int, kT - 1>{}, 8, sl);
    // D layout: value v of a lane is row 8 (v / 4) + 4 half + v % 4, column fr
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int row = m0 + (wm * kMI + i) * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
            if (row >= a.M) continue;
            uint16_t* o = a.y + (size_t)row * a.N;
#pragma unroll
            for (int j = 0; j < kNI; ++j) {
                const int n = n0 + (wn * kNI + j) * 32 + fr;
                if (n < a.N) o[n] = f32_to_bf16(acc[i][j][v]);
            }
        }
}

template <typename F>
static moe_status lin_launch(LinArgs a, int BM, int BN, int threads, F kernel, hipStream_t st) {
    const int64_t mt = ((int64_t)a.M + BM - 1) / BM, nt = ((int64_t)a.N + BN - 1) / BN, R = mt * nt;
    a.m_tiles = (int)mt;
    a.n_tiles = (int)nt;
    if (R > (1 << 22)) return MOE_ERR_UNSUPPORTED;  // (a launch holds fewer than 2^32 threads)
    kernel<<<dim3((unsigned)((R + 7) / 8 * 8)), dim3(threads), 0, st>>>(a);
    return launch_status();
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_a8(const uint8_t* x_codes, const int8_t* x_exps, int32_t exp_pitch,
                                    int32_t M, int32_t N, int32_t K, const uint8_t* w, const float* s_w,
                                    uint16_t* y, void* stream) {
    if (M < 0 || N < 1 || K < 1) return MOE_ERR_INVALID_ARG;
    if (K % 128 != 0 || K > MOE_LINEAR_MAX_K) return MOE_ERR_UNSUPPORTED;
    if (exp_pitch < K / 128) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (!x_codes || !x_exps || !w || !s_w || !y || !aligned16(x_codes) || !aligned16(x_exps) ||
        !aligned16(w) || !aligned16(s_w) || !aligned16(y))
        return MOE_ERR_INVALID_ARG;
    LinArgs a{x_codes, x_exps, exp_pitch, M, N, K, w, s_w, y, 0, 0};
    hipStream_t st = as_stream(stream);
    // Streaming or tiles, by the time each would take: the streaming kernel reads MT + kG tiles of 16 rows
    // for every MT x kG of them (at the 7 TB/s that its loads come from the caches with), the small tiles
    // take 0.75 us a K step where every CU has at most one, else 1.13 us a round of two.  Up to 64 rows always
    // stream (the weights pass once).  128 x 7168 x 7168: 25 us streamed, 42 us in tiles; 256 x 7168 x
    // 7168: 59 by that rule, 41 us in tiles.
    const int MT = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    const int64_t rows = ((int64_t)M + 16 * MT - 1) / (16 * MT);
    const int64_t cols = ((int64_t)N + 15) / 16;
    // as many column groups a workgroup as leave one for most CUs
    const int kG = rows * ((cols + 3) / 4) >= 192 ? 4 : rows * ((cols + 1) / 2) >= 192 ? 2 : 1;
    const double stream_us = (double)rows * ((cols + kG - 1) / kG) * (MT + kG) * 16 * K / 7e6;
    const int64_t small = (((int64_t)M + 127) / 128) * (((int64_t)N + 127) / 128);
    const double tile_us = K / 128 * (small <= 256 ? 0.75 : 1.13 * ((small + 511) / 512));
    if (M <= 64 || (M <= 1024 && stream_us < tile_us)) {
#define MOE_STREAM(T_, G_) \
    if (MT == T_ && kG == G_) return lin_launch(a, 16 * T_, 16 * G_, kLinWaves * 64, linear_stream_kernel<T_, G_>, st);
        MOE_STREAM(1, 1) MOE_STREAM(1, 2) MOE_STREAM(1, 4)
        MOE_STREAM(2, 1) MOE_STREAM(2, 2) MOE_STREAM(2, 4)
        MOE_STREAM(4, 1) MOE_STREAM(4, 2) MOE_STREAM(4, 4)
#undef MOE_STREAM
    }
    const int64_t large = (((int64_t)M + 255) / 256) * (((int64_t)N + 255) / 256);
    if (large >= 192) return lin_launch(a, 256, 256, 512, linear_tile_kernel<4, 2, 4, 2>, st);
    // four steps in LDS where a CU has one workgroup, else two for two of them (512 x 7168 x 7168, 224 tiles: 43
    // us, with two steps 45; 1024 x 7168 x 7168, 448 tiles: two steps 63 us, four 86)
    if (small <= 256) return lin_launch(a, 128, 128, 256, linear_tile_kernel<2, 2, 2, 4>, st);
    return lin_launch(a, 128, 128, 256, linear_tile_kernel<2, 2, 2, 2>, st);
}
