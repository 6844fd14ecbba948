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
//   stream  few rows: the weights' bytes bound it.  A workgroup owns 16 columns, its eight waves a part
//           of K each, streamed through a ring of register stages (as in moe_few.hip); every weight
//           stage meets 1, 2 or 4 tiles of 16 rows.  One 16x16x128 instruction is a whole 128-block.
//   tile    many rows: the matrix cores bound it.  256 x 256 tiles (eight waves of 128 x 64), or 128 x 128
//           (four waves of 64 x 64, two workgroups a CU) where the large ones would leave CUs idle.
//           A K step is one 128-block, loaded directly to LDS in two buffers, one barrier a step.
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

constexpr int kLinWaves = 8, kLinRing = 4;
constexpr int kLinLD = 128 + 16;  // LDS row stride of a wave's 16 weight rows

// MT row tiles of 16
template <int MT>
__global__ __launch_bounds__(kLinWaves * 64) void linear_stream_kernel(LinArgs a) {
    constexpr int D = kLinRing;
    __shared__ __attribute__((aligned(16))) uint8_t sW[kLinWaves][16 * kLinLD];
    __shared__ int8_t sE[MT * 16][kLinMaxBlocks];
    __shared__ f32x4 red[kLinWaves][MT][kWave];
    int mt, nt;
    if (!lin_tile<16>(a, mt, nt)) return;
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int m = lane & 15, q = lane >> 4;
    const int K = a.K, kb_all = K / 128, m0 = mt * MT * 16, n0 = nt * 16;
    const int st0 = kb_all * wave / kLinWaves, ns = kb_all * (wave + 1) / kLinWaves - st0;
    uint8_t* lds = sW[wave];

    // weights: instruction i loads rows 8 i + lane / 8, 16-byte chunk lane % 8 (whole 128-byte lines);
    // activations: row m of each tile, chunks q and q + 4 (the operand layout: which K a chunk holds
    // does not matter as long as both operands agree)
    const gbytes W = held(a.w), A = held(a.a);
    gbytes wp[2], xp[MT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wp[i] = W + (size_t)min(n0 + 8 * i + (lane >> 3), a.N - 1) * K + (size_t)st0 * 128 + (lane & 7) * 16;
#pragma unroll
    for (int t = 0; t < MT; ++t)
        xp[t] = A + (size_t)min(m0 + 16 * t + m, a.M - 1) * K + (size_t)st0 * 128 + q * 16;
    const gbytes sp = held(a.s) + 4 * ((size_t)(n0 / 128) * kb_all + st0);
    u32x4 bw[D][2], ax[D][MT][2];
    float sc[D];
    int is = 0;
    auto issue = [&](auto tag) {  // past the wave's part its last block is loaded again (not used)
        constexpr int d = decltype(tag)::value;
        const size_t at = (size_t)is * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) bw[d][i] = __builtin_nontemporal_load((gvec<u32x4>)(wp[i] + at));
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            ax[d][t][0] = *(gvec<u32x4>)(xp[t] + at);
            ax[d][t][1] = *(gvec<u32x4>)(xp[t] + at + 64);
        }
        sc[d] = *(gvec<float>)(sp + 4 * is);
        is = min(is + 1, ns - 1);
    };
    // block exponents of the workgroup's rows, all of K
    for (int i = tid; i < MT * 16 * kb_all; i += kLinWaves * 64) {
        const int r = i / kb_all, b = i - r * kb_all;
        sE[r][b] = a.e[(size_t)min(m0 + r, a.M - 1) * a.pitch + b];
    }
    __syncthreads();
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (ns > 0) {
        // (in slot order, as the loop has them: the waits count on it)
        each_slot<D>([&](auto tag) {
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
        });
        int kb = st0;
        ring_loop<D>(ns, [&](auto tag) {
            constexpr int d = decltype(tag)::value;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *(u32x4*)&lds[(8 * i + (lane >> 3)) * kLinLD + (lane & 7) * 16] = bw[d][i];
            __builtin_amdgcn_wave_barrier();  // (a wave's LDS operations complete in order)
            const i32x8 fb = lin_join(*(const u32x4*)&lds[m * kLinLD + q * 16],
                                      *(const u32x4*)&lds[m * kLinLD + 64 + q * 16]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const f32x4 p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    lin_join(ax[d][t][0], ax[d][t][1]), fb, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0,
                    (int)sE[16 * t + m][kb] + 127, 0, kLinE8M0One);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][r] = fmaf(p[r], sc[d], acc[t][r]);
                asm volatile("" : "+v"(acc[t]));  // (taken before the slot is loaded again)
            }
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_sched_barrier(0);
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
            ++kb;
        });
    }
    // the waves' sums, in wave order: wave t finishes row tile t
#pragma unroll
    for (int t = 0; t < MT; ++t) red[wave][t][lane] = acc[t];
    __syncthreads();
    if (wave < MT) {
        f32x4 v = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kLinWaves; ++w) v += red[w][wave][lane];
        const int n = n0 + m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = m0 + 16 * wave + 4 * q + r;
            if (row < a.M && n < a.N) a.y[(size_t)row * a.N + n] = f32_to_bf16(v[r]);
        }
    }
}

// kMI x kNI subtiles of 32 x 32 a wave, kWM x kWN waves.
// LDS rows are 128 bytes (one block's codes), eight 16-byte chunks, chunk c at slot c ^ ((row >> 1) & 7):
// 16 consecutive rows' reads of one chunk fall in distinct banks.  32x32x64 operands: lane l holds row
// l % 32, chunks 4 j + l / 32 and 4 j + 2 + l / 32 of half j of the block (both operands alike).
template <int kMI, int kNI, int kWM, int kWN>
__global__ __launch_bounds__(kWM * kWN * 64) void linear_tile_kernel(LinArgs a) {
    constexpr int kWaves = kWM * kWN, BM = 32 * kMI * kWM, BN = 32 * kNI * kWN;
    constexpr int kIA = BM / 8 / kWaves, kIB = BN / 8 / kWaves;  // direct loads a wave a step (8 rows each)
    static_assert(32 * kNI <= 128 && 128 % (32 * kNI) == 0, "one weight scale a wave");
    __shared__ __attribute__((aligned(1024))) uint8_t sA[2][BM * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t sB[2][BN * 128];
    int mt, nt;
    if (!lin_tile<8>(a, mt, nt)) return;
    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    const int wm = wave / kWN, wn = wave % kWN, fr = lane & 31, half = lane >> 5;
    const int K = a.K, kb_all = K / 128, m0 = mt * BM, n0 = nt * BN;

    gbytes ap[kIA], bp[kIB];
#pragma unroll
    for (int i = 0; i < kIA; ++i) {
        const int r = 8 * (kIA * wave + i) + (lane >> 3);
        ap[i] = (gbytes)a.a + (size_t)min(m0 + r, a.M - 1) * K + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
#pragma unroll
    for (int i = 0; i < kIB; ++i) {
        const int r = 8 * (kIB * wave + i) + (lane >> 3);
        bp[i] = (gbytes)a.w + (size_t)min(n0 + r, a.N - 1) * K + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
    }
    gbytes ep[kMI];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
        ep[i] = (gbytes)a.e + (size_t)min(m0 + (wm * kMI + i) * 32 + fr, a.M - 1) * a.pitch;
    const int sg = min(n0 + wn * 32 * kNI, a.N - 1) / 128;  // (columns past the end are not stored)
    const gbytes sp = (gbytes)a.s + 4 * (size_t)sg * kb_all;
    const uint32_t la = lds_address(sA), lb = lds_address(sB);
    int en[kMI];
    float sn;
    auto issue = [&](int kb) {
        const int buf = kb & 1;
#pragma unroll
        for (int i = 0; i < kIA; ++i)
            lds_dma16_at((const void*)(ap[i] + (size_t)kb * 128), la + (buf * BM + 8 * (kIA * wave + i)) * 128);
#pragma unroll
        for (int i = 0; i < kIB; ++i)
            lds_dma16_at((const void*)(bp[i] + (size_t)kb * 128), lb + (buf * BN + 8 * (kIB * wave + i)) * 128);
        // the block's scales, to registers: complete with the direct loads, at the next step's wait
#pragma unroll
        for (int i = 0; i < kMI; ++i) en[i] = *(gvec<int8_t>)(ep[i] + kb);
        sn = *(gvec<float>)(sp + 4 * kb);
    };
    int arow[kMI], brow[kNI];
#pragma unroll
    for (int i = 0; i < kMI; ++i) arow[i] = (wm * kMI + i) * 32 + fr;
#pragma unroll
    for (int i = 0; i < kNI; ++i) brow[i] = (wn * kNI + i) * 32 + fr;
    auto frag = [&](const uint8_t* s, int row, int j) {
        const int x = (row >> 1) & 7;
        return lin_join(*(const u32x4*)&s[row * 128 + (((4 * j + half) ^ x) << 4)],
                        *(const u32x4*)&s[row * 128 + (((4 * j + 2 + half) ^ x) << 4)]);
    };
    f32x16 acc[kMI][kNI];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const f32x16 zero = {};
    issue(0);
    for (int kb = 0; kb < kb_all; ++kb) {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        __syncthreads();  // step kb is in LDS, and every wave has left step kb - 1's buffer
        int ec[kMI];
#pragma unroll
        for (int i = 0; i < kMI; ++i) ec[i] = en[i] + 127;
        const float s = sn;
        if (kb + 1 < kb_all) issue(kb + 1);
        const uint8_t *A = sA[kb & 1], *B = sB[kb & 1];
        i32x8 fb[kNI][2];
#pragma unroll
        for (int j = 0; j < kNI; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) fb[j][h] = frag(B, brow[j], h);
#pragma unroll
        for (int i = 0; i < kMI; ++i) {
            i32x8 fa[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) fa[h] = frag(A, arow[i], h);
            f32x16 p[kNI];
#pragma unroll
            for (int j = 0; j < kNI; ++j)
                p[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[0], fb[j][0], zero, 0, 0, 0, ec[i], 0, kLinE8M0One);
#pragma unroll
            for (int j = 0; j < kNI; ++j)
                p[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa[1], fb[j][1], p[j], 0, 0, 0, ec[i], 0, kLinE8M0One);
#pragma unroll
            for (int j = 0; j < kNI; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = fmaf(p[j][v], s, acc[i][j][v]);
        }
    }
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

constexpr int kLinStreamM = 256;  // most rows of the streaming kernel

template <typename F>
static moe_status lin_launch(LinArgs a, int BM, int BN, int threads, F kernel, hipStream_t st) {
    a.m_tiles = (a.M + BM - 1) / BM;
    a.n_tiles = (a.N + BN - 1) / BN;
    const int64_t R = (int64_t)a.m_tiles * a.n_tiles;
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
    if (M <= 16) return lin_launch(a, 16, 16, kLinWaves * 64, linear_stream_kernel<1>, st);
    if (M <= 32) return lin_launch(a, 32, 16, kLinWaves * 64, linear_stream_kernel<2>, st);
    if (M <= kLinStreamM) return lin_launch(a, 64, 16, kLinWaves * 64, linear_stream_kernel<4>, st);
    const int64_t large = ((int64_t)(M + 255) / 256) * ((N + 255) / 256);
    if (large >= 192) return lin_launch(a, 256, 256, 512, linear_tile_kernel<4, 2, 2, 4>, st);
    return lin_launch(a, 128, 128, 256, linear_tile_kernel<2, 2, 2, 2>, st);
}
