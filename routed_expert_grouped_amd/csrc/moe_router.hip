// moe_router.hip -- the router's product: scores[t][e] = sum_h x[t][h] W[e][h], fp32.
//
// The gate of a sparse MoE layer scores every expert for every token (CMU 11-868 appendix A2 notes,
// 4.1; "gating" in the OSDI'26 hybrid-inference article, DSLP section); moe_route ranks these
// scores, so they stay in fp32: bf16 products are exact in fp32 and every sum is held in fp32.
//
// Two shapes:
//   few tokens  one workgroup per expert (and per group of up to 8 tokens): its four waves read the
//               expert's row once, each lane multiplies its chunks with every token's, and the lanes'
//               sums are joined in a fixed order.  W's bytes and the launch bound it.
//   more        tiles on the matrix cores (32x32x16 bf16), operands through LDS.  When the tiles alone
//               do not fill the chip, K is split over workgroups into fp32 partial scores in the
//               caller's workspace, and a second launch adds them in order.  Small batches take
//               64 x 64 tiles staged through registers, large ones tiles of 128 x 256, 192 or 128 loaded
//               directly to LDS, three stages deep.
//
// Measured, 7168 values a row, 256 experts, bf16 W: 1 token 6 us (the call), 512 tokens 13 us, 8192 tokens 46 us
// (663 TFLOP/s), 32768 tokens 140 to 147 us (837 TFLOP/s, 3.3 TB/s of x: loads to LDS and matrix cores bound it
// together); fp32 W at 32768 tokens 362 us (1.0 PFLOP/s of bf16 products).
//
// fp32 W goes to the matrix cores as three bf16 parts, w = hi + mid + lo (8 + 8 + 8 significand bits:
// exact for every finite w whose parts are not subnormal), so no bits of W are lost.  The small tiles split
// it while staging; for the large ones a launch before writes the parts to the workspace.
#include "libmoe.h"
#include "moe_device.h"
#include "moe_host.h"
#include "moe_lds.h"
#include "moe_ring.h"

#include <algorithm>

namespace moe {

constexpr int kDotThreads = 256;
constexpr int kDotWaves = kDotThreads / kWave;
constexpr int kRouterDotT = 16;  // most tokens of the per-expert kernel

// eight values of a weight row from chunk c (8 consecutive values)
template <bool kF32>
__device__ __forceinline__ void load_w8(const void* row, int c, float* w) {
    if constexpr (kF32) {
        const f32x4 a = ((const f32x4*)row)[2 * c], b = ((const f32x4*)row)[2 * c + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = a[i], w[4 + i] = b[i];
    } else {
        const u32x4 a = ((const u32x4*)row)[c];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = __uint_as_float(a[i] << 16);
            w[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
    }
}

template <bool kF32, int TT>
__global__ __launch_bounds__(kDotThreads) void router_dot_kernel(const uint16_t* __restrict__ x, int T,
                                                                 int H, const void* __restrict__ w,
                                                                 int E, float* __restrict__ scores) {
    __shared__ float part[kDotWaves][TT];
    const int e = (int)blockIdx.x, t0 = (int)blockIdx.y * TT;
    const int tid = (int)threadIdx.x, chunks = H / 8;
    const void* wrow = (const char*)w + (size_t)e * H * (kF32 ? 4 : 2);
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.0f;
#pragma unroll 4
    for (int c = tid; c < chunks; c += kDotThreads) {
        float wv[8];
        load_w8<kF32>(wrow, c, wv);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            // tokens past the last read the last one's row; their sums are not stored
            const u32x4 xv = ((const u32x4*)(x + (size_t)min(t0 + t, T - 1) * H))[c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[t] = fmaf(__uint_as_float(xv[i] << 16), wv[2 * i], acc[t]);
                acc[t] = fmaf(__uint_as_float(xv[i] & 0xffff0000u), wv[2 * i + 1], acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
#pragma unroll
        for (int d = kWave / 2; d > 0; d >>= 1) acc[t] += __shfl_xor(acc[t], d, kWave);
        if (lane_id() == 0) part[tid / kWave][t] = acc[t];
    }
    __syncthreads();
    if (tid < TT && t0 + tid < T) {
        float s = part[0][tid];
#pragma unroll
        for (int v = 1; v < kDotWaves; ++v) s += part[v][tid];
        scores[(size_t)(t0 + tid) * E + e] = s;
    }
}

// The three bf16 parts of two floats (a in the low halves), each the upper half of what is left: cut off, not
// rounded, so that the next difference is exact and has eight significant bits less.  An infinity is all in the
// first part; a NaN whose first part is an infinity has a NaN as its second.
__device__ __forceinline__ void split3(float a, float b, uint32_t* parts) {
    const auto upper = [](float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); };
    const auto pack = [](float lo, float hi) { return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u); };
    const float ah = upper(a), bh = upper(b);
    parts[0] = pack(a, b);
    a = a == ah ? 0.0f : a - ah;
    b = b == bh ? 0.0f : b - bh;
    parts[1] = pack(a, b);
    parts[2] = pack(a - upper(a), b - upper(b));
}

// 64 x 64 tile, four waves of 32 x 32, K in steps of 64 through two LDS buffers (fp32 W: three planes), one
// barrier a step.  With K split over the chip a workgroup has but a few steps, so latency is what they cost:
// the operands of four steps are in flight in registers.
constexpr int kRtK = 64;
constexpr int kRtLd = kRtK * 2 + 16;  // LDS row bytes: 16 consecutive rows' 16-byte reads hit distinct banks

template <bool kF32>
__global__ __launch_bounds__(256) void router_gemm_kernel(const uint16_t* __restrict__ x, int T, int H,
                                                          const void* __restrict__ w, int E, int n_tiles,
                                                          int tiles, int splits, float* __restrict__ out) {
    constexpr int kPlanes = kF32 ? 3 : 1, kWB = kF32 ? 2 : 1;  // (16-byte words of 8 weights)
    constexpr int kM = 64, kN = 64, kL = kM / 32, D = 4;       // staging loads a thread and operand, steps in flight
    __shared__ __attribute__((aligned(16))) uint8_t sA[2][kM * kRtLd];
    __shared__ __attribute__((aligned(16))) uint8_t sB[2][kPlanes][kN * kRtLd];
    // consecutive workgroups go to the 8 XCDs in turn: XCD i takes the contiguous range i of logical
    // tiles, so that the column tiles of a row tile share its x rows in one L2
    const int R8 = (tiles * splits + 7) / 8;
    const int L = ((int)blockIdx.x & 7) * R8 + ((int)blockIdx.x >> 3);
    if (L >= tiles * splits) return;
    const int split = L / tiles, tile = L - split * tiles;
    const int m0 = tile / n_tiles * kM, n0 = tile % n_tiles * kN;
    const int steps_all = (H + kRtK - 1) / kRtK;
    const int k0 = (int)((int64_t)steps_all * split / splits), k1 = (int)((int64_t)steps_all * (split + 1) / splits);

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, half = lane >> 5;
    // staging: thread loads 16-byte chunk tid % 8 of rows tid / 8 + 32 i; rows past the end read the last
    // row (not stored), chunks past H the last chunk, and are staged as zeros (both operands: 0 times garbage
    // could be NaN)
    const int lc = tid & 7, lr = tid >> 3;
    const uint16_t* xr[kL];
    const char* wr[kL];
#pragma unroll
    for (int i = 0; i < kL; ++i) {
        xr[i] = x + (size_t)min(m0 + lr + 32 * i, T - 1) * H;
        wr[i] = (const char*)w + (size_t)min(n0 + lr + 32 * i, E - 1) * H * (kF32 ? 4 : 2);
    }
    u32x4 ra[D][kL], rb[D][kL][kWB];
    auto load = [&](auto tag, int step) {
        constexpr int d = decltype(tag)::value;
        const int c = min(step * (kRtK / 8) + lc, H / 8 - 1);
#pragma unroll
        for (int i = 0; i < kL; ++i) ra[d][i] = ((const u32x4*)xr[i])[c];
#pragma unroll
        for (int i = 0; i < kL; ++i)
#pragma unroll
            for (int p = 0; p < kWB; ++p) rb[d][i][p] = ((const u32x4*)wr[i])[kWB * c + p];
    };
    auto stage = [&](auto tag, int buf, int step) {
        constexpr int d = decltype(tag)::value;
        const uint32_t keep = step * (kRtK / 8) + lc < H / 8 ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int i = 0; i < kL; ++i) *(u32x4*)&sA[buf][(lr + 32 * i) * kRtLd + lc * 16] = ra[d][i] & keep;
#pragma unroll
        for (int i = 0; i < kL; ++i) {
            const int at = (lr + 32 * i) * kRtLd + lc * 16;
            if constexpr (kF32) {
                u32x4 pl[3];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t q[3];
                    split3(__uint_as_float(rb[d][i][j >> 1][(2 * j) & 3] & keep),
                           __uint_as_float(rb[d][i][j >> 1][(2 * j + 1) & 3] & keep), q);
#pragma unroll
                    for (int p = 0; p < 3; ++p) pl[p][j] = q[p];
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) *(u32x4*)&sB[buf][p][at] = pl[p];
            } else {
                *(u32x4*)&sB[buf][0][at] = rb[d][i][0] & keep;
            }
        }
    };
    f32x16 acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    auto compute = [&](int buf) {
#pragma unroll
        for (int ks = 0; ks < kRtK / 16; ++ks) {
            const bf16x8 fa = as_bf16x8(*(const u32x4*)&sA[buf][(wm * 32 + fr) * kRtLd + ks * 32 + half * 16]);
#pragma unroll
            for (int p = kPlanes - 1; p >= 0; --p) {  // the small parts first
                const bf16x8 fb = as_bf16x8(*(const u32x4*)&sB[buf][p][(wn * 32 + fr) * kRtLd + ks * 32 + half * 16]);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
            }
        }
    };
    // (in slot order, as the loop has them: the waits count on it; past the end the last step is loaded again)
    each_slot<D>([&](auto tag) {
        load(tag, min(k0 + decltype(tag)::value, k1 - 1));
        __builtin_amdgcn_sched_barrier(0);
    });
    int s = k0;
    ring_loop<D>(k1 - k0, [&](auto tag) {
        const int buf = (s - k0) & 1;  // (its readers of two steps ago have passed the last step's barrier)
        stage(tag, buf, s);
        __builtin_amdgcn_sched_barrier(0);
        load(tag, min(s + D, k1 - 1));
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        compute(buf);
        ++s;
    });
    // D layout: value v of a lane is row 8 (v / 4) + 4 half + v % 4, column fr
    float* o = out + (size_t)split * T * E;
    const int e = n0 + wn * 32 + fr;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int t = m0 + wm * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
        if (t < T && e < E) o[(size_t)t * E + e] = acc[v];
    }
}

// fp32 W to its three bf16 parts [3][E][H]
__global__ __launch_bounds__(256) void router_split_kernel(const float* __restrict__ w, int64_t chunks,
                                                           uint16_t* __restrict__ parts) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= chunks) return;
    float v[8];
    load_w8<true>(w, (int)c, v);
    u32x4 pl[3];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t q[3];
        split3(v[2 * j], v[2 * j + 1], q);
#pragma unroll
        for (int p = 0; p < 3; ++p) pl[p][j] = q[p];
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) ((u32x4*)parts)[p * chunks + c] = pl[p];
}

__device__ const u32x4 kRouterZeros = {0u, 0u, 0u, 0u};

// 128 x (32 kNI kWN) tile, eight waves, K in stages of 64 and (fp32 W) of one of its planes, the small
// parts first: stage s is K step s / planes.  Operand rows are 128 bytes in LDS, eight 16-byte chunks, chunk
// c at slot c ^ ((row >> 1) & 7), so that 16 consecutive rows' reads of one chunk fall in distinct banks.
//
// Loads go directly to LDS, three buffers.  A stage is four products' depths; each depth's fragments are read
// while the one before is multiplied.  The stage's barrier stands before its last depth: every wave then
// has all of the stage in registers, the next stage has landed (the one after it may be in flight: the
// wait's count), and the freed buffer takes the stage after those.  The loop has no branch: past the end the
// first stages are loaded again, into buffers that are not read.  Neighbouring workgroups of an XCD start one
// K step apart and go round: rows of a whole number of 2 KiB have all of one step's lines in the same
// memory channel (32768 x 7168 x 256: 144 us, all from the first step 149).
// Rows past the end read the last row (not stored).  A last step of fewer than 64 values follows the loop,
// with zeros for the chunks past H.
template <int kMI, int kNI, int kWM, int kWN>
__global__ __launch_bounds__(512) void router_dma_kernel(const uint16_t* __restrict__ x, int T, int H,
                                                         const uint16_t* __restrict__ w, int planes, int E,
                                                         int n_tiles, int tiles, int splits,
                                                         float* __restrict__ out) {
    constexpr int kM = 32 * kMI * kWM, kN = 32 * kNI * kWN, kIA = kM / 64, kIB = kN / 64;
    static_assert(kWM * kWN == 8 && kM == 128, "eight waves, 128 rows");
    __shared__ __attribute__((aligned(1024))) uint8_t sA[3][kM * 128];
    __shared__ __attribute__((aligned(1024))) uint8_t sB[3][kN * 128];
    const int R8 = (tiles * splits + 7) / 8;
    const int L = ((int)blockIdx.x & 7) * R8 + ((int)blockIdx.x >> 3);
    if (L >= tiles * splits) return;
    const int split = L / tiles, tile = L - split * tiles;
    const int m0 = uniform(tile / n_tiles * kM), n0 = uniform(tile % n_tiles * kN);
    const int stages = H / kRtK * planes;  // (of whole steps)
    const int k0 = (int)((int64_t)stages * split / splits), k1 = (int)((int64_t)stages * (split + 1) / splits);

    const int lane = lane_id(), wave = uniform((int)threadIdx.x >> 6);
    const int wm = wave / kWN, wn = wave % kWN, fr = lane & 31, half = lane >> 5;
    uint32_t ao[kIA], bo[kIB];  // byte offsets from the tile's first row
    const int chunk = (lane & 7) ^ ((lane >> 4) & 3);  // (rows 8 i + lane / 8: the swizzle's third bit is i's)
#pragma unroll
    for (int i = 0; i < kIA; ++i)
        ao[i] = (uint32_t)(min(8 * (kIA * wave + i) + (lane >> 3), T - 1 - m0) * H) * 2 +
                16 * (chunk ^ (4 * ((kIA * wave + i) & 1)));
#pragma unroll
    for (int i = 0; i < kIB; ++i)
        bo[i] = (uint32_t)(min(8 * (kIB * wave + i) + (lane >> 3), E - 1 - n0) * H) * 2 +
                16 * (chunk ^ (4 * ((kIB * wave + i) & 1)));
    const char *xb = (const char*)(x + (size_t)m0 * H), *wb = (const char*)(w + (size_t)n0 * H);
    const size_t plane_bytes = (size_t)E * H * 2;
    const uint32_t la = lds_address(sA) + 1024 * kIA * wave, lb = lds_address(sB) + 1024 * kIB * wave;
    const int n_stages = k1 - k0;
    int next = n_stages > 0 ? k0 + ((int)(blockIdx.x >> 3) * planes) % n_stages : 0;  // the next stage to load
    size_t at = (size_t)(next / planes) * 128;
    int plane = planes - 1 - next % planes;
    auto issue = [&](uint32_t buf) {
        const char *a = xb + at, *b = wb + at + plane * plane_bytes;
#pragma unroll
        for (int i = 0; i < kIA; ++i) lds_dma16_from(a, ao[i], la + buf * (kM * 128) + 1024 * i);
#pragma unroll
        for (int i = 0; i < kIB; ++i) lds_dma16_from(b, bo[i], lb + buf * (kN * 128) + 1024 * i);
        const bool again = next + 1 == k1, wrap = plane == 0;
        next = again ? k0 : next + 1;
        at = again ? (size_t)(k0 / planes) * 128 : wrap ? at + 128 : at;
        plane = again ? planes - 1 - k0 % planes : wrap ? planes - 1 : plane - 1;
    };
    f32x16 acc[kMI][kNI];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    bf16x8 fa[2][kMI], fb[2][kNI];
    const uint32_t sw = (fr >> 1) & 7;
    auto read = [&](int set, uint32_t buf, int ks) {  // depth ks: chunk 2 ks + half
        const uint32_t c = ((2 * ks + half) ^ sw) << 4;
#pragma unroll
        for (int i = 0; i < kMI; ++i) fa[set][i] = as_bf16x8(*(const u32x4*)&sA[buf][((wm * kMI + i) * 32 + fr) * 128 + c]);
#pragma unroll
        for (int j = 0; j < kNI; ++j) fb[set][j] = as_bf16x8(*(const u32x4*)&sB[buf][((wn * kNI + j) * 32 + fr) * 128 + c]);
    };
    auto multiply = [&](int set) {
#pragma unroll
        for (int i = 0; i < kMI; ++i)
#pragma unroll
            for (int j = 0; j < kNI; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
    };
    if (k0 < k1) {
        issue(0);
        issue(1);
        issue(2);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * (kIA + kIB)));
        __syncthreads();
        read(0, 0, 0);
        uint32_t buf = 0;
        for (int s = k0; s < k1; ++s) {
            const uint32_t after = buf == 2 ? 0 : buf + 1;
            read(1, buf, 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            read(0, buf, 2);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1);
            __builtin_amdgcn_sched_barrier(0);
            read(1, buf, 3);
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(kIA + kIB));
            __syncthreads();
            read(0, after, 0);  // (after the last stage: not used)
            issue(buf);
            __builtin_amdgcn_sched_barrier(0);
            multiply(1);
            __builtin_amdgcn_sched_barrier(0);
            buf = after;
        }
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    }
    if (H % kRtK != 0 && split == splits - 1) {
        const int left = H % kRtK / 8;  // chunks of the last step
        for (int p = planes - 1; p >= 0; --p) {
            __syncthreads();  // every wave has left the buffer
            const char *a = xb + (size_t)(H / kRtK) * 128, *b = wb + (size_t)(H / kRtK) * 128 + p * plane_bytes;
#pragma unroll
            for (int i = 0; i < kIA; ++i)
                lds_dma16_at((chunk ^ (4 * ((kIA * wave + i) & 1))) < left ? a + ao[i] : (const char*)&kRouterZeros,
                             la + 1024 * i);
#pragma unroll
            for (int i = 0; i < kIB; ++i)
                lds_dma16_at((chunk ^ (4 * ((kIB * wave + i) & 1))) < left ? b + bo[i] : (const char*)&kRouterZeros,
                             lb + 1024 * i);
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                read(0, 0, ks);
                multiply(0);
            }
        }
    }
    float* o = out + (size_t)split * T * E;
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int t = m0 + (wm * kMI + i) * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
            if (t >= T) continue;
#pragma unroll
            for (int j = 0; j < kNI; ++j) {
                const int e = n0 + (wn * kNI + j) * 32 + fr;
                if (e < E) o[(size_t)t * E + e] = acc[i][j][v];
            }
        }
}

// The parts' sums, in part order, eight loads in flight.
__global__ __launch_bounds__(256) void router_join_kernel(const float* __restrict__ part, int64_t n,
                                                          int splits, float* __restrict__ scores) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.0f;
    int k = 0;
    for (; k + 8 <= splits; k += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = part[(size_t)(k + j) * n + i];
#pragma unroll
        for (int j = 0; j < 8; ++j) s += v[j];
    }
    for (; k < splits; ++k) s += part[(size_t)k * n + i];
    scores[i] = s;
}

// Which tiles T tokens take, and into how many parts K goes.
struct RouterPlan {
    bool dma;
    int kM, kN, n_tiles, tiles, splits;
    size_t w_bytes, part_bytes;  // workspace: fp32 W's parts, then the partial scores
};

// From so many 64 x 64 tiles on the large ones are faster (2048 x 7168 x 256, 128 tiles: 21 us against 28; 3000 x
// 7168 x 256, 188 tiles: 31 against 28; 1500 x 7168 x 384, 144 tiles: 24 against 22)
constexpr int kRouterDmaTiles = 148;

static RouterPlan router_plan(int T, int H, int E, bool f32) {
    RouterPlan p{};
    p.dma = ((int64_t)T + 63) / 64 * ((E + 63) / 64) >= kRouterDmaTiles;
    p.kM = p.dma ? 128 : 64;
    // of 256, 192 and 128 columns the width that loads the fewest rows, kN of W and 128 of x a tile
    // (32768 x 7168 x 384: 192 columns 203 us, 128 columns 229)
    p.kN = 64;
    if (p.dma) {
        int best = INT32_MAX;
        for (int kN : {256, 192, 128}) {
            const int rows = (E + kN - 1) / kN * (kN + 128);
            if (rows < best) best = rows, p.kN = kN;
        }
    }
    p.n_tiles = (E + p.kN - 1) / p.kN;
    p.tiles = (int)(((int64_t)T + p.kM - 1) / p.kM) * p.n_tiles;
    // one round of workgroups (two a CU of the small tiles), at least four K steps each
    const int steps = (H + kRtK - 1) / kRtK;
    p.splits = std::max(1, std::min((p.dma ? 256 : 512) / p.tiles, steps / 4));
    p.w_bytes = p.dma && f32 ? ((size_t)3 * E * H * 2 + 255) & ~size_t(255) : 0;
    p.part_bytes = p.splits > 1 ? (size_t)p.splits * T * E * sizeof(float) : 0;
    return p;
}

static moe_status check_router(int32_t T, int32_t H, int32_t E, int32_t w_dtype) {
    if (T < 0 || H < 1 || E < 1) return MOE_ERR_INVALID_ARG;
    if (w_dtype != MOE_ROUTER_W_BF16 && w_dtype != MOE_ROUTER_W_F32) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > MOE_MAX_DIM || E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    // (a launch holds fewer than 2^32 threads, 512 for 128 rows)
    if ((int64_t)T * E > INT32_MAX || T > 1 << 29) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

static size_t router_ws(int T, int H, int E, bool f32) {
    if (T <= kRouterDotT) return 0;
    const RouterPlan p = router_plan(T, H, E, f32);
    return p.w_bytes + p.part_bytes;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router_scores_workspace_size(int32_t T, int32_t H, int32_t E, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status s = check_router(T, H, E, MOE_ROUTER_W_BF16);
    if (s != MOE_OK) return s;
    *bytes = std::max(router_ws(T, H, E, false), router_ws(T, H, E, true));
    return MOE_OK;
}

extern "C" moe_status moe_router_scores(const uint16_t* x, int32_t T, int32_t H, const void* w,
                                        int32_t w_dtype, int32_t E, float* scores, void* ws,
                                        size_t ws_bytes, void* stream) {
    const moe_status s = check_router(T, H, E, w_dtype);
    if (s != MOE_OK || T == 0) return s;
    if (!x || !w || !scores || !aligned16(x) || !aligned16(w) || !aligned16(scores))
        return MOE_ERR_INVALID_ARG;
    const bool f32 = w_dtype == MOE_ROUTER_W_F32;
    const size_t need = router_ws(T, H, E, f32);
    if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    if (need && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    hipStream_t st = as_stream(stream);
    if (T <= kRouterDotT) {
        const int TT = T == 1 ? 1 : T == 2 ? 2 : T <= 4 ? 4 : 8;
        const dim3 grid((unsigned)E, (unsigned)((T + TT - 1) / TT)), block(kDotThreads);
#define MOE_DOT(N)                                                                        \
    case N:                                                                               \
        f32 ? router_dot_kernel<true, N><<<grid, block, 0, st>>>(x, T, H, w, E, scores)   \
            : router_dot_kernel<false, N><<<grid, block, 0, st>>>(x, T, H, w, E, scores); \
        break;
        switch (TT) { MOE_DOT(1) MOE_DOT(2) MOE_DOT(4) MOE_DOT(8) }
#undef MOE_DOT
        return launch_status();
    }
    const RouterPlan p = router_plan(T, H, E, f32);
    const int splits = p.splits;
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.w_bytes);
    float* o = splits > 1 ? part : scores;
    const dim3 grid((unsigned)(((int64_t)p.tiles * splits + 7) & ~int64_t(7)));
    if (p.dma) {
        const uint16_t* wb = static_cast<const uint16_t*>(w);
        if (f32) {
            uint16_t* parts = static_cast<uint16_t*>(ws);
            const int64_t chunks = (int64_t)E * H / 8;
            router_split_kernel<<<dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, st>>>(
                static_cast<const float*>(w), chunks, parts);
            wb = parts;
        }
        const int planes = f32 ? 3 : 1;
        if (p.kN == 256)
            router_dma_kernel<2, 2, 2, 4><<<grid, dim3(512), 0, st>>>(x, T, H, wb, planes, E, p.n_tiles, p.tiles, splits, o);
        else if (p.kN == 192)
            router_dma_kernel<1, 3, 4, 2><<<grid, dim3(512), 0, st>>>(x, T, H, wb, planes, E, p.n_tiles, p.tiles, splits, o);
        else
            router_dma_kernel<1, 2, 4, 2><<<grid, dim3(512), 0, st>>>(x, T, H, wb, planes, E, p.n_tiles, p.tiles, splits, o);
    } else if (f32) {
        router_gemm_kernel<true><<<grid, dim3(256), 0, st>>>(x, T, H, w, E, p.n_tiles, p.tiles, splits, o);
    } else {
        router_gemm_kernel<false><<<grid, dim3(256), 0, st>>>(x, T, H, w, E, p.n_tiles, p.tiles, splits, o);
    }
    moe_status r = launch_status();
    if (r != MOE_OK || splits == 1) return r;
    const int64_t n = (int64_t)T * E;
    router_join_kernel<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(part, n, splits, scores);
    return launch_status();
}
