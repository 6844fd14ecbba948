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
//   many tokens 128 x 128 tiles on the matrix cores (32x32x16 bf16), operands through LDS.  When
//               the tiles alone do not fill the chip, K is split over workgroups into fp32 partial
//               scores in the caller's workspace, and a second launch adds them in order.
//
// fp32 W goes to the matrix cores as three bf16 parts, w = hi + mid + lo (8 + 8 + 8 significand bits:
// exact for every finite w whose parts are not subnormal), so no bits of W are lost.
#include "libmoe.h"
#include "moe_device.h"
#include "moe_host.h"

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

// 128 x 128 tile, four waves of 64 x 64 each, K in steps of 64.  The next step's operands are loaded to
// registers before the current step's products and written to the other LDS buffer after them, one
// barrier a step (fp32 W, three planes of it, has room for one buffer and takes two barriers).
constexpr int kRtM = 128, kRtN = 128, kRtK = 64;
constexpr int kRtLd = kRtK * 2 + 16;  // LDS row bytes: 16 consecutive rows' 16-byte reads hit distinct banks

template <bool kF32>
__global__ __launch_bounds__(256, 2) void router_gemm_kernel(const uint16_t* __restrict__ x, int T,
                                                             int H, const void* __restrict__ w, int E,
                                                             int n_tiles, int tiles, int splits,
                                                             float* __restrict__ out) {
    constexpr int kPlanes = kF32 ? 3 : 1, kBufs = kF32 ? 1 : 2;
    __shared__ __attribute__((aligned(16))) uint8_t sA[kBufs][kRtM * kRtLd];
    __shared__ __attribute__((aligned(16))) uint8_t sB[kBufs][kPlanes][kRtN * kRtLd];
    // consecutive workgroups go to the 8 XCDs in turn: XCD i takes the contiguous range i of logical
    // tiles, so that the column tiles of a row tile share its x rows in one L2
    const int R8 = (tiles * splits + 7) / 8;
    const int L = ((int)blockIdx.x & 7) * R8 + ((int)blockIdx.x >> 3);
    if (L >= tiles * splits) return;
    const int split = L / tiles, tile = L - split * tiles;
    const int m0 = tile / n_tiles * kRtM, n0 = tile % n_tiles * kRtN;
    const int steps_all = (H + kRtK - 1) / kRtK;
    const int k0 = (int)((int64_t)steps_all * split / splits), k1 = (int)((int64_t)steps_all * (split + 1) / splits);

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, half = lane >> 5;
    // staging: thread loads 16-byte chunk tid % 8 of rows tid / 8 + 32 i; rows past the end read the last
    // row (not stored), chunks past H are zeros (both operands: 0 times garbage could be NaN)
    const int lc = tid & 7, lr = tid >> 3;
    const uint16_t* ap[4];
    const char* bp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ap[i] = x + (size_t)min(m0 + lr + 32 * i, T - 1) * H;
        bp[i] = (const char*)w + (size_t)min(n0 + lr + 32 * i, E - 1) * H * (kF32 ? 4 : 2);
    }
    u32x4 ra[4], rb[4][kF32 ? 2 : 1];
    auto load = [&](int step) {
        const int c = step * (kRtK / 8) + lc;
        const bool in = c < H / 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ra[i] = in ? ((const u32x4*)ap[i])[c] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int p = 0; p < (kF32 ? 2 : 1); ++p)
                rb[i][p] = in ? ((const u32x4*)bp[i])[kF32 ? 2 * c + p : c] : u32x4{0u, 0u, 0u, 0u};
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (lr + 32 * i) * kRtLd + lc * 16;
            *(u32x4*)&sA[buf][at] = ra[i];
            if constexpr (kF32) {
                u32x4 pl[3];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float a = __uint_as_float(rb[i][j >> 1][(2 * j) & 3]), b = __uint_as_float(rb[i][j >> 1][(2 * j + 1) & 3]);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        const uint32_t v = f32x2_to_bf16x2(a, b);
                        pl[p][j] = v;
                        const float ha = __uint_as_float(v << 16), hb = __uint_as_float(v & 0xffff0000u);
                        a = isfinite(ha) ? a - ha : 0.0f;  // an infinity or a NaN is all in the first part
                        b = isfinite(hb) ? b - hb : 0.0f;
                    }
                }
#pragma unroll
                for (int p = 0; p < 3; ++p) *(u32x4*)&sB[buf][p][at] = pl[p];
            } else {
                *(u32x4*)&sB[buf][0][at] = rb[i][0];
            }
        }
    };
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    auto compute = [&](int buf) {
#pragma unroll
        for (int ks = 0; ks < kRtK / 16; ++ks) {
            bf16x8 fa[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                fa[i] = as_bf16x8(*(const u32x4*)&sA[buf][(wm * 64 + i * 32 + fr) * kRtLd + ks * 32 + half * 16]);
#pragma unroll
            for (int p = kPlanes - 1; p >= 0; --p) {  // the small parts first
                bf16x8 fb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    fb[j] = as_bf16x8(*(const u32x4*)&sB[buf][p][(wn * 64 + j * 32 + fr) * kRtLd + ks * 32 + half * 16]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }
    };
    load(k0);
    stage(0);
    __syncthreads();
    for (int s = k0; s < k1; ++s) {
        const int buf = kBufs == 2 ? (s - k0) & 1 : 0;
        if (s + 1 < k1) load(s + 1);
        compute(buf);
        if (s + 1 < k1) {
            if (kBufs == 1) __syncthreads();
            stage(kBufs == 2 ? buf ^ 1 : 0);
        }
        __syncthreads();
    }
    // D layout: value v of a lane is row 8 (v / 4) + 4 half + v % 4, column fr
    float* o = out + (size_t)split * T * E;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int t = m0 + wm * 64 + i * 32 + 8 * (v >> 2) + 4 * half + (v & 3);
            if (t >= T) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = n0 + wn * 64 + j * 32 + fr;
                if (e < E) o[(size_t)t * E + e] = acc[i][j][v];
            }
        }
}

__global__ __launch_bounds__(256) void router_join_kernel(const float* __restrict__ part, int64_t n,
                                                          int splits, float* __restrict__ scores) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = part[i];
    for (int k = 1; k < splits; ++k) s += part[(size_t)k * n + i];
    scores[i] = s;
}

// K splits of the tile kernel: enough workgroups for two on every CU, at least four K steps each
static int router_splits(int T, int H, int E) {
    const int64_t tiles = (int64_t)((T + kRtM - 1) / kRtM) * ((E + kRtN - 1) / kRtN);
    const int steps = (H + kRtK - 1) / kRtK;
    const int64_t want = 512 / std::max<int64_t>(1, tiles);
    return (int)std::max<int64_t>(1, std::min<int64_t>(want, steps / 4));
}

static moe_status check_router(int32_t T, int32_t H, int32_t E, int32_t w_dtype) {
    if (T < 0 || H < 1 || E < 1) return MOE_ERR_INVALID_ARG;
    if (w_dtype != MOE_ROUTER_W_BF16 && w_dtype != MOE_ROUTER_W_F32) return MOE_ERR_INVALID_ARG;
    if (H % 8 != 0 || H > MOE_MAX_DIM || E > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)T * E > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

static size_t router_ws(int T, int H, int E) {
    if (T <= kRouterDotT) return 0;
    const int s = router_splits(T, H, E);
    return s > 1 ? (size_t)s * T * E * sizeof(float) : 0;
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_router_scores_workspace_size(int32_t T, int32_t H, int32_t E, size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status s = check_router(T, H, E, MOE_ROUTER_W_BF16);
    if (s != MOE_OK) return s;
    *bytes = router_ws(T, H, E);
    return MOE_OK;
}

extern "C" moe_status moe_router_scores(const uint16_t* x, int32_t T, int32_t H, const void* w,
                                        int32_t w_dtype, int32_t E, float* scores, void* ws,
                                        size_t ws_bytes, void* stream) {
    const moe_status s = check_router(T, H, E, w_dtype);
    if (s != MOE_OK || T == 0) return s;
    if (!x || !w || !scores || !aligned16(x) || !aligned16(w) || !aligned16(scores))
        return MOE_ERR_INVALID_ARG;
    const size_t need = router_ws(T, H, E);
    if (need && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    if (need && !aligned16(ws)) return MOE_ERR_INVALID_ARG;
    hipStream_t st = as_stream(stream);
    const bool f32 = w_dtype == MOE_ROUTER_W_F32;
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
    const int splits = router_splits(T, H, E);
    const int n_tiles = (E + kRtN - 1) / kRtN, tiles = (T + kRtM - 1) / kRtM * n_tiles;
    const int64_t wgs = ((int64_t)tiles * splits + 7) & ~int64_t(7);
    float* o = splits > 1 ? (float*)ws : scores;
    const dim3 grid((unsigned)wgs), block(256);
    if (f32) router_gemm_kernel<true><<<grid, block, 0, st>>>(x, T, H, w, E, n_tiles, tiles, splits, o);
    else router_gemm_kernel<false><<<grid, block, 0, st>>>(x, T, H, w, E, n_tiles, tiles, splits, o);
    moe_status r = launch_status();
    if (r != MOE_OK || splits == 1) return r;
    const int64_t n = (int64_t)T * E;
    router_join_kernel<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>((const float*)ws, n, splits, scores);
    return launch_status();
}
