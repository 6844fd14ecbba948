// moe_norm.hip -- RMS norm with the residual's addition, bf16 and FP8 outputs.
//
//     s = bf16(x + r)      (s = x without a residual)
//     v = fp32( s / sqrt(mean(s^2) + eps) * g )
//     y = bf16(v),  e_b = smallest integer with max|v| over 128-block b <= 448 * 2^e_b,
//     code = E4M3FN(v * 2^-e_b)
//
// One pass: a workgroup owns a row, every thread keeps its 8, 16 or 32 values of it in registers between
// the sum of squares and the outputs, so each input is read once and each output written once.  The sum
// of squares and the two products run in double and v is rounded to fp32 once: the squares of bf16
// values are exact there, and the codes then follow the exact v but for values within about 2^-50 of
// a rounding border.  (235 M values of the largest prefill batch need about 1.5 G double operations, a
// tenth of the time its bytes take.)
//
// Lane layout: chunk c of a row is its values 8c .. 8c + 7 (16 bytes); thread i owns chunks i,
// i + threads, ...  With a workgroup of whole waves a 128-block is 16 consecutive lanes, whose maximum
// is taken by DPP without LDS.
//
// Bound by HBM at many rows: 32768 x 7168 with everything on 374 us, 5.7 TB/s of reads and writes together (a
// copy of torch's reaches 4.8, a read alone 6.8).  One row: 3.5 us, the latency of load, sum and store.
#include "libmoe.h"
#include "moe_device.h"
#include "moe_host.h"
#include "moe_route.h"

#include <math.h>

namespace moe {

constexpr int kNormMaxThreads = 512;

// sum_out may be x or r (each value is read by the thread that writes it, before it writes), so
// those pointers are not restrict
template <int V>
__global__ __launch_bounds__(kNormMaxThreads) void rmsnorm_kernel(
    const uint16_t* x, const uint16_t* r, const uint16_t* __restrict__ g, int rows, int K,
    double eps, uint16_t* sum_out, uint16_t* __restrict__ y, uint8_t* __restrict__ codes,
    int8_t* __restrict__ exps, int exp_pitch) {
    __shared__ double part[2][kNormMaxThreads / kWave];  // two: a row's sums are read while the next row's arrive
    const int tid = (int)threadIdx.x, threads = (int)blockDim.x;
    const int chunks = K / 8, waves = threads / kWave;
    u32x4 gv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * threads;
        gv[i] = c < chunks ? *(const u32x4*)(g + 8 * c) : u32x4{0u, 0u, 0u, 0u};
    }
    int parity = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
        const size_t at = (size_t)row * K;
        u32x4 xv[V], rv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * threads;
            xv[i] = c < chunks ? __builtin_nontemporal_load((const u32x4*)(x + at + 8 * c)) : u32x4{0u, 0u, 0u, 0u};
        }
        if (r) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = tid + i * threads;
                rv[i] = c < chunks ? __builtin_nontemporal_load((const u32x4*)(r + at + 8 * c)) : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    xv[i][w] = f32x2_to_bf16x2(
                        bf16_to_f32((uint16_t)xv[i][w]) + bf16_to_f32((uint16_t)rv[i][w]),
                        bf16_to_f32((uint16_t)(xv[i][w] >> 16)) + bf16_to_f32((uint16_t)(rv[i][w] >> 16)));
            if (sum_out) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = tid + i * threads;
                    if (c < chunks) __builtin_nontemporal_store(xv[i], (u32x4*)(sum_out + at + 8 * c));
                }
            }
        }
        double sq = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const double a = (double)bf16_to_f32((uint16_t)xv[i][w]);
                const double b = (double)bf16_to_f32((uint16_t)(xv[i][w] >> 16));
                sq = fma(a, a, sq);
                sq = fma(b, b, sq);
            }
        sq = wave_sum_f64(sq);
        if (waves > 1) {
            if (lane_id() == 0) part[parity][tid / kWave] = sq;
            __syncthreads();
            sq = 0.0;
            for (int w = 0; w < waves; ++w) sq += part[parity][w];
        }
        const double scale = 1.0 / sqrt(sq / (double)K + eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = tid + i * threads;
            float v[8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                v[2 * w] = (float)((double)bf16_to_f32((uint16_t)xv[i][w]) * scale *
                                   (double)bf16_to_f32((uint16_t)gv[i][w]));
                v[2 * w + 1] = (float)((double)bf16_to_f32((uint16_t)(xv[i][w] >> 16)) * scale *
                                       (double)bf16_to_f32((uint16_t)(gv[i][w] >> 16)));
            }
            if (y && c < chunks) {
                u32x4 o;
#pragma unroll
                for (int w = 0; w < 4; ++w) o[w] = f32x2_to_bf16x2(v[2 * w], v[2 * w + 1]);
                *(u32x4*)(y + at + 8 * c) = o;
            }
            if (codes) {  // (K is a multiple of 128: the 16 lanes of a block are in or out together)
                float amax = 0.0f;
#pragma unroll
                for (int w = 0; w < 8; ++w) amax = fmaxf(amax, fabsf(v[w]));  // a NaN takes no part
                amax = __uint_as_float(row16_max_u32(__float_as_uint(amax)));
                const int e = isinf(amax) ? 127 : act_scale_exp(amax);
                uint32_t q[2];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(v[4 * w], -e), ldexpf(v[4 * w + 1], -e), 0, false);
                    q[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(ldexpf(v[4 * w + 2], -e), ldexpf(v[4 * w + 3], -e), lo, true);
                }
                if (c < chunks) {
                    *(uint2*)(codes + at + 8 * c) = make_uint2(q[0], q[1]);
                    if ((c & 15) == 0) exps[(size_t)row * exp_pitch + c / 16] = (int8_t)e;
                }
            }
        }
    }
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_rmsnorm_quantize_act(const uint16_t* x, const uint16_t* residual,
                                               const uint16_t* weight, int32_t rows, int32_t K,
                                               float eps, uint16_t* sum_out, uint16_t* y,
                                               uint8_t* codes, int8_t* exps, int32_t exp_pitch,
                                               void* stream) {
    if (rows < 0 || K < 1 || !(eps > 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARG;
    if ((codes == nullptr) != (exps == nullptr)) return MOE_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > MOE_MAX_DIM || (codes && K % 128 != 0)) return MOE_ERR_UNSUPPORTED;
    if (codes && exp_pitch < K / 128) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!x || !weight || (!y && !codes) || (sum_out && !residual)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)x, (const void*)residual, (const void*)weight, (const void*)sum_out,
                          (const void*)y, (const void*)codes, (const void*)exps})
        if (!aligned16(p)) return MOE_ERR_INVALID_ARG;
    // 1, 2 or 4 chunks a thread, so that a row is one workgroup of at most 512 threads
    const int chunks = K / 8;
    const int V = chunks <= kNormMaxThreads ? 1 : chunks <= 2 * kNormMaxThreads ? 2 : 4;
    const int threads = ((chunks + V - 1) / V + kWave - 1) / kWave * kWave;
    // (a launch holds fewer than 2^32 threads: longer batches loop)
    const dim3 grid((unsigned)(rows < (1 << 22) ? rows : (1 << 22))), block(threads);
    hipStream_t st = as_stream(stream);
#define MOE_NORM(N) rmsnorm_kernel<N><<<grid, block, 0, st>>>(x, residual, weight, rows, K, (double)eps, sum_out, y, codes, exps, exp_pitch)
    if (V == 1) MOE_NORM(1);
    else if (V == 2) MOE_NORM(2);
    else MOE_NORM(4);
#undef MOE_NORM
    return launch_status();
}
