// moe_few.hip -- a whole MoE layer for up to eight tokens in two launches.
//
// Decode of a few sequences reads every touched expert's three matrices once and does next to no
// arithmetic on them (2 to 16 flops a byte): the weights' bytes bound it, and around them the launches and
// the steps between them.  The layer is two streaming kernels:
//
//   few_gate_up   every workgroup routes the tokens for itself (scores are a few KB), then streams gate and
//                 up rows of the touched experts: h_te = SiLU(Wg_e x_t) * (Wu_e x_t), stored as w_te * h_te.
//   few_down      out_t = S_t + sum_e Wd_e (w_te h_te): with the gate weights already in h, the combine is
//                 the same sum as the projection's.  A workgroup owns a few columns of out and runs one
//                 product whose contraction is all touched experts' I in a row; no y, no permutation.
//
// Matrix tile (16x16x32 bf16, weights expanded exactly as in moe_ffn.hip): row m is token m, for every
// expert, so that the activations need no gather: in few_gate_up all eight tokens' rows are multiplied and
// those not routed to the expert are not stored; in few_down a token's sum takes the experts that it
// is routed to, by a select when the expert's blocks end (so that what a weight does to one token's sum
// cannot reach another's).  few_gate_up with MXFP4 weights takes the scaled 16x16x128 instruction instead:
// weights and their scales as they are stored, x as two E4M3 codes in rows t and 8 + t (few_codes).
//
// h keeps fp32's precision: w_te * h_te goes on as two bf16 values, hi + lo (16 significand bits), in rows
// t and 8 + t of the tile that eight tokens leave half empty, at no matrix instruction more.
//
// Work split: 8-wave workgroups, every wave a part of K.  few_gate_up: one workgroup per CU, looping over
// units of 8 h columns (8 gate + 8 up rows); each wave streams its K part of unit after unit through a
// ring of register stages that never drains between units, and the waves' sums meet in LDS once a
// unit.  x (all tokens) stays in LDS, so that the ring's loads are weights alone: loads complete in
// order, and a load of x behind them would wait for all of them.  The scores and x are loaded first, then
// the shared expert's first unit, whose loads are in flight while the routing runs.  few_down: a wave takes
// an even share of all (expert, 128-block) stages of the workgroup's columns, and the waves' sums meet once
// at the end; where the columns alone leave CUs idle, several workgroups share the stages of a tile.
//
// Measured, 7168 x 2048, 256 experts, top-8 and a shared expert: 1 token 67 us FP8 (gate/up 45, down 23; the
// weights alone 58 at 6.8 TB/s), 46 us MXFP4, 125 us bf16; 8 tokens 367 to 392 us FP8, 234 to 248 us MXFP4 (gate/up
// 147 to 156 at 6.2 TB/s, down 88 to 93: bound by the instructions that expand 4-bit weights).  4 x 256 x 128:
// 10 us, two dependent launches of 5.7 and 3.9.
#include "libmoe.h"
#include "moe_device.h"
#include "moe_ffn.h"
#include "moe_host.h"
#include "moe_lds.h"
#include "moe_ring.h"
#include "moe_route.h"

#include <algorithm>

namespace moe {

constexpr int kFewT = MOE_FEW_MAX_TOKENS;
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewXBytes = 114816;   // LDS for x: 8 rows of 7168 bf16, padded by 16 bytes each ...
constexpr int kFewCodeBytes = kFewXBytes + 16 * kFewT;  // ... or 16 of codes, as many more
constexpr int kFewList = kFewT * MOE_MAX_TOPK;  // most touched experts
constexpr int kFewShared = 0xFFFF;   // the shared expert's id in the list
constexpr int kFewParts = 8;         // most workgroups of a few_down tile
// workspace: list (count, then id | token mask << 16), arrivals of few_down's tiles, h, their parts' sums
constexpr size_t kFewCounts = 2048, kFewHead = kFewCounts + MOE_MAX_DIM / 32 * sizeof(int32_t);
static_assert((kFewList + 2) * sizeof(int32_t) <= kFewCounts, "the list fits before the arrivals");

struct FewArgs {
    const float* scores;
    const uint16_t* x;
    int T, E, k, H, I, score_fn, renorm;
    const void *g, *u, *d;     // routed experts
    const void *sg, *su, *sd;  // their scales
    const void *xg, *xu, *xd;  // the shared expert (null: none)
    const void *xsg, *xsu, *xsd;
    int32_t* ids;
    float* wts;
    int32_t* list;
    uint16_t* h;  // [list index][2 T][pitch]: hi rows 0..T-1, lo rows T..2T-1
    int pitch;    // I rounded up to 256 (two blocks), the rest zeros
    int down_g, parts;  // few_down: 16-column groups of a tile, workgroups of a tile
    int32_t* arrived;   // [tile]
    float* part;        // [part][tile][group][8][16]
    uint16_t* out;
};

constexpr int kFewBF16 = 0, kFewFP8 = 1, kFewMX = 2;

// A stage is 128 bytes (a cache line) of each of 16 weight rows.  A load instruction covers 8 rows; the
// stage then goes through the wave's LDS rows once, to change from that layout to the matrix operand's.
template <int kFmt>
struct FewFmt {
    static constexpr int kSV = kFmt == kFewMX ? 256 : kFmt == kFewFP8 ? 128 : 64;  // values of a row per stage
    static constexpr int kNM = kSV / 32;  // matrix instructions per stage and 16 rows
    __device__ static size_t row_bytes(int K) { return kFmt == kFewMX ? K / 2 : kFmt == kFewFP8 ? K : 2 * (size_t)K; }
    // The value (within the stage) of the first of the 8 values that lane quarter kq holds in
    // instruction i: a quarter's values are consecutive weight bytes, a scale group in MXFP4
    __device__ static int value(int i, int kq) {
        return kFmt == kFewMX ? (i >> 2) * 128 + kq * 32 + (i & 3) * 8 : kq * (kSV / 4) + i * 8;
    }
};
constexpr int kFewRing = 4;       // stages in flight a wave and 16 rows: 8 KB, 64 KB a CU
constexpr int kFewLD = 128 + 16;  // LDS row stride of a stage: conflict-free reads

// MXFP4 scales: the stage's 16 kG rows have 8 bytes each, far apart.  One load instruction takes them all,
// lane 2 r + b the dword of row r's block b: two lanes a row, 32 accesses.  (With every lane loading the
// dword of its own row and block, four quarters asking for the same one, the address unit took 64 cycles for
// each of 2 kG instructions a stage, and bounded the kernel: 284 K of 415 K cycles at 8 tokens.)
__device__ __forceinline__ int mx_row(int lane, int kG) { return (lane >> 1) & (16 * kG - 1); }

// One stage of kG times 16 weight rows, times the activation fragments x(i).  Each group goes through the
// same LDS rows (a wave's LDS operations complete in order), all groups before the first product; the
// products run in two chains a group, so that a wave has 2 kG independent ones in flight.  The chains add
// to acc; FP8 (post-scaled: acc += stage * sc) starts them at zero.
// MXFP4: sv holds the stage's scale dwords (four scale bytes, one a quarter, per row and block) as
// mx_row() says, row r's block b in lane 2 r + b.  The conversion takes its scale operand's exponent
// field and nothing else, so the quarter's byte is rotated there with its neighbours left in the sign
// and mantissa.  A last stage of one block has its second block's x as zeros (and the first block's
// weights again).
template <int kFmt, int kG, typename X>
__device__ __forceinline__ void few_stage(uint8_t* lds, const u32x4 (*w)[2], int lane, uint32_t sv, float sc,
                                          X&& x, f32x4 (*acc)[2]) {
    using F = FewFmt<kFmt>;
    const int m = lane & 15, kq = lane >> 4;
    const uint8_t* row = lds + m * kFewLD;
    u32x4 v[kG][2];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *(u32x4*)&lds[(8 * i + (lane >> 3)) * kFewLD + (lane & 7) * 16] = w[g][i];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) v[g][i] = *(const u32x4*)&row[kFmt == kFewMX ? 64 * i + 16 * kq : 32 * kq + 16 * i];
        __builtin_amdgcn_wave_barrier();
    }
    float f[kG][2];
    if (kFmt == kFewMX) {
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const uint32_t w4 = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (2 * (16 * g + m) + b), (int)sv);
                f[g][b] = __uint_as_float(__builtin_amdgcn_alignbit(w4, w4, (8 * kq + 9) & 31));
            }
    }
    constexpr int kHalf = F::kNM / 2;
    f32x4 q[kG][2];
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int c = 0; c < 2; ++c) q[g][c] = kFmt == kFewFP8 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[g][c];
#pragma unroll
    for (int j = 0; j < kHalf; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int i = c * kHalf + j;
            const bf16x8 xv = x(i);
#pragma unroll
            for (int g = 0; g < kG; ++g) {
                const uint32_t* u = (const uint32_t*)v[g];
                const bf16x8 wv = kFmt == kFewFP8 ? fp8x8_to_bf16x8(u[2 * (i & 3)], u[2 * (i & 3) + 1])
                                : kFmt == kFewMX  ? fp4x8_to_bf16x8(u[i], f[g][i >> 2])
                                                  : as_bf16x8(v[g][i & 1]);
                q[g][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, wv, q[g][c], 0, 0, 0);
            }
        }
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        if (kFmt == kFewFP8) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[g][0][r] = fmaf(q[g][0][r] + q[g][1][r], sc, acc[g][0][r]);
        } else {
            acc[g][0] = q[g][0], acc[g][1] = q[g][1];
        }
        // the sums are taken here, not where they are next used: a scale that outlived its slot would be
        // copied to another register every round, and that copy would wait for the whole ring
        asm volatile("" : "+v"(acc[g][0]), "+v"(acc[g][1]));
    }
}

typedef int i32x8 __attribute__((__vector_size__(8 * sizeof(int))));
constexpr int kFewFP8Codes = 0, kFewFP4Codes = 4;  // the scaled instruction's operand formats

// Eight bf16 values of x (16 consecutive lanes have a 128-block) as two E4M3 values each, x = 2^e hi +
// 2^(e - 4) lo: hi holds the first four significand bits, and what is left is at most half of hi's last
// place, 16 2^e, with four significand bits: lo holds it exactly.  Only where hi is subnormal (below 2^-14 of
// the block's largest, which is over 224 2^e) may lo lose bits, at most 2^-14 2^e: less than 2^-21 of
// the block's largest value.  Returns e (>= -123, so that e - 4 is an E8M0 scale too).
__device__ __forceinline__ int few_codes(u32x4 v, uint2& hi, uint2& lo) {
    float f[8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));  // (a NaN takes no part)
    }
    amax = __uint_as_float(row16_max_u32(__float_as_uint(amax)));
    const int e = isinf(amax) ? 127 : max(-123, act_scale_exp(amax));
    uint32_t h[2], l[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * w + i] = ldexpf(f[4 * w + i], -e);
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * w], f[4 * w + 1], 0, false);
        c = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * w + 2], f[4 * w + 3], c, true);
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(c, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(c, true);
        h[w] = (uint32_t)c;
        c = __builtin_amdgcn_cvt_pk_fp8_f32(16.0f * (f[4 * w] - a[0]), 16.0f * (f[4 * w + 1] - a[1]), 0, false);
        l[w] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(16.0f * (f[4 * w + 2] - b[0]), 16.0f * (f[4 * w + 3] - b[1]), c, true);
    }
    hi = make_uint2(h[0], h[1]);
    lo = make_uint2(l[0], l[1]);
    return e;
}

// An MXFP4 stage of kG times 16 weight rows times x in codes (few_codes): the scaled 16x16x128
// instruction takes both operands' codes and scales as they are, a block each.  Its 4-bit operand has 32
// consecutive values in a lane quarter, kq's block of scale group kq; the 8-bit one 16 from 16 kq and 16 from
// 64 + 16 kq.  se: the E8M0 scales of this lane's row of x, blocks 0 and 1 in bytes 0 and 1.
template <int kG>
__device__ __forceinline__ void few_stage_codes(uint8_t* lds, const u32x4 (*w)[2], int lane, uint32_t sv, int se,
                                                const i32x8 (&x)[2], f32x4 (*acc)[2]) {
    const int m = lane & 15, kq = lane >> 4;
    const uint8_t* row = lds + m * kFewLD;
    u32x4 v[kG][2];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *(u32x4*)&lds[(8 * i + (lane >> 3)) * kFewLD + (lane & 7) * 16] = w[g][i];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < 2; ++i) v[g][i] = *(const u32x4*)&row[64 * i + 16 * kq];
        __builtin_amdgcn_wave_barrier();
    }
    int f[kG][2];
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            f[g][b] = (int)((uint32_t)__builtin_amdgcn_ds_bpermute(4 * (2 * (16 * g + m) + b), (int)sv) >> (8 * kq));
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        const i32x8 w0 = {(int)v[g][0][0], (int)v[g][0][1], (int)v[g][0][2], (int)v[g][0][3], 0, 0, 0, 0};
        const i32x8 w1 = {(int)v[g][1][0], (int)v[g][1][1], (int)v[g][1][2], (int)v[g][1][3], 0, 0, 0, 0};
        acc[g][0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x[0], w0, acc[g][0], kFewFP8Codes, kFewFP4Codes,
                                                                    0, se, 0, f[g][0]);
        acc[g][1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x[1], w1, acc[g][1], kFewFP8Codes, kFewFP4Codes,
                                                                    1, se, 0, f[g][1]);
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) asm volatile("" : "+v"(acc[g][0]), "+v"(acc[g][1]));  // (as in few_stage)
}

template <int kG>
__device__ __forceinline__ void few_clear(f32x4 (*acc)[2]) {
#pragma unroll
    for (int g = 0; g < kG; ++g) acc[g][0] = acc[g][1] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Waits for this wave's LDS operations, then the workgroup; loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// kG: 16-row groups (8 gate + 8 up rows) of a unit
template <int kFmt, int kG>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs a) {
    using F = FewFmt<kFmt>;
    constexpr int D = kFewRing, kCols = 8 * kG;
    constexpr bool kCodes = kFmt == kFewMX;  // x in LDS: E4M3 codes (rows t hi, T + t lo), else bf16
    __shared__ __attribute__((aligned(16))) uint8_t sX[kCodes ? kFewCodeBytes : kFewXBytes];
    __shared__ __attribute__((aligned(16))) uint8_t sE[kCodes ? kFewCodeBytes / 128 + 2 * kFewT : 2];  // the codes' E8M0 scales
    __shared__ __attribute__((aligned(16))) uint8_t sZero[128];
    __shared__ __attribute__((aligned(16))) uint8_t sW[kFewWaves][16 * kFewLD];
    __shared__ float red[2][kFewWaves][kG][32 * 4];
    __shared__ int32_t sids[kFewList];
    __shared__ float swts[kFewList];
    __shared__ uint32_t bits[MOE_MAX_EXPERTS / 32];
    __shared__ int32_t base[MOE_MAX_EXPERTS / 32];  // touched experts before the word's
    __shared__ uint32_t list[kFewList];             // touched experts, ascending: id | token mask << 16
    __shared__ float wt[kFewList][kFewT];           // their gate weights for each token
    __shared__ int32_t count;

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int m = lane & 15, kq = lane >> 4;
    const int T = a.T, H = a.H, I = a.I, k = a.k;
    const gbytes Wg = held(a.g), Wu = held(a.u), Xg = held(a.xg), Xu = held(a.xu);
    const gbytes Sg = held(a.sg), Su = held(a.su), XSg = held(a.xsg), XSu = held(a.xsu);
    const int grid = (int)gridDim.x;
    const int sh = a.xg != nullptr ? 1 : 0;
    const int tiles = I / kCols;
    const int kb_all = H / 128, st_all = (H + F::kSV - 1) / F::kSV;
    const int st0 = st_all * wave / kFewWaves, ns = st_all * (wave + 1) / kFewWaves - st0;
    const size_t row_bytes = F::row_bytes(H);
    const int lrow = lane >> 3, lchunk = lane & 7;
    uint8_t* lds = sW[wave];

    // ---- the ring of weight stages
    u32x4 bw[D][kG][2];
    float sc[D];              // FP8: the scale of this lane's column (gate for columns 0..7, up for 8..15)
    uint32_t mx[D];           // MXFP4: the stage's scales, a row and block a lane (mx_row)
    const int mr = mx_row(lane, kG);
    int iu = (int)blockIdx.x, ib = 0;   // issue cursor: unit, stage of this wave
    int n_units = sh * tiles;  // (the shared expert's, until the routing is known)
    gbytes gp{}, up{};         // the unit's gate / up rows, at the wave's part of K (uniform)
    gbytes sp{};               // this lane's scales
    const uint32_t wofs = (uint32_t)lrow * (uint32_t)row_bytes + lchunk * 16;  // this lane's bytes of a stage
    auto unit_of = [&](int unit) {  // pointers of a unit
        const int u = unit / tiles, n0 = (unit - u * tiles) * kCols;
        const bool xg = u < sh;
        const int e = xg ? 0 : uniform((int)(list[u - sh] & 0xFFFFu));
        const size_t at = ((size_t)e * I + n0) * row_bytes + (size_t)st0 * 128;
        gp = pick(xg, Xg, Wg) + at;
        up = pick(xg, Xu, Wu) + at;
        const bool gate = (kFmt == kFewMX ? mr & 8 : m & 8) == 0;
        const gbytes s = pick(gate, pick(xg, XSg, Sg), pick(xg, XSu, Su));
        if (kFmt == kFewFP8) sp = s + 4 * (((size_t)e * (I / 128) + n0 / 128) * kb_all + st0);
        if (kFmt == kFewMX) sp = s + ((size_t)e * I + n0 + 8 * (mr >> 4) + (mr & 7)) * (H / 32);
    };
    // loads of the cursor's stage into slot d, then one step of the cursor; past the last unit the last
    // stage is loaded again (into slots that are not used), so that the loop's loads are unconditional
    auto issue = [&](auto tag) {
        constexpr int d = decltype(tag)::value;
        const int kb = 2 * (st0 + ib);  // MXFP4
        // a short last MXFP4 stage: the chunks of the missing block reload the first
        const uint32_t ofs = kFmt == kFewMX && kb + 1 >= kb_all && lchunk >= 4 ? wofs - 64 : wofs;
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            const size_t at = (size_t)8 * g * row_bytes + (size_t)ib * 128;
            bw[d][g][0] = __builtin_nontemporal_load((gvec<u32x4>)(gp + at + ofs));
            bw[d][g][1] = __builtin_nontemporal_load((gvec<u32x4>)(up + at + ofs));
        }
        if (kFmt == kFewFP8) sc[d] = *(gvec<float>)(sp + 4 * ib);
        if (kFmt == kFewMX) mx[d] = *(gvec<uint32_t>)(sp + 4 * min(kb + (lane & 1), kb_all - 1));
        if (ib + 1 < ns) {
            ++ib;
        } else if (iu + grid < n_units) {
            iu += grid;
            ib = 0;
            unit_of(iu);
        }
    };

    // ---- loads in the order they are needed in: the scores (token t by wave t), x, and the shared expert's
    // first stages, which are in flight while the routing runs
    float sv[MOE_MAX_EXPERTS / kWave];
    if (wave < T) {
#pragma unroll
        for (int i = 0; i < MOE_MAX_EXPERTS / kWave; ++i)
            if (kWave * i < a.E) {
                const int e = lane + kWave * i;
                sv[i] = e < a.E ? a.scores[(size_t)wave * a.E + e] : 0.0f;
            }
    }
    constexpr int kX = (kFewXBytes / 16 + kFewThreads - 1) / kFewThreads;  // chunks of x a thread, at most
    const int chunks = H / 8;
    u32x4 xc[kX];
#pragma unroll
    for (int i = 0; i < kX; ++i)
        if (kFewThreads * i < T * chunks) xc[i] = ((const u32x4*)a.x)[min(tid + kFewThreads * i, T * chunks - 1)];
    __builtin_amdgcn_sched_barrier(0);
    const int pre = iu < n_units ? min(D, ns) : 0;
    if (pre > 0) {
        unit_of(iu);
        each_slot<D>([&](auto tag) {
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
        });
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(D * (2 * kG + (kFmt == kFewBF16 ? 0 : 1))));  // (all but the ring's)
        if (pre == ns) {  // the cursor back to the unit's last stage: slots from `pre` on are loaded again below
            iu = (int)blockIdx.x;
            ib = ns - 1;
        }
    } else {
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    }
    // ---- x into LDS, rows padded by 16 bytes (row m starts 4 m banks on)
    const int xrow = (kCodes ? H : 2 * H) + 16, epitch = (kb_all + 1) & ~1;
    const uint32_t inv = 0xFFFFFFFFu / (uint32_t)chunks + 1;  // c / chunks is the product's high half (c < 2^13)
    if (tid < 8) *(u32x4*)&sZero[16 * tid] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        const int c = tid + kFewThreads * i;
        if (c >= T * chunks) break;
        const int t = (int)__umulhi((uint32_t)c, inv), j = c - t * chunks;
        if (kCodes) {  // (chunks is a multiple of 16: a block's 16 lanes are here together)
            uint2 hi, lo;
            const int e = few_codes(xc[i], hi, lo);
            *(uint2*)&sX[t * xrow + 8 * j] = hi;
            *(uint2*)&sX[(T + t) * xrow + 8 * j] = lo;
            if ((j & 15) == 0) {
                const int b = j / 16;
                sE[t * epitch + b] = (uint8_t)(127 + e);
                sE[(T + t) * epitch + b] = (uint8_t)(123 + e);
                if (b + 1 == kb_all && b + 1 < epitch) sE[t * epitch + b + 1] = sE[(T + t) * epitch + b + 1] = 127;
            }
        } else {
            *(u32x4*)&sX[t * xrow + 16 * j] = xc[i];
        }
    }
    // ---- routing
    if (tid < MOE_MAX_EXPERTS / 32) bits[tid] = 0u;
    if (tid < kFewList) list[tid] = 0u;
    if (wave < T) {
        int32_t* ri = sids + wave * k;
        float* rw = swts + wave * k;
        if (a.E <= 64) route_values<1>(sv, a.E, k, a.score_fn, a.renorm, ri, rw);
        else if (a.E <= 128) route_values<2>(sv, a.E, k, a.score_fn, a.renorm, ri, rw);
        else if (a.E <= 256) route_values<4>(sv, a.E, k, a.score_fn, a.renorm, ri, rw);
        else if (a.E <= 512) route_values<8>(sv, a.E, k, a.score_fn, a.renorm, ri, rw);
        else route_values<16>(sv, a.E, k, a.score_fn, a.renorm, ri, rw);
    }
    __syncthreads();
    if (tid < T * k) atomicOr(&bits[sids[tid] >> 5], 1u << (sids[tid] & 31));
    __syncthreads();
    if (wave == 0) {
        const int n = __popc(lane < MOE_MAX_EXPERTS / 32 ? bits[lane] : 0u), incl = wave_inclusive_scan(n);
        if (lane < MOE_MAX_EXPERTS / 32) base[lane] = incl - n;
        if (lane == kWave - 1) count = incl;
    }
    __syncthreads();
    if (tid < T * k) {
        const int e = sids[tid], t = tid / k;
        const int u = base[e >> 5] + __popc(bits[e >> 5] & ((1u << (e & 31)) - 1u));
        atomicOr(&list[u], (uint32_t)e | 1u << (16 + t));
        wt[u][t] = swts[tid];
    }
    __syncthreads();
    const int n_exp = uniform(count) + sh;
    n_units = n_exp * tiles;
    if (blockIdx.x == 0) {  // for the second kernel and the caller
        for (int i = tid; i < T * k; i += kFewThreads) {
            a.ids[i] = sids[i];
            a.wts[i] = swts[i];
        }
        for (int i = tid; i < n_exp; i += kFewThreads)
            a.list[1 + i] = i < sh ? (int32_t)(kFewShared | ((1u << T) - 1) << 16) : (int32_t)list[i - sh];
        if (tid == 0) a.list[0] = n_exp;
        if (a.parts > 1)
            for (int i = tid; i < H / 32; i += kFewThreads) a.arrived[i] = 0;
    }
    if ((int)blockIdx.x >= n_units) return;  // (whole workgroups)
    if (ns > 0) {
        // the issue cursor: at the shared unit's stage `pre`, or at the first unit's start
        if (pre == 0) {
            iu = (int)blockIdx.x;
            ib = 0;
            unit_of(iu);
        } else if (pre == ns && iu + grid < n_units) {
            // the whole shared unit is loaded, and its successor was not known yet
            iu += grid;
            ib = 0;
            unit_of(iu);
        }
        each_slot<D>([&](auto tag) {
            if (decltype(tag)::value >= pre) issue(tag);
        });
        // the conditional loads above end here, so that the loop's waits count its own loads only
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    }

    // this lane's x row, at its quarter; rows past the last token repeat token 0 (not stored)
    // (codes: rows 8 + t are the lo codes)
    const int xr = kCodes ? ((m & 7) < T ? (m & 7) : 0) + (m < 8 ? 0 : T) : m < T ? m : 0;
    const uint8_t* xm = sX + xr * xrow + (kCodes ? 16 * kq : 2 * F::value(0, kq));
    const uint8_t* em = sE + xr * epitch;
    f32x4 acc[kG][2];
    few_clear<kG>(acc);
    auto compute = [&](auto tag, int st) {
        constexpr int d = decltype(tag)::value;
        if constexpr (kCodes) {
            const uint8_t* x0 = xm + st * F::kSV;
            const uint8_t* x1 = 2 * st + 1 >= kb_all ? sZero : x0 + 128;  // the second block
            i32x8 xv[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const u32x4 p = *(const u32x4*)(b ? x1 : x0), q = *(const u32x4*)((b ? x1 : x0) + 64);
#pragma unroll
                for (int i = 0; i < 4; ++i) xv[b][i] = (int)p[i], xv[b][4 + i] = (int)q[i];
            }
            few_stage_codes<kG>(lds, bw[d], lane, mx[d], *(const uint16_t*)(em + 2 * st), xv, acc);
        } else {
            const uint8_t* x0 = xm + 2 * st * F::kSV;
            bf16x8 xv[F::kNM];
#pragma unroll
            for (int i = 0; i < F::kNM; ++i) xv[i] = as_bf16x8(*(const u32x4*)&x0[16 * i]);
            few_stage<kFmt, kG>(lds, bw[d], lane, 0u, kFmt == kFewFP8 ? sc[d] : 0.0f, [&](int i) { return xv[i]; }, acc);
        }
    };
    int cu = (int)blockIdx.x, seq = 0;  // the unit being computed
    // Joins the waves' sums of the unit; kG of the waves, in turn, then finish its columns: wave
    // kG seq + g takes group g, lane 8 t + c token t's column c.
    auto finish = [&]() {
#pragma unroll
        for (int g = 0; g < kG; ++g) {
            // tokens 0..7 are rows 0..7: lanes 0..31 (and rows 8..15 their lo parts: lanes 32..63)
            f32x4 v = kFmt == kFewFP8 ? acc[g][0] : acc[g][0] + acc[g][1];
            if (kCodes) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] += __shfl_xor(v[r], 32, kWave);
            }
            if (lane < 32) *(f32x4*)&red[seq & 1][wave][g][4 * lane] = v;
        }
        few_clear<kG>(acc);
        lds_barrier();
        const int g = (wave - kG * seq) & (kFewWaves - 1);
        if (g < kG) {
            const int t = lane >> 3, c = lane & 7;
            // D layout: token t is value t % 4 of lanes 16 (t / 4) + column; gate column c, up column 8 + c
            const int at = 64 * (t >> 2) + 4 * c + (t & 3);
            float gv = 0.0f, uv = 0.0f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) {
                gv += red[seq & 1][w][g][at];
                uv += red[seq & 1][w][g][at + 32];
            }
            const int u = cu / tiles, n0 = (cu - u * tiles) * kCols;
            const uint32_t mask = u < sh ? (1u << T) - 1 : list[u - sh] >> 16;
            const float hv = (u < sh ? 1.0f : wt[u - sh][t]) * silu_mul(gv, uv);
            if (mask >> t & 1) {
                const uint16_t hi = f32_to_bf16(hv);
                const float rest = hv - bf16_to_f32(hi);
                uint16_t* h = a.h + ((size_t)u * 2 * T + t) * a.pitch + n0 + 8 * g + c;
                h[0] = hi;
                h[(size_t)T * a.pitch] = f32_to_bf16(isfinite(rest) ? rest : 0.0f);
                if (n0 + 8 * g + 8 == I)  // the row's padding
                    for (int i = 8; I + i <= a.pitch; i += 8) h[i] = h[(size_t)T * a.pitch + i] = 0;
            }
        }
        ++seq;
        cu += grid;
    };
    const int units = (n_units - (int)blockIdx.x + grid - 1) / grid;
    if (ns == 0) {  // fewer stages than waves: this wave only takes part in the joins
        for (int i = 0; i < units; ++i) finish();
        return;
    }
    int cs = 0;
    ring_loop<D>(units * ns, [&](auto tag) {
        compute(tag, st0 + cs);
        __builtin_amdgcn_sched_barrier(0);
        issue(tag);
        __builtin_amdgcn_sched_barrier(0);
        if (++cs == ns) {
            cs = 0;
            finish();
        }
    });
}

// kG: 16-column groups of a workgroup; TT: at least T.  Up to four tokens a stage's h rows, hi and lo of TT
// tokens, are loaded as whole lines, 1024 / (2 kSV) rows an instruction, and go through LDS to the operand's
// layout; eight fill that layout's 16 rows, and are loaded in it.  (7168 x 2048, MXFP4: the layer of 1 to 4 tokens
// took 2 to 3% longer the other way, FP8 and bf16 1%; of 8 tokens this phase took 98 us against 93.)
template <int kFmt, int kG, int TT>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs a) {
    using F = FewFmt<kFmt>;
    constexpr int D = kFmt == kFewMX && TT == 8 ? 3 : kFewRing;  // (an MXFP4 stage holds two blocks of h)
    constexpr int kRowLanes = F::kSV / 8, kRows = 64 / kRowLanes;  // of an h load
    constexpr bool kDirect = TT == 8;
    constexpr int kHL = kDirect ? F::kNM : 2 * TT <= kRows ? 1 : 2 * TT / kRows, kHLD = 2 * F::kSV + 16;
    constexpr int kHO = kDirect ? 1 : kHL;  // offsets a lane
    __shared__ __attribute__((aligned(16))) uint8_t sW[kFewWaves][16 * kFewLD];
    __shared__ __attribute__((aligned(16))) uint8_t sH[kFewWaves][kDirect ? 16 : 2 * TT * kHLD];
    __shared__ f32x4 red[kFewWaves][kG][kWave];
    __shared__ uint32_t list[kFewList + 1];
    __shared__ int before;

    const int tid = (int)threadIdx.x, lane = lane_id(), wave = uniform(tid >> 6);
    const int m = lane & 15, kq = lane >> 4;
    const int T = a.T, H = a.H, I = a.I;
    const gbytes Wd = held(a.d), Xd = held(a.xd), Sd = held(a.sd), XSd = held(a.xsd), Hb = held(a.h);
    const int tiles = H / (16 * kG), my_part = (int)blockIdx.x / tiles, tile = (int)blockIdx.x - my_part * tiles;
    const int n0 = tile * 16 * kG;
    // (entries past the count are loaded too, not to wait for it first; the head has room for all of them)
    static_assert(kFewThreads >= kFewList + 1 && kFewHead >= (kFewList + 2) * sizeof(int32_t), "one entry a thread");
    const uint32_t entry = (uint32_t)a.list[1 + min(tid, kFewList)];
    const int n_exp = uniform(a.list[0]);
    if (tid <= kFewList) list[tid] = entry;
    __syncthreads();
    const int kb_all = I / 128, st_e = (I + F::kSV - 1) / F::kSV;  // stages of an expert
    const int S = n_exp * st_e;
    const int share = my_part * kFewWaves + wave, shares = a.parts * kFewWaves;
    const int q0 = (int)((int64_t)S * share / shares), q1 = (int)((int64_t)S * (share + 1) / shares);
    const size_t row_bytes = F::row_bytes(I);
    const int lrow = lane >> 3, lchunk = lane & 7;
    uint8_t* lds = sW[wave];

    u32x4 bw[D][kG][2], hx[D][kHL];
    float sc[D];
    uint32_t mx[D];
    int iu = 0, is = 0;       // issue cursor: list index, stage of the expert
    gbytes wp{}, hp{}, sp{};  // the expert's weight rows and h rows (uniform), this lane's scales
    const uint32_t wofs = (uint32_t)lrow * (uint32_t)row_bytes + lchunk * 16;  // this lane's bytes of a stage
    uint32_t hofs[kHO];       // this lane's chunks of the stage's h rows: row 2 t is token t's hi row, 2 t + 1 lo
    auto hrow = [&](int j) { return kDirect ? 2 * (m & 7) + (m >> 3) : (j * kRows + lane / kRowLanes) & (2 * TT - 1); };
    uint8_t* hlds = sH[wave];
    auto expert_of = [&](int u) {
        const uint32_t entry = (uint32_t)uniform((int)list[u]);
        const int id = (int)(entry & 0xFFFF), mask = (int)(entry >> 16);
        const bool xg = id == kFewShared;
        const int e = xg ? 0 : id;
        wp = pick(xg, Xd, Wd) + ((size_t)e * H + n0) * row_bytes;
        hp = Hb + 2 * (size_t)u * 2 * T * a.pitch;
        // rows of tokens that are not routed here hold nothing: another's row is read, and its sums are not
        // taken
        const int any = __ffs(mask) - 1;
#pragma unroll
        for (int j = 0; j < kHO; ++j) {
            const int r = hrow(j), t = (mask >> (r >> 1)) & 1 ? r >> 1 : any;
            hofs[j] = 2 * (uint32_t)(t + (r & 1) * T) * (uint32_t)a.pitch + (kDirect ? 2 * F::value(0, kq) : 16 * (lane & (kRowLanes - 1)));
        }
        const gbytes s = pick(xg, XSd, Sd);
        if (kFmt == kFewFP8) sp = s + 4 * ((size_t)e * (H / 128) + n0 / 128) * kb_all;
        if (kFmt == kFewMX) sp = s + ((size_t)e * H + n0 + mx_row(lane, kG)) * (I / 32);
    };
    int left = 0;  // stages not yet issued
    auto issue = [&](auto tag) {
        constexpr int d = decltype(tag)::value;
        const int kb = 2 * is;  // MXFP4
        const uint32_t ofs = kFmt == kFewMX && kb + 1 >= kb_all && lchunk >= 4 ? wofs - 64 : wofs;
#pragma unroll
        for (int g = 0; g < kG; ++g)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                bw[d][g][i] = __builtin_nontemporal_load(
                    (gvec<u32x4>)(wp + ((size_t)(16 * g + 8 * i) * row_bytes + (size_t)is * 128) + ofs));
#pragma unroll
        for (int j = 0; j < kHL; ++j) hx[d][j] = *(gvec<u32x4>)(hp + (2 * is * F::kSV + (kDirect ? 2 * F::value(j, 0) : 0)) + hofs[kDirect ? 0 : j]);
        if (kFmt == kFewFP8) sc[d] = *(gvec<float>)(sp + 4 * is);
        if (kFmt == kFewMX) mx[d] = *(gvec<uint32_t>)(sp + 4 * min(kb + (lane & 1), kb_all - 1));
        if (--left > 0) {  // (past the wave's share its last stage is loaded again, into unused slots)
            if (++is == st_e) {
                is = 0;
                expert_of(++iu);
            }
        }
    };
    f32x4 acc[kG], pe[kG][2];  // sums of the experts done, and of the current one
#pragma unroll
    for (int g = 0; g < kG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};
    few_clear<kG>(pe);
    if (q0 < q1) {
        iu = q0 / st_e;
        is = q0 - iu * st_e;
        int cu = iu, cs = is;  // the stage being computed
        left = q1 - q0;
        expert_of(iu);
        // (in slot order, as the loop has them: the waits count on it)
        each_slot<D>([&](auto tag) {
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
        });
        auto compute = [&](auto tag) {
            constexpr int d = decltype(tag)::value;
            bf16x8 xv[F::kNM];
            if constexpr (kDirect) {
#pragma unroll
                for (int i = 0; i < F::kNM; ++i) xv[i] = as_bf16x8(hx[d][i]);
            } else {
#pragma unroll
                for (int j = 0; j < kHL; ++j) *(u32x4*)&hlds[hrow(j) * kHLD + 16 * (lane & (kRowLanes - 1))] = hx[d][j];
                __builtin_amdgcn_wave_barrier();
                const uint8_t* hm = hlds + (2 * min(m & 7, TT - 1) + (m >> 3)) * kHLD + 2 * F::value(0, kq);
#pragma unroll
                for (int i = 0; i < F::kNM; ++i) xv[i] = as_bf16x8(*(const u32x4*)&hm[2 * F::value(i, 0)]);
            }
            few_stage<kFmt, kG>(lds, bw[d], lane, kFmt == kFewMX ? mx[d] : 0u, kFmt == kFewFP8 ? sc[d] : 0.0f,
                                [&](int i) { return xv[i]; }, pe);
        };
        auto flush = [&]() {  // the expert's sums, for the tokens routed to it (a wave's share may
                              // begin or end inside an expert)
            const int mask = (int)((uint32_t)uniform((int)list[cu]) >> 16);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool mine = (mask >> ((4 * kq + r) & 7)) & 1;
#pragma unroll
                for (int g = 0; g < kG; ++g) acc[g][r] += mine ? pe[g][0][r] + pe[g][1][r] : 0.0f;
            }
            few_clear<kG>(pe);
        };
        ring_loop<D>(q1 - q0, [&](auto tag) {
            compute(tag);
            __builtin_amdgcn_sched_barrier(0);
            issue(tag);
            __builtin_amdgcn_sched_barrier(0);
            if (++cs == st_e) {
                flush();
                cs = 0;
                ++cu;
            }
        });
        if (cs != 0) flush();
    }
#pragma unroll
    for (int g = 0; g < kG; ++g) red[wave][g][lane] = acc[g];
    __syncthreads();
    // wave g joins group g, in wave order, and adds the lo rows to the hi rows: value r is column m of token
    // 4 kq + r (lanes 0..31)
    f32x4 v{};
    if (wave < kG) {
        v = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) v += red[w][wave][lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] += __shfl(v[r], lane | 32, kWave);
    }
    const bool mine = wave < kG && lane < 32;
    if (a.parts > 1) {
        // The tile's workgroups leave their sums in memory, past the XCDs' caches (agent scope); the one that
        // arrives last adds them all, in part order.  A sum is there before its arrival is counted: the
        // stores are waited for.
        const auto at = [&](int p, int r) {
            return a.part + ((((size_t)p * tiles + tile) * kG + wave) * kFewT + 4 * kq + r) * 16 + m;
        };
        if (mine) {
#pragma unroll
            for (int r = 0; r < 4; ++r) __hip_atomic_store(at(my_part, r), v[r], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0) before = __hip_atomic_fetch_add(&a.arrived[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (before != a.parts - 1 || !mine) return;
        f32x4 p[kFewParts];
#pragma unroll
        for (int i = 0; i < kFewParts; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                p[i][r] = i < a.parts ? __hip_atomic_load(at(i, r), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0f;
        v = p[0];
#pragma unroll
        for (int i = 1; i < kFewParts; ++i) v += p[i];
    }
    if (mine) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * kq + r;
            if (t < T) a.out[(size_t)t * H + n0 + 16 * wave + m] = f32_to_bf16(v[r]);
        }
    }
}

static moe_status check_few(int32_t T, int32_t k, const moe_expert_weights* w) {
    if (T < 0 || k < 1) return MOE_ERR_INVALID_ARG;
    const moe_status s = check_weights(w);
    if (s != MOE_OK) return s;
    if (k > w->n_groups) return MOE_ERR_INVALID_ARG;
    if (k > MOE_MAX_TOPK || T > MOE_FEW_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (T * (2 * w->H + 16) > kFewXBytes) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

static int few_pitch(int I) { return (I + 255) & ~255; }

// few_down's tiles and the workgroups that share one, by the time each choice would take: a round of the chip's
// CUs costs 4 us before its loads arrive, a workgroup streams at most the rate below (the chip 6.8 KB/ns), and
// a join costs 3 us.  Measured, us a layer (groups x parts; the rule's choice marked):
//   2048 x 1408, FP8, 8 tokens     1x1 84   2x1 98   2x2 78   2x4 69*  2x8 73
//   4096 x 1536, MXFP4, 8 tokens   1x1 112  2x1 123  2x2 102* 2x4 107  2x8 118
//   5120 x 1536, FP8, 8 tokens     1x1 237  2x1 212  2x2 221  2x3 202* 2x8 214
//   7168 x 2048, MXFP4, 1 token    1x1 50   2x1 46*  2x2 53   2x8 75
struct FewDown {
    int g, parts;
};
static FewDown few_down_plan(int64_t experts, int H, int fmt, double row_bytes) {
    static const double rate[3][2] = {{33, 42}, {24, 36}, {14, 21}};  // bytes/ns: bf16, FP8, MXFP4; one group, two
    FewDown best{1, 1};
    double best_ns = 1e30;
    for (int g : {1, 2})
        for (int parts = 1; parts <= (g == 2 ? kFewParts : 1); ++parts) {
            const int groups = H / (16 * g) * parts, rounds = (groups + 255) / 256;
            const double bytes = 16.0 * g * (double)experts * row_bytes / parts;  // of a workgroup
            const double ns = 4000.0 * rounds + std::max(rounds * bytes / rate[fmt][g - 1], groups * bytes / 6800.0) +
                              (parts > 1 ? 3000.0 : 0.0);
            if (ns < best_ns) best_ns = ns, best = {g, parts};
        }
    return best;
}

static int64_t few_experts(int T, int k, const moe_expert_weights* w) {  // the most there can be, and the shared one
    return std::min<int64_t>((int64_t)T * k, w->n_groups) + 1;
}

static FewDown few_down_of(int T, int k, const moe_expert_weights* w) {
    const int64_t experts = few_experts(T, k, w);
    switch (w->dtype) {
        case MOE_W_BF16: return few_down_plan(experts, w->H, kFewBF16, 2.0 * w->I);
        case MOE_W_FP8_E4M3_B128: return few_down_plan(experts, w->H, kFewFP8, w->I);
        default: return few_down_plan(experts, w->H, kFewMX, w->I * 17.0 / 32);
    }
}

static size_t few_h_bytes(int T, int k, const moe_expert_weights* w) {
    return few_experts(T, k, w) * 2 * T * (size_t)few_pitch(w->I) * sizeof(uint16_t);
}

static size_t few_ws(int T, int k, const moe_expert_weights* w) {
    if (T == 0) return 0;
    const int parts = few_down_of(T, k, w).parts;
    return kFewHead + few_h_bytes(T, k, w) + (parts > 1 ? (size_t)parts * kFewT * w->H * sizeof(float) : 0);
}

template <int kFmt>
static moe_status launch_few(const FewArgs& a, hipStream_t st) {
    // units of 16 columns where there are many of them, of 8 where whole rounds of the workgroups matter
    const int64_t experts = std::min(a.T * a.k, a.E) + 1;
    const bool wide = experts * a.I >= 16 * 4096;
    const int64_t units = experts * (a.I / (wide ? 16 : 8));
    const dim3 grid((unsigned)std::min<int64_t>(units, 256)), block(kFewThreads);
    if (wide) few_gate_up_kernel<kFmt, 2><<<grid, block, 0, st>>>(a);
    else few_gate_up_kernel<kFmt, 1><<<grid, block, 0, st>>>(a);
    const moe_status s = launch_status();
    if (s != MOE_OK) return s;
    auto down = [&](auto tag) {
        constexpr int TT = decltype(tag)::value;
        const dim3 grid((unsigned)(a.H / (16 * a.down_g) * a.parts));
        if (a.down_g == 2) few_down_kernel<kFmt, 2, TT><<<grid, block, 0, st>>>(a);
        else few_down_kernel<kFmt, 1, TT><<<grid, block, 0, st>>>(a);
    };
    if (a.T <= 2) down(std::integral_constant<int, 2>{});
    else if (a.T <= 4) down(std::integral_constant<int, 4>{});
    else down(std::integral_constant<int, 8>{});
    return launch_status();
}

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_layer_few_workspace_size(int32_t T, int32_t k, const moe_expert_weights* w,
                                                   size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status s = check_few(T, k, w);
    if (s != MOE_OK) return s;
    *bytes = few_ws(T, k, w);
    return MOE_OK;
}

extern "C" moe_status moe_layer_few(const float* scores, const uint16_t* x, int32_t T, int32_t k,
                                    int32_t score_fn, int32_t renorm, const moe_expert_weights* w,
                                    const moe_expert_weights* shared, int32_t* topk_ids, float* topk_w,
                                    uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
    if (score_fn != MOE_SCORE_SOFTMAX && score_fn != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    moe_status s = check_few(T, k, w);
    if (s != MOE_OK) return s;
    if (shared) {
        if ((s = check_weights(shared)) != MOE_OK) return s;
        if (shared->n_groups != 1 || shared->dtype != w->dtype || shared->H != w->H || shared->I != w->I)
            return MOE_ERR_INVALID_ARG;
    }
    if (T == 0) return MOE_OK;
    if (!scores || !x || !topk_ids || !topk_w || !out || !aligned16(scores) || !aligned16(x) ||
        !aligned16(topk_ids) || !aligned16(topk_w) || !aligned16(out))
        return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < few_ws(T, k, w)) return MOE_ERR_WORKSPACE;
    if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
    FewArgs a{};
    a.scores = scores;
    a.x = x;
    a.T = T, a.E = w->n_groups, a.k = k, a.H = w->H, a.I = w->I;
    a.score_fn = score_fn, a.renorm = renorm;
    a.g = w->w_gate, a.u = w->w_up, a.d = w->w_down;
    a.sg = w->s_gate, a.su = w->s_up, a.sd = w->s_down;
    if (shared) {
        a.xg = shared->w_gate, a.xu = shared->w_up, a.xd = shared->w_down;
        a.xsg = shared->s_gate, a.xsu = shared->s_up, a.xsd = shared->s_down;
    }
    a.ids = topk_ids;
    a.wts = topk_w;
    a.list = static_cast<int32_t*>(ws);
    a.h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(ws) + kFewHead);
    a.pitch = few_pitch(w->I);
    const FewDown down = few_down_of(T, k, w);
    a.down_g = down.g, a.parts = down.parts;
    a.arrived = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kFewCounts);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kFewHead + few_h_bytes(T, k, w));
    a.out = out;
    hipStream_t st = as_stream(stream);
    switch (w->dtype) {
        case MOE_W_BF16: return launch_few<kFewBF16>(a, st);
        case MOE_W_FP8_E4M3_B128: return launch_few<kFewFP8>(a, st);
        default: return launch_few<kFewMX>(a, st);
    }
}
