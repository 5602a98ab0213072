// Kernels of the fused INT8 W8A16 linear layer that the plain one has not:
//   out[t][r] = rnd(residual[t][r] + act(sum_k x[t][k] (q[r][k] - 128) s[r][k/G] + bias[r]))
//
//   * int8_short_fused_kernel: many tokens, K <= 320 (the hyper-connection up
//     projection);
//   * int8_ksplit_kernel: more than four tokens and few 32 x 32 output tiles
//     (the down projection): the waves of one workgroup split K and meet in
//     LDS, so no partial sum goes through memory;
//   * int8_gemv_wide_kernel: few tokens on wide matrices (lm_head): up to 16,
//     from 5 on, or from 3 on where N * K >= kInt8WideMinWeights.
//
// The first two use v_mfma_f32_32x32x16_f16 on exact fp16 codes and activations, a
// group's sum starting from zero and folded into the accumulator with the
// group's scale by one FMA, as int8_gemm_kernel does.  In the result a lane
// holds one column (weight row, lane % 32) of 16 tokens: rows
// 8 (j / 4) + 4 (lane / 32) + j % 4.
#include "int8.h"

namespace moe {

namespace {

struct FusedArgs {
    const uint16_t *x;        // bf16 [T][K], rows e.x_stride apart
    const int32_t *wq;        // [N][K/4]
    const uint16_t *ws;       // bf16 [N][K/G]
    int T, N, K, gshift;
    int mtiles, ntiles;
    int mstep;                // short K: workgroups per weight-row tile; wide GEMV: waves per row block
    float *part;              // fp32 [K splits][pstride], or null
    size_t pstride;
    Int8Epilogue e;
};

// ---------------------------------------------------------------------------
// Short K: a workgroup keeps 128 weight rows (32 per wave, all of K in
// registers) and takes one 64-token tile after the other; three workgroups to
// a CU cover each other's waits.  The residual is on its way while the sums
// pass through LDS, which they do so that a lane's accesses to residual
// and out are 8 or 16 bytes wide and a row's lanes consecutive: one or two
// elements per lane straight from the accumulators issue four to eight times
// the memory instructions (8192 tokens, N = 10240, K = 320, bf16 out and
// residual: 114 us against 142 and 173).  Columns that share no aligned word
// (odd N, odd strides) go element by element through the same LDS, a row's
// lanes consecutive: 188 us for 8192 x 10239 in fp32, 59 for 4919 x 3435 with
// GELU, where four columns per lane, an element at a time, took 411 and 91.
// What bounds it: with fp32 out and residual the memory (680 MB in 146 us, 94 %
// of a copy's rate); with bf16 the work per tile of three workgroups per CU (a
// fourth would need its registers spilled), two thirds of it vector
// instructions.
// ---------------------------------------------------------------------------
constexpr int kSpM = 64, kSpN = 128, kSpThreads = 256, kSpKS = 64;
constexpr int kSpCs = kSpN + 8;   // padded row of sums (fp32 words)

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// M rows of `cols` elements from token m on, as a buffer: accesses beyond the
// last token, and those of columns past N (placed beyond any buffer by
// lane_offset), read zero and store nothing.
template <int M>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const void *base, size_t stride, int bytes, int m, int T,
                                                              int cols)
{
    const int rows = min(M, T - m);
    const char *p = static_cast<const char *>(base) + (size_t)m * stride * bytes;
    const uint32_t size = rows > 0 ? (uint32_t)(((size_t)(rows - 1) * stride + cols) * bytes) : 0u;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), (short)0, (int)size, kBufferWord3);
}

// NS: K / 64; GS: stages per scale group; RES: bytes of a residual element (0:
// none); VEC: four columns lie on an aligned word in residual and out.
template <int NS, int GS, int RES, bool VEC>
__global__ __launch_bounds__(kSpThreads, 3) void int8_short_fused_kernel(FusedArgs g)
{
    constexpr int LR = NS * kSpKS + 8;    // padded activation row (fp16)
    constexpr int CH = NS * 8;            // 16-byte chunks per activation row
    constexpr int XPER = kSpM * CH / kSpThreads;
    constexpr int NG = NS / GS;           // scale groups
    constexpr int SPER = (NG * kSpN + kSpThreads - 1) / kSpThreads;
    static_assert(NS % GS == 0 && kSpM * CH % kSpThreads == 0, "whole groups, whole passes");
    // the activation tile, then the tile's sums
    constexpr int kBytes = kSpM * LR * 2 > kSpM * kSpCs * 4 ? kSpM * LR * 2 : kSpM * kSpCs * 4;
    __shared__ __align__(16) unsigned char s_raw[kBytes];
    _Float16 *s_x = reinterpret_cast<_Float16 *>(s_raw);
    float *s_c = reinterpret_cast<float *>(s_raw);
    __shared__ uint16_t s_sc[NG * kSpN];   // [group][row]

    // ---- work: each XCD takes a contiguous range of workgroups, those of
    // one token tile back to back; the workgroup's token tiles are g.mstep
    // apart ----
    const int per = gridDim.x >> 3;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= g.mstep * g.ntiles) return;
    const int n0 = tile % g.ntiles * kSpN;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, half = lane >> 5;
    const int n = n0 + 32 * wave + (lane & 31);

    u32x4_t rx[XPER];
    auto load_x = [&](int m0) {
        const __amdgpu_buffer_rsrc_t xs = rows_buffer<kSpM>(g.x, g.e.x_stride, 2, m0, g.T, g.K);
#pragma unroll
        for (int u = 0; u < XPER; ++u) {
            const uint32_t c = tid + kSpThreads * u;
            rx[u] = __builtin_amdgcn_raw_buffer_load_b128(xs, (int)(c / CH * (uint32_t)(2 * g.e.x_stride) + c % CH * 16), 0, 0);
        }
    };
    const u32x4_t *bsrc = reinterpret_cast<const u32x4_t *>(g.wq + (size_t)min(n, g.N - 1) * (g.K / 4)) + 2 * half;
    u32x4_t rb[NS][2];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        rb[s][0] = bsrc[4 * s];
        rb[s][1] = bsrc[4 * s + 1];
    }
#pragma unroll
    for (int u = 0; u < SPER; ++u) {   // a row's scales are consecutive
        const int i = tid + kSpThreads * u;
        if (i < NG * kSpN) s_sc[i % NG * kSpN + i / NG] = g.ws[(size_t)min(n0 + i / NG, g.N - 1) * NG + i % NG];
    }
    // epilogue: this thread's four columns of rows tid / 32 + 8 u
    const int r0 = tid >> 5, c4 = 4 * (tid & 31), nn = n0 + c4;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g.e.bias) {
        if constexpr (VEC)
            bias = load_typed4(g.e.bias, g.e.bias_type, min(nn, g.N - 4));
        else
            bias = make_float4(load_typed(g.e.bias, g.e.bias_type, min(nn, g.N - 1)),
                               load_typed(g.e.bias, g.e.bias_type, min(nn + 1, g.N - 1)),
                               load_typed(g.e.bias, g.e.bias_type, min(nn + 2, g.N - 1)),
                               load_typed(g.e.bias, g.e.bias_type, min(nn + 3, g.N - 1)));
    }
    // at residual and out these columns, or, element by element, column
    // tid % 128 of rows tid / 128 + 2 u
    constexpr int kRowStep = VEC ? 8 : 2;
    const int rr = VEC ? r0 : tid >> 7, rc = VEC ? c4 : tid & 127;
    auto lane_offset = [&](size_t stride, int bytes) {
        return n0 + rc < g.N ? ((uint32_t)rr * (uint32_t)stride + (uint32_t)(n0 + rc)) * (uint32_t)bytes : 0x80000000u;
    };
    // the bias where no activation has taken it in
    const float4 late = g.e.activation == kActNone ? bias : make_float4(0.f, 0.f, 0.f, 0.f);
    const int ob = type_bytes(g.e.out_type);
    const uint32_t roff = lane_offset(g.e.residual_stride, RES), rstep = kRowStep * (uint32_t)g.e.residual_stride * RES;
    const uint32_t ooff = lane_offset(g.e.out_stride, ob), ostep = kRowStep * (uint32_t)g.e.out_stride * ob;

    for (int mi = tile / g.ntiles; mi < g.mtiles; mi += g.mstep) {
    const int m0 = mi * kSpM, rows = min(kSpM, g.T - m0);
    load_x(m0);
    if (mi >= g.mstep) __syncthreads();   // the tile before has been read
#pragma unroll
    for (int u = 0; u < XPER; ++u) {
        const int c = tid + kSpThreads * u;
        *reinterpret_cast<u32x4_t *>(s_x + (c / CH) * LR + 8 * (c % CH)) = bf16x8_to_f16x8(rx[u]);
    }
    // the codes are unpacked anew for every tile: kept as fp16, they would
    // take twice the registers
#pragma unroll
    for (int s = 0; s < NS; ++s) asm volatile("" : "+v"(rb[s][0]), "+v"(rb[s][1]));
    __syncthreads();

    f32x16_t acc[2];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[mt][q] = 0.f;
    f32x16_t tmp[2];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        const bool gfirst = s % GS == 0, glast = s % GS == GS - 1;
        const u32x4_t w0 = rb[s][0], w1 = rb[s][1];
        const _Float16 *A = s_x + (lane & 31) * LR + kSpKS * s + 32 * half;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t wa = j < 2 ? w0[2 * j] : w1[2 * j - 4];
            const uint32_t wb = j < 2 ? w0[2 * j + 1] : w1[2 * j - 3];
            const h2_t p0 = code_pair<0>(wa), p1 = code_pair<1>(wa);
            const h2_t p2 = code_pair<0>(wb), p3 = code_pair<1>(wb);
            const f16x8_t bf = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                const f16x8_t af = *reinterpret_cast<const f16x8_t *>(A + 32 * mt * LR + 8 * j);
                const f32x16_t z = {};
                tmp[mt] = __builtin_amdgcn_mfma_f32_32x32x16_f16(af, bf, gfirst && j == 0 ? z : tmp[mt], 0, 0, 0);
            }
        }
        if (glast) {
            const float sf = bf16_to_f32(s_sc[(s / GS) * kSpN + 32 * wave + (lane & 31)]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[mt][v] = fmaf(sf, tmp[mt][v], acc[mt][v]);
        }
        // the fold happens here: sunk into the epilogue's branch, it would keep
        // every stage's sums in registers
        asm volatile("" : "+v"(acc[0]), "+v"(acc[1]));
    }

    // ---- epilogue ----
    constexpr int kPer = 32 / kRowStep;   // accesses per thread to 32 rows
    u32x4_t res[VEC ? 2 * kPer : 1];
    uint32_t res1[VEC ? 1 : 2 * kPer];
    auto load_residual = [&](int h) {
        const __amdgpu_buffer_rsrc_t rs = rows_buffer<32>(g.e.residual, g.e.residual_stride, RES, m0 + 32 * h, g.T, g.N);
        uint32_t off = roff;
        if constexpr (!VEC) asm volatile("" : "+v"(off));   // 16 offsets made here, not kept over the tiles
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int at = (int)(off + u * rstep);
            if constexpr (!VEC) {
                if constexpr (RES == 4) res1[kPer * h + u] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
                else res1[kPer * h + u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
            } else if constexpr (RES == 4) {
                res[kPer * h + u] = __builtin_amdgcn_raw_buffer_load_b128(rs, at, 0, 0);
            } else {
                const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(rs, at, 0, 0);
                res[kPer * h + u][0] = w[0];
                res[kPer * h + u][1] = w[1];
            }
        }
    };
    if constexpr (RES > 0) {
        load_residual(0);
        if constexpr (VEC) load_residual(1);
    }
    __syncthreads();   // the activations have been read
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            s_c[(32 * mt + 8 * (j >> 2) + 4 * half + (j & 3)) * kSpCs + 32 * wave + (lane & 31)] = acc[mt][j];
    __syncthreads();
    if constexpr (RES > 0 && !VEC) load_residual(1);   // the accumulators' registers are free
    // an activation in place (this thread's own words), in a loop of its own:
    // unrolled with the stores it was 25 KB of code, fetched at every launch
    if (g.e.activation != kActNone || (!VEC && g.e.bias)) {
#pragma unroll 1
        for (int u = 0; u < kSpM / 8; ++u) {
            float4 *w = reinterpret_cast<float4 *>(s_c + (8 * u + r0) * kSpCs + c4);
            const float4 f = *w;
            *w = make_float4(activate(f.x + bias.x, g.e.activation), activate(f.y + bias.y, g.e.activation),
                             activate(f.z + bias.z, g.e.activation), activate(f.w + bias.w, g.e.activation));
        }
    }
    if constexpr (!VEC) __syncthreads();   // the words of other threads
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (32 * h >= rows) break;
        const __amdgpu_buffer_rsrc_t rs = rows_buffer<32>(g.e.out, g.e.out_stride, ob, m0 + 32 * h, g.T, g.N);
        uint32_t off = ooff;
        if constexpr (!VEC) asm volatile("" : "+v"(off));
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int at = (int)(off + u * ostep);
            if constexpr (!VEC) {
                float v = s_c[(32 * h + kRowStep * u + rr) * kSpCs + rc];
                if constexpr (RES > 0) {
                    const uint32_t w = res1[kPer * h + u];
                    v += RES == 4                       ? __uint_as_float(w)
                         : g.e.residual_type == kBf16 ? bf16_lo(w)
                                                        : (float)__builtin_bit_cast(f16x2_t, w)[0];
                }
                if (g.e.out_type == kF32)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rs, at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b16(
                        g.e.out_type == kBf16 ? (uint16_t)f32_to_bf16(v) : __builtin_bit_cast(uint16_t, (_Float16)v), rs, at, 0, 0);
                continue;
            }
            const float4 f = *reinterpret_cast<const float4 *>(s_c + (32 * h + 8 * u + r0) * kSpCs + c4);
            float v[4] = {f.x + late.x, f.y + late.y, f.z + late.z, f.w + late.w};
            const u32x4_t w = res[VEC ? kPer * h + u : 0];
            if constexpr (RES == 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t e = w[q];
                    v[q] += __uint_as_float(e);
                }
            } else if constexpr (RES == 2) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t e = w[q];
                    const f16x2_t hh = __builtin_bit_cast(f16x2_t, e);
                    const bool bf = g.e.residual_type == kBf16;
                    v[2 * q] += bf ? bf16_lo(e) : (float)hh[0];
                    v[2 * q + 1] += bf ? bf16_hi(e) : (float)hh[1];
                }
            }
            if (g.e.out_type == kF32) {
                const u32x4_t o = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
                __builtin_amdgcn_raw_buffer_store_b128(o, rs, at, 0, 0);
            } else {
                const f16x2_t lo = {(_Float16)v[0], (_Float16)v[1]}, hi = {(_Float16)v[2], (_Float16)v[3]};
                const bool bf = g.e.out_type == kBf16;
                const u32x2_t o = {bf ? f32x2_to_bf16x2(v[0], v[1]) : __builtin_bit_cast(uint32_t, lo),
                                   bf ? f32x2_to_bf16x2(v[2], v[3]) : __builtin_bit_cast(uint32_t, hi)};
                __builtin_amdgcn_raw_buffer_store_b64(o, rs, at, 0, 0);
            }
        }
    }
    }
}

// ---------------------------------------------------------------------------
// K across the waves: a workgroup owns one output tile of 32 tokens x 32
// weight rows, and each of its (up to 16) waves a run of whole scale groups of
// K, which it stages through LDS of its own without a barrier, the loads two
// stages ahead.  The waves' sums meet in LDS and are added in wave order, so
// no partial sum goes through memory, unless K is split over workgroups too
// (gridDim.y) because the tiles alone would leave CUs idle.
//
// What bounds it: no one unit.  [320, 10240] at 512 tokens takes 19 us (3.4
// GFLOP) in 160 workgroups, each alone on its CU (the LDS is reserved for 16
// waves, 128 KB, however many there are), so 96 CUs idle.  On the others the
// vector ALU issues half of the time (32 instructions to an MFMA: a stage
// converts 32 x 64 activations, which the ten weight-row tiles of a mixer
// repeat, and folds 16 sums), the matrix cores work an eighth of it, and a wave
// waits for data or a barrier two fifths of it.  Tiles of 64 x 64, which halve
// the conversions, leave 40 workgroups, and with K over six workgroups each
// take as long.
// ---------------------------------------------------------------------------
constexpr int kKwWaves = 16;
constexpr int kKwTile = 32;
constexpr int kKwXPitch = 72;   // fp16 per staged activation row: 16-byte reads of 8 rows fall in different banks
constexpr int kKwWPitch = 80;   // bytes per staged weight row, likewise

template <int GS>
__global__ __launch_bounds__(64 * kKwWaves) void int8_ksplit_kernel(FusedArgs g)
{
    constexpr int kPitch = kKwTile + 8;   // fp32 words per row of sums: the half-waves' rows, 4 apart, in different banks
    constexpr int kWaveLds = kKwTile * (kKwXPitch * 2 + kKwWPitch);
    static_assert(kWaveLds >= kKwTile * kPitch * 4, "a wave's sums fit its staging area");
    constexpr int kScGroups = 16;
    __shared__ __align__(16) unsigned char s_raw[kKwWaves][kWaveLds];
    __shared__ uint16_t s_scale[kKwWaves][kScGroups * kKwTile];
    const int per = gridDim.x >> 3;
    const int tile = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (tile >= g.mtiles * g.ntiles) return;
    const int m0 = tile / g.ntiles * kKwTile, n0 = tile % g.ntiles * kKwTile;
    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int waves = blockDim.x >> 6, groups = g.K >> g.gshift;
    // this wave's groups; at least one (the launch sees to it)
    const int parts = waves * gridDim.y, part = blockIdx.y * waves + wave;
    const int g0 = (int)((long)part * groups / parts), g1 = (int)((long)(part + 1) * groups / parts);
    const int s1 = (g1 - g0) * GS;   // stages of 64 inputs

    // loads: eight lanes on the 128 bytes of a token, four on the 64 of a
    // weight row; rows past the last repeat it and are never stored.  (The
    // tile's rows from a uniform base: 32-bit offsets are enough, 31 rows of
    // at most 2^24 elements, and take half the registers.)
    const char *xb = reinterpret_cast<const char *>(g.x + m0 * g.e.x_stride + (size_t)g0 * GS * 64);
    const char *wb = reinterpret_cast<const char *>(g.wq) + (size_t)n0 * g.K + (size_t)g0 * GS * 64;
    const uint16_t *sb = g.ws + (size_t)n0 * groups + g0;
    uint32_t xo[4], wo[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        xo[i] = min(8 * i + (lane >> 3), g.T - 1 - m0) * (uint32_t)(2 * g.e.x_stride) + 16 * (lane & 7);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        wo[i] = min(16 * i + (lane >> 2), g.N - 1 - n0) * (uint32_t)g.K + 16 * (lane & 3);
    // scales: kScGroups groups of every row at a time, 16 lanes on those of one
    // row (a load of one scale per row would cost as many cache accesses as
    // the row's 64 codes)
    uint16_t *s_sc = s_scale[wave];   // [group][row]
    uint32_t sv[kScGroups * kKwTile / 64];
    auto load_scales = [&](int grp) {
#pragma unroll
        for (int i = 0; i < kScGroups * kKwTile / 64; ++i)
            sv[i] = sb[min(4 * i + (lane >> 4), g.N - 1 - n0) * (uint32_t)groups + min(grp + (lane & 15), g1 - g0 - 1)];
    };
    auto store_scales = [&]() {
#pragma unroll
        for (int i = 0; i < kScGroups * kKwTile / 64; ++i) s_sc[(lane & 15) * kKwTile + 4 * i + (lane >> 4)] = (uint16_t)sv[i];
    };
    _Float16 *s_x = reinterpret_cast<_Float16 *>(s_raw[wave]);
    unsigned char *s_w = s_raw[wave] + kKwTile * kKwXPitch * 2;

    struct Stage {
        u32x4_t x[4], w[2];
    };
    auto load = [&](int s, Stage &r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.x[i] = *reinterpret_cast<const u32x4_t *>(xb + (xo[i] + 128u * s));
#pragma unroll
        for (int i = 0; i < 2; ++i) r.w[i] = *reinterpret_cast<const u32x4_t *>(wb + (wo[i] + 64u * s));
    };
    f32x16_t acc, tmp;
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[q] = 0.f;
    // stage s, whose data r holds: through LDS into MFMA order (the area is
    // this wave's own, and its LDS operations run in order), with the loads
    // of stage s + 2 issued in between
    auto stage = [&](int s, Stage &r, bool gfirst, bool glast) {
        if (s > 0 && s % (kScGroups * GS) == 0) {   // the next groups' scales
            load_scales(s / GS);
            store_scales();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<u32x4_t *>(s_x + (8 * i + (lane >> 3)) * kKwXPitch + 8 * (lane & 7)) = bf16x8_to_f16x8(r.x[i]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<u32x4_t *>(s_w + (16 * i + (lane >> 2)) * kKwWPitch + 16 * (lane & 3)) = r.w[i];
        load(min(s + 2, s1 - 1), r);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        u32x4_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = *reinterpret_cast<const u32x4_t *>(s_w + (lane & 31) * kKwWPitch + 32 * half + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t wa = w[j >> 1][2 * (j & 1)], wb = w[j >> 1][2 * (j & 1) + 1];
            const h2_t p0 = code_pair<0>(wa), p1 = code_pair<1>(wa);
            const h2_t p2 = code_pair<0>(wb), p3 = code_pair<1>(wb);
            const f16x8_t bf = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
            const f16x8_t af = *reinterpret_cast<const f16x8_t *>(s_x + (lane & 31) * kKwXPitch + 32 * half + 8 * j);
            const f32x16_t z = {};
            tmp = __builtin_amdgcn_mfma_f32_32x32x16_f16(af, bf, gfirst && j == 0 ? z : tmp, 0, 0, 0);
        }
        if (glast) {
            const float sf = bf16_to_f32(s_sc[s / GS % kScGroups * kKwTile + (lane & 31)]);
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[v] = fmaf(sf, tmp[v], acc[v]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // nothing of the next stage before here: its data would be waited for
        __builtin_amdgcn_sched_barrier(0);
    };
    Stage r0, r1;
    load_scales(0);
    load(0, r0);
    load(min(1, s1 - 1), r1);
    store_scales();
    int s = 0;
    for (; s + 1 < s1; s += 2) {   // s is even: with two stages per group the first and the last of one
        stage(s, r0, true, GS == 1);
        stage(s + 1, r1, GS == 1, true);
    }
    if (s < s1) stage(s, r0, true, true);   // one stage per group

    float *sums = reinterpret_cast<float *>(s_raw[wave]);
#pragma unroll
    for (int j = 0; j < 16; ++j) sums[(8 * (j >> 2) + 4 * half + (j & 3)) * kPitch + (lane & 31)] = acc[j];
    __syncthreads();
    for (int i = tid; i < kKwTile * kKwTile; i += blockDim.x) {
        const int r = i / kKwTile, c = i % kKwTile, t = m0 + r, n = n0 + c;
        float v = 0.f;
        for (int w = 0; w < waves; ++w) v += reinterpret_cast<const float *>(s_raw[w])[r * kPitch + c];
        if (t >= g.T || n >= g.N) continue;
        if (gridDim.y > 1) g.part[blockIdx.y * g.pstride + (size_t)t * g.N + n] = v;
        else finish(g.e, t, n, v);
    }
}

// ---------------------------------------------------------------------------
// Few tokens on wide matrices (lm_head): one read of the weights at the
// memory's rate.  A wave owns 16 weight rows at a time.  Per step of 128 inputs
// eight lanes load the 128 consecutive bytes of a row, and the 16 x 128 block
// passes through LDS of the wave's own into the B operand of
// v_mfma_f32_16x16x32_f16 (column = weight row, lane % 16; the A operand is
// the activations, fp16 in LDS, row = token).  kGwAhead steps are on their
// way, across row blocks.  Rows past T repeat the last token and are never
// stored.
//
// What bounds it: memory, 248320 x 2560 at 8 tokens in 114 us (5.7 TB/s of
// 654 MB); loads that put 16 rows of 64 bytes into one instruction reach 4.2.
// Six steps ahead need more registers than two workgroups per CU have: 113 us
// with one of them, and 20 us instead of 14 for 10240 x 2560.
// ---------------------------------------------------------------------------
constexpr int kGwWaves = 8, kGwThreads = 64 * kGwWaves;
constexpr int kGwRows = 16;
constexpr int kGwStep = kInt8WideStep;
constexpr int kGwAhead = kInt8WideAhead;
constexpr int kGwPitch = kGwStep + 16;   // bytes per staged row
constexpr int kGwScGroups = 16;          // scale groups staged at a time

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2w_t __attribute__((ext_vector_type(2)));

template <int G>
__global__ __launch_bounds__(kGwThreads, 4) void int8_gemv_wide_kernel(FusedArgs g)
{
    constexpr int GPS = kGwStep / G;   // scale groups per step
    __shared__ __align__(16) unsigned char s_w[kGwWaves][kGwRows * kGwPitch];
    __shared__ uint16_t s_scale[kGwWaves][kGwScGroups * kGwRows];
    extern __shared__ u32x4_t s_xv[];   // [T][K / 8 + 1]: one unit of padding per row
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // ks waves share a row block, each with a range of its steps (more than
    // one: every wave has at most one block)
    const int ks = g.mstep, part = wave % ks;
    const int first = (blockIdx.x * kGwWaves + wave) / ks, waves = gridDim.x * kGwWaves / ks;
    const int nrb = (g.N + kGwRows - 1) / kGwRows, groups = g.K / G;
    const int s0 = part * (g.K / kGwStep) / ks, steps = (part + 1) * (g.K / kGwStep) / ks - s0;
    const int blocks = first < nrb ? (nrb - first + waves - 1) / waves : 0;
    const int U = blocks * steps;

    // load cursor: step s0 + lst of row block lb; past the last unit it stays
    int lb = 0, lst = 0;
    const char *wb = nullptr;
    uint32_t wo[2];
    auto aim = [&]() {
        const int row0 = (first + lb * waves) * kGwRows;
        wb = reinterpret_cast<const char *>(g.wq) + (size_t)row0 * g.K + (size_t)s0 * kGwStep;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            wo[i] = min(8 * i + (lane >> 3), g.N - 1 - row0) * (uint32_t)g.K + 16 * (lane & 7);
    };
    struct Raw {
        u32x4_t w[2];
    };
    auto load_next = [&](Raw &r) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(wb + (wo[i] + (uint32_t)(kGwStep * lst))));
        if (lst + 1 < steps) {
            ++lst;
        } else if (lb + 1 < blocks) {
            lst = 0;
            ++lb;
            aim();
        }
    };
    // scales of the groups from s0 GPS + grp on of block b, 16 lanes on those of a row
    uint32_t sv[4];
    auto load_scales = [&](int b, int grp) {
        const int row0 = (first + b * waves) * kGwRows;
        const uint16_t *sb = g.ws + (size_t)row0 * groups;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sv[i] = sb[min(4 * i + (lane >> 4), g.N - 1 - row0) * (uint32_t)groups +
                       min(s0 * GPS + grp + (lane & 15), groups - 1)];
    };
    Raw raw[kGwAhead];
    if (U > 0) {
        aim();
        load_scales(0, 0);
#pragma unroll
        for (int q = 0; q < kGwAhead; ++q) load_next(raw[q]);
    }
    const int K8 = g.K >> 3, xs = K8 + 1;
    for (int i = tid; i < g.T * K8; i += kGwThreads) {
        const int t = i / K8, c = i - t * K8;
        s_xv[t * xs + c] = bf16x8_to_f16x8(*reinterpret_cast<const u32x4_t *>(g.x + t * g.e.x_stride + 8 * c));
    }
    __syncthreads();

    const int n = lane & 15, kq = lane >> 4;
    const u32x4_t *xrow = s_xv + min(n, g.T - 1) * xs + kq + s0 * (kGwStep / 8);
    uint16_t *s_sc = s_scale[wave];   // [group][row]
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    int cb = 0, cst = 0;
    // a finished block's sums and its number, until the epilogue comes round
    // (one copy of it, between runs of kGwAhead steps: no two blocks end in one)
    f32x4_t done = acc;
    int db = -1;
    auto compute = [&](Raw &r) {
        const int grp = cst * GPS;
        if (grp % kGwScGroups == 0) {   // this chunk of scales to LDS, the next on its way
#pragma unroll
            for (int i = 0; i < 4; ++i) s_sc[(lane & 15) * kGwRows + 4 * i + (lane >> 4)] = (uint16_t)sv[i];
            const bool more = grp + kGwScGroups < steps * GPS;
            load_scales(more ? cb : min(cb + 1, blocks - 1), more ? grp + kGwScGroups : 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<u32x4_t *>(s_w[wave] + (8 * i + (lane >> 3)) * kGwPitch + 16 * (lane & 7)) = r.w[i];
        load_next(r);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        f32x4_t tmp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const u32x2w_t w = *reinterpret_cast<const u32x2w_t *>(s_w[wave] + n * kGwPitch + 32 * m + 8 * kq);
            const uint32_t wa = w[0], wc = w[1];
            const h2_t p0 = code_pair<0>(wa), p1 = code_pair<1>(wa);
            const h2_t p2 = code_pair<0>(wc), p3 = code_pair<1>(wc);
            const f16x8_t bf = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
            const u32x4_t xv = xrow[cst * (kGwStep / 8) + 4 * m];
            tmp = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, xv), bf, tmp, 0, 0, 0);
            if (GPS == 1 ? m == 3 : m & 1) {
                const float sf = bf16_to_f32(s_sc[(grp + (GPS == 2 ? m >> 1 : 0)) % kGwScGroups * kGwRows + n]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j] = fmaf(sf, tmp[j], acc[j]);
                    tmp[j] = 0.f;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (++cst == steps) {
            done = acc;
            db = cb;
            acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
            cst = 0;
            ++cb;
        }
        __builtin_amdgcn_sched_barrier(0);   // nothing of the next step: its data would be waited for
    };
    auto store = [&]() {   // the lane holds tokens 4 kq + j of row n
        int nn = n, t0 = 4 * kq;
        asm volatile("" : "+v"(nn), "+v"(t0));   // the addresses are made here, not kept in registers all along
        const int row = (first + db * waves) * kGwRows + nn;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t0 + j < g.T && row < g.N) finish(g.e, t0 + j, row, done[j]);
        db = -1;
    };
    for (int u = 0; u < U; u += kGwAhead) {
        if (u + kGwAhead <= U) {
#pragma unroll
            for (int q = 0; q < kGwAhead; ++q) compute(raw[q]);
        } else {
#pragma unroll
            for (int q = 0; q < kGwAhead; ++q)
                if (u + q < U) compute(raw[q]);
        }
        if (ks == 1 && db >= 0) store();
    }
    if (ks > 1) {   // the waves' sums, in wave order
        float *sums = reinterpret_cast<float *>(s_w[wave]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[4 * lane + j] = done[j];
        __syncthreads();
        if (part == 0 && blocks > 0) {
            for (int w = 1; w < ks; ++w)
#pragma unroll
                for (int j = 0; j < 4; ++j) done[j] += reinterpret_cast<const float *>(s_w[wave + w])[4 * lane + j];
            store();
        }
    }
}

template <int RES, bool VEC>
void launch_short(const FusedArgs &a, int grid, hipStream_t st)
{
    const int ns = a.K / kSpKS;
    if (a.gshift == 6) {
        switch (ns) {
        case 1: int8_short_fused_kernel<1, 1, RES, VEC><<<grid, kSpThreads, 0, st>>>(a); break;
        case 2: int8_short_fused_kernel<2, 1, RES, VEC><<<grid, kSpThreads, 0, st>>>(a); break;
        case 3: int8_short_fused_kernel<3, 1, RES, VEC><<<grid, kSpThreads, 0, st>>>(a); break;
        case 4: int8_short_fused_kernel<4, 1, RES, VEC><<<grid, kSpThreads, 0, st>>>(a); break;
        default: int8_short_fused_kernel<5, 1, RES, VEC><<<grid, kSpThreads, 0, st>>>(a); break;
        }
    } else {
        if (ns == 2) int8_short_fused_kernel<2, 2, RES, VEC><<<grid, kSpThreads, 0, st>>>(a);
        else int8_short_fused_kernel<4, 2, RES, VEC><<<grid, kSpThreads, 0, st>>>(a);
    }
}

FusedArgs fused_args(const uint16_t *x, const int32_t *wq, const uint16_t *ws, int T, int N, int K, int G,
                     const Int8Epilogue &e, int tm, int tn)
{
    return FusedArgs{x, wq, ws, T, N, K, G == 64 ? 6 : 7, (T + tm - 1) / tm, (N + tn - 1) / tn, 0, nullptr, 0, e};
}

}  // namespace

hipError_t launch_int8_short_fused(const uint16_t *x, const int32_t *wq, const uint16_t *ws, int T, int N, int K,
                                  int G, const Int8Epilogue &e, hipStream_t st)
{
    FusedArgs a = fused_args(x, wq, ws, T, N, K, G, e, kSpM, kSpN);
    // three workgroups to a CU; as many per weight-row tile as give each of
    // them the same number of token tiles
    constexpr int kSlots = 768;
    const int most = kSlots / a.ntiles > 0 ? kSlots / a.ntiles : 1, turns = (a.mtiles + most - 1) / most;
    a.mstep = (a.mtiles + turns - 1) / turns;
    const int grid = (a.mstep * a.ntiles + 7) / 8 * 8;
    const int res = !e.residual ? 0 : type_bytes(e.residual_type);
    if (res == 0) e.vec ? launch_short<0, true>(a, grid, st) : launch_short<0, false>(a, grid, st);
    else if (res == 4) e.vec ? launch_short<4, true>(a, grid, st) : launch_short<4, false>(a, grid, st);
    else e.vec ? launch_short<2, true>(a, grid, st) : launch_short<2, false>(a, grid, st);
    return hipGetLastError();
}

size_t int8_gemv_wide_lds(int T, int K) { return (size_t)T * (K / 8 + 1) * 16; }

hipError_t launch_int8_gemv_wide(const uint16_t *x, const int32_t *wq, const uint16_t *ws, int T, int N, int K, int G,
                                 const Int8Epilogue &e, hipStream_t st)
{
    FusedArgs a = fused_args(x, wq, ws, T, N, K, G, e, 16, kGwRows);
    // two workgroups to a CU (one where the activations take most of its LDS),
    // with the same number of row blocks per wave; fewer blocks than waves are
    // shared out
    const size_t lds = int8_gemv_wide_lds(T, K);
    const int most = (lds <= 57344 ? 2 : 1) * 256 * kGwWaves, turns = (a.ntiles + most - 1) / most;
    a.mstep = 1;
    while (turns == 1 && 2 * a.mstep <= kGwWaves && 2 * a.mstep * a.ntiles <= most && 2 * a.mstep * kGwStep <= K)
        a.mstep *= 2;
    const int grid = (a.ntiles * a.mstep + turns * kGwWaves - 1) / (turns * kGwWaves);
    if (lds > 65536) {
        const void *f = G == 64 ? reinterpret_cast<const void *>(int8_gemv_wide_kernel<64>)
                                : reinterpret_cast<const void *>(int8_gemv_wide_kernel<128>);
        const hipError_t rc = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (rc != hipSuccess) return rc;
    }
    if (G == 64) int8_gemv_wide_kernel<64><<<grid, kGwThreads, lds, st>>>(a);
    else int8_gemv_wide_kernel<128><<<grid, kGwThreads, lds, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_int8_ksplit(const uint16_t *x, const int32_t *wq, const uint16_t *ws, int T, int N, int K, int G,
                              const Int8Epilogue &e, int ksplit, float *part, size_t pstride, hipStream_t st)
{
    FusedArgs a = fused_args(x, wq, ws, T, N, K, G, e, kKwTile, kKwTile);
    a.part = part;
    a.pstride = pstride;
    const dim3 grid((unsigned)((a.mtiles * a.ntiles + 7) / 8 * 8), (unsigned)ksplit);
    const int groups = K / G / ksplit, waves = groups < kKwWaves ? groups : kKwWaves;
    if (G == 64) int8_ksplit_kernel<1><<<grid, 64 * waves, 0, st>>>(a);
    else int8_ksplit_kernel<2><<<grid, 64 * waves, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
