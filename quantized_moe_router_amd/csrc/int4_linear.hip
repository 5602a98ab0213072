// INT4 W4A16 linear layer and the products grouped by expert:
//   out[o] = residual[o] + row_weights[o] act(x[i] W_e^T + bias[e])
//
// Codes become bf16 by placing a nibble n = code + 8 in the mantissa of 16.0:
// 0x4180 | n << 3 is 16 + n = code + 24 exactly, so a word takes four shifts
// and four AND-ORs for its eight codes.  The 24 too much is taken off by the
// matrix cores: the accumulators of a group begin at the product of x with a
// matrix of -24 (one such product serves every column tile of the wave), and
// what the group's products leave there is sum x code, exact up to fp32's
// additions.  The group's scale multiplies that sum in fp32, so neither x nor
// a weight is ever rounded.
//
// A word's pairs are its codes (0,4)(1,5)(2,6)(3,7); x is put in that order.
#include "int8.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Word -> MFMA operand: eight bf16 values code + 24 in pair order.
__device__ __forceinline__ bf16x8_t codes24(uint32_t w)
{
    const uint32_t m = vconst(0x00780078u), b = vconst(0x41804180u);
    u32x4_t p;
    p[0] = ((w << 3) & m) | b;
    p[1] = ((w >> 1) & m) | b;
    p[2] = ((w >> 5) & m) | b;
    p[3] = ((w >> 9) & m) | b;
    return __builtin_bit_cast(bf16x8_t, p);
}

__device__ __forceinline__ bf16x8_t minus24()
{
    const uint32_t c = 0xC1C0C1C0u;
    const u32x4_t p = {c, c, c, c};
    return __builtin_bit_cast(bf16x8_t, p);
}

// Eight bf16 values of a row -> pair order.
__device__ __forceinline__ bf16x8_t pair_octet(u32x4_t v)
{
    const uint32_t in[4] = {v[0], v[1], v[2], v[3]};
    uint32_t out[4];
    octet_to_pair_order(in, out);
    const u32x4_t p = {out[0], out[1], out[2], out[3]};
    return __builtin_bit_cast(bf16x8_t, p);
}

// One element of the products -> its place in out.
__device__ __forceinline__ void finish_int4(const Int4Args &g, int expert, int o, int r, float v)
{
    const Int8Epilogue &e = g.e;
    if (e.bias) v += load_typed(e.bias, e.bias_type, (size_t)expert * g.N + r);
    v = activate(v, e.activation);
    if (g.row_weights) v *= g.row_weights[o];
    if (e.residual) v += load_typed(e.residual, e.residual_type, o * e.residual_stride + r);
    store_typed(e.out, e.out_type, o * e.out_stride + r, v);
}

// The expert of a place, and the places that it has: every table entry is read
// by some thread (experts <= 4 * NT by four loads each).  False: no expert.
template <int NT>
__device__ __forceinline__ bool find_expert(const Int4Args &g, int p, int *s_e, int &e, int &begin, int &end)
{
    if (threadIdx.x == 0) *s_e = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < g.experts; i += NT)
        if (g.offsets[i] <= p && p < g.offsets[i + 1]) atomicMax(s_e, i);
    __syncthreads();
    e = *s_e;
    if (e < 0) return false;
    begin = max(g.offsets[e], 0);
    end = min(g.offsets[e + 1], g.places);
    return true;
}

// Few rows: a wave takes 16 NT weight rows and a share of K, 16 rows of x as
// the other side of v_mfma_f32_16x16x32_bf16.  Lane (q = lane / 16, c = lane %
// 16) holds the words of weight row c that lie in quarter q of a group, 16
// bytes at once, and x of row c at the same inputs.  The KS waves of a
// workgroup share K, and their sums meet in LDS.
template <int G, int NT, int KS>
__global__ __launch_bounds__(KS * kWave) void int4_rows_kernel(Int4Args g, int tiles)
{
    constexpr int kWords = G / 32;   // of a lane and group
    typedef uint32_t words_t __attribute__((ext_vector_type(kWords)));
    __shared__ int s_e;
    __shared__ float s_sum[KS][NT * 4][kWave];
    const int nb = blockIdx.x, tile = blockIdx.z * gridDim.y + blockIdx.y;
    if (tile >= tiles) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, q = lane >> 4;

    int e = 0, first = tile * 16, rows = min(16, g.places - first);
    if (g.offsets) {
        int begin, end;
        first = tile;
        if (!find_expert<KS * kWave>(g, first, &s_e, e, begin, end) || (first - begin) % 16) return;
        rows = min(16, end - first);
    }
    // the row of x of this lane's place (a row of zeros reads row 0 and is cleared at the end)
    const int place = first + min(c, rows - 1);
    int xr = g.gather ? g.gather[place] : place;
    if (g.gather) xr = xr < 0 ? -1 : xr / g.gather_div;
    const uint16_t *x = g.x + (xr >= 0 && xr < g.x_rows ? xr : 0) * g.x_stride + 8 * kWords * q;

    const int ng = g.K / G, g0 = ng * wave / KS, g1 = ng * (wave + 1) / KS;
    const int n0 = nb * (16 * NT);
    const int32_t *wq[NT];
    const uint16_t *ws[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const size_t row = (size_t)e * g.N + min(n0 + 16 * t + c, g.N - 1);
        wq[t] = g.wq + row * (g.K / 8) + kWords * q;
        ws[t] = g.ws + row * ng;
    }
    f32x4_t sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int gi = g0; gi < g1; ++gi) {
        words_t w[NT];
        u32x4_t xv[kWords];
        float scale[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            w[t] = *reinterpret_cast<const words_t *>(wq[t] + gi * (G / 8));
            scale[t] = bf16_to_f32(ws[t][gi]);
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) xv[j] = *reinterpret_cast<const u32x4_t *>(x + gi * G + 8 * j);
        bf16x8_t xb[kWords];
        f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            xb[j] = pair_octet(xv[j]);
            zero = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j], minus24(), zero, 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            f32x4_t a = zero;
#pragma unroll
            for (int j = 0; j < kWords; ++j)
                a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j], codes24(w[t][j]), a, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[t][i] = fmaf(scale[t], a[i], sum[t][i]);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_sum[wave][4 * t + i][lane] = sum[t][i];
    __syncthreads();
    for (int i = tid; i < NT * 4 * kWave; i += KS * kWave) {
        const int l = i & 63, ti = i >> 6;
        float v = s_sum[0][ti][l];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += s_sum[w][ti][l];
        const int row = 4 * (l >> 4) + (ti & 3), r = n0 + 16 * (ti >> 2) + (l & 15);
        if (row >= rows || r >= g.N) continue;
        const int p = first + row, o = g.scatter ? g.scatter[p] : p;
        if (o < 0 || o >= g.out_rows) continue;
        if (g.gather) {
            const int s = g.gather[p];
            if (s < 0 || s / g.gather_div >= g.x_rows) v = 0.f;
        }
        finish_int4(g, e, o, r, v);
    }
}

}  // namespace

size_t int4_workspace(const Int4Args &a) { return 0; }

hipError_t launch_int4_linear(const Int4Args &a, void *workspace, hipStream_t st)
{
    constexpr int NT = 2, KS = 4;
    const int tiles = a.offsets ? a.places : (a.places + 15) / 16;
    const unsigned ny = tiles < 32768 ? tiles : 32768;
    const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), ny, (tiles + ny - 1) / ny);
    if (a.G == 128) int4_rows_kernel<128, NT, KS><<<grid, KS * kWave, 0, st>>>(a, tiles);
    else int4_rows_kernel<64, NT, KS><<<grid, KS * kWave, 0, st>>>(a, tiles);
    return hipGetLastError();
}

}  // namespace moe
