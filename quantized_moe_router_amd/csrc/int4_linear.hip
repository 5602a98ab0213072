// INT4 W4A16 linear layer and the products grouped by expert:
//   out[o] = residual[o] + row_weights[o] act(x[i] W_e^T + bias[e])
//
// Two kernels.  Few rows of a matrix: its codes go through the matrix cores as
// bf16 values, unscaled, against bf16 x.  Many: x and the scaled codes are fp16
// values, each row times a power of two of its own.
//
// A word's pairs are its codes (0,4)(1,5)(2,6)(3,7); x is put in that order.
#include <type_traits>

#include "int8.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Global memory straight into LDS: lane l's 16 bytes from `at` + `more` bytes
// into a buffer go to `to` + 16 l bytes, `more` and `to` the same for the whole
// wave.  The wave waits for them with wait_loads.  (By buffer, for the compiler
// takes the form with a pointer for one that may be out of order among the
// loads, and waits for all of them where it needs one.)
typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ void load_to_lds(rsrc_t from, uint32_t at, uint32_t more, void *to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, at, more, 0, 0);
}
__device__ __forceinline__ rsrc_t buffer_of(const void *p, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, kBufferWord3);
}

// Until at most N of the wave's loads from global memory are on their way, and
// none from LDS.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);
}

__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }   // lgkmcnt(0)

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

// Columns r, r + step, .. (four, those below N) of P rows o (below 0: none).
template <int TYPE, int P>
__device__ __forceinline__ void store_columns(const Int4Args &g, const int (&o)[P], int r, int step, const float4 (&v)[P])
{
    constexpr int kBytes = TYPE == kF32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (o[i] < 0) continue;
        char *row = static_cast<char *>(g.e.out) + (o[i] * g.e.out_stride + r) * kBytes;
        const float y[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r + j * step < g.N) store_typed(row + j * step * kBytes, TYPE, 0, y[j]);
    }
}

// The same columns of the residual.
template <int TYPE, int P>
__device__ __forceinline__ void load_columns(const Int4Args &g, const int (&o)[P], int r, int step, float4 (&v)[P])
{
    constexpr int kBytes = TYPE == kF32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const char *row = static_cast<const char *>(g.e.residual) + max(o[i], 0) * g.e.residual_stride * kBytes;
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = load_typed(row, TYPE, min(r + j * step, g.N - 1));
        v[i] = make_float4(y[0], y[1], y[2], y[3]);
    }
}

// Columns r .. r + 3 of P rows, as one word.
template <int TYPE, int P>
__device__ __forceinline__ void store_words(const Int4Args &g, const int (&o)[P], int r, const float4 (&v)[P])
{
    constexpr int kBytes = TYPE == kF32 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (o[i] >= 0) store_typed4(static_cast<char *>(g.e.out) + (o[i] * g.e.out_stride + r) * kBytes, TYPE, 0, v[i]);
}

// Four columns of P rows o (below 0: none) with their weights f: r .. r + 3 where
// such words are aligned, else r, r + step, .., so that the lanes of a row move
// consecutive elements.  The residual of all rows is asked for first, so that it
// is waited for once.
template <int P>
__device__ __forceinline__ void finish_rows_int4(const Int4Args &g, int expert, const int (&o)[P], const float (&f)[P], int r, int step, float4 (&v)[P])
{
    const Int8Epilogue &e = g.e;
    if (!e.vec) {
        if (e.bias || e.residual || e.activation != kActNone || g.row_weights) {
            float4 res[P];
#pragma unroll
            for (int i = 0; i < P; ++i) res[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (e.residual) {
                if (e.residual_type == kF32) load_columns<kF32>(g, o, r, step, res);
                else if (e.residual_type == kBf16) load_columns<kBf16>(g, o, r, step, res);
                else load_columns<kF16>(g, o, r, step, res);
            }
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const float b = e.bias ? load_typed(e.bias, e.bias_type, (size_t)expert * g.N + min(r + j * step, g.N - 1)) : 0.f;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    float y = activate(v[i].x + b, e.activation) * f[i];
                    if (e.residual) y += res[i].x;
                    v[i] = make_float4(v[i].y, v[i].z, v[i].w, y);   // four turns: in order again
                    res[i] = make_float4(res[i].y, res[i].z, res[i].w, 0.f);
                }
            }
        }
        if (e.out_type == kF32) store_columns<kF32>(g, o, r, step, v);
        else if (e.out_type == kBf16) store_columns<kBf16>(g, o, r, step, v);
        else store_columns<kF16>(g, o, r, step, v);
        return;
    }
    if (e.bias || e.residual || e.activation != kActNone || g.row_weights) {
        float4 res[P];
        if (e.residual)
#pragma unroll
            for (int i = 0; i < P; ++i) res[i] = load_typed4(e.residual, e.residual_type, max(o[i], 0) * e.residual_stride + min(r, g.N - 4));
        float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
        if (e.bias) b = load_typed4(e.bias, e.bias_type, (size_t)expert * g.N + min(r, g.N - 4));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float4 y = make_float4(v[i].x + b.x, v[i].y + b.y, v[i].z + b.z, v[i].w + b.w);
            if (e.activation != kActNone)
                y = make_float4(activate(y.x, e.activation), activate(y.y, e.activation), activate(y.z, e.activation),
                                activate(y.w, e.activation));
            y = make_float4(y.x * f[i], y.y * f[i], y.z * f[i], y.w * f[i]);
            if (e.residual) y = make_float4(y.x + res[i].x, y.y + res[i].y, y.z + res[i].z, y.w + res[i].w);
            v[i] = y;
        }
    }
    if (e.out_type == kF32) store_words<kF32>(g, o, r, v);
    else if (e.out_type == kBf16) store_words<kBf16>(g, o, r, v);
    else store_words<kF16>(g, o, r, v);
}

// Which rows a workgroup takes: `count` tiles of at most 16 rows of one expert.
struct Int4Tiles {
    int count;            // with a list: the most there can be
    const int4 *list;     // [0].x: how many, then {expert, first place, rows, 0}; null: none
};

// Few rows: a wave takes 16 NT weight rows and a share of K, 16 rows of x as
// the other side of v_mfma_f32_16x16x32_bf16.  The KS waves of a workgroup
// share K, and their sums meet in LDS.
//
// K goes in units of 128 inputs, the codes (64 bytes of each weight row) and x
// (256 bytes of a row) straight into a wave's own part of LDS, double-buffered:
// a load whose neighbouring lanes read along a row costs a quarter of one in
// the order of the matrix operands, whose neighbouring lanes are neighbouring
// rows.  No wave waits for another before the end.  XR: rows of x that are
// copied (4 of few tokens, the products of the others are of no use).
//
// Codes become bf16 by placing a nibble n = code + 8 in the mantissa of 16.0:
// 0x4180 | n << 3 is 16 + n = code + 24 exactly, so a word takes four shifts
// and four AND-ORs for its eight codes.  The 24 too much is taken off by the
// matrix cores: the accumulators of a group begin at the product of x with a
// matrix of -24 (one such product serves every column tile of the wave), and
// what the group's products leave there is sum x code, exact up to fp32's
// additions.  These pass through 24 sum |x| of a group: for x of one sign an
// output is off by up to 1.0e-6 of its size (a plain fp32 sum 2e-7), for x of
// both signs by 1.2e-7 (2.6e-7; K of 2560, groups of 128).  The group's scale
// multiplies that sum in fp32, so neither x nor a weight is ever rounded.  (The
// 24 taken off after every 32 inputs, in each column tile: 2.3e-7 for x of one
// sign, and 1 to 3.5 % more time, 216 -> 218 us for 5120 places, 27.1 -> 28.1
// for 128 tokens of [10240, 2560].)
//
// What bounds it: memory where it is large (one token of [248320, 2560] 72 us,
// 4.6 TB/s, nearly the rate of a copy; 5120 places of 512 experts, [1280, 2560],
// 216 us, 4.1 TB/s, with the vector ALU busy 55 % of the time), and the way
// through its dependent loads where it is small (one token of [2560, 2560]: 6
// us, of which the matrix takes 0.7).  Between them, 17 to 512 rows of a matrix
// (64 tokens of [10240, 2560] 17 us, where memory takes 3), it makes the codes
// anew for every 16 rows.  The buffer of the codes is held in vector registers
// (for the clamp of its rows), so each copy of codes is a loop over it.  Straight
// to LDS against loads into registers in the operands' order: 70 us against 82,
// and 12.6 against 15.0 for 32 tokens of [10240, 2560] (11.1 with two column tiles
// a wave).
template <int G, int NT, int KS, int WC, int XR>
__global__ __launch_bounds__(KS * WC * kWave) void int4_rows_kernel(Int4Args g, Int4Tiles tl, int nblocks)
{
    constexpr int kGroups = 128 / G, kWords = G / 32;   // groups of a unit; words of a lane and group
    constexpr int kWaves = KS * WC, kThreads = kWaves * kWave, kCols = 16 * NT * WC;
    constexpr int kXCopies = WC == 1 ? XR / 4 : (XR / 4 + WC - 1) / WC;   // of a wave and unit
    constexpr int kLoads = NT + kXCopies;
    constexpr int kBufs = WC == 1 ? 2 : 3;              // (see the loops)
    constexpr int kAhead = 8;                           // units whose scales a wave holds
    typedef uint32_t words_t __attribute__((ext_vector_type(kWords)));
    __shared__ struct __align__(16) {
        uint32_t w[kWaves][kBufs][NT * 16 * 16];
        uint16_t x[KS][kBufs][XR * 128];
        uint16_t scale[kWaves][kAhead * kGroups][16 * NT];
        int out[16];   // row of out of each row of the tile, -1: none; with bit 30 set its row of x is zeros
        int e;
    } s;
    static_assert(sizeof(s.w) + sizeof(s.x) >= sizeof(float) * kWaves * NT * 4 * kWave, "the sums take the place of the operands");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int wc = wave % WC, ks = wave / WC;
    // every XCD has consecutive tiles, all weight blocks of one after the other:
    // the tiles of an expert find its weights in one L2
    const int total = tl.list ? tl.list[0].x : tl.count, per = (total * nblocks + 7) / 8;
    const int at = blockIdx.x >> 3, work = (blockIdx.x & 7) * per + at, tile = work / nblocks, nb = work - tile * nblocks;
    if (at >= per || tile >= total) return;

    int e = 0, first, rows;
    if (!g.offsets) {
        first = tile * 16;
        rows = min(16, g.places - first);
    } else if (tl.list) {
        const int4 t = tl.list[1 + tile];
        e = t.x, first = t.y, rows = t.z;
    } else {   // a workgroup for each place: the first of sixteen of an expert works
        first = tile;
        if (tid == 0) s.e = -1;
        __syncthreads();
        for (int i = tid; i < g.experts; i += kThreads)
            if (g.offsets[i] <= first && first < g.offsets[i + 1]) atomicMax(&s.e, i);
        __syncthreads();
        e = __builtin_amdgcn_readfirstlane(s.e);
        if (e < 0 || (first - max(g.offsets[e], 0)) % 16) return;
        rows = min(16, min(g.offsets[e + 1], g.places) - first);
    }
    const int units = (g.K + 127) / 128, ng = g.K / G, kw = g.K / 8;
    const int u0 = units * ks / KS, u1 = units * (ks + 1) / KS;
    const int n0 = nb * kCols, nw = n0 + 16 * NT * wc, nrows = max(0, min(16 * NT, g.N - nw));
    if (tid < 16) {
        const int p = first + min(tid, rows - 1);
        int o = g.scatter ? g.scatter[p] : p;
        if (tid >= rows || o < 0 || o >= g.out_rows) o = -1;
        if (g.gather && o >= 0) {
            const int slot = g.gather[p];
            if (slot < 0 || slot / g.gather_div >= g.x_rows) o |= 1 << 30;
        }
        s.out[tid] = o;
    }

    // Codes: copy t takes 16 rows, lane l piece (l % 4) ^ (row / 4 % 4) of row l
    // / 4; behind the matrix, zeros come.  x: copy i takes rows 4 i .. 4 i + 3,
    // lane l piece (l % 16) ^ row of row l / 16.  Reads meet no bank twice.
    const rsrc_t w_buf = buffer_of(g.wq + ((size_t)e * g.N + min(nw, g.N - 1)) * kw, (uint32_t)nrows * (uint32_t)kw * 4u);
    const uint32_t wsrc = 4u * (uint32_t)(lane >> 2) * (uint32_t)kw + 16 * ((lane & 3) ^ (lane >> 4 & 3));
    // (without gather the rows are consecutive: their first is the buffer's)
    const rsrc_t x_buf = buffer_of(g.x + (g.gather ? 0 : (size_t)first * g.x_stride),
                                   2u * ((uint32_t)((g.gather ? g.x_rows : rows) - 1) * (uint32_t)g.x_stride + (uint32_t)g.K));
    uint32_t xsrc[kXCopies];
    int slot[kXCopies];
    auto copied = [&](int i) __attribute__((always_inline)) { return WC == 1 ? i : (wc + i * WC) % (XR / 4); };   // which of x
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) slot[i] = min(4 * copied(i) + (lane >> 4), rows - 1);
    if (g.gather)
#pragma unroll
        for (int i = 0; i < kXCopies; ++i) slot[i] = g.gather[first + slot[i]];
#pragma unroll
    for (int i = 0; i < kXCopies; ++i) {   // (a row of zeros reads row 0 and is cleared at the end)
        const int xr = slot[i] < 0 ? 0 : slot[i] / g.gather_div;
        xsrc[i] = 2u * (uint32_t)(xr < g.x_rows ? xr : 0) * (uint32_t)g.x_stride + 16 * ((lane & 15) ^ (lane >> 4) ^ (4 * copied(i)));
    }
    auto copy = [&](int u, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) load_to_lds(w_buf, wsrc + (uint32_t)(64 * t) * (uint32_t)kw, 64 * u, s.w[wave][buf] + t * 256);
#pragma unroll
        for (int i = 0; i < kXCopies; ++i)   // (half a unit at K's end: what comes behind it is not used)
            load_to_lds(x_buf, xsrc[i], 256 * u, s.x[ks][buf] + copied(i) * 512);
    };
    // scales of kAhead units, a lane a row
    auto scales = [&](int u) __attribute__((always_inline)) {
        if (lane < 16 * NT) {
            const uint16_t *ws = g.ws + ((size_t)e * g.N + min(nw + lane, g.N - 1)) * ng;
            if (ng >= 4) {   // four at a time; behind the last, none are used
                struct __attribute__((packed, aligned(2))) four_t { uint64_t v; };
                uint64_t v[kAhead * kGroups / 4];
#pragma unroll
                for (int i = 0; i < kAhead * kGroups / 4; ++i)
                    v[i] = reinterpret_cast<const four_t *>(ws + min(u * kGroups + 4 * i, ng - 4))->v;
#pragma unroll
                for (int i = 0; i < kAhead * kGroups / 4; ++i) {
                    v[i] >>= 16 * (min(u * kGroups + 4 * i - min(u * kGroups + 4 * i, ng - 4), 3));
#pragma unroll
                    for (int j = 0; j < 4; ++j) s.scale[wave][4 * i + j][lane] = (uint16_t)(v[i] >> (16 * j));
                }
            } else {
                for (int i = u * kGroups; i < ng; ++i) s.scale[wave][i - u * kGroups][lane] = ws[i];
            }
        }
    };
    f32x4_t sum[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) sum[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // The quarter of a group that lane quarter q takes.  LDS serves lanes 0-3,
    // 12-15 and 20-27 of a half wave together, then the others: with quarters 0
    // and 3 beside each other (and 1 and 2) those meet no bank twice, in order
    // they met every one.  (Half groups, of 64, do in order.)
    const int qk = G == 128 ? (q == 0 ? 0 : q == 1 ? 3 : q - 1) : q;
    auto compute = [&](int u, int buf) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < kGroups; ++a) {
            if (a && u * kGroups + a >= ng) break;
            bf16x8_t xb[kWords];
            f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                const int octet = (G / 8) * a + kWords * qk + j, row = c % XR;
                xb[j] = pair_octet(*reinterpret_cast<const u32x4_t *>(s.x[ks][buf] + row * 128 + 8 * (octet ^ row)));
                zero = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j], minus24(), zero, 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                // the lane's words: bytes 4 kWords qk of the group's
                const int byte = (G / 2) * a + 4 * kWords * qk;
                const words_t w = *reinterpret_cast<const words_t *>(
                    s.w[wave][buf] + t * 256 + c * 16 + 4 * ((byte >> 4) ^ (c >> 2 & 3)) + (byte >> 2 & 3));
                f32x4_t v = zero;
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j], codes24(w[j]), v, 0, 0, 0);
                const float f = bf16_to_f32(s.scale[wave][(u - u0) % kAhead * kGroups + a][16 * t + c]);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[t][i] = fmaf(f, v[i], sum[t][i]);
            }
        }
    };
    if (u0 < u1) copy(u0, 0);
    if (u0 + 1 < u1) copy(u0 + 1, 1);
    if constexpr (WC == 1) {
        // each wave by itself: a unit's place is free when its reads have ended
        auto unit = [&](int u, int buf) __attribute__((always_inline)) {
            if ((u - u0) % kAhead == 0) scales(u);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            if (u + 1 < u1) wait_loads<kLoads>();
            else wait_loads<0>();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            compute(u, buf);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            if (u + 2 < u1) {
                wait_lds();
                copy(u + 2, buf);
            }
        };
        for (int u = u0; u < u1; u += 2) {
            unit(u, 0);
            if (u + 1 < u1) unit(u + 1, 1);
        }
    } else {
        // x is shared: behind the barrier a unit is there for every wave, and the
        // place of the one before it is free
        auto unit = [&](int u, int buf) __attribute__((always_inline)) {
            if ((u - u0) % kAhead == 0) scales(u);
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            if (u + 1 < u1) wait_loads<kLoads>();
            else wait_loads<0>();
            __builtin_amdgcn_s_barrier();
            __atomic_signal_fence(__ATOMIC_SEQ_CST);
            if (u + 2 < u1) copy(u + 2, (buf + 2) % 3);
            compute(u, buf);
        };
        for (int u = u0; u < u1; u += 3) {
            unit(u, 0);
            if (u + 1 < u1) unit(u + 1, 1);
            if (u + 2 < u1) unit(u + 2, 2);
        }
    }
    __syncthreads();
    float (*s_sum)[NT * 4][kWave] = reinterpret_cast<float (*)[NT * 4][kWave]>(&s.w);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s_sum[wave][4 * t + i][lane] = sum[t][i];
    __syncthreads();
    for (int i = tid; i < rows * kCols; i += kThreads) {
        // consecutive threads: consecutive columns of a row
        const int col = i % kCols, row = i / kCols, r = n0 + col, cw = col % (16 * NT);
        const int ti = 4 * (cw >> 4) + (row & 3), l = 16 * (row >> 2) + (cw & 15), w0 = col / (16 * NT);
        const int o = s.out[row];
        if (o < 0 || r >= g.N) continue;
        float v = s_sum[w0][ti][l];
#pragma unroll
        for (int w = 1; w < KS; ++w) v += s_sum[w * WC + w0][ti][l];
        finish_int4(g, e, o & ~(1 << 30), r, o >> 30 ? 0.f : v);
    }
}

// ---------------------------------------------------------------------------
// Many rows.  A pass over x writes it as fp16 in pair order, each row times a
// power of two of its own; then a workgroup takes a chunk of up to 32 MAXMA
// sorted rows of one expert and 32 WAVES weight rows, 32 of them to a wave, as
// v_mfma_f32_32x32x16_f16 tiles whose sums stay in registers over all of K.  K
// goes in stages of 128: x and codes straight into LDS (16-byte pieces,
// exclusive-or'ed by the row, so that reads meet no bank twice), two stages
// ahead.  A wave makes its 32 rows' weights once a stage, in registers, for all
// row tiles.
//
// The scale goes into the fp16 weight, not onto a group's sum as in the kernel
// above: there sixteen products with it per tile and group, and a sum of x per
// row, cost more here than the three instructions a word more do (81920 places
// of 512 experts, [1280, 2560]: 820 us against 749).
//
// What bounds it: at 81920 places (684 to 708 us, 758 to 785 TFLOP/s, 61 % of a
// large library product) the matrix cores are busy 45 % of the cycles, the vector
// ALU 26 %, LDS 27 %; waves wait two fifths of their time, most of it where a
// stage begins: a barrier, the first reads of LDS and the first weights follow
// each other (about 1300 cycles of a stage's 3400 with 128 rows; a row tile more
// costs what its products cost).  Part of that is that the scales cross the loop
// in registers: where a turn of the loop begins (three stages; of chunks of 192
// six, and there in the second stage, too) the compiler waits for every load
// before it reads them, the copies for the next stages among them.  512 tokens of
// [10240, 2560] (49 us): 160 workgroups for 256 CUs besides, and 11 us of the
// pass over x, the start and the end.
// ---------------------------------------------------------------------------
constexpr int kStageK = 128;

// What the pass over x leaves in the workspace.  It takes 5 us for 512 rows of
// 2560, 22 us for 8192.
struct Int4Plan {
    int rows;       // rows of xp: those of x, or the places where x has more; and one of zeros behind them
    bool by_place;
    int kp;         // K rounded up to a stage
    int most;       // rows of a chunk
    int tiles;      // most chunks that there can be
    size_t exps_at, list_at, bytes;
};

// The tiles of each expert, in its order: nearly equal parts of at most `most`
// rows.  One workgroup of 256; list[0].x: how many.
__device__ inline void list_tiles(const Int4Args &g, int most, int slots, int4 *list)
{
    __shared__ int s_sum[4];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 256) {
        const int e = e0 + threadIdx.x;
        int begin = 0, cnt = 0;
        if (e < g.experts) {
            begin = min(max(g.offsets[e], 0), g.places);
            cnt = max(min(g.offsets[e + 1], g.places) - begin, 0);
        }
        const int nc = (cnt + most - 1) / most;
        int incl = nc;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(incl, off, 64);
            if (lane >= off) incl += o;
        }
        __syncthreads();
        if (lane == 63) s_sum[wave] = incl;
        __syncthreads();
        int at = base + incl - nc;
        for (int w = 0; w < 4; ++w) {
            if (w < wave) at += s_sum[w];
            base += s_sum[w];
        }
        for (int i = 0; i < nc && at + i < slots; ++i) {
            const int b = (int)((long)cnt * i / nc), en = (int)((long)cnt * (i + 1) / nc);
            list[1 + at + i] = make_int4(e, begin + b, en - b, 0);
        }
    }
    if (threadIdx.x == 0) list[0] = make_int4(min(base, slots), 0, 0, 0);
}

__global__ __launch_bounds__(256) void int4_list_kernel(Int4Args g, int most, int slots, int4 *list)
{
    list_tiles(g, most, slots, list);
}

__global__ __launch_bounds__(256) void int4_prepare_kernel(Int4Args g, Int4Plan pl, uint16_t *xp, int *exps, int4 *list)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int row_blocks = (pl.rows + 1 + 3) / 4;
    if ((int)blockIdx.x >= row_blocks) {
        list_tiles(g, pl.most, pl.tiles, list);
        return;
    }
    const int row = blockIdx.x * 4 + wave;
    if (row > pl.rows) return;
    int xr = row < pl.rows ? row : -1;   // behind the last: the row of zeros
    if (pl.by_place && xr >= 0 && g.gather) {
        const int s = g.gather[row];
        xr = s < 0 ? -1 : s / g.gather_div;
        if (xr >= g.x_rows) xr = -1;
    }
    const uint16_t *x = g.x + max(xr, 0) * g.x_stride;
    // the row's largest exponent, then its values times a power of two that
    // brings the largest below 2^15; up to 4096 inputs stay in registers
    constexpr int kHeld = 8;
    u32x4_t v[kHeld];
    auto read = [&](int k0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int k = k0 + 512 * i + 8 * lane;
            v[i] = u32x4_t{0u, 0u, 0u, 0u};
            if (xr >= 0 && k < g.K) v[i] = *reinterpret_cast<const u32x4_t *>(x + k);
        }
    };
    uint32_t top = 0;
    for (int k0 = 0; k0 < g.K; k0 += 512 * kHeld) {
        read(k0);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max(v[i][j] & 0x7F80u, (v[i][j] >> 16) & 0x7F80u));
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
    const int e = max((int)(top >> 7), 1), shift = e == 255 ? 0 : 141 - e;
    if (lane == 0) exps[row] = -shift;
    for (int k0 = 0; k0 < pl.kp; k0 += 512 * kHeld) {
        if (g.K > 512 * kHeld) read(k0);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            u32x4_t y;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // element j with element j + 4
                const uint32_t a = v[i][j >> 1], b = v[i][2 + (j >> 1)];
                const float fa = j & 1 ? bf16_hi(a) : bf16_lo(a), fb = j & 1 ? bf16_hi(b) : bf16_lo(b);
                y[j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(ldexpf(fa, shift), ldexpf(fb, shift)));
            }
            if (e == 255) y = u32x4_t{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};   // NaN
            const int k = k0 + 512 * i + 8 * lane;
            if (k < pl.kp) *reinterpret_cast<u32x4_t *>(xp + (size_t)row * pl.kp + k) = y;
        }
    }
}

// The weight blocks of a chunk are dealt to one XCD in units of `unit` blocks,
// so that what they share of x stays in its L2.
struct Int4Grid {
    int nblocks, unit, units;   // weight blocks, blocks of a unit, units of a chunk
};

// Word -> MFMA operand: eight fp16 values code * s in pair order.  fp16 0x4C00
// is 16 with a mantissa step of 1/64, so a nibble in bits 6-9 makes 16 + n; (16
// + n) s - 24 s is (n - 8) s, exact in one fused step: at most eleven bits.
__device__ __forceinline__ f16x8_t codes_times(uint32_t w, h2_t s, h2_t s24)
{
    const uint32_t m = vconst(0x03C003C0u), b = vconst(0x4C004C00u);
    const uint32_t p[4] = {((w << 6) & m) | b, ((w << 2) & m) | b, ((w >> 2) & m) | b, ((w >> 6) & m) | b};
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        v[j] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(h2_t, p[j]), s, s24));
    return __builtin_bit_cast(f16x8_t, v);
}

template <int G, int MAXMA, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void int4_tile_kernel(Int4Args g, Int4Plan pl, Int4Grid gr, const uint16_t *xp, const int *exps, const int4 *list)
{
    constexpr int NT = WAVES * kWave, kRows = 32 * MAXMA, kCols = 32 * WAVES, kGroups = kStageK / G;
    constexpr int kBufs = MAXMA <= 4 ? 3 : 2;   // of x: as many as fit LDS beside three of codes
    constexpr int kX = kRows * 16 / NT;         // copies of a wave and stage, beside two of codes
    // loads that may be on their way when a stage begins (see there)
    constexpr int kFlight = kBufs == 3 ? kX + 2 + 2 * kGroups : 2 + kGroups;
    // one object: with several the compiler waits for every copy on its way
    // before it reads any of them
    __shared__ struct __align__(16) {
        uint16_t x[kBufs][kRows * kStageK];
        uint32_t w[3][kCols * kStageK / 8];
        int exp[kRows];
        int row[kRows];
        int out[kRows];
        float weight[kRows];
    } s;
    const int xcd = blockIdx.x & 7, r = blockIdx.x >> 3;
    const int u = (r / gr.unit) * 8 + xcd, chunk = u / gr.units, nb = (u % gr.units) * gr.unit + r % gr.unit;
    if (chunk >= pl.tiles || nb >= gr.nblocks) return;
    int e = 0, first, rows;
    if (g.offsets) {
        const int count = list[0].x;
        const int4 t = list[1 + chunk];   // (of a slot that is not filled it is not used)
        if (chunk >= count) return;
        e = t.x, first = t.y, rows = t.z;
    } else {
        first = (int)((long)g.places * chunk / pl.tiles);
        rows = (int)((long)g.places * (chunk + 1) / pl.tiles) - first;
    }
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 31, h = lane >> 5;
    const int stages = pl.kp / kStageK, mtiles = (rows + 31) / 32;
    const int n0 = nb * kCols, nrows = min(kCols, g.N - n0);   // weight rows of the workgroup
    const int kw = g.K / 8, ng = g.K / G;

    // Codes: a wave copies the 64 bytes of its own 32 rows, 16 rows at once;
    // lane l takes piece (l % 4) ^ (row / 4 % 4) of its row, so that the reads
    // meet no bank twice.  Behind the last row of the matrix, zeros come.
    const rsrc_t w_buf = buffer_of(g.wq + ((size_t)e * g.N + n0) * kw, (uint32_t)nrows * (uint32_t)kw * 4u);
    uint32_t wsrc[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        const int row = 16 * o + (lane >> 2);
        wsrc[o] = 4u * (uint32_t)(32 * wave + row) * (uint32_t)kw + 16 * ((lane & 3) ^ (row >> 2 & 3));
    }
    auto copy_w = [&](int st, int buf, int o) __attribute__((always_inline)) {
        load_to_lds(w_buf, wsrc[o], kStageK / 2 * min(st, stages - 1), s.w[buf] + (32 * wave + 16 * o) * (kStageK / 8));
    };
#pragma unroll
    for (int o = 0; o < 4; ++o) copy_w(o >> 1, o >> 1, o & 1);

    for (int i = tid; i < kRows; i += NT) {
        int at = pl.rows;   // zeros
        if (i < rows) {
            at = first + i;
            if (!pl.by_place && g.gather) {
                const int slot = g.gather[first + i];
                at = slot < 0 ? pl.rows : min(slot / g.gather_div, pl.rows);
            }
        }
        s.row[i] = at;
    }
    __syncthreads();

    // x: copy o of a wave takes rows 4 (WAVES o + wave) .. + 3, lane l piece (l
    // % 16) ^ (row % 16) of its row
    const rsrc_t x_buf = buffer_of(xp, (uint32_t)(pl.rows + 1) * (uint32_t)pl.kp * 2u);
    uint32_t src[kX];   // bytes
#pragma unroll
    for (int o = 0; o < kX; ++o) {
        const int row = 4 * (WAVES * o + wave) + (lane >> 4);
        src[o] = 2u * (uint32_t)s.row[row] * (uint32_t)pl.kp + 16 * ((lane & 15) ^ (row & 15));
    }
    auto copy_x = [&](int st, int buf, int o) __attribute__((always_inline)) {
        load_to_lds(x_buf, src[o], 2 * kStageK * min(st, stages - 1), s.x[buf] + 4 * (WAVES * o + wave) * kStageK);
    };
#pragma unroll
    for (int o = 0; o < kX; ++o) copy_x(0, 0, o);
    if (kBufs == 3)
#pragma unroll
        for (int o = 0; o < kX; ++o) copy_x(1, 1, o);

    // The scales of a weight row are taken times a power of two that brings the
    // largest finite one below 2^11: then 24 s, and with it code * s, is within
    // fp16's range, and scales down to 2^-24 of it are exact.
    const uint16_t *ws = g.ws + ((size_t)e * g.N + min(n0 + 32 * wave + c, g.N - 1)) * ng;
    uint32_t sc[3][kGroups];
    auto fetch = [&](int st, int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) sc[set][i] = ws[min(st * kGroups + i, ng - 1)];
    };
    uint32_t top = 0;
#pragma unroll 8
    for (int i = h; i < ng; i += 2) {
        const uint32_t b = ws[i] & 0x7F80u;
        top = max(top, b == 0x7F80u ? 0u : b);
    }
    // what the epilogue needs of the rows, while their x is on its way
    for (int i = tid; i < kRows; i += NT) {
        int o = -1;   // nowhere
        if (i < rows) {
            o = g.scatter ? g.scatter[first + i] : first + i;
            if (o < 0 || o >= g.out_rows) o = -1;
        }
        s.exp[i] = exps[s.row[i]];
        s.out[i] = o;
        s.weight[i] = g.row_weights && o >= 0 ? g.row_weights[o] : 1.f;
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    const int wshift = 137 - max((int)(top >> 7), 1);

    f32x16_t acc[MAXMA];
#pragma unroll
    for (int m = 0; m < MAXMA; ++m)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[m][j] = 0.f;

    // A stage's loads are issued in the order x, codes, scales: with three
    // buffers of x all for the stage after the next (scales one later), with
    // two x for the next.  What a stage reads has arrived when at most the
    // kFlight loads issued after it are on their way.  Behind the barrier that
    // holds for every wave, and the buffers of the stage before are free.  A
    // stage is 2 MA steps of four products; while those of a step run, x of the
    // next is read, and a weight operand is made between the products of the
    // first row tile, just before its use.
    auto stage = [&](auto ma_c, int st, int set, int xset) __attribute__((always_inline)) {
        constexpr int MA = decltype(ma_c)::value, kSteps = 2 * MA;
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        wait_loads<kFlight>();
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        // this lane's row and its piece 4 h; opaque, so that the eight places
        // made from it are formed anew instead of held over all stages
        uint32_t at = 2 * kStageK * c + 16 * ((c & 15) ^ (4 * h));
        asm volatile("" : "+v"(at));
        // lane half h takes pieces h and 2 + h of its weight row's 64 bytes; word
        // j of the p-th holds the inputs of octet 8 p + 4 h + j of the stage
        u32x4_t wv[2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
            wv[p] = *reinterpret_cast<const u32x4_t *>(s.w[set] + (32 * wave + c) * (kStageK / 8) + 4 * ((2 * p + h) ^ (c >> 2 & 3)));
        f16x8_t x[2][4], w[8];
        auto read_x = [&](int step) __attribute__((always_inline)) {
            const char *xm = reinterpret_cast<const char *>(s.x[xset]) + 32 * (step >> 1) * (2 * kStageK);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[step & 1][j] = *reinterpret_cast<const f16x8_t *>(xm + (at ^ 16 * (8 * (step & 1) + j)));
        };
        read_x(0);
        h2_t scale[kGroups], s24[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const _Float16 f = (_Float16)ldexpf(bf16_to_f32((uint16_t)sc[set][i]), wshift);
            scale[i] = h2_t{f, f};
            s24[i] = scale[i] * h2_t{(_Float16)-24.f, (_Float16)-24.f};
            asm volatile("" : "+v"(scale[i]), "+v"(s24[i]));
        }
        __builtin_amdgcn_sched_barrier(0);
        // the loads of the stage, spread over its steps: all at once, behind the
        // barrier, they would hold every wave up before its first product
        auto load = [&](int i) __attribute__((always_inline)) {
            // kFlight counts on the order of the three kinds, and to the compiler
            // a scale's load into a register is independent of copies into LDS
            if (i == kX || i == kX + 2) {
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (i < kX) copy_x(kBufs == 3 ? st + 2 : st + 1, kBufs == 3 ? (set + 2) % 3 : xset ^ 1, i);
            else if (i < kX + 2) copy_w(st + 2, (set + 2) % 3, i - kX);
            else fetch(st + 3, set);
        };
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            if (step + 1 < kSteps) read_x(step + 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = 4 * (step & 1) + j, p = step & 1;
                if (step < 2) w[k] = codes_times(wv[p][j], scale[p % kGroups], s24[p % kGroups]);
                acc[step >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[p][j], w[k], acc[step >> 1], 0, 0, 0);
            }
#pragma unroll
            for (int i = (kX + 3) * step / kSteps; i < (kX + 3) * (step + 1) / kSteps; ++i) load(i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto all = [&](auto ma_c) __attribute__((always_inline)) {
        fetch(0, 0);
        fetch(1, 1);
        fetch(2, 2);
        wait_loads<3 * kGroups>();   // the first copies: fewer loads follow them than later ones
        if constexpr (kBufs == 3) {
            for (int st = 0; st < stages; st += 3) {
                stage(ma_c, st, 0, 0);
                if (st + 1 < stages) stage(ma_c, st + 1, 1, 1);
                if (st + 2 < stages) stage(ma_c, st + 2, 2, 2);
            }
        } else {
            for (int st = 0; st < stages; st += 6) {
                stage(ma_c, st, 0, 0);
                if (st + 1 < stages) stage(ma_c, st + 1, 1, 1);
                if (st + 2 < stages) stage(ma_c, st + 2, 2, 0);
                if (st + 3 < stages) stage(ma_c, st + 3, 0, 1);
                if (st + 4 < stages) stage(ma_c, st + 4, 1, 0);
                if (st + 5 < stages) stage(ma_c, st + 5, 2, 1);
            }
        }
    };
    static_assert(MAXMA == 4 || MAXMA == 6, "a case for each number of row tiles");
    if (mtiles == 1) all(std::integral_constant<int, 1>{});
    else if (mtiles == 2) all(std::integral_constant<int, 2>{});
    else if (mtiles == 3) all(std::integral_constant<int, 3>{});
    else if (MAXMA == 4 || mtiles == 4) all(std::integral_constant<int, 4>{});
    else if constexpr (MAXMA == 6) {
        if (mtiles == 5) all(std::integral_constant<int, 5>{});
        else all(std::integral_constant<int, 6>{});
    }
    wait_loads<0>();   // the copies of stages that do not come, too

    // 32 rows at a time through LDS, so that a thread has four columns of a row;
    // one body for all row tiles, for its code is fetched anew at every launch
    constexpr int kPitch = kCols + 4, kPer = 32 * kCols / 4 / NT;   // rows of a thread
    static_assert(2 * sizeof(float) * 32 * kPitch <= sizeof(s.x), "staging of the epilogue");
    const int col = (g.e.vec ? 4 : 1) * (tid % (kCols / 4)), n = n0 + col, row0 = tid / (kCols / 4);
#pragma unroll 1
    for (int m = 0; m < mtiles; ++m) {
        if (m == 0) __syncthreads();   // every wave's last reads of x
        // two places in turn: a wave writes the next rows while others read
        float *s_y = reinterpret_cast<float *>(s.x) + (m & 1) * (32 * kPitch);
#pragma unroll
        for (int mm = 0; mm < MAXMA; ++mm)
            if (m == mm)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int row = 8 * (j >> 2) + 4 * h + (j & 3);
                    s_y[row * kPitch + 32 * wave + c] = ldexpf(acc[mm][j], s.exp[32 * m + row] - wshift);
                }
        __syncthreads();
        int o[kPer];
        float f[kPer];
        float4 v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int row = row0 + i * (NT / (kCols / 4));
            o[i] = n < g.N ? s.out[32 * m + row] : -1;
            f[i] = s.weight[32 * m + row];
            const float *y = s_y + row * kPitch + col;
            if (g.e.vec) v[i] = *reinterpret_cast<const float4 *>(y);
            else v[i] = make_float4(y[0], y[kCols / 4], y[2 * (kCols / 4)], y[3 * (kCols / 4)]);
        }
        finish_rows_int4(g, e, o, f, n, kCols / 4, v);
    }
}

template <int G, int MAXMA>
void launch_tiles(const Int4Args &a, const Int4Plan &pl, uint16_t *xp, int *exps, int4 *list, hipStream_t st)
{
    constexpr int WAVES = 8;
    Int4Grid gr;
    gr.nblocks = (a.N + 32 * WAVES - 1) / (32 * WAVES);
    // whole chunks, where eight units for each XCD are left
    const long blocks = (long)gr.nblocks * pl.tiles;
    gr.unit = blocks / 64 < 1 ? 1 : (blocks / 64 < gr.nblocks ? (int)(blocks / 64) : gr.nblocks);
    gr.units = (gr.nblocks + gr.unit - 1) / gr.unit;
    const unsigned grid = (unsigned)((pl.tiles * gr.units + 7) / 8 * 8) * (unsigned)gr.unit;
    int4_tile_kernel<G, MAXMA, WAVES><<<grid, WAVES * kWave, 0, st>>>(a, pl, gr, xp, exps, list);
}

template <int NT, int KS, int WC, int XR>
void launch_rows(const Int4Args &a, const Int4Tiles &tl, hipStream_t st)
{
    const int nblocks = (a.N + 16 * NT * WC - 1) / (16 * NT * WC);
    const unsigned grid = ((unsigned)tl.count * (unsigned)nblocks + 7) / 8 * 8;
    if (a.G == 128) int4_rows_kernel<128, NT, KS, WC, XR><<<grid, KS * WC * kWave, 0, st>>>(a, tl, nblocks);
    else int4_rows_kernel<64, NT, KS, WC, XR><<<grid, KS * WC * kWave, 0, st>>>(a, tl, nblocks);
}

// Most tiles of `most` rows that the places can make.
int most_tiles(const Int4Args &a, int most)
{
    if (!a.grouped) return (a.places + most - 1) / most;
    return a.places / most + (a.experts < a.places ? a.experts : a.places);
}

// Whether the rows are many enough for the kernel that makes a copy of x: a
// third of the chip's CUs with a tile of 128 x 256 (512 tokens of [10240, 2560]
// 49 us, by sixteen rows 81; 256 tokens 40 and 43; 128 tokens, which stay with
// the other, 39 and 27; of [2560, 2560], 512 tokens 41 and 25), and 32 rows to an
// expert (20480 places of 512 experts 334 us against 455; 10240 places 288, 278).
bool many_rows(const Int4Args &a)
{
    return a.places >= 32L * a.experts && (long)((a.places + 127) / 128) * ((a.N + 255) / 256) >= 80;
}
// Few places: the workgroups find their experts themselves, 256 threads for each
// place and 128 columns.  Where these would be 2^32 (of 2^24 columns) the list,
// which has a tile for every sixteen places and expert, stays below.
bool listed(const Int4Args &a)
{
    return a.grouped && (a.places > 128 || (long)a.places * ((a.N + 127) / 128) >= 1L << 24);
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

Int4Plan tile_plan(const Int4Args &a)
{
    Int4Plan p{};
    p.by_place = a.x_rows > a.places;
    p.rows = p.by_place ? a.places : a.x_rows;
    p.kp = (a.K + kStageK - 1) / kStageK * kStageK;
    // 192 rows where the experts have more than 96 each (81920 places of 512
    // experts 706 us, with 128 rows 738), 128 otherwise (20480 places 334, 348;
    // 512 tokens of one matrix 49, 63: the last round of tiles fills the chip better)
    p.most = a.grouped && a.places > 96L * a.experts ? 192 : 128;
    p.tiles = most_tiles(a, p.most);
    p.exps_at = up256(2 * (size_t)(p.rows + 1) * p.kp);
    p.list_at = p.exps_at + up256(4 * (size_t)(p.rows + 1));
    p.bytes = p.list_at + up256(16 * (size_t)(p.tiles + 1));
    return p;
}

}  // namespace

size_t int4_workspace(const Int4Args &a)
{
    if (a.places <= 0) return 0;
    if (many_rows(a)) return tile_plan(a).bytes;
    return listed(a) ? up256(16 * (size_t)(most_tiles(a, 16) + 1)) : 0;
}

hipError_t launch_int4_linear(const Int4Args &a, void *workspace, hipStream_t st)
{
    char *ws = static_cast<char *>(workspace);
    if (many_rows(a)) {
        const Int4Plan pl = tile_plan(a);
        uint16_t *xp = reinterpret_cast<uint16_t *>(ws);
        int *exps = reinterpret_cast<int *>(ws + pl.exps_at);
        int4 *list = reinterpret_cast<int4 *>(ws + pl.list_at);
        int4_prepare_kernel<<<(pl.rows + 4) / 4 + (a.grouped ? 1 : 0), 256, 0, st>>>(a, pl, xp, exps, list);
        if (a.G == 128) pl.most == 192 ? launch_tiles<128, 6>(a, pl, xp, exps, list, st) : launch_tiles<128, 4>(a, pl, xp, exps, list, st);
        else pl.most == 192 ? launch_tiles<64, 6>(a, pl, xp, exps, list, st) : launch_tiles<64, 4>(a, pl, xp, exps, list, st);
        return hipGetLastError();
    }
    Int4Tiles tl{};
    if (listed(a)) {
        tl.count = most_tiles(a, 16);
        int4 *list = reinterpret_cast<int4 *>(ws);
        int4_list_kernel<<<1, 256, 0, st>>>(a, 16, tl.count, list);
        tl.list = list;
    } else {
        tl.count = a.grouped ? a.places : (a.places + 15) / 16;
    }
    // Enough columns to go round: the waves of a workgroup take columns and share
    // x (640 places of 512 experts, [2560, 640]: 71 us, with K over the waves 141,
    // with that and four column tiles a wave 119).  Fewer: four of them share K (8
    // tokens of [10240, 2560] 8.0 us, with columns over the waves 15.7, with four
    // column tiles a wave 8.5; 64 tokens 16.8, 21.0 and 18.9).  A long K of few
    // columns takes eight, where columns are very few with one column tile a wave
    // (16 tokens of [5120, 5120] 8.3 us against 9.7 with four; 32 of [33, 10240]
    // 8.5, 14.5).
    const bool four = !a.grouped && a.places <= 4;
    const long columns = (long)tl.count * ((a.N + 31) / 32);
    if (columns >= 2048) four ? launch_rows<2, 1, 4, 4>(a, tl, st) : launch_rows<2, 1, 4, 16>(a, tl, st);
    else if (a.K >= 4096 && columns <= 64) four ? launch_rows<1, 8, 1, 4>(a, tl, st) : launch_rows<1, 8, 1, 16>(a, tl, st);
    else if (a.K >= 4096 && columns <= 256) four ? launch_rows<2, 8, 1, 4>(a, tl, st) : launch_rows<2, 8, 1, 16>(a, tl, st);
    else four ? launch_rows<2, 4, 1, 4>(a, tl, st) : launch_rows<2, 4, 1, 16>(a, tl, st);
    return hipGetLastError();
}

}  // namespace moe
