// Rules on the logits of a decoding step (penalties for repeated tokens,
// biases, temperature, grammar masks), one pass over the rows:
//   v in the history:  l = l > 0 ? l / repetition : l * repetition
//   c > 0:             l = l - (frequency c + presence)
//   v has a bias:      l = l + bias
//   temperature > 0:   l = l / temperature
//   mask bit clear:    l = -inf
// with c the count of v behind the prompt; fp32, one rounding at the store.
//
// A workgroup takes a slab of kSlab consecutive tokens of one row.  The
// slab's logits go to registers first, and while they are on their way the
// workgroup reads the row's whole history and counts, in LDS, the tokens that
// fall into its slab.  Counts are integers, so the order of the LDS atomics
// does not show; nothing is kept in global memory, so there is no workspace
// and nothing to clear.
#include "common.h"

namespace moe {

namespace {

constexpr int kLgThreads = 1024;
constexpr int kLgPer = 8;                          // logits per thread
constexpr int kSlab = kLgThreads * kLgPer;         // tokens per workgroup
constexpr uint32_t kSeen = 0x80000000u;            // counter bit: in the prompt

template <int TYPE>
__device__ __forceinline__ void load8(const void *p, size_t i, int left, bool vec, float (&v)[kLgPer])
{
    if (vec && left >= kLgPer) {
#pragma unroll
        for (int q = 0; q < kLgPer / 4; ++q) {
            const float4 f = load_typed4(p, TYPE, i + 4 * q);
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kLgPer; ++j) v[j] = j < left ? load_typed(p, TYPE, i + j) : 0.f;
}

template <int TYPE>
__device__ __forceinline__ void store8(void *p, size_t i, int left, bool vec, const float (&v)[kLgPer])
{
    if (vec && left >= kLgPer) {
#pragma unroll
        for (int q = 0; q < kLgPer / 4; ++q)
            store_typed4(p, TYPE, i + 4 * q, make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < kLgPer; ++j)
        if (j < left) store_typed(p, TYPE, i + j, v[j]);
}

template <int TIN, int TOUT>
__global__ __launch_bounds__(kLgThreads) void logits_kernel(LogitsArgs a, int slabs, bool vec_in, bool vec_out)
{
    __shared__ uint32_t s_n[kSlab];
    const int row = blockIdx.x / slabs, v0 = (blockIdx.x % slabs) * kSlab;
    const int tid = threadIdx.x, mine = v0 + tid * kLgPer, left = a.vocab - mine;
    const uint32_t span = (uint32_t)min(kSlab, a.vocab - v0);

    float l[kLgPer];
    load8<TIN>(a.logits, row * a.logits_stride + mine, left, vec_in, l);
    uint32_t allowed = 0xFFu;   // bit j: token mine + j
    if (a.mask && left > 0) allowed = a.mask[row * a.mask_stride + (mine >> 5)] >> (mine & 31);

    // ---- repeated tokens ----
    const int hist = a.history_width ? (a.history_lengths ? min(max(a.history_lengths[row], 0), a.history_width)
                                                          : a.history_width) : 0;
    if (hist > 0) {
        const int prompt = a.prompt_lengths ? min(max(a.prompt_lengths[row], 0), hist) : 0;
#pragma unroll
        for (int j = 0; j < kLgPer; ++j) s_n[tid + j * kLgThreads] = 0u;
        __syncthreads();
        const int32_t *h = a.history + row * a.history_stride;
        for (int i = tid; i < hist; i += kLgThreads) {
            const uint32_t at = (uint32_t)h[i] - (uint32_t)v0;
            if (at < span) {
                if (i < prompt) atomicOr(&s_n[at], kSeen);
                else atomicAdd(&s_n[at], 1u);
            }
        }
        __syncthreads();
        const float rep = a.repetition ? a.repetition[row] : 1.f;
        const float freq = a.frequency ? a.frequency[row] : 0.f, pres = a.presence ? a.presence[row] : 0.f;
#pragma unroll
        for (int j = 0; j < kLgPer; ++j) {
            const uint32_t n = s_n[tid * kLgPer + j], c = n & ~kSeen;
            if (n) l[j] = l[j] > 0.f ? l[j] / rep : l[j] * rep;
            if (c) l[j] -= freq * (float)c + pres;
        }
        __syncthreads();
    }

    // ---- biases: the last entry of a token holds ----
    const int nb = a.bias_width ? (a.bias_lengths ? min(max(a.bias_lengths[row], 0), a.bias_width)
                                                  : a.bias_width) : 0;
    if (nb > 0) {
#pragma unroll
        for (int j = 0; j < kLgPer; ++j) s_n[tid + j * kLgThreads] = 0u;
        __syncthreads();
        const int32_t *ids = a.bias_ids + row * a.bias_stride;
        for (int i = tid; i < nb; i += kLgThreads) {
            const uint32_t at = (uint32_t)ids[i] - (uint32_t)v0;
            if (at < span) atomicMax(&s_n[at], (uint32_t)i + 1u);
        }
        __syncthreads();
        const float *values = a.bias_values + row * a.bias_stride;
#pragma unroll
        for (int j = 0; j < kLgPer; ++j) {
            const uint32_t n = s_n[tid * kLgPer + j];
            if (n) l[j] += values[n - 1];
        }
    }

    const float t = a.temperature ? a.temperature[row] : 1.f;
#pragma unroll
    for (int j = 0; j < kLgPer; ++j) {
        if (t > 0.f) l[j] /= t;
        if (!((allowed >> j) & 1u)) l[j] = -__builtin_inff();
    }
    store8<TOUT>(a.out, row * a.out_stride + mine, left, vec_out, l);
}

template <int TIN>
void launch_out(const LogitsArgs &a, int out_type, unsigned grid, int slabs, bool vi, bool vo, hipStream_t st)
{
    switch (out_type) {
    case kBf16: logits_kernel<TIN, kBf16><<<grid, kLgThreads, 0, st>>>(a, slabs, vi, vo); break;
    case kF16: logits_kernel<TIN, kF16><<<grid, kLgThreads, 0, st>>>(a, slabs, vi, vo); break;
    default: logits_kernel<TIN, kF32><<<grid, kLgThreads, 0, st>>>(a, slabs, vi, vo); break;
    }
}

// Whether four elements at a multiple of four of every row are aligned.
bool rows_aligned4(const void *p, size_t stride, int rows, int type)
{
    return (uintptr_t)p % (4 * type_bytes(type)) == 0 && (rows == 1 || stride % 4 == 0);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs &a, int in_type, int out_type, hipStream_t st)
{
    const int slabs = (a.vocab + kSlab - 1) / kSlab;
    const unsigned grid = (unsigned)slabs * (unsigned)a.rows;
    const bool vi = rows_aligned4(a.logits, a.logits_stride, a.rows, in_type);
    const bool vo = rows_aligned4(a.out, a.out_stride, a.rows, out_type);
    switch (in_type) {
    case kBf16: launch_out<kBf16>(a, out_type, grid, slabs, vi, vo, st); break;
    case kF16: launch_out<kF16>(a, out_type, grid, slabs, vi, vo, st); break;
    default: launch_out<kF32>(a, out_type, grid, slabs, vi, vo, st); break;
    }
    return hipGetLastError();
}

}  // namespace moe
