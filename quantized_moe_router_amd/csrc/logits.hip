// Rules on the logits of a decoding step (penalties for repeated tokens,
// biases, temperature, grammar masks), one pass over the rows:
//   v in the history:  l = l > 0 ? l / repetition : l * repetition
//   c > 0:             l = l - (frequency c + presence)
//   v has a bias:      l = l + bias
//   temperature > 0:   l = l / temperature
//   mask bit clear:    l = -inf
// with c the count of v behind the prompt; fp32, one rounding at the store.
//
// A workgroup takes a slab of consecutive tokens of one row, and counts in LDS
// those tokens of the row's history that fall into its slab, so the row is
// read and written once, nothing is kept in global memory (no workspace,
// nothing to clear) and, counts being integers, the order of the LDS atomics
// does not show.  Every slab reads the whole history, from L2 after the first.
//
// What bounds it: the row's bytes, at the rate of a copy (256 x 248320 bf16
// logits, masked, histories of 1024: 49 us, as long as a copy takes), as long
// as the loads do not wait for each other.  Loads return in order, and one
// under a branch is waited for where the branch ends; so the history's start,
// the biases, the mask and the logits are asked for first of all, in the order
// of their use, without a branch and whatever the row's lengths turn out to be
// (with branches the same call took 63 us).  The temperature is one product
// with its inverse: the quotient's ten instructions cost as much as the rest.
//
// Rows that do not all begin on 16 bytes (8 where a lane's four elements are 16
// bits wide) are taken an element at a time: the logits and out by each lane's
// own 4 or 8 (256 x 50257 bf16 with a mask 33 us, 256 x 50256 16), the history
// without any id on its way while one is counted (2 rows of 248320 with 131071
// ids each 24 us, with 131072 12; where the history is short beside the logits
// it hides: 64 rows with 4097 ids 24, with 4096 22).
#include "common.h"

namespace moe {

namespace {

constexpr uint32_t kSeen = 0x80000000u;            // counter bit: in the prompt

// C consecutive logits (4 or 8) as they lie in memory.
template <int TYPE, int C>
struct __align__(C * (TYPE == kF32 ? 4 : 2) < 16 ? C * (TYPE == kF32 ? 4 : 2) : 16) Raw {
    static constexpr int kWords = C * (TYPE == kF32 ? 4 : 2) / 4;
    uint32_t w[kWords];
};

// Logits v .. v + C - 1 of a row of `vocab`.  The loads are unconditional, at
// places pulled back into the row (what they bring from there is never
// stored): loads under a branch would be waited for where it ends.
template <int TYPE, int C, bool VEC>
__device__ __forceinline__ void load_chunk(const void *row, int v, int vocab, Raw<TYPE, C> &r)
{
    if constexpr (VEC) {   // aligned chunks; vocab is at least C
        constexpr int kBytes = TYPE == kF32 ? 4 : 2;
        const int at = min(v, vocab / C * C - C);
        r = *reinterpret_cast<const Raw<TYPE, C> *>(static_cast<const char *>(row) + (size_t)at * kBytes);
    } else {
        uint32_t e[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int at = min(v + j, vocab - 1);
            e[j] = TYPE == kF32 ? static_cast<const uint32_t *>(row)[at] : static_cast<const uint16_t *>(row)[at];
        }
#pragma unroll
        for (int j = 0; j < Raw<TYPE, C>::kWords; ++j)
            r.w[j] = TYPE == kF32 ? e[j] : e[2 * j % C] | e[2 * j % C + 1] << 16;
    }
}

template <int TYPE, int C>
__device__ __forceinline__ float chunk_value(const Raw<TYPE, C> &r, int j)
{
    if (TYPE == kF32) return __uint_as_float(r.w[j]);
    const uint32_t w = r.w[j / 2];
    if (TYPE == kBf16) return j & 1 ? bf16_hi(w) : bf16_lo(w);
    return (float)__builtin_bit_cast(f16x2_t, w)[j & 1];
}

// Stores a chunk at v of a row of `vocab`, as one word where `vec` allows it.
template <int TYPE, int C>
__device__ __forceinline__ void store_type(void *row, int v, int vocab, bool vec, const float (&l)[C])
{
    if (vec && v + C <= vocab) {
        Raw<TYPE, C> r;
#pragma unroll
        for (int j = 0; j < Raw<TYPE, C>::kWords; ++j) {
            if constexpr (TYPE == kF32) {
                r.w[j] = __float_as_uint(l[j]);
            } else if constexpr (TYPE == kBf16) {
                r.w[j] = f32x2_to_bf16x2(l[2 * j], l[2 * j + 1]);
            } else {
                const f16x2_t h = {(_Float16)l[2 * j], (_Float16)l[2 * j + 1]};
                r.w[j] = __builtin_bit_cast(uint32_t, h);
            }
        }
        *reinterpret_cast<Raw<TYPE, C> *>(static_cast<char *>(row) + (size_t)v * (TYPE == kF32 ? 4 : 2)) = r;
        return;
    }
#pragma unroll
    for (int j = 0; j < C; ++j)
        if (v + j < vocab) store_typed(row, TYPE, v + j, l[j]);
}

template <int C>
__device__ __forceinline__ void store_chunk(void *row, int type, int v, int vocab, bool vec, const float (&l)[C])
{
    if (type == kF32) store_type<kF32, C>(row, v, vocab, vec, l);
    else if (type == kBf16) store_type<kBf16, C>(row, v, vocab, vec, l);
    else store_type<kF16, C>(row, v, vocab, vec, l);
}

// x / d as one product with 1 / d (an ulp more than the quotient, a tenth of
// its instructions), where 1 / d keeps fp32's full precision.
__device__ __forceinline__ bool has_inverse(float d) { return d > 0x1p-100f && d < 0x1p100f; }

constexpr int kAhead = 4;   // groups of four history entries per thread in flight

template <int NT, int CHUNKS, int C, int TIN, bool VEC, bool LONG>
__global__ __launch_bounds__(NT) void logits_kernel(LogitsArgs a, int slabs, int out_type, bool vec_out, bool vec_hist)
{
    constexpr int kStep = NT * C, kSlab = kStep * CHUNKS;
    __shared__ __align__(16) uint32_t s_n[kSlab];   // counts behind the prompt and kSeen; then bias entries
    const int row = blockIdx.x / slabs, v0 = (blockIdx.x % slabs) * kSlab;
    const int tid = threadIdx.x;
    const uint32_t span = (uint32_t)min(kSlab, a.vocab - v0);

    // ---- every load that depends on nothing, in the order of its use (loads
    // return in order): the start of the history and of the biases, whatever
    // the row's lengths, then the mask and the logits ----
    const int32_t *h = a.history + row * a.history_stride;
    constexpr int kTurn = kAhead * NT;
    const int groups = vec_hist ? a.history_width / 4 : 0;   // whole groups of four
    int4 ahead[kAhead];
    auto fetch = [&](int4 (&to)[kAhead], int g0) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            to[u] = *reinterpret_cast<const int4 *>(reinterpret_cast<const char *>(h) +
                                                    16u * (uint32_t)min(g0 + tid + u * NT, groups - 1));
    };
    if (groups > 0) fetch(ahead, 0);
    const int32_t *ids = a.bias_ids + row * a.bias_stride;
    int32_t first_id = 0;
    float first_value = 0.f;
    if (a.bias_width > 0) {
        first_id = ids[min(tid, a.bias_width - 1)];
        first_value = (a.bias_values + row * a.bias_stride)[min(tid, a.bias_width - 1)];
    }

    uint32_t allowed[CHUNKS];   // bit j: token j of the chunk
#pragma unroll
    for (int q = 0; q < CHUNKS; ++q) allowed[q] = ~0u;
    if (a.mask) {
        const uint32_t *mask = a.mask + row * a.mask_stride;
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            const int v = min(v0 + q * kStep + tid * C, a.vocab - 1);
            allowed[q] = mask[v >> 5] >> (v & (32 - C));
        }
    }
    const char *in = static_cast<const char *>(a.logits) + row * a.logits_stride * (TIN == kF32 ? 4 : 2);
    Raw<TIN, C> raw[CHUNKS];
#pragma unroll
    for (int q = 0; q < CHUNKS; ++q) load_chunk<TIN, C, VEC>(in, v0 + q * kStep + tid * C, a.vocab, raw[q]);
    if (VEC && span < (uint32_t)kSlab && a.vocab % C) {   // the row's last, partial chunk
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            const int v = v0 + q * kStep + tid * C;
            if (v < a.vocab && v + C > a.vocab) load_chunk<TIN, C, false>(in, v, a.vocab, raw[q]);
        }
    }

    // ---- the row's numbers ----
    int hist = a.history_width, prompt = 0, nb = a.bias_width;
    float rep = 1.f, freq = 0.f, pres = 0.f, t = 1.f;
    if (a.history_lengths) hist = a.history_lengths[row];
    if (a.prompt_lengths) prompt = a.prompt_lengths[row];
    if (a.bias_lengths) nb = a.bias_lengths[row];
    if (a.repetition) rep = a.repetition[row];
    if (a.frequency) freq = a.frequency[row];
    if (a.presence) pres = a.presence[row];
    if (a.temperature) t = a.temperature[row];
    hist = min(max(hist, 0), a.history_width);
    prompt = min(max(prompt, 0), hist);
    nb = min(max(nb, 0), a.bias_width);

    // this thread's own counters, read and cleared for what comes next
    uint4 *own = reinterpret_cast<uint4 *>(s_n) + tid * (C / 4);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto take = [&](int q, uint32_t (&n)[C]) {
#pragma unroll
        for (int c = 0; c < C / 4; ++c) {
            const uint4 w = own[q * (kStep / 4) + c];
            if (nb > 0) own[q * (kStep / 4) + c] = zero;
            n[4 * c] = w.x, n[4 * c + 1] = w.y, n[4 * c + 2] = w.z, n[4 * c + 3] = w.w;
        }
    };
    if (hist > 0 || nb > 0) {
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q)
#pragma unroll
            for (int c = 0; c < C / 4; ++c) own[q * (kStep / 4) + c] = zero;
        __syncthreads();
    }

    // ---- repeated tokens: count those of the slab ----
    if (hist > 0) {
        auto one = [&](int i, int32_t id) {
            const uint32_t at = (uint32_t)id - (uint32_t)v0;
            if (at < span && i < hist) {
                if (i < prompt) atomicOr(&s_n[at], kSeen);
                else atomicAdd(&s_n[at], 1u);
            }
        };
        // the groups from g0 on, kAhead per thread
        auto count = [&](const int4 (&now)[kAhead], int g0) {
            // all of it prompt, all of it behind the prompt, or something of both
            const int g1 = g0 + kTurn;
            const bool all_prompt = 4 * g1 <= prompt, all_after = 4 * g0 >= prompt && 4 * g1 <= min(hist, 4 * groups);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int32_t id[4] = {now[u].x, now[u].y, now[u].z, now[u].w};
                const int g = g0 + tid + u * NT;
                if (all_prompt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((uint32_t)id[e] - (uint32_t)v0 < span) atomicOr(&s_n[id[e] - v0], kSeen);
                } else if (all_after) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((uint32_t)id[e] - (uint32_t)v0 < span) atomicAdd(&s_n[id[e] - v0], 1u);
                } else if (g < groups) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) one(4 * g + e, id[e]);
                }
            }
        };
        auto more = [&](int g0) { return g0 < groups && 4 * g0 < hist; };
        if constexpr (LONG) {
            // the next groups are on their way while these are counted; two
            // buffers by name, for moving one into the other took as many
            // vector instructions as the counting (a million ids: 56 us
            // against 63)
            int4 next[kAhead];
            for (int g0 = 0; more(g0); g0 += 2 * kTurn) {
                fetch(next, g0 + kTurn);
                count(ahead, g0);
                if (!more(g0 + kTurn)) break;
                fetch(ahead, g0 + 2 * kTurn);
                count(next, g0 + kTurn);
            }
        } else {
            for (int g0 = 0; more(g0); g0 += kTurn) {
                if (g0 > 0) fetch(ahead, g0);
                count(ahead, g0);
            }
        }
        for (int i = 4 * groups + tid; i < hist; i += NT) one(i, h[i]);   // behind the groups
        __syncthreads();
    }

    float l[CHUNKS][C];
#pragma unroll
    for (int q = 0; q < CHUNKS; ++q)
#pragma unroll
        for (int j = 0; j < C; ++j) l[q][j] = chunk_value<TIN, C>(raw[q], j);
    if (hist > 0) {
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            uint32_t n[C];
            take(q, n);
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (n[j]) {   // few tokens of a slab
                    float &x = l[q][j];
                    x = x > 0.f ? x / rep : x * rep;
                    const uint32_t c = n[j] & ~kSeen;
                    if (c) x -= freq * (float)c + pres;
                }
        }
        if (nb > 0) __syncthreads();
    }

    // ---- biases: the last entry of a token holds.  Its place in the list
    // is found first, then its value takes that place (a bias of zero leaves
    // a clear word, and changes nothing) ----
    if (nb > 0) {
        auto each = [&](auto &&f) {
            for (int i = tid; i < nb; i += NT) {
                const uint32_t at = (uint32_t)(i < NT ? first_id : ids[i]) - (uint32_t)v0;
                if (at < span) f(i, &s_n[at]);
            }
        };
        each([&](int i, uint32_t *w) { atomicMax(w, (uint32_t)i + 1u); });
        __syncthreads();
        const float *values = a.bias_values + row * a.bias_stride;
        each([&](int i, uint32_t *w) {
            if (*w != (uint32_t)i + 1u) return;
            // a value whose bits could be taken for a place (at most 2^24: 2^-125) is zero
            const uint32_t bits = __float_as_uint(i < NT ? first_value : values[i]);
            *w = bits <= (1u << 24) ? 0u : bits;
        });
        __syncthreads();
#pragma unroll
        for (int q = 0; q < CHUNKS; ++q) {
            uint32_t n[C];
            take(q, n);
#pragma unroll
            for (int j = 0; j < C; ++j) l[q][j] += __uint_as_float(n[j]);
        }
    }

    const bool inverse = has_inverse(t);
    const float it = inverse ? 1.f / t : 1.f;
    char *out = static_cast<char *>(a.out) + row * a.out_stride * type_bytes(out_type);
#pragma unroll
    for (int q = 0; q < CHUNKS; ++q) {
        const int v = v0 + q * kStep + tid * C;
        if (!inverse && t > 0.f) {
#pragma unroll
            for (int j = 0; j < C; ++j) l[q][j] /= t;
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) l[q][j] *= it;
        }
#pragma unroll
        for (int j = 0; j < C; ++j) {
            // all ones where the bit is set: the logit, else -infinity
            const uint32_t m = (uint32_t)((int32_t)(allowed[q] << (31 - j)) >> 31);
            l[q][j] = __uint_as_float((__float_as_uint(l[q][j]) & m) | (0xFF800000u & ~m));
        }
        store_chunk(out, out_type, v, a.vocab, vec_out, l[q]);
    }
}

// Whether chunks of `per` elements at multiples of `per` in every row are
// aligned to 16 bytes, or to their size where that is less.
bool rows_aligned(const void *p, size_t stride, int rows, int type, int per)
{
    const int bytes = per * type_bytes(type), word = bytes < 16 ? bytes : 16;
    return (uintptr_t)p % word == 0 && (rows == 1 || stride * type_bytes(type) % word == 0);
}

template <int NT, int PER, int C, int TIN, bool LONG>
void launch_shape(const LogitsArgs &a, int out_type, hipStream_t st)
{
    const int slab = NT * PER, slabs = (a.vocab + slab - 1) / slab;
    const unsigned grid = (unsigned)slabs * (unsigned)a.rows;
    const bool vo = rows_aligned(a.out, a.out_stride, a.rows, out_type, C);
    const bool vh = rows_aligned(a.history, a.history_stride, a.rows, kF32, 4);
    if (a.vocab >= C && rows_aligned(a.logits, a.logits_stride, a.rows, TIN, C))
        logits_kernel<NT, PER / C, C, TIN, true, LONG><<<grid, NT, 0, st>>>(a, slabs, out_type, vo, vh);
    else
        logits_kernel<NT, PER / C, C, TIN, false, LONG><<<grid, NT, 0, st>>>(a, slabs, out_type, vo, vh);
}

template <int C, int TIN>
void launch_in(const LogitsArgs &a, int out_type, hipStream_t st)
{
    // Slabs of 8192 by workgroups of 512, four to a CU, once they fill the
    // chip: at 64 x 248320 logits (bf16 to fp32, a history of 512) 21.7 us,
    // against 22.6 with 256 threads and slabs of 2048, and 29.0 against 45.3
    // with histories of 16384, which a smaller slab scans more often.
    if ((long)a.rows * ((a.vocab + 8191) / 8192) > 512) launch_shape<512, 16, C, TIN, false>(a, out_type, st);
    // Below that, small workgroups start and end soonest (one row of 248320
    // and a history of 512: 3.8 us against 5.4), but every workgroup scans the
    // whole history, so for wide tables it gets all the threads it can have
    // (one row, a history of 131072: 11.5 us against 21), with one chunk each
    // where that takes no more workgroups than CUs (fp32: 10.7; two to a CU
    // share its issue slots, 8 rows take 18.8 against 14.2).
    else if (a.history_width > 8192 && (long)a.rows * ((a.vocab + 1024 * C - 1) / (1024 * C)) <= 256)
        launch_shape<1024, C, C, TIN, true>(a, out_type, st);
    else if (a.history_width > 8192) launch_shape<1024, 8, C, TIN, true>(a, out_type, st);
    else launch_shape<256, 8, C, TIN, false>(a, out_type, st);
}

}  // namespace

hipError_t launch_logits(const LogitsArgs &a, int in_type, int out_type, hipStream_t st)
{
    // Eight at a time where both sides are 16 bits wide; with fp32 on a side,
    // four, so that the lanes of one store (or load) cover whole lines.
    const bool narrow = out_type != kF32;
    if (in_type == kF32) launch_in<4, kF32>(a, out_type, st);
    else if (in_type == kBf16) narrow ? launch_in<8, kBf16>(a, out_type, st) : launch_in<4, kBf16>(a, out_type, st);
    else narrow ? launch_in<8, kF16>(a, out_type, st) : launch_in<4, kF16>(a, out_type, st);
    return hipGetLastError();
}

}  // namespace moe
