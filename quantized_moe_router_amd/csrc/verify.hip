// Verification of drafted tokens: softmax of target and draft rows, acceptance
// by given random numbers, and the next token from what the target has over the
// draft.
//
// Three launches over slabs of 8192 tokens of the vocabulary, each of a
// workgroup whose threads hold their logits in registers:
//   stats  each slab's largest logit, its first place (greedy sequences) and
//          the sum of exponentials relative to it, for all rows that count;
//   mass   each sequence's decision, from its rows' slabs; where a draft was
//          refused, the mass of max(0, p - q) in each 256 tokens and slab;
//   pick   the slab, the 256 tokens and the token that the pick falls on.
// Behind the last draft the token comes from p itself, whose slabs' masses the
// first launch has left, so the second has nothing to do for such a sequence
// and is left out where there are no drafts at all.
//
// Probabilities and sums are in 64 bits: among 10^5 tokens a pick falls within
// fp32's error of some border about once in a hundred.
//
// What bounds it: 64 sequences with three drafts over 248320 tokens (fp32) take
// 106 to 112 us.  One by one, under a profiler, which parts the launches, the
// first takes 75 (the rows' bytes at the rate of a copy, with the vector ALU busy
// 70 % of the time), the second 30, of which half goes by before a workgroup has
// its sequence's decision, made anew by each of them from a few hundred slabs, and
// the third 11.  One sequence takes 20, so parted 6, 5 and 5 to 8, dependent loads
// all of them; 8 sequences 40, where the bytes take 9: three launches and the
// decisions.  Rows that do not begin on a word of four tokens, and the last slab
// of every row, are loaded token by token (33 sequences of 16-bit rows: 33 us,
// where the bytes take 4).  Every slab's workgroup deciding for itself saves a
// launch; the third reads what the second has decided (28 us for one sequence
// when it decided again).
#include "common.h"

namespace moe {

namespace {

constexpr int kSlab = 8192, kThreads = 256, kWaves = kThreads / 64;
constexpr int kTurns = kSlab / (4 * kThreads);   // of four tokens a thread
constexpr int kChunk = 256;                      // tokens of a wave's turn
constexpr int kChunks = kSlab / kChunk;
constexpr int kMostDrafts = 64;                  // a lane each

// What a slab of a row leaves: its largest logit (-infinity: none) and the first
// place of it, and the sum of exp(l - largest).
struct Part {
    double sum;
    float top;
    int32_t at;
};

// e^d for d <= 0, within 2^-52 of it: 2^k e^r with |r| <= ln 2 / 2.  e^r is 1 + r
// + r^2 g(r), g the polynomial of degree 9 through (e^r - 1 - r) / r^2 at the ten
// Chebyshev nodes of the interval, which leaves 2^-55.8 (the Taylor sum with as
// many terms: 2^-46.7; with two more: 2^-58, at 113 us instead of 108 for 64
// sequences).  Far below, and for a NaN, 0.
__device__ __forceinline__ double exp_below(double d)
{
    d = fmax(d, -2000.0);   // of a NaN, too, the other one
    const double k = rint(d * 1.4426950408889634074);
    // ln 2 as a double with 32 bits, times k exact, and the rest of it
    double r = fma(k, -0x1.62e42fefp-1, d);
    r = fma(k, -0x1.473de6af278edp-34, r);
    double y = 0x1.af389ecfcbdafp-26;
    y = fma(y, r, 0x1.28917c89aa05dp-22);
    y = fma(y, r, 0x1.71de0db2f6ae9p-19);
    y = fma(y, r, 0x1.a019b9149a3cep-16);
    y = fma(y, r, 0x1.a01a01a7c2efep-13);
    y = fma(y, r, 0x1.6c16c17889ef1p-10);
    y = fma(y, r, 0x1.11111111109b5p-7);
    y = fma(y, r, 0x1.5555555553d68p-5);
    y = fma(y, r, 0x1.5555555555556p-3);
    y = fma(y, r, 0.5);
    y = fma(y, r, 1.0);
    y = fma(y, r, 1.0);
    return ldexp(y, (int)k);
}

// exp(l - top), top the largest of its row or slab; +infinities share the
// probability; -infinity and NaN have none.
__device__ __forceinline__ double term(float l, float top)
{
    if (top == INFINITY) return l == INFINITY ? 1.0 : 0.0;
    return exp_below((double)l - (double)top);
}

// Sum over the wave, the same for every lane, in a fixed order.
template <int CTRL>
__device__ __forceinline__ double dpp_move64(double v)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double read_lane64(double v, int l)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum64(double v)
{
    v += dpp_move64<kDppXor1>(v);
    v += dpp_move64<kDppXor2>(v);
    v += dpp_move64<kDppHalfMirror>(v);
    v += dpp_move64<kDppMirror>(v);
    return (read_lane64(v, 0) + read_lane64(v, 16)) + (read_lane64(v, 32) + read_lane64(v, 48));
}

// The workgroup's, for its first thread.
__device__ __forceinline__ double block_sum(double v, double *s)
{
    v = wave_sum64(v);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += s[w];
    return v;
}

// The smallest of a workgroup's ints.
__device__ __forceinline__ int block_min(int v, int *s)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) v = min(v, __shfl_xor(v, off, 64));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v = min(v, s[w]);
    return v;
}

// A row of logits.
struct Row {
    const char *p;
    int type;
};
__device__ __forceinline__ Row target_row(const VerifyArgs &a, int seq, int i)
{
    return {static_cast<const char *>(a.target) + ((size_t)seq * (a.width + 1) + i) * a.target_stride * type_bytes(a.target_type),
            a.target_type};
}
__device__ __forceinline__ Row draft_row(const VerifyArgs &a, int seq, int i)
{
    return {static_cast<const char *>(a.draft) + ((size_t)seq * a.width + i) * a.draft_stride * type_bytes(a.draft_type),
            a.draft_type};
}

// This thread's logits of a slab: four consecutive ones a turn, -infinity
// behind the vocabulary.  All loads are issued before any is used.
template <int TYPE>
__device__ __forceinline__ void load_slab_as(const char *row, int v0, int vocab, float (&l)[kTurns][4])
{
    constexpr int kBytes = TYPE == kF32 ? 4 : 2;
    const int v = v0 + 4 * threadIdx.x;
    if ((uintptr_t)row % (4 * kBytes) == 0 && v0 + kSlab <= vocab) {
        uint32_t w[kTurns][kBytes];
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const void *at = row + (size_t)(v + 4 * kThreads * i) * kBytes;
            if constexpr (TYPE == kF32) {
                const uint4 q = *static_cast<const uint4 *>(at);
                w[i][0] = q.x, w[i][1] = q.y, w[i][2] = q.z, w[i][3] = q.w;
            } else {
                const uint2 q = *static_cast<const uint2 *>(at);
                w[i][0] = q.x, w[i][1] = q.y;
            }
        }
#pragma unroll
        for (int i = 0; i < kTurns; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (TYPE == kF32) l[i][j] = __uint_as_float(w[i][j]);
                else if constexpr (TYPE == kBf16) l[i][j] = j & 1 ? bf16_hi(w[i][j >> 1]) : bf16_lo(w[i][j >> 1]);
                else l[i][j] = (float)__builtin_bit_cast(f16x2_t, w[i][j >> 1])[j & 1];
            }
        return;
    }
    uint32_t w[kTurns][4];
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = min(v + 4 * kThreads * i + j, vocab - 1);
            w[i][j] = TYPE == kF32 ? reinterpret_cast<const uint32_t *>(row)[at] : reinterpret_cast<const uint16_t *>(row)[at];
        }
#pragma unroll
    for (int i = 0; i < kTurns; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f;
            if (TYPE == kF32) f = __uint_as_float(w[i][j]);
            else if (TYPE == kBf16) f = __uint_as_float(w[i][j] << 16);
            else f = (float)__builtin_bit_cast(_Float16, (uint16_t)w[i][j]);
            l[i][j] = v + 4 * kThreads * i + j < vocab ? f : -INFINITY;
        }
}

__device__ __forceinline__ void load_slab(const Row &r, int v0, int vocab, float (&l)[kTurns][4])
{
    if (r.type == kF32) load_slab_as<kF32>(r.p, v0, vocab, l);
    else if (r.type == kBf16) load_slab_as<kBf16>(r.p, v0, vocab, l);
    else load_slab_as<kF16>(r.p, v0, vocab, l);
}

__device__ __forceinline__ int drafts_of(const VerifyArgs &a, int seq)
{
    return a.lengths ? min(max(a.lengths[seq], 0), a.width) : a.width;
}
__device__ __forceinline__ bool greedy(const VerifyArgs &a, int seq)
{
    return a.temperature && !(a.temperature[seq] > 0.f);
}

__global__ __launch_bounds__(kThreads) void verify_stats_kernel(VerifyArgs a, int slabs, Part *parts)
{
    __shared__ double s_sum[kWaves];
    __shared__ float s_top[kWaves];
    __shared__ int s_at[kWaves];
    const int row = blockIdx.x / slabs, slab = blockIdx.x - row * slabs, v0 = slab * kSlab;
    const int targets = a.seqs * (a.width + 1);
    const bool t = row < targets;
    const int seq = t ? row / (a.width + 1) : (row - targets) / a.width;
    const int i = t ? row - seq * (a.width + 1) : row - targets - seq * a.width;
    const Row r = t ? target_row(a, seq, i) : draft_row(a, seq, i);
    const int drafts = drafts_of(a, seq);
    const bool first_only = greedy(a, seq);
    if (t ? i > drafts : i >= drafts || first_only) return;   // a row that no decision looks at
    float l[kTurns][4];
    load_slab(r, v0, a.vocab, l);

    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < kTurns; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, l[k][j]);   // passes over a NaN
#pragma unroll
    for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_top[w]);
    int at = 0x7FFFFFFF;
    double sum = 0.0;
    if (first_only) {
#pragma unroll
        for (int k = kTurns - 1; k >= 0; --k)
#pragma unroll
            for (int j = 3; j >= 0; --j)
                if (l[k][j] == top) at = v0 + 4 * (int)threadIdx.x + 4 * kThreads * k + j;
        at = block_min(at, s_at);
    } else if (top == INFINITY) {
#pragma unroll
        for (int k = 0; k < kTurns; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += l[k][j] == top ? 1.0 : 0.0;
        sum = block_sum(sum, s_sum);
    } else if (top > -INFINITY) {
#pragma unroll
        for (int k = 0; k < kTurns; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += exp_below((double)l[k][j] - (double)top);
        sum = block_sum(sum, s_sum);
    }
    if (threadIdx.x == 0) parts[(size_t)row * slabs + slab] = Part{sum, top, at};
}

// A row's largest logit and the first place of it (greedy), or the sum of its
// exponentials, from its slabs; by one wave.
__device__ __forceinline__ Part row_of(const Part *p, int slabs, bool first_only)
{
    const int lane = threadIdx.x & 63;
    const Part none{0.0, -INFINITY, 0x7FFFFFFF};
    const Part mine = lane < slabs ? p[lane] : none;   // all of them, up to half a million tokens
    Part r = none;
    r.top = mine.top;
    for (int i = lane + 64; i < slabs; i += 64) r.top = fmaxf(r.top, p[i].top);
#pragma unroll
    for (int off = 32; off; off >>= 1) r.top = fmaxf(r.top, __shfl_xor(r.top, off, 64));
    if (!(r.top > -INFINITY)) return r;
    if (first_only) {
        if (mine.top == r.top) r.at = mine.at;
        for (int i = lane + 64; i < slabs; i += 64)
            if (p[i].top == r.top) r.at = min(r.at, p[i].at);
#pragma unroll
        for (int off = 32; off; off >>= 1) r.at = min(r.at, __shfl_xor(r.at, off, 64));
        return r;
    }
    r.sum = mine.sum > 0.0 ? mine.sum * term(mine.top, r.top) : 0.0;
    for (int i = lane + 64; i < slabs; i += 64)
        if (p[i].sum > 0.0) r.sum += p[i].sum * term(p[i].top, r.top);
    r.sum = wave_sum64(r.sum);
    return r;
}

// What a sequence's drafts come to: how many are accepted, and the rows that the
// next token is drawn from.
struct Decision {
    int accepted, drafts;
    bool first_only;   // greedy
    Part p, q;         // of the row behind the accepted drafts; q.sum 0: nothing is taken off
};

__device__ __forceinline__ double probability(const Part &r, float l)
{
    return r.sum > 0.0 ? term(l, r.top) / r.sum : 0.0;
}

struct DecisionSpace {
    Part p[kMostDrafts + 1], q[kMostDrafts];
    int accepted;
};

// By all threads of a workgroup: a wave takes a row at a time, then a lane each
// draft.
__device__ __forceinline__ Decision decide(const VerifyArgs &a, const Part *parts, int slabs, int seq, DecisionSpace &s)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Decision d;
    d.drafts = drafts_of(a, seq);
    d.first_only = greedy(a, seq);
    const bool have_q = a.draft && !d.first_only;
    // this lane's draft and its logits
    int x = -1;
    float lp = -INFINITY, lq = -INFINITY, coin = 0.f;
    if (wave == 0 && lane < d.drafts) {
        x = a.tokens[seq * a.width + lane];
        coin = a.coins[seq * a.width + lane];
        if (x >= 0 && x < a.vocab && !d.first_only) {
            const Row rp = target_row(a, seq, lane);
            lp = load_typed(rp.p, rp.type, x);
            if (have_q) {
                const Row rq = draft_row(a, seq, lane);
                lq = load_typed(rq.p, rq.type, x);
            }
        }
    }
    const Part *pt = parts + (size_t)seq * (a.width + 1) * slabs;
    const Part *pd = parts + ((size_t)a.seqs * (a.width + 1) + (size_t)seq * a.width) * slabs;
    const int rows = d.drafts + 1 + (have_q ? d.drafts : 0);
    for (int i = wave; i < rows; i += kWaves) {
        const bool t = i <= d.drafts;
        const Part r = row_of(t ? pt + (size_t)i * slabs : pd + (size_t)(i - d.drafts - 1) * slabs, slabs, d.first_only);
        if (lane == 0) (t ? s.p[i] : s.q[i - d.drafts - 1]) = r;
    }
    __syncthreads();
    if (wave == 0) {
        bool good = false;
        if (lane < d.drafts) {
            const Part p = s.p[lane];
            if (d.first_only) {
                good = p.top > -INFINITY && x == p.at;
            } else if (x >= 0 && x < a.vocab) {
                const double qx = a.draft ? probability(s.q[lane], lq) : 1.0;
                good = (double)coin * qx < probability(p, lp);
            }
        }
        const uint64_t bad = ~__ballot(good);   // beyond the drafts, too
        if (lane == 0) s.accepted = bad ? min(d.drafts, __ffsll((unsigned long long)bad) - 1) : d.drafts;
    }
    __syncthreads();
    d.accepted = s.accepted;
    d.p = s.p[d.accepted];
    d.q = Part{0.0, -INFINITY, -1};
    if (d.accepted < d.drafts && !d.first_only) {
        if (a.draft) {
            d.q = s.q[d.accepted];
        } else {   // all of q at the drafted token
            const int at = a.tokens[seq * a.width + d.accepted];
            d.q = Part{at >= 0 && at < a.vocab ? 1.0 : 0.0, -INFINITY, at};
        }
    }
    return d;
}

// p and r = max(0, p - q) of one token.  ip, iq: 1 / sum, or 0.  A quotient is
// a product with them: an ulp more of 64 bits.  Both products are rounded before
// the subtraction: with one of them inside a fused step, equal rows would leave
// the other's rounding error.
__device__ __forceinline__ double token_r(const VerifyArgs &a, const Decision &d, double ip, double iq, int v, float lp, float lq)
{
#pragma clang fp contract(off)
    const double p = term(lp, d.p.top) * ip;
    const double q = a.draft ? term(lq, d.q.top) * iq : (v == d.q.at ? iq : 0.0);
    const double r = p - q;
    return r > 0.0 ? r : 0.0;
}
__device__ __forceinline__ double inverse(double s) { return s > 0.0 ? 1.0 / s : 0.0; }

// The masses of r: chunks[seq][slab][kChunks] and slabs_r[seq][slab].
__global__ __launch_bounds__(kThreads, 4) void verify_mass_kernel(VerifyArgs a, int slabs, const Part *parts, double *chunks, double *slab_r, Decision *decisions)
{
    __shared__ DecisionSpace s;
    __shared__ double s_sum[kWaves];
    const int seq = blockIdx.x / slabs, slab = blockIdx.x - seq * slabs, v0 = slab * kSlab;
    const Decision d = decide(a, parts, slabs, seq, s);
    if (slab == 0 && threadIdx.x == 0) decisions[seq] = d;
    if (d.first_only || !(d.q.sum > 0.0)) return;   // the largest, or p itself
    float lp[kTurns][4], lq[kTurns][4];
    load_slab(target_row(a, seq, d.accepted), v0, a.vocab, lp);
    if (a.draft) load_slab(draft_row(a, seq, d.accepted), v0, a.vocab, lq);
    const double ip = inverse(d.p.sum), iq = inverse(d.q.sum);
    double all = 0.0;
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
        const int v = v0 + 4 * (int)threadIdx.x + 4 * kThreads * k;
        double r = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) r += token_r(a, d, ip, iq, v + j, lp[k][j], a.draft ? lq[k][j] : 0.f);
        r = wave_sum64(r);
        if ((threadIdx.x & 63) == 0) chunks[((size_t)seq * slabs + slab) * kChunks + k * kWaves + (threadIdx.x >> 6)] = r;
        all += r;
    }
    if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) all += s_sum[w];
        slab_r[(size_t)seq * slabs + slab] = all;
    }
}

// The first of `count` masses up to which their sum, with `before`, exceeds
// `mark`; else the last that is not zero (rounding), -1 if all are.  before:
// becomes the sum of those ahead of it.  By one wave, the same for every lane;
// `mine`: the mass of this lane's place in the first 64.
template <class Mass>
__device__ __forceinline__ int find_mass(int count, Mass mass, double mine, double mark, double &before)
{
    const int lane = threadIdx.x & 63;
    double ahead = before, last_ahead = before;
    int last = -1;
    for (int i0 = 0; i0 < count; i0 += 64) {
        const int i = i0 + lane;
        const double m = i0 == 0 ? mine : i < count ? mass(i) : 0.0;
        double run = m;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(run, off, 64);
            if (lane >= off) run += o;
        }
        const double here = __shfl(run, 63, 64);
        run += ahead;
        const uint64_t some = __ballot(m > 0.0), over = __ballot(m > 0.0 && run > mark);
        if (some) {
            const int l = over ? __ffsll((unsigned long long)over) - 1 : 63 - __clzll((long long)some);
            last = i0 + l;
            last_ahead = __shfl(run - m, l, 64);
        }
        if (over) break;
        ahead += here;
    }
    before = last_ahead;
    return last;
}

// One workgroup per sequence; its first wave chooses.
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs a, int slabs, const Part *parts, const double *chunks, const double *slab_r, const Decision *decisions)
{
    __shared__ DecisionSpace s;
    __shared__ double s_chunk[kChunks], s_token[kChunk], s_before, s_mark;
    __shared__ int s_slab, s_place, s_rest;
    const int seq = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Decision d = a.width ? decisions[seq] : decide(a, parts, slabs, seq, s);
    int token = -1;
    if (d.first_only) {
        token = d.p.top > -INFINITY ? d.p.at : -1;
    } else if (d.p.sum > 0.0) {
        const Row rp = target_row(a, seq, d.accepted);
        if (wave == 0) {
            const Part *pt = parts + ((size_t)seq * (a.width + 1) + d.accepted) * slabs;
            const double *mr = slab_r + (size_t)seq * slabs;
            bool rest = d.q.sum > 0.0;
            auto mass = [&](int i) { return rest ? mr[i] : pt[i].sum > 0.0 ? pt[i].sum * term(pt[i].top, d.p.top) : 0.0; };
            double mine, total;
            auto add = [&]() {
                mine = lane < slabs ? mass(lane) : 0.0;
                double all = mine;
                for (int i = lane + 64; i < slabs; i += 64) all += mass(i);
                total = wave_sum64(all);
            };
            add();
            if (rest && !(total > 0.0)) {   // the draft has all that the target has
                rest = false;
                add();
            }
            double before = 0.0;
            const double mark = (double)a.picks[seq] * total;
            const int slab = find_mass(slabs, mass, mine, mark, before);
            if (lane == 0) s_slab = slab, s_before = before, s_mark = mark, s_rest = rest;
        }
        __syncthreads();
        const bool rest = s_rest;
        const int slab = s_slab;
        const double mark = s_mark;
        // (of p the masses are exp(l - top) here, without the division by their sum)
        if (!rest) {
            float lp[kTurns][4];
            load_slab(rp, slab * kSlab, a.vocab, lp);
#pragma unroll
            for (int k = 0; k < kTurns; ++k) {
                double m = 0.0;
#pragma unroll
                for (int j = 0; j < 4; ++j) m += term(lp[k][j], d.p.top);
                m = wave_sum64(m);
                if (lane == 0) s_chunk[k * kWaves + wave] = m;
            }
            __syncthreads();
        }
        double before = s_before;
        if (wave == 0) {
            const double mine = lane >= kChunks ? 0.0 : rest ? chunks[((size_t)seq * slabs + slab) * kChunks + lane] : s_chunk[lane];
            const int chunk = find_mass(kChunks, [](int) { return 0.0; }, mine, mark, before);
            if (lane == 0) s_place = slab * kSlab + chunk * kChunk;
        }
        __syncthreads();
        const int v0 = s_place, v = v0 + tid;
        double m = 0.0;
        if (v < a.vocab) {
            const float lp = load_typed(rp.p, rp.type, v);
            if (rest) {
                float lq = 0.f;
                if (a.draft) {
                    const Row rq = draft_row(a, seq, d.accepted);
                    lq = load_typed(rq.p, rq.type, v);
                }
                m = token_r(a, d, inverse(d.p.sum), inverse(d.q.sum), v, lp, lq);
            } else {
                m = term(lp, d.p.top);
            }
        }
        s_token[tid] = m;
        __syncthreads();
        // (the other waves' `before` is of no use, nor is what they find)
        token = v0 + find_mass(kChunk, [&](int i) { return s_token[i]; }, s_token[lane], mark, before);
    }
    if (wave) return;
    for (int i = lane; i <= a.width; i += 64)
        a.out_tokens[(size_t)seq * (a.width + 1) + i] = i < d.accepted ? a.tokens[seq * a.width + i] : i == d.accepted ? token : -1;
    if (lane == 0) a.accepted[seq] = d.accepted;
}
static_assert(kThreads == kChunk && kChunks <= 64, "a thread for each token of 256, a lane for each 256 of a slab");

int slabs_of(int vocab) { return (vocab + kSlab - 1) / kSlab; }

// Parts of all rows, the masses of chunks and slabs, the decisions; in whole 8-byte words.
struct Space {
    size_t parts, chunks, slab_r, decisions, bytes;
};
Space space_of(int seqs, int width, int vocab)
{
    const size_t slabs = slabs_of(vocab);
    Space s;
    s.parts = 0;
    s.chunks = (size_t)seqs * (2 * width + 1) * slabs * sizeof(Part);
    s.slab_r = s.chunks + (width ? (size_t)seqs * slabs * kChunks * sizeof(double) : 0);
    s.decisions = s.slab_r + (width ? (size_t)seqs * slabs * sizeof(double) : 0);
    s.bytes = s.decisions + (width ? (size_t)seqs * sizeof(Decision) : 0);
    return s;
}

}  // namespace

size_t verify_workspace(int seqs, int width, int vocab) { return space_of(seqs, width, vocab).bytes; }

hipError_t launch_verify(const VerifyArgs &a, void *workspace, hipStream_t st)
{
    const int slabs = slabs_of(a.vocab);
    const Space sp = space_of(a.seqs, a.width, a.vocab);
    char *ws = static_cast<char *>(workspace);
    Part *parts = reinterpret_cast<Part *>(ws + sp.parts);
    double *chunks = reinterpret_cast<double *>(ws + sp.chunks), *slab_r = reinterpret_cast<double *>(ws + sp.slab_r);
    Decision *decisions = reinterpret_cast<Decision *>(ws + sp.decisions);
    const int rows = a.seqs * (a.draft ? 2 * a.width + 1 : a.width + 1);
    verify_stats_kernel<<<rows * slabs, kThreads, 0, st>>>(a, slabs, parts);
    if (a.width) verify_mass_kernel<<<a.seqs * slabs, kThreads, 0, st>>>(a, slabs, parts, chunks, slab_r, decisions);
    verify_pick_kernel<<<a.seqs, kThreads, 0, st>>>(a, slabs, parts, chunks, slab_r, decisions);
    return hipGetLastError();
}

}  // namespace moe
