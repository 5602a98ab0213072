// Verification of drafted tokens: softmax of target and draft rows, acceptance
// by given random numbers, and the next token from what the target has over the
// draft.
//
// Three launches over slabs of the vocabulary: each slab's largest logit, its
// first place and the sum of exponentials relative to it, for all rows; each
// sequence's decision, and by slabs the mass of its next token's distribution;
// the slab and the token that the pick falls on.  Probabilities and sums are in
// 64 bits: among 10^5 tokens a pick falls within fp32's error of some border
// about once in a hundred.
#include "common.h"

namespace moe {

namespace {

constexpr int kSlab = 8192, kThreads = 256;

// What a slab of a row leaves: its largest logit (-infinity: none) and the first
// place of it, and the sum of exp(l - largest).
struct Part {
    double sum;
    float top;
    int32_t at;
};

// exp(l - top), with +infinities sharing the probability.
__device__ __forceinline__ double term(float l, double top)
{
    if (!(l > -INFINITY)) return 0.0;   // NaN too
    const double d = (double)l - top;
    return (double)l == top ? 1.0 : exp(d);
}

__device__ __forceinline__ void larger(float &top, int &at, float other, int place)
{
    if (other > top || (other == top && place < at)) {
        top = other;
        at = place;
    }
}

// Sum over the workgroup, in a fixed order.
__device__ __forceinline__ double block_sum(double v, double *s)
{
#pragma unroll
    for (int off = 32; off; off >>= 1) v += __shfl_xor(v, off, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < kThreads / 64; ++w) v += s[w];
    return v;
}

__global__ __launch_bounds__(kThreads) void verify_stats_kernel(VerifyArgs a, int slabs, Part *parts)
{
    __shared__ double s_sum[4];
    __shared__ float s_top[4];
    __shared__ int s_at[4];
    const int row = blockIdx.x / slabs, slab = blockIdx.x - row * slabs;
    const int targets = a.seqs * (a.width + 1);
    const bool t = row < targets;
    const char *p = static_cast<const char *>(t ? a.target : a.draft);
    const int type = t ? a.target_type : a.draft_type;
    p += (t ? row * a.target_stride : (row - targets) * a.draft_stride) * type_bytes(type);
    const int v0 = slab * kSlab, v1 = min(a.vocab, v0 + kSlab);
    float top = -INFINITY;
    int at = 0x7FFFFFFF;
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
        const float l = load_typed(p, type, v);
        if (l > top) top = l, at = v;
    }
#pragma unroll
    for (int off = 32; off; off >>= 1) larger(top, at, __shfl_xor(top, off, 64), __shfl_xor(at, off, 64));
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top, s_at[threadIdx.x >> 6] = at;
    __syncthreads();
    for (int w = 0; w < kThreads / 64; ++w) larger(top, at, s_top[w], s_at[w]);
    double sum = 0.0;
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) sum += term(load_typed(p, type, v), (double)top);
    sum = block_sum(sum, s_sum);
    if (threadIdx.x == 0) parts[(size_t)row * slabs + slab] = Part{sum, top, at};
}

// A row's largest logit, its place and the sum of its exponentials, from its slabs.
__device__ __forceinline__ Part row_of(const Part *p, int slabs)
{
    Part r{0.0, -INFINITY, 0x7FFFFFFF};
    for (int i = 0; i < slabs; ++i) larger(r.top, r.at, p[i].top, p[i].at);
    for (int i = 0; i < slabs; ++i)
        if (p[i].top > -INFINITY) r.sum += p[i].sum * term(p[i].top, (double)r.top);
    return r;
}

__device__ __forceinline__ double probability(const Part &r, float l)
{
    return r.sum > 0.0 ? term(l, (double)r.top) / r.sum : 0.0;
}

// What a sequence's drafts come to: how many are accepted, and the rows that the
// next token is drawn from.
struct Decision {
    int accepted, drafts;
    bool greedy;
    Part p, q;
};

__device__ __forceinline__ Decision decide(const VerifyArgs &a, const Part *parts, int slabs, int seq)
{
    Decision d{};
    d.drafts = a.lengths ? min(max(a.lengths[seq], 0), a.width) : a.width;
    d.greedy = a.temperature && !(a.temperature[seq] > 0.f);
    const Part *pt = parts + (size_t)seq * (a.width + 1) * slabs;
    const Part *pd = parts + ((size_t)a.seqs * (a.width + 1) + (size_t)seq * a.width) * slabs;
    for (int n = 0;; ++n) {
        d.accepted = n;
        d.p = row_of(pt + (size_t)n * slabs, slabs);
        if (n == d.drafts) return d;
        const int x = a.tokens[seq * a.width + n];
        const bool in = x >= 0 && x < a.vocab;
        if (d.greedy) {
            if (!(d.p.top > -INFINITY) || x != d.p.at) return d;
            continue;
        }
        double px = 0.0, qx = in ? 1.0 : 0.0;
        if (in)
            px = probability(d.p, load_typed(a.target, a.target_type, ((size_t)seq * (a.width + 1) + n) * a.target_stride + x));
        if (a.draft) {
            d.q = row_of(pd + (size_t)n * slabs, slabs);
            if (in)
                qx = probability(d.q, load_typed(a.draft, a.draft_type, ((size_t)seq * a.width + n) * a.draft_stride + x));
        }
        if (!((double)a.coins[seq * a.width + n] * qx < px)) return d;
    }
}

// r of one token.
__device__ __forceinline__ double over(const VerifyArgs &a, const Decision &d, int seq, int v, bool rest)
{
    const double p = probability(d.p, load_typed(a.target, a.target_type, ((size_t)seq * (a.width + 1) + d.accepted) * a.target_stride + v));
    if (d.accepted == d.drafts || !rest) return p;
    double q;
    if (a.draft)
        q = probability(d.q, load_typed(a.draft, a.draft_type, ((size_t)seq * a.width + d.accepted) * a.draft_stride + v));
    else
        q = v == a.tokens[seq * a.width + d.accepted] ? 1.0 : 0.0;
    return fmax(p - q, 0.0);
}

// masses[seq][slab] = {sum of max(0, p - q), sum of p}
__global__ __launch_bounds__(kThreads) void verify_mass_kernel(VerifyArgs a, int slabs, const Part *parts, double2 *masses)
{
    __shared__ double s_sum[4];
    const int seq = blockIdx.x / slabs, slab = blockIdx.x - seq * slabs;
    const Decision d = decide(a, parts, slabs, seq);
    if (d.greedy) return;
    const int v0 = slab * kSlab, v1 = min(a.vocab, v0 + kSlab);
    double r = 0.0, p = 0.0;
    for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
        r += over(a, d, seq, v, true);
        p += over(a, d, seq, v, false);
    }
    r = block_sum(r, s_sum);
    p = block_sum(p, s_sum);
    if (threadIdx.x == 0) masses[(size_t)seq * slabs + slab] = make_double2(r, p);
}

// One workgroup per sequence: the slab of the pick, then its token.
__global__ __launch_bounds__(kThreads) void verify_pick_kernel(VerifyArgs a, int slabs, const Part *parts, const double2 *masses)
{
    __shared__ double s_run[kThreads];
    const int seq = blockIdx.x, tid = threadIdx.x;
    const Decision d = decide(a, parts, slabs, seq);
    int token = -1;
    if (d.greedy) {
        token = d.p.top > -INFINITY ? d.p.at : -1;
    } else if (d.p.sum > 0.0) {
        const double2 *m = masses + (size_t)seq * slabs;
        double total = 0.0, all = 0.0;
        for (int i = 0; i < slabs; ++i) total += m[i].x, all += m[i].y;
        const bool rest = total > 0.0;
        if (!rest) total = all;
        const double mark = (double)a.picks[seq] * total;
        // the first slab whose end passes the mark; the last with any mass, where rounding leaves none
        double before = 0.0, run = 0.0;
        int slab = 0;
        for (int i = 0; i < slabs; ++i) {
            const double w = rest ? m[i].x : m[i].y;
            if (w > 0.0) {
                slab = i, before = run;
                run += w;
                if (run > mark) break;
            }
        }
        // 32 consecutive tokens to a thread
        constexpr int kPer = kSlab / kThreads;
        const int v0 = slab * kSlab + tid * kPer, v1 = min(a.vocab, v0 + kPer);
        double mine = 0.0;
        for (int v = v0; v < v1; ++v) mine += over(a, d, seq, v, rest);
        s_run[tid] = mine;
        __syncthreads();
        run = before;
        for (int i = 0; i < tid; ++i) run += s_run[i];
        int last = -1;
        bool found = false;
        for (int v = v0; v < v1 && !found; ++v) {
            const double w = over(a, d, seq, v, rest);
            if (w > 0.0) {
                run += w;
                last = v;
                found = run > mark;
            }
        }
        // the first found; else the slab's last token with any mass
        __shared__ int s_first, s_last;
        if (tid == 0) s_first = 0x7FFFFFFF, s_last = -1;
        __syncthreads();
        if (found) atomicMin(&s_first, last);
        if (last >= 0) atomicMax(&s_last, last);
        __syncthreads();
        token = s_first != 0x7FFFFFFF ? s_first : s_last;
    }
    for (int i = tid; i <= a.width; i += kThreads)
        a.out_tokens[(size_t)seq * (a.width + 1) + i] = i < d.accepted ? a.tokens[seq * a.width + i] : i == d.accepted ? token : -1;
    if (tid == 0) a.accepted[seq] = d.accepted;
}

int slabs_of(int vocab) { return (vocab + kSlab - 1) / kSlab; }
size_t parts_bytes(int seqs, int width, int vocab)
{
    return (size_t)seqs * (2 * width + 1) * slabs_of(vocab) * sizeof(Part);
}

}  // namespace

size_t verify_workspace(int seqs, int width, int vocab)
{
    return parts_bytes(seqs, width, vocab) + (size_t)seqs * slabs_of(vocab) * sizeof(double2);
}

hipError_t launch_verify(const VerifyArgs &a, void *workspace, hipStream_t st)
{
    const int slabs = slabs_of(a.vocab);
    Part *parts = static_cast<Part *>(workspace);
    double2 *masses = reinterpret_cast<double2 *>(static_cast<char *>(workspace) + parts_bytes(a.seqs, a.width, a.vocab));
    const int rows = a.seqs * (a.draft ? 2 * a.width + 1 : a.width + 1);
    verify_stats_kernel<<<rows * slabs, kThreads, 0, st>>>(a, slabs, parts);
    verify_mass_kernel<<<a.seqs * slabs, kThreads, 0, st>>>(a, slabs, parts, masses);
    verify_pick_kernel<<<a.seqs, kThreads, 0, st>>>(a, slabs, parts, masses);
    return hipGetLastError();
}

}  // namespace moe
