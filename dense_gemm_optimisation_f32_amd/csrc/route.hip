// route.hip -- routing of tokens to experts: scores, the choice of k experts per
// token, their weights, the rows sorted by expert; its gradient; the weighted
// sum of the experts' rows back to tokens and its gradient.
//
// Figures below are of one MI355X, kernel times from a tracer unless said otherwise.
#include "routed_internal.h"
#include "epilogue.h"
#include "wave.h"

#include <type_traits>

namespace mi355gemm {
namespace {

// A choice score as an unsigned key that orders like it: larger scores larger
// keys, NaN below every number; 0 is left for an expert that cannot be chosen.
constexpr uint64_t kNanKey = 1ull << 32;
__device__ __forceinline__ uint64_t score_key(double c)
{
    if (c != c) return kNanKey;
    const uint64_t b = __builtin_bit_cast(uint64_t, c);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t logit_key(float c)
{
    if (c != c) return kNanKey;
    const unsigned b = __builtin_bit_cast(unsigned, c + 0.f);   // (-0 counts as 0)
    return (uint64_t)((b >> 31) ? ~b : (b | 0x80000000u)) << 32;
}

__device__ __forceinline__ unsigned max_u(unsigned a, unsigned b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned min_u(unsigned a, unsigned b) { return a < b ? a : b; }

// A lane's NE keys in descending order: bitonic merges of runs of w into runs of
// 2w, the second run read backwards.
template <int NE, class K>
__device__ __forceinline__ void sort_keys(K *key)
{
#pragma unroll
    for (int w = 1; w < NE; w <<= 1)
#pragma unroll
        for (int d = w; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int o = d == w ? (i / (2 * w)) * 2 * w + (2 * w - 1 - i % (2 * w)) : i ^ d;
                if (o > i) {
                    const K u = key[i], v = key[o];
                    key[i] = u > v ? u : v;
                    key[o] = u > v ? v : u;
                }
            }
}

// The same with each key's place, at[i] = 0 .. NE-1, equal keys in the order of their places.
template <int NE>
__device__ __forceinline__ void sort_placed(uint64_t *key, int *at)
{
#pragma unroll
    for (int w = 1; w < NE; w <<= 1)
#pragma unroll
        for (int d = w; d > 0; d >>= 1)
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int o = d == w ? (i / (2 * w)) * 2 * w + (2 * w - 1 - i % (2 * w)) : i ^ d;
                if (o > i) {
                    const uint64_t u = key[i], v = key[o];
                    const int a = at[i], b = at[o];
                    const bool first = u > v || (u == v && a < b);
                    key[i] = first ? u : v;
                    key[o] = first ? v : u;
                    at[i] = first ? a : b;
                    at[o] = first ? b : a;
                }
            }
}

// v[i] = row[lane*NE + i], `none` from E on: 16-byte loads where all four are inside.
template <int NE>
__device__ __forceinline__ void load_experts(const float *row, int lane, int E, float none, float *v)
{
    const int e0 = lane * NE;
    if constexpr (NE % 4 == 0) {
        if (e0 + NE <= E) {
#pragma unroll
            for (int i = 0; i < NE; i += 4) {
                const f32x4_t q = *reinterpret_cast<const f32x4_g *>(row + e0 + i);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i + j] = q[j];
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = e0 + i < E ? row[e0 + i] : none;
}

// ---------------------------------------------------------------- routing
//
// A block takes `chunk` consecutive tokens, a wave one token at a time; lane l
// holds experts l*NE .. l*NE + NE-1.
//   choose: choice scores are formed and compared in 64 bits, since neighbouring
//     scores of a token are often nearer than 32 bits can tell and the choice is
//     a whole number that is either right or not.  A score becomes a 64-bit key of all its
//     bits, which a lane sorts together with the experts' places, so that equal scores come in
//     the order of the experts.  A round of the choice is a maximum of the lanes' upper words;
//     the lower words are looked at only where two lanes tie.  Where the logits order the
//     experts like the scores (BY_LOGIT: no bias, a group's best score alone) no score is
//     formed, and a key is a logit's 32 bits with the place in the lowest log2(NE) below them.
//   layout: choices are numbered by expert in token order: within 64 choices by
//     comparing ids over the wave, across the block's (at most kSegments) runs of
//     64 by a prefix over their counts, so the order never depends on timing.
//     With one block the counts are scanned here; otherwise they go to `counts`
//     and place_kernel turns local numbers into rows.
// Where scores are needed, 32 bits decide first (choose32): scores between -3.9 and 3.9
// as whole numbers of 2^-27, and a choice stands if every decision in it (a group
// kept or not, a choice before the next) is by more than the errors of what it compares;
// else the token is done again in 64 bits.  With scores of some hundred experts spread over a
// unit a few tokens in a thousand are.  With groups of experts that are not 1, 2, 4, 8 or 16 whole lanes
// (lanes_per_group = 0: 160 experts in 8 groups) every token is, after its 32-bit scores were formed.
// Bound by instructions, not by its reads: 32768 tokens of 256 experts (the best 4 of 8 groups, 8 choices, bias,
// sigmoid) take 40 us, vector instructions on 67% of the cycles; their 33.6 MB are 7.1 us at a copy's rate.  Of a
// call without the layout, 36 us, a round of the choice takes 2 each, the groups 6, loads, scores, sort and
// weights 14.  Two waves per SIMD for every one (64 registers) gave 39 us against 41 and a longer prefix.  16
// tokens: 8.4 us, one token's chain of dependent steps, then a layout that clears and scans 16 runs of
// choices where these fill two.
// log2(e) as a 32-bit value and what that leaves out, ln(2)
constexpr float kLog2e = 1.4426950408889634, kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e), kLn2 = 0.6931471805599453;
// e^(x + low) for |x| <= 200 and a low of some u |x| (below 2^-126: 0): the exponential instruction on the rounded
// x log2(e), and what that rounding left out, with low, to first order; off by 3 u.  (The library's function takes about
// twice the instructions.)
__device__ __forceinline__ float exp_of(float x, float low = 0.f)
{
    const float p = x * kLog2e, left = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -p));
    const float e = __builtin_amdgcn_exp2f(p);
    return __builtin_fmaf(e, __builtin_fmaf(left, kLn2, low), e);
}
constexpr float kUnits = 1 << 27, kZero = 4.f * (1 << 27);   // key = score * kUnits + kZero; 0: unavailable
// Error of a key: exp, sum and quotient 4e-6, the rounding of score + 4 2.4e-7, the place of
// the expert in the lowest 4 bits 1.2e-7; together below 2^-17.
constexpr unsigned kNear = 1 << 10;

// The k choices (lane j's is `mine`), or false.  x: logits, b: biases (-inf: unavailable).
template <int NE>
__device__ __forceinline__ bool choose32(const RouteProblem &p, const float *x, const float *b, float mx, int lane,
                                         int lanes_per_group, int *mine)
{
    float s[NE];
    if (p.score == 0) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = __builtin_amdgcn_exp2f((x[i] - mx) * kLog2e);
            sum += s[i];
        }
        sum = __builtin_amdgcn_rcpf(wave_sum(sum));
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] *= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x[i] * kLog2e));
    }
    unsigned key[NE];
    bool odd = false;   // a score that this path does not take
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const float c = s[i] + b[i];
        const bool gone = x[i] == -INFINITY || b[i] == -INFINITY;
        odd |= !gone && !(fabsf(c) < 3.9f);
        key[i] = gone ? 0u : ((unsigned)__builtin_fmaf(c, kUnits, kZero) & ~(unsigned)(NE - 1)) | (NE - 1 - i);
    }
    if (__ballot(odd)) return false;
    sort_keys<NE>(key);
    if (p.groups > 1) {
        if (lanes_per_group == 0) return false;
        // the group's two best keys by exchanges between its lanes
        unsigned k1 = key[0], k2 = NE > 1 ? key[NE > 1 ? 1 : 0] : 0u;
        auto merge = [&](unsigned o1, unsigned o2) {
            k2 = max_u(min_u(k1, o1), max_u(k2, o2));
            k1 = max_u(k1, o1);
        };
        if (lanes_per_group > 1) merge(dpp<0xB1, 0xF>(0u, k1), dpp<0xB1, 0xF>(0u, k2));     // lane ^ 1
        if (lanes_per_group > 2) merge(dpp<0x4E, 0xF>(0u, k1), dpp<0x4E, 0xF>(0u, k2));     // lane ^ 2
        if (lanes_per_group > 4) merge(dpp<0x141, 0xF>(0u, k1), dpp<0x141, 0xF>(0u, k2));   // mirrored in 8
        if (lanes_per_group > 8) merge(dpp<0x140, 0xF>(0u, k1), dpp<0x140, 0xF>(0u, k2));   // mirrored in 16
        // two keys' sum below 2^31; a lone one's other half is the score 0
        int score = (int)k1;
        if (p.group_top == 2) score = k1 == 0 ? 0 : (int)k1 + (int)(k2 == 0 ? (unsigned)kZero : k2);
        int surely = 0, maybe = 0;   // groups that come before this lane's
        for (int g = 0; g < p.groups; ++g) {
            const int d = (int)lane_value((unsigned)score, g * lanes_per_group) - score;
            surely += d > (int)(4 * kNear);
            maybe += d > -(int)(4 * kNear);
        }
        const bool kept = maybe - 1 < p.group_k;   // (its own group counts once)
        if (__ballot(lane < p.groups * lanes_per_group && !kept && surely < p.group_k)) return false;
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = kept ? key[i] : 0u;
    }
    unsigned gap = ~0u, last = ~0u;
    uint64_t twice = 0;   // two lanes' keys were equal
    unsigned top = wave_max(key[0]);
    for (int j = 0; j < p.k && top != 0; ++j) {
        gap = min_u(gap, last - top);
        last = top;
        const bool won = key[0] == top;
        const uint64_t at = __ballot(won);
        twice |= at & (at - 1);
        const int win = __builtin_ctzll(at);
        const int e = win * NE + (NE - 1 - (int)(top & (NE - 1)));
        *mine = lane == j ? e : *mine;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const unsigned here = key[i], next = i + 1 < NE ? key[i + 1 < NE ? i + 1 : i] : 0u;   // (values, not places, to choose from)
            key[i] = won ? next : here;
        }
        top = wave_max(key[0]);
    }
    if (top != 0) gap = min_u(gap, last - top);   // the first that is not chosen
    return gap > 2 * kNear && twice == 0;
}

constexpr int kSegments = 16;                  // runs of 64 choices in a block
constexpr int kChunkIds = 64 * kSegments;

template <int NE, int NT, bool BY_LOGIT>
__global__ __launch_bounds__(NT) void route_kernel(RouteProblem p, int chunk, int lanes_per_group)
{
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int T = p.T, E = p.E, k = p.k;
    const int t0 = blockIdx.x * chunk, t1 = t0 + chunk < T ? t0 + chunk : T;
    // group scores of odd sizes (64-bit, one row per wave), later the counts of
    // the runs (16-bit, kSegments rows)
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    __shared__ int cid[kChunkIds];
    __shared__ int total[kMaxExperts + 2];
    double *sc = reinterpret_cast<double *>(smem) + (size_t)wave * E;

    float b[NE];
    if (p.bias)
        load_experts<NE>(p.bias, lane, E, -INFINITY, b);
    else
#pragma unroll
        for (int i = 0; i < NE; ++i) b[i] = 0.f;
    float x[NE], ahead[NE];   // a token's logits are read while the one before it is chosen for
    if (t0 + wave < t1) load_experts<NE>(p.logits + (long long)(t0 + wave) * p.ldl, lane, E, -INFINITY, ahead);
    for (int t = t0 + wave; t < t1; t += NW) {
        const float *row = p.logits + (long long)t * p.ldl;
#pragma unroll
        for (int i = 0; i < NE; ++i) x[i] = ahead[i];
        if (t + NW < t1) load_experts<NE>(row + NW * p.ldl, lane, E, -INFINITY, ahead);
        float mx = -INFINITY;
        bool bad = false;   // a softmax whose scores are NaN: the row holds NaN or +inf
        uint64_t key[NE];
        int at_place[NE];   // of the sorted keys (BY_LOGIT: in the keys)
        if (BY_LOGIT || p.score == 0) {
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                mx = fmaxf(mx, x[i]);
                bad |= x[i] != x[i] || x[i] == INFINITY;
            }
            bad = __ballot(bad) != 0;
            mx = wave_max(mx);
        }
        if constexpr (BY_LOGIT) {
#pragma unroll
            for (int i = 0; i < NE; ++i)
                key[i] = x[i] == -INFINITY ? 0
                         : p.score == 0 && bad ? kNanKey | (NE - 1 - i)
                                               : logit_key(x[i]) | (NE - 1 - i);
        }
        auto sum32 = [&]() {   // the softmax's sum (32 bits: it only scales weights)
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < NE; ++i) v += x[i] == -INFINITY ? 0.f : expf(x[i] - mx);
            return wave_sum(v);
        };
        int mine = -1;   // lane j: choice j
        bool done = false;
        if constexpr (!BY_LOGIT) {
            done = !bad && choose32<NE>(p, x, b, mx, lane, lanes_per_group, &mine);
            if (!done) mine = -1;
        }
        if (!BY_LOGIT && !done) {
            double c[NE];
            if (p.score == 0) {
                double sum = 0.0;
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    c[i] = x[i] == -INFINITY ? 0.0 : exp((double)x[i] - (double)mx);
                    sum += c[i];
                }
                sum = wave_sum(sum);
#pragma unroll
                for (int i = 0; i < NE; ++i) c[i] /= sum;
            } else {
#pragma unroll
                for (int i = 0; i < NE; ++i) c[i] = 1.0 / (1.0 + exp(-(double)x[i]));
            }
            bool nan = false;
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                c[i] += (double)b[i];
                const bool gone = x[i] == -INFINITY || b[i] == -INFINITY;
                key[i] = gone ? 0 : score_key(c[i]);
                at_place[i] = i;
                if (gone) c[i] = -INFINITY;
                nan |= c[i] != c[i];
            }
            if (p.groups > 1) {
                bool kept;
                if (lanes_per_group > 0 && __ballot(nan) == 0) {
                    // a group is 1, 2, 4, 8 or 16 whole lanes: its two best scores by
                    // exchanges between them (-inf: no available expert)
                    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        b2 = fmax(b2, fmin(b1, c[i]));
                        b1 = fmax(b1, c[i]);
                    }
                    auto merge = [&](double o1, double o2) {
                        b2 = fmax(fmin(b1, o1), fmax(b2, o2));
                        b1 = fmax(b1, o1);
                    };
                    if (lanes_per_group > 1) merge(dpp<0xB1, 0xF>(b1, b1), dpp<0xB1, 0xF>(b2, b2));     // lane ^ 1
                    if (lanes_per_group > 2) merge(dpp<0x4E, 0xF>(b1, b1), dpp<0x4E, 0xF>(b2, b2));     // lane ^ 2
                    if (lanes_per_group > 4) merge(dpp<0x141, 0xF>(b1, b1), dpp<0x141, 0xF>(b2, b2));   // mirrored in 8
                    if (lanes_per_group > 8) merge(dpp<0x140, 0xF>(b1, b1), dpp<0x140, 0xF>(b2, b2));   // mirrored in 16
                    const double mine = p.group_top == 2 && b2 != -INFINITY ? b1 + b2 : b1;
                    const int group = lane / lanes_per_group;
                    int before = 0;   // groups that come before this lane's
                    for (int g = 0; g < p.groups; ++g) {
                        const double o = lane_value(mine, g * lanes_per_group);
                        before += o > mine || (o == mine && g < group);
                    }
                    kept = before < p.group_k;
#pragma unroll
                    for (int i = 0; i < NE; ++i)
                        if (!kept) key[i] = 0;
                } else {
                    // lane g walks group g
#pragma unroll
                    for (int i = 0; i < NE; ++i)
                        if (lane * NE + i < E) sc[lane * NE + i] = c[i];
                    __builtin_amdgcn_wave_barrier();
                    const int size = E / p.groups;
                    uint64_t k1 = 0, k2 = 0;
                    double b1 = 0.0, b2 = 0.0;
                    if (lane < p.groups)
                        for (int m = 0; m < size; ++m) {
                            const double v = sc[lane * size + m];
                            const uint64_t kv = v == -INFINITY ? 0 : score_key(v);
                            if (kv > k1) {
                                k2 = k1; b2 = b1; k1 = kv; b1 = v;
                            } else if (kv > k2) {
                                k2 = kv; b2 = v;
                            }
                        }
                    const uint64_t mine = k1 == 0 ? 0 : score_key(p.group_top == 2 && k2 ? b1 + b2 : b1);
                    int before = 0;
                    for (int g = 0; g < p.groups; ++g) {
                        const uint64_t o = ((uint64_t)lane_value((unsigned)(mine >> 32), g) << 32) | lane_value((unsigned)mine, g);
                        before += o > mine || (o == mine && g < lane);
                    }
                    const uint64_t keep = __ballot(lane < p.groups && before < p.group_k);
#pragma unroll
                    for (int i = 0; i < NE; ++i) {
                        const int e = lane * NE + i;
                        if (e < E && !((keep >> (e / size)) & 1)) key[i] = 0;
                    }
                    __builtin_amdgcn_wave_barrier();
                }
            }
        }
        if constexpr (BY_LOGIT) {
            if (p.groups > 1) {
                // a group's score is its best logit's key; groups by lanes as above, or lane by lane
                const int size = E / p.groups;
                uint64_t *sk = reinterpret_cast<uint64_t *>(sc);
#pragma unroll
                for (int i = 0; i < NE; ++i)
                    if (lane * NE + i < E) sk[lane * NE + i] = key[i] & ~(uint64_t)(NE - 1);
                __builtin_amdgcn_wave_barrier();
                uint64_t mine = 0;
                if (lane < p.groups)
                    for (int m = 0; m < size; ++m) {
                        const uint64_t v = sk[lane * size + m];
                        mine = v > mine ? v : mine;
                    }
                int before = 0;
                for (int g = 0; g < p.groups; ++g) {
                    const uint64_t o = ((uint64_t)lane_value((unsigned)(mine >> 32), g) << 32) | lane_value((unsigned)mine, g);
                    before += o > mine || (o == mine && g < lane);
                }
                const uint64_t keep = __ballot(lane < p.groups && before < p.group_k);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    const int e = lane * NE + i;
                    if (e < E && !((keep >> (e / size)) & 1)) key[i] = 0;
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
        if constexpr (BY_LOGIT)
            sort_keys<NE>(key);
        else if (!done)
            sort_placed<NE>(key, at_place);
        for (int j = 0; !done && j < k; ++j) {
            const unsigned top = wave_max((unsigned)(key[0] >> 32));
            if (top == 0) break;
            uint64_t at = __ballot((unsigned)(key[0] >> 32) == top);
            if (at & (at - 1)) {   // lanes whose upper words are equal: the larger lower word, then the lower lane
                const bool in = (at >> lane) & 1;
                const unsigned low = in ? (unsigned)key[0] & ~(BY_LOGIT ? NE - 1u : 0u) : 0u;
                const unsigned most = wave_max(low);   // (every lane takes part)
                at = __ballot(in && low == most);
            }
            const int win = __builtin_ctzll(at);
            int place;
            if constexpr (BY_LOGIT)
                place = NE - 1 - (int)(lane_value((unsigned)key[0], win) & (NE - 1));
            else
                place = (int)lane_value((unsigned)at_place[0], win);
            if (lane == j) mine = win * NE + place;
            if (lane == win) {
#pragma unroll
                for (int i = 0; i + 1 < NE; ++i) {
                    key[i] = key[i + 1];
                    if constexpr (!BY_LOGIT) at_place[i] = at_place[i + 1];
                }
                key[NE - 1] = 0;
            }
        }
        // weights, from the chosen logits alone where they are renormalised; in 64
        // bits where scores that 32 bits lose still have a quotient.  In 32 bits the difference of logits
        // is carried with its rounding error, so that no weight's error grows with the logits: an
        // exponential 3 u, 1 + e and a reciprocal 3, the sum of the k 6 and theirs, the quotient 4: 22 u
        // renormalised (5 measured).  Not renormalised, a softmax's sum over E experts is off by what its terms
        // are, 3 u and their differences' rounding (their share of the sum weighs that: ln E), and 21 additions.
        const bool has = lane < k && mine >= 0;
        const float xl = has ? row[mine] : -INFINITY;
        const float ref = p.score == 1 ? 0.f : p.renorm ? wave_max(xl) : mx;
        const float over = p.renorm || p.score == 1 ? 1.f : sum32();   // (every lane takes part)
        float weight = 0.f;
        if (__ballot(has && (bad || !(fabsf(xl - ref) < 60.f))) == 0) {
            const float d = xl - ref, back = d - xl, low = (xl - (d - back)) - (ref + back);   // d + low = xl - ref
            float w = p.score == 1 ? exp_of(-d) : exp_of(d, low);                              // (sigmoid: ref = 0)
            if (p.score == 1) w = __builtin_amdgcn_rcpf(1.f + w);
            if (!has) w = 0.f;
            const float all = p.renorm ? wave_sum(w) : over;
            if (has) weight = w * __builtin_amdgcn_rcpf(all) * p.scale;
        } else {
            double w = 0.0;
            if (p.score == 1)
                w = has ? 1.0 / (1.0 + exp(-(double)xl)) : 0.0;
            else
                w = !has ? 0.0 : bad ? (double)NAN : exp((double)xl - (double)ref) / (double)over;
            if (p.renorm) {
                const double s = wave_sum(w);
                if (s != 0.0) w /= s;   // scores that are all zero keep weights of zero
            }
            if (has) weight = (float)(w * (double)p.scale);
        }
        if (lane < k) {
            p.ids[(long long)t * k + lane] = mine;
            p.weights[(long long)t * k + lane] = weight;
            cid[(t - t0) * k + lane] = mine < 0 ? E : mine;
        }
    }
    if (p.offsets == nullptr) return;

    const int n = (t1 - t0) * k;   // at most kChunkIds
    const int first = t0 * k;      // T*k fits an int
    const int per = E + 1;
    uint16_t *seg = reinterpret_cast<uint16_t *>(smem);
    __syncthreads();
    for (int i = tid; i < kSegments * per; i += NT) seg[i] = 0;
    __syncthreads();
    constexpr int IT = (kChunkIds + NT - 1) / NT;
    int mine[IT], rank[IT];
    const int bits = 32 - __builtin_clz((unsigned)E);   // E itself is an id
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int i = it * NT + tid;
        const int e = i < n ? cid[i] : 0;
        uint64_t same = __ballot(i < n);
        for (int bit = 0; bit < bits; ++bit) {
            const bool one = (e >> bit) & 1;
            const uint64_t m = __ballot(one);
            same &= one ? m : ~m;
        }
        mine[it] = e;
        rank[it] = __popcll(same & ((1ull << lane) - 1));
        if (i < n && rank[it] == 0) seg[(i >> 6) * per + e] = (uint16_t)__popcll(same);
    }
    __syncthreads();
    for (int e = tid; e < per; e += NT) {
        int run = 0;
#pragma unroll
        for (int g = 0; g < kSegments; ++g) {
            const int v = seg[g * per + e];
            seg[g * per + e] = (uint16_t)run;
            run += v;
        }
        total[e] = run;
        if (gridDim.x > 1) p.counts[(long long)blockIdx.x * per + e] = run;
    }
    __syncthreads();
    const bool alone = gridDim.x == 1;
    if (alone && wave == 0) {
        int carry = 0;
        for (int e0 = 0; e0 < per; e0 += 64) {
            const int e = e0 + lane;
            const int v = e < per ? total[e] : 0;
            const int s = wave_scan(v);
            if (e < per) {
                total[e] = carry + s - v;
                p.offsets[e] = carry + s - v;
            }
            carry += __builtin_amdgcn_readlane(s, 63);
        }
    }
    if (alone) __syncthreads();
#pragma unroll
    for (int it = 0; it < IT; ++it) {
        const int i = it * NT + tid;
        if (i >= n) continue;
        const int e = mine[it], local = seg[(i >> 6) * per + e] + rank[it];
        if (!alone) {
            p.slots[first + i] = local;
        } else {
            const int at = total[e] + local;
            p.slots[i] = e < E ? at : -1;
            p.rows[at] = e < E ? i / k : -1;
        }
    }
}

// The chunks' counts (chunks rows of E + 1) to the counts before each chunk, in
// place, and their totals as one more row.  A block takes 64 experts, one per
// lane; its waves take 16 chunks each in turn, read at once (256 chunks of 257 counts: 4.8 us, two trips to
// memory and a launch).
__global__ __launch_bounds__(1024) void prefix_kernel(RouteProblem p, int chunks)
{
    constexpr int PW = 16;   // chunks per wave and turn
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int per = p.E + 1, e = blockIdx.x * 64 + lane;
    __shared__ int part[2][16][64];   // (two: one barrier a turn)
    int carry = 0;
    for (int b0 = 0, turn = 0; b0 < chunks; b0 += 16 * PW, turn ^= 1) {
        const int first = b0 + wave * PW;
        int v[PW], sum = 0;
#pragma unroll
        for (int i = 0; i < PW; ++i) v[i] = e < per && first + i < chunks ? p.counts[(long long)(first + i) * per + e] : 0;
#pragma unroll
        for (int i = 0; i < PW; ++i) sum += v[i];
        part[turn][wave][lane] = sum;
        __syncthreads();
        int run = carry;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int s = part[turn][w][lane];
            run += w < wave ? s : 0;
            carry += s;
        }
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            if (e < per && first + i < chunks) p.counts[(long long)(first + i) * per + e] = run;
            run += v[i];
        }
    }
    if (wave == 0 && e < per) p.counts[(long long)chunks * per + e] = carry;
}

// Local numbers to rows.  PREFIXED: prefix_kernel has run; otherwise each block
// adds up the counts of the chunks before its own, and of all of them.  262144 choices: 5.0 us, of
// which the 4 MB moved are 0.9: a chain of loads, a scan and scattered stores.
template <bool PREFIXED>
__global__ __launch_bounds__(1024) void place_kernel(RouteProblem p, int chunk, int chunks)
{
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, k = p.k, E = p.E, per = E + 1;
    __shared__ int base[kMaxExperts + 2], total[kMaxExperts + 2];
    const int t0 = blockIdx.x * chunk, t1 = t0 + chunk < p.T ? t0 + chunk : p.T;
    // a thread's choice (a block has at most 1024), on its way while the counts are added up
    const int i = t0 * k + tid;
    const bool has = i < t1 * k;
    const int id = has ? p.ids[i] : -1, local = has ? p.slots[i] : 0;
    if constexpr (PREFIXED) {
        for (int e = tid; e < per; e += 1024) {
            base[e] = p.counts[(long long)blockIdx.x * per + e];
            total[e] = p.counts[(long long)chunks * per + e];
        }
    } else {
        for (int e = tid; e < per; e += 1024) base[e] = total[e] = 0;
        __syncthreads();
        const int runs = (per + 63) / 64;   // (64 experts) x (an eighth of the chunks) per wave and turn
        for (int it = wave; it < 8 * runs; it += 16) {
            const int e = it / 8 * 64 + lane;
            if (e >= per) continue;
            int before = 0, all = 0;
#pragma unroll 4
            for (int b = it % 8; b < chunks; b += 8) {
                const int v = p.counts[(long long)b * per + e];
                all += v;
                before += b < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&base[e], before);   // whole numbers in LDS: the order does not matter
            atomicAdd(&total[e], all);
        }
    }
    __syncthreads();
    if (wave == 0) {
        int carry = 0;
        for (int e0 = 0; e0 < per; e0 += 64) {
            const int e = e0 + lane;
            const int v = e < per ? total[e] : 0;
            const int s = wave_scan(v);
            if (e < per) {
                base[e] += carry + s - v;
                if (blockIdx.x == 0) p.offsets[e] = carry + s - v;
            }
            carry += __builtin_amdgcn_readlane(s, 63);
        }
    }
    __syncthreads();
    if (!has) return;
    const int at = base[id < 0 ? E : id] + local;
    p.slots[i] = id < 0 ? -1 : at;
    p.rows[at] = id < 0 ? -1 : i / k;
}
static_assert(kChunkIds <= 1024, "place_kernel: a choice per thread");

// Tokens per block.  One block for a few tokens (one launch); else 16 tokens or
// more, such that 256 blocks hold all of them while a block's choices fit
// kChunkIds.
int route_chunk(int T, int k)
{
    const int most = kChunkIds / k;
    if (T <= 64 && T <= most) return T < 1 ? 1 : T;
    const int c = (T + 255) / 256;
    const int least = most < 16 ? most : 16;
    return c < least ? least : c < most ? c : most;
}

constexpr int kDirectChunks = 64;   // up to these many chunks place_kernel adds the counts up itself

template <int NE, bool BY_LOGIT>
hipError_t route_ne(const RouteProblem &p, hipStream_t stream)
{
    constexpr int NT = NE <= 4 ? 1024 : 512;
    const int chunk = route_chunk(p.T, p.k), chunks = p.T > 0 ? (p.T + chunk - 1) / chunk : 1;
    // lanes that hold a group: whole ones, a power of two up to a row of 16
    const int size = p.E / p.groups, lanes = size % NE == 0 ? size / NE : 0;
    const int fast = lanes > 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    const size_t scores = p.groups > 1 ? (size_t)(NT / 64) * p.E * sizeof(double) : 0;
    const size_t counts = p.offsets ? (size_t)kSegments * (p.E + 1) * sizeof(uint16_t) : 0;
    hipLaunchKernelGGL((route_kernel<NE, NT, BY_LOGIT>), dim3(chunks), dim3(NT), scores > counts ? scores : counts, stream, p,
                       chunk, fast);
    if (chunks > 1 && p.offsets) {
        if (chunks <= kDirectChunks) {
            hipLaunchKernelGGL(place_kernel<false>, dim3(chunks), dim3(1024), 0, stream, p, chunk, chunks);
        } else {
            hipLaunchKernelGGL(prefix_kernel, dim3((p.E + 64) / 64), dim3(1024), 0, stream, p, chunks);
            hipLaunchKernelGGL(place_kernel<true>, dim3(chunks), dim3(1024), 0, stream, p, chunk, chunks);
        }
    }
    return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
//
// A wave per token.  s: the scores of all experts (softmax) or of the chosen
// ones; g_j = scale * dweights_j.
//   renormalised, p_j = s_j / sum of the chosen s:  q_j = p_j (g_j - sum_i p_i g_i);
//     softmax: dl = q_j (the softmax's own sum cancels; other experts 0),  sigmoid: dl = q_j (1 - s_j)
//   otherwise  softmax: dl_e = s_e (g_e - sum_i g_i s_i) over all experts,  sigmoid: dl = g_j s_j (1 - s_j)
// A router that is sure of its experts makes g_e and the sum nearly equal (and 1 - s_j small), so neither difference is
// formed.  With r the chosen expert of the largest score, D_j = dweights_j - dweights_r, and u the sum of the scores that
// are not chosen, added up by itself:
//   g_e - sum_i g_i s_i = scale (D_e - sum_i D_i s_i + dweights_r u),   q_j = p_j scale (D_j - sum_i p_i D_i),
//   1 - s = s(-x) for sigmoid scores.
// D_r is 0, so what stands at r are the small terms alone.  (Where u is 1/2 or more, or the largest score of all is not
// chosen, nothing cancels and dweights_r is taken as 0.)  Renormalised, the k values are formed in 64 bits, all else in
// 32.  They reach their experts' lanes through a row in LDS, of which a wave has one of its own (64 NE floats).
// 16384 tokens of 128 experts, softmax, 8 choices: 17.8 MB in 7.7 us (6.3 at the least), 2.3 TB/s, 3.8 us at a copy's
// rate.  Vector instructions take 75% of the cycles: a wave holds one token, two experts a lane, read
// and written a dword at a time, and its three reductions are a chain.

template <int NE>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradProblem p)
{
    __shared__ __attribute__((aligned(16))) float rows[4][64 * NE];
    __shared__ unsigned marks[4][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    const int E = p.E, k = p.k;
    if (t >= p.T) return;
    const float *row = p.logits + (long long)t * p.ldl;
    const int32_t *ids = p.ids + (long long)t * k;
    const float *dw = p.dweights + (long long)t * k;
    int id = lane < k ? ids[lane] : -1;
    const bool whole = p.score == 0 && !p.renorm;   // every expert gets a gradient
    float s[NE];
    if (whole) load_experts<NE>(row, lane, E, -INFINITY, s);
    const bool has = (unsigned)id < (unsigned)E;
    const float xl = has && !whole ? row[id] : -INFINITY;
    float *mine = rows[wave];
#pragma unroll
    for (int i = 0; i < NE; ++i) mine[lane * NE + i] = 0.f;
    const float d = has ? dw[lane] : 0.f;
    float acc[NE];
    if (whole) {
        // the chosen experts: a bit of their lane's word each, and their dweights (added up where the ids name one twice)
        unsigned *mark = marks[wave];
        mark[lane] = 0;
        if (has) {
            atomicOr(&mark[id / NE], 1u << (id % NE));
            atomicAdd(&mine[id], d);
        }
        __builtin_amdgcn_wave_barrier();
        const unsigned bits = mark[lane];
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            acc[i] = mine[lane * NE + i];
            mx = s[i] > mx ? s[i] : mx;
        }
        const float lane_mx = mx;
        mx = wave_max(mx);
        const uint64_t best = __ballot(lane_mx == mx);
        mx = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f, others = 0.f, top = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            top = s[i] == mx ? acc[i] : top;   // (0 if it is not chosen)
            const float x = s[i] - mx;
            s[i] = exp_of(x < -200.f ? -200.f : x);
            sum += s[i];
            others += (bits >> i) & 1 ? 0.f : s[i];
        }
        sum = wave_sum(sum);
        others = wave_sum(others);
        const float over = sum == 0.f ? 0.f : 1.f / sum, u = others * over;
        const float gr = best != 0 && u < 0.5f ? lane_value(top, __builtin_ctzll(best)) : 0.f;
        float mean = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            acc[i] = (bits >> i) & 1 ? acc[i] - gr : 0.f;
            mean = __builtin_fmaf(s[i], acc[i], mean);
        }
        mean = wave_sum(mean) * over;
        const float dot = __builtin_fmaf(gr, 1.f - u, mean);   // sum of g_i s_i; gr = 0 unless 1 - u > 1/2
        const float rest = __builtin_fmaf(gr, u, -mean), by = p.scale * over;
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = by * s[i] * ((bits >> i) & 1 ? acc[i] + rest : -dot);
    } else {
        float v;   // lane j: the value choice j adds to its expert
        if (p.renorm) {
            const float cm = wave_max(xl);
            double raw = 0.0, rest = 1.0;   // the score (softmax: up to a factor), and for sigmoid 1 less it
            if (has && p.score == 1) {
                const double e = exp(-fabs((double)xl)), q = 1.0 / (1.0 + e);
                raw = xl < 0.f ? e * q : q;
                rest = xl < 0.f ? q : e * q;
            } else if (has) {
                raw = xl == -INFINITY ? 0.0 : exp((double)xl - (double)cm);
            }
            const double sum = wave_sum(raw);
            const double pj = sum != 0.0 ? raw / sum : 0.0;
            const uint64_t best = __ballot(has && xl == cm);
            const double dj = (double)d - (best ? (double)lane_value(d, __builtin_ctzll(best)) : 0.0);
            const double mean = wave_sum(pj * dj);
            v = (float)((double)p.scale * (pj * (dj - mean) * rest));
        } else {
            // s (1 - s) = s(x) s(-x), neither factor a difference
            const float e = expf(-fabsf(xl)), q = 1.f / (1.f + e);
            v = p.scale * d * (e * q * q);
        }
        if (has) atomicAdd(&mine[id], v);   // (distinct experts: no two lanes add to one)
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < NE; ++i) acc[i] = mine[lane * NE + i];
    }
    float *out = p.dlogits + (long long)t * p.lddl;
    const int e0 = lane * NE;
    if constexpr (NE % 4 == 0) {
        if (e0 + NE <= E) {
#pragma unroll
            for (int i = 0; i < NE; i += 4)
                *reinterpret_cast<f32x4_g *>(out + e0 + i) = f32x4_t{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i)
        if (e0 + i < E) out[e0 + i] = acc[i];
}

// ---------------------------------------------------------------- combining
//
// C[t,:] = sum_j w_j Y[slot_j,:] + beta C[t,:]: four columns per thread, added in the order of
// the choices, one after another: a slot and its weight, then its row (and with beta C's four values one by one).
// With many tokens other waves' rows are on their way meanwhile and the bytes are the bound (4096 tokens of 2048
// columns, 8 choices: 302 MB in 49 us, 6.2 TB/s, part of Y being in the memory-side cache still; 61 us on
// other data each call); a few tokens' time is 2 k trips to memory in turn.
constexpr int kCombineCols = 1024;   // columns of a block of 256 threads

__global__ __launch_bounds__(256) void combine_kernel(CombineProblem p)
{
    const int t = blockIdx.x, k = p.k;
    const long long col = (long long)blockIdx.y * kCombineCols + 4 * threadIdx.x;
    if (col >= p.N) return;
    const bool four = col + 3 < p.N;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < k; ++j) {
        const int slot = p.slots[(long long)t * k + j];
        if (slot < 0 || slot >= p.R) continue;
        const float w = p.weights ? p.weights[(long long)t * k + j] : 1.f;
        const float *y = p.Y + (long long)slot * p.ldy + col;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
        if (four)
            v = *reinterpret_cast<const f32x4_g *>(y);
        else
            for (int e = 0; e < 3; ++e)
                if (col + e < p.N) v[e] = y[e];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(w, v[e], acc[e]);
    }
    float *dst = p.C + (long long)t * p.ldc + col;
    for (int e = 0; e < 4; ++e)
        if (p.beta != 0.f && col + e < p.N) acc[e] = __builtin_fmaf(p.beta, dst[e], acc[e]);
    if (four)
        *reinterpret_cast<f32x4_g *>(dst) = acc;
    else
        for (int e = 0; e < 3; ++e)
            if (col + e < p.N) dst[e] = acc[e];
}

template <bool BF>
__device__ __forceinline__ unsigned round16(float v)
{
    if constexpr (BF)
        return __builtin_bit_cast(unsigned short, (__bf16)v);
    else
        return __builtin_bit_cast(unsigned short, (_Float16)v);
}
typedef unsigned int u32x2_g __attribute__((ext_vector_type(2), aligned(4)));

// dY[slot_j,:] = w_j dC[t,:] rounded once to 16 bits, which is what the experts'
// gradient products take; dw_j = <dC[t,:], Y[slot_j,:]> summed in 32 bits: each
// thread its columns, then the wave, then the block's four waves in order.  A block takes a
// token, so that dC's row is read once for its k choices.  Bound by its bytes (8192 tokens of 1024
// columns, 4 choices: 235 MB in 38.9 us, 6.1 TB/s; 54 us on other data each call).
template <bool BF>
__global__ __launch_bounds__(256) void combine_grad_kernel(CombineGradProblem p)
{
    constexpr int JB = 8;   // choices per pass over the row
    const int t = blockIdx.x, k = p.k, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    __shared__ float part[4][JB];
    const bool pair = p.lddy % 2 == 0 && reinterpret_cast<uintptr_t>(p.dY) % 4 == 0;   // dword-aligned rows
    const float *dc = p.dC + (long long)t * p.lddc;
    for (int j0 = 0; j0 < k; j0 += JB) {
        const int nj = k - j0 < JB ? k - j0 : JB;
        float dot[JB];
        int slot[JB];
        float w[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            dot[j] = 0.f;
            slot[j] = -1;
            w[j] = 1.f;
            if (j < nj) {
                slot[j] = p.slots[(long long)t * k + j0 + j];
                if (slot[j] >= p.R) slot[j] = -1;
                if (p.weights) w[j] = p.weights[(long long)t * k + j0 + j];
            }
        }
        for (int col = 4 * tid; col < p.N; col += 1024) {
            const bool four = col + 3 < p.N;
            f32x4_t d = {0.f, 0.f, 0.f, 0.f};
            if (four)
                d = *reinterpret_cast<const f32x4_g *>(dc + col);
            else
                for (int e = 0; e < 3; ++e)
                    if (col + e < p.N) d[e] = dc[col + e];
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                if (slot[j] < 0) continue;
                const float *y = p.Y + (long long)slot[j] * p.ldy + col;
                uint16_t *o = p.dY + (long long)slot[j] * p.lddy + col;
                f32x4_t v = {0.f, 0.f, 0.f, 0.f};
                if (four)
                    v = *reinterpret_cast<const f32x4_g *>(y);
                else
                    for (int e = 0; e < 3; ++e)
                        if (col + e < p.N) v[e] = y[e];
                unsigned r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dot[j] = __builtin_fmaf(d[e], v[e], dot[j]);
                    r[e] = round16<BF>(w[j] * d[e]);
                }
                if (four && pair)
                    *reinterpret_cast<u32x2_g *>(o) = u32x2_g{r[0] | (r[1] << 16), r[2] | (r[3] << 16)};
                else
                    for (int e = 0; e < 4; ++e)
                        if (col + e < p.N) o[e] = (uint16_t)r[e];
            }
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            if (j >= nj) break;
            const float s = wave_sum(dot[j]);
            if (lane == 0) part[wave][j] = s;
        }
        __syncthreads();
        if (tid < nj) p.dweights[(long long)t * k + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
    }
}

}  // namespace

size_t route_workspace(int T, int E, int k)
{
    const int chunk = route_chunk(T, k), chunks = (T + chunk - 1) / chunk;
    return chunks > 1 ? (size_t)(chunks + 1) * (E + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_route(const RouteProblem &p, hipStream_t stream)
{
    const bool by_logit = p.bias == nullptr && (p.groups == 1 || p.group_top == 1);
    auto run = [&](auto ne) {
        constexpr int NE = decltype(ne)::value;
        return by_logit ? route_ne<NE, true>(p, stream) : route_ne<NE, false>(p, stream);
    };
    if (p.E <= 64) return run(std::integral_constant<int, 1>{});
    if (p.E <= 128) return run(std::integral_constant<int, 2>{});
    if (p.E <= 256) return run(std::integral_constant<int, 4>{});
    if (p.E <= 512) return run(std::integral_constant<int, 8>{});
    return run(std::integral_constant<int, 16>{});
}

hipError_t launch_route_grad(const RouteGradProblem &p, hipStream_t stream)
{
    const dim3 grid((p.T + 3) / 4), block(256);
    if (p.E <= 64)
        hipLaunchKernelGGL(route_grad_kernel<1>, grid, block, 0, stream, p);
    else if (p.E <= 128)
        hipLaunchKernelGGL(route_grad_kernel<2>, grid, block, 0, stream, p);
    else if (p.E <= 256)
        hipLaunchKernelGGL(route_grad_kernel<4>, grid, block, 0, stream, p);
    else if (p.E <= 512)
        hipLaunchKernelGGL(route_grad_kernel<8>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(route_grad_kernel<16>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_combine(const CombineProblem &p, hipStream_t stream)
{
    hipLaunchKernelGGL(combine_kernel, dim3(p.T, (p.N + kCombineCols - 1) / kCombineCols), dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_combine_grad(const CombineGradProblem &p, bool bf, hipStream_t stream)
{
    if (bf)
        hipLaunchKernelGGL(combine_grad_kernel<true>, dim3(p.T), dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL(combine_grad_kernel<false>, dim3(p.T), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace mi355gemm
