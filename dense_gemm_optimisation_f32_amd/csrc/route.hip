// route.hip -- routing of tokens to experts: scores, the choice of k experts per
// token, their weights, the rows sorted by expert; its gradient; the weighted
// sum of the experts' rows back to tokens and its gradient.
#include "routed_internal.h"
#include "epilogue.h"

#include <float.h>

namespace mi355gemm {
namespace {

// ---------------------------------------------------------------- wave helpers
template <class T>
__device__ __forceinline__ T wave_max(T v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const T o = __shfl_xor(v, d);
        v = o > v ? o : v;
    }
    return v;
}
template <class T>
__device__ __forceinline__ T wave_sum(T v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// A choice score as an unsigned key that orders like it: larger scores larger
// keys, NaN below every number (key 1), an expert that cannot be chosen last
// (key 0).  -inf is never an available expert's score, so no key clashes.
__device__ __forceinline__ uint64_t score_key(double c)
{
    if (c != c) return 1;
    const uint64_t b = (uint64_t)__double_as_longlong(c);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// ---------------------------------------------------------------- routing
//
// A block takes `chunk` consecutive tokens, a wave one token at a time.
//   choose: every lane holds the scores of experts lane, lane + 64, ...; the k
//     choices are k rounds of a maximum over the wave (ties to the lowest
//     index).  Choice scores are formed and compared in 64 bits: neighbouring
//     scores of one token are often nearer than 32 bits can tell, and the
//     choice is a whole number that either is right or is not.
//   layout: the block counts its choices by expert (expert E: the unfilled
//     choices) and numbers them in token order; one thread per expert walks
//     the chunk's ids, so the order never depends on timing.  With one block
//     the counts are scanned here; otherwise they go to `hist` and
//     place_kernel turns local numbers into rows.
template <int NE, int NT>
__global__ __launch_bounds__(NT) void route_kernel(RouteProblem p, int chunk)
{
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int T = p.T, E = p.E, k = p.k;
    const int t0 = blockIdx.x * chunk, t1 = t0 + chunk < T ? t0 + chunk : T;
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    double *sc = reinterpret_cast<double *>(smem) + (size_t)wave * (p.groups > 1 ? E : 0);
    int *cid = reinterpret_cast<int *>(smem + (p.groups > 1 ? (size_t)NW * E * sizeof(double) : 0));   // chunk x k ids

    for (int t = t0 + wave; t < t1; t += NW) {
        const float *row = p.logits + (long long)t * p.ldl;
        float x[NE];
        float mx = -INFINITY;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            x[i] = e < E ? row[e] : -INFINITY;
            mx = x[i] > mx ? x[i] : mx;
            nan |= x[i] != x[i];
        }
        mx = wave_max(mx);
        double sum = 0.0;
        double c[NE];
        if (p.score == 0) {
            // (a row of -inf alone has no available expert; its scores are not used)
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
        uint64_t key[NE];
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            const float b = p.bias && e < E ? p.bias[e] : 0.f;
            c[i] += (double)b;
            key[i] = x[i] == -INFINITY || b == -INFINITY ? 0 : score_key(c[i]);
        }
        if (p.groups > 1) {
            // lane g sums the best group_top available scores of group g; the
            // group_k best groups stay (ties to the lowest group)
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                if (e < E) sc[e] = key[i] == 0 ? -INFINITY : c[i];
            }
            __builtin_amdgcn_wave_barrier();
            const int size = E / p.groups;
            uint64_t gkey = 0;
            if (lane < p.groups) {
                uint64_t k1 = 0, k2 = 0;
                double b1 = 0.0, b2 = 0.0;
                for (int m = 0; m < size; ++m) {
                    const double v = sc[lane * size + m];
                    const uint64_t kv = v == -INFINITY ? 0 : score_key(v);
                    if (kv > k1) {
                        k2 = k1; b2 = b1; k1 = kv; b1 = v;
                    } else if (kv > k2) {
                        k2 = kv; b2 = v;
                    }
                }
                if (k1) gkey = score_key(p.group_top == 2 && k2 ? b1 + b2 : b1);
            }
            bool kept = false;
            for (int j = 0; j < p.group_k; ++j) {
                const uint64_t best = wave_max(kept || lane >= p.groups ? (uint64_t)0 : gkey + 1);
                if (best == 0) break;
                const uint64_t m = __ballot(!kept && lane < p.groups && gkey + 1 == best);
                if (lane == __builtin_ctzll(m)) kept = true;
            }
            const uint64_t keep = __ballot(kept);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                const int e = lane + 64 * i;
                if (e < E && !((keep >> (e / size)) & 1)) key[i] = 0;
            }
            __builtin_amdgcn_wave_barrier();
        }
        // k rounds: the largest key, of equal ones the lowest expert
        int mine = -1;   // lane j: choice j
        for (int j = 0; j < k; ++j) {
            uint64_t b = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (key[i] > b) {
                    b = key[i];
                    at = i;
                }
            const uint64_t best = wave_max(b);
            if (best == 0) break;
            int e = b == best ? lane + 64 * at : INT_MAX;
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) {
                const int o = __shfl_xor(e, d);
                e = o < e ? o : e;
            }
            if (lane == j) mine = e;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (lane + 64 * i == e) key[i] = 0;
        }
        // weights, from the chosen logits alone where they are renormalised
        const bool has = lane < k && mine >= 0;
        const float xl = has ? row[mine] : -INFINITY;
        double w = 0.0;
        if (p.score == 1)
            w = has ? 1.0 / (1.0 + exp(-(double)xl)) : 0.0;
        else if (p.renorm) {
            // (of a row that holds NaN or +inf every softmax score is NaN)
            const bool bad = __ballot(nan) != 0 || mx == INFINITY;
            const float cm = wave_max(xl);
            w = has ? (bad ? (double)NAN : exp((double)xl - (double)cm)) : 0.0;
        } else {
            w = has ? exp((double)xl - (double)mx) / sum : 0.0;
        }
        if (p.renorm) {
            const double s = wave_sum(w);
            if (s != 0.0) w /= s;   // scores that are all zero keep weights of zero
        }
        if (lane < k) {
            p.ids[(long long)t * k + lane] = mine;
            p.weights[(long long)t * k + lane] = (float)(has ? w * (double)p.scale : 0.0);
            cid[(t - t0) * k + lane] = mine < 0 ? E : mine;
        }
    }
    if (p.offsets == nullptr) return;
    __syncthreads();
    const int n = (t1 - t0) * k;
    const int first = t0 * k;   // T*k fits an int
    if (gridDim.x > 1) {
        int32_t *hist = p.hist + (long long)blockIdx.x * (E + 1);
        for (int e = tid; e <= E; e += NT) {
            int cnt = 0;
            for (int i = 0; i < n; ++i)
                if (cid[i] == e) p.slots[first + i] = cnt++;
            hist[e] = cnt;
        }
        return;
    }
    // one block: scan the counts here.  Thread e holds expert e's, then E's.
    __shared__ int total[kMaxExperts + 2];
    for (int e = tid; e <= E; e += NT) {
        int cnt = 0;
        for (int i = 0; i < n; ++i) cnt += cid[i] == e;
        total[e] = cnt;
    }
    __syncthreads();
    if (wave == 0) {
        int carry = 0;
        for (int b = 0; b <= E; b += 64) {
            const int e = b + lane;
            const int v = e <= E ? total[e] : 0;
            int s = v;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(s, d);
                if (lane >= d) s += o;
            }
            if (e <= E) total[e] = carry + s - v;
            carry += __shfl(s, 63);
        }
    }
    __syncthreads();
    for (int e = tid; e <= E; e += NT) {
        int at = total[e];
        p.offsets[e] = at;
        for (int i = 0; i < n; ++i)
            if (cid[i] == e) {
                p.slots[i] = e < E ? at : -1;
                p.rows[at++] = e < E ? i / k : -1;
            }
    }
}

// Local numbers to rows: block b adds up the counts of the chunks before its
// own (and of all, for the experts' starts) and places its chunk's choices.
__global__ __launch_bounds__(1024) void place_kernel(RouteProblem p, int chunk, int chunks)
{
    const int tid = threadIdx.x, E = p.E, k = p.k;
    __shared__ int base[kMaxExperts + 2], total[kMaxExperts + 2];
    for (int e = tid; e <= E; e += 1024) base[e] = total[e] = 0;
    __syncthreads();
    // threads share the (chunk, expert) counts by rows of chunks
    const int per = E + 1;
    for (int e = tid % 512; e < per; e += 512) {
        int before = 0, all = 0;
        for (int b = tid / 512; b < chunks; b += 2) {
            const int v = p.hist[(long long)b * per + e];
            all += v;
            if (b < (int)blockIdx.x) before += v;
        }
        atomicAdd(&base[e], before);   // whole numbers: the order does not matter
        atomicAdd(&total[e], all);
    }
    __syncthreads();
    if (tid < 64) {
        int carry = 0;
        for (int b = 0; b < per; b += 64) {
            const int e = b + tid;
            const int v = e < per ? total[e] : 0;
            int s = v;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(s, d);
                if (tid >= d) s += o;
            }
            if (e < per) {
                base[e] += carry + s - v;
                if (blockIdx.x == 0) p.offsets[e] = carry + s - v;
            }
            carry += __shfl(s, 63);
        }
    }
    __syncthreads();
    const int t0 = blockIdx.x * chunk, t1 = t0 + chunk < p.T ? t0 + chunk : p.T;
    for (int i = t0 * k + tid; i < t1 * k; i += 1024) {
        const int e = p.ids[i];
        const int at = base[e < 0 ? E : e] + p.slots[i];
        p.slots[i] = e < 0 ? -1 : at;
        p.rows[at] = e < 0 ? -1 : i / k;
    }
}

// Tokens per block: one block for up to 64 tokens, else 32 or more tokens such
// that place_kernel reads the counts of at most 256 chunks while a chunk's ids
// fit 16 KB of LDS.
int route_chunk(int T, int k)
{
    if (T <= 64) return 64;
    const int c = (T + 255) / 256, most = 4096 / k;
    return c < 32 ? 32 : c < most ? c : most;
}

template <int NE>
hipError_t route_ne(const RouteProblem &p, hipStream_t stream)
{
    const int chunk = route_chunk(p.T, p.k), chunks = p.T > 0 ? (p.T + chunk - 1) / chunk : 1;
    constexpr int NT1 = NE <= 4 ? 1024 : 256;   // threads of a single block (32 KB of group scores either way)
    const int nt = chunks == 1 ? NT1 : 256;
    const size_t lds = (p.groups > 1 ? (size_t)(nt / 64) * p.E * sizeof(double) : 0) + (size_t)chunk * p.k * sizeof(int);
    if (chunks == 1)
        hipLaunchKernelGGL((route_kernel<NE, NT1>), dim3(1), dim3(NT1), lds, stream, p, chunk);
    else
        hipLaunchKernelGGL((route_kernel<NE, 256>), dim3(chunks), dim3(256), lds, stream, p, chunk);
    if (chunks > 1 && p.offsets)
        hipLaunchKernelGGL(place_kernel, dim3(chunks), dim3(1024), 0, stream, p, chunk, chunks);
    return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
//
// A wave per token.  s: the scores of all experts (softmax) or of the chosen
// ones; g_j = scale * dweights_j.
//   renormalised, p_j = s_j / sum of the chosen s: ds-side factor
//     q_j = p_j (g_j - sum_i p_i g_i);   softmax: dl = q_j (the softmax's own sum cancels; other experts 0),
//     sigmoid: dl = q_j (1 - s_j)
//   otherwise  softmax: dl_e = s_e (g_e - sum_i g_i s_i) over all experts,  sigmoid: dl = g_j s_j (1 - s_j)
// The k chosen values are formed in 64 bits (differences of near numbers), the
// row in 32.
template <int NE>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradProblem p)
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int t = blockIdx.x * 4 + wave;
    const int E = p.E, k = p.k;
    if (t >= p.T) return;
    const float *row = p.logits + (long long)t * p.ldl;
    float *out = p.dlogits + (long long)t * p.lddl;
    int id = lane < k ? p.ids[(long long)t * k + lane] : -1;
    if (id >= E) id = -1;
    const bool has = id >= 0;
    const double g = has ? (double)p.scale * (double)p.dweights[(long long)t * k + lane] : 0.0;
    const float xl = has ? row[id] : -INFINITY;
    const bool whole = p.score == 0 && !p.renorm;   // every expert gets a gradient
    float s[NE];
    float v = 0.f;          // lane j: the gradient of choice j's own logit (g_j where whole)
    float dot = 0.f;
    if (whole) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int e = lane + 64 * i;
            s[i] = e < E ? row[e] : -INFINITY;
            mx = s[i] > mx ? s[i] : mx;
        }
        mx = wave_max(mx);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = s[i] == -INFINITY ? 0.f : expf(s[i] - mx);
            sum += s[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] = sum == 0.f ? 0.f : s[i] / sum;
        const double sl = !has ? 0.0 : xl == -INFINITY ? 0.0 : exp((double)xl - (double)mx) / (double)sum;
        dot = (float)wave_sum(g * sl);
        v = (float)g;
    } else {
        double sl, d = g;
        if (p.score == 0) {
            const float cm = wave_max(xl);
            sl = !has || xl == -INFINITY ? 0.0 : exp((double)xl - (double)cm);
        } else {
            sl = has ? 1.0 / (1.0 + exp(-(double)xl)) : 0.0;
        }
        const double raw = sl;
        if (p.renorm) {
            const double sum = wave_sum(sl);
            sl = sum != 0.0 ? sl / sum : 0.0;
            d = g - wave_sum(sl * g);
        }
        v = (float)(sl * d * (p.score == 1 ? 1.0 - raw : 1.0));
        if (!has) v = 0.f;
    }
    float acc[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) acc[i] = 0.f;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl(id, j);
        const float d = __shfl(v, j);
#pragma unroll
        for (int i = 0; i < NE; ++i)
            if (lane + 64 * i == e) acc[i] += d;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        const int e = lane + 64 * i;
        if (e < E) out[e] = whole ? s[i] * (acc[i] - dot) : acc[i];
    }
}

// ---------------------------------------------------------------- combining
//
// C[t,:] = sum_j w_j Y[slot_j,:] + beta C[t,:]: four columns per thread, the k
// rows read independently of one another, added in the order of the choices.
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
// thread its columns, then the wave, then the block's four waves in order.
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
    return chunks > 1 ? (size_t)chunks * (E + 1) * sizeof(int32_t) : 0;
}

hipError_t launch_route(const RouteProblem &p, hipStream_t stream)
{
    if (p.E <= 64) return route_ne<1>(p, stream);
    if (p.E <= 128) return route_ne<2>(p, stream);
    if (p.E <= 256) return route_ne<4>(p, stream);
    if (p.E <= 512) return route_ne<8>(p, stream);
    return route_ne<16>(p, stream);
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
