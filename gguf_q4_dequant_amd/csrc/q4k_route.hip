// Top-k routing and the grouping of (token, choice) pairs by expert.
//
// Routing.  One wave per token; lane l holds the logits of experts l, 64 + l,
// 128 + l, ... in registers.  The k choices are k rounds of a wave maximum
// (DPP moves inside the vector unit, no LDS round trip) followed by a ballot
// that finds the lowest expert holding it: a round costs about a hundred
// cycles, against the three thousand of comparing every pair of 128 scores.
//
// Grouping is a stable counting sort without atomics whose order could change
// a result.  Up to kSingleTokens tokens one workgroup of sixteen waves routes
// and groups in one launch: pairs are taken 64 at a time by a wave, each lane
// finds the lanes with its own expert by one ballot per bit of the expert
// number (its rank is the number of them below it), and per-wave counts per
// expert, summed over the waves in order, give every wave its first place in
// every group.  Above, a second launch has one workgroup per expert, which
// reads the whole table of choices: a ballot of "before my expert" gives the
// group's offset, one of "my expert" the places.  Every workgroup reads all P
// choices, but from the L2 and 64 at a time, and no counts cross workgroups.
//
// Both are bound by latency: one token over 128 experts, top 8, takes 5.2 us in
// one launch; 4096 tokens over 256 experts (sigmoid and bias, top 8) 9.3 us for
// the choices and 6.7 us for the groups, 4.6 MB in all.  Two launches take over
// where a wave of the one workgroup would have a second token: 128 experts
// without a bias, in graph replays: 16 tokens 6.7 us in one launch, 32 tokens
// 9.7 in one against 7.7 in two; 256 experts under a bias 10.0 at 16 in one
// against 9.2 at 17 in two.
#include <math.h>

#include "../../include/q4k_moe.h"
#include "q4k_internal.h"

namespace q4k {
namespace {

constexpr int kSingleTokens = 16;  // tokens routed and grouped by one workgroup: one a wave
constexpr int kSingleThreads = 1024;
constexpr int kThreads = 256;

template <int kCtrl>
__device__ __forceinline__ float dpp(float v, float identity) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(identity), __float_as_int(v), kCtrl, 0xF, 0xF,
                                                      false));
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v, double identity) {
    const int2 a = __builtin_bit_cast(int2, v), i = __builtin_bit_cast(int2, identity);
    int2 r;
    r.x = __builtin_amdgcn_update_dpp(i.x, a.x, kCtrl, 0xF, 0xF, false);
    r.y = __builtin_amdgcn_update_dpp(i.y, a.y, kCtrl, 0xF, 0xF, false);
    return __builtin_bit_cast(double, r);
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    int2 a = __builtin_bit_cast(int2, v);
    a.x = __builtin_amdgcn_readlane(a.x, lane);
    a.y = __builtin_amdgcn_readlane(a.y, lane);
    return __builtin_bit_cast(double, a);
}

// op over the 64 lanes, uniform: row shifts by 1, 2, 4 and 8 leave each row
// of 16 in its last lane, the two row broadcasts join the rows in lane 63.
template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, T identity, Op op) {
    v = op(v, dpp<0x111>(v, identity));
    v = op(v, dpp<0x112>(v, identity));
    v = op(v, dpp<0x114>(v, identity));
    v = op(v, dpp<0x118>(v, identity));
    v = op(v, dpp<0x142>(v, identity));
    v = op(v, dpp<0x143>(v, identity));
    return lane_value(v, 63);
}
template <class T>
__device__ __forceinline__ T wave_max(T v) {
    return wave_reduce(v, static_cast<T>(-INFINITY), [](T a, T b) { return a > b ? a : b; });
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
    return wave_reduce(v, static_cast<T>(0), [](T a, T b) { return a + b; });
}

// Floats as unsigned integers of the same order, all above 0 (-0 as +0), and back.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
    return __uint_as_float(o ^ (static_cast<uint32_t>(static_cast<int>(~o) >> 31) | 0x80000000u));
}

// The largest over the 64 lanes, uniform; one instruction a step, since 0 is
// the identity of the unsigned maximum and what a move from outside reads.
template <int kCtrl, int kRows>
__device__ __forceinline__ uint32_t max_step(uint32_t v) {
    const uint32_t o = __builtin_amdgcn_update_dpp(0, v, kCtrl, kRows, 0xF, kRows == 0xF);
    return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_step<0x111, 0xF>(v);
    v = max_step<0x112, 0xF>(v);
    v = max_step<0x114, 0xF>(v);
    v = max_step<0x118, 0xF>(v);
    v = max_step<0x142, 0xA>(v);
    v = max_step<0x143, 0xC>(v);
    return __builtin_amdgcn_readlane(v, 63);
}

// The softmax's numerator: 1 at the largest logit also where that is +inf.
__device__ __forceinline__ float softmax_term(float l, float mx) { return l == mx ? 1.f : expf(l - mx); }
__device__ __forceinline__ double softmax_term(double l, double mx) { return l == mx ? 1.0 : exp(l - mx); }

// The sigmoid with the exponential of -|l|, which cannot overflow: a low logit's
// score e^l / (1 + e^l) stays above 0 as long as a double holds e^l.
__device__ __forceinline__ double sigmoid_of(double l) {
    const double t = exp(-fabs(l));
    return (l < 0.0 ? t : 1.0) / (1.0 + t);
}

// Routes one token; lane j < top_k ends with choice j.
//   Without a bias the logits decide, which needs no arithmetic.  With one the
// scores do, and close scores have to be told apart: they are computed in
// float32, whose error here is below 2^-19 + 2^-24 |score + bias| (of a score
// of at most 1: an exponential and a quotient of a few 2^-24, for the softmax
// also its argument's, at most 0.4, and its sum of 16 terms a lane over 64
// lanes, 22; and the rounding of the last sum), and where another candidate
// comes within twice that of a round's best, the scores are computed once more
// in double, for the whole token, and decide.  (In double throughout, 4096
// tokens over 256 experts took 10.6 us, 1000 vector instructions a token.)
template <int VPL, bool kBias>
__device__ __forceinline__ void route_token(const float *logits, const float *bias, int E, int top_k, int flags,
                                            float scale, int lane, int &expert, float &weight) {
    const bool sigmoid = (flags & Q4K_ROUTE_SIGMOID) != 0;
    float l[VPL], bs[kBias ? VPL : 1];
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = v * 64 + lane;
        l[v] = e < E ? logits[e] : -INFINITY;
        if constexpr (kBias) bs[v] = e < E ? bias[e] : 0.f;
    }
    // keys: the order of the logits (of the scores under a bias), 0: not to be chosen
    uint32_t key[VPL], top = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        key[v] = l[v] > -INFINITY ? ordered(l[v]) : 0;  // NaN: 0 too
        top = key[v] > top ? key[v] : top;
    }
    const float mx = from_ordered(wave_max(top));
    float sum = 1.f;  // of the softmax's numerators
    float term[VPL];
    if (!sigmoid && (kBias || !(flags & Q4K_ROUTE_NORMALIZE))) {
        sum = 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            term[v] = key[v] != 0 ? softmax_term(l[v], mx) : 0.f;
            sum += term[v];
        }
        sum = wave_sum(sum);
    }
    if constexpr (kBias) {
        if (sigmoid) {
#pragma unroll
            for (int v = 0; v < VPL; ++v) term[v] = 1.f / (1.f + expf(-l[v]));
        }
        const float share = 1.f / sum;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const float s = term[v] * share + bs[v];
            key[v] = key[v] != 0 && s > -INFINITY ? ordered(s) : 0;
        }
    }
    double exact[kBias ? VPL : 1];
    bool have_exact = false;
    expert = -1;
    float mine = 0.f;  // the choice's logit
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int v = 1; v < VPL; ++v) best = key[v] > best ? key[v] : best;
        best = wave_max(best);
        if (best == 0) break;  // uniform: nothing left to choose
        uint64_t at[VPL];      // the lanes of the best (without close ones: exactly one)
        uint32_t least = best;
        if constexpr (kBias) {
            const float f = from_ordered(best), near = f - (0x1p-18f + 0x1p-22f * fabsf(f));
            least = near > -INFINITY ? ordered(near) : best;  // NaN where the best is infinite
        }
        int found = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            at[v] = __ballot(key[v] >= least);
            found += __builtin_popcountll(at[v]);
        }
        if constexpr (kBias) {
            if (found > 1) {
                if (!have_exact) {
                    have_exact = true;
                    double total = 0.0;
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        float z = l[v];
                        asm volatile("" : "+v"(z));  // keeps the doubles out of the common path (and one at a time)
                        exact[v] = !(z > -INFINITY) ? 0.0
                                   : sigmoid       ? sigmoid_of(static_cast<double>(z))
                                                   : softmax_term(static_cast<double>(z), static_cast<double>(mx));
                        total += exact[v];
                    }
                    total = sigmoid ? 1.0 : wave_sum(total);
#pragma unroll
                    for (int v = 0; v < VPL; ++v)
                        exact[v] = exact[v] / total + static_cast<double>(bias[min(v * 64 + lane, E - 1)]);
                }
                double largest = -INFINITY;
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    if (key[v] >= least && exact[v] > largest) largest = exact[v];
                largest = wave_max(largest);
#pragma unroll
                for (int v = 0; v < VPL; ++v) at[v] = __ballot(key[v] >= least && exact[v] == largest);
            }
        }
        int owner = 0, slot = -1;
#pragma unroll
        for (int v = VPL - 1; v >= 0; --v) {
            slot = at[v] != 0 ? v : slot;
            owner = at[v] != 0 ? __builtin_ctzll(at[v]) : owner;
        }
        float val = l[0];
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            val = slot == v ? l[v] : val;
            key[v] = slot == v && lane == owner ? 0 : key[v];
        }
        val = lane_value(val, owner);
        if (lane == j) {
            expert = slot * 64 + owner;
            mine = val;
        }
    }
    // One value per lane from here: in double, where a sigmoid does not
    // underflow before -745 (nor lose bits before -708) and the shares of very
    // low scores stay exact.
    double w = 0.0;
    if (expert >= 0)
        w = sigmoid ? sigmoid_of(static_cast<double>(mine))
                    : softmax_term(static_cast<double>(mine), static_cast<double>(mx));
    if (flags & Q4K_ROUTE_NORMALIZE) {
        const double total = wave_sum(w);
        w = total > 0.0 ? w / total : 0.0;
    } else {
        w = w / static_cast<double>(sum);
    }
    weight = expert >= 0 ? scale * static_cast<float>(w) : 0.f;
}

__device__ __forceinline__ int expert_bits(int E) { return E <= 1 ? 0 : 32 - __builtin_clz(E - 1); }

// The lanes of the wave that hold this lane's expert (0 for a lane without).
__device__ __forceinline__ uint64_t same_expert(int e, bool valid, int bits) {
    uint64_t mask = __ballot(valid);
    for (int b = 0; b < bits; ++b) {
        const bool bit = (e >> b) & 1;
        const uint64_t with = __ballot(bit);
        mask &= bit ? with : ~with;
    }
    return valid ? mask : 0;
}

__device__ __forceinline__ uint64_t lanes_below(int lane) { return (1ull << lane) - 1; }

// The waves of a workgroup that share [0, count) in chunks of 64: a few pairs
// leave most of them, and their rows of hist, out.
__device__ __forceinline__ int sharing_waves(int count, int waves) {
    const int chunks = (count + 63) / 64, per = (chunks + waves - 1) / waves;
    return (chunks + per - 1) / per;
}

// hist[wave][e] += pairs of expert e among this wave's share of [0, count).
template <class F>
__device__ __forceinline__ void count_pairs(F expert_of, int count, int E, int *hist) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int chunks = (count + 63) / 64, per = (chunks + waves - 1) / waves, bits = expert_bits(E);
    for (int c = wave * per; c < min(chunks, (wave + 1) * per); ++c) {
        const int i = c * 64 + lane;
        const int e = i < count ? expert_of(i) : -1;
        const bool valid = static_cast<unsigned>(e) < static_cast<unsigned>(E);
        const uint64_t same = same_expert(e, valid, bits);
        if (valid && (same & lanes_below(lane)) == 0) atomicAdd(&hist[wave * E + e], __builtin_popcountll(same));
    }
}

// Places the pairs of one workgroup: hist [sharing waves][E] holds the counts
// of count_pairs, tot [E + 1] is scratch, both in LDS.
template <class F>
__device__ __forceinline__ void place_pairs(F expert_of, int count, int E, int *hist, int *tot, int *offsets,
                                            int *rows) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int sharing = sharing_waves(count, waves);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int run = 0;
        for (int w = 0; w < sharing; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = run;
            run += c;
        }
        tot[e] = run;
    }
    __syncthreads();
    if (wave == 0) {  // exclusive scan of the totals over the experts
        int carry = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int c = e0 + lane < E ? tot[e0 + lane] : 0;
            int incl = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int up = __shfl_up(incl, o);
                incl += lane >= o ? up : 0;
            }
            if (e0 + lane < E) tot[e0 + lane] = carry + incl - c;
            carry += __shfl(incl, 63);
        }
        if (lane == 0) tot[E] = carry;
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += blockDim.x) offsets[e] = tot[e];
    const int chunks = (count + 63) / 64, per = (chunks + waves - 1) / waves, bits = expert_bits(E);
    for (int c = wave * per; c < min(chunks, (wave + 1) * per); ++c) {
        const int i = c * 64 + lane;
        const int e = i < count ? expert_of(i) : -1;
        const bool valid = static_cast<unsigned>(e) < static_cast<unsigned>(E);
        const uint64_t same = same_expert(e, valid, bits);
        const uint64_t below = same & lanes_below(lane);
        if (valid) {
            rows[tot[e] + hist[wave * E + e] + __builtin_popcountll(below)] = i;
            if (below == 0) atomicAdd(&hist[wave * E + e], __builtin_popcountll(same));
        }
    }
    for (int i = tot[E] + threadIdx.x; i < count; i += blockDim.x) rows[i] = -1;
}

struct RouteArgs {
    const float *logits, *bias;
    int *expert;
    float *weight;
    int *offsets, *rows;
    int M, E, top_k, flags;
    float scale;
};

// One workgroup: routing and grouping.  LDS: hist [sharing waves][E], tot
// [E + 1] and the choices [M][top_k].
// (Half the waves where sixteen scores a lane and their doubles need more than
// a sixteenth of the registers.)
template <int VPL, bool kBias>
constexpr int kGroupThreads = VPL > 8 && kBias ? kSingleThreads / 2 : kSingleThreads;

template <int VPL, bool kBias>
__global__ __launch_bounds__((kGroupThreads<VPL, kBias>)) void route_group_kernel(RouteArgs a) {
    extern __shared__ int lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const int count = a.M * a.top_k, counts = sharing_waves(count, waves) * a.E;
    int *hist = lds, *tot = hist + counts, *chosen = tot + a.E + 1;
    for (int i = threadIdx.x; i < counts; i += blockDim.x) hist[i] = 0;
    for (int m = wave; m < a.M; m += waves) {
        int e;
        float w;
        route_token<VPL, kBias>(a.logits + static_cast<size_t>(m) * a.E, a.bias, a.E, a.top_k, a.flags, a.scale, lane, e, w);
        if (lane < a.top_k) {
            chosen[m * a.top_k + lane] = e;
            a.expert[m * a.top_k + lane] = e;
            a.weight[m * a.top_k + lane] = w;
        }
    }
    __syncthreads();
    const auto expert_of = [&](int i) { return chosen[i]; };
    count_pairs(expert_of, count, a.E, hist);
    place_pairs(expert_of, count, a.E, hist, tot, a.offsets, a.rows);
}

// Routing only: one token per wave.
template <int VPL, bool kBias>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 63;
    const size_t m = static_cast<size_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6);
    if (m >= static_cast<size_t>(a.M)) return;
    int e;
    float w;
    route_token<VPL, kBias>(a.logits + m * a.E, a.bias, a.E, a.top_k, a.flags, a.scale, lane, e, w);
    if (lane < a.top_k) {
        a.expert[m * a.top_k + lane] = e;
        a.weight[m * a.top_k + lane] = w;
    }
}

// Grouping: workgroup e places the pairs of expert e; the last one also closes
// the offsets and fills the tail of rows.  A wave reads its share of the
// choices in rounds of kAhead steps of 64, all of a round's loads requested
// together; up to kAhead * 1024 pairs there is one round, whose choices stay
// in registers from the counts to the places (256 experts: 5.9 us); beyond, every
// workgroup reads the table twice (10.4 us just above, 20 at 131072 pairs, 143 at
// 2^20).
__global__ __launch_bounds__(kSingleThreads) void group_kernel(const int *expert, int P, int E, int *offsets, int *rows) {
    constexpr int kWaves = kSingleThreads / 64, kAhead = 32;
    __shared__ int s_less[kWaves], s_same[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int mine = blockIdx.x;
    // this wave's share, in steps of 64 pairs (unsigned: a step may pass P)
    const unsigned steps = (static_cast<unsigned>(P) + 63) / 64, per = (steps + kWaves - 1) / kWaves;
    const unsigned i0 = wave * per * 64, i1 = min(static_cast<unsigned>(P), i0 + per * 64);
    int e[kAhead];
    const auto load = [&](unsigned i) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) e[k] = i + k * 64 + lane < i1 ? expert[i + k * 64 + lane] : -1;
    };
    int less = 0, same = 0;
    for (unsigned i = i0; i < i1; i += 64 * kAhead) {
        load(i);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            // as unsigned, -1 and every other negative number is above any expert
            less += __builtin_popcountll(__ballot(static_cast<unsigned>(e[k]) < static_cast<unsigned>(mine)));
            same += __builtin_popcountll(__ballot(e[k] == mine));
        }
    }
    if (lane == 0) {
        s_less[wave] = less;
        s_same[wave] = same;
    }
    __syncthreads();
    int base = 0, before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        base += s_less[w];
        before += w < wave ? s_same[w] : 0;
        all += s_same[w];
    }
    if (threadIdx.x == 0) offsets[mine] = base;
    int at = base + before;
    for (unsigned i = i0; i < i1; i += 64 * kAhead) {
        if (per > kAhead) load(i);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint64_t with = __ballot(e[k] == mine);
            if (with == 0) continue;  // uniform
            if (e[k] == mine) rows[at + __builtin_popcountll(with & lanes_below(lane))] = static_cast<int>(i + k * 64 + lane);
            at += __builtin_popcountll(with);
        }
    }
    if (mine == E - 1) {
        if (threadIdx.x == 0) offsets[E] = base + all;
        for (unsigned i = base + all + threadIdx.x; i < static_cast<unsigned>(P); i += kSingleThreads) rows[i] = -1;
    }
}

hipError_t launch_group(const int *expert, int P, int E, int *offsets, int *rows, hipStream_t stream) {
    hipLaunchKernelGGL(group_kernel, dim3(E), dim3(kSingleThreads), 0, stream, expert, P, E, offsets, rows);
    return hipGetLastError();
}

template <int VPL, bool kBias>
hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
    if (a.M <= kSingleTokens) {
        constexpr int kThreads1 = kGroupThreads<VPL, kBias>, waves = kThreads1 / 64;
        const int bytes = (waves * a.E + a.E + 1 + a.M * a.top_k) * 4;
        const hipError_t err = allow_dynamic_lds(reinterpret_cast<const void *>(route_group_kernel<VPL, kBias>), 96 << 10);
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL((route_group_kernel<VPL, kBias>), dim3(1), dim3(kThreads1), bytes, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((route_kernel<VPL, kBias>), dim3((a.M - 1) / (kThreads / 64) + 1), dim3(kThreads), 0, stream, a);
    const hipError_t err = hipGetLastError();
    return err != hipSuccess ? err : launch_group(a.expert, a.M * a.top_k, a.E, a.offsets, a.rows, stream);
}

template <bool kBias>
hipError_t launch_route_for(const RouteArgs &a, hipStream_t stream) {
    if (a.E <= 64) return launch_route<1, kBias>(a, stream);
    if (a.E <= 128) return launch_route<2, kBias>(a, stream);
    if (a.E <= 256) return launch_route<4, kBias>(a, stream);
    if (a.E <= 512) return launch_route<8, kBias>(a, stream);
    return launch_route<16, kBias>(a, stream);
}

bool misaligned4(const void *a, const void *b = nullptr, const void *c = nullptr, const void *d = nullptr,
                 const void *e = nullptr, const void *f = nullptr) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
             reinterpret_cast<uintptr_t>(d) | reinterpret_cast<uintptr_t>(e) | reinterpret_cast<uintptr_t>(f)) & 3u) != 0;
}

int status(hipError_t err) {
    if (err == hipErrorOutOfMemory || err == hipErrorMemoryAllocation) return Q4K_ERR_ALLOC;
    return err == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_moe_route(const float *logits, const float *bias, int M, int E, int top_k, int flags,
                             float scale, int *expert, float *weight, int *offsets, int *rows, hipStream_t stream) {
    using namespace q4k;
    if (M < 0 || E < 1 || E > Q4K_MAX_EXPERTS || top_k < 1 || top_k > E || top_k > Q4K_MAX_TOP_K ||
        static_cast<int64_t>(M) * top_k > INT_MAX || (flags & ~(Q4K_ROUTE_SIGMOID | Q4K_ROUTE_NORMALIZE)) != 0)
        return Q4K_ERR_BAD_DIM;
    if (!offsets || (M > 0 && (!logits || !expert || !weight || !rows))) return Q4K_ERR_NULL;
    if (misaligned4(logits, bias, expert, weight, offsets, rows)) return Q4K_ERR_ALIGN;
    const int dev_rc = check_device();
    if (dev_rc != Q4K_OK) return dev_rc;
    if (M == 0) return status(launch_group(nullptr, 0, E, offsets, rows, stream));
    const RouteArgs a = {logits, bias, expert, weight, offsets, rows, M, E, top_k, flags, scale};
    return status(bias ? launch_route_for<true>(a, stream) : launch_route_for<false>(a, stream));
}

extern "C" int q4k_moe_group(const int *expert, int P, int E, int *offsets, int *rows, hipStream_t stream) {
    using namespace q4k;
    if (P < 0 || E < 1 || E > Q4K_MAX_EXPERTS) return Q4K_ERR_BAD_DIM;
    if (!offsets || (P > 0 && (!expert || !rows))) return Q4K_ERR_NULL;
    if (misaligned4(expert, offsets, rows)) return Q4K_ERR_ALIGN;
    const int dev_rc = check_device();
    if (dev_rc != Q4K_OK) return dev_rc;
    return status(launch_group(expert, P, E, offsets, rows, stream));
}
