// Products grouped by expert over packed Q4_K weights: y[p] = x[row of p] .
// dequant(W[e])^T for every pair p of group e (include/q4k_moe.h), the gate/up
// form with its SwiGLU epilogue, and the weighted sum over a token's experts.
//
// What is computed.  A Q4_K weight is w = d * sc_j * q - dmin * m_j with the
// 6-bit sc_j, m_j of its 32-weight sub-block j and the 4-bit quant q, so for a
// token t, a row n of W and one super-block
//   y += d * (sum_k x_k * (sc q)_k) - dmin * (sum_j m_j X_j),   X_j = sum of x over sub-block j.
//   * sc * q <= 945 is an integer below 2^11: exact as a binary16.  A nibble in
//     the low bits of a 16-bit lane is the binary16 subnormal q * 2^-24 (one AND
//     for two weights), times sc in binary16 (v_pk_mul_f16) the subnormal
//     sc * q * 2^-24, still exact; the matrix cores keep subnormals.  Both
//     scales d and dmin stay out of the operand and are applied to the fp32
//     sums once per super-block of 256, so nothing of W is ever rounded.
//   * x is scaled by a power of two per row, 2^e, that puts the row's largest
//     magnitude in [2^14, 2^15), and split into two binary16 values, hi =
//     rn(x'), lo = rn(x' - hi): about 22 bits of every value, and an absolute
//     error of at most 2^-39 of the row's maximum where lo is subnormal (half
//     of its step of 2^-24, against a maximum of 2^14 at least).  Both
//     enter the same fp32 accumulator: two v_mfma_f32_16x16x32_f16 per 32
//     weights, half the binary16 matrix rate at fp32 accuracy.
//   * The min term is one more MFMA per super-block: the eight X_j (hi and lo
//     in k-quarters 0 and 1) times the eight m_j as subnormals.  X_j is split
//     after a division by 2^6 that keeps it in range: to 2^-33 of the maximum.
//
// k order.  The order of k inside an MFMA is free as long as both operands
// agree.  Lane quarter c of a wave (lanes 16c .. 16c + 15, one row of W each)
// takes group c of the super-block, 32 contiguous quant bytes = sub-blocks 2c
// (low nibbles) and 2c + 1 (high): a lane reads 32 bytes of its row in two
// 16-byte loads and needs two of the eight scales.  Step s = 2i + h uses bytes
// 8i .. 8i + 7 of every group, nibble h; inside a step a lane's eight k are
// 8i + {0, 2, 1, 3, 4, 6, 5, 7} (bytes 0, 2 and 1, 3 of a dword come out of one
// AND each).  The staged x is laid out in that order once per call.
#include <limits.h>
#include <math.h>

#include "../../include/q4k_moe.h"
#include "q4k_internal.h"
#include "q4k_rows.h"

namespace q4k {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));

constexpr int kImageBlock = 1024;  // staged bytes per super-block of a row: 8 steps x (hi, lo) x 4 quarters x 16
constexpr int kSumsBlock = 32;     // eight sub-block sums, hi then lo

struct Staged {
    const uint8_t *img;   // [rows][K / 256][kImageBlock]
    const uint8_t *sums;  // [rows][K / 256][kSumsBlock]
    const float *back;    // [rows]: 2^(8 - e)
};

// The e of the scale 2^e that puts a largest magnitude mx in [2^14, 2^15),
// limited so that 2^e is a float (zeros and subnormals: 127, infinity and NaN:
// 0); the largest float has -113.  The way back, 2^(24 - e) with the quants'
// 2^24, does not fit a float there: it is 2^(8 - e), always a normal one, after
// 2^16, which the sums take without rounding and without overflow (they stay
// below 2^43 for any K).
__device__ __forceinline__ int scale_exponent(float mx) {
    const int E = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu);
    const int e = E == 0 ? 127 : (E == 255 ? 0 : 141 - E);
    return max(-113, min(127, e));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
constexpr float kBackFirst = 65536.f;

// Stages eight consecutive values of a row at k (see above); the four threads
// of a sub-block are neighbours and join its sum.
__device__ __forceinline__ void stage_eight(const float4 a, const float4 b, int k, float up, uint8_t *im, uint8_t *sm) {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    constexpr int order[8] = {0, 2, 1, 3, 4, 6, 5, 7};
    half8 hi, lo;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = v[order[i]] * up;
        hi[i] = static_cast<_Float16>(t);
        lo[i] = static_cast<_Float16>(t - static_cast<float>(hi[i]));
        s += t;
    }
    const int blk = k / kBlockWeights, in = k % kBlockWeights;
    const int quarter = in >> 6, h = (in >> 5) & 1, i = (in >> 3) & 3;
    uint8_t *o = im + blk * kImageBlock + (2 * i + h) * 128 + quarter * 16;
    *reinterpret_cast<half8 *>(o) = hi;
    *reinterpret_cast<half8 *>(o + 64) = lo;
    // 32 values below 2^15 each: times 2^-6 to stay in binary16's range
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    s *= 0.015625f;
    if (i == 0) {
        const _Float16 sh = static_cast<_Float16>(s);
        _Float16 *so = reinterpret_cast<_Float16 *>(sm + blk * kSumsBlock) + (in >> 5);
        so[0] = sh;
        so[8] = static_cast<_Float16>(s - static_cast<float>(sh));
    }
}

// Stages one row of x per workgroup: the row's first kKept * 8 values of every
// thread stay in registers between the maximum and the conversion.  Bound by
// memory: 8192 rows of 1024 (68 MB read and written) 13 us, 5.0 TB/s.
constexpr int kStageThreads = 1024, kKept = 2;
__global__ __launch_bounds__(kStageThreads) void stage_rows_kernel(const float *x, int K, uint8_t *img, uint8_t *sums,
                                                                   float *back) {
    __shared__ float wave_mx[kStageThreads / 64];
    const size_t row = blockIdx.x;
    const float *xr = x + row * K;
    const int step = blockDim.x * 8, k0 = threadIdx.x * 8;
    float4 a[kKept], b[kKept];
#pragma unroll
    for (int j = 0; j < kKept; ++j) {
        a[j] = b[j] = float4{0.f, 0.f, 0.f, 0.f};
        if (k0 + j * step < K) {
            a[j] = *reinterpret_cast<const float4 *>(xr + k0 + j * step);
            b[j] = *reinterpret_cast<const float4 *>(xr + k0 + j * step + 4);
        }
    }
    const auto largest = [](float mx, const float4 v) {
        return fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
    };
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < kKept; ++j) mx = largest(largest(mx, a[j]), b[j]);
    for (int64_t k = k0 + static_cast<int64_t>(kKept) * step; k < K; k += step)
        mx = largest(largest(mx, *reinterpret_cast<const float4 *>(xr + k)), *reinterpret_cast<const float4 *>(xr + k + 4));
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    if ((threadIdx.x & 63) == 0) wave_mx[threadIdx.x >> 6] = mx;
    __syncthreads();
    for (unsigned w = 0; w < blockDim.x >> 6; ++w) mx = fmaxf(mx, wave_mx[w]);
    const int e = scale_exponent(mx);
    const float up = power_of_two(e);
    if (threadIdx.x == 0) back[row] = power_of_two(8 - e);
    uint8_t *im = img + row * (K / kBlockWeights) * kImageBlock;
    uint8_t *sm = sums + row * (K / kBlockWeights) * kSumsBlock;
#pragma unroll
    for (int j = 0; j < kKept; ++j)
        if (k0 + j * step < K) stage_eight(a[j], b[j], k0 + j * step, up, im, sm);
    for (int64_t k = k0 + static_cast<int64_t>(kKept) * step; k < K; k += step)
        stage_eight(*reinterpret_cast<const float4 *>(xr + k), *reinterpret_cast<const float4 *>(xr + k + 4),
                    static_cast<int>(k), up, im, sm);
}

struct Grouped {
    const uint8_t *w, *w2;  // [E][N][K/256*144]; w2: the up matrices (SwiGLU) or null
    Staged x;
    const int *offsets, *rows;
    float *y;
    int E, P, N, K, x_div;
};

struct Tile {
    int e, first, count;  // rows[first .. first + count) of expert e
};

// The groups cut into tiles of TM rows.  Lane l of a wave owns experts 4l ..
// 4l + 3 of each 256; every wave scans the offsets by itself (one memory round
// trip and a scan in the vector unit for up to 256 experts).
template <int TM>
struct Tiles {
    const int *offsets;
    int E, P, lane;
    int first[4], count[4], before;  // of the 256 experts from e0; before: tiles of this lane's predecessors
    int sum;                         // tiles of these 256 experts

    __device__ __forceinline__ void load(int e0) {
        int o[5];
#pragma unroll
        for (int i = 0; i < 5; ++i) o[i] = min(max(offsets[min(e0 + 4 * lane + i, E)], 0), P);
        int own = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            first[i] = o[i];
            count[i] = max(o[i + 1] - o[i], 0);
            own += (count[i] + TM - 1) / TM;
        }
        int v = own;  // inclusive scan: within rows of 16 lanes, then across them
        v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
        v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
        v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
        v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
        v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
        v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
        before = v - own;
        sum = __builtin_amdgcn_readlane(v, 63);
    }

    __device__ __forceinline__ Tiles(const int *off, int experts, int pairs, int ln)
        : offsets(off), E(experts), P(pairs), lane(ln) {
        load(0);
    }

    // Tiles of all experts.  Leaves the first 256 experts loaded.
    __device__ __forceinline__ int total() {
        if (E <= 256) return sum;
        int n = 0;
        for (int e0 = (E - 1) / 256 * 256; e0 >= 0; e0 -= 256) {
            load(e0);
            n += sum;
        }
        return n;
    }

    // Tile number t (count 0: there is none); the first 256 experts are loaded.
    __device__ __forceinline__ Tile find(int t) {
        for (int e0 = 0;;) {
            if (t < sum) {
                // the last lane with before <= t owns it
                const int owner = 63 - __builtin_clzll(__ballot(before <= t));
                int at = t - __builtin_amdgcn_readlane(before, owner);
                if (at < 0) return {0, 0, 0};  // a table whose groups overlap may claim more tiles than an int counts
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = __builtin_amdgcn_readlane(count[i], owner), n = (c + TM - 1) / TM;
                    if (at < n)
                        return {e0 + 4 * owner + i, __builtin_amdgcn_readlane(first[i], owner) + at * TM,
                                min(TM, c - at * TM)};
                    at -= n;
                }
            }
            t -= sum;
            e0 += 256;
            if (e0 >= E) return {0, 0, 0};
            load(e0);
        }
    }
};

// One lane's part of one super-block of its row of W.
struct WBlock {
    uint4 head, q0, q1;
};
__device__ __forceinline__ WBlock load_block(const uint8_t *row, int b, int quarter) {
    const uint8_t *p = row + static_cast<size_t>(b) * kBlockBytes;
    return {*reinterpret_cast<const uint4 *>(p), *reinterpret_cast<const uint4 *>(p + 16 + 32 * quarter),
            *reinterpret_cast<const uint4 *>(p + 32 + 32 * quarter)};
}

struct WScales {
    float d, nm;  // d, -64 * dmin
    half2v s;     // the lane's two scales, the second / 16 (its nibbles are 16q)
    half8 mins;   // m_0..m_7 as subnormals m * 2^-24
};
__device__ __forceinline__ WScales block_scales(const uint4 hd, int quarter) {
    WScales s;
    s.d = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hd.x & 0xFFFFu)));
    s.nm = -64.f * static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hd.x >> 16)));
    const uint32_t scA = hd.y & 0x3F3F3F3Fu, mnA = hd.z & 0x3F3F3F3Fu;
    const uint32_t scB = (hd.w & 0x0F0F0F0Fu) | ((hd.y >> 2) & 0x30303030u);
    const uint32_t mnB = ((hd.w >> 4) & 0x0F0F0F0Fu) | ((hd.z >> 2) & 0x30303030u);
    // bytes 2 quarter and 2 quarter + 1 of scA, scB as 16-bit lanes; 0x6400 |
    // sc is the binary16 1024 + sc
    const uint32_t two = __builtin_amdgcn_perm(scB, scA, 0x0C010C00u + 0x00020002u * quarter);
    const half2v sc = __builtin_bit_cast(half2v, two | 0x64006400u) - half2v{1024, 1024};
    s.s = sc * half2v{1, static_cast<_Float16>(0.0625f)};
    uint4 m;  // bytes to 16-bit lanes
    m.x = __builtin_amdgcn_perm(0u, mnA, 0x0C010C00u);
    m.y = __builtin_amdgcn_perm(0u, mnA, 0x0C030C02u);
    m.z = __builtin_amdgcn_perm(0u, mnB, 0x0C010C00u);
    m.w = __builtin_amdgcn_perm(0u, mnB, 0x0C030C02u);
    s.mins = __builtin_bit_cast(half8, m);
    return s;
}

// The operand of step 2i + h (h = 0: low nibbles, 1: high) from two dwords.
__device__ __forceinline__ half2v scaled(uint32_t bits, half2v s) { return __builtin_bit_cast(half2v, bits) * s; }
__device__ __forceinline__ half8 join(half2v a, half2v b, half2v c, half2v d) {
    return half8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ half8 operand(uint32_t u, uint32_t v, const WScales &s, int h) {
    const uint32_t mask = h ? 0x00F000F0u : 0x000F000Fu;
    const half2v sc = h ? half2v{s.s.y, s.s.y} : half2v{s.s.x, s.s.x};
    return join(scaled(u & mask, sc), scaled((u >> 8) & mask, sc), scaled(v & mask, sc), scaled((v >> 8) & mask, sc));
}

__device__ __forceinline__ float4v mfma(half8 a, half8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// ---- many rows per expert: tiles of RT * 16 rows times 64 NC columns ----------

// LDS of a workgroup: two buffers of x (a quarter of a super-block: two steps,
// 256 bytes a row), two of its sub-block sums, one super-block of each wave's
// own rows of W, and the tile's pairs and factors.
template <int RT, int NC>
struct TileLds {
    static constexpr int kRows = RT * 16;
    static constexpr int kX = kRows * 256, kSums = kRows * kSumsBlock, kW = 16 * NC * kBlockBytes;
    static constexpr int kSumsAt = 2 * kX, kWAt = kSumsAt + 2 * kSums, kPairsAt = kWAt + 4 * kW;
    static constexpr int kBackAt = kPairsAt + kRows * 4, kBytes = kBackAt + kRows * 4;
};

typedef uint32_t rsrc_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

// LDS byte address of a uniform pointer.
__device__ __forceinline__ uint32_t lds_address(uint8_t *p) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_u8 *)p)));
}

// 16 bytes per lane from memory to LDS at dst + 16 * lane.  Written in
// assembly because the compiler waits for every such copy before the next LDS
// read, whichever buffer that reads; no register is written, and the kernel
// waits for vmcnt and the barrier before it reads a buffer.
// m0, which the compiler keeps to itself, is named as clobbered, so that no use
// of its own is moved across; it remarks that the register is reserved.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(const uint8_t *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory", "m0");
}
// The same from a buffer (offsets behind its end read zeros).
__device__ __forceinline__ void copy_to_lds(rsrc_t buffer, uint32_t offset, uint32_t base, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(offset), "s"(buffer),
                 "s"(__builtin_amdgcn_readfirstlane(base)), "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory", "m0");
}
#pragma clang diagnostic pop
// A raw buffer of bytes at p (both uniform).
__device__ __forceinline__ rsrc_t buffer_at(const uint8_t *p, uint32_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    rsrc_t r;
    r.x = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    r.y = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32) & 0xFFFFu);
    r.z = __builtin_amdgcn_readfirstlane(bytes);
    r.w = 0x00020000u;
    return r;
}

// Every copy and LDS operation of this wave has ended.
__device__ __forceinline__ void wait_all() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("" ::: "memory");
}
// Every LDS operation of this wave has ended (copies may be on their way).
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}
// All but the last VM copies of this wave, and every LDS operation, have ended.
template <int VM>
__device__ __forceinline__ void wait_copies() {
    static_assert(VM < 16, "one field of the counter");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | VM);
    asm volatile("" ::: "memory");
}
// The workgroup's barrier (what its waves have waited for is then there for all).
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A wave's 16 NC rows of W, copied to its own LDS slot one super-block at a
// time, 144 bytes a row: two halves of 8 NC rows (SwiGLU: gate and up), row
// 16c + r of the slot being column r of the wave's column tile c.  Rows behind
// N read zeros, or row N - 1 where a half has no other; their columns are never
// stored.  (No copy is left out: the waits count them.)
template <int NC, bool kSwiglu>
struct WTile {
    static constexpr int kHalfRows = 8 * NC, kPieces = 9 * kHalfRows, kCopies = (kPieces + 63) / 64;
    static constexpr int kLast = kPieces - 64 * (kCopies - 1);  // lanes of the last copy
    static constexpr int kBytes = 2 * kPieces * 16;
    static constexpr int kN = kSwiglu ? 8 * NC : 16 * NC;  // outputs of a wave
    uint32_t off[kCopies];
    rsrc_t buf[2];
    uint32_t lds;
    int lane;

    __device__ __forceinline__ WTile(const Grouped &g, int e, int n0, uint8_t *slot, int ln)
        : lds(lds_address(slot)), lane(ln) {
        const uint32_t row_bytes = static_cast<uint32_t>(g.K / kBlockWeights) * kBlockBytes;
#pragma unroll
        for (int k = 0; k < kCopies; ++k) {
            const int piece = k * 64 + lane, j = piece / 9;
            off[k] = j * row_bytes + (piece - 9 * j) * 16;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const RowWindow r = row_window(n0 + (kSwiglu ? 0 : kHalfRows * h), kHalfRows, g.N);
            buf[h] = buffer_at((kSwiglu && h ? g.w2 : g.w) + (static_cast<size_t>(e) * g.N + r.first) * row_bytes,
                               r.rows * row_bytes);
        }
    }
    __device__ __forceinline__ void copy(int b) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < kCopies; ++k)
                if (k < kCopies - 1 || lane < kLast)
                    copy_to_lds(buf[h], off[k], b * kBlockBytes, lds + h * (kPieces * 16) + k * 1024);
    }
};

// The address of workgroup `id` in the work of `tiles` row tiles times n_tiles
// column tiles (-1: none).  Workgroups go to the eight XCDs in turn: each XCD
// takes one contiguous eighth of the work, column tiles fastest, so that the
// workgroups that share rows of x or an expert's matrix share an L2.
__device__ __forceinline__ int place_in_work(unsigned id, int tiles, int n_tiles) {
    const int64_t work = static_cast<int64_t>(tiles) * n_tiles, per = (work + 7) / 8;
    const int64_t at = (id & 7) * per + (id >> 3);
    // (a table whose offsets do not ascend may claim more than a call can hold)
    return (id >> 3) >= per || at >= work || at > INT_MAX ? -1 : static_cast<int>(at);
}

// Pair i of the tile, the last one again behind its end; -1 for an entry
// outside [0, P).
__device__ __forceinline__ int pair_of(const Grouped &g, const Tile &t, int i) {
    const int at = t.first + min(i, t.count - 1);
    const int p = g.rows ? g.rows[at] : at;
    return static_cast<unsigned>(p) < static_cast<unsigned>(g.P) ? p : -1;
}

// The tile's pairs.
__device__ __forceinline__ void load_pairs(const Grouped &g, const Tile &t, int rows, int *pairs) {
    if (threadIdx.x < rows) pairs[threadIdx.x] = pair_of(g, t, threadIdx.x);
}
// The factors of their rows, which only the end needs: asked for behind the
// first copies of x, and there with the barrier that waits for those.
__device__ __forceinline__ void load_factors(const Grouped &g, int rows, const int *pairs, float *back) {
    if (threadIdx.x < rows) back[threadIdx.x] = g.x.back[max(pairs[threadIdx.x], 0) / g.x_div];
}

// Writes row i of the tile's columns: acc[c] for column n0 + 16c + c16
// (SwiGLU: tiles 0 .. NC / 2 - 1 gate, the others up).
template <int NC, bool kSwiglu>
__device__ __forceinline__ void store_row(const Grouped &g, int p, float back, int n0, int c16, const float acc[NC]) {
    float *yr = g.y + static_cast<size_t>(p) * g.N;
    constexpr int kOut = kSwiglu ? NC / 2 : NC;
#pragma unroll
    for (int c = 0; c < kOut; ++c) {
        const float v = acc[c] * kBackFirst * back;
        const float out = kSwiglu ? swiglu(v, acc[(c + kOut) % NC] * kBackFirst * back) : v;
        if (n0 + 16 * c + c16 < g.N) yr[n0 + 16 * c + c16] = out;
    }
}

// The arithmetic of one tile over its first RT row tiles of 16.  Every wave
// reads all of the tile's x from LDS and builds the operands of its own columns
// of W in registers: RT row tiles share an operand, NC column tiles a fragment
// of x, and two waves a SIMD (RT = 3, NC = 4, 241 registers) hide each other's
// waits.  Bound by the power of the matrix cores: 16384 pairs over 64 experts of
// 2 x 1024 x 2048 take 290 us, 0.95 PFLOP/s of binary16 (1.20 for a large plain
// product on this card), with the pipes busy half of the cycles at 1.9 GHz; the
// same work with a quarter fewer vector instructions took the same time at a
// lower clock.  Three buffers of x, copied two quarters ahead: 314 against 302 us.
template <int RT, class L, int NC, bool kSwiglu>
__device__ __forceinline__ void run_tile(const Grouped &g, const Tile &t, const WTile<NC, kSwiglu> &w, uint8_t *lds, int wave,
                                         int lane, int n0) {
    const int c16 = lane & 15, quarter = lane >> 4;
    const int *pairs = reinterpret_cast<const int *>(lds + L::kPairsAt);
    float *back = reinterpret_cast<float *>(lds + L::kBackAt);
    const uint8_t *const wslot = lds + L::kWAt + wave * L::kW;
    const int KB = g.K / kBlockWeights;

    // x: this wave copies rows 4 RT wave .. + 4 RT of the tile, four per
    // instruction; a row's 16-byte pieces are exchanged by its number (piece c
    // in slot c ^ (row % 16)), so that a column of pieces reads 16 banks apart.
    const uint8_t *xsrc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
        const int row = wave * RT * 4 + j * 4 + quarter;
        const size_t xr = max(pairs[row], 0) / g.x_div;
        xsrc[j] = g.x.img + xr * KB * kImageBlock + ((c16 ^ (row & 15)) * 16);
    }
    const uint8_t *ssrc = g.x.sums;
    if (lane < RT * 8) {
        const size_t xr = max(pairs[wave * RT * 4 + (lane >> 1)], 0) / g.x_div;
        ssrc += xr * KB * kSumsBlock + (lane & 1) * 16;
    }
    const uint32_t lds0 = lds_address(lds);
    const auto copy_x = [&](int b, int i, int buf) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
            copy_to_lds(xsrc[j] + (static_cast<size_t>(b) * kImageBlock + i * 256), lds0 + buf * L::kX + (wave * RT + j) * 1024);
    };
    const auto copy_sums = [&](int b) {
        if (lane < RT * 8)
            copy_to_lds(ssrc + static_cast<size_t>(b) * kSumsBlock, lds0 + L::kSumsAt + (b & 1) * L::kSums + wave * RT * 128);
    };
    float4v acc[RT][NC];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
    copy_x(0, 0, 0);
    copy_sums(0);
    load_factors(g, RT * 16, pairs, back);
    for (int b = 0; b < KB; ++b) {
        WScales ws[NC];
        float4v blk[RT][NC];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // x of this quarter has arrived; the others' too behind the barrier
            wait_all();
            barrier();
            if (i < 3) copy_x(b, i + 1, (i + 1) & 1);
            else if (b + 1 < KB) {
                copy_x(b + 1, 0, 0);
                copy_sums(b + 1);
            }
            if (i == 0) {
                half8 am[RT];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint4 s = *reinterpret_cast<const uint4 *>(lds + L::kSumsAt + (b & 1) * L::kSums +
                                                                     (r * 16 + c16) * kSumsBlock + (quarter & 1) * 16);
                    am[r] = __builtin_bit_cast(half8, quarter < 2 ? s : uint4{0, 0, 0, 0});
                }
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    ws[c] = block_scales(*reinterpret_cast<const uint4 *>(wslot + (c * 16 + c16) * kBlockBytes), quarter);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float4v cm = mfma(am[r], ws[c].mins, float4v{0.f, 0.f, 0.f, 0.f});
                        blk[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[r][c][k] = __builtin_fmaf(ws[c].nm, cm[k], acc[r][c][k]);
                    }
                }
            }
            uint2 q[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c)
                q[c] = *reinterpret_cast<const uint2 *>(wslot + (c * 16 + c16) * kBlockBytes + 16 + 32 * quarter + 8 * i);
            if (i == 3 && b + 1 < KB) {
                // every read of this wave's W slot has returned: refill it
                wait_lds();
                w.copy(b + 1);
            }
            const uint8_t *xb = lds + (i & 1) * L::kX + c16 * 256;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __builtin_amdgcn_sched_barrier(0);  // one step's operands in registers at a time
                half8 op[NC];
#pragma unroll
                for (int c = 0; c < NC; ++c) op[c] = operand(q[c].x, q[c].y, ws[c], h);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    half8 a[RT];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
                        a[r] = *reinterpret_cast<const half8 *>(xb + ((((h * 2 + part) * 4 + quarter) ^ c16) * 16) + r * 4096);
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int r = 0; r < RT; ++r) blk[r][c] = mfma(a[r], op[c], blk[r][c]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[r][c][k] = __builtin_fmaf(ws[c].d, blk[r][c][k], acc[r][c][k]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = r * 16 + 4 * quarter + k, p = pairs[i];
            if (i >= t.count || p < 0) continue;
            float v[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) v[c] = acc[r][c][k];
            store_row<NC, kSwiglu>(g, p, back[i], n0, c16, v);
        }
}

template <int RT, int NC, bool kSwiglu>
__global__ __launch_bounds__(256, 2) void tile_kernel(Grouped g) {
    using L = TileLds<RT, NC>;
    using W = WTile<NC, kSwiglu>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Tiles<L::kRows> tiles(g.offsets, g.E, g.P, lane);
    const int n_tiles = (g.N - 1) / (4 * W::kN) + 1;
    const int at = place_in_work(blockIdx.x, tiles.total(), n_tiles);
    if (at < 0) return;
    const Tile t = tiles.find(at / n_tiles);
    if (t.count == 0) return;
    const int n0 = (at % n_tiles * 4 + wave) * W::kN;
    const W w(g, t.e, n0, lds + L::kWAt + wave * L::kW, lane);
    w.copy(0);
    load_pairs(g, t, L::kRows, reinterpret_cast<int *>(lds + L::kPairsAt));
    __syncthreads();
    const int active = (t.count + 15) / 16;  // uniform: a group's last tile takes the row tiles that it fills
    if (active >= RT) run_tile<RT, L>(g, t, w, lds, wave, lane, n0);
    else if (RT > 2 && active == 2) run_tile<2, L>(g, t, w, lds, wave, lane, n0);
    else run_tile<1, L>(g, t, w, lds, wave, lane, n0);
}

// ---- up to about sixteen rows per expert ---------------------------------------

// One row tile of 16: here the stream of W sets the pace.  W moves to
// registers at the start of a super-block and its slot is refilled at once, so
// that copies are on their way during all of the arithmetic; x comes half a
// super-block (512 bytes a row) at a time in two buffers.  That keeps a
// workgroup within a quarter of the LDS, and four to a CU.  Where the tiles
// leave CUs idle, KS such groups of four waves split K by super-blocks (group s
// takes blocks s, s + KS, ...), and the first adds the others' sums in order:
// 64 pairs over 8 experts of 1024 x 2048 15.5 -> 13.6 us.  (Staging x inside
// this kernel instead of by a launch of its own was slower: 32 against 29 us
// for 48 x 8 rows over 64 experts of 2048 x 1024, 66 against 48 us at 128 x 8.)
// Bound by the stream of W: those 48 x 8 rows read 75 MB in 20 us (3.7 TB/s, one
// round of workgroups, its start and end with it), 32 x 8 rows over 64 experts of
// 2 x 1024 x 2048 read 151 MB in 29 us (5.2 TB/s); copying only the rows of x that
// a tile has changed neither.
template <int NC>
struct ThinLds {
    static constexpr int kX = 16 * kImageBlock / 2, kSums = 16 * kSumsBlock, kW = 16 * NC * kBlockBytes;
    static constexpr int kSumsAt = 2 * kX, kWAt = kSumsAt + 2 * kSums, kGroup = kWAt + 4 * kW;
    static constexpr int bytes(int groups) { return groups * kGroup + 16 * 8; }
};

// Adds the wave groups' sums (R values of a thread each): groups 1 .. KS - 1
// leave them in LDS, group 0 returns true with all of them.
template <int KS, int R>
__device__ __forceinline__ bool join_groups(float *acc, uint8_t *lds, int group) {
    if constexpr (KS == 1) return true;
    float *red = reinterpret_cast<float *>(lds) + (threadIdx.x & 255);
    wait_all();
    barrier();  // every group has left its buffers
    if (group != 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) red[((group - 1) * R + i) * 256] = acc[i];
    }
    __syncthreads();
    if (group != 0) return false;
#pragma unroll
    for (int s = 1; s < KS; ++s)
#pragma unroll
        for (int i = 0; i < R; ++i) acc[i] += red[((s - 1) * R + i) * 256];
    return true;
}

template <int NC, int KS, bool kSwiglu>
__global__ __launch_bounds__(256 * KS, 4) void thin_kernel(Grouped g) {
    using L = ThinLds<NC>;
    using W = WTile<NC, kSwiglu>;
    extern __shared__ __align__(16) uint8_t all_lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) & 3);
    const int group = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    uint8_t *const lds = all_lds + group * L::kGroup;
    const int c16 = lane & 15, quarter = lane >> 4;
    Tiles<16> tiles(g.offsets, g.E, g.P, lane);
    const int n_tiles = (g.N - 1) / (4 * W::kN) + 1;
    const int at = place_in_work(blockIdx.x, tiles.total(), n_tiles);
    if (at < 0) return;
    const Tile t = tiles.find(at / n_tiles);
    if (t.count == 0) return;
    const int n0 = (at % n_tiles * 4 + wave) * W::kN;
    uint8_t *const wslot = lds + L::kWAt + wave * L::kW;
    const W w(g, t.e, n0, wslot, lane);
    const int KB = g.K / kBlockWeights;
    if (group < KB) w.copy(group);
    int *pairs = reinterpret_cast<int *>(all_lds + KS * L::kGroup);
    float *back = reinterpret_cast<float *>(pairs + 16);
    load_pairs(g, t, 16, pairs);
    __syncthreads();
    // x: this wave copies rows 4 wave .. + 4, two per instruction, their pieces
    // exchanged by the row's number as in tile_kernel
    const uint8_t *xsrc[2], *ssrc = g.x.sums;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = wave * 4 + j * 2 + (lane >> 5);
        const size_t xr = max(pairs[row], 0) / g.x_div;
        xsrc[j] = g.x.img + xr * KB * kImageBlock + (((lane & 31) ^ row) * 16);
    }
    if (lane < 8) {
        const size_t xr = max(pairs[wave * 4 + (lane >> 1)], 0) / g.x_div;
        ssrc += xr * KB * kSumsBlock + (lane & 1) * 16;
    }
    const uint32_t lds0 = lds_address(lds);
    const auto copy_x = [&](int b, int half) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            copy_to_lds(xsrc[j] + (static_cast<size_t>(b) * kImageBlock + half * (kImageBlock / 2)),
                        lds0 + half * L::kX + (wave * 2 + j) * 1024);
    };
    const auto copy_sums = [&](int b, int buf) {
        if (lane < 8)
            copy_to_lds(ssrc + static_cast<size_t>(b) * kSumsBlock, lds0 + L::kSumsAt + buf * L::kSums + wave * 128);
    };
    float4v acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
    if (group < KB) {
        copy_x(group, 0);
        copy_sums(group, 0);
    }
    load_factors(g, 16, pairs, back);
    int parity = 0;  // of the sums' buffers
    for (int b0 = 0; b0 < KB; b0 += KS, parity ^= 1) {
        const int b = b0 + group;
        wait_all();
        barrier();
        if (KS > 1 && b >= KB) {  // uniform over a wave; the barriers are the workgroup's
            barrier();
            continue;
        }
        WBlock wb[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) wb[c] = load_block(wslot + (c * 16 + c16) * kBlockBytes, 0, quarter);
        wait_lds();  // W is in registers
        copy_x(b, 1);
        const bool more = b + KS < KB;
        if (more) w.copy(b + KS);
        WScales ws[NC];
        float4v blk[NC];
        const uint4 s = *reinterpret_cast<const uint4 *>(lds + L::kSumsAt + parity * L::kSums + c16 * kSumsBlock + (quarter & 1) * 16);
        const half8 am = __builtin_bit_cast(half8, quarter < 2 ? s : uint4{0, 0, 0, 0});
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            ws[c] = block_scales(wb[c].head, quarter);
            const float4v cm = mfma(am, ws[c].mins, float4v{0.f, 0.f, 0.f, 0.f});
            blk[c] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][k] = __builtin_fmaf(ws[c].nm, cm[k], acc[c][k]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i == 2) {
                // the second half of x, requested before W of the next block,
                // which may stay on its way
                if (more) wait_copies<2 * W::kCopies>();
                else wait_all();
                barrier();
                if (more) {
                    copy_x(b + KS, 0);
                    copy_sums(b + KS, parity ^ 1);
                }
            }
            __builtin_amdgcn_sched_barrier(0);  // the operands of one pair of steps in registers at a time
            const uint8_t *xb = lds + (i >> 1) * L::kX + c16 * (kImageBlock / 2) + (i & 1) * 256;
            half8 a[4];
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) a[s4] = *reinterpret_cast<const half8 *>(xb + ((4 * s4 + quarter) ^ c16) * 16);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const uint4 qq = i < 2 ? wb[c].q0 : wb[c].q1;
                const uint32_t u = i & 1 ? qq.z : qq.x, v = i & 1 ? qq.w : qq.y;
                const half8 low = operand(u, v, ws[c], 0), high = operand(u, v, ws[c], 1);
                blk[c] = mfma(a[0], low, blk[c]);
                blk[c] = mfma(a[1], low, blk[c]);
                blk[c] = mfma(a[2], high, blk[c]);
                blk[c] = mfma(a[3], high, blk[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[c][k] = __builtin_fmaf(ws[c].d, blk[c][k], acc[c][k]);
    }
    if (!join_groups<KS, NC * 4>(reinterpret_cast<float *>(acc), all_lds, group)) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = 4 * quarter + k, p = pairs[i];
        if (i >= t.count || p < 0) continue;
        float v[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) v[c] = acc[c][k];
        store_row<NC, kSwiglu>(g, p, back[i], n0, c16, v);
    }
}

// ---- few rows per expert -----------------------------------------------------

// Four rows of x times 32 rows of W (SwiGLU: 16 gate and the same 16 up rows)
// per workgroup; the waves split K by super-blocks, each with its own LDS:
// one super-block of the 32 rows of W, the staged x and its factors.  Without a
// launch for the staging, and with K in eight parts, a call is about three memory
// round trips (the offsets; the rows' numbers, beside the first of W; x): 8 of 128
// experts of 2 x 1024 x 2048 for one token (18.9 MB) 9.3 us, or 7.5 with the weights
// still in the L2s, 2 of 16 of 4096 x 2048 (9.4 MB) 5.6 us, of which an empty launch
// is about 2.
constexpr int kFewRows = 4;
struct FewLds {
    static constexpr int kW = 32 * kBlockBytes, kX = kFewRows * kImageBlock, kSums = kFewRows * kSumsBlock;
    static constexpr int kXAt = kW, kSumsAt = kXAt + kX, kBackAt = kSumsAt + kSums, kWave = kBackAt + 16;
};

template <int kCtrl>
__device__ __forceinline__ float dpp_move(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, false));
}

// Stages one super-block of four rows for the wave: lane 16r + p holds values
// 16p .. 16p + 15 of row r.  The four quarters' pieces of a step are exchanged
// by the row's number, so that the rows read different banks.  The scale is per row and super-block here, so
// that a wave needs nothing from the others.
__device__ __forceinline__ void stage_few(const float4 v[4], int lane, uint8_t *base) {
    const int r = lane >> 4, p = lane & 15;
    const float x[16] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w,
                         v[2].x, v[2].y, v[2].z, v[2].w, v[3].x, v[3].y, v[3].z, v[3].w};
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(x[i]));
    mx = fmaxf(mx, dpp_move<0x121>(mx));  // rotations by 1, 2, 4, 8 within the row of 16 lanes
    mx = fmaxf(mx, dpp_move<0x122>(mx));
    mx = fmaxf(mx, dpp_move<0x124>(mx));
    mx = fmaxf(mx, dpp_move<0x128>(mx));
    const int e = scale_exponent(mx);
    const float up = power_of_two(e);
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        constexpr int order[8] = {0, 2, 1, 3, 4, 6, 5, 7};
        half8 hi, lo;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = x[8 * u + order[i]] * up;
            hi[i] = static_cast<_Float16>(t);
            lo[i] = static_cast<_Float16>(t - static_cast<float>(hi[i]));
            s += t;
        }
        // k = 16p + 8u: quarter p / 4, half (p / 2) % 2, step pair 2 (p % 2) + u
        const int quarter = p >> 2, h = (p >> 1) & 1, i = 2 * (p & 1) + u;
        uint8_t *o = base + FewLds::kXAt + r * kImageBlock + (2 * i + h) * 128 + (quarter ^ r) * 16;
        *reinterpret_cast<half8 *>(o) = hi;
        *reinterpret_cast<half8 *>(o + 64) = lo;
    }
    s += dpp_move<0xB1>(s);  // the other half of the sub-block (lanes exchanged in pairs)
    s *= 0.015625f;
    if ((p & 1) == 0) {
        const _Float16 sh = static_cast<_Float16>(s);
        _Float16 *so = reinterpret_cast<_Float16 *>(base + FewLds::kSumsAt + r * kSumsBlock) + (p >> 1);
        so[0] = sh;
        so[8] = static_cast<_Float16>(s - static_cast<float>(sh));
    }
    if (p == 0) reinterpret_cast<float *>(base + FewLds::kBackAt)[r] = power_of_two(8 - e);
}

template <int WAVES, bool kSwiglu>
__global__ __launch_bounds__(64 * WAVES, 4) void few_kernel(Grouped g, const float *x) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, quarter = lane >> 4;
    const Tile t = Tiles<kFewRows>(g.offsets, g.E, g.P, lane).find(blockIdx.y);
    if (t.count == 0) return;
    const int KB = g.K / kBlockWeights;
    using W = WTile<2, kSwiglu>;
    const int n0 = blockIdx.x * W::kN;
    uint8_t *const base = lds + wave * FewLds::kWave;
    const W w(g, t.e, n0, base, lane);
    if (wave < KB) w.copy(wave);
    // lane 16r + p reads values 16p .. of row r (the last row again behind the end)
    const float *xr = x + static_cast<size_t>(max(pair_of(g, t, quarter), 0) / g.x_div) * g.K + c16 * 16;
    float4 xv[4];
    const auto load_x = [&](int b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const float4 *>(xr + static_cast<size_t>(b) * kBlockWeights + i * 4);
    };
    if (wave < KB) load_x(wave);
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const int arow = min(c16, kFewRows - 1);
    for (int b = wave; b < KB; b += WAVES) {
        stage_few(xv, lane, base);
        wait_all();  // W has arrived, x is staged (both this wave's own)
        WBlock wb[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) wb[c] = load_block(base + (c * 16 + c16) * kBlockBytes, 0, quarter);
        wait_lds();  // W is in registers: its slot may be filled again
        if (b + WAVES < KB) {
            w.copy(b + WAVES);
            load_x(b + WAVES);
        }
        WScales ws[2];
        float4v blk[2][2], cm[2];
        const uint4 sm = *reinterpret_cast<const uint4 *>(base + FewLds::kSumsAt + arow * kSumsBlock + (quarter & 1) * 16);
        const half8 am = __builtin_bit_cast(half8, quarter < 2 ? sm : uint4{0, 0, 0, 0});
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            ws[c] = block_scales(wb[c].head, quarter);
            cm[c] = mfma(am, ws[c].mins, float4v{0.f, 0.f, 0.f, 0.f});
            blk[c][0] = blk[c][1] = float4v{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);  // the operands of one pair of steps in registers at a time
            half8 a[4];
#pragma unroll
            for (int s = 0; s < 4; ++s)
                a[s] = *reinterpret_cast<const half8 *>(base + FewLds::kXAt + arow * kImageBlock + (4 * i + s) * 64 + (quarter ^ arow) * 16);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 qq = i < 2 ? wb[c].q0 : wb[c].q1;
                const uint32_t u = i & 1 ? qq.z : qq.x, v = i & 1 ? qq.w : qq.y;
                const half8 low = operand(u, v, ws[c], 0), high = operand(u, v, ws[c], 1);
                blk[c][0] = mfma(a[0], low, blk[c][0]);
                blk[c][1] = mfma(a[2], high, blk[c][1]);
                blk[c][0] = mfma(a[1], low, blk[c][0]);
                blk[c][1] = mfma(a[3], high, blk[c][1]);
            }
        }
        const float4 back = *reinterpret_cast<const float4 *>(base + FewLds::kBackAt);
        const float bk[4] = {back.x, back.y, back.z, back.w};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float d = ws[c].d * kBackFirst, nm = ws[c].nm * kBackFirst;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[c][r] = __builtin_fmaf(bk[r], __builtin_fmaf(nm, cm[c][r], d * (blk[c][0][r] + blk[c][1][r])), acc[c][r]);
        }
        asm volatile("" ::: "memory");
    }
    // rows 0..3 of the tile are in lanes 0..15 (column c16): join the waves
    float *red = reinterpret_cast<float *>(base);
    asm volatile("" ::: "memory");
    if (quarter == 0) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[(c * 4 + r) * 16 + c16] = acc[c][r];
    }
    __syncthreads();
    if (threadIdx.x >= 128) return;
    const int c = threadIdx.x >> 6, r = (threadIdx.x >> 4) & 3;  // column tile and row of this thread's output
    if ((kSwiglu && c) || r >= t.count) return;
    const int p = pair_of(g, t, r);
    const int n = n0 + 16 * c + c16;
    if (n >= g.N || p < 0) return;
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const float *part = reinterpret_cast<const float *>(lds + w * FewLds::kWave);
        s[0] += part[(c * 4 + r) * 16 + c16];
        if (kSwiglu) s[1] += part[(4 + r) * 16 + c16];
    }
    g.y[static_cast<size_t>(p) * g.N + n] = kSwiglu ? swiglu(s[0], s[1]) : s[0];
}

// out[m, n] = sum_j weight[m, j] * y[m * top_k + j, n] over the choices with a
// valid expert, in ascending j; a thread holds four columns and requests eight
// choices' values before it adds the first.  Bound by memory: 1024 x 8 rows of
// 2048 (75 MB, mostly still in the last-level cache) 13.5 us.
typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));  // rows of odd N start anywhere
__global__ __launch_bounds__(256) void combine_kernel(const float *y, const int *expert, const float *weight,
                                                      float *out, int E, int M, int top_k, int N) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
    if (n >= N) return;
    for (int m = blockIdx.y; m < M; m += gridDim.y) {
        float4u acc = {0.f, 0.f, 0.f, 0.f};
        const size_t p0 = static_cast<size_t>(m) * top_k;
        for (int j0 = 0; j0 < top_k; j0 += 8) {
            // every choice's values are requested, and dropped where it has no expert
            float4u v[8];
            float w[8];
            bool use[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const size_t p = p0 + min(j0 + i, top_k - 1);
                const float *src = y + p * N + n;
                if (n + 4 <= N) v[i] = *reinterpret_cast<const float4u *>(src);
                else
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][k] = src[min(k, N - 1 - n)];
                use[i] = j0 + i < top_k && static_cast<unsigned>(expert[p]) < static_cast<unsigned>(E);
                w[i] = weight[p];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k] = use[i] ? __builtin_fmaf(w[i], v[i][k], acc[k]) : acc[k];
        }
        float *o = out + static_cast<size_t>(m) * N + n;
        if (n + 4 <= N) *reinterpret_cast<float4u *>(o) = acc;
        else
            for (int k = 0; k < 3; ++k)
                if (n + k < N) o[k] = acc[k];
    }
}

bool misaligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int status(hipError_t err) {
    if (err == hipErrorOutOfMemory || err == hipErrorMemoryAllocation) return Q4K_ERR_ALLOC;
    return err == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}

int check_sizes(int E, int P, int N, int K) {
    if (E < 1 || E > Q4K_MAX_EXPERTS || P < 0 || N < 0 || K < 0) return Q4K_ERR_BAD_DIM;
    if (P == 0 || N == 0) return Q4K_OK;
    // 32 rows of W are addressed as one buffer of 32-bit offsets
    if (K == 0 || K % kBlockWeights != 0 || K > (1 << 26)) return Q4K_ERR_BAD_DIM;
    return Q4K_OK;
}

int check_grouped(const void *w, const void *w2, const float *x, int x_div, const int *offsets, const int *rows,
                  const float *y, int E, int P, int N, int K) {
    const int rc = check_sizes(E, P, N, K);
    if (rc != Q4K_OK) return rc;
    if (x_div < 1) return Q4K_ERR_BAD_DIM;
    if (P == 0 || N == 0) return Q4K_OK;
    if (!w || !w2 || !x || !offsets || !y) return Q4K_ERR_NULL;
    if (misaligned(w, 16) || misaligned(w2, 16) || misaligned(x, 16) || misaligned(y, 16) || misaligned(offsets, 4) ||
        misaligned(rows, 4))
        return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

enum class Variant { kFew = kFewRows, kThin = 16, kTile = 32, kLargeTile = 48 };  // the rows of a tile

// The kernel for a call, and the parts its workgroups split K into, from what
// the host knows (the groups' sizes are on the device): P pairs over E experts.  Expected times in us, of a pair of
// expected tile counts: with the pairs spread evenly E (1 - exp(-P / E))
// experts are in use, and tiles of r rows are that many and one more for every
// r pairs above half a tile each.  The unit of work is a super-block of one
// column tile; the rates are those measured with the card full (tiles of 16
// rows are then bound by W's 4.6 TB/s), the other side of each maximum is one
// tile's own time over its K blocks, and 5 us is the staging launch that tiles
// of four rows do without.  Measured, rows of four / of sixteen / of 32 rows by
// 128 columns, in us:
//     64 experts of 1024 x 2048 (SwiGLU), 8 pairs a token: 1 token 8 / 13 / 18,
//         4 tokens 24 / 21 / 23, 64 tokens 105 / 41 / 38, 256 tokens 343 / 72 / 64
//     16 experts of 4096 x 2048, 2 pairs: 8 tokens 18 / 21 / 22, 128 tokens
//         96 / 31 / 34, 256 tokens 176 / 41 / 42
//     40 experts of 50 x 2560, 5 pairs, 242 tokens: 16 / 25 / 35
// From 64 pairs per expert, and where that gives four workgroups to every CU
// (two rounds of them), 48 rows by 256 columns; in us, against 32 by 128:
//     64 experts of 1024 x 2048 (SwiGLU): 64 rows each 105 against 101, 128
//         rows 165 / 173, 256 rows 302 / 321
//     16 experts of 4096 x 2048: 128 rows each (811 workgroups) 105 / 96, 192
//         (1152) 134 / 138, 256 rows 165 / 187, 500 rows 302 / 339
//     2 experts of 2000 x 4096: 1000 rows each 101 / 93
Variant choose(int pairs, int experts, int N, int K, bool swiglu, int *parts) {
    const double P = pairs, E = experts, KB = K / kBlockWeights, columns = swiglu ? 2.0 * N : N;
    const double used = P <= E / 8 ? P : E * (1.0 - exp(-P / E));
    const auto tiles = [&](double rows) { return used + fmax(0.0, P / rows - 0.5 * used); };
    const double thin_workgroups = tiles(16) * ceil(columns / 128);
    const int groups = thin_workgroups <= 256 && KB >= 4 ? 4 : thin_workgroups <= 512 && KB >= 2 ? 2 : 1;
    const double few = tiles(4) * ceil(columns / 32) * KB / 750;
    const double thin = fmax(thin_workgroups * KB / 250, 3.0 * KB / groups);
    const double tile = fmax(tiles(32) * ceil(columns / 128) * KB / 158, 1.9 * KB);
    *parts = KB > 4 ? 8 : 4;
    if (few < 5 + fmin(thin, tile) && tiles(4) < 16384) return Variant::kFew;
    *parts = 1;
    if (P >= 64 * E && (P / 48 + 0.5 * E) * columns / 256 >= 1024) return Variant::kLargeTile;
    if (thin > tile) return Variant::kTile;
    *parts = groups;
    return Variant::kThin;
}

// No call has more tiles of `rows` rows: every group has at most one that is not
// full, and every tile has a pair.
int most_tiles(const Grouped &g, int rows) {
    const int64_t tiles = static_cast<int64_t>(g.P) / rows + (g.E < g.P ? g.E : g.P);
    return static_cast<int>(tiles < g.P ? tiles : g.P);
}

template <int WAVES, bool kSwiglu>
hipError_t launch_few(const Grouped &g, const float *x, hipStream_t stream) {
    constexpr int kBytes = WAVES * FewLds::kWave, kTileN = kSwiglu ? 16 : 32;
    const hipError_t err = allow_dynamic_lds(reinterpret_cast<const void *>(few_kernel<WAVES, kSwiglu>), kBytes);
    if (err != hipSuccess) return err;
    const dim3 grid((g.N - 1) / kTileN + 1, most_tiles(g, kFewRows));
    hipLaunchKernelGGL((few_kernel<WAVES, kSwiglu>), grid, dim3(64 * WAVES), kBytes, stream, g, x);
    return hipGetLastError();
}

hipError_t launch_tiles(void (*kernel)(Grouped), const Grouped &g, int rows, int cols, int threads, int bytes,
                        hipStream_t stream) {
    const hipError_t err = allow_dynamic_lds(reinterpret_cast<const void *>(kernel), bytes);
    if (err != hipSuccess) return err;
    const int64_t tiles = most_tiles(g, rows);
    const int64_t blocks = (tiles * ((g.N - 1) / cols + 1) + 7) / 8 * 8;
    if (blocks > INT_MAX) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), bytes, stream, g);
    return hipGetLastError();
}
template <int RT, int NC>
hipError_t launch_tile(const Grouped &g, hipStream_t stream) {
    constexpr int kBytes = TileLds<RT, NC>::kBytes;
    if (g.w2) return launch_tiles(tile_kernel<RT, NC, true>, g, RT * 16, 4 * WTile<NC, true>::kN, 256, kBytes, stream);
    return launch_tiles(tile_kernel<RT, NC, false>, g, RT * 16, 4 * WTile<NC, false>::kN, 256, kBytes, stream);
}
template <int NC, int KS>
hipError_t launch_thin(const Grouped &g, hipStream_t stream) {
    constexpr int kBytes = ThinLds<NC>::bytes(KS);
    if (g.w2) return launch_tiles(thin_kernel<NC, KS, true>, g, 16, 4 * WTile<NC, true>::kN, 256 * KS, kBytes, stream);
    return launch_tiles(thin_kernel<NC, KS, false>, g, 16, 4 * WTile<NC, false>::kN, 256 * KS, kBytes, stream);
}

// Stages x, then the products.  g.x is filled in here.
hipError_t run_grouped(Grouped g, const float *x, hipStream_t stream) {
    const size_t xrows = (static_cast<size_t>(g.P) + g.x_div - 1) / g.x_div, KB = g.K / kBlockWeights;
    int parts = 1;
    const Variant variant = choose(g.P, g.E, g.N, g.K, g.w2 != nullptr, &parts);
    if (variant == Variant::kFew) {
        if (g.w2) return parts == 8 ? launch_few<8, true>(g, x, stream) : launch_few<4, true>(g, x, stream);
        return parts == 8 ? launch_few<8, false>(g, x, stream) : launch_few<4, false>(g, x, stream);
    }
    float *ws = nullptr;
    hipError_t err = workspace(stream, xrows * (KB * (kImageBlock + kSumsBlock) + 16), &ws);
    if (err != hipSuccess) return err;
    uint8_t *img = reinterpret_cast<uint8_t *>(ws), *sums = img + xrows * KB * kImageBlock;
    float *back = reinterpret_cast<float *>(sums + xrows * KB * kSumsBlock);
    g.x = {img, sums, back};
    const int threads = g.K >= 8 * kStageThreads ? kStageThreads : (g.K / 8 + 63) / 64 * 64;
    hipLaunchKernelGGL(stage_rows_kernel, dim3(static_cast<unsigned>(xrows)), dim3(threads), 0, stream, x, g.K, img,
                       sums, back);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    switch (variant) {
    case Variant::kThin:
        return parts == 4   ? launch_thin<2, 4>(g, stream)
               : parts == 2 ? launch_thin<2, 2>(g, stream)
                            : launch_thin<2, 1>(g, stream);
    case Variant::kTile: return launch_tile<2, 2>(g, stream);
    default: return launch_tile<3, 4>(g, stream);
    }
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_grouped_tile(int E, int P, int N, int K, int swiglu, int *parts) {
    using namespace q4k;
    if (parts) *parts = 0;
    const int rc = check_sizes(E, P, N, K);
    if (rc != Q4K_OK || P == 0 || N == 0) return rc;
    int split = 1;
    const int rows = static_cast<int>(choose(P, E, N, K, swiglu != 0, &split));
    if (parts) *parts = split;
    return rows;
}

extern "C" int q4k_matmul_grouped(const void *w_packed, const float *x, int x_div, const int *offsets,
                                  const int *rows, float *y, int E, int P, int N, int K, hipStream_t stream) {
    using namespace q4k;
    int rc = check_grouped(w_packed, w_packed, x, x_div, offsets, rows, y, E, P, N, K);
    if (rc != Q4K_OK || P == 0 || N == 0) return rc;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    return status(run_grouped({static_cast<const uint8_t *>(w_packed), nullptr, {}, offsets, rows, y, E, P, N, K, x_div},
                              x, stream));
}

extern "C" int q4k_matmul_grouped_swiglu(const void *w_gate, const void *w_up, const float *x, int x_div,
                                         const int *offsets, const int *rows, float *out, int E, int P, int N,
                                         int K, hipStream_t stream) {
    using namespace q4k;
    int rc = check_grouped(w_gate, w_up, x, x_div, offsets, rows, out, E, P, N, K);
    if (rc != Q4K_OK || P == 0 || N == 0) return rc;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    return status(run_grouped({static_cast<const uint8_t *>(w_gate), static_cast<const uint8_t *>(w_up), {}, offsets,
                               rows, out, E, P, N, K, x_div},
                              x, stream));
}

extern "C" int q4k_matmul_grouped_combine(const void *w_packed, const float *x, const int *expert,
                                          const float *weight, const int *offsets, const int *rows, float *out,
                                          int E, int M, int top_k, int N, int K, hipStream_t stream) {
    using namespace q4k;
    if (M < 0 || top_k < 1 || static_cast<int64_t>(M) * top_k > INT_MAX) return Q4K_ERR_BAD_DIM;
    const int P = M * top_k;
    int rc = check_grouped(w_packed, w_packed, x, 1, offsets, rows, out, E, P, N, K);
    if (rc != Q4K_OK || P == 0 || N == 0) return rc;
    if (!rows || !expert || !weight) return Q4K_ERR_NULL;
    if (misaligned(expert, 4) || misaligned(weight, 4)) return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    float *y = nullptr;
    if (workspace(stream, static_cast<size_t>(P) * N * sizeof(float), &y, 1) != hipSuccess) return Q4K_ERR_ALLOC;
    hipError_t err = run_grouped({static_cast<const uint8_t *>(w_packed), nullptr, {}, offsets, rows, y, E, P, N, K, 1},
                                 x, stream);
    if (err != hipSuccess) return status(err);
    hipLaunchKernelGGL(combine_kernel, dim3((N - 1) / 1024 + 1, M < 65535 ? M : 65535), dim3(256), 0, stream, y, expert,
                       weight, out, E, M, top_k, N);
    return status(hipGetLastError());
}
