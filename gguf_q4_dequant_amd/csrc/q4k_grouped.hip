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
//     error below 2^-40 of the row's maximum where lo is subnormal.  Both
//     enter the same fp32 accumulator: two v_mfma_f32_16x16x32_f16 per 32
//     weights, half the binary16 matrix rate at fp32 accuracy.
//   * The min term is one more MFMA per super-block: the eight X_j (hi and lo
//     in k-quarters 0 and 1) times the eight m_j as subnormals.
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
    const float *back;    // [rows]: 2^(24 - e)
};

// The e of the scale 2^e that puts a largest magnitude mx in [2^14, 2^15),
// limited so that 2^e and 2^(24 - e) are normal (zeros and subnormals: 127,
// infinity and NaN: 0).
__device__ __forceinline__ int scale_exponent(float mx) {
    const int E = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFFu);
    const int e = E == 0 ? 127 : (E == 255 ? 0 : 141 - E);
    return max(-103, min(127, e));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Stages one row of x per workgroup (see above): thread u takes eight
// consecutive values at a time.
__global__ __launch_bounds__(256) void stage_rows_kernel(const float *x, int K, uint8_t *img, uint8_t *sums,
                                                         float *back) {
    __shared__ float wave_mx[4];
    const size_t row = blockIdx.x;
    const float *xr = x + row * K;
    float mx = 0.f;
    for (int k = threadIdx.x * 8; k < K; k += 256 * 8) {
        const float4 a = *reinterpret_cast<const float4 *>(xr + k), b = *reinterpret_cast<const float4 *>(xr + k + 4);
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))));
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
    if ((threadIdx.x & 63) == 0) wave_mx[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(wave_mx[0], wave_mx[1]), fmaxf(wave_mx[2], wave_mx[3]));
    const int e = scale_exponent(mx);
    const float up = power_of_two(e);
    if (threadIdx.x == 0) back[row] = power_of_two(24 - e);
    uint8_t *im = img + row * (K / kBlockWeights) * kImageBlock;
    uint8_t *sm = sums + row * (K / kBlockWeights) * kSumsBlock;
    for (int k = threadIdx.x * 8; k < K; k += 256 * 8) {
        const float4 a = *reinterpret_cast<const float4 *>(xr + k), b = *reinterpret_cast<const float4 *>(xr + k + 4);
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        constexpr int order[8] = {0, 2, 1, 3, 4, 6, 5, 7};
        half8 hi, lo;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float t = v[order[i]] * up;
            hi[i] = static_cast<_Float16>(t);
            lo[i] = static_cast<_Float16>(t - static_cast<float>(hi[i]));
            s += v[i] * up;
        }
        const int blk = k / kBlockWeights, in = k % kBlockWeights;
        const int quarter = in >> 6, h = (in >> 5) & 1, i = (in >> 3) & 3;
        uint8_t *o = im + blk * kImageBlock + (2 * i + h) * 128 + quarter * 16;
        *reinterpret_cast<half8 *>(o) = hi;
        *reinterpret_cast<half8 *>(o + 64) = lo;
        // the sub-block's sum over its four threads (32 values below 2^15
        // each), times 2^-6 to stay in binary16's range
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

// Tile number t of the groups cut into tiles of TM rows (count 0: no such
// tile).  Every wave scans the offsets by itself, 64 experts at a time.
template <int TM>
__device__ __forceinline__ Tile find_tile(const int *offsets, int E, int P, int t, int lane) {
    int done = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        int b = 0, c = 0;
        if (e0 + lane < E) {
            b = min(max(offsets[e0 + lane], 0), P);
            c = max(min(offsets[e0 + lane + 1], P) - b, 0);
        }
        const int tiles = (c + TM - 1) / TM;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int up = __shfl_up(incl, o);
            incl += lane >= o ? up : 0;
        }
        const uint64_t past = __ballot(done + incl > t);
        if (past != 0) {
            const int owner = __builtin_ctzll(past);
            const int begin = __builtin_amdgcn_readlane(b, owner), all = __builtin_amdgcn_readlane(c, owner);
            const int at = t - done - (__builtin_amdgcn_readlane(incl, owner) - __builtin_amdgcn_readlane(tiles, owner));
            return {e0 + owner, begin + at * TM, min(TM, all - at * TM)};
        }
        done += __builtin_amdgcn_readlane(incl, 63);
    }
    return {0, 0, 0};
}

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
    float d, nm;    // d, -64 * dmin
    half2v s0, s1;  // the lane's two scales, the second / 16 (its nibbles are 16q)
    half8 mins;     // m_0..m_7 as subnormals m * 2^-24
};
__device__ __forceinline__ WScales block_scales(const uint4 hd, int quarter) {
    WScales s;
    s.d = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hd.x & 0xFFFFu)));
    s.nm = -64.f * static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(hd.x >> 16)));
    const uint32_t scA = hd.y & 0x3F3F3F3Fu, mnA = hd.z & 0x3F3F3F3Fu;
    const uint32_t scB = (hd.w & 0x0F0F0F0Fu) | ((hd.y >> 2) & 0x30303030u);
    const uint32_t mnB = ((hd.w >> 4) & 0x0F0F0F0Fu) | ((hd.z >> 2) & 0x30303030u);
    const uint32_t two = (quarter & 2 ? scB : scA) >> (16 * (quarter & 1));
    const _Float16 a = static_cast<_Float16>(static_cast<float>(two & 0xFFu));
    const _Float16 b = static_cast<_Float16>(0.0625f * static_cast<float>((two >> 8) & 0xFFu));
    s.s0 = half2v{a, a};
    s.s1 = half2v{b, b};
    uint4 m;
    m.x = (mnA & 0xFFu) | ((mnA & 0xFF00u) << 8);
    m.y = ((mnA >> 16) & 0xFFu) | ((mnA >> 8) & 0xFF0000u);
    m.z = (mnB & 0xFFu) | ((mnB & 0xFF00u) << 8);
    m.w = ((mnB >> 16) & 0xFFu) | ((mnB >> 8) & 0xFF0000u);
    s.mins = __builtin_bit_cast(half8, m);
    return s;
}

// The operands of steps 2i (low nibbles) and 2i + 1 (high) from two dwords.
__device__ __forceinline__ half2v scaled(uint32_t bits, half2v s) { return __builtin_bit_cast(half2v, bits) * s; }
__device__ __forceinline__ half8 join(half2v a, half2v b, half2v c, half2v d) {
    return half8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ void operands(uint32_t u, uint32_t v, const WScales &s, half8 &low, half8 &high) {
    const uint32_t LM = 0x000F000Fu, HM = 0x00F000F0u;
    const uint32_t u8 = u >> 8, v8 = v >> 8;
    low = join(scaled(u & LM, s.s0), scaled(u8 & LM, s.s0), scaled(v & LM, s.s0), scaled(v8 & LM, s.s0));
    high = join(scaled(u & HM, s.s1), scaled(u8 & HM, s.s1), scaled(v & HM, s.s1), scaled(v8 & HM, s.s1));
}

// The operand of one of the two steps.
__device__ __forceinline__ void operand(uint32_t u, uint32_t v, const WScales &s, int h, half8 &op) {
    const uint32_t mask = h ? 0x00F000F0u : 0x000F000Fu;
    const half2v sc = h ? s.s1 : s.s0;
    op = join(scaled(u & mask, sc), scaled((u >> 8) & mask, sc), scaled(v & mask, sc), scaled((v >> 8) & mask, sc));
}

__device__ __forceinline__ float4v mfma(half8 a, half8 b, float4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// 16 rows of x times 32 rows of W (SwiGLU: 16 gate and the same 16 up rows)
// per wave, four waves side by side; operands straight from memory.
template <bool kSwiglu>
__global__ __launch_bounds__(256) void grouped_kernel(Grouped g) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, quarter = lane >> 4;
    const Tile t = find_tile<16>(g.offsets, g.E, g.P, blockIdx.y, lane);
    if (t.count == 0) return;
    constexpr int kWaveN = kSwiglu ? 16 : 32;
    const int n0 = (blockIdx.x * 4 + wave) * kWaveN;
    if (n0 >= g.N) return;
    const int KB = g.K / kBlockWeights;
    const size_t row_bytes = static_cast<size_t>(KB) * kBlockBytes;
    const uint8_t *wrow[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int n = min(n0 + (kSwiglu ? 0 : 16 * c) + c16, g.N - 1);
        wrow[c] = (kSwiglu && c ? g.w2 : g.w) + (static_cast<size_t>(t.e) * g.N + n) * row_bytes;
    }
    // this lane's row of x as the A operand: row c16 of the tile (the last one again behind the end)
    const auto pair_at = [&](int i) {
        const int at = t.first + min(i, t.count - 1);
        return g.rows ? g.rows[at] : at;
    };
    int pair = pair_at(c16);
    pair = static_cast<unsigned>(pair) < static_cast<unsigned>(g.P) ? pair : 0;
    const size_t xr = pair / g.x_div;
    const uint8_t *img = g.x.img + xr * KB * kImageBlock + quarter * 16;
    const uint8_t *sums = g.x.sums + xr * KB * kSumsBlock + (quarter & 1) * 16;
    float4v acc[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < KB; ++b) {
        WBlock wb[2];
        WScales ws[2];
        float4v blk[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            wb[c] = load_block(wrow[c], b, quarter);
            blk[c] = float4v{0.f, 0.f, 0.f, 0.f};
        }
        half8 a[16];
#pragma unroll
        for (int s = 0; s < 16; ++s) a[s] = *reinterpret_cast<const half8 *>(img + b * kImageBlock + s * 64);
        const uint4 sm = *reinterpret_cast<const uint4 *>(sums + b * kSumsBlock);
        const half8 am = __builtin_bit_cast(half8, quarter < 2 ? sm : uint4{0, 0, 0, 0});
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            ws[c] = block_scales(wb[c].head, quarter);
            const uint32_t q[8] = {wb[c].q0.x, wb[c].q0.y, wb[c].q0.z, wb[c].q0.w,
                                   wb[c].q1.x, wb[c].q1.y, wb[c].q1.z, wb[c].q1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                half8 low, high;
                operands(q[2 * i], q[2 * i + 1], ws[c], low, high);
                blk[c] = mfma(a[4 * i + 0], low, blk[c]);
                blk[c] = mfma(a[4 * i + 1], low, blk[c]);
                blk[c] = mfma(a[4 * i + 2], high, blk[c]);
                blk[c] = mfma(a[4 * i + 3], high, blk[c]);
            }
            const float4v cm = mfma(am, ws[c].mins, float4v{0.f, 0.f, 0.f, 0.f});
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[c][r] = __builtin_fmaf(ws[c].nm, cm[r], __builtin_fmaf(ws[c].d, blk[c][r], acc[c][r]));
        }
    }
    // lane l holds rows 4 * (l / 16) + r of the tile for column l % 16
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 4 * quarter + r;
        const int p = pair_at(i);
        if (i >= t.count || static_cast<unsigned>(p) >= static_cast<unsigned>(g.P)) continue;
        const float back = g.x.back[p / g.x_div];
        float *yr = g.y + static_cast<size_t>(p) * g.N;
        if (kSwiglu) {
            if (n0 + c16 < g.N) yr[n0 + c16] = swiglu(acc[0][r] * back, acc[1][r] * back);
        } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (n0 + 16 * c + c16 < g.N) yr[n0 + 16 * c + c16] = acc[c][r] * back;
        }
    }
}

// ---- many rows per expert: tiles of RT * 16 rows times 256 columns ----------

// LDS of a workgroup: two buffers of x (a quarter of a super-block: two steps,
// 256 bytes a row), two of its sub-block sums, one super-block of each wave's
// own 64 rows of W, and the tile's pair numbers.
template <int RT>
struct TileLds {
    static constexpr int kRows = RT * 16;
    static constexpr int kX = kRows * 256, kSums = kRows * kSumsBlock, kW = 64 * kBlockBytes;
    static constexpr int kSumsAt = 2 * kX, kWAt = kSumsAt + 2 * kSums, kPairsAt = kWAt + 4 * kW;
    static constexpr int kBytes = kPairsAt + kRows * 4;
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
__device__ __forceinline__ void copy_to_lds(const uint8_t *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(dst) : "memory");
}
// The same from a buffer (offsets behind its end read zeros).
__device__ __forceinline__ void copy_to_lds(rsrc_t buffer, uint32_t offset, uint32_t base, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(offset), "s"(buffer),
                 "s"(base), "s"(dst)
                 : "memory");
}
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

// At most VM vector-memory operations of this wave outstanding and no LDS
// operation, then the workgroup's barrier.
template <int VM>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (VM & 15));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int RT, bool kSwiglu>
__global__ __launch_bounds__(256, 2) void tile_kernel(Grouped g) {
    using L = TileLds<RT>;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, quarter = lane >> 4;
    const Tile t = find_tile<L::kRows>(g.offsets, g.E, g.P, blockIdx.y, lane);
    if (t.count == 0) return;
    int *pairs = reinterpret_cast<int *>(lds + L::kPairsAt);
    if (threadIdx.x < L::kRows) {
        const int at = t.first + min(static_cast<int>(threadIdx.x), t.count - 1);
        const int p = g.rows ? g.rows[at] : at;
        pairs[threadIdx.x] = static_cast<unsigned>(p) < static_cast<unsigned>(g.P) ? p : -1;
    }
    __syncthreads();
    const int KB = g.K / kBlockWeights;
    const size_t row_bytes = static_cast<size_t>(KB) * kBlockBytes;
    constexpr int kWaveN = kSwiglu ? 32 : 64;
    const int n0 = (blockIdx.x * 4 + wave) * kWaveN;

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
    // W: two halves of 32 rows, 288 pieces of 16 bytes each (4.5 instructions);
    // row 16c + r of the wave's 64 is column r of its tile c (SwiGLU: the
    // halves are gate and up).  Rows behind N read zeros.
    uint32_t woff[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        const int piece = k * 64 + lane, j = piece / 9, part = piece - 9 * j;
        woff[k] = j * static_cast<uint32_t>(row_bytes) + part * 16;
    }
    rsrc_t wbuf[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int first = min(n0 + (kSwiglu ? 0 : 32 * h), g.N), rows = min(32, g.N - first);
        wbuf[h] = buffer_at((kSwiglu && h ? g.w2 : g.w) + (static_cast<size_t>(t.e) * g.N + first) * row_bytes,
                            rows * static_cast<uint32_t>(row_bytes));
    }
    uint8_t *const wlds = lds + L::kWAt + wave * L::kW;
    const uint32_t lds0 = lds_address(lds), wlds0 = lds0 + L::kWAt + wave * L::kW;
    const auto copy_x = [&](int b, int i, int buf) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
            copy_to_lds(xsrc[j] + (static_cast<size_t>(b) * kImageBlock + i * 256), lds0 + buf * L::kX + (wave * RT + j) * 1024);
    };
    const auto copy_sums = [&](int b) {
        if (lane < RT * 8)
            copy_to_lds(ssrc + static_cast<size_t>(b) * kSumsBlock, lds0 + L::kSumsAt + (b & 1) * L::kSums + wave * RT * 128);
    };
    const auto copy_w = [&](int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (k < 4 || lane < 32)
                    copy_to_lds(wbuf[h], woff[k], b * kBlockBytes, wlds0 + h * (L::kW / 2) + k * 1024);
    };
    float4v acc[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
    copy_w(0);
    copy_x(0, 0, 0);
    copy_sums(0);
    for (int b = 0; b < KB; ++b) {
        WScales ws[4];
        float4v blk[RT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // x of this quarter has arrived; the others' too behind the barrier
            wait_and_barrier<0>();
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
                for (int c = 0; c < 4; ++c) {
                    __builtin_amdgcn_sched_barrier(0);
                    ws[c] = block_scales(*reinterpret_cast<const uint4 *>(wlds + (c * 16 + c16) * kBlockBytes), quarter);
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
                        const float4v cm = mfma(am[r], ws[c].mins, float4v{0.f, 0.f, 0.f, 0.f});
                        blk[r][c] = float4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[r][c][k] = __builtin_fmaf(ws[c].nm, cm[k], acc[r][c][k]);
                    }
                }
            }
            uint2 q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                q[c] = *reinterpret_cast<const uint2 *>(wlds + (c * 16 + c16) * kBlockBytes + 16 + 32 * quarter + 8 * i);
            if (i == 3 && b + 1 < KB) {
                // every read of this wave's W slot has returned: refill it
                asm volatile("" ::: "memory");
                __builtin_amdgcn_s_waitcnt(0xC07F);
                copy_w(b + 1);
            }
            const uint8_t *xb = lds + (i & 1) * L::kX;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __builtin_amdgcn_sched_barrier(0);  // one step's operands in registers at a time
                half8 a[RT][2];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        a[r][part] = *reinterpret_cast<const half8 *>(
                            xb + (r * 16 + c16) * 256 + (((h * 2 + part) * 4 + quarter) ^ c16) * 16);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    half8 op;
                    operand(q[c].x, q[c].y, ws[c], h, op);
#pragma unroll
                    for (int r = 0; r < RT; ++r) blk[r][c] = mfma(a[r][0], op, blk[r][c]);
#pragma unroll
                    for (int r = 0; r < RT; ++r) blk[r][c] = mfma(a[r][1], op, blk[r][c]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[r][c][k] = __builtin_fmaf(ws[c].d, blk[r][c][k], acc[r][c][k]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = r * 16 + 4 * quarter + k;
            const int p = pairs[i];
            if (i >= t.count || p < 0) continue;
            const float back = g.x.back[p / g.x_div];
            float *yr = g.y + static_cast<size_t>(p) * g.N;
            if (kSwiglu) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (n0 + 16 * c + c16 < g.N)
                        yr[n0 + 16 * c + c16] = swiglu(acc[r][c][k] * back, acc[r][2 + c][k] * back);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n0 + 16 * c + c16 < g.N) yr[n0 + 16 * c + c16] = acc[r][c][k] * back;
            }
        }
}

// ---- few rows per expert -----------------------------------------------------

// Four rows of x times 32 rows of W (SwiGLU: 16 gate and the same 16 up rows)
// per workgroup; the waves split K by super-blocks, each with its own LDS:
// one super-block of the 32 rows of W, the staged x and its factors.
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
// 16p .. 16p + 15 of row r.  The scale is per row and super-block here, so
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
        uint8_t *o = base + FewLds::kXAt + r * kImageBlock + (2 * i + h) * 128 + quarter * 16;
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
    if (p == 0) reinterpret_cast<float *>(base + FewLds::kBackAt)[r] = power_of_two(24 - e);
}

template <int WAVES, bool kSwiglu>
__global__ __launch_bounds__(64 * WAVES, 4) void few_kernel(Grouped g, const float *x) {
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c16 = lane & 15, quarter = lane >> 4;
    const Tile t = find_tile<kFewRows>(g.offsets, g.E, g.P, blockIdx.y, lane);
    if (t.count == 0) return;
    const auto pair_at = [&](int i) {
        const int at = t.first + min(i, t.count - 1);
        return g.rows ? g.rows[at] : at;
    };
    const int KB = g.K / kBlockWeights;
    const size_t row_bytes = static_cast<size_t>(KB) * kBlockBytes;
    constexpr int kTileN = kSwiglu ? 16 : 32;
    const int n0 = blockIdx.x * kTileN;
    uint8_t *const base = lds + wave * FewLds::kWave;
    const uint32_t wlds = lds_address(base);
    // two halves of 16 rows (SwiGLU: gate and up), 144 pieces of 16 bytes each
    uint32_t woff[3];
    rsrc_t wbuf[2];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int piece = k * 64 + lane, j = piece / 9, part = piece - 9 * j;
        woff[k] = j * static_cast<uint32_t>(row_bytes) + part * 16;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int first = min(n0 + (kSwiglu ? 0 : 16 * h), g.N), rows = min(16, g.N - first);
        wbuf[h] = buffer_at((kSwiglu && h ? g.w2 : g.w) + (static_cast<size_t>(t.e) * g.N + first) * row_bytes,
                            rows * static_cast<uint32_t>(row_bytes));
    }
    const auto copy_w = [&](int b) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (k < 2 || lane < 16)
                    copy_to_lds(wbuf[h], woff[k], b * kBlockBytes, wlds + h * (FewLds::kW / 2) + k * 1024);
    };
    if (wave < KB) copy_w(wave);
    // lane 16r + p reads values 16p .. of row r (the last row again behind the end)
    int pair = pair_at(quarter);
    pair = static_cast<unsigned>(pair) < static_cast<unsigned>(g.P) ? pair : 0;
    const float *xr = x + static_cast<size_t>(pair / g.x_div) * g.K + c16 * 16;
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
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);  // W has arrived, x is staged (both this wave's own)
        asm volatile("" ::: "memory");
        WBlock wb[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) wb[c] = load_block(base + (c * 16 + c16) * kBlockBytes, 0, quarter);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);  // W is in registers: its slot may be filled again
        if (b + WAVES < KB) {
            copy_w(b + WAVES);
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
                a[s] = *reinterpret_cast<const half8 *>(base + FewLds::kXAt + arow * kImageBlock + (4 * i + s) * 64 + quarter * 16);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const uint4 qq = i < 2 ? wb[c].q0 : wb[c].q1;
                const uint32_t u = i & 1 ? qq.z : qq.x, v = i & 1 ? qq.w : qq.y;
                half8 low, high;
                operand(u, v, ws[c], 0, low);
                operand(u, v, ws[c], 1, high);
                blk[c][0] = mfma(a[0], low, blk[c][0]);
                blk[c][1] = mfma(a[2], high, blk[c][1]);
                blk[c][0] = mfma(a[1], low, blk[c][0]);
                blk[c][1] = mfma(a[3], high, blk[c][1]);
            }
        }
        const float4 back = *reinterpret_cast<const float4 *>(base + FewLds::kBackAt);
        const float bk[4] = {back.x, back.y, back.z, back.w};
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[c][r] = __builtin_fmaf(bk[r], __builtin_fmaf(ws[c].nm, cm[c][r], ws[c].d * (blk[c][0][r] + blk[c][1][r])),
                                           acc[c][r]);
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
    const int c = threadIdx.x >> 6, r = (threadIdx.x >> 4) & 3;
    if ((kSwiglu && c) || r >= t.count) return;
    const int p = pair_at(r);
    const int n = n0 + 16 * c + c16;
    if (n >= g.N || static_cast<unsigned>(p) >= static_cast<unsigned>(g.P)) return;
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
// valid expert, in ascending j.
__global__ __launch_bounds__(256) void combine_kernel(const float *y, const int *expert, const float *weight,
                                                      float *out, int E, int top_k, int N) {
    const int m = blockIdx.y;
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= N) return;
    float acc = 0.f;
    for (int j = 0; j < top_k; ++j) {
        const size_t p = static_cast<size_t>(m) * top_k + j;
        if (static_cast<unsigned>(expert[p]) >= static_cast<unsigned>(E)) continue;
        acc = __builtin_fmaf(weight[p], y[p * N + n], acc);
    }
    out[static_cast<size_t>(m) * N + n] = acc;
}

bool misaligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int status(hipError_t err) {
    if (err == hipErrorOutOfMemory || err == hipErrorMemoryAllocation) return Q4K_ERR_ALLOC;
    return err == hipSuccess ? Q4K_OK : Q4K_ERR_LAUNCH;
}

int check_grouped(const void *w, const void *w2, const float *x, int x_div, const int *offsets, const int *rows,
                  const float *y, int E, int P, int N, int K) {
    if (E < 1 || E > Q4K_MAX_EXPERTS || P < 0 || N < 0 || K < 0 || x_div < 1) return Q4K_ERR_BAD_DIM;
    if (P == 0 || N == 0) return Q4K_OK;
    if (K == 0 || K % kBlockWeights != 0) return Q4K_ERR_BAD_DIM;
    if (!w || !w2 || !x || !offsets || !y) return Q4K_ERR_NULL;
    if (misaligned(w, 16) || misaligned(w2, 16) || misaligned(x, 16) || misaligned(y, 16) || misaligned(offsets, 4) ||
        misaligned(rows, 4))
        return Q4K_ERR_ALIGN;
    return Q4K_OK;
}

bool few_rows(const Grouped &g) { return g.P <= 2 * g.E; }

template <int WAVES, bool kSwiglu>
hipError_t launch_few(const Grouped &g, const float *x, hipStream_t stream) {
    constexpr int kBytes = WAVES * FewLds::kWave, kTileN = kSwiglu ? 16 : 32;
    const hipError_t err = allow_dynamic_lds(reinterpret_cast<const void *>(few_kernel<WAVES, kSwiglu>), kBytes);
    if (err != hipSuccess) return err;
    const dim3 grid((g.N + kTileN - 1) / kTileN, g.P / kFewRows + (g.E < g.P ? g.E : g.P));
    hipLaunchKernelGGL((few_kernel<WAVES, kSwiglu>), grid, dim3(64 * WAVES), kBytes, stream, g, x);
    return hipGetLastError();
}

// Stages x, then the products.  g.x is filled in here.
hipError_t run_grouped(Grouped g, const float *x, hipStream_t stream) {
    const size_t xrows = (static_cast<size_t>(g.P) + g.x_div - 1) / g.x_div, KB = g.K / kBlockWeights;
    if (few_rows(g)) {
        if (g.w2) return KB > 4 ? launch_few<8, true>(g, x, stream) : launch_few<4, true>(g, x, stream);
        return KB > 4 ? launch_few<8, false>(g, x, stream) : launch_few<4, false>(g, x, stream);
    }
    float *ws = nullptr;
    hipError_t err = workspace(stream, xrows * (KB * (kImageBlock + kSumsBlock) + 16), &ws);
    if (err != hipSuccess) return err;
    uint8_t *img = reinterpret_cast<uint8_t *>(ws), *sums = img + xrows * KB * kImageBlock;
    float *back = reinterpret_cast<float *>(sums + xrows * KB * kSumsBlock);
    g.x = {img, sums, back};
    hipLaunchKernelGGL(stage_rows_kernel, dim3(static_cast<unsigned>(xrows)), dim3(256), 0, stream, x, g.K, img, sums,
                       back);
    err = hipGetLastError();
    if (err != hipSuccess) return err;
    if (g.P >= 24 * g.E) {
        const int tiles = g.P / 48 + (g.E < g.P ? g.E : g.P);
        const dim3 grid((g.N + (g.w2 ? 127 : 255)) / (g.w2 ? 128 : 256), tiles);
        const void *k = g.w2 ? reinterpret_cast<const void *>(tile_kernel<3, true>) : reinterpret_cast<const void *>(tile_kernel<3, false>);
        err = allow_dynamic_lds(k, TileLds<3>::kBytes);
        if (err != hipSuccess) return err;
        if (g.w2) hipLaunchKernelGGL((tile_kernel<3, true>), grid, dim3(256), TileLds<3>::kBytes, stream, g);
        else hipLaunchKernelGGL((tile_kernel<3, false>), grid, dim3(256), TileLds<3>::kBytes, stream, g);
        return hipGetLastError();
    }
    const int tiles = g.P / 16 + (g.E < g.P ? g.E : g.P);
    const int cols = g.w2 ? 64 : 128;
    const dim3 grid((g.N + cols - 1) / cols, tiles);
    if (g.w2) hipLaunchKernelGGL(grouped_kernel<true>, grid, dim3(256), 0, stream, g);
    else hipLaunchKernelGGL(grouped_kernel<false>, grid, dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace
}  // namespace q4k

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
    hipLaunchKernelGGL(combine_kernel, dim3((N + 255) / 256, M), dim3(256), 0, stream, y, expert, weight, out, E,
                       top_k, N);
    return status(hipGetLastError());
}
