// Attention over the paged cache (include/q4k_layer.h).
//
// Rows.  The queries of one sequence that read key head h are rows
// r = i * group + g (new token i, query head h * group + g), so that the heads of
// a group share every key and value that is loaded.  A workgroup takes a tile
// of rows and walks over the keys with the running maximum and sum of the
// softmax.
//
// Products.  Scores are computed transposed, S^T = K Q^T, and so is the output,
// O^T = V^T P^T: in the matrix instructions' layout a lane then holds scores of
// ONE row, maximum, sum and the output's correction are a lane's own numbers, and
// the scores' registers are the second product's operand as they are (the order
// of the keys within a step is free, as long as V^T is read in the same one).
// The queries (times scale, log2 e and a power of two per row) and the weights
// are float32 values split into two of 16 bits, so both products run twice:
// 8 * head_dim operations per row and key instead of 4, at float32 accuracy.
//
// Copies.  Keys and values go from memory to LDS as they are stored, 16 bytes a
// lane, one tile ahead of the products; what has no place (behind the sequence,
// a missing page, dimensions behind head_dim) is copied from a line of zeros.
// The 16-byte pieces of a row are permuted by an exclusive or with bits of the
// row, so that neither the rows read by pieces (K) nor the transposing reads (V)
// meet the same banks.  e4m3 is widened to binary16 (exactly) when it is read.
//
// What a row does not see.  Scores get -inf by a bit per key; weights are then 0,
// and 0 times a NaN or an infinity in V would be NaN.  Values behind a sequence
// are zeros, so this concerns later new tokens only: a tile that some rows see
// in part is looked through, and if it holds such a value (never, in earnest)
// its values are multiplied as zeros and the rows that see one are made NaN.
//
// Few tiles are split along the keys (find_unit): the total of key tiles is
// divided by the workgroups that fill the card, each takes at most that many of
// one sequence, and a second launch joins the parts.  The lengths stay on the
// device; every workgroup works the division out by itself.
#include <math.h>

#include "q4k_cache.h"

namespace q4k {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

struct Attend {
    Paged p;
    const float *q;
    float *out;
    const unsigned *mask;  // null: causal
    float *part;           // split: outputs of the units, [units * kv_heads][rows][head_dim] ...
    float *part_ml;        // ... and their maxima and sums, [units * kv_heads][rows][2]
    int words;
    int q_heads;
    int group;   // query heads of a key head
    int target;  // split: workgroups of a key head to aim at; 0: one unit per tile
    int least;   // split: key tiles of a unit at least
    int units;   // workgroups of a key head in the grid
    int tiles;   // row tiles at most
    float scale;
};

__device__ const __align__(16) uint8_t kZeros[16] = {};

constexpr float kBias = 13.f;  // weights are 2^(s - max + 13): binary16's subnormal numbers begin 2^-27 below the largest
constexpr float kLog2e = 1.4426950408889634f;

template <int kType>
struct Math {  // binary16 (e4m3 widened to it)
    typedef half8v v8;
    static constexpr bool kScaled = true;
    __device__ static f32x16 mfma32(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    __device__ static f32x4 mfma16(v8 a, v8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    __device__ static void split(const float *x, v8 &hi, v8 &lo) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const half2v h = __builtin_convertvector((f32x2{x[i], x[i + 1]}), half2v);
            const half2v l = __builtin_convertvector(
                (f32x2{fmaf(static_cast<float>(h.x), -1.f, x[i]), fmaf(static_cast<float>(h.y), -1.f, x[i + 1])}), half2v);
            hi[i] = h.x;
            hi[i + 1] = h.y;
            lo[i] = l.x;
            lo[i + 1] = l.y;
        }
    }
};
template <>
struct Math<Q4K_KV_BF16> {
    typedef bf8v v8;
    static constexpr bool kScaled = false;
    __device__ static f32x16 mfma32(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    __device__ static f32x4 mfma16(v8 a, v8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    __device__ static void split(const float *x, v8 &hi, v8 &lo) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const bf2v h = __builtin_convertvector((f32x2{x[i], x[i + 1]}), bf2v);
            const bf2v l = __builtin_convertvector(
                (f32x2{x[i] - static_cast<float>(h.x), x[i + 1] - static_cast<float>(h.y)}), bf2v);
            hi[i] = h.x;
            hi[i + 1] = h.y;
            lo[i] = l.x;
            lo[i + 1] = l.y;
        }
    }
};

// Eight e4m3 values (two words) in binary16.
__device__ __forceinline__ half8v widened(uint32_t a, uint32_t b) {
    const half2v x0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
    const half2v x1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
    const half2v x2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
    const half2v x3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
    return half8v{x0.x, x0.y, x1.x, x1.y, x2.x, x2.y, x3.x, x3.y};
}

// ---- copies -------------------------------------------------------------------

__device__ __forceinline__ uint32_t lds_address(const uint8_t *p) {
    return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const lds_u8 *)p)));
}

// 16 bytes per lane from memory to LDS at dst + 16 * lane, in assembly because
// the compiler would wait for every such copy before the next LDS read,
// whichever buffer that reads.  No register is written; the kernels wait for
// vmcnt before they read a buffer.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(const uint8_t *src, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src),
                 "s"(__builtin_amdgcn_readfirstlane(dst))
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// All but the last VM memory operations of this wave, and every LDS operation, have ended.
template <int VM>
__device__ __forceinline__ void wait_copies() {
    static_assert(VM < 64, "the counter's six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (VM & 15) | (VM >> 4) << 14);
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The place of 16-byte piece c of a row in LDS is c ^ swizzle(row).  RB: bytes of a
// row.  K: sixteen neighbouring rows, the same piece.  V: eight rows, a
// 64-byte stretch (or sixteen rows, 32 bytes), by 8-byte halves of pieces.
template <int RB>
__device__ __forceinline__ int swizzle_k(int row) {
    return RB == 64 ? (row >> 2) & 3 : RB == 128 ? (row >> 1) & 7 : row & 15;
}
template <int RB>
__device__ __forceinline__ int swizzle_v(int row) {
    return RB == 64    ? ((row >> 2) & 1) << 1 | ((row >> 3) & 1)
           : RB == 128 ? ((row >> 1) & 3) << 1 | ((row >> 3) & 1)
                       : (row & 7) << 1 | ((row >> 3) & 1);
}

// Where a sequence's keys and values are.  Lane l keeps entry first + l of the
// sequence's row of the table: 64 pages, looked up again when the keys pass them.
struct Pages {
    const int *row;
    const uint8_t *k, *v;  // of the key head
    uint64_t page_bytes;
    int first, entry;
    int max_pages, pages, shift, row_bytes;
    int stop;  // keys at and behind it are not there

    __device__ Pages(const Paged &p, int b, int head, int stop_, int size) {
        row = p.table + static_cast<size_t>(b) * p.max_pages;
        row_bytes = p.head_dim * size;
        const uint64_t head_bytes = static_cast<uint64_t>(row_bytes) << p.shift;
        k = p.k + head * head_bytes;
        v = p.v + head * head_bytes;
        page_bytes = head_bytes * p.kv_heads;
        max_pages = p.max_pages;
        pages = p.pages;
        shift = p.shift;
        stop = stop_;
        first = -64;
        entry = -1;
    }
    // Makes the pages of keys j0 .. j0 + 63 at most available.
    __device__ void look_up(int j0, int keys) {
        if (((j0 + keys - 1) >> shift) >= first + 64 || first < 0) {
            first = j0 >> shift;
            const int at = first + (threadIdx.x & 63);
            entry = at < max_pages ? row[at] : -1;
            if (entry >= pages) entry = -1;
        }
    }
    // The page of key j (of this look_up's keys), -1 if it is not there.
    __device__ int page_of(int j) const {
        const int page = __builtin_amdgcn_ds_bpermute(((j >> shift) - first) << 2, entry);
        return j < stop ? page : -1;
    }
    __device__ uint64_t offset(int page, int j) const {
        return static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_bytes +
               static_cast<uint32_t>((j & ((1 << shift) - 1)) * row_bytes);
    }
};

// Copies COPIES KB of a tile's keys and of its values, from byte `at` of the tile on.
template <int RB, int COPIES>
__device__ __forceinline__ void copy_rows(const Pages &g, int j0, int at, uint32_t k_lds, uint32_t v_lds) {
    constexpr int kPieces = RB / 16, kRows = 1024 / RB;
    const int lane = threadIdx.x & 63;
#pragma unroll 4
    for (int i = 0; i < COPIES; ++i) {
        const int row = (at + i * 1024) / RB + lane / kPieces, piece = lane % kPieces;
        const int j = j0 + row, page = g.page_of(j);
        const uint64_t off = g.offset(page, j);
        const int ck = (piece ^ swizzle_k<RB>(row)) * 16, cv = (piece ^ swizzle_v<RB>(row)) * 16;
        const uint8_t *ks = page >= 0 && ck < g.row_bytes ? g.k + off + ck : kZeros;
        const uint8_t *vs = page >= 0 && cv < g.row_bytes ? g.v + off + cv : kZeros;
        copy_to_lds(ks, k_lds + at + i * 1024);
        copy_to_lds(vs, v_lds + at + i * 1024);
    }
    static_assert(kRows >= 1, "a row is at most a copy");
}

// Bit l: key j0 + l has a place (keys: 32 or 64).
__device__ __forceinline__ uint64_t there(const Pages &g, int j0, int keys) {
    const int lane = threadIdx.x & 63;
    const int page = g.page_of(j0 + min(lane, keys - 1));
    return __ballot(page >= 0 && lane < keys);
}

// Values in LDS from byte `at` on, BYTES of a tile, looked through by the lanes of a
// wave: NaN and infinities are made zeros, and marks[row * DP + d bits] say where
// they were.  Returns whether there were any.
template <int kType, int RB, int BYTES>
__device__ __forceinline__ bool set_apart(uint8_t *v, int at, uint8_t *marks) {
    constexpr int kSize = kType == Q4K_KV_E4M3 ? 1 : 2, kPieces = RB / 16;
    uint32_t any = 0;
#pragma unroll 1
    for (int i = at + (threadIdx.x & 63) * 16; i < at + BYTES; i += 1024) {
        u32x4 w = *reinterpret_cast<const u32x4 *>(v + i);
        const int row = i / RB, piece = i / 16 % kPieces ^ swizzle_v<RB>(row);
        uint32_t found = 0, bits = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // the highest bit of every value that is a NaN or an infinity
            const uint32_t f = kType == Q4K_KV_E4M3   ? ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u
                               : kType == Q4K_KV_BF16 ? ((w[k] & 0x7fff7fffu) + 0x00800080u) & 0x80008000u
                                                      : ((w[k] & 0x7fff7fffu) + 0x04000400u) & 0x80008000u;
            found |= f;
            if (kSize == 1) {
                bits |= ((f >> 7 & 1) | (f >> 14 & 2) | (f >> 21 & 4) | (f >> 28 & 8)) << (4 * k);
                w[k] &= ~((f >> 7) * 0xffu);
            } else {
                bits |= ((f >> 15 & 1) | (f >> 30 & 2)) << (2 * k);
                w[k] &= ~((f >> 15) * 0xffffu);
            }
        }
        if (kSize == 1) *reinterpret_cast<uint16_t *>(marks + (row * kPieces + piece) * 2) = static_cast<uint16_t>(bits);
        else marks[row * kPieces + piece] = static_cast<uint8_t>(bits);
        if (found) *reinterpret_cast<u32x4 *>(v + i) = w;
        any |= found;
    }
    return __ballot(any != 0) != 0;
}

// ---- the division of the work ---------------------------------------------------

struct Unit {
    int b, first, n;    // sequence, its first row of q, its new tokens
    int length;         // its tokens
    int tile;           // of its row tiles
    int chunk, chunks;  // of its keys
    int size;           // key tiles of a chunk
    int64_t unit0;      // the tile's first unit
};

// Unit (kByTile: row tile) number id of a key head.  Sequences have
// tiles_b = ceil(n_b * group / ROWS) tiles of chunks_b = ceil(keys_b / size) units.
// Every lane returns the same; false where there is no such unit.
template <int ROWS, int KT, bool kByTile>
__device__ __forceinline__ bool find_unit(const Attend &a, int64_t id, Unit &u) {
    const Paged &p = a.p;
    const int lane = threadIdx.x & 63;
    const int capacity = p.max_pages << p.shift;
    int first = 0, n = 0, length = 0;
    int64_t tiles = 0, key_tiles = 0;
    const auto load = [&](int b) {
        first = n = length = 0;
        if (b < p.count) {
            first = offset_of(p, b);
            n = max(offset_of(p, b + 1) - first, 0);
            length = max(p.lengths[b], 0);  // (without tokens nothing is seen)
        }
        tiles = (static_cast<int64_t>(n) * a.group + ROWS - 1) / ROWS;
        key_tiles = (min(length, capacity) + KT - 1) / KT;
    };
    int size = INT_MAX;
    if (a.target) {
        int64_t all = 0;
        for (int b = lane; b < ((p.count + 63) & ~63); b += 64) {
            load(b);
            all += tiles * key_tiles;
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o);
        size = static_cast<int>(max((all + a.target - 1) / a.target, static_cast<int64_t>(a.least)));
    }
    int64_t before = 0, units_before = 0;  // of the sequences looked through
    for (int b0 = 0; b0 < p.count; b0 += 64) {
        if (!a.target || p.count > 64) load(b0 + lane);
        const int64_t chunks = max(key_tiles / size + (key_tiles % size != 0), static_cast<int64_t>(1));
        const int64_t units = tiles * chunks, mine = kByTile ? tiles : units;
        int64_t sum = mine, unit_sum = units;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t x = __shfl_up(sum, o), y = __shfl_up(unit_sum, o);
            if (lane >= o) {
                sum += x;
                unit_sum += y;
            }
        }
        const uint64_t behind = __ballot(before + sum > id);
        if (behind) {
            const int l = __builtin_ctzll(behind);
            const int64_t rest = id - before - (__shfl(sum, l) - __shfl(mine, l));
            u.b = b0 + l;
            u.first = __builtin_amdgcn_readfirstlane(__shfl(first, l));
            u.n = __builtin_amdgcn_readfirstlane(__shfl(n, l));
            u.length = __builtin_amdgcn_readfirstlane(__shfl(length, l));
            u.chunks = __builtin_amdgcn_readfirstlane(static_cast<int>(__shfl(chunks, l)));
            const int kt = __builtin_amdgcn_readfirstlane(static_cast<int>(__shfl(key_tiles, l)));
            const int r = __builtin_amdgcn_readfirstlane(static_cast<int>(rest));
            u.tile = kByTile ? r : r / u.chunks;
            u.chunk = kByTile ? 0 : r % u.chunks;
            u.size = (kt + u.chunks - 1) / u.chunks;
            u.unit0 = units_before + (__shfl(unit_sum, l) - __shfl(units, l)) + static_cast<int64_t>(u.tile) * u.chunks;
            return true;
        }
        before += __shfl(sum, 63);
        units_before += __shfl(unit_sum, 63);
    }
    return false;
}

// A lane's row: its query, its place in the outputs and what it sees.
struct Row {
    bool real;
    int64_t at;  // element of q and out
    int stop;    // causal: the keys below it are seen; tree: the length
    const unsigned *mask;
};

__device__ __forceinline__ Row row_of(const Attend &a, const Unit &u, int r, int head) {
    Row w;
    const int i = r / a.group, g = r - i * a.group;
    w.real = i < u.n;
    const int64_t t = static_cast<int64_t>(u.first) + (w.real ? i : 0);
    w.at = (t * a.q_heads + head * a.group + (w.real ? g : 0)) * a.p.head_dim;
    w.stop = a.mask || !w.real ? u.length : u.length - u.n + i + 1;
    w.mask = a.mask ? a.mask + t * a.words : nullptr;
    return w;
}

// Bit k: the row sees key j0 + k, for 64 keys (before: the index of the first new token).
__device__ __forceinline__ uint64_t seen(const Attend &a, const Row &w, int before, int j0) {
    if (!a.mask || !w.real) {
        const int left = w.stop - j0;
        return left >= 64 ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1;
    }
    // new tokens of the window: bits from word (j0 - before) / 32 on
    const int64_t from = static_cast<int64_t>(j0) - before;
    if (from <= -64) return ~0ull;
    const auto word = [&](int64_t i) { return i >= 0 && i < a.words ? static_cast<uint64_t>(w.mask[i]) : 0ull; };
    if (from < 0) return (word(0) | word(1) << 32) << -from | ((1ull << -from) - 1);
    const int64_t i = from >> 5;
    const int s = static_cast<int>(from & 31);
    const uint64_t low = word(i) | word(i + 1) << 32;
    return s ? low >> s | word(i + 2) << (64 - s) : low;
}

// The query's power of two: |x| * 2^e of the largest is in [2^13, 2^14).
__device__ __forceinline__ int exponent_for(float largest) {
    if (!(largest > 0.f) || !(largest < INFINITY)) return 0;
    return min(14 - (static_cast<int>(__builtin_amdgcn_frexp_expf(largest))), 100);
}

// Eight values of the query from dimension d on, times `by`.
__device__ __forceinline__ void load_query(const Attend &a, const Row &w, int d, float by, float *x) {
    f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0;
    if (w.real && d < a.p.head_dim) {
        x0 = *reinterpret_cast<const f32x4 *>(a.q + w.at + d);
        x1 = *reinterpret_cast<const f32x4 *>(a.q + w.at + d + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = x0[i] * by;
        x[4 + i] = x1[i] * by;
    }
}

__device__ __forceinline__ float nan_value() { return __builtin_nanf(""); }

// ---- many rows -------------------------------------------------------------------
//
// 128 rows per workgroup, 32 a wave; tiles of KT keys, in LDS for all waves, two
// buffers.  Products of 32 x 32 x 16.

constexpr int kTileRows = 128;

template <int kType, int DP>
struct TileShape {
    static constexpr int kSize = kType == Q4K_KV_E4M3 ? 1 : 2;
    static constexpr int RB = DP * kSize;             // bytes of a row
    static constexpr int KT = DP == 256 ? 32 : 64;    // keys of a tile
    static constexpr int kBytes = KT * RB;            // of K, and of V
    static constexpr int kCopies = kBytes / 4096;     // of a wave
    static constexpr int kMarks = KT * DP / 8;        // a bit per value
    static constexpr int kLds = 4 * kBytes + kMarks + 16;
};

template <int kType, int DP>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void attend_tiles(const Attend a) {
    typedef TileShape<kType, DP> S;
    typedef Math<kType> M;
    typedef typename M::v8 v8;
    constexpr int RB = S::RB, KT = S::KT, KS = KT / 32, NS = DP / 16, ND = DP / 32;
    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t *const marks = lds + 4 * S::kBytes;
    int *const flag = reinterpret_cast<int *>(marks + S::kMarks);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
    const int head = blockIdx.x % a.p.kv_heads;
    // the last tiles of a prompt have the most keys: they go first
    const int64_t id = a.units - 1 - static_cast<int64_t>(blockIdx.x / a.p.kv_heads);
    Unit u;
    if (!find_unit<kTileRows, KT, false>(a, id, u)) return;
    const int before = u.length - u.n;
    const int row0 = u.tile * kTileRows, rows = u.n * a.group;
    const int capacity = a.p.max_pages << a.p.shift;
    // keys that some row of the tile may see, and those that every one sees
    const int last = min((row0 + kTileRows - 1) / a.group, u.n - 1);
    const int most = a.mask ? u.length : before + last + 1;
    const int common = a.mask ? before : before + row0 / a.group + 1;
    const int stop = max(min(most, capacity), 0);
    const int t0 = u.chunk * u.size, t1 = min((stop + KT - 1) / KT, u.chunks == 1 ? INT_MAX : t0 + u.size);
    const Row w = row_of(a, u, row0 + wave * 32 + col, head);
    const bool idle = row0 + wave * 32 >= rows;  // no row of this wave is real

    Pages pages(a.p, u.b, head, min(u.length, capacity), S::kSize);
    const uint32_t base = lds_address(lds);
    const int piece0 = wave * S::kCopies * 1024;
    uint64_t here = 0;
    if (threadIdx.x == 0) *flag = -1;
    if (t0 < t1) {
        pages.look_up(t0 * KT, KT);
        here = there(pages, t0 * KT, KT);
        copy_rows<RB, S::kCopies>(pages, t0 * KT, piece0, base, base + 2 * S::kBytes);
    }

    // the wave's queries as the second operand of S^T = K Q^T: lane's row, 8 dimensions a step
    v8 qh[NS], ql[NS];
    float factor = 1.f;
    {
        const float by = a.scale * kLog2e * a.p.k_scale;
        const auto dim = [&](int s) {
            return kType == Q4K_KV_E4M3 ? 32 * (s >> 1) + 16 * half + 8 * (s & 1) : 16 * s + 8 * half;
        };
        const auto load = [&](int s, float *x) {
            load_query(a, w, dim(s), by, x);
        };
        int e = 0;
        if constexpr (M::kScaled) {
            float largest = 0.f;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                float x[8];
                load(s, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) largest = fmaxf(largest, __builtin_fabsf(x[i]));
            }
            e = exponent_for(fmaxf(largest, __shfl_xor(largest, 32)));
            factor = ldexpf(1.f, -e);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            float x[8];
            load(s, x);
            if constexpr (M::kScaled) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = ldexpf(x[i], e);
            }
            M::split(x, qh[s], ql[s]);
        }
    }

    // where this lane reads: K by pieces of its row, V by halves of pieces, four keys (e4m3: eight) at a time
    const int k_at = col * RB, k_x = half ^ swizzle_k<RB>(col);
    const int li = lane & 15, dh = (lane >> 4) & 1;
    int v_row, v_c;
    if constexpr (kType == Q4K_KV_E4M3) {
        const int r = li >> 1;
        v_row = (r < 4 ? 0 : 4) + 4 * half + r;
        v_c = dh;
    } else {
        v_row = 4 * half + (li >> 2);
        v_c = 2 * dh + ((li & 3) >> 1);
    }
    const int v_at = v_row * RB + 8 * (li & 1), v_x = v_c ^ swizzle_v<RB>(v_row);
    const int v_at2 = v_at + 8 * RB, v_x2 = v_c ^ swizzle_v<RB>(v_row + 8);

    f32x16 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] = 0.f;
    float m = -INFINITY, sum = 0.f;

    for (int t = t0; t < t1; ++t) {
        const int buf = (t - t0) & 1;
        wait_copies<0>();
        barrier();
        const uint64_t now = here;
        if (t + 1 < t1) {
            pages.look_up((t + 1) * KT, KT);
            here = there(pages, (t + 1) * KT, KT);
            copy_rows<RB, S::kCopies>(pages, (t + 1) * KT, piece0, base + (buf ^ 1) * S::kBytes,
                                      base + (2 + (buf ^ 1)) * S::kBytes);
        }
        const uint8_t *kt = lds + buf * S::kBytes;
        uint8_t *vt = lds + (2 + buf) * S::kBytes;
        // rows that see different parts of the tile: is there a value to be kept from some?
        bool apart = false;
        if (t * KT + KT > common) {
            if (set_apart<kType, RB, S::kBytes / 4>(vt, wave * (S::kBytes / 4), marks) && lane == 0) *flag = t;
            __syncthreads();
            apart = *flag == t;
        }
        if (idle) continue;
        uint64_t vis = seen(a, w, before, t * KT) & now;
        const uint64_t whole = KT == 64 ? ~0ull : 0xFFFFFFFFull;
        vis &= whole;
        if (__ballot(vis != 0) == 0) continue;  // nothing for this wave
        f32x16 s[KS];
        int kx = k_x;
        asm volatile("" : "+v"(kx));  // the pieces' places are worked out again, not kept: registers are short here
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[k][r] = 0.f;
#pragma unroll
            for (int c = 0; c < RB / 32; ++c) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(kt + k * 32 * RB + k_at + (((2 * c) ^ kx) << 4));
                if constexpr (kType == Q4K_KV_E4M3) {
                    const half8v x0 = widened(x.x, x.y), x1 = widened(x.z, x.w);
                    s[k] = M::mfma32(x0, qh[2 * c], s[k]);
                    s[k] = M::mfma32(x0, ql[2 * c], s[k]);
                    s[k] = M::mfma32(x1, qh[2 * c + 1], s[k]);
                    s[k] = M::mfma32(x1, ql[2 * c + 1], s[k]);
                } else {
                    const v8 x0 = __builtin_bit_cast(v8, x);
                    s[k] = M::mfma32(x0, qh[c], s[k]);
                    s[k] = M::mfma32(x0, ql[c], s[k]);
                }
            }
        }
        const bool masked = __ballot(vis != whole) != 0;
        const uint64_t mine = vis >> (4 * half);
        if (masked) {
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!((mine >> (32 * k + 8 * (r >> 2) + (r & 3))) & 1)) s[k][r] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[k][r]);
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m1 = fmaxf(m, top * factor);
        const float zero = m1 == -INFINITY ? 0.f : m1;
        const float fade = __builtin_amdgcn_exp2f(m - zero);
        m = m1;
        const float shift = kBias - zero;
        float part = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[k][r] = __builtin_amdgcn_exp2f(fmaf(s[k][r], factor, shift));
                part += s[k][r];
            }
        sum = fmaf(sum, fade, part);
        if (__ballot(fade != 1.f) != 0) {
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[d][r] *= fade;
        }
#pragma unroll
        for (int q = 0; q < KT / 16; ++q) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s[q >> 1][8 * (q & 1) + i];
            v8 ph, pl;
            M::split(x, ph, pl);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                v8 y;
                const uint8_t *vq = vt + q * 16 * RB;
                if constexpr (kType == Q4K_KV_E4M3) {
                    const i32x2 z = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                        (__attribute__((address_space(3))) i32x2 *)(vq + v_at + (((2 * d) ^ v_x) << 4)));
                    y = widened(z.x, z.y);
                } else {
                    const s16x4 z0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s16x4 *)(vq + v_at + (((4 * d) ^ v_x) << 4)));
                    const s16x4 z1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (__attribute__((address_space(3))) s16x4 *)(vq + v_at2 + (((4 * d) ^ v_x2) << 4)));
                    y = __builtin_bit_cast(v8, __builtin_shufflevector(z0, z1, 0, 1, 2, 3, 4, 5, 6, 7));
                }
                acc[d] = M::mfma32(y, ph, acc[d]);
                acc[d] = M::mfma32(y, pl, acc[d]);
            }
        }
        if (apart) {  // rows that see a marked value get NaN there
#pragma unroll 1
            for (int i = 0; i < KT * DP / 8; ++i) {
                uint32_t bits = marks[i];
                if (!((vis >> (i / (DP / 8))) & 1)) bits = 0;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int at = 32 * d + 8 * (r >> 2) + 4 * half + (r & 3) - i % (DP / 8) * 8;
                        if (static_cast<unsigned>(at) < 8u && ((bits >> at) & 1)) acc[d][r] = nan_value();
                    }
            }
        }
    }

    sum += __shfl_xor(sum, 32);
    if (idle || !w.real) return;
    if (u.chunks == 1) {
        int r0 = row0 + wave * 32 + col;
        asm volatile("" : "+v"(r0));  // worked out again rather than kept over the loop
        float *const out = a.out + row_of(a, u, r0, head).at;
        const float f = sum == 0.f ? 0.f : a.p.v_scale / sum;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int at = 32 * d + 2 * r + 4 * half;
                if (at < a.p.head_dim) {
                    f32x4 y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = sum == 0.f ? 0.f : acc[d][r + i] * f;
                    *reinterpret_cast<f32x4 *>(out + at) = y;
                }
            }
    } else {
        const int64_t at0 = (id * a.p.kv_heads + head) * kTileRows + wave * 32 + col;
        if (half == 0) {
            a.part_ml[2 * at0] = m;
            a.part_ml[2 * at0 + 1] = sum;
        }
        if (t0 >= t1) return;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int at = 32 * d + 2 * r + 4 * half;
                if (at < a.p.head_dim)
                    *reinterpret_cast<f32x4 *>(a.part + at0 * a.p.head_dim + at) =
                        f32x4{acc[d][r], acc[d][r + 1], acc[d][r + 2], acc[d][r + 3]};
            }
    }
}

// ---- few rows --------------------------------------------------------------------
//
// 16 rows per workgroup; its waves take key tiles of 32 in turn, each with its
// own two buffers in LDS and its own maximum, sum and output, and nothing to
// wait for but its own copies; the waves' parts are joined at the end.
// Products of 16 x 16 x 32.

constexpr int kFewRows = 16;

template <int kType, int DP>
struct FewShape {
    static constexpr int kSize = kType == Q4K_KV_E4M3 ? 1 : 2;
    static constexpr int RB = DP * kSize;
    static constexpr int kWaves = RB == 512 ? 2 : 4;
    static constexpr int kBytes = 32 * RB;  // of a tile's K, and of its V
    static constexpr int kCopies = kBytes / 1024;
    static constexpr int kJoin = kWaves * kFewRows * (DP + 4) * 4;
    static constexpr int kMarks = 32 * DP / 8;  // a bit per value
    static constexpr int kOwn = 4 * kBytes + kMarks;
    static constexpr int kLds = kWaves * kOwn > kJoin ? kWaves * kOwn : kJoin;
};

template <int kType, int DP>
__global__ __launch_bounds__((FewShape<kType, DP>::kWaves * 64)) void attend_few(const Attend a) {
    typedef FewShape<kType, DP> S;
    typedef Math<kType> M;
    typedef typename M::v8 v8;
    constexpr int RB = S::RB, KT = 32 * S::kWaves, NS = DP / 32, ND = DP / 16;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quarter = lane >> 4;
    const int head = blockIdx.x % a.p.kv_heads;
    const int64_t id = blockIdx.x / a.p.kv_heads;
    Unit u;
    if (!find_unit<kFewRows, KT, false>(a, id, u)) return;
    const int before = u.length - u.n;
    const int row0 = u.tile * kFewRows;
    const int capacity = a.p.max_pages << a.p.shift;
    const int last = min((row0 + kFewRows - 1) / a.group, u.n - 1);
    const int most = a.mask ? u.length : before + last + 1;
    const int common = a.mask ? before : before + row0 / a.group + 1;
    const int stop = max(min(most, capacity), 0);
    // tiles of 32 keys: this wave's are first, first + kWaves, ...
    const int t0 = u.chunk * u.size * S::kWaves + wave;
    const int t1 = min((stop + 31) / 32, u.chunks == 1 ? INT_MAX : (u.chunk + 1) * u.size * S::kWaves);
    const Row w = row_of(a, u, row0 + col, head);

    Pages pages(a.p, u.b, head, min(u.length, capacity), S::kSize);
    uint8_t *const own = lds + wave * S::kOwn;
    const uint32_t base = lds_address(own);
    const auto copy = [&](int t, int buf) {
        pages.look_up(t * 32, 32);
        const uint64_t is = there(pages, t * 32, 32);
        copy_rows<RB, S::kCopies>(pages, t * 32, 0, base + buf * 2 * S::kBytes, base + (buf * 2 + 1) * S::kBytes);
        return is;
    };
    uint64_t here = 0;
    if (t0 < t1) here = copy(t0, 0);

    v8 qh[NS], ql[NS];
    float factor = 1.f;
    {
        const float by = a.scale * kLog2e * a.p.k_scale;
        const auto load = [&](int s, float *x) {
            const int d = kType == Q4K_KV_E4M3 ? 64 * (s >> 1) + 16 * quarter + 8 * (s & 1) : 32 * s + 8 * quarter;
            load_query(a, w, d, by, x);
        };
        int e = 0;
        if constexpr (M::kScaled) {
            float largest = 0.f;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                float x[8];
                load(s, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) largest = fmaxf(largest, __builtin_fabsf(x[i]));
            }
            largest = fmaxf(largest, __shfl_xor(largest, 16));
            largest = fmaxf(largest, __shfl_xor(largest, 32));
            e = exponent_for(largest);
            factor = ldexpf(1.f, -e);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            float x[8];
            load(s, x);
            if constexpr (M::kScaled) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = ldexpf(x[i], e);
            }
            M::split(x, qh[s], ql[s]);
        }
    }

    const int k_at = col * RB, k_x = quarter ^ swizzle_k<RB>(col);
    int v_row, v_c;
    if constexpr (kType == Q4K_KV_E4M3) {
        const int r = col >> 1;
        v_row = (r < 4 ? 0 : 12) + 4 * quarter + r;
        v_c = 0;
    } else {
        v_row = 4 * quarter + (col >> 2);
        v_c = (col & 3) >> 1;
    }
    const int v_at = v_row * RB + 8 * (col & 1), v_x = v_c ^ swizzle_v<RB>(v_row);

    f32x4 acc[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;
    int buf = 0;
    for (int t = t0; t < t1; t += S::kWaves, buf ^= 1) {
        const uint64_t now = here;
        if (t + S::kWaves < t1) {
            here = copy(t + S::kWaves, buf ^ 1);
            wait_copies<2 * S::kCopies>();
        } else {
            wait_copies<0>();
        }
        const uint8_t *kt = own + buf * 2 * S::kBytes;
        uint8_t *vt = own + (buf * 2 + 1) * S::kBytes, *marks = own + 4 * S::kBytes;
        const bool apart = t * 32 + 32 > common && set_apart<kType, RB, S::kBytes>(vt, 0, marks);
        const uint32_t vis = static_cast<uint32_t>(seen(a, w, before, t * 32) & now);
        if (__ballot(vis != 0) == 0) continue;
        f32x4 s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            s[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < RB / 64; ++c) {
                const u32x4 x = *reinterpret_cast<const u32x4 *>(kt + k * 16 * RB + k_at + (((4 * c) ^ k_x) << 4));
                if constexpr (kType == Q4K_KV_E4M3) {
                    const half8v x0 = widened(x.x, x.y), x1 = widened(x.z, x.w);
                    s[k] = M::mfma16(x0, qh[2 * c], s[k]);
                    s[k] = M::mfma16(x0, ql[2 * c], s[k]);
                    s[k] = M::mfma16(x1, qh[2 * c + 1], s[k]);
                    s[k] = M::mfma16(x1, ql[2 * c + 1], s[k]);
                } else {
                    const v8 x0 = __builtin_bit_cast(v8, x);
                    s[k] = M::mfma16(x0, qh[c], s[k]);
                    s[k] = M::mfma16(x0, ql[c], s[k]);
                }
            }
        }
        const uint32_t mine = vis >> (4 * quarter);
        if (__ballot(vis != 0xFFFFFFFFu) != 0) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!((mine >> (16 * k + r)) & 1)) s[k][r] = -INFINITY;
        }
        float top = s[0][0];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) top = fmaxf(top, s[k][r]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m1 = fmaxf(m, top * factor);
        const float zero = m1 == -INFINITY ? 0.f : m1;
        const float fade = __builtin_amdgcn_exp2f(m - zero);
        m = m1;
        const float shift = kBias - zero;
        float x[8], part = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_amdgcn_exp2f(fmaf(s[i >> 2][i & 3], factor, shift));
            part += x[i];
        }
        sum = fmaf(sum, fade, part);
        v8 ph, pl;
        M::split(x, ph, pl);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            acc[d] *= fade;
            v8 y;
            if constexpr (kType == Q4K_KV_E4M3) {
                const i32x2 z = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (__attribute__((address_space(3))) i32x2 *)(vt + v_at + ((d ^ v_x) << 4)));
                y = widened(z.x, z.y);
            } else {
                const uint8_t *at = vt + v_at + (((2 * d) ^ v_x) << 4);
                const s16x4 z0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at);
                const s16x4 z1 =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(at + 16 * RB));
                y = __builtin_bit_cast(v8, __builtin_shufflevector(z0, z1, 0, 1, 2, 3, 4, 5, 6, 7));
            }
            acc[d] = M::mfma16(y, ph, acc[d]);
            acc[d] = M::mfma16(y, pl, acc[d]);
        }
        if (apart) {
#pragma unroll 1
            for (int i = 0; i < 32 * DP / 8; ++i) {
                uint32_t bits = marks[i];
                if (!((vis >> (i / (DP / 8))) & 1)) bits = 0;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int at = 16 * d + 4 * quarter + r - i % (DP / 8) * 8;
                        if (static_cast<unsigned>(at) < 8u && ((bits >> at) & 1)) acc[d][r] = nan_value();
                    }
            }
        }
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);

    // the waves' parts: [wave][row][DP] and [wave][row] maxima and sums (row stride DP + 4 words)
    wait_copies<0>();
    barrier();
    float *const po = reinterpret_cast<float *>(lds);
    constexpr int kStride = DP + 4;
    {
        float *mine = po + (wave * kFewRows + col) * kStride;
#pragma unroll
        for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(mine + 16 * d + 4 * quarter) = acc[d];
        if (quarter == 0) {
            mine[DP] = m;
            mine[DP + 1] = sum;
        }
    }
    __syncthreads();
    const int quads = a.p.head_dim / 4;
    for (int i = threadIdx.x; i < kFewRows * quads; i += S::kWaves * 64) {
        const int r = i / quads, d = (i - r * quads) * 4;
        const Row o = row_of(a, u, row0 + r, head);
        if (!o.real) continue;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < S::kWaves; ++k) top = fmaxf(top, po[(k * kFewRows + r) * kStride + DP]);
        const float zero = top == -INFINITY ? 0.f : top;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < S::kWaves; ++k) {
            const float *from = po + (k * kFewRows + r) * kStride;
            // a wave without keys has nothing to add (its maximum is -inf)
            const float f = __builtin_amdgcn_exp2f(from[DP] - zero);
            total = fmaf(from[DP + 1], f, total);
            y += *reinterpret_cast<const f32x4 *>(from + d) * f;
        }
        if (u.chunks == 1) {
            const float f = a.p.v_scale / total;
            if (total == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
            else y *= f;
            *reinterpret_cast<f32x4 *>(a.out + o.at + d) = y;
        } else {
            const int64_t at = (id * a.p.kv_heads + head) * kFewRows + r;
            *reinterpret_cast<f32x4 *>(a.part + at * a.p.head_dim + d) = y;
            if (d == 0) {
                a.part_ml[2 * at] = top;
                a.part_ml[2 * at + 1] = total;
            }
        }
    }
}

// ---- the units' parts joined -------------------------------------------------------
//
// A wave per row: its units' maxima and sums by lanes, then their outputs in
// ascending order.  A unit whose maximum is -inf has seen nothing (and may have
// written no output).

template <int ROWS, int KT>
__global__ __launch_bounds__(256) void join_units(const Attend a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int head = blockIdx.x % a.p.kv_heads;
    const int rest = blockIdx.x / a.p.kv_heads;
    const int tile = rest / (ROWS / 4), r = rest % (ROWS / 4) * 4 + wave;
    Unit u;
    if (!find_unit<ROWS, KT, true>(a, tile, u) || u.chunks == 1 || u.unit0 + u.chunks > a.units) return;
    const Row w = row_of(a, u, u.tile * ROWS + r, head);
    if (!w.real) return;
    const int D = a.p.head_dim;
    const auto place = [&](int c) { return ((u.unit0 + c) * a.p.kv_heads + head) * ROWS + r; };
    float top = -INFINITY;
    for (int c = lane; c < u.chunks; c += 64) top = fmaxf(top, a.part_ml[2 * place(c)]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float zero = top == -INFINITY ? 0.f : top;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
    for (int c0 = 0; c0 < u.chunks; c0 += 64) {
        float f = 0.f;
        bool any = false;
        if (c0 + lane < u.chunks) {
            const float mc = a.part_ml[2 * place(c0 + lane)];
            any = mc != -INFINITY;
            f = __builtin_amdgcn_exp2f(mc - zero);
            total = fmaf(a.part_ml[2 * place(c0 + lane) + 1], f, total);
        }
        uint64_t with = __ballot(any);
        while (with) {
            const int l = __builtin_ctzll(with);
            with &= with - 1;
            const float fc = __shfl(f, l);
            if (lane * 4 < D) y += *reinterpret_cast<const f32x4 *>(a.part + place(c0 + l) * D + lane * 4) * fc;
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
    const float f = a.p.v_scale / total;
    if (total == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
    else y *= f;
    if (lane * 4 < D) *reinterpret_cast<f32x4 *>(a.out + w.at + lane * 4) = y;
}

// ---- launches ------------------------------------------------------------------------

constexpr int kCus = 256;

// Row tiles of a key head at most: sum of ceil(n_b * group / rows) <= T * group / rows + count.
int64_t tiles_at_most(const Attend &a, int rows) {
    return static_cast<int64_t>(a.p.tokens) * a.group / rows + min(a.p.count, a.p.tokens);
}

template <int ROWS, int KT, class Kernel>
int launch(Attend &a, Kernel kernel, int threads, int lds, int per_cu, int least, hipStream_t stream) {
    const int64_t tiles = tiles_at_most(a, ROWS), heads = a.p.kv_heads;
    int64_t target = (static_cast<int64_t>(kCus) * per_cu + heads - 1) / heads;
    if (tiles >= target) target = 0;
    a.target = static_cast<int>(target);
    a.least = least;
    const int64_t units = tiles + target;
    if (units * heads > INT_MAX || tiles * heads * (ROWS / 4) > INT_MAX) return Q4K_ERR_LAUNCH;
    a.units = static_cast<int>(units);
    a.tiles = static_cast<int>(tiles);
    if (target) {
        const size_t rows = static_cast<size_t>(units) * heads * ROWS;
        float *ws = nullptr;
        if (workspace(stream, rows * (a.p.head_dim + 2) * sizeof(float), &ws, 0) != hipSuccess) return Q4K_ERR_ALLOC;
        a.part = ws;
        a.part_ml = ws + rows * a.p.head_dim;
    }
    if (lds > 65536 && allow_dynamic_lds(reinterpret_cast<const void *>(kernel), lds) != hipSuccess) return Q4K_ERR_LAUNCH;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(units * heads)), dim3(threads), lds, stream, a);
    if (hipGetLastError() != hipSuccess) return Q4K_ERR_LAUNCH;
    if (target) {
        hipLaunchKernelGGL((join_units<ROWS, KT>), dim3(static_cast<unsigned>(tiles * heads * (ROWS / 4))), dim3(256), 0, stream, a);
        if (hipGetLastError() != hipSuccess) return Q4K_ERR_LAUNCH;
    }
    return Q4K_OK;
}

template <int kType, int DP>
int launch_shape(Attend &a, hipStream_t stream) {
    // Rows of a sequence on average: the smaller tiles where they would be the emptier ones.
    const int64_t rows = static_cast<int64_t>(a.p.tokens) * a.group;
    if (rows <= 16ll * a.p.count) {
        typedef FewShape<kType, DP> S;
        return launch<kFewRows, 32 * S::kWaves>(a, attend_few<kType, DP>, S::kWaves * 64, S::kLds,
                                                S::kLds > 81920 ? 1 : 2, 1, stream);
    }
    typedef TileShape<kType, DP> S;
    return launch<kTileRows, S::KT>(a, attend_tiles<kType, DP>, 256, S::kLds, S::kLds > 81920 ? 1 : 2, 4, stream);
}

template <int kType>
int launch_type(Attend &a, hipStream_t stream) {
    const int D = a.p.head_dim;
    return D <= 64 ? launch_shape<kType, 64>(a, stream) : D <= 128 ? launch_shape<kType, 128>(a, stream) : launch_shape<kType, 256>(a, stream);
}

bool misaligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
bool misaligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int attend(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences, const unsigned *mask, int words,
           float scale, float *out, int T, int q_heads, hipStream_t stream) {
    Attend a = {};
    if (q_heads < 1) return Q4K_ERR_BAD_DIM;
    int rc = check_paged(cache, sequences, T, q_heads, &a.p);
    if (rc != Q4K_OK || T == 0 || sequences->count == 0) return rc;
    if (!q || !out) return Q4K_ERR_NULL;
    if (misaligned16(q) || misaligned16(out) || misaligned4(mask)) return Q4K_ERR_ALIGN;
    rc = check_device();
    if (rc != Q4K_OK) return rc;
    a.q = q;
    a.out = out;
    a.mask = mask;
    a.words = words;
    a.q_heads = q_heads;
    a.group = q_heads / cache->kv_heads;
    a.scale = scale;
    return cache->type == Q4K_KV_F16    ? launch_type<Q4K_KV_F16>(a, stream)
           : cache->type == Q4K_KV_BF16 ? launch_type<Q4K_KV_BF16>(a, stream)
                                        : launch_type<Q4K_KV_E4M3>(a, stream);
}

}  // namespace
}  // namespace q4k

extern "C" int q4k_attention(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences, float scale,
                             float *out, int T, int q_heads, hipStream_t stream) {
    return q4k::attend(q, cache, sequences, nullptr, 0, scale, out, T, q_heads, stream);
}

extern "C" int q4k_attention_tree(const float *q, const q4k_kv_cache *cache, const q4k_sequences *sequences,
                                  const unsigned *mask, int mask_words, float scale, float *out, int T, int q_heads,
                                  hipStream_t stream) {
    if (mask_words < 1) return Q4K_ERR_BAD_DIM;
    if (T > 0 && sequences && sequences->count > 0 && !mask) return Q4K_ERR_NULL;
    return q4k::attend(q, cache, sequences, mask, mask_words, scale, out, T, q_heads, stream);
}
