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
// are float32 values split into two binary16 numbers (over a bfloat16 cache, three
// bfloat16 ones), so both products run twice (three times): 8 (12) * head_dim
// operations per row and key instead of 4, at float32 accuracy.
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
// Few row tiles are split along the keys (Piece): the workgroups that fill the
// card take equal shares of all key tiles, and the parts of a row are joined, by
// the last of them to end or by a second launch.  The lengths stay on the
// device; every workgroup works its share out by itself.
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

struct Part {  // a row tile's units
    int unit0, units;
};

struct Attend {
    Paged p;
    const float *q;
    float *out;
    const unsigned *mask;  // null: causal
    float *part;           // split: outputs of the units, [units * kv_heads][rows][head_dim] ...
    float *part_ml;        // ... and their maxima and sums, [units * kv_heads][rows][2]
    Part *plan;            // split, many rows: [slots], for the launch that joins them
    uint32_t *counters;    // split, few rows: the units of a row tile that have ended
    uint32_t *next;        // split, few rows: counters to be cleared for the next call
    int64_t slots;
    int words;
    int q_heads;
    int group;   // query heads of a key head
    int target;  // split: workgroups of a key head; 0: one for every row tile
    int spread;  // not split: workgroups of a key head if the lengths are so uneven that it is after all; 0: it never is
    int least;   // split: key tiles of a workgroup at least
    int units;   // split: of a key head, at most
    float scale;
};

__device__ const __align__(16) uint8_t kZeros[16] = {};

constexpr int kCus = 256;
static_assert(kCounters >= 2 * kCus, "a counter for every row tile that is joined in its launch");
constexpr float kSlack = 2.75f;  // a row's maximum may be this much above the one in use
constexpr float kLog2e = 1.4426950408889634f;

// x less the lower or upper half of h, exactly: the instruction reads binary16 halves as
// they are (the compiler would convert each of them first).
__device__ __forceinline__ float less_low(float x, half2v h) {
    float y;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(y) : "v"(h), "v"(x));
    return y;
}
__device__ __forceinline__ float less_high(float x, half2v h) {
    float y;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(y) : "v"(h), "v"(x));
    return y;
}

// Float32 values in parts of 16 bits: two of binary16 (22 bits), three of bfloat16 (24).
// Weights are 2^(s - max + kBias).  Binary16: 13, its subnormal numbers begin 2^-27 below the
// largest weight, and with kSlack weights stay below 2^15.75.  Bfloat16 has float32's range and
// values up to 2^128: with -13 the sum of 2^(13 - kSlack) = 1217 weights is at most 1, so that
// sums of weights times values stay finite (the exponential's argument then rounds a little
// more coarsely: errors of 32 tokens behind 4000 6.2e-7 -> 7.4e-7 of the result).
template <int kType>
struct Math {  // binary16 (e4m3 widened to it)
    typedef half8v v8;
    static constexpr int kParts = 2;
    static constexpr float kBias = 13.f;
    static constexpr bool kScaled = true;
    __device__ static f32x16 mfma32(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
    __device__ static f32x4 mfma16(v8 a, v8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    __device__ static void split(const float *x, v8 *parts) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const half2v h = __builtin_convertvector((f32x2{x[i], x[i + 1]}), half2v);
            const half2v l = __builtin_convertvector((f32x2{less_low(x[i], h), less_high(x[i + 1], h)}), half2v);
            parts[0][i] = h.x;
            parts[0][i + 1] = h.y;
            parts[1][i] = l.x;
            parts[1][i + 1] = l.y;
        }
    }
};
template <>
struct Math<Q4K_KV_BF16> {
    typedef bf8v v8;
    static constexpr int kParts = 3;
    static constexpr float kBias = -13.f;
    static constexpr bool kScaled = false;
    __device__ static f32x16 mfma32(v8 a, v8 b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
    __device__ static f32x4 mfma16(v8 a, v8 b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    __device__ static void split(const float *x, v8 *parts) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            f32x2 rest = {x[i], x[i + 1]};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const bf2v h = __builtin_convertvector(rest, bf2v);
                parts[k][i] = h.x;
                parts[k][i + 1] = h.y;
                rest = f32x2{rest.x - static_cast<float>(h.x), rest.y - static_cast<float>(h.y)};
            }
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
// The same from base + offset, the base uniform.
__device__ __forceinline__ void copy_to_lds(const uint8_t *base, uint32_t offset, uint32_t dst) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base),
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
// Every LDS operation of this wave has ended (copies may be on their way).
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}
// What lanes of this wave have put into LDS is there for its other lanes (which execute
// in order; the compiler may otherwise move accesses that it finds to be apart).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
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
    uint64_t missing;  // lanes whose entry is no page
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
        missing = ~0ull;
    }
    // Makes the pages of keys j0 .. j0 + 63 at most available.
    __device__ void look_up(int j0, int keys) {
        if (((j0 + keys - 1) >> shift) >= first + 64 || first < 0) {
            first = j0 >> shift;
            const int at = first + (threadIdx.x & 63);
            entry = at < max_pages ? row[at] : -1;
            if (entry >= pages) entry = -1;
            missing = __ballot(entry < 0);
        }
    }
    // Whether keys j0 .. j0 + keys - 1 are all there.
    __device__ bool whole(int j0, int keys) const {
        const int at = (j0 >> shift) - first, more = ((j0 + keys - 1) >> shift) - (j0 >> shift);
        return j0 + keys <= stop && (missing >> at & (2ull << more) - 1) == 0;
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
template <int RB, int COPIES, int UNROLL>
__device__ __forceinline__ void copy_rows(const Pages &g, int j0, bool whole, int at, uint32_t k_lds, uint32_t v_lds) {
    constexpr int kPieces = RB / 16, kRows = 1024 / RB;
    const int lane = threadIdx.x & 63;
    if (whole && g.row_bytes == RB && 1 << g.shift >= kRows) {
        // Every copy's rows are in one page: a uniform address, and the lane's place
        // behind it.  The swizzles are exclusive ors of bits of the row, and the
        // copy's number has bits of its own in it.
        static_assert((COPIES & (COPIES - 1)) == 0, "rows of a copy: the first copy's with bits set");
        const int row = at / RB + lane / kPieces;
        const uint32_t in_copy = lane / kPieces * RB;
        uint32_t xk = (lane % kPieces ^ swizzle_k<RB>(row)) * 16, xv = (lane % kPieces ^ swizzle_v<RB>(row)) * 16;
        asm volatile("" : "+v"(xk), "+v"(xv));  // (two registers kept, not two for every copy)
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int j = __builtin_amdgcn_readfirstlane(j0 + (at + i * 1024) / RB);
            const int page = __builtin_amdgcn_readlane(g.entry, (j >> g.shift) - g.first);
            const uint64_t off = g.offset(page, j);
            copy_to_lds(g.k + off, in_copy + (xk ^ swizzle_k<RB>(i * kRows) * 16), k_lds + at + i * 1024);
            copy_to_lds(g.v + off, in_copy + (xv ^ swizzle_v<RB>(i * kRows) * 16), v_lds + at + i * 1024);
        }
        return;
    }
#pragma unroll UNROLL
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
__device__ __forceinline__ uint64_t there(const Pages &g, int j0, bool whole, int keys) {
    if (whole) return ~0ull;
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
#pragma unroll 4
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
    wave_sync();
    return __ballot(any != 0) != 0;
}

// ---- the division of the work ---------------------------------------------------
//
// A key head's work is one line of key tiles: those of the first row tile of the
// first sequence that has new tokens, those of the next one, and so on.  Where
// there are fewer row tiles than workgroups that the card holds (a.target), the
// line is cut into that many equal pieces, so that all of them end at the same
// time whatever the lengths are; workgroup w takes piece w.  What it has of a row
// tile is a unit.  At most one row tile begins in a workgroup and goes on in the
// next: what workgroup w has of the one that begins in w0 has number w0 + w, so a
// row tile's units follow each other, and the next such row tile (which begins in
// the last one's workgroup or later) has higher numbers.  With as many row tiles
// or more, every workgroup takes one, the most keys first; but where the longest
// would take far longer than its share (a.spread), the line is cut all the same.

struct Unit {
    int b, first, n;  // sequence, its first row of q, its new tokens
    int length;       // its tokens
    int tile;         // of its row tiles
    int begin, end;   // key tiles
    int64_t number;
    int unit0, units;  // the row tile's
    int64_t w0;        // the workgroup that it begins in
};

// Where the plan of a sequence's row tile is kept (below tokens * group / ROWS + count).
template <int ROWS>
__device__ __forceinline__ int64_t slot_of(const Attend &a, int b, int first, int64_t tile) {
    return static_cast<int64_t>(first) * a.group / ROWS + b + tile;
}

// The launch behind this one finds the row tile's units there.
template <int ROWS>
__device__ __forceinline__ void note_units(const Attend &a, const Unit &u) {
    const int64_t slot = slot_of<ROWS>(a, u.b, u.first, u.tile);
    if (slot < a.slots) a.plan[slot] = Part{u.unit0, u.units};
}

__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t low = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
    const uint32_t high = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(x) >> 32));
    return static_cast<int64_t>(static_cast<uint64_t>(high) << 32 | low);
}

// 64 sequences from b on, one a lane: their row tiles, the key tiles of one (at
// least 1: a row that sees nothing has its zeros written), and both summed up to
// and with them.
template <int ROWS, int KT>
struct Span {
    int first, n, length, key_tiles;
    int64_t tiles, line, tiles_sum, line_sum;
    __device__ Span(const Attend &a, bool line_wanted, int b, int64_t tiles_before, int64_t line_before) {
        const Paged &p = a.p;
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));  // (no addresses kept from one unit to the next)
        first = n = length = 0;
        if (line_wanted && b + lane < p.count) {
            first = offset_of(p, b + lane);
            n = max(offset_of(p, b + lane + 1) - first, 0);
            length = max(p.lengths[b + lane], 0);  // (without tokens nothing is seen)
        }
        tiles = (static_cast<int64_t>(n) * a.group + ROWS - 1) / ROWS;
        key_tiles = max((min(length, p.max_pages << p.shift) + KT - 1) / KT, 1);
        line = tiles * key_tiles;
        tiles_sum = tiles;
        line_sum = line;
        if (p.count == 1 || !line_wanted) {  // (one user's token: 0.3 us less)
            tiles_sum = uniform(tiles);
            line_sum = uniform(line);
            return;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int64_t x = __shfl_up(tiles_sum, o), y = __shfl_up(line_sum, o);
            if (lane >= o) {
                tiles_sum += x;
                line_sum += y;
            }
        }
        tiles_sum += tiles_before;
        line_sum += line_before;
    }
};

// a / b of uniform numbers, a not negative, b positive, by way of a double (the
// compiler's four divisions of 64 bits took 2 us of a workgroup's start).  The
// hardware's reciprocal is far coarser than a double, so that the first quotient may be
// off by more than one where it is large; the loop makes it exact, by a true division
// of what remains.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    asm volatile("" : "+v"(b));  // (its double is not kept over the products)
    int64_t q = static_cast<int64_t>(static_cast<double>(a) * __builtin_amdgcn_rcp(static_cast<double>(b)));
    int64_t rest = a - q * b;
    while (rest < 0 || rest >= b) {
        const int64_t more = static_cast<int64_t>(floor(static_cast<double>(rest) / static_cast<double>(b)));
        q += more;
        rest -= more * b;
    }
    return q;
}

__device__ __forceinline__ float uniform_of(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// A sum (or largest) over a wave's lanes, of numbers not below 0; uniform.
template <typename Op>
__device__ __forceinline__ int reduced(int x, Op op) {
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false));  // a row of 16 lanes: from 1 below,
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false));  // 2,
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false));  // 4,
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false));  // 8;
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false));  // lane 15 to the second row, 47 to the fourth,
    x = op(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false));  // lane 31 to the upper half
    return __builtin_amdgcn_readlane(x, 63);
}

// As many row tiles as workgroups: their line is cut all the same where the longest context has so many key tiles,
// and so many times a workgroup's share.  A workgroup by itself walks over 128 keys of 128 x 16 bits in 1.84 us, 512
// at once in 6.5, so that the longest row tile lasts beyond the others from 3.5 times the share on.  (One token of
// each of 64 sequences, one of them over 131072 keys and 63 over 300: 1870 us uncut and 127 cut; over 16000 keys and
// 2000, 289 and 110; comparing the lengths costs 1% of a batch of 200 over 1000 keys.)
constexpr int kUnevenTiles = 32;
constexpr float kUneven = 4.f;

// Sequences whose row tiles are ranked together.
constexpr int sequences_at_once(int rows) { return rows < 128 ? 256 : 64; }

// A workgroup's piece of the line.  kKeep: the 64 sequences last looked through stay
// in registers; without it (where the products need them) they are looked through
// again for every unit.  kCut: as many row tiles as workgroups may be cut (parts are joined without a launch).
template <int ROWS, int KT, bool kKeep, bool kCut>
struct Piece {
    typedef Span<ROWS, KT> S;
    const Attend &a;
    S kept;
    int kept_b;
    int cut_target;
    // Workgroups of a key head that share the line; 0: each has a row tile.
    __device__ __forceinline__ int target() const { return kCut ? cut_target : a.target; }
    static constexpr int kAtOnce = sequences_at_once(ROWS), kSets = kAtOnce / 64;
    int64_t at, stop, size, workgroup;

    __device__ Piece(const Attend &a_, int64_t w)
        : a(a_), kept(a_, a_.target != 0, 0, 0, 0), kept_b(0), size(1), workgroup(w) {
        if constexpr (kCut) cut_target = a.target;
        if (target()) {
            share_line();
        } else {
            at = w;
            stop = at + 1;
        }
        // Of more sequences than are ranked together, those that a workgroup's rank falls to begin at the
        // slot of their first tile (some slots have no tile).  (Going through the sets instead took 3000 us
        // for one token of each of 8192 sequences over 16 keys, with this 1070; of 65535, 139700 and 8800.)
        if (!target() && a.p.count > kAtOnce) {
            const auto start = [&](int s) { return slot_of<ROWS>(a, s * kAtOnce, offset_of(a.p, s * kAtOnce), 0); };
            const int s = last_started((a.p.count + kAtOnce - 1) / kAtOnce, w, start);
            kept_b = s * kAtOnce;
            at = w - uniform(start(s));
            stop = max(at, int64_t{0}) + 1;
        }
    }
    // The line's total, and the workgroup's piece of it.
    __device__ __forceinline__ void share_line() {
        int64_t all = __shfl(kept.line_sum, 63), rows = __shfl(kept.tiles_sum, 63);
        for (int b = 64; b < a.p.count; b += 64) {
            const S x(a, true, b, rows, all);
            all = __shfl(x.line_sum, 63);
            rows = __shfl(x.tiles_sum, 63);
        }
        all = uniform(all);
        // (16-row tiles over few keys: one key tile a workgroup as long as the parts are few, 500 keys 11.3 ->
        // 9.8 us; with 32 parts of 4000 keys it took 15.7 us instead of 13.4)
        const int least = kKeep && all <= 12 * uniform(rows) ? 1 : a.least;
        size = max(uniform(quotient(all + target() - 1, target())), static_cast<int64_t>(least));
        at = workgroup * size;
        stop = !kCut || workgroup < target() ? at + size : at;
    }
    // Every workgroup has one row tile, and the ones with the most keys go first: the one of rank at by the tokens
    // before its end (counted in row tiles), of every 256 sequences (where there are many rows: 64).  Tile t of a
    // sequence has level context + t, and the tiles of a level and above are quickly counted, so the rank's level is
    // found by halving.  (In the batch's order or against it the longest may start last: seven prompts up to 1531
    // tokens 116 -> 103 us, 96 tokens over up to 4000 keys 166 -> 147, 64 chunks of 8 behind up to 4000 164 -> 116;
    // where all are alike it takes 1 us: 64 tokens over 500 keys 29.6 -> 30.7.)
    __device__ __forceinline__ bool most_keys_first(Unit &u) {
        if (at >= stop) return false;
        const Paged &p = a.p;
        const auto sum = [](int x, int y) { return x + y; };
        int lane = threadIdx.x & 63, rank = static_cast<int>(at);
        at = stop;
        u.begin = 0;
        u.end = INT_MAX;
        u.number = u.w0 = u.unit0 = 0;
        u.units = 1;
        if (p.count == 1) {  // (1 us less)
            u.b = 0;
            u.first = offset_of(p, 0);
            u.n = max(offset_of(p, 1) - u.first, 0);
            u.length = max(p.lengths[0], 0);
            u.tile = static_cast<int>((static_cast<int64_t>(u.n) * a.group + ROWS - 1) / ROWS) - 1 - rank;
            return u.tile >= 0;
        }
        int first[kSets], n[kSets], length[kSets], tiles[kSets], lowest[kSets], all = 0, end = 0, below = 0;
        constexpr int kHighest = 1 << 29;
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            const int b = kept_b + 64 * k + lane;
            first[k] = n[k] = length[k] = 0;
            if (b < p.count) {
                first[k] = offset_of(p, b);
                n[k] = max(offset_of(p, b + 1) - first[k], 0);
                length[k] = max(p.lengths[b], 0);  // (without tokens nothing is seen)
            }
        }
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            tiles[k] = static_cast<int>((static_cast<int64_t>(n[k]) * a.group + ROWS - 1) / ROWS);
            const int64_t context = static_cast<int64_t>(max(length[k] - n[k], 0)) * a.group / ROWS;
            lowest[k] = static_cast<int>(min(context, int64_t{kHighest}));
            all += tiles[k];
            if (tiles[k]) {
                end = max(end, lowest[k] + tiles[k]);
                below = max(below, kHighest - lowest[k]);
            }
        }
        const auto larger = [](int x, int y) { return max(x, y); };
        if constexpr (kCut) {
            if (a.spread) {  // (all sequences are in these sets)
                float line = 0.f;
                int longest = 0;
#pragma unroll
                for (int k = 0; k < kSets; ++k) {
                    const int key_tiles = max((min(length[k], p.max_pages << p.shift) + KT - 1) / KT, 1);
                    line += static_cast<float>(tiles[k]) * static_cast<float>(key_tiles);
                    longest = max(longest, tiles[k] ? key_tiles : 0);
                }
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) line += __shfl_xor(line, o);
                longest = reduced(longest, larger);
                if (longest >= kUnevenTiles && static_cast<float>(longest) * static_cast<float>(a.spread) > kUneven * uniform_of(line)) {
                    cut_target = a.spread;
                    kept = S(a, true, 0, 0, 0);
                    share_line();
                    return false;
                }
            }
        }
        all = reduced(all, sum);
        if (rank < 0 || rank >= all) return false;
        int low = kHighest - reduced(below, larger), high = reduced(end, larger), above = 0;
        while (high - low > 1) {
            const int middle = (low + high) >> 1;
            int more = 0;
#pragma unroll
            for (int k = 0; k < kSets; ++k) more += min(max(lowest[k] + tiles[k] - middle, 0), tiles[k]);
            more = reduced(more, sum);
            if (more > rank) {
                low = middle;
            } else {
                high = middle;
                above = more;
            }
        }
        int index = rank - above;  // among those of the level
#pragma unroll
        for (int k = 0; k < kSets; ++k) {
            uint64_t level = __ballot(lowest[k] <= low && low < lowest[k] + tiles[k]);
            if (index < __popcll(level)) {
                for (; index > 0; --index) level &= level - 1;
                const int l = __builtin_ctzll(level);
                u.b = kept_b + 64 * k + l;
                u.first = __builtin_amdgcn_readlane(first[k], l);
                u.n = __builtin_amdgcn_readlane(n[k], l);
                u.length = __builtin_amdgcn_readlane(length[k], l);
                u.tile = low - __builtin_amdgcn_readlane(lowest[k], l);
                return true;
            }
            index -= __popcll(level);
        }
        return false;  // (offsets out of order, more tiles than a word counts)
    }
    // The piece's next unit; false behind its last.  Every lane has the same.
    __device__ bool next(Unit &u) {
        if (!target()) {
            const bool taken = most_keys_first(u);
            if (!target()) return taken;
        }
        if (at >= stop) return false;
        if constexpr (!kKeep) {
            kept = S(a, true, 0, 0, 0);
            kept_b = 0;
        }
        uint64_t behind;
        while ((behind = __ballot(kept.line_sum > at)) == 0) {
            kept_b += 64;
            if (kept_b >= a.p.count) return false;
            kept = S(a, true, kept_b, __shfl(kept.tiles_sum, 63), __shfl(kept.line_sum, 63));
        }
        const int l = __builtin_ctzll(behind);
        u.b = kept_b + l;
        u.first = __builtin_amdgcn_readlane(kept.first, l);
        u.n = __builtin_amdgcn_readlane(kept.n, l);
        u.length = __builtin_amdgcn_readlane(kept.length, l);
        const int64_t rest = at - uniform(__shfl(kept.line_sum - kept.line, l));
        const int keys = __builtin_amdgcn_readlane(kept.key_tiles, l);
        u.tile = rest < keys ? 0 : static_cast<int>(uniform(quotient(rest, keys)));
        u.begin = static_cast<int>(rest - static_cast<int64_t>(u.tile) * keys);
        u.end = static_cast<int>(min(static_cast<int64_t>(keys), u.begin + (stop - at)));
        const int64_t begin = at - u.begin;  // the row tile's place on the line
        u.w0 = u.begin == 0 ? workgroup : uniform(quotient(begin, size));
        const int64_t w1 = begin + keys <= stop ? workgroup : uniform(quotient(begin + keys - 1, size));
        u.number = u.w0 + workgroup;
        u.unit0 = static_cast<int>(min(2 * u.w0, static_cast<int64_t>(a.units)));
        u.units = static_cast<int>(w1 - u.w0) + 1;
        at += u.end - u.begin;
        return true;
    }
};

// A lane's row: its query, its place in the outputs and what it sees (rows behind the
// last see anything).
struct Row {
    int64_t at;  // element of q and out; -1: no row
    int stop;    // causal: the keys below it are seen; tree: the length
    const unsigned *mask;
};

__device__ __forceinline__ Row row_of(const Attend &a, const Unit &u, int r, int head) {
    Row w;
    const int i = r / a.group, g = r - i * a.group;
    const bool real = i < u.n;
    const int64_t t = static_cast<int64_t>(u.first) + (real ? i : 0);
    w.at = real ? (t * a.q_heads + head * a.group + g) * a.p.head_dim : -1;
    w.stop = a.mask || !real ? u.length : u.length - u.n + i + 1;
    w.mask = a.mask ? a.mask + t * a.words : nullptr;
    return w;
}

// Bit k: the row sees key j0 + k, for 64 keys (before: the index of the first new token).
__device__ __forceinline__ uint64_t seen(const Attend &a, const Row &w, int before, int j0) {
    const int left = w.stop - j0;
    const uint64_t below = left >= 64 ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1;
    if (!a.mask) return below;
    const int64_t from = static_cast<int64_t>(j0) - before;  // the new token of bit 0
    if (from <= -64) return ~0ull;
    // bits from word first on, all three words asked for at once
    const int64_t first = from < 0 ? 0 : from >> 5;
    uint64_t word[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const uint32_t x = w.mask[min(first + i, static_cast<int64_t>(a.words - 1))];
        word[i] = first + i < a.words ? x : 0u;
    }
    const uint64_t low = word[0] | word[1] << 32;
    const int s = static_cast<int>(from & 31);
    const uint64_t bits = from < 0 ? low << -from | ((1ull << -from) - 1) : s ? low >> s | word[2] << (64 - s) : low;
    return bits;
}

// The query's power of two: |x| * 2^e of the largest is in [2^13, 2^14).
__device__ __forceinline__ int exponent_for(float largest) {
    if (!(largest > 0.f) || !(largest < INFINITY)) return 0;
    return min(14 - (static_cast<int>(__builtin_amdgcn_frexp_expf(largest))), 100);
}

// Eight values of the query from dimension d on.
__device__ __forceinline__ void load_query(const Attend &a, const Row &w, int d, float *x) {
    f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = x0;
    if (w.at >= 0 && d < a.p.head_dim) {
        x0 = *reinterpret_cast<const f32x4 *>(a.q + w.at + d);
        x1 = *reinterpret_cast<const f32x4 *>(a.q + w.at + d + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = x0[i];
        x[4 + i] = x1[i];
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
    static constexpr int KT = DP == 256 || (kType == Q4K_KV_BF16 && DP == 128) ? 32 : 64;  // keys of a tile
    static constexpr int kBytes = KT * RB;            // of K, and of V
    static constexpr int kCopies = kBytes / 4096;     // of a wave
    static constexpr int kMarks = KT * DP / 8;        // a bit per value
    static constexpr int kThird = kType == Q4K_KV_BF16 ? kTileRows * DP * 2 : 0;  // the queries' third parts
    static constexpr int kLds = 4 * kBytes + kMarks + 16 + kThird;
    // Workgroups, as the registers allow (64 dimensions, two: seven prompts up to 1531 tokens 94 -> 103 us).
    static constexpr int kPerCu = DP == 64 ? 3 : DP == 128 ? 2 : 1;
};

template <int kType, int DP>
__global__ __launch_bounds__(256, (TileShape<kType, DP>::kPerCu)) void attend_tiles(const Attend a) {
    typedef TileShape<kType, DP> S;
    typedef Math<kType> M;
    typedef typename M::v8 v8;
    constexpr int RB = S::RB, KT = S::KT, KS = KT / 32, NS = DP / 16, ND = DP / 32;
    extern __shared__ __align__(16) uint8_t lds[];
    uint8_t *const marks = lds + 4 * S::kBytes;
    int *const flag = reinterpret_cast<int *>(marks + S::kMarks);
    const int head = blockIdx.x % a.p.kv_heads;
    Piece<kTileRows, KT, false, false> piece(a, blockIdx.x / a.p.kv_heads);
    for (Unit u; piece.next(u); __syncthreads()) {
        int thread = threadIdx.x;
        asm volatile("" : "+v"(thread));  // (what follows from it is worked out for every unit, not kept over them)
        const int lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6), col = lane & 31, half = lane >> 5;
        const int before = u.length - u.n;
        const int row0 = u.tile * kTileRows, rows = u.n * a.group;
        const int capacity = a.p.max_pages << a.p.shift;
        // keys that some row of the tile may see, and those that every one sees
        const int last = min((row0 + kTileRows - 1) / a.group, u.n - 1);
        const int most = a.mask ? u.length : before + last + 1;
        const int common = a.mask ? before : before + row0 / a.group + 1;
        const int stop = max(min(most, capacity), 0);
        const int t0 = u.begin, t1 = min((stop + KT - 1) / KT, u.end);
        if (a.target && u.begin == 0 && head == 0 && threadIdx.x == 0) note_units<kTileRows>(a, u);
        const Row w = row_of(a, u, row0 + wave * 32 + col, head);
        const bool idle = row0 + wave * 32 >= rows;  // no row of this wave is real

        Pages pages(a.p, u.b, head, min(u.length, capacity), S::kSize);
        const uint32_t base = lds_address(lds);
        const int piece0 = wave * S::kCopies * 1024;
        // the wave's queries as the second operand of S^T = K Q^T: lane's row, 8 dimensions a
        // step; asked for before the first copies, whose addresses have to be looked up first
        float held[NS][8];
#pragma unroll
        for (int s = 0; s < NS; ++s)
            load_query(a, w, kType == Q4K_KV_E4M3 ? 32 * (s >> 1) + 16 * half + 8 * (s & 1) : 16 * s + 8 * half, held[s]);
        uint64_t here = 0;
        if (threadIdx.x == 0) *flag = -1;
        if (t0 < t1) {
            pages.look_up(t0 * KT, KT);
            const bool whole = pages.whole(t0 * KT, KT);
            here = there(pages, t0 * KT, whole, KT);
            copy_rows<RB, S::kCopies, 4>(pages, t0 * KT, whole, piece0, base, base + 2 * S::kBytes);
        }

        v8 qh[NS], ql[NS];
        // (for the third parts there are too few registers)
        u32x4 *const third = reinterpret_cast<u32x4 *>(lds + 4 * S::kBytes + S::kMarks + 16) + wave * NS * 64 + lane;
        float factor = 1.f;
        {
            const float by = a.scale * kLog2e * a.p.k_scale;
            int e = 0;
            if constexpr (M::kScaled) {
                float largest = 0.f;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 8; ++i) largest = fmaxf(largest, __builtin_fabsf(held[s][i] * by));
                e = exponent_for(fmaxf(largest, __shfl_xor(largest, 32)));
                factor = ldexpf(1.f, -e);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = held[s][i] * by;
                    if constexpr (M::kScaled) x[i] = ldexpf(x[i], e);
                }
                v8 parts[M::kParts];
                M::split(x, parts);
                qh[s] = parts[0];
                ql[s] = parts[1];
                if constexpr (M::kParts == 3) third[s * 64] = __builtin_bit_cast(u32x4, parts[2]);
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
        constexpr int kEight = 1;  // swizzle_v(row + 8) ^ swizzle_v(row), row below 8
        const int v_at = v_row * RB + 8 * (li & 1), v_x = v_c ^ swizzle_v<RB>(v_row);

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
                const bool whole = pages.whole((t + 1) * KT, KT);
                here = there(pages, (t + 1) * KT, whole, KT);
                copy_rows<RB, S::kCopies, 4>(pages, (t + 1) * KT, whole, piece0, base + (buf ^ 1) * S::kBytes,
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
            int kx = k_x, vx = v_x;
            asm volatile("" : "+v"(kx), "+v"(vx));  // the pieces' places are worked out again, not kept: registers are short here
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
                        if constexpr (M::kParts == 3) s[k] = M::mfma32(x0, __builtin_bit_cast(v8, third[c * 64]), s[k]);
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
            top *= factor;
            // The output is corrected only where a maximum has risen by more than kSlack (or from nothing).
            if (__ballot(!(top - m <= kSlack) && top != -INFINITY) != 0) {
                const float m1 = fmaxf(m, top);
                const float fade = m1 == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - m1);
                m = m1;
                sum *= fade;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[d][r] *= fade;
            }
            const float shift = M::kBias - (m == -INFINITY ? 0.f : m);
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    s[k][r] = __builtin_amdgcn_exp2f(fmaf(s[k][r], factor, shift));
                    part += s[k][r];
                }
            sum += part;
#pragma unroll
            for (int q = 0; q < KT / 16; ++q) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = s[q >> 1][8 * (q & 1) + i];
                v8 parts[M::kParts];
                M::split(x, parts);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    v8 y;
                    const uint8_t *vq = vt + q * 16 * RB;
                    if constexpr (kType == Q4K_KV_E4M3) {
                        const i32x2 z = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                            (__attribute__((address_space(3))) i32x2 *)(vq + v_at + (((2 * d) ^ vx) << 4)));
                        y = widened(z.x, z.y);
                    } else {
                        const s16x4 z0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4 *)(vq + v_at + (((4 * d) ^ vx) << 4)));
                        const s16x4 z1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                            (__attribute__((address_space(3))) s16x4 *)(vq + v_at + 8 * RB + (((4 * d) ^ vx ^ kEight) << 4)));
                        y = __builtin_bit_cast(v8, __builtin_shufflevector(z0, z1, 0, 1, 2, 3, 4, 5, 6, 7));
                    }
#pragma unroll
                    for (int i = 0; i < M::kParts; ++i) acc[d] = M::mfma32(y, parts[i], acc[d]);
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
        int r0 = row0 + wave * 32 + col, D = a.p.head_dim;
        asm volatile("" : "+v"(r0), "+s"(D));  // worked out again rather than kept over the loops
        const Row o = row_of(a, u, r0, head);
        if (o.at < 0) continue;
        float *to = a.out + o.at;
        // (v_scale / sum could be a subnormal number or infinite where the output is neither)
        float f = sum == 0.f ? 0.f : 1.f / sum, v_scale = a.p.v_scale;
        if (u.units > 1) {
            if (u.number >= a.units) continue;  // (offsets out of order)
            const int64_t at = (u.number * a.p.kv_heads + head) * kTileRows + wave * 32 + col;
            if (half == 0) {
                a.part_ml[2 * at] = m;
                a.part_ml[2 * at + 1] = sum;
            }
            if (m == -INFINITY && sum == 0.f) continue;  // the output is not read
            to = a.part + at * D;
            f = v_scale = 1.f;
        }
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const int at = 32 * d + 2 * r + 4 * half;
                if (at < D) {
                    f32x4 y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = f == 0.f ? 0.f : acc[d][r + i] * f * v_scale;
                    *reinterpret_cast<f32x4 *>(to + at) = y;
                }
            }
    }
}

// ---- few rows --------------------------------------------------------------------
//
// 16, 32 or 64 rows per workgroup, all of them in every wave; the waves take key
// tiles of 32 in turn, each with its own two buffers in LDS and its own maxima,
// sums and outputs, and nothing to wait for but its own copies; the waves' parts
// are joined at the end.  Products of 16 x 16 x 32, blocks of 16 rows: every
// value that is read from LDS serves all blocks.
//
// Units of one row tile of 16 are joined by the workgroup of the last one to end,
// without a second launch (which takes 4 to 5 us; with 64 rows it was this
// workgroup's work that took long, 20 us of 38 over 16 units).  Their parts
// go past the L2s, which the card's eight dies do not share: stores and loads of
// the agent's scope, each wave's stores waited for before the workgroup counts
// its unit as ended.  They are added in the units' order whichever came last.

// Two numbers to and from memory that all dies see.
__device__ __forceinline__ void share(float *at, float x, float y) {
    const uint64_t pair = static_cast<uint64_t>(__float_as_uint(y)) << 32 | __float_as_uint(x);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(at), pair, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2 shared_pair(const float *at) {
    const uint64_t pair = __hip_atomic_load(reinterpret_cast<const uint64_t *>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return f32x2{__uint_as_float(static_cast<uint32_t>(pair)), __uint_as_float(static_cast<uint32_t>(pair >> 32))};
}

template <int kType, int DP, int NB, bool kPaired>
struct FewShape {
    static constexpr int kRows = 16 * NB;
    static constexpr int kSize = kType == Q4K_KV_E4M3 ? 1 : 2;
    static constexpr int RB = DP * kSize;
    // Two workgroups on a CU where their LDS allows it.  Of 512-byte rows there is room for one buffer a
    // wave, of 256-byte ones too where two workgroups are wanted: a wave then computes while the
    // others' copies are on their way.
    static constexpr int kWaves = 4;
    static constexpr int kBuffers = RB == 512 || kPaired ? 1 : 2;  // of a wave
    static constexpr int kBytes = 32 * RB;  // of a tile's K, and of its V
    static constexpr int kCopies = kBytes / 1024;
    static constexpr int kJoin = kWaves * kRows * (DP + 4) * 4;
    static constexpr int kMarks = 32 * DP / 8;  // a bit per value
    static constexpr int kOwn = 2 * kBuffers * kBytes + kMarks;
    static constexpr int kEnded = kWaves * kOwn > kJoin ? kWaves * kOwn : kJoin;
    static constexpr bool kLow = NB * DP > 256;  // the queries' second parts in LDS: there are too few registers
    static constexpr int kLds = kEnded + 16 + (kLow ? kRows * DP * 2 : 0);
    static constexpr bool kJoined = NB == 1;  // in the same launch
    static constexpr int kPerCu = NB < 4 && kLds <= 81920 ? 2 : 1;
    static constexpr int kPerSimd = kPerCu;  // waves
};

template <int kType, int DP, int NB, bool kPaired>
__global__ __launch_bounds__((FewShape<kType, DP, NB, kPaired>::kWaves * 64), (FewShape<kType, DP, NB, kPaired>::kPerSimd))
    void attend_few(const Attend a) {
    typedef FewShape<kType, DP, NB, kPaired> S;
    typedef Math<kType> M;
    typedef typename M::v8 v8;
    constexpr int RB = S::RB, KT = 32 * S::kWaves, NS = DP / 32, ND = DP / 16, kRows = S::kRows;
    extern __shared__ __align__(16) uint8_t lds[];
    int *const ended = reinterpret_cast<int *>(lds + S::kEnded);
    if (S::kJoined && a.next && blockIdx.x == 0)
        for (int i = threadIdx.x; i < kCounters; i += S::kWaves * 64)
            __hip_atomic_store(a.next + i, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int head = blockIdx.x % a.p.kv_heads;
    Piece<kRows, KT, true, S::kJoined> piece(a, blockIdx.x / a.p.kv_heads);
    for (Unit u; piece.next(u); __syncthreads()) {
        int thread = threadIdx.x;
        asm volatile("" : "+v"(thread));  // (what follows from it is worked out for every unit, not kept over them)
        const int lane = thread & 63, wave = __builtin_amdgcn_readfirstlane(thread >> 6), col = lane & 15, quarter = lane >> 4;
        const int before = u.length - u.n;
        const int row0 = u.tile * kRows;
        const int capacity = a.p.max_pages << a.p.shift;
        const int last = min((row0 + kRows - 1) / a.group, u.n - 1);
        const int most = a.mask ? u.length : before + last + 1;
        const int common = a.mask ? before : before + row0 / a.group + 1;
        const int stop = max(min(most, capacity), 0);
        // tiles of 32 keys: this wave's are first, first + kWaves, ...
        const int t0 = u.begin * S::kWaves + wave;
        const int t1 = u.end == INT_MAX ? (stop + 31) / 32 : min((stop + 31) / 32, u.end * S::kWaves);
        if (!S::kJoined && a.target && u.begin == 0 && head == 0 && threadIdx.x == 0) note_units<kRows>(a, u);
        Row w[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) w[n] = row_of(a, u, row0 + 16 * n + col, head);

        Pages pages(a.p, u.b, head, min(u.length, capacity), S::kSize);
        uint8_t *const own = lds + wave * S::kOwn;
        const uint32_t base = lds_address(own);
        const auto copy = [&](int t, int buf) __attribute__((always_inline)) {
            pages.look_up(t * 32, 32);
            const bool whole = pages.whole(t * 32, 32);
            const uint64_t is = there(pages, t * 32, whole, 32);
            copy_rows<RB, S::kCopies, NB == 1 ? 4 : 1>(pages, t * 32, whole, 0, base + buf * 2 * S::kBytes,
                                                       base + (buf * 2 + 1) * S::kBytes);
            return is;
        };
        static_assert(!S::kLow || M::kParts == 2, "one part in LDS");
        v8 query[NB][NS][S::kLow ? 1 : M::kParts];
        u32x4 *const low = reinterpret_cast<u32x4 *>(lds + S::kEnded + 16) + lane;  // (every wave writes the same)
        float factor[NB];
        const float by = a.scale * kLog2e * a.p.k_scale;
        // (asked for before the first copies, whose addresses have to be looked up first)
        float held[NB][NS][8];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int d = kType == Q4K_KV_E4M3 ? 64 * (s >> 1) + 16 * quarter + 8 * (s & 1) : 32 * s + 8 * quarter;
                load_query(a, w[n], d, held[n][s]);
            }
        uint64_t here = 0;
        if (t0 < t1) here = copy(t0, 0);

#pragma unroll
        for (int n = 0; n < NB; ++n) {
            int e = 0;
            factor[n] = 1.f;
            if constexpr (M::kScaled) {
                float largest = 0.f;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 8; ++i) largest = fmaxf(largest, __builtin_fabsf(held[n][s][i] * by));
                largest = fmaxf(largest, __shfl_xor(largest, 16));
                largest = fmaxf(largest, __shfl_xor(largest, 32));
                e = exponent_for(largest);
                factor[n] = ldexpf(1.f, -e);
            }
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = held[n][s][i] * by;
                    if constexpr (M::kScaled) x[i] = ldexpf(x[i], e);
                }
                v8 split[M::kParts];
                M::split(x, split);
                query[n][s][0] = split[0];
                if constexpr (S::kLow) {
                    low[(n * NS + s) * 64] = __builtin_bit_cast(u32x4, split[1]);
                } else {
#pragma unroll
                    for (int i = 1; i < M::kParts; ++i) query[n][s][i] = split[i];
                }
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

        f32x4 acc[NB][ND];
        float m[NB], sum[NB];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            m[n] = -INFINITY;
            sum[n] = 0.f;
#pragma unroll
            for (int d = 0; d < ND; ++d) acc[n][d] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        int buf = 0;
        const auto turn = [&](int t) {
            if (S::kBuffers == 2) {
                buf ^= 1;
            } else if (t + S::kWaves < t1) {
                wait_lds();  // (nothing is on its way to the buffer any more)
                here = copy(t + S::kWaves, 0);
            }
        };
        for (int t = t0; t < t1; turn(t), t += S::kWaves) {
            const uint64_t now = here;
            if (S::kBuffers == 2 && t + S::kWaves < t1) {
                here = copy(t + S::kWaves, buf ^ 1);
                wait_copies<2 * S::kCopies>();
            } else {
                wait_copies<0>();
            }
            const uint8_t *kt = own + buf * 2 * S::kBytes;
            uint8_t *vt = own + (buf * 2 + 1) * S::kBytes, *marks = own + 2 * S::kBuffers * S::kBytes;
            const bool apart = t * 32 + 32 > common && set_apart<kType, RB, S::kBytes>(vt, 0, marks);
            uint32_t vis[NB], any = 0;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                vis[n] = static_cast<uint32_t>(seen(a, w[n], before, t * 32) & now);
                any |= vis[n];
            }
            if (__ballot(any != 0) == 0) continue;
            const auto part_of = [&](int n, int s, int i) {
                if constexpr (S::kLow)
                    if (i == 1) return __builtin_bit_cast(v8, low[(n * NS + s) * 64]);
                return query[n][s][S::kLow ? 0 : i];
            };
            f32x4 s[NB][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int n = 0; n < NB; ++n) s[n][k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < RB / 64; ++c) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(kt + k * 16 * RB + k_at + (((4 * c) ^ k_x) << 4));
                    if constexpr (kType == Q4K_KV_E4M3) {
                        const half8v x0 = widened(x.x, x.y), x1 = widened(x.z, x.w);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int n = 0; n < NB; ++n) {
                                s[n][k] = M::mfma16(x0, part_of(n, 2 * c, i), s[n][k]);
                                s[n][k] = M::mfma16(x1, part_of(n, 2 * c + 1, i), s[n][k]);
                            }
                    } else {
#pragma unroll
                        for (int i = 0; i < M::kParts; ++i)
#pragma unroll
                            for (int n = 0; n < NB; ++n)
                                s[n][k] = M::mfma16(__builtin_bit_cast(v8, x), part_of(n, c, i), s[n][k]);
                    }
                }
            }
            v8 parts[NB][M::kParts];
            float fade[NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint32_t mine = vis[n] >> (4 * quarter);
                if (__ballot(vis[n] != 0xFFFFFFFFu) != 0) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (!((mine >> (16 * k + r)) & 1)) s[n][k][r] = -INFINITY;
                }
                float top = s[n][0][0];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int r = 0; r < 4; ++r) top = fmaxf(top, s[n][k][r]);
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float m1 = fmaxf(m[n], top * factor[n]);
                const float zero = m1 == -INFINITY ? 0.f : m1;
                fade[n] = __builtin_amdgcn_exp2f(m[n] - zero);
                m[n] = m1;
                const float shift = M::kBias - zero;
                float x[8], part = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] = __builtin_amdgcn_exp2f(fmaf(s[n][i >> 2][i & 3], factor[n], shift));
                    part += x[i];
                }
                sum[n] = fmaf(sum[n], fade[n], part);
                M::split(x, parts[n]);
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
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
#pragma unroll
                for (int n = 0; n < NB; ++n) acc[n][d] *= fade[n];
#pragma unroll
                for (int i = 0; i < M::kParts; ++i)
#pragma unroll
                    for (int n = 0; n < NB; ++n) acc[n][d] = M::mfma16(y, parts[n][i], acc[n][d]);
            }
            if (apart) {
#pragma unroll 1
                for (int i = 0; i < 32 * DP / 8; ++i) {
                    const uint32_t marked = marks[i];
                    if (marked == 0) continue;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const uint32_t bits = (vis[n] >> (i / (DP / 8))) & 1 ? marked : 0;
#pragma unroll
                        for (int d = 0; d < ND; ++d)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int at = 16 * d + 4 * quarter + r - i % (DP / 8) * 8;
                                if (static_cast<unsigned>(at) < 8u && ((bits >> at) & 1)) acc[n][d][r] = nan_value();
                            }
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            sum[n] += __shfl_xor(sum[n], 16);
            sum[n] += __shfl_xor(sum[n], 32);
        }

        // the waves' parts: [wave][row][DP] and behind them maximum, sum and the row's place (stride DP + 4 words)
        wait_copies<0>();
        barrier();
        float *const po = reinterpret_cast<float *>(lds);
        constexpr int kStride = DP + 4;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            float *mine = po + (wave * kRows + 16 * n + col) * kStride;
#pragma unroll
            for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4 *>(mine + 16 * d + 4 * quarter) = acc[n][d];
            if (quarter == 0) {
                mine[DP] = m[n];
                mine[DP + 1] = sum[n];
                *reinterpret_cast<int64_t *>(mine + DP + 2) = w[n].at;
            }
        }
        __syncthreads();
        const int quads = a.p.head_dim / 4;
        // (offsets out of order can give more units or row tiles than there is room for)
        const int64_t counter = u.w0 * a.p.kv_heads + head;
        const bool shared = u.units > 1 && u.unit0 + u.units <= a.units && (!S::kJoined || counter < kCounters);
        const int at_once = S::kWaves * 64 / quads;  // rows
        const auto at_of = [&](int r) { return *reinterpret_cast<const int64_t *>(po + r * kStride + DP + 2); };
        const int real = min(u.n * a.group - row0, kRows), d = (thread % quads) * 4;
        for (int r = thread / quads; r < real; r += at_once) {
            if (thread >= at_once * quads) break;
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < S::kWaves; ++k) top = fmaxf(top, po[(k * kRows + r) * kStride + DP]);
            const float zero = top == -INFINITY ? 0.f : top;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
            float total = 0.f;
#pragma unroll
            for (int k = 0; k < S::kWaves; ++k) {
                const float *from = po + (k * kRows + r) * kStride;
                // a wave without keys has nothing to add (its maximum is -inf)
                const float f = __builtin_amdgcn_exp2f(from[DP] - zero);
                total = fmaf(from[DP + 1], f, total);
                y += *reinterpret_cast<const f32x4 *>(from + d) * f;
            }
            if (u.units == 1) {
                if (total == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
                else y = y * (1.f / total) * a.p.v_scale;
                *reinterpret_cast<f32x4 *>(a.out + at_of(r) + d) = y;
            } else if (shared) {
                const int64_t at = (u.number * a.p.kv_heads + head) * kRows + r;
                if constexpr (S::kJoined) {
                    share(a.part + at * a.p.head_dim + d, y.x, y.y);
                    share(a.part + at * a.p.head_dim + d + 2, y.z, y.w);
                    if (d == 0) share(a.part_ml + 2 * at, top, total);
                } else {
                    *reinterpret_cast<f32x4 *>(a.part + at * a.p.head_dim + d) = y;
                    if (d == 0) *reinterpret_cast<f32x2 *>(a.part_ml + 2 * at) = f32x2{top, total};
                }
            }
        }
        if (!S::kJoined || !shared) continue;
        // the row tile's last unit to end joins them all
        wait_copies<0>();  // what this wave has shared is there for the others
        __syncthreads();
        if (threadIdx.x == 0) {
            const bool last = __hip_atomic_fetch_add(a.counters + counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                              static_cast<uint32_t>(u.units - 1);
            if (last) __hip_atomic_store(a.counters + counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *ended = last;
        }
        __syncthreads();
        if (!*ended) continue;
        const auto place = [&](int c, int r) { return (static_cast<int64_t>(u.unit0 + c) * a.p.kv_heads + head) * kRows + r; };
        for (int r = thread / quads; r < real; r += at_once) {
            if (thread >= at_once * quads) break;
            float top = -INFINITY, total = 0.f;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
            const float *from = a.part + place(0, r) * a.p.head_dim + d, *from_ml = a.part_ml + 2 * place(0, r);
            const int64_t step = static_cast<int64_t>(a.p.kv_heads) * kRows;
            constexpr int kAtOnce = 8;  // all asked for together (behind the last unit: that one again)
            for (int c0 = 0; c0 < u.units; c0 += kAtOnce) {
                f32x2 ml[kAtOnce], y0[kAtOnce], y1[kAtOnce];
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) {
                    const int64_t at = min(c0 + c, u.units - 1) * step;
                    ml[c] = shared_pair(from_ml + 2 * at);
                    y0[c] = shared_pair(from + at * a.p.head_dim);
                    y1[c] = shared_pair(from + at * a.p.head_dim + 2);
                }
                float top1 = top;
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) top1 = fmaxf(top1, ml[c].x);
                const float zero = top1 == -INFINITY ? 0.f : top1, fade = __builtin_amdgcn_exp2f(top - zero);
                top = top1;
                total *= fade;
                y *= fade;
#pragma unroll
                for (int c = 0; c < kAtOnce; ++c) {
                    const float f = c0 + c < u.units ? __builtin_amdgcn_exp2f(ml[c].x - zero) : 0.f;
                    if (c0 + c < u.units) {
                        total = fmaf(ml[c].y, f, total);
                        y += f32x4{y0[c].x, y0[c].y, y1[c].x, y1[c].y} * f;
                    }
                }
            }
            if (total == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
            else y = y * (1.f / total) * a.p.v_scale;
            *reinterpret_cast<f32x4 *>(a.out + at_of(r) + d) = y;
        }
    }
}

// ---- the units' parts joined -------------------------------------------------------
//
// A row's units: their maxima and sums by lanes, then their outputs, four values
// a lane; the lanes that one unit's output leaves free take the next units, and
// their sums are added in a fixed order.  A unit whose maximum is -inf has seen
// nothing, or NaN only (and may have written no output).  kThreads a row: a
// workgroup where there are few rows (and many units), else a wave.

template <int ROWS, int kThreads>
__global__ __launch_bounds__(256) void join_units(const Attend a) {
    constexpr int kRows = 256 / kThreads;
    __shared__ float weights[256];
    __shared__ __align__(16) f32x4 sums[256];
    __shared__ float tops[4], totals[4];
    const int mine = threadIdx.x / kThreads, tid = threadIdx.x % kThreads, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kRows + mine;  // query t, head h: uniform in a wave
    const int t = static_cast<int>(id / a.q_heads), h = static_cast<int>(id - static_cast<int64_t>(t) * a.q_heads);
    const Paged &p = a.p;
    Part part = {0, 0};
    int head = 0, r = 0;
    if (t < p.tokens) {
        const int b = last_started(p.count, t, [&](int i) { return offset_of(p, i); });
        const int first = offset_of(p, b), end = offset_of(p, b + 1);
        if (t >= first && t < end) {
            head = h / a.group;
            const int64_t row = static_cast<int64_t>(t - first) * a.group + h % a.group;
            r = static_cast<int>(row % ROWS);
            const int64_t slot = slot_of<ROWS>(a, b, first, row / ROWS);
            if (slot < a.slots) part = a.plan[slot];
        }
    }
    // (what offsets out of order left in the plan is not followed)
    const bool here = part.units > 1 && part.unit0 >= 0 && part.units <= a.units - part.unit0;
    const int units = here ? part.units : 0;
    const int D = p.head_dim, quads = D / 4, streams = kThreads / quads;
    const int quad = tid % quads, stream = tid / quads;
    const auto place = [&](int c) { return (static_cast<int64_t>(part.unit0 + c) * p.kv_heads + head) * ROWS + r; };
    const auto sync = [&] {
        if (kThreads > 64) __syncthreads();
        else wave_sync();
    };
    float top = -INFINITY;
    for (int c = tid; c < units; c += kThreads) top = fmaxf(top, a.part_ml[2 * place(c)]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (kThreads > 64) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    }
    const float zero = top == -INFINITY ? 0.f : top;
    float *const weight = weights + mine * kThreads;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
    for (int c0 = 0; c0 < units; c0 += kThreads) {
        sync();
        const int n = min(units - c0, kThreads);
        if (tid < n) {
            const float m = a.part_ml[2 * place(c0 + tid)];
            const float f = __builtin_amdgcn_exp2f(m - zero);
            weight[tid] = m == -INFINITY ? -1.f : f;  // -1: nothing to add, and nothing to read
            total = fmaf(a.part_ml[2 * place(c0 + tid) + 1], f, total);  // (a sum of NaN only has no maximum)
        }
        sync();
        if (stream < streams) {
            const float *from = a.part + place(c0) * D + quad * 4;
            const int64_t step = static_cast<int64_t>(p.kv_heads) * ROWS * D;
#pragma unroll 8
            for (int c = stream; c < n; c += streams) {
                const float f = weight[c];
                if (!(f < 0.f)) y += *reinterpret_cast<const f32x4 *>(from + c * step) * f;
            }
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o);
    sums[threadIdx.x] = y;
    if (kThreads > 64) {
        if (lane == 0) totals[wave] = total;
        __syncthreads();
        total = (totals[0] + totals[1]) + (totals[2] + totals[3]);
    } else {
        sync();
    }
    if (!here || tid >= quads) return;
    for (int k = 1; k < streams; ++k) y += sums[mine * kThreads + k * quads + tid];
    if (total == 0.f) y = f32x4{0.f, 0.f, 0.f, 0.f};
    else y = y * (1.f / total) * p.v_scale;
    *reinterpret_cast<f32x4 *>(a.out + id * D + tid * 4) = y;
}

// ---- launches ------------------------------------------------------------------------

// Row tiles of a key head at most: the sum of ceil(n_b * group / rows) over the
// sequences that have new tokens (at most T of them).
int64_t tiles_at_most(const Attend &a, int rows) {
    return (static_cast<int64_t>(a.p.tokens) * a.group + static_cast<int64_t>(min(a.p.count, a.p.tokens)) * (rows - 1)) / rows;
}

template <int ROWS, int KT, bool kJoined, class Kernel>
int launch(Attend &a, Kernel kernel, int threads, int lds, int per_cu, int least, hipStream_t stream) {
    const int64_t tiles = tiles_at_most(a, ROWS), heads = a.p.kv_heads;
    const int64_t capacity = static_cast<int64_t>(a.p.max_pages) << a.p.shift;
    int64_t target = (static_cast<int64_t>(kCus) * per_cu + heads - 1) / heads;
    const int64_t held = target;
    // (as many row tiles, or not two workgroups' worth of keys in the longest sequence that can be)
    if (tiles >= target || capacity <= static_cast<int64_t>(least) * KT) target = 0;
    // (lengths may be uneven: several sequences, as many as a workgroup ranks, and a table wide enough)
    const bool cut = kJoined && !target && held > 1 && a.p.count > 1 && a.p.count <= sequences_at_once(ROWS) &&
                     capacity >= kUnevenTiles * KT;
    a.target = static_cast<int>(target);
    a.spread = cut ? static_cast<int>(held) : 0;
    a.least = least;
    a.slots = static_cast<int64_t>(a.p.tokens) * a.group / ROWS + a.p.count;
    a.units = static_cast<int>(2 * held);
    const int64_t workgroups = target ? target : a.p.count > sequences_at_once(ROWS) ? a.slots : tiles;
    if (workgroups * heads * threads > UINT32_MAX) return Q4K_ERR_LAUNCH;
    if (target || cut) {
        const size_t rows = static_cast<size_t>(a.units) * heads * ROWS;
        float *ws = nullptr;
        const size_t bytes = rows * (a.p.head_dim + 2) * sizeof(float) + (target ? a.slots * sizeof(Part) : 0);
        if (workspace(stream, bytes, &ws, 0) != hipSuccess) return Q4K_ERR_ALLOC;
        a.part = ws;
        a.part_ml = ws + rows * a.p.head_dim;
        a.plan = reinterpret_cast<Part *>(a.part_ml + 2 * rows);
        // (row tiles that are cut, of all key heads: one for each workgroup but the last of a head, below kCus * per_cu)
        if (kJoined && counters(stream, &a.counters, &a.next) != hipSuccess) return Q4K_ERR_ALLOC;
    }
    if (lds > 65536 && allow_dynamic_lds(reinterpret_cast<const void *>(kernel), lds) != hipSuccess) return Q4K_ERR_LAUNCH;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(workgroups * heads)), dim3(threads), lds, stream, a);
    if (hipGetLastError() != hipSuccess) return Q4K_ERR_LAUNCH;
    if constexpr (!kJoined) {
        if (target) {
            const int outputs = a.p.tokens * a.q_heads;
            if (outputs <= 2048)
                hipLaunchKernelGGL((join_units<ROWS, 256>), dim3(outputs), dim3(256), 0, stream, a);
            else
                hipLaunchKernelGGL((join_units<ROWS, 64>), dim3((outputs + 3) / 4), dim3(256), 0, stream, a);
            if (hipGetLastError() != hipSuccess) return Q4K_ERR_LAUNCH;
        }
    }
    return Q4K_OK;
}

template <int kType, int DP, int NB, bool kPaired = false>
int launch_few(Attend &a, hipStream_t stream) {
    typedef FewShape<kType, DP, NB, kPaired> S;
    return launch<S::kRows, 32 * S::kWaves, S::kJoined>(a, attend_few<kType, DP, NB, kPaired>, S::kWaves * 64, S::kLds,
                                                        S::kPerCu, 2, stream);
}

template <int kType, int DP>
int launch_shape(Attend &a, hipStream_t stream) {
    // Rows of a sequence on average: the smallest tiles that hold them (as far as the registers go).  (The lengths
    // are on the device, so a batch of unlike sequences takes what its average asks for: 31 tokens and a chunk of 256,
    // all behind 2000 keys, 32/8 heads of 128 x 16 bits, 142 us where the two alone take 45 and 43; with a chunk of 64
    // 51 against 45 and 30; seven tokens and a chunk of 512 74 against 17 and 62.)
    constexpr bool kBf16 = kType == Q4K_KV_BF16;
    const int64_t rows = (static_cast<int64_t>(a.p.tokens) * a.group + a.p.count - 1) / a.p.count;
    // Few tiles of 16 rows over a short context: each takes its keys by itself, which costs less than
    // the wider tiles' longer steps and second launch (8, 16 and 32 tokens, four query heads a key head,
    // 4000 keys of 128 x 16 bits: 21 -> 18, 29 -> 18, 27 -> 20 us; from 8000 keys on the keys read again
    // cost more: 22 -> 28, 30 -> 32, 28 -> 41).  The table's width says how long a context can be.  With more rows
    // the gain gets small over 4000 keys (33, 48 and 64 tokens 27 -> 26, 28 -> 29, 30 -> 26 us, two chunks of 32
    // 37 -> 37) and stays over 1000 (28 -> 18, 30 -> 20, 33 -> 18): the limit is on the safe side.
    const bool narrow = rows <= 128 && tiles_at_most(a, 16) * a.p.kv_heads <= kCus / 4 &&
                        static_cast<int64_t>(a.p.max_pages) << a.p.shift <= 6000;
    if (rows <= 16 || narrow) {
        // 128 KB of LDS are one workgroup on a CU with two buffers a wave, or two with one: with
        // many row tiles a workgroup's start hides behind the other's copies and eight waves
        // compute (48 sequences of 4096 keys on average, 128 x 16 bits: 105 -> 85 us, 16 of 16000:
        // 202 -> 187, eight tiles over 4000 keys: 24.5 -> 21.9), with a few there would be twice
        // the parts to join (one sequence of 16000 keys: 21 -> 25 us, four tiles over 4000:
        // 17.7 -> 21.8).
        if constexpr (FewShape<kType, DP, 1, false>::RB == 256)
            if (4 * tiles_at_most(a, 16) * a.p.kv_heads >= kCus) return launch_few<kType, DP, 1, true>(a, stream);
        return launch_few<kType, DP, 1>(a, stream);
    }
    if constexpr (DP <= (kBf16 ? 128 : 256))
        if (rows <= 32) return launch_few<kType, DP, 2>(a, stream);
    if constexpr (DP <= (kBf16 ? 64 : 128))
        if (rows <= 64) return launch_few<kType, DP, 4>(a, stream);
    typedef TileShape<kType, DP> S;
    // (split for two a CU at most: with three, 64 row tiles a key head are split too, 59 -> 96 us)
    return launch<kTileRows, S::KT, false>(a, attend_tiles<kType, DP>, 256, S::kLds, S::kPerCu < 2 ? 1 : 2, 4, stream);
}

template <int kType>
int launch_type(Attend &a, hipStream_t stream) {
    const int D = a.p.head_dim;
    return D <= 64    ? launch_shape<kType, 64>(a, stream)
           : D <= 128 ? launch_shape<kType, 128>(a, stream)
                      : launch_shape<kType, 256>(a, stream);
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
