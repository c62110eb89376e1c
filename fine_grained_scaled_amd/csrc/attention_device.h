// attention_device.h -- device helpers shared by the attention kernels:
// where a workgroup's rows lie in the packed sequences, staging of row tiles
// in LDS, and the reads of matrix operands from it (internal header of libfgs).
#pragma once

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_v4;

__device__ __forceinline__ f32x16 mfma(const bf16x8& a, const bf16x8& b, const f32x16& c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The lane halves of a 32x32 accumulator tile: register i of lane l holds
// column l % 32 and row 8 (i / 4) + 4 (l / 32) + i % 4.
__device__ __forceinline__ int acc_row(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

__device__ __forceinline__ float swap_half(float x)
{
    auto r = __builtin_amdgcn_permlane32_swap(as_u32(x), as_u32(x), false, false);
    return as_f32((threadIdx.x & 32) ? r[0] : r[1]);
}

// Eight accumulator registers as the B operand of a 16-deep product whose
// contraction runs over the accumulator's rows.  Operand slot (half, j) then
// stands for row 4 half + j (j < 4) or 8 + 4 half + j - 4: the rows that the
// lane already holds, so nothing crosses lanes; read_tr() below brings the
// other operand in the same order.
__device__ __forceinline__ bf16x8 pack8(const f32x16& s, int i0)
{
    bf16x8 r;
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (__bf16)s[i0 + j];
    return r;
}

// ------------------------------------------------------------------------
// Rows of D bf16 in LDS, D * 2 bytes apart, in 16-byte chunks; chunk c of
// row r sits in slot c ^ f(r).  f is chosen so that both kinds of read touch
// every bank once: 16 rows of one chunk (the row-major operand), and 4 rows
// of 4 neighbouring chunks (the transposed one).
// ------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ constexpr uint32_t swizzle(uint32_t r)
{
    return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
}

// Global -> LDS copies of 16 bytes a lane that pass no register: lane i
// fills bytes 16 i .. of the wave's 1 KiB span at lds_addr (uniform).  They
// are issued from assembly so that the compiler does not make every later
// LDS read wait for them; publish() waits for them by hand.
__device__ __forceinline__ void g2lds16(const void* base, uint32_t off, uint32_t lds_addr)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(lds_addr) : "memory", "m0");
}
__device__ __forceinline__ void g2lds4(const void* base, uint32_t off, uint32_t lds_addr)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :: "v"(off), "s"(base), "s"(lds_addr) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_ptr)p));
}
template <class T>
__device__ __forceinline__ const T* uniform_ptr(const T* q)
{
    const uint64_t v = reinterpret_cast<uint64_t>(q);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const T*>(((uint64_t)hi << 32) | lo);
}

// This wave's copies have landed and its LDS reads are done, and so for
// every other wave of the workgroup.
__device__ __forceinline__ void publish()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Every load into registers so far has landed, in a form that the compiler
// sees: before a loop that issues copies, or its waits for those registers
// inside the loop would wait for the copies as well.
__device__ __forceinline__ void registers_landed() { __builtin_amdgcn_s_waitcnt(0x0F70); }   // vmcnt(0)

// ROWS rows at `base` (uniform; row stride ld bytes, below 2^24) into LDS at
// `lds`, split over the workgroup's WAVES waves.  Rows past `last` repeat row
// `last`, so nothing outside the sequence is read.
template <int D, int ROWS, int WAVES>
__device__ __forceinline__ void stage(const void* base, uint32_t ld, int last, uint32_t lds, int wave, int lane)
{
    constexpr int SLOTS = D / 8, PER = 64 / SLOTS, N = ROWS / PER / WAVES;
    static_assert(N * PER * WAVES == ROWS, "whole copies");
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int copy = wave * N + j;
        const int r = copy * PER + lane / SLOTS;
        const uint32_t c = (uint32_t)(lane % SLOTS) ^ swizzle<D>(r);
        g2lds16(base, __umul24((uint32_t)min(r, last), ld) + c * 16, lds + copy * 1024);
    }
}

// The row-major operand of rows r0 + l % 32 (r0 a multiple of 16): 8 values
// of the 16-deep step ks, values 16 ks + 8 (l / 32) .. .
template <int D>
__device__ __forceinline__ bf16x8 read_rows(const char* tile, int r0, int ks, int lane)
{
    const uint32_t r = r0 + (lane & 31);
    const uint32_t c = (uint32_t)(2 * ks + (lane >> 5)) ^ swizzle<D>(lane & 31);
    return *reinterpret_cast<const bf16x8*>(tile + r * (D * 2) + c * 16);
}

// The transposed operand: columns 32 dt + l % 32 of the tile, contracted
// over rows r0 .. r0 + 15 (r0 a multiple of 16) in the order of pack8().
// One ds_read_b64_tr_b16 gives each lane 4 rows of its column: the 16 lanes
// of a group address 4 rows of 16 columns, 8 bytes each.
template <int D>
__device__ __forceinline__ bf16x8 read_tr(const char* tile, int r0, int dt, int lane)
{
    const int half = lane >> 5, i = lane & 15;
    const uint32_t c = 4 * dt + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    const uint32_t ra = r0 + 4 * half + (i >> 2), rb = ra + 8;
    const uint32_t fa = swizzle<D>(4 * half + (i >> 2)), fb = swizzle<D>(8 + 4 * half + (i >> 2));
    union { s16x4 s[2]; bf16x8 v; } u;
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(tile + ra * (D * 2) + (c ^ fa) * 16 + 8 * (i & 1)));
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(tile + rb * (D * 2) + (c ^ fb) * 16 + 8 * (i & 1)));
    return u.v;
}

// The same operands by LDS address.  A tile starts at a multiple of 256
// bytes, so the swizzled chunk of step ks (of column block dt) is one XOR
// away from that of step 0: a kernel short of registers keeps one address
// for the tile instead of one for each step.
typedef const __attribute__((address_space(3))) bf16x8* lds_operand;
template <int D>
__device__ __forceinline__ uint32_t rows_address(int lane)
{
    return (lane & 31) * (D * 2) + (((uint32_t)(lane >> 5) ^ swizzle<D>(lane & 31)) << 4);
}
__device__ __forceinline__ bf16x8 read_rows_at(uint32_t address, int ks, uint32_t offset)
{
    return *(lds_operand)(uintptr_t)((address ^ (ks << 5)) + offset);
}
template <int D>
__device__ __forceinline__ uint32_t tr_address(int lane)
{
    const int half = lane >> 5, i = lane & 15;
    const uint32_t r = 4 * half + (i >> 2), c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    return r * (D * 2) + ((c ^ swizzle<D>(r)) << 4) + 8 * (i & 1);
}
template <int D>
__device__ __forceinline__ bf16x8 read_tr_at(uint32_t address, int r0, int dt, uint32_t offset)
{
    // eight rows on, one bit of the swizzle differs
    constexpr uint32_t flip = swizzle<D>(8) << 4;
    union { s16x4 s[2]; bf16x8 v; } u;
    const uint32_t a = address ^ (dt << 6);
    u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(uintptr_t)(a + (r0 * (D * 2) + offset)));
    u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(uintptr_t)((a ^ flip) + ((r0 + 8) * (D * 2) + offset)));
    return u.v;
}

// Two rows' product, from the halves that two lanes hold.
template <int D>
__device__ __forceinline__ float dot_rows(const uint16_t* a, const uint16_t* b, int half)
{
    float dot = 0.0f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const bf16x8 x = *reinterpret_cast<const bf16x8*>(a + 16 * ks + 8 * half);
        const bf16x8 y = *reinterpret_cast<const bf16x8*>(b + 16 * ks + 8 * half);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = __builtin_fmaf((float)x[j], (float)y[j], dot);
    }
    return dot + swap_half(dot);
}
// acc += f times a row, the lane's values of it.
template <int D>
__device__ __forceinline__ void add_row(f32x16* acc, float f, const uint16_t* row, int half)
{
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const bf16x4 x = *reinterpret_cast<const bf16x4*>(row + 32 * dt + 8 * g + 4 * half);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[dt][4 * g + j] = __builtin_fmaf(f, (float)x[j], acc[dt][4 * g + j]);
        }
}

// Whether a lane's row or key came out non-finite, in both of its halves.
template <int D>
__device__ __forceinline__ bool non_finite(const f32x16* acc)
{
    float bad = 0.0f;                          // 0 * x is NaN for a non-finite x and 0 otherwise
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) bad = __builtin_fmaf(0.0f, acc[dt][i], bad);
    bad += swap_half(bad);
    return bad != bad;
}
// Whether a NaN or Inf is among rows first .. first + ROWS - 1 of `base` (rows
// past `last` are not read): the largest magnitude of all, as integers.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
template <int D, int ROWS>
__device__ __forceinline__ bool rows_non_finite(const uint16_t* base, int64_t ld, int first, int last, int lane)
{
    u16x2 top = {0, 0};
#pragma unroll 4
    for (int j = 0; j < ROWS * D / 512; ++j) {
        const int row = min(first + (64 * j + lane) / (D / 8), last);
        const u32x4 w = *reinterpret_cast<const u32x4*>(base + row * ld + 8 * (lane % (D / 8)));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i] & 0x7FFF7FFFu));
    }
    return __any(max(top[0], top[1]) >= 0x7F80);
}

// An accumulator tile set acc[D / 32] (rows: values of the head, column: the
// lane's row) written as bf16 to one row per lane, times f: the lane halves
// swap 4-value pieces so that each lane writes 16 bytes.
template <int D>
__device__ __forceinline__ void store_row(uint16_t* row, const f32x16* acc, float f, int lane, bool write)
{
    const int half = lane >> 5;
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * (g + (k >> 1)) + 2 * (k & 1);
                bf16x2 p = {(__bf16)(acc[dt][i] * f), (__bf16)(acc[dt][i + 1] * f)};
                w[k] = __builtin_bit_cast(uint32_t, p);
            }
            auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
            auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
            if (write)
                *reinterpret_cast<uint4*>(row + 32 * dt + 8 * (g + half)) = make_uint4(a[0], b[0], a[1], b[1]);
        }
}

// ------------------------------------------------------------------------
// The packed sequences.  Segment 0 is what lies before cu[0], segment i in
// 1..S is sequence i - 1 and segment S + 1 what lies after cu[S]; segment i
// owns the tiles from floor(start_i / rows) + i on, so a tile finds its
// segment without a scan, and there are at most T / rows + S + 2 tiles.
// Offsets that leave [0, T] are clamped, and where they decrease a tile may
// come out in front of its segment: it has no rows then.  The rows touched
// stay inside the buffers, whatever cu holds.
// ------------------------------------------------------------------------
struct Where {
    int64_t start;   // first token of the segment
    int len;         // its tokens
    int tile;        // this workgroup's tile within it
    bool sequence;   // a sequence, not what lies outside all of them
    int part = 0, parts = 1, slot = 0;   // its share of the tile's work, and the share's number
};
__device__ __forceinline__ int64_t segment_start(const int32_t* cu, int S, int64_t T, int i)
{
    if (i == 0) return 0;
    if (i > S + 1) return T;
    return min(max((int64_t)cu[i - 1], (int64_t)0), T);
}
__device__ __forceinline__ Where find_tile(const int32_t* cu, int S, int64_t T, int shift, int tile, int lane)
{   // tiles of 1 << shift rows
    // every lane tests one segment: how many start at or before this tile
    Where w;
    int n = 0;
    if (S + 2 < 64) {                   // and keeps its start: one read of cu in all
        const int start = (int)segment_start(cu, S, T, lane);
        const int seg = __popcll(__ballot(lane < S + 2 && (start >> shift) + lane <= tile)) - 1;
        const int a = __builtin_amdgcn_readlane(start, seg), b = __builtin_amdgcn_readlane(start, seg + 1);
        w.start = a;
        const int at = tile - ((a >> shift) + seg);
        w.tile = max(at, 0);
        w.len = b > a && at >= 0 ? b - a : 0;
        w.sequence = seg > 0 && seg <= S;
        return w;
    }
    for (int i0 = 0; i0 < S + 2; i0 += 64) {
        const int i = i0 + lane;
        const bool before = i < S + 2 && (int)(segment_start(cu, S, T, i) >> shift) + i <= tile;
        n += __popcll(__ballot(before));
    }
    const int seg = __builtin_amdgcn_readfirstlane(n - 1);
    const int64_t a = segment_start(cu, S, T, seg), b = segment_start(cu, S, T, seg + 1);
    w.start = __builtin_amdgcn_readfirstlane((int)a);
    const int at = __builtin_amdgcn_readfirstlane(tile - ((int)(a >> shift) + seg));
    w.tile = max(at, 0);
    w.len = __builtin_amdgcn_readfirstlane(b > a && at >= 0 ? (int)(b - a) : 0);
    w.sequence = seg > 0 && seg <= S;
    return w;
}

// The sum over the wave of non-negative values, in every lane.
__device__ __forceinline__ int wave_total(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, DPP_XOR1, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, DPP_XOR2, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, DPP_HALF_MIRROR, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, DPP_MIRROR, 0xF, 0xF, false);
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = (int)(a[0] + a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return __builtin_amdgcn_readfirstlane((int)(b[0] + b[1]));
}

__device__ __forceinline__ float wave_total(float v)
{
    auto add = [&](int moved) { v += as_f32((uint32_t)moved); };
    add(__builtin_amdgcn_update_dpp(0, (int)as_u32(v), DPP_XOR1, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, (int)as_u32(v), DPP_XOR2, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, (int)as_u32(v), DPP_HALF_MIRROR, 0xF, 0xF, false));
    add(__builtin_amdgcn_update_dpp(0, (int)as_u32(v), DPP_MIRROR, 0xF, 0xF, false));
    const auto a = __builtin_amdgcn_permlane16_swap(as_u32(v), as_u32(v), false, false);
    v = as_f32(a[0]) + as_f32(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(as_u32(v), as_u32(v), false, false);
    return as_f32(__builtin_amdgcn_readfirstlane((int)as_u32(as_f32(b[0]) + as_f32(b[1]))));
}

// Key tiles that are larger than a compute unit's fair share of the work are
// cut into parts, so that a long sequence among short ones, or one key head,
// does not leave a few workgroups running at the end.
struct Split {
    int extra;        // workgroups a head that the launch has beyond one a tile; 0: no parts
    int least;        // tiles up to this size stay whole
    float fair;       // heads / compute units
};
constexpr int MOST_PARTS = 8;

// The key tiles by the work they stand for, most first: the m-th tile from
// the end of its segment is seen by the m last tiles' queries and has size m,
// and workgroup `rank` takes the rank-th tile (or part) in order of falling
// size, so that the longest workgroups start first and the shortest fill the
// end.  Up to SORTED - 2 sequences; each lane holds a few segments, whose
// bounds are read once.
constexpr int SORTED = 256;
__device__ __forceinline__ Where find_tile_by_size(const int32_t* cu, int S, int64_t T, int shift, const Split& split,
                                                   int rank, int lane)
{
    constexpr int C = SORTED / 64;
    int start[C], len[C], n[C], segments = 0;
    float work = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int i = 64 * j + lane;
        start[j] = len[j] = n[j] = 0;
        if (64 * j < S + 2 && i < S + 2) {
            const int64_t a = segment_start(cu, S, T, i), b = segment_start(cu, S, T, i + 1);
            start[j] = (int)a;
            len[j] = b > a ? (int)(b - a) : 0;
            n[j] = (int)(((uint32_t)len[j] + (1u << shift) - 1) >> shift);
            if (i > 0 && i <= S) work += 0.5f * (float)n[j] * (float)(n[j] + 1);
        }
        segments += __popcll(__ballot(n[j] > 0));
    }
    auto larger = [&](int m) {          // tiles of a size above m
        int v = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) v += max(n[j] - m, 0);
        return wave_total(v);
    };
    int most = 0;
#pragma unroll
    for (int j = 0; j < C; ++j) most = max(most, n[j]);
    most = (int)__builtin_amdgcn_readfirstlane(max_xor32(max_xor16(max_lanes16((uint32_t)most))));
    int whole = most, cut = 0, parts = 1;      // sizes above `whole` are cut, `cut` tiles of them
    if (split.extra > 0) {
        const int fair = max(split.least, (int)ceilf(fminf(wave_total(work) * split.fair, 1e9f)));
        if (most > fair) {
            cut = max(larger(fair), 1);
            parts = min(min(max((most + fair / 2) / fair, 2), MOST_PARTS), 1 + split.extra / cut);
            whole = fair;
        }
    }
    auto above = [&](int m) {           // workgroups for the tiles of a size above m
        const int v = larger(m);
        return v + (parts - 1) * (m < whole ? cut : v);
    };
    Where w{0, 0, 0, false};
    const int all = above(0);
    if (rank >= all) return w;
    int size, r = 0;
    if (segments == 1 && parts == 1) {
        size = all - rank;              // one sequence: its tiles in order
    } else {
        int lo = 1, hi = most;          // the smallest size with at most `rank` workgroups above it
        while (lo < hi) {
            const int m = (lo + hi) / 2;
            if (above(m) <= rank) hi = m;
            else lo = m + 1;
        }
        size = lo;
        r = rank - above(size);
        if (size > whole && rank < 2 * split.extra) {      // (always, with offsets that do not decrease)
            w.parts = parts;
            w.part = r % parts;
            w.slot = rank;
            r /= parts;
        }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {       // the r-th segment that has a tile of this size
        const uint64_t has = __ballot(n[j] >= size);
        const int c = __popcll(has), before = __popcll(has & ((1ull << lane) - 1));
        const uint64_t hit = __ballot(n[j] >= size && before == r);
        if (r >= 0 && r < c) {
            const int at = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
            w.start = __builtin_amdgcn_readlane(start[j], at);
            w.len = __builtin_amdgcn_readlane(len[j], at);
            w.tile = __builtin_amdgcn_readlane(n[j], at) - size;
            w.sequence = 64 * j + at > 0 && 64 * j + at <= S;
        }
        r -= c;
    }
    return w;
}

// Division of a launch's numbers (below 2^31) by one that the host knows: a
// product with floor((2^32 - 1) / d) is at most one too small.  A division
// proper costs a workgroup of a short sequence more than its matrix products.
struct Divisor {
    uint32_t d = 1, m = 0xFFFFFFFFu;
    Divisor() = default;
    explicit Divisor(uint32_t by) : d(by), m(0xFFFFFFFFu / by) {}
};
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& by)
{
    const uint32_t q = __umulhi(n, by.m);
    return n - q * by.d >= by.d ? q + 1 : q;
}

// A grid of `tiles` x `groups` workgroups, the groups of heads innermost.
// Workgroups go round the 8 XCDs, each with its own L2: with a multiple of 8
// groups, one XCD keeps the same heads.
struct Order {
    int tiles = 0, groups = 1;
    Divisor by;          // groups / 8 if that is whole, or else groups
    Order() = default;
    Order(int tiles_, int groups_)
        : tiles(tiles_), groups(groups_), by((uint32_t)(groups_ % 8 == 0 ? groups_ / 8 : groups_)) {}
};
// This workgroup's tile and its group of heads.
struct Mine { Where at; int group; };
struct Place { int rank, group; };
__device__ __forceinline__ Place my_place(const Order& o)
{
    const uint32_t b = blockIdx.x;
    const bool by_xcd = (o.groups & 7) == 0;
    const uint32_t x = by_xcd ? b >> 3 : b;
    const int rank = (int)divide(x, o.by);
    const int in = (int)(x - rank * o.by.d);
    return {rank, by_xcd ? (int)((b & 7) * o.by.d) + in : in};
}
// Query tiles go by their place, the last ones first: by size, neighbours
// come from different sequences and share no keys (61 prompts: 46.0 -> 49.2 us).
__device__ __forceinline__ Mine my_queries(const int32_t* cu, int S, int64_t T, int shift, const Order& o, int lane)
{
    const Place p = my_place(o);
    return {find_tile(cu, S, T, shift, o.tiles - 1 - p.rank, lane), p.group};
}
__device__ __forceinline__ Mine my_keys(const int32_t* cu, int S, int64_t T, int shift, const Order& o,
                                        const Split& split, int lane)
{
    const Place p = my_place(o);
    if (S + 2 <= SORTED) return {find_tile_by_size(cu, S, T, shift, split, p.rank, lane), p.group};
    return {find_tile(cu, S, T, shift, p.rank, lane), p.group};
}

} // namespace attn
} // namespace fgs
