// product_device.h -- tiles of C[m][n] = sum over k of A[m][k] B[n][k] on the
// BF16 matrix instructions, for operands whose contraction runs along their
// rows or across them (internal header of libfgs).
//
// A workgroup of NWM x NWN waves owns a BM x BN tile of C, each wave TI x TJ
// accumulators of 32 x 32.  The contraction advances in steps of BK values (64
// or 32), staged in LDS by copies that pass no register, into a ring of stages.
// An operand whose contraction runs along its rows is staged as BM (or BN) rows
// of 2 BK bytes and read 16 bytes a lane; one whose contraction runs across its
// rows as BK rows of BM (or BN) values, read by the transposing loads, so no
// operand has to be transposed in memory first.
//
// Bound by the matrix units: 8192 x 128000 over 4096 values 6.47 ms (1.33
// PFLOP/s, 73% busy, on a card where the library's product of 8192^3 reaches
// 1.38), both operands read along their rows; 6.38 ms with both across them.
#pragma once

#include <type_traits>

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {
namespace prod {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) s16x4* lds_v4;
typedef const __attribute__((address_space(3))) bf16x8* lds_v8;

enum Side { ALONG, ACROSS };                 // the contraction runs along an operand's rows, or across them

// (BK: contraction values a stage)
template <int NWM_, int NWN_, int TI_, int TJ_, int BK_, int STAGES_>
struct Shape {
    static constexpr int NWM = NWM_, NWN = NWN_, TI = TI_, TJ = TJ_, BK = BK_, STAGES = STAGES_;
    static_assert((STAGES & (STAGES - 1)) == 0, "a stage's place is its number's low bits");
    static constexpr int NW = NWM * NWN, THREADS = 64 * NW;
    static constexpr int WM = 32 * TI, WN = 32 * TJ;                 // a wave's part of the tile
    static constexpr int BM = WM * NWM, BN = WN * NWN;
    static constexpr int A_BYTES = BM * BK * 2, STAGE = (BM + BN) * BK * 2, LDS = STAGES * STAGE;
};

// The lane halves of a 32x32 accumulator tile: register i of lane l holds
// m = l % 32 and n = 8 (i / 4) + 4 (l / 32) + i % 4 (the B fragment goes first).
__device__ __forceinline__ int acc_n(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

__device__ __forceinline__ float swap_half(float x)
{
    auto r = __builtin_amdgcn_permlane32_swap(as_u32(x), as_u32(x), false, false);
    return as_f32((threadIdx.x & 32) ? r[0] : r[1]);
}

__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b)
{
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t lds_offset(const void* p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>((lds_ptr)p));
}

// Global -> LDS copies of 16 bytes a lane: lane i fills bytes 16 i .. of the
// wave's 1 KiB span at lds_addr (uniform).  Issued from assembly so that the
// compiler does not make every later LDS read wait for them; publish() waits.
__device__ __forceinline__ void g2lds16(const char* at, uint32_t lds_addr)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(at), "s"(lds_addr) : "memory", "m0");
}

// All but the last LEFT of this wave's copies have landed and its LDS reads are
// done, and so for every other wave of the workgroup.
template <int LEFT>
__device__ __forceinline__ void publish()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(LEFT) : "memory");
}

// 16-byte chunk c of staged row r sits in slot c ^ f(r): 16 rows of one chunk
// (ALONG), or 4 rows of 4 neighbouring chunks (ACROSS), touch every bank once.
template <Side SIDE, int EXT, int BK>
__device__ __forceinline__ constexpr uint32_t swizzle(uint32_t r)
{
    static_assert(BK == 32 || BK == 64, "rows of 64 or 128 bytes");
    return SIDE == ALONG ? (BK == 64 ? (r >> 1) & 7 : (r >> 2) & 3) : EXT >= 128 ? (r & 3) << 2 : ((r >> 1) & 1) << 2;
}

// One operand's copies: EXT rows (ALONG) or columns (ACROSS) of the tile.
template <Side SIDE, int EXT, int NW, int BK>
struct Loader {
    static constexpr int SLOTS = SIDE == ALONG ? BK / 8 : EXT / 8;   // chunks a staged row
    static constexpr int PER = 64 / SLOTS;                           // staged rows a copy
    static constexpr int N = EXT * BK / 512 / NW;                    // copies a wave and stage
    static_assert(N * NW * 512 == EXT * BK && PER * SLOTS == 64, "whole copies");
    const char* at[N];
    int64_t ld;                                                      // bytes (ACROSS)

    __device__ __forceinline__ static int row(int wave, int lane, int j) { return (wave * N + j) * PER + lane / SLOTS; }
    __device__ __forceinline__ static int chunk(int wave, int lane, int j)
    {
        return (lane % SLOTS) ^ swizzle<SIDE, EXT, BK>(row(wave, lane, j));
    }
    // ALONG: where(r) is row r's first contraction value
    template <class F>
    __device__ __forceinline__ void rows(F where, int wave, int lane)
    {
#pragma unroll
        for (int j = 0; j < N; ++j)
            at[j] = reinterpret_cast<const char*>(where(row(wave, lane, j))) + 16 * chunk(wave, lane, j);
    }
    // ACROSS: the operand's first contraction row, from the tile's first column on; columns past the last of `width`
    // repeat the last eight
    __device__ __forceinline__ void columns(const uint16_t* base, int64_t ld_, int64_t first, int64_t width, int wave, int lane)
    {
        ld = 2 * ld_;
#pragma unroll
        for (int j = 0; j < N; ++j)
            at[j] = reinterpret_cast<const char*>(base) + row(wave, lane, j) * ld +
                    2 * min(first + 8 * chunk(wave, lane, j), width - 8);
    }
    // copy j of the next stage
    __device__ __forceinline__ void issue(int j, uint32_t lds, int wave)
    {
        g2lds16(at[j], lds + (wave * N + j) * 1024);
        at[j] += SIDE == ALONG ? 2 * BK : BK * ld;
    }
    // the next stage is the last and has only `left` rows (ACROSS): later ones repeat the last
    __device__ __forceinline__ void shorten(int left, int wave, int lane)
    {
        if constexpr (SIDE == ACROSS) {
#pragma unroll
            for (int j = 0; j < N; ++j) at[j] -= max(0, row(wave, lane, j) - (left - 1)) * ld;
        }
    }
};

// The operand fragment of values 16 ks .. 16 ks + 15 of the stage and rows
// (columns) first + l % 32 of the tile; address: fragment_address() of the lane.
template <Side SIDE, int EXT, int BK>
__device__ __forceinline__ uint32_t fragment_address(int first, int lane)
{
    if constexpr (SIDE == ALONG) {
        const uint32_t r = first + (lane & 31);
        return r * (2 * BK) + (((uint32_t)(lane >> 5) ^ swizzle<ALONG, EXT, BK>(lane & 31)) << 4);
    } else {
        const int i = lane & 15;
        const uint32_t r = 8 * (lane >> 5) + (i >> 2);
        const uint32_t c = first / 8 + 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        return r * (2 * EXT) + ((c ^ swizzle<ACROSS, EXT, BK>(r)) << 4) + 8 * (i & 1);
    }
}
template <Side SIDE, int EXT>
__device__ __forceinline__ bf16x8 fragment(uint32_t address, uint32_t tile, int ks)
{
    if constexpr (SIDE == ALONG) {
        return *(lds_v8)(uintptr_t)((address ^ (ks << 5)) + tile);
    } else {
        union { s16x4 s[2]; bf16x8 v; } u;       // rows 16 ks + 8 half + 0..3 and + 4..7
        u.s[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(uintptr_t)(address + tile + 16 * ks * (2 * EXT)));
        u.s[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4)(uintptr_t)(address + tile + (16 * ks + 4) * (2 * EXT)));
        return u.v;
    }
}

// acc = the tile's sums over `values` contraction values (ACROSS operands have
// rows for them all; a stage past them repeats rows that the other operand
// meets with zeros).  smem: S::LDS bytes, free again for every wave after the
// call.
template <class S, Side SA, Side SB>
__device__ __forceinline__ void product(f32x16 (&acc)[S::TI][S::TJ], Loader<SA, S::BM, S::NW, S::BK>& la,
                                        Loader<SB, S::BN, S::NW, S::BK>& lb, int64_t values, char* smem)
{
    constexpr int BK = S::BK, KS = BK / 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    const uint32_t lds = lds_offset(smem);
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j) acc[i][j] = f32x16{};
    const int steps = (int)((values + BK - 1) / BK);
    if (steps == 0) return;
    uint32_t aa[S::TI], ab[S::TJ];
#pragma unroll
    for (int i = 0; i < S::TI; ++i) aa[i] = fragment_address<SA, S::BM, BK>(wm * S::WM + 32 * i, lane);
#pragma unroll
    for (int j = 0; j < S::TJ; ++j) ab[j] = fragment_address<SB, S::BN, BK>(wn * S::WN + 32 * j, lane);

    bf16x8 fa[2][S::TI], fb[2][S::TJ];
    constexpr int READS = S::TI + S::TJ, MMAS = S::TI * S::TJ;
    constexpr int A_COPIES = Loader<SA, S::BM, S::NW, BK>::N,
                  COPIES = A_COPIES + Loader<SB, S::BN, S::NW, BK>::N;
    auto place = [&](int step) { return lds + (step & (S::STAGES - 1)) * S::STAGE; };
    auto read = [&](int f, int set, uint32_t stage, int ks) {
        if (f < S::TI) fa[set][f] = fragment<SA, S::BM>(aa[f], stage, ks);
        else fb[set][f - S::TI] = fragment<SB, S::BN>(ab[f - S::TI], stage + S::A_BYTES, ks);
    };
    auto multiply = [&](int t, int set) {
        const int i = t / S::TJ, j = t % S::TJ;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
    };
    const int last = (int)(values - (int64_t)(steps - 1) * BK);       // values of the last stage
    auto copy = [&](int c, int step) {
        if (c == 0 && step == steps - 1 && last < BK) {
            la.shorten(last, wave, lane);
            lb.shorten(last, wave, lane);
        }
        if (c < A_COPIES) la.issue(c, place(step), wave);
        else lb.issue(c - A_COPIES, place(step) + S::A_BYTES, wave);
    };
#pragma unroll
    for (int step = 0; step < S::STAGES; ++step)
        if (step < steps)
#pragma unroll
            for (int c = 0; c < COPIES; ++c) copy(c, step);
    if (steps >= S::STAGES) publish<(S::STAGES - 1) * COPIES>();
    else publish<0>();
#pragma unroll
    for (int f = 0; f < READS; ++f) read(f, 0, lds, 0);
    // The order below is kept as it is written: a fragment is read a whole
    // k-step before its products, and a copy starts beside a product, so that
    // neither is waited for (left to the compiler, reads stand right before
    // their products).  The stage's last products run after the barrier that
    // publishes the next stage, beside that stage's first reads and, every wave
    // being past its reads of this one, the copies that take its place.
    // fill: there are such copies; more: there is a next stage.
    auto advance = [&](int step, auto fill, auto more) {
#pragma unroll
        for (int ks = 0; ks < KS - 1; ++ks)
#pragma unroll
            for (int t = 0; t < MMAS; ++t) {
                multiply(t, ks & 1);
#pragma unroll
                for (int f = t * READS / MMAS; f < (t + 1) * READS / MMAS; ++f) read(f, (ks + 1) & 1, place(step), ks + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
        publish<fill ? (S::STAGES - 2) * COPIES : 0>();
#pragma unroll
        for (int t = 0; t < MMAS; ++t) {
            multiply(t, 1);
            if constexpr (more) {
#pragma unroll
                for (int f = t * READS / MMAS; f < (t + 1) * READS / MMAS; ++f) read(f, 0, place(step + 1), 0);
            }
            if constexpr (fill) {
#pragma unroll
                for (int c = t * COPIES / MMAS; c < (t + 1) * COPIES / MMAS; ++c) copy(c, step + S::STAGES);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int step = 0;
    for (; step < steps - S::STAGES; ++step) advance(step, std::true_type{}, std::true_type{});
    for (; step < steps - 1; ++step) advance(step, std::false_type{}, std::true_type{});
    advance(step, std::false_type{}, std::false_type{});
}

// Tile `id` of tm x tn of them: workgroups are dealt round-robin to the 8
// XCDs; each XCD gets a contiguous range of an order that runs down 4 m-tiles,
// then to the next n-tile, so that the tiles in flight share panels in its L2.
__device__ __forceinline__ void tile_of(int64_t id, int tm, int tn, int& m, int& n)
{
    const int64_t total = (int64_t)tm * tn, each = total >> 3, more = total & 7, x = id & 7;
    const uint32_t at = (uint32_t)(x * each + min(x, more) + (id >> 3));
    const uint32_t group = at / (4u * tn), first = group * 4, size = min((uint32_t)tm - first, 4u);
    const uint32_t in = at - group * 4u * tn;
    n = (int)(in / size);
    m = (int)(first + in - n * size);
}

} // namespace prod
} // namespace fgs
