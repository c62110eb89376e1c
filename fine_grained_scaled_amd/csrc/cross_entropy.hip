// cross_entropy.hip -- the output head with softmax cross entropy, on gfx950,
// forward and backward, without keeping the logits.
//
//   z = x w^T,  lse = log sum_v exp z[v],  loss = lse - z[target],
//   dz = dloss (softmax(z) - onehot(target)) + dlse softmax(z),
//   dx = dz w,  dw = dz^T x.
//
// Forward: a tile of z stays in the accumulators; each row leaves its maximum
// and its sum of exponents over the tile's vocabulary, and a second kernel
// joins them over the tiles in a fixed order.  Backward: the vocabulary goes in
// pieces; for each, z is formed again (2 T V K operations more than the
// gradients' 4 T V K, against T x V values kept and read), dz is written in
// BF16, and two products over it add to dx (FP32 sums in the workspace) and
// write the piece's rows of dw.  No atomics: the same inputs give the same bits.
//
// Tokens without a target take no part.  The rows that have one are listed on
// the device first, and everything after works on that list, so a batch of
// mostly masked tokens costs what its targets cost, and NaN in the rows of the
// others reach nothing.
//
// The pieces' width and the number of workgroups that share a tile of dx follow
// from that list too, on the device: few rows take wide pieces.
//
// dz goes to the matrix units in BF16, divided by the largest |dloss| (|dlse|)
// of the call, which the results are multiplied with again in FP32: under a
// mean over the tokens the values are then softmax - onehot itself, whose
// largest, those of the targets, round best (-1 exactly).
//
// Measured, the fastest card to the slowest: 8192 tokens, 128000 x 4096, forward
// and backward 26.2 to 27.6 ms, 8 T V K operations at 1.31 to 1.25 PFLOP/s; 4099
// tokens, 50021 x 2048 forward 728 to 799 us; 5 tokens, 32003 x 512 forward 12.7 us,
// of which the kernel that reads w takes 9.0.
#include <algorithm>
#include <cmath>

#include "product_device.h"

namespace fgs {

namespace {

using namespace prod;

// 256 x 256, 8 waves of 128 x 64 (4 waves of 128 x 128, 8192 tokens: 29.4 ms for
// 28.4).  An operand that is read along its rows comes in whole lines of 128
// bytes with stages of 64 values, two of them; with four of 32 the copies start
// a stage earlier, which pays where no operand is (dw: 841 us a piece for 869,
// the scores 7180 for 6910).
using Big = Shape<2, 4, 4, 2, 64, 2>;
using Deep = Shape<2, 4, 4, 2, 32, 4>;
// 128 x 256: a last tile of up to 128 rows (300 tokens, 32003 x 1024: 33.9 us for 36.4)
using Half = Shape<2, 4, 2, 2, 64, 2>;
// 128 x 128, up to 128 tokens: bound by the loads of w
using Small = Shape<2, 4, 2, 1, 64, 4>;

constexpr float LOG2E = 1.44269504088896340736f;

// What the rows with a target need, in their order (padded with zeros to a
// multiple of 256 rows).
struct Rows {
    int32_t* count;        // [3]: the rows; backward: a piece's width, workgroups that share a tile of dx
    float* most;           // [1]: the largest |dloss|, |dlse| (1 where that is 0 or not finite)
    int32_t* place;        // [T]: a token's row, -1 without a target
    int32_t* token;        // [Tp]
    int32_t* target;       // [Tp]
    float *lse, *dloss, *dlse;    // [Tp] (backward)
};

__device__ __forceinline__ int target_of(const void* targets, int wide, int64_t t, int64_t V)
{
    const int64_t v = wide ? static_cast<const int64_t*>(targets)[t] : static_cast<const int32_t*>(targets)[t];
    return v >= 0 && v < V ? (int)v : -1;
}

// How the backward pass is cut, from the number of rows.
struct Cut {
    int64_t V, room;       // values of dz that the workspace holds
    int bm, tiles_n;       // rows a tile of dx, tiles along its width
    int slots, most;       // tiles' sums that the workspace holds, workgroups a tile at most
    int cus;
};

__host__ __device__ inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

__host__ __device__ inline int64_t piece_width(const Cut& c, int64_t rows)
{
    const int64_t fits = c.room / up(rows > 0 ? rows : 1, 256) / 256 * 256;
    return fits < up(c.V, 256) ? fits : up(c.V, 256);
}

// Workgroups that share a tile of dx, each a part of the piece: the fewest
// microseconds.  A step of 64 values is taken to cost a compute unit 1.9 us per
// 256 x 256 and a part's first loads 3 us; its sums are read and written again,
// 0.117 us of the chip's time (512 KiB at 4.5 TB/s).  The present main loop takes
// 1.53 us a step and 1.5 us besides its sums (4096 tokens, 2048 to 16384 words x
// 4096: 65 to 409 us): with these the choice differs at 100 of 2808 sizes from 1
// to 32768 tokens, by at most 2% of the time.  A 128 x 128 tile counts as a quarter.
// (By the 64 lanes of a wave.)
__device__ inline int dx_splits(const Cut& c, int64_t rows, int64_t width)
{
    const int n = (int)((rows + c.bm - 1) / c.bm) * c.tiles_n;
    const float size = c.bm / 256.0f * (c.bm / 256.0f);
    uint64_t best = ~0ull;             // the time's bits (no float here is negative) and the number
    for (int s = 1 + (threadIdx.x & 63); s <= c.most && (s == 1 || n * s <= c.slots); s += 64) {
        const float t = (float)((n * s + c.cus - 1) / c.cus) * (width / (float)s * 0.0292f * size + 3.0f) + n * s * 0.117f * size;
        best = min(best, (uint64_t)as_u32(t) << 32 | (uint32_t)s);
    }
    for (int m = 1; m < 64; m *= 2) best = min(best, (uint64_t)__shfl_xor((unsigned long long)best, m));
    return (int)best;
}

// One workgroup lists the rows with a target.
__global__ __launch_bounds__(1024) void ce_rows_kernel(const void* targets, int wide, int64_t T, int64_t V, Rows r,
                                                       const float* dloss, const float* dlse, const float* lse, Cut cut)
{
    const bool backward = cut.V > 0;       // (dloss of no tokens may be a null pointer)
    __shared__ int s_count[16];
    __shared__ float s_top[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before = 0;
    float top = 0.0f;
    bool bad = false;
    for (int64_t t0 = 0; t0 < T; t0 += 1024) {
        const int64_t t = t0 + threadIdx.x;
        const int target = t < T ? target_of(targets, wide, t, V) : -1;
        const uint64_t some = __ballot(target >= 0);
        if (lane == 0) s_count[wave] = __popcll(some);
        __syncthreads();
        int at = before, all = 0;
        for (int i = 0; i < 16; ++i) {
            const int c = s_count[i];
            if (i < wave) at += c;
            all += c;
        }
        __syncthreads();
        before += all;
        at += __popcll(some & ((1ull << lane) - 1));
        if (t < T) r.place[t] = target >= 0 ? at : -1;
        if (target >= 0) {
            r.token[at] = (int)t;
            r.target[at] = target;
            if (backward) {
                const float b = dloss[t], e = dlse ? dlse[t] : 0.0f;
                r.dloss[at] = b;
                r.dlse[at] = e;
                r.lse[at] = lse[t];
                top = fmaxf(top, fmaxf(fabsf(b), fabsf(e)));
                bad |= b - b != 0.0f || e - e != 0.0f;
            }
        }
    }
    const int padded = (before + 255) & ~255;
    for (int i = before + threadIdx.x; i < padded; i += 1024) {
        r.token[i] = 0;
        r.target[i] = -1;
        if (backward) r.dloss[i] = r.dlse[i] = r.lse[i] = 0.0f;
    }
    if (backward) {
        if (bad) top = INFINITY;
        for (int m = 1; m < 64; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
        if (lane == 0) s_top[wave] = top;
        __syncthreads();
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s_top[i]);
    }
    if (wave != 0) return;
    const int64_t width = backward ? piece_width(cut, before) : 0;
    const int splits = backward ? dx_splits(cut, before, width) : 0;
    if (lane == 0) {
        r.count[0] = before;
        r.count[1] = (int)width;
        r.count[2] = splits;
        if (backward) *r.most = top > 0.0f && top < INFINITY ? top : 1.0f;
    }
}

// Token t's row of x to its place among the rows with a target; without one,
// zeros to its row of dx.  The rows from the count to a multiple of 256 get zeros.
__global__ __launch_bounds__(256) void ce_gather_kernel(const uint16_t* x, int64_t ldx, int64_t T, int K, Rows r,
                                                        uint16_t* xc, uint16_t* dx)
{
    int64_t t = blockIdx.x;
    const uint4* from = nullptr;
    uint4* to;
    if (t < T) {
        const int at = r.place[t];
        if (at >= 0) from = reinterpret_cast<const uint4*>(x + t * ldx);
        to = reinterpret_cast<uint4*>(at >= 0 ? xc + (int64_t)at * K : dx + t * K);
    } else {
        const int64_t n = *r.count, at = n + t - T;
        if (at >= ((n + 255) & ~(int64_t)255)) return;
        to = reinterpret_cast<uint4*>(xc + at * K);
    }
    for (int i = threadIdx.x; i < K / 8; i += 256) to[i] = from ? from[i] : make_uint4(0, 0, 0, 0);
}

// ------------------------------------------------------------------------
// Forward: tiles of z, of which each row leaves (maximum, sum of exponents)
// and the target's value.
// ------------------------------------------------------------------------
struct ScoreArgs {
    const uint16_t *x, *w;
    int64_t ldx, ldw, T, V;
    int K, tiles_n;                    // tiles along the vocabulary (forward)
    int piece;                         // of the vocabulary (backward)
    const void* targets;               // the forward pass without a list of rows
    int wide;
    Rows r;                            // r.count nullptr: every token is a row
    int64_t Tp;
    float2* part;                      // [tiles_n][Tp]
    float* z_target;                   // [Tp]
    uint16_t* dz;                      // [rows][a piece's width] (backward)
};

// The workgroup's tile of z: body(S{}, its place), or body(Half{}, ..) where a
// last tile of Big has at most 128 rows.
template <class S, class F>
__device__ __forceinline__ void score_place(int64_t rows, int64_t v0, int tiles_n, F body)
{
    const int tiles_m = (int)((rows + S::BM - 1) / S::BM);
    if ((int64_t)blockIdx.x >= (int64_t)tiles_m * tiles_n) return;
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * S::BM, n0 = v0 + (int64_t)tn * S::BN;
    if constexpr (std::is_same_v<S, Big>) {
        if (rows - m0 <= Half::BM) return body(Half{}, m0, n0, tn);
    }
    body(S{}, m0, n0, tn);
}

template <class S>
__device__ __forceinline__ void score_product(const ScoreArgs& p, f32x16 (&acc)[S::TI][S::TJ], int64_t rows, int64_t m0,
                                              int64_t n0, char* smem)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Loader<ALONG, S::BM, S::NW, S::BK> la;
    Loader<ALONG, S::BN, S::NW, S::BK> lb;
    la.rows([&](int r) {
        int64_t row = min(m0 + r, rows - 1);
        if (p.r.token) row = p.r.token[row];
        return p.x + row * p.ldx;
    }, wave, lane);
    lb.rows([&](int r) { return p.w + min(n0 + r, p.V - 1) * p.ldw; }, wave, lane);
    product<S, ALONG, ALONG>(acc, la, lb, p.K, smem);
}

template <class S>
__device__ __forceinline__ void score_tile(const ScoreArgs& p, int64_t rows, int64_t m0, int64_t n0, int tn, char* smem)
{
    f32x16 acc[S::TI][S::TJ];
    score_product<S>(p, acc, rows, m0, n0, smem);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    const int64_t nw = n0 + wn * S::WN;
    if (nw + S::WN > p.V) {
#pragma unroll
        for (int i = 0; i < S::TI; ++i)
#pragma unroll
            for (int j = 0; j < S::TJ; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (nw + 32 * j + acc_n(k, half) >= p.V) acc[i][j][k] = -INFINITY;
    }
    float2* red = reinterpret_cast<float2*>(smem);      // [NWN][BM]
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
        const int row = wm * S::WM + 32 * i + (lane & 31);
        float top = acc[i][0][0];
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, acc[i][j][k]);
        top = fmaxf(top, swap_half(top));
        // the distance first, then log2 e: z log2 e by itself is off by up to 2^-24 of its size, from 2^31 on more than
        // an exponent holds (one multiply-add a score instead: 4099 tokens, 50021 x 2048 760 us for 764)
        const float base = top == -INFINITY ? 0.0f : top;
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) sum += __builtin_amdgcn_exp2f((acc[i][j][k] - base) * LOG2E);
        sum += swap_half(sum);
        if (half == 0) red[wn * S::BM + row] = make_float2(top, sum);
        // the target's value, from the lane that holds it
        int target = -1;
        if (m0 + row < rows) target = p.r.count ? p.r.target[m0 + row] : target_of(p.targets, p.wide, m0 + row, p.V);
        const int64_t in = target - nw;
        if (__any(target >= 0 && in >= 0 && in < S::WN)) {
#pragma unroll
            for (int j = 0; j < S::TJ; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (target >= 0 && in == 32 * j + acc_n(k, half)) p.z_target[m0 + row] = acc[i][j][k];
        }
    }
    __syncthreads();
    for (int row = threadIdx.x; row < S::BM; row += S::THREADS) {
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < S::NWN; ++i) top = fmaxf(top, red[i * S::BM + row].x);
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < S::NWN; ++i) {
            const float2 v = red[i * S::BM + row];
            sum += v.y * __builtin_amdgcn_exp2f((v.x - base) * LOG2E);
        }
        if (m0 + row < rows) p.part[(int64_t)tn * p.Tp + m0 + row] = make_float2(top, sum);
    }
}

template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_score_kernel(ScoreArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const int64_t rows = p.r.count ? *p.r.count : p.T;
    score_place<S>(rows, 0, p.tiles_n, [&](auto shape, int64_t m0, int64_t n0, int tn) {
        score_tile<decltype(shape)>(p, rows, m0, n0, tn, smem);
    });
}

// Every token's loss and lse from its row's parts: 16 rows a workgroup, 64
// threads a row.
__global__ __launch_bounds__(1024) void ce_join_kernel(ScoreArgs p, float* loss, float* lse)
{
    __shared__ float2 red[64][16];
    const int r = threadIdx.x & 15, split = threadIdx.x >> 4;
    const int64_t t = (int64_t)blockIdx.x * 16 + r;
    int64_t row = -1;
    if (t < p.T) row = p.r.count ? p.r.place[t] : target_of(p.targets, p.wide, t, p.V) >= 0 ? t : -1;
    float top = -INFINITY, sum = 0.0f;
    if (row >= 0) {
        for (int i = split; i < p.tiles_n; i += 64) {
            const float2 v = p.part[(int64_t)i * p.Tp + row];
            const float now = fmaxf(top, v.x), base = now == -INFINITY ? 0.0f : now;
            sum = sum * __builtin_amdgcn_exp2f((top - base) * LOG2E) + v.y * __builtin_amdgcn_exp2f((v.x - base) * LOG2E);
            top = now;
        }
    }
    red[split][r] = make_float2(top, sum);
    __syncthreads();
    for (int n = 32; n > 0; n >>= 1) {
        if (split < n) {
            const float2 o = red[split + n][r];
            const float now = fmaxf(top, o.x), base = now == -INFINITY ? 0.0f : now;
            sum = sum * __builtin_amdgcn_exp2f((top - base) * LOG2E) + o.y * __builtin_amdgcn_exp2f((o.x - base) * LOG2E);
            top = now;
            red[split][r] = make_float2(top, sum);
        }
        __syncthreads();
    }
    if (split == 0 && t < p.T) {
        const float ln = logf(sum);
        lse[t] = row >= 0 ? top + ln : 0.0f;
        loss[t] = row >= 0 ? (top - p.z_target[row]) + ln : 0.0f;      // 0 + ln where the target is the largest
    }
}

// ------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------

// A piece of the vocabulary: words v0 .. v0 + width - 1, padded to a multiple of
// 256 columns of dz, whose rows are ld apart; none where v0 is past the last.
struct Piece {
    int64_t v0, width, padded, ld;
};
__device__ __forceinline__ Piece piece_of(const Rows& r, int piece, int64_t V)
{
    Piece p;
    p.ld = r.count[1];
    p.v0 = piece * p.ld;
    p.width = min(p.ld, max(V - p.v0, (int64_t)0));
    p.padded = up(p.width, 256);
    return p;
}

// A tile's values as BF16 through LDS, so that whole rows are written: f(i, j,
// k) is the lane's value, write(row, chunk) where 16 bytes of the tile go, or
// nullptr.  16-byte chunk c of row r sits in slot c ^ (r % 32).
template <class S, class F, class W>
__device__ __forceinline__ void store_tile(char* smem, F f, W write)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    constexpr int CHUNKS = S::BN / 8, MASK = std::min(CHUNKS, 32) - 1;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
        const int row = wm * S::WM + 32 * i + (lane & 31);
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = (wn * S::WN + 32 * j) / 8 + g;
                uint2 v;
                v.x = bf16x2_rne(f(i, j, 4 * g), f(i, j, 4 * g + 1));
                v.y = bf16x2_rne(f(i, j, 4 * g + 2), f(i, j, 4 * g + 3));
                *reinterpret_cast<uint2*>(smem + row * (2 * S::BN) + ((c ^ (row & MASK)) << 4) + 8 * half) = v;
            }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < S::BM * CHUNKS; e += S::THREADS) {
        const int row = e / CHUNKS, c = e % CHUNKS;
        const uint4 v = *reinterpret_cast<const uint4*>(smem + row * (2 * S::BN) + ((c ^ (row & MASK)) << 4));
        if (uint16_t* to = write(row, c)) *reinterpret_cast<uint4*>(to) = v;
    }
}

// A tile of dz: z again, then the softmax from the row's lse.
template <class S>
__device__ __forceinline__ void gradient_tile(const ScoreArgs& p, int64_t rows, int64_t v0, int64_t m0, int64_t n0, char* smem)
{
    f32x16 acc[S::TI][S::TJ];
    score_product<S>(p, acc, rows, m0, n0, smem);
    const int64_t ld = p.r.count[1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    const int64_t nw = n0 + wn * S::WN;
    const float most = *p.r.most;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
        const int64_t row = m0 + wm * S::WM + 32 * i + (lane & 31);      // within the padded rows
        const float lse = p.r.lse[row], b = p.r.dloss[row] / most, a = b + p.r.dlse[row] / most;
        const int64_t in = p.r.target[row] - nw;
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[i][j][k] = a * __builtin_amdgcn_exp2f((acc[i][j][k] - lse) * LOG2E);
        if (__any(in >= 0 && in < S::WN)) {
#pragma unroll
            for (int j = 0; j < S::TJ; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (in == 32 * j + acc_n(k, half)) acc[i][j][k] -= b;
        }
        // rows and words that only fill the tile up
        if (m0 + S::BM > rows || nw + S::WN > p.V) {
#pragma unroll
            for (int j = 0; j < S::TJ; ++j)
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (row >= rows || nw + 32 * j + acc_n(k, half) >= p.V) acc[i][j][k] = 0.0f;
        }
    }
    store_tile<S>(smem, [&](int i, int j, int k) { return acc[i][j][k]; },
                  [&](int row, int c) { return p.dz + (m0 + row) * ld + (n0 - v0) + 8 * c; });
}

template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_gradient_kernel(ScoreArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const Piece at = piece_of(p.r, p.piece, p.V);
    const int64_t rows = p.r.count[0];
    score_place<S>(rows, at.v0, (int)(at.padded / S::BN), [&](auto shape, int64_t m0, int64_t n0, int) {
        gradient_tile<decltype(shape)>(p, rows, at.v0, m0, n0, smem);
    });
}

struct GradArgs {
    const uint16_t *dz, *w, *xc;
    int64_t ldw, V;
    int K, piece, tiles_n;             // tiles along dx's width
    Rows r;
    float* sums;                       // [slots][bm x 256 (128)]
    uint16_t *dx, *dw;
};

// dx += dz w over the piece's vocabulary, or a part of it; the sums stay in
// the accumulators' order.
template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_dx_kernel(GradArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const Piece at = piece_of(p.r, p.piece, p.V);
    const int64_t rows = p.r.count[0];
    const int splits = p.r.count[2], tiles_m = (int)((rows + S::BM - 1) / S::BM);
    const int64_t each = (int64_t)tiles_m * p.tiles_n;
    if (at.width == 0 || (int64_t)blockIdx.x >= each * splits) return;
    const int split = (int)(blockIdx.x / each);
    int tm, tn;
    tile_of(blockIdx.x - split * each, tiles_m, p.tiles_n, tm, tn);
    const int64_t per = up((at.padded + splits - 1) / splits, S::BK);
    const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN, k0 = split * per;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t values = max((int64_t)0, min(per, at.width - k0));
    Loader<ALONG, S::BM, S::NW, S::BK> la;
    Loader<ACROSS, S::BN, S::NW, S::BK> lb;
    la.rows([&](int r) { return p.dz + (m0 + r) * at.ld + k0; }, wave, lane);
    lb.columns(p.w + min(at.v0 + k0, p.V - 1) * p.ldw, p.ldw, n0, p.K, wave, lane);
    f32x16 acc[S::TI][S::TJ];
    product<S, ALONG, ACROSS>(acc, la, lb, values, smem);
    float4* sums = reinterpret_cast<float4*>(p.sums) + ((int64_t)(tm * p.tiles_n + tn) * splits + split) * (S::BM * S::BN / 4) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float4* to = sums + ((i * S::TJ + j) * 4 + g) * S::THREADS;
                float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
                if (p.piece > 0) {
                    const float4 o = *to;
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                *to = v;
            }
}

// The parts' sums to the tokens' rows of dx.  A thread takes two of a lane's
// groups of 4 columns, which the lane halves swap so that each writes 16 bytes.
template <class S>
__global__ __launch_bounds__(256) void ce_dx_store_kernel(GradArgs p)
{
    constexpr int PAIRS = S::TI * S::TJ * 2, PER = S::BM * S::BN / 4;      // pairs of groups a lane, float4 a tile
    const int64_t rows = p.r.count[0];
    const int splits = p.r.count[2];
    const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t tile = e / (PAIRS * S::THREADS);
    const int64_t m0 = tile / p.tiles_n * S::BM, n0 = tile % p.tiles_n * S::BN;
    if (m0 >= rows) return;
    const int in = (int)(e % (PAIRS * S::THREADS)), pair = in / S::THREADS, thread = in % S::THREADS;
    const int lane = thread & 63, wave = thread >> 6, half = lane >> 5;
    const float4* sums = reinterpret_cast<const float4*>(p.sums) + tile * splits * PER + 2 * pair * S::THREADS + thread;
    float4 a = {}, b = {};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) {
        const float4 u = sums[(int64_t)s * PER], v = sums[(int64_t)s * PER + S::THREADS];
        a.x += u.x, a.y += u.y, a.z += u.z, a.w += u.w;
        b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
    }
    const float scale = *p.r.most;
    const auto lo = __builtin_amdgcn_permlane32_swap(bf16x2_rne(a.x * scale, a.y * scale), bf16x2_rne(b.x * scale, b.y * scale), false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(bf16x2_rne(a.z * scale, a.w * scale), bf16x2_rne(b.z * scale, b.w * scale), false, false);
    const int i = pair / 2 / S::TJ, j = pair / 2 % S::TJ, g = 2 * (pair & 1);
    const int64_t row = m0 + wave / S::NWN * S::WM + 32 * i + (lane & 31);
    const int64_t col = n0 + wave % S::NWN * S::WN + 32 * j + 8 * (g + half);
    if (row < rows && col < p.K)
        *reinterpret_cast<uint4*>(p.dx + (int64_t)p.r.token[row] * p.K + col) = make_uint4(lo[0], hi[0], lo[1], hi[1]);
}

// The piece's rows of dw = dz^T x.
template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_dw_kernel(GradArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const Piece at = piece_of(p.r, p.piece, p.V);
    const int64_t rows = p.r.count[0];
    const int tiles_m = (int)(at.padded / S::BM), tiles_n = (p.K + S::BN - 1) / S::BN;
    if ((int64_t)blockIdx.x >= (int64_t)tiles_m * tiles_n) return;
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Loader<ACROSS, S::BM, S::NW, S::BK> la;
    Loader<ACROSS, S::BN, S::NW, S::BK> lb;
    la.columns(p.dz, at.ld, m0, at.ld, wave, lane);
    lb.columns(p.xc, p.K, n0, p.K, wave, lane);
    f32x16 acc[S::TI][S::TJ];
    product<S, ACROSS, ACROSS>(acc, la, lb, up(rows, 64), smem);
    const float scale = *p.r.most;
    store_tile<S>(smem, [&](int i, int j, int k) { return acc[i][j][k] * scale; },
                  [&](int row, int c) -> uint16_t* {
                      if (m0 + row >= at.width || n0 + 8 * c >= p.K) return nullptr;
                      return p.dw + (at.v0 + m0 + row) * p.K + n0 + 8 * c;
                  });
}

// Up to 128 tokens the pass is bound by reading w, and a 256 x 256 tile's rows
// would be padding for the most part: 128 x 128 with three stages on their way
// takes 64 us for 100 tokens, 32000 x 4096 forward (107 with 256 x 256), 207 for
// 128 tokens, 128000 x 4096 (252).  (64 x 128 in 4 waves: 2% less at 5 tokens,
// 14 to 30% more from 65 on.)  Above, 256 x 256 pays from 257 tokens on and not
// yet at 129 to 256, where two rows of 128 x 128 tiles would take less: 32000 x
// 4096 forward 101 us for 84 at 129 tokens and 108 for 91 at 256, then 105 for 120
// at 257 and 179 for 200 at 600; forward and backward 406 for 349, 428 for 388,
// and 479 for 499 at 300; 32003 x 1024 forward 28 for 25 at 129, 34 for 38 at 257.
constexpr int64_t SMALL = Small::BM;
// dz of one piece of the vocabulary: 256 MiB, or 8192 words where that is more.
constexpr int64_t PIECE_VALUES = (int64_t)1 << 27, PIECE_LEAST = 8192;
// Parts of dx: sums of 1280 tiles at most, where their number is not more
// already, and one for each 1024 words of the vocabulary at most (of one piece that
// is 1024 values of the contraction each at least; where there are several, the
// times above choose no shorter ones at any of those 2808 sizes).
constexpr int64_t SLOTS = 1280, PART_LEAST = 1024;

// The workspace's parts, each at a multiple of 256 bytes.
struct Layout {
    size_t bytes = 0;
    char* base;
    explicit Layout(void* at) : base(static_cast<char*>(at)) {}
    template <class T> T* take(int64_t n)
    {
        T* p = reinterpret_cast<T*>(base + bytes);
        bytes += (size_t)up(n * (int64_t)sizeof(T), 256);
        return p;
    }
};

struct Plan {
    Rows r{};
    int64_t Tp;
    bool small, list;
    int tiles_n = 0;                   // forward
    Cut cut{};                         // backward
    int pieces = 0;
    float2* part = nullptr;
    float *z_target = nullptr, *sums = nullptr;
    uint16_t *xc = nullptr, *dz = nullptr;
    size_t bytes;
};

Plan make_plan(int64_t T, int64_t V, int64_t K, bool backward, void* workspace)
{
    Plan p;
    Layout at(workspace);
    p.small = T <= SMALL;
    const int bm = p.small ? Small::BM : Big::BM, bn = p.small ? Small::BN : Big::BN;
    p.Tp = up(std::max<int64_t>(T, 1), 256);
    // the forward pass of one tile's tokens gains nothing from a list of rows
    p.list = backward || T > Big::BM;
    if (p.list) {
        p.r.count = at.take<int32_t>(3);
        p.r.most = at.take<float>(1);
        p.r.place = at.take<int32_t>(p.Tp);
        p.r.token = at.take<int32_t>(p.Tp);
        p.r.target = at.take<int32_t>(p.Tp);
    }
    if (!backward) {
        p.tiles_n = (int)(up(V, bn) / bn);
        p.part = at.take<float2>(p.tiles_n * p.Tp);
        p.z_target = at.take<float>(p.Tp);
    } else {
        p.r.lse = at.take<float>(p.Tp), p.r.dloss = at.take<float>(p.Tp), p.r.dlse = at.take<float>(p.Tp);
        p.xc = at.take<uint16_t>(p.Tp * K);
        Cut& c = p.cut;
        c.V = V;
        // (all of the vocabulary for any number of rows, where that is less)
        c.room = std::min(p.Tp * up(V, 256), std::max(PIECE_VALUES, p.Tp * PIECE_LEAST));
        p.pieces = (int)((V + piece_width(c, p.Tp) - 1) / piece_width(c, p.Tp));
        p.dz = at.take<uint16_t>(c.room);
        c.bm = bm, c.tiles_n = (int)(up(K, bn) / bn);
        const int64_t tiles = up(std::max<int64_t>(T, 1), bm) / bm * c.tiles_n;
        c.most = (int)std::max<int64_t>(1, up(V, 256) / PART_LEAST);
        c.slots = (int)std::max(tiles, std::min(SLOTS, tiles * c.most));
        p.sums = at.take<float>((int64_t)c.slots * bm * bn);
    }
    p.bytes = at.bytes;
    return p;
}

template <class S, class A>
hipError_t go(void (*kernel)(A), int64_t grid, const A& a, hipStream_t stream)
{
    constexpr int LDS = std::max(S::LDS, 2 * S::BM * S::BN);       // the stages, then the tile on its way out
    if (LDS > 64 * 1024)
        if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, LDS); e != hipSuccess)
            return e;
    kernel<<<(uint32_t)grid, S::THREADS, LDS, stream>>>(a);
    return hipGetLastError();
}

ScoreArgs score_args(const CrossEntropyArgs& c, const Plan& p)
{
    ScoreArgs s{};
    s.x = static_cast<const uint16_t*>(c.x), s.w = static_cast<const uint16_t*>(c.w);
    s.ldx = c.ldx, s.ldw = c.ldw, s.T = c.T, s.V = c.V, s.K = (int)c.K;
    s.targets = c.targets, s.wide = c.wide, s.r = p.r, s.Tp = p.Tp;
    s.part = p.part, s.z_target = p.z_target, s.tiles_n = p.tiles_n;
    return s;
}

} // namespace

size_t cross_entropy_workspace_bytes(int64_t T, int64_t V, int64_t K, int backward)
{
    return make_plan(T, V, K, backward != 0, nullptr).bytes;
}

hipError_t launch_cross_entropy_fwd(const CrossEntropyArgs& c, hipStream_t stream)
{
    const Plan p = make_plan(c.T, c.V, c.K, false, c.workspace);
    const ScoreArgs s = score_args(c, p);
    if (p.list) ce_rows_kernel<<<1, 1024, 0, stream>>>(c.targets, c.wide, c.T, c.V, p.r, nullptr, nullptr, nullptr, p.cut);
    hipError_t e = p.small ? go<Small>(ce_score_kernel<Small>, p.tiles_n, s, stream)
                           : go<Big>(ce_score_kernel<Big>, p.Tp / Big::BM * p.tiles_n, s, stream);
    if (e != hipSuccess) return e;
    ce_join_kernel<<<(uint32_t)((c.T + 15) / 16), 1024, 0, stream>>>(s, c.loss, c.lse);
    return hipGetLastError();
}

template <class S>
static hipError_t backward(const CrossEntropyArgs& c, Plan& p, hipStream_t stream)
{
    int device;
    if (hipError_t e = hipGetDevice(&device); e != hipSuccess) return e;
    if (hipError_t e = hipDeviceGetAttribute(&p.cut.cus, hipDeviceAttributeMultiprocessorCount, device); e != hipSuccess) return e;
    ScoreArgs s = score_args(c, p);
    ce_rows_kernel<<<1, 1024, 0, stream>>>(c.targets, c.wide, c.T, c.V, p.r, c.dloss, c.dlse, c.lse, p.cut);
    ce_gather_kernel<<<(uint32_t)(c.T + 256), 256, 0, stream>>>(s.x, c.ldx, c.T, (int)c.K, p.r, p.xc, static_cast<uint16_t*>(c.dx));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    s.x = p.xc, s.ldx = c.K, s.r.token = nullptr;
    s.dz = p.dz;
    GradArgs g{};
    g.dz = p.dz, g.w = s.w, g.xc = p.xc, g.ldw = c.ldw, g.V = c.V, g.K = (int)c.K;
    g.tiles_n = p.cut.tiles_n, g.r = p.r, g.sums = p.sums;
    g.dx = static_cast<uint16_t*>(c.dx), g.dw = static_cast<uint16_t*>(c.dw);
    // grids for any number of rows; workgroups without a tile end at once
    const int64_t words = up(c.V, 256), tiles_m = up(std::max<int64_t>(c.T, 1), S::BM) / S::BM;
    const int64_t scores = std::min(tiles_m * (words / S::BN), (p.cut.room + (int64_t)S::BM * S::BN - 1) / (S::BM * S::BN));
    for (int i = 0; i < p.pieces; ++i) {
        s.piece = g.piece = i;
        if (hipError_t e = go<S>(ce_gradient_kernel<S>, scores, s, stream); e != hipSuccess) return e;
        if (hipError_t e = go<S>(ce_dx_kernel<S>, p.cut.slots, g, stream); e != hipSuccess) return e;
        // (the first piece may be all of the vocabulary, a later one is no wider than the rest)
        const int64_t rest = up(c.V - i * piece_width(p.cut, p.Tp), 256);
        if (hipError_t e = go<Deep>(ce_dw_kernel<Deep>, rest / Deep::BM * (up(c.K, Deep::BN) / Deep::BN), g, stream); e != hipSuccess) return e;
    }
    if (c.T == 0) return hipSuccess;
    ce_dx_store_kernel<S><<<(uint32_t)(tiles_m * g.tiles_n * (S::BM * S::BN / 8 / 256)), 256, 0, stream>>>(g);
    return hipGetLastError();
}

hipError_t launch_cross_entropy_bwd(const CrossEntropyArgs& c, hipStream_t stream)
{
    Plan p = make_plan(c.T, c.V, c.K, true, c.workspace);
    return p.small ? backward<Small>(c, p, stream) : backward<Big>(c, p, stream);
}

} // namespace fgs
