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
// dz goes to the matrix units in BF16, divided by the largest |dloss| (|dlse|)
// of the call, which the results are multiplied with again in FP32: under a
// mean over the tokens the values are then softmax - onehot itself, whose
// largest, those of the targets, round best (-1 exactly).
#include <algorithm>
#include <cmath>

#include "product_device.h"

namespace fgs {

namespace {

using namespace prod;

using Big = Shape<2, 4, 4, 2>;         // 256 x 256, 8 waves of 128 x 64
using Small = Shape<1, 4, 2, 1>;       // 64 x 128, 4 waves of 64 x 32: up to 64 tokens

constexpr float LOG2E = 1.44269504088896340736f;

// What the rows with a target need, in their order (padded with zeros to a
// multiple of 256 rows).
struct Rows {
    int32_t* count;        // [1]
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

// One workgroup lists the rows with a target.
__global__ __launch_bounds__(1024) void ce_rows_kernel(const void* targets, int wide, int64_t T, int64_t V, Rows r,
                                                       const float* dloss, const float* dlse, const float* lse)
{
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
            if (dloss) {
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
        if (dloss) r.dloss[i] = r.dlse[i] = r.lse[i] = 0.0f;
    }
    if (dloss) {
        if (bad) top = INFINITY;
        for (int m = 1; m < 64; m *= 2) top = fmaxf(top, __shfl_xor(top, m));
        if (lane == 0) s_top[wave] = top;
        __syncthreads();
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s_top[i]);
    }
    if (threadIdx.x == 0) {
        *r.count = before;
        if (dloss) *r.most = top > 0.0f && top < INFINITY ? top : 1.0f;
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
    int64_t ldx, ldw, T, V, v0;        // the vocabulary from v0 on
    int K, tiles_n;
    const void* targets;               // the forward pass without a list of rows
    int wide;
    Rows r;                            // r.count nullptr: every token is a row
    int64_t Tp;
    float2* part;                      // [tiles_n][Tp]
    float* z_target;                   // [Tp]
    uint16_t* dz;                      // [Tp][ldz] (backward)
    int64_t ldz;
};

template <class S>
__device__ __forceinline__ bool score_tile(const ScoreArgs& p, f32x16 (&acc)[S::TI][S::TJ], int64_t& rows, int64_t& m0,
                                           int64_t& n0, int& tn, char* smem)
{
    rows = p.r.count ? *p.r.count : p.T;
    const int tiles_m = (int)((rows + S::BM - 1) / S::BM);
    if ((int64_t)blockIdx.x >= (int64_t)tiles_m * p.tiles_n) return false;
    int tm;
    tile_of(blockIdx.x, tiles_m, p.tiles_n, tm, tn);
    m0 = (int64_t)tm * S::BM, n0 = p.v0 + (int64_t)tn * S::BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Loader<ALONG, S::BM, S::NW> la;
    Loader<ALONG, S::BN, S::NW> lb;
    la.rows([&](int r) {
        int64_t row = min(m0 + r, rows - 1);
        if (p.r.token) row = p.r.token[row];
        return p.x + row * p.ldx;
    }, wave, lane);
    lb.rows([&](int r) { return p.w + min(n0 + r, p.V - 1) * p.ldw; }, wave, lane);
    product<S, ALONG, ALONG>(acc, la, lb, p.K, smem);
    return true;
}

template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_score_kernel(ScoreArgs p)
{
    extern __shared__ __align__(256) char smem[];
    f32x16 acc[S::TI][S::TJ];
    int64_t rows, m0, n0;
    int tn;
    if (!score_tile<S>(p, acc, rows, m0, n0, tn, smem)) return;
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
__global__ __launch_bounds__(S::THREADS, 1) void ce_gradient_kernel(ScoreArgs p)
{
    extern __shared__ __align__(256) char smem[];
    f32x16 acc[S::TI][S::TJ];
    int64_t rows, m0, n0;
    int tn;
    if (!score_tile<S>(p, acc, rows, m0, n0, tn, smem)) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, half = lane >> 5;
    const int wm = wave / S::NWN, wn = wave % S::NWN;
    const int64_t nw = n0 + wn * S::WN;
    const float most = *p.r.most;
#pragma unroll
    for (int i = 0; i < S::TI; ++i) {
        const int64_t row = m0 + wm * S::WM + 32 * i + (lane & 31);      // within the padded rows
        const float lse = p.r.lse[row], b = p.r.dloss[row] / most, a = b + p.r.dlse[row] / most;
        const int target = p.r.target[row];
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const int64_t n = nw + 32 * j + acc_n(k, half);
                float v = a * __builtin_amdgcn_exp2f((acc[i][j][k] - lse) * LOG2E);
                if (n == target) v -= b;
                acc[i][j][k] = row < rows && n < p.V ? v : 0.0f;
            }
    }
    store_tile<S>(smem, [&](int i, int j, int k) { return acc[i][j][k]; },
                  [&](int row, int c) { return p.dz + (m0 + row) * p.ldz + (n0 - p.v0) + 8 * c; });
}

struct GradArgs {
    const uint16_t *dz, *w, *xc;
    int64_t ldz, ldw, V, v0, width;    // width: vocabulary of the piece, padded to 256
    int K, tiles_n, tiles_m, splits, first;
    int64_t per;                       // contraction values a split (dx)
    Rows r;
    float* sums;                       // [splits][tiles_m][tiles_n][BM x BN]
    uint16_t *dx, *dw;
};

// dx += dz w over the piece's vocabulary, or a split of it; the sums stay in
// the accumulators' order.
template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_dx_kernel(GradArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const int64_t rows = *p.r.count;
    const int tiles_m = (int)((rows + S::BM - 1) / S::BM);
    const int64_t each = (int64_t)tiles_m * p.tiles_n;
    if ((int64_t)blockIdx.x >= each * p.splits) return;
    const int split = (int)(blockIdx.x / each);
    int tm, tn;
    tile_of(blockIdx.x - split * each, tiles_m, p.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN, k0 = split * p.per;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t values = max((int64_t)0, min(p.per, min(p.width, p.V - p.v0) - k0));
    Loader<ALONG, S::BM, S::NW> la;
    Loader<ACROSS, S::BN, S::NW> lb;
    la.rows([&](int r) { return p.dz + (m0 + r) * p.ldz + k0; }, wave, lane);
    lb.columns(p.w + min(p.v0 + k0, p.V - 1) * p.ldw, p.ldw, n0, p.K, wave, lane);
    f32x16 acc[S::TI][S::TJ];
    product<S, ALONG, ACROSS>(acc, la, lb, values, smem);
    float4* sums = reinterpret_cast<float4*>(p.sums) +
                   (((int64_t)split * p.tiles_m + tm) * p.tiles_n + tn) * (S::BM * S::BN / 4) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float4* at = sums + ((i * S::TJ + j) * 4 + g) * S::THREADS;
                float4 v = make_float4(acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
                if (!p.first) {
                    const float4 o = *at;
                    v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                }
                *at = v;
            }
}

// The splits' sums to the tokens' rows of dx.
template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_dx_store_kernel(GradArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const int64_t rows = *p.r.count;
    const int tm = blockIdx.x / p.tiles_n, tn = blockIdx.x % p.tiles_n;
    const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN;
    if (m0 >= rows) return;
    const float scale = *p.r.most;
    f32x16 acc[S::TI][S::TJ];
#pragma unroll
    for (int i = 0; i < S::TI; ++i)
#pragma unroll
        for (int j = 0; j < S::TJ; ++j) acc[i][j] = f32x16{};
    for (int s = 0; s < p.splits; ++s) {
        const float4* sums = reinterpret_cast<const float4*>(p.sums) +
                             (((int64_t)s * p.tiles_m + tm) * p.tiles_n + tn) * (S::BM * S::BN / 4) + threadIdx.x;
#pragma unroll
        for (int i = 0; i < S::TI; ++i)
#pragma unroll
            for (int j = 0; j < S::TJ; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float4 v = sums[((i * S::TJ + j) * 4 + g) * S::THREADS];
                    acc[i][j][4 * g] += v.x, acc[i][j][4 * g + 1] += v.y;
                    acc[i][j][4 * g + 2] += v.z, acc[i][j][4 * g + 3] += v.w;
                }
    }
    store_tile<S>(smem, [&](int i, int j, int k) { return acc[i][j][k] * scale; },
                  [&](int row, int c) -> uint16_t* {
                      if (m0 + row >= rows || n0 + 8 * c >= p.K) return nullptr;
                      return p.dx + (int64_t)p.r.token[m0 + row] * p.K + n0 + 8 * c;
                  });
}

// The piece's rows of dw = dz^T x.
template <class S>
__global__ __launch_bounds__(S::THREADS, 1) void ce_dw_kernel(GradArgs p)
{
    extern __shared__ __align__(256) char smem[];
    const int64_t rows = *p.r.count;
    int tm, tn;
    tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * S::BM, n0 = (int64_t)tn * S::BN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Loader<ACROSS, S::BM, S::NW> la;
    Loader<ACROSS, S::BN, S::NW> lb;
    la.columns(p.dz, p.ldz, m0, p.ldz, wave, lane);
    lb.columns(p.xc, p.K, n0, p.K, wave, lane);
    f32x16 acc[S::TI][S::TJ];
    product<S, ACROSS, ACROSS>(acc, la, lb, (rows + BK - 1) / BK * BK, smem);
    const float scale = *p.r.most;
    store_tile<S>(smem, [&](int i, int j, int k) { return acc[i][j][k] * scale; },
                  [&](int row, int c) -> uint16_t* {
                      const int64_t v = p.v0 + m0 + row;
                      if (v >= p.V || m0 + row >= p.width || n0 + 8 * c >= p.K) return nullptr;
                      return p.dw + v * p.K + n0 + 8 * c;
                  });
}

// Up to 64 tokens the rows of a 256 x 256 tile would be padding for the most
// part, and its 8 waves would wait for one tile's loads.
constexpr int64_t SMALL = 64;
// dz of one piece of the vocabulary: 256 MiB at most where that is 8192 wide or more.
constexpr int64_t PIECE_VALUES = (int64_t)1 << 27, PIECE_LEAST = 8192;

int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

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
    int64_t Tp, piece = 0;
    bool small, list;
    int tiles_n = 0, splits = 1, dx_m = 0, dx_n = 0;
    int64_t per = 0;
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
    p.Tp = up(std::max<int64_t>(T, 1), 256);
    // the forward pass of one tile of tokens gains nothing from a list of rows
    p.list = backward || T > Big::BM;
    if (p.list) {
        p.r.count = at.take<int32_t>(1);
        p.r.most = at.take<float>(1);
        p.r.place = at.take<int32_t>(p.Tp);
        p.r.token = at.take<int32_t>(p.Tp);
        p.r.target = at.take<int32_t>(p.Tp);
    }
    if (!backward) {
        p.tiles_n = (int)(up(V, p.small ? Small::BN : Big::BN) / (p.small ? Small::BN : Big::BN));
        p.part = at.take<float2>(p.tiles_n * p.Tp);
        p.z_target = at.take<float>(p.Tp);
    } else {
        p.r.lse = at.take<float>(p.Tp), p.r.dloss = at.take<float>(p.Tp), p.r.dlse = at.take<float>(p.Tp);
        p.xc = at.take<uint16_t>(p.Tp * K);
        p.piece = std::min(up(V, 256), std::max(PIECE_VALUES / p.Tp / 256 * 256, PIECE_LEAST));
        p.dz = at.take<uint16_t>(p.Tp * p.piece);
        const int bm = p.small ? Small::BM : Big::BM, bn = p.small ? Small::BN : Big::BN;
        p.dx_m = (int)(up(std::max<int64_t>(T, 1), bm) / bm), p.dx_n = (int)(up(K, bn) / bn);
        // few tiles of dx: the vocabulary is split over workgroups, 1024 values each at least
        const int64_t tiles = (int64_t)p.dx_m * p.dx_n;
        p.splits = (int)std::max<int64_t>(1, std::min(512 / tiles, p.piece / 1024));
        p.per = up((p.piece + p.splits - 1) / p.splits, BK);
        p.sums = at.take<float>(p.splits * tiles * bm * bn);
    }
    p.bytes = at.bytes;
    return p;
}

template <class S, class A>
hipError_t go(void (*kernel)(A), int64_t grid, const A& a, hipStream_t stream)
{
    if (grid == 0) return hipSuccess;
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
    if (p.list) ce_rows_kernel<<<1, 1024, 0, stream>>>(c.targets, c.wide, c.T, c.V, p.r, nullptr, nullptr, nullptr);
    hipError_t e = p.small ? go<Small>(ce_score_kernel<Small>, p.tiles_n, s, stream)
                           : go<Big>(ce_score_kernel<Big>, p.Tp / Big::BM * p.tiles_n, s, stream);
    if (e != hipSuccess) return e;
    ce_join_kernel<<<(uint32_t)((c.T + 15) / 16), 1024, 0, stream>>>(s, c.loss, c.lse);
    return hipGetLastError();
}

hipError_t launch_cross_entropy_bwd(const CrossEntropyArgs& c, hipStream_t stream)
{
    const Plan p = make_plan(c.T, c.V, c.K, true, c.workspace);
    ScoreArgs s = score_args(c, p);
    ce_rows_kernel<<<1, 1024, 0, stream>>>(c.targets, c.wide, c.T, c.V, p.r, c.dloss, c.dlse, c.lse);
    ce_gather_kernel<<<(uint32_t)(c.T + 256), 256, 0, stream>>>(s.x, c.ldx, c.T, (int)c.K, p.r, p.xc, static_cast<uint16_t*>(c.dx));
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    s.x = p.xc, s.ldx = c.K, s.r.token = nullptr;
    s.dz = p.dz, s.ldz = p.piece;
    GradArgs g{};
    g.dz = p.dz, g.w = s.w, g.xc = p.xc, g.ldz = p.piece, g.ldw = c.ldw, g.V = c.V, g.K = (int)c.K;
    g.splits = p.splits, g.per = p.per, g.r = p.r, g.sums = p.sums;
    g.dx = static_cast<uint16_t*>(c.dx), g.dw = static_cast<uint16_t*>(c.dw);
    for (int64_t v0 = 0; v0 < c.V; v0 += p.piece) {
        const int64_t width = up(std::min(p.piece, c.V - v0), 256);
        s.v0 = g.v0 = v0, g.width = width;
        g.first = v0 == 0;
        s.tiles_n = (int)(width / (p.small ? Small::BN : Big::BN));
        hipError_t e = p.small ? go<Small>(ce_gradient_kernel<Small>, s.tiles_n, s, stream)
                               : go<Big>(ce_gradient_kernel<Big>, p.Tp / Big::BM * s.tiles_n, s, stream);
        if (e != hipSuccess) return e;
        g.tiles_m = p.dx_m, g.tiles_n = p.dx_n;
        const int64_t grid = (int64_t)p.dx_m * p.dx_n * p.splits;
        e = p.small ? go<Small>(ce_dx_kernel<Small>, grid, g, stream) : go<Big>(ce_dx_kernel<Big>, grid, g, stream);
        if (e != hipSuccess) return e;
        g.tiles_m = (int)(width / Big::BM), g.tiles_n = (int)(up(c.K, Big::BN) / Big::BN);
        if ((e = go<Big>(ce_dw_kernel<Big>, (int64_t)g.tiles_m * g.tiles_n, g, stream)) != hipSuccess) return e;
    }
    if (c.T == 0) return hipSuccess;
    g.tiles_m = p.dx_m, g.tiles_n = p.dx_n;
    const int64_t grid = (int64_t)p.dx_m * p.dx_n;
    return p.small ? go<Small>(ce_dx_store_kernel<Small>, grid, g, stream) : go<Big>(ce_dx_store_kernel<Big>, grid, g, stream);
}

} // namespace fgs
