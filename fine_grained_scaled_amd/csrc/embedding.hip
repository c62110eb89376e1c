// embedding.hip -- token embedding and its gradient by sorted tokens, on gfx950.
//
//   out[t] = scale w[token[t]],
//   dw[v]  = scale times the sum of dout[t] over the t with token[t] = v
//            (added to dw, or with zeros where no token is v).
//
// Tokens outside the vocabulary read as zeros and have no gradient.
//
// The forward pass moves whole rows, bound by memory.  The gradient sorts the
// tokens first, stably, so that every sum runs over a contiguous piece of the
// sorted list in the order of the positions: no atomics, the same bits on every
// run, and each row of dout is read once.  The sort counts: within chunks of
// 4096 tokens an entry's place is the number of entries before it (16 waves
// compare 64 entries with the whole chunk from LDS), and a chunk's entries find
// their places among the other chunks by binary search.  Two launches for any
// number of tokens; the first also clears dw, which takes longer than the sort.
//
// The sorted list is cut into pieces of equal length whatever the tokens are, so
// that one token in most positions (padding) is summed by as many workgroups as
// any other input.  A sum that lies in one piece is written at once; the parts
// of one that spans pieces go to the workspace, and a last kernel adds them in
// the pieces' order.
#include <algorithm>
#include <climits>

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {

namespace {

constexpr int CHUNK = 4096;            // tokens sorted at once
constexpr int TABLE = 64;              // entries a workgroup places

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t t)
{
    return wide ? static_cast<const int64_t*>(tokens)[t] : static_cast<const int32_t*>(tokens)[t];
}

// Eight values of a row, as FP32.
template <bool BF16> struct Eight;
template <> struct Eight<true> {
    uint4 v;
    __device__ __forceinline__ void load(const void* row, int64_t vec) { v = static_cast<const uint4*>(row)[vec]; }
    __device__ __forceinline__ void get(float f[8]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
    }
    __device__ __forceinline__ static void store(void* row, int64_t vec, const float f[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2 p = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, p);
        }
        static_cast<uint4*>(row)[vec] = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<false> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* row, int64_t vec)
    {
        a = static_cast<const float4*>(row)[2 * vec];
        b = static_cast<const float4*>(row)[2 * vec + 1];
    }
    __device__ __forceinline__ void get(float f[8]) const
    {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    __device__ __forceinline__ static void store(void* row, int64_t vec, const float f[8])
    {
        static_cast<float4*>(row)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4*>(row)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

template <bool BF16>
__device__ __forceinline__ const char* row_of(const void* base, int64_t row, int64_t ld)
{
    return static_cast<const char*>(base) + row * ld * (BF16 ? 2 : 4);
}

// ------------------------------------------------------------------------
// Forward: `lanes` threads a row.
// ------------------------------------------------------------------------
template <bool WB, bool OB>
__global__ __launch_bounds__(256) void embedding_rows_kernel(const void* tokens, int wide, int64_t T, const void* w,
                                                             int64_t ldw, int64_t V, int vecs, int shift, float scale, void* out)
{
    const int64_t t = ((int64_t)blockIdx.x << (8 - shift)) + (threadIdx.x >> shift);
    if (t >= T) return;
    const int64_t v = token_at(tokens, wide, t);
    const bool in = v >= 0 && v < V;
    const char* from = row_of<WB>(w, in ? v : 0, ldw);
    char* to = const_cast<char*>(row_of<OB>(out, t, 8 * (int64_t)vecs));
    for (int i = threadIdx.x & ((1 << shift) - 1); i < vecs; i += 1 << shift) {
        float f[8] = {};
        if (in) {
            Eight<WB> e;
            e.load(from, i);
            e.get(f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= scale;
        }
        Eight<OB>::store(to, i, f);
    }
}

// ------------------------------------------------------------------------
// The sort.  Tokens outside the vocabulary take the key V, behind all others.
// ------------------------------------------------------------------------
struct SortArgs {
    const void* tokens;
    int wide;
    int T, V;
    int2 *sorted, *merged;             // (key, position): by chunk, and of all
    uint4* clear;                      // dw, where the call clears it
    int64_t clear_vecs;
    int sorters;                       // workgroups that sort; the others clear
};

__global__ __launch_bounds__(1024) void embedding_sort_kernel(SortArgs p)
{
    __shared__ int s_key[CHUNK];
    __shared__ int s_rank[TABLE];
    if ((int)blockIdx.x >= p.sorters) {
        const int64_t step = (int64_t)(gridDim.x - p.sorters) * 1024;
        for (int64_t i = (int64_t)(blockIdx.x - p.sorters) * 1024 + threadIdx.x; i < p.clear_vecs; i += step)
            p.clear[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int first = blockIdx.x * TABLE, base = first & ~(CHUNK - 1);
    for (int i = threadIdx.x; i < CHUNK; i += 1024) {
        int key = INT_MAX;
        if (base + i < p.T) {
            const int64_t v = token_at(p.tokens, p.wide, base + i);
            key = v >= 0 && v < p.V ? (int)v : p.V;
        }
        s_key[i] = key;
    }
    if (threadIdx.x < TABLE) s_rank[threadIdx.x] = 0;
    __syncthreads();
    const int mine = first - base + lane, key = min(s_key[mine], p.V);
    const int n = min(CHUNK, p.T - base), per = CHUNK / 16;
    const int lo = wave * per, hi = min(lo + per, n);
    const int4* keys = reinterpret_cast<const int4*>(s_key);
    int rank = 0;
    for (int k = lo; k < hi; k += 4) {             // entries past n hold the largest key and count for none
        const int4 q = keys[k / 4];
        rank += q.x < key + (k < mine);            // an equal key in front of this one counts
        rank += q.y < key + (k + 1 < mine);
        rank += q.z < key + (k + 2 < mine);
        rank += q.w < key + (k + 3 < mine);
    }
    atomicAdd(&s_rank[lane], rank);
    __syncthreads();
    if (wave == 0 && first + lane < p.T) p.sorted[base + s_rank[lane]] = make_int2(key, first + lane);
}

__global__ __launch_bounds__(1024) void embedding_merge_kernel(SortArgs p)
{
    __shared__ int s_rank[TABLE];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int first = blockIdx.x * TABLE, chunk = first / CHUNK;
    if (threadIdx.x < TABLE) s_rank[threadIdx.x] = 0;
    __syncthreads();
    const int e = min(first + lane, p.T - 1);
    const int2 entry = p.sorted[e];
    const int chunks = (p.T + CHUNK - 1) / CHUNK;
    int rank = 0;
    for (int c = wave; c < chunks; c += 16) {
        if (c == chunk) continue;
        const int2* at = p.sorted + c * CHUNK;
        const int n = min(CHUNK, p.T - c * CHUNK), below = entry.x + (c < chunk);      // keys below this one come first
        int found = 0;
        for (int step = CHUNK; step > 0; step >>= 1)
            if (found + step <= n && at[found + step - 1].x < below) found += step;
        rank += found;
    }
    atomicAdd(&s_rank[lane], rank);
    __syncthreads();
    if (wave == 0 && first + lane < p.T) p.merged[e - chunk * CHUNK + s_rank[lane]] = entry;
}

// ------------------------------------------------------------------------
// The sums over pieces of the sorted list
// ------------------------------------------------------------------------
struct SumArgs {
    const int2* list;                  // T entries
    int T, V, vecs, piece, pieces, shift;
    const void* dout;
    int64_t ldd;
    void* dw;
    float scale;
    int add;                           // to what dw holds
    float* parts;                      // [pieces][2][8 vecs]: a piece's first and its last sum
};

template <bool WB>
__device__ __forceinline__ void write_sum(const SumArgs& p, int key, int vec, const float sum[8])
{
    char* row = const_cast<char*>(row_of<WB>(p.dw, key, 8 * (int64_t)p.vecs));
    float f[8] = {};
    if (p.add) {
        Eight<WB> old;
        old.load(row, vec);
        old.get(f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] += p.scale * sum[k];
    Eight<WB>::store(row, vec, f);
}

template <bool DB, bool WB>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs p)
{
    constexpr int AHEAD = 8;
    const int piece = ((int)blockIdx.x << (8 - p.shift)) + (threadIdx.x >> p.shift);
    const int vec = (int)(blockIdx.y << p.shift) + (threadIdx.x & ((1 << p.shift) - 1));
    if (piece >= p.pieces || vec >= p.vecs) return;
    const int begin = piece * p.piece, end = min(begin + p.piece, p.T);
    const int before = begin > 0 ? p.list[begin - 1].x : -1, after = end < p.T ? p.list[end].x : -1;
    float* part = p.parts + ((int64_t)piece * 2 * p.vecs + vec) * 8;
    float sum[8] = {};
    int key = p.list[begin].x;
    bool first = true;                 // the run in hand began in front of the piece, or at its first entry
    // the run in hand is complete, or the piece ends
    auto flush = [&](bool last) {
        if (key >= p.V) return;
        const bool cut_before = first && before == key, cut_after = last && after == key;
        if (!cut_before && !cut_after) return write_sum<WB>(p, key, vec, sum);
        // a whole piece of one token counts as a first sum
        Eight<false>::store(part + (cut_before ? 0 : 8 * (int64_t)p.vecs), 0, sum);
    };
    for (int i = begin; i < end; i += AHEAD) {
        int2 e[AHEAD];
        Eight<DB> row[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) e[k] = p.list[min(i + k, end - 1)];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) row[k].load(row_of<DB>(p.dout, e[k].y, p.ldd), vec);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i + k >= end) break;
            if (e[k].x != key) {
                flush(false);
                key = e[k].x;
                first = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
            }
            float f[8];
            row[k].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += f[j];
        }
    }
    flush(true);
}

// The sums that span pieces: the piece in which one begins finds the last that
// it reaches and adds the parts, 16 at a time over the workgroup's rows.
template <bool WB>
__global__ __launch_bounds__(1024) void embedding_join_kernel(SumArgs p)
{
    __shared__ float s_sum[16][64][9];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int piece = blockIdx.x;                          // there is one behind it
    const int begin = piece * p.piece, next = begin + p.piece;
    const int key = p.list[next - 1].x;
    if (key >= p.V || p.list[next].x != key) return;
    const bool whole = p.list[begin].x == key;
    if (whole && begin > 0 && p.list[begin - 1].x == key) return;      // began earlier
    int last = piece;
    for (;;) {
        const int c = last + 1 + lane;
        const uint64_t same = __ballot(c < p.pieces && p.list[(int64_t)c * p.piece].x == key);
        const int run = same == ~0ull ? 64 : __builtin_ctzll(~same);
        last += run;
        if (run < 64) break;
    }
    const int vec = (int)blockIdx.y * 64 + lane;
    const int64_t row = 8 * (int64_t)p.vecs;
    float sum[8] = {};
    if (vec < p.vecs) {
        for (int c = piece + wave; c <= last; c += 16) {
            Eight<false> e;
            e.load(p.parts + 2 * row * c + (c == piece ? row : 0), vec);
            float f[8];
            e.get(f);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += f[k];
        }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s_sum[wave][lane][k] = sum[k];
    __syncthreads();
    if (wave == 0 && vec < p.vecs) {
        const int waves = min(16, last - piece + 1);
        for (int w = 1; w < waves; ++w)
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += s_sum[w][lane][k];
        write_sum<WB>(p, key, vec, sum);
    }
}

struct Plan {
    int vecs, shift, columns, piece, pieces;
    int64_t sorted, merged, parts, bytes;      // offsets into the workspace
};

// threads a row: a power of two, 256 at most
int row_shift(int64_t vecs)
{
    int s = 0;
    while (s < 8 && (1 << s) < vecs) ++s;
    return s;
}

Plan make_plan(int64_t T, int64_t W)
{
    Plan p;
    p.vecs = (int)(W / 8);
    p.shift = row_shift(p.vecs);
    p.columns = (p.vecs + (1 << p.shift) - 1) >> p.shift;
    // pieces long enough for a thread's loads to overlap, short enough for about 1024 workgroups
    const int64_t work = (T * p.columns) >> (8 - p.shift);
    p.piece = 16;
    while (p.piece < 256 && work / p.piece > 1024) p.piece *= 2;
    p.pieces = (int)((T + p.piece - 1) / p.piece);
    const auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.sorted = 0;
    p.merged = up(8 * T);
    p.parts = p.merged + (T > CHUNK ? up(8 * T) : 0);
    p.bytes = p.parts + (p.pieces > 1 ? 8 * p.pieces * W : 0);
    return p;
}

} // namespace

size_t embedding_workspace_bytes(int64_t T, int64_t W) { return (size_t)make_plan(T, W).bytes; }

hipError_t launch_embedding_fwd(const EmbeddingArgs& a, hipStream_t stream)
{
    const int vecs = (int)(a.W / 8), shift = row_shift(vecs);
    const uint32_t grid = (uint32_t)((a.T + (256 >> shift) - 1) / (256 >> shift));
    auto kernel = a.weight_bf16 ? a.bf16 ? embedding_rows_kernel<true, true> : embedding_rows_kernel<true, false>
                                : a.bf16 ? embedding_rows_kernel<false, true> : embedding_rows_kernel<false, false>;
    kernel<<<grid, 256, 0, stream>>>(a.tokens, a.wide, a.T, a.weight, a.ldw, a.V, vecs, shift, a.scale, a.out);
    return hipGetLastError();
}

hipError_t launch_embedding_bwd(const EmbeddingArgs& a, hipStream_t stream)
{
    const Plan p = make_plan(a.T, a.W);
    char* ws = static_cast<char*>(a.workspace);
    SortArgs s{};
    s.tokens = a.tokens, s.wide = a.wide, s.T = (int)a.T, s.V = (int)a.V;
    s.sorted = reinterpret_cast<int2*>(ws + p.sorted), s.merged = reinterpret_cast<int2*>(ws + p.merged);
    s.sorters = (int)((a.T + TABLE - 1) / TABLE);
    int64_t clearers = 0;
    if (!a.add) {
        s.clear = static_cast<uint4*>(a.dweight);
        s.clear_vecs = a.V * a.W * (a.weight_bf16 ? 2 : 4) / 16;
        clearers = std::min<int64_t>(2048, (s.clear_vecs + 1023) / 1024);
    }
    if (s.sorters + clearers == 0) return hipSuccess;
    embedding_sort_kernel<<<(uint32_t)(s.sorters + clearers), 1024, 0, stream>>>(s);
    if (a.T == 0) return hipGetLastError();
    const bool chunks = a.T > CHUNK;
    if (chunks) embedding_merge_kernel<<<(uint32_t)s.sorters, 1024, 0, stream>>>(s);
    SumArgs m{};
    m.list = chunks ? s.merged : s.sorted;
    m.T = s.T, m.V = s.V, m.vecs = p.vecs, m.piece = p.piece, m.pieces = p.pieces, m.shift = p.shift;
    m.dout = a.dout, m.ldd = a.ldd, m.dw = a.dweight, m.scale = a.scale, m.add = a.add;
    m.parts = reinterpret_cast<float*>(ws + p.parts);
    const dim3 grid((uint32_t)((p.pieces + (256 >> p.shift) - 1) / (256 >> p.shift)), (uint32_t)p.columns);
    auto sum = a.bf16 ? a.weight_bf16 ? embedding_sum_kernel<true, true> : embedding_sum_kernel<true, false>
                      : a.weight_bf16 ? embedding_sum_kernel<false, true> : embedding_sum_kernel<false, false>;
    sum<<<grid, 256, 0, stream>>>(m);
    if (p.pieces > 1) {
        auto join = a.weight_bf16 ? embedding_join_kernel<true> : embedding_join_kernel<false>;
        join<<<dim3((uint32_t)(p.pieces - 1), (uint32_t)((p.vecs + 63) / 64)), 1024, 0, stream>>>(m);
    }
    return hipGetLastError();
}

} // namespace fgs
