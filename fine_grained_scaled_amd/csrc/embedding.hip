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
// 2048 tokens an entry's place is the number of entries before it (16 waves
// compare 64 entries with the whole chunk from LDS), and a chunk's entries find
// their places among the other chunks by binary search: two launches for any
// number of tokens.
//
// The sorted list is cut into pieces of equal length whatever the tokens are, so
// that one token in most positions (padding) is summed by as many workgroups as
// any other input.  A sum that lies in one piece is written at once; the parts
// of one that spans pieces go to the workspace, and a last kernel adds them in
// a fixed order (one sum's by a workgroup for each 256 columns).  The rows that no token is get their zeros from workgroups of
// their own in the launch that sums, so each row of dw is written once.
//
// Measured: 16381 rows of 7168 FP32 values 160 us (5.9 TB/s); gradient of 8192
// tokens, 128000 x 4096 FP32, 423 us, 395 of them the launch that sums and clears
// (5.3 TB/s written), the sort 12; 61440 tokens, 70% of them the same, 32003 x 1024
// BF16 from FP32, 109 us: the sums 60, the sort 26, the long sum's parts 14.
#include <algorithm>
#include <climits>

#include "fgs_device.h"
#include "operators_internal.h"

namespace fgs {

namespace {

constexpr int CHUNK = 2048;            // tokens sorted at once
constexpr int TABLE = 64;              // entries a workgroup places
constexpr int SEARCHES = 4;            // chunks that a wave searches at once
constexpr int ZERO_ROWS = 64;          // rows of dw that a workgroup looks up and clears
constexpr int JOINERS = 8;             // waves that add one sum's parts
constexpr int MERGERS = 8;             // waves that search for the same entries

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
    int* spanning;                     // a counter to clear
};

__global__ __launch_bounds__(1024) void embedding_sort_kernel(SortArgs p)
{
    __shared__ __align__(16) int s_key[CHUNK];       // read four at a time
    __shared__ int s_rank[TABLE];
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.spanning = 0;
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
    const int block = first - base;                // the entries placed here
    int rank = 0;
    int k = lo;
    // equal keys in front of an entry come before it, those behind it do not;
    // what lies past the tokens holds the largest key and counts for none
    for (; k < min(hi, block); k += 4) {
        const int4 q = keys[k / 4];
        rank += (q.x <= key) + (q.y <= key) + (q.z <= key) + (q.w <= key);
    }
    for (; k < min(hi, block + TABLE); k += 4) {
        const int4 q = keys[k / 4];
        rank += (q.x < key + (k < mine)) + (q.y < key + (k + 1 < mine)) + (q.z < key + (k + 2 < mine)) + (q.w < key + (k + 3 < mine));
    }
    for (; k < hi; k += 4) {
        const int4 q = keys[k / 4];
        rank += (q.x < key) + (q.y < key) + (q.z < key) + (q.w < key);
    }
    atomicAdd(&s_rank[lane], rank);
    __syncthreads();
    if (wave == 0 && first + lane < p.T) p.sorted[base + s_rank[lane]] = make_int2(key, first + lane);
}

__global__ __launch_bounds__(64 * MERGERS) void embedding_merge_kernel(SortArgs p)
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
    for (int c0 = wave; c0 < chunks; c0 += MERGERS * SEARCHES) {
        // several chunks at a time: a search is a chain of loads
        const int2* at[SEARCHES];
        int n[SEARCHES], below[SEARCHES], found[SEARCHES] = {};
#pragma unroll
        for (int k = 0; k < SEARCHES; ++k) {
            const int c = c0 + MERGERS * k;
            at[k] = p.sorted + min(c, chunks - 1) * CHUNK;
            n[k] = c < chunks ? min(CHUNK, p.T - c * CHUNK) : 0;
            below[k] = entry.x + (c < chunk);          // keys below this one come first
        }
#pragma unroll
        for (int step = CHUNK; step > 0; step >>= 1) {
            int key[SEARCHES];
#pragma unroll
            for (int k = 0; k < SEARCHES; ++k) key[k] = at[k][max(min(found[k] + step, n[k]) - 1, 0)].x;
#pragma unroll
            for (int k = 0; k < SEARCHES; ++k) found[k] += found[k] + step <= n[k] && key[k] < below[k] ? step : 0;
        }
#pragma unroll
        for (int k = 0; k < SEARCHES; ++k) rank += c0 + MERGERS * k != chunk ? found[k] : 0;
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
    int T, V, W, piece, pieces, shift;
    const void* dout;
    int64_t ldd;
    void* dw;
    float scale;
    int add;                           // to what dw holds
    float* parts;                      // [pieces][2][W]: a piece's first and its last sum
    int* spanning;                     // how many sums span pieces, and the pieces in which they begin (in any order)
    int summers, columns;              // workgroups that sum, in front of those that write zeros; blocks along a row
};

// Zeros to those of rows first .. first + ZERO_ROWS - 1 of dw that no token is:
// a thread looks a row up in the sorted list.
template <bool WB>
__device__ __forceinline__ void write_zeros(const SumArgs& p, int64_t first)
{
    __shared__ uint8_t s_idle[ZERO_ROWS];
    const int rows = (int)min((int64_t)ZERO_ROWS, p.V - first);
    if ((int)threadIdx.x < rows) {
        const int key = (int)first + threadIdx.x;
        int found = 0;                 // entries below the key
        for (int step = 1 << (31 - __builtin_clz(p.T | 1)); step > 0; step >>= 1)
            if (found + step <= p.T && p.list[found + step - 1].x < key) found += step;
        s_idle[threadIdx.x] = found == p.T || p.list[found].x != key;
    }
    __syncthreads();
    const int vecs = p.W * (WB ? 2 : 4) / 16;
    uint4* base = static_cast<uint4*>(p.dw) + first * vecs;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (vecs >= 256) {
        for (int r = 0; r < rows; ++r)
            if (s_idle[r])
                for (int i = threadIdx.x; i < vecs; i += 256) base[(int64_t)r * vecs + i] = zero;
    } else {
        for (int i = threadIdx.x; i < rows * vecs; i += 256)
            if (s_idle[i / vecs]) base[i] = zero;
    }
}

// dw's row `key`, columns col .. col + N - 1
template <bool WB, int N>
__device__ __forceinline__ void write_sum(const SumArgs& p, int key, int col, const float* sum)
{
    if constexpr (WB) {
        uint16_t* at = static_cast<uint16_t*>(p.dw) + (int64_t)key * p.W + col;
        uint32_t w[N / 2] = {};
        if (p.add) {
            if constexpr (N == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(at);
            else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const bf16x2 v = {(__bf16)(bf16_lo(w[i]) + p.scale * sum[2 * i]), (__bf16)(bf16_hi(w[i]) + p.scale * sum[2 * i + 1])};
            w[i] = __builtin_bit_cast(uint32_t, v);
        }
        if constexpr (N == 8) *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(w);
        else *reinterpret_cast<uint2*>(at) = *reinterpret_cast<const uint2*>(w);
    } else {
        float4* at = reinterpret_cast<float4*>(static_cast<float*>(p.dw) + (int64_t)key * p.W + col);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            float4 v = p.add ? at[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v.x += p.scale * sum[4 * i], v.y += p.scale * sum[4 * i + 1];
            v.z += p.scale * sum[4 * i + 2], v.w += p.scale * sum[4 * i + 3];
            at[i] = v;
        }
    }
}

// 16 bytes of a row a thread: 8 BF16 or 4 FP32 columns.  WAVES: a piece takes
// whole waves, which then read the list once for all their lanes.
template <bool DB, bool WB, bool WAVES>
__global__ __launch_bounds__(256) void embedding_sum_kernel(SumArgs p)
{
    constexpr int N = DB ? 8 : 4, AHEAD = 16;
    if ((int)blockIdx.x >= p.summers) return write_zeros<WB>(p, (int64_t)((int)blockIdx.x - p.summers) * ZERO_ROWS);
    const int block = blockIdx.x, across = block % p.columns;
    int piece = (block / p.columns << (8 - p.shift)) + (threadIdx.x >> p.shift);
    if (WAVES) piece = __builtin_amdgcn_readfirstlane(piece);
    const int wanted = N * ((across << p.shift) + (threadIdx.x & ((1 << p.shift) - 1)));
    if (piece >= p.pieces) return;
    const int col = min(wanted, p.W - N);          // lanes past the row stay to hand out the list, and write nothing
    const int begin = piece * p.piece, end = min(begin + p.piece, p.T);
    const int before = begin > 0 ? p.list[begin - 1].x : -1, after = end < p.T ? p.list[end].x : -1;
    float* part = p.parts + (int64_t)piece * 2 * p.W + col;
    float sum[N] = {};
    int key = p.list[begin].x;
    bool first = true;                 // the run in hand began in front of the piece, or at its first entry
    // the run in hand is complete, or the piece ends
    auto flush = [&](bool last) {
        if (key >= p.V || wanted >= p.W) return;
        const bool cut_before = first && before == key, cut_after = last && after == key;
        if (!cut_before && !cut_after) return write_sum<WB, N>(p, key, col, sum);
        if (!cut_before && col == 0) p.spanning[1 + atomicAdd(p.spanning, 1)] = piece;
        // a whole piece of one token counts as a first sum
        float4* to = reinterpret_cast<float4*>(part + (cut_before ? 0 : p.W));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) to[i] = make_float4(sum[4 * i], sum[4 * i + 1], sum[4 * i + 2], sum[4 * i + 3]);
    };
    for (int i = begin; i < end; i += AHEAD) {
        int2 e[AHEAD];
        uint4 row[AHEAD];
        if constexpr (WAVES) {         // a lane's entry each, handed to all
            const int2 mine = p.list[min(i + (int)(threadIdx.x & (AHEAD - 1)), end - 1)];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                e[k] = make_int2(__builtin_amdgcn_readlane(mine.x, k), __builtin_amdgcn_readlane(mine.y, k));
        } else {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) e[k] = p.list[min(i + k, end - 1)];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            row[k] = *reinterpret_cast<const uint4*>(row_of<DB>(p.dout, e[k].y, p.ldd) + (DB ? 2 : 4) * (int64_t)col);
        // all loads are on their way before the first is used: the compiler would
        // move each behind the branches in front of its use
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) asm volatile("" : "+v"(row[k].x), "+v"(row[k].y), "+v"(row[k].z), "+v"(row[k].w));
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const bool there = i + k < end;
            if (there && e[k].x != key) {
                flush(false);
                key = e[k].x;
                first = false;
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] = 0.0f;
            }
            const uint32_t w[4] = {row[k].x, row[k].y, row[k].z, row[k].w};
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float v = DB ? j & 1 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]) : as_f32(w[j]);
                sum[j] = there ? sum[j] + v : sum[j];
            }
        }
    }
    flush(true);
}

// The sums that span pieces: from the piece in which one begins to the last that
// it reaches, the parts are added in the order of their numbers' residues by 8
// (a wave each, four columns a lane).
template <bool WB>
__global__ __launch_bounds__(64 * JOINERS) void embedding_join_kernel(SumArgs p)
{
    __shared__ float4 s_sum[JOINERS][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int count = p.spanning[0], col = 4 * ((int)blockIdx.y * 64 + lane);
    for (int i = blockIdx.x; i < count; i += gridDim.x) {
        const int piece = p.spanning[1 + i];
        const int key = p.list[(piece + 1) * p.piece].x;
        // the pieces that begin with the key: of the next 64, and where these all do, of the workgroup's threads at a time
        auto begins = [&](int64_t c) { return c < p.pieces && p.list[c * p.piece].x == key; };
        const uint64_t same = __ballot(begins(piece + 2 + lane));
        int last = piece + 1 + (same == ~0ull ? 64 : __builtin_ctzll(~same));
        for (int more = last == piece + 65 ? 64 * JOINERS : 0; more == 64 * JOINERS; last += more) more = __syncthreads_count(begins(last + 1 + (int)threadIdx.x));
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (col < p.W) {
#pragma unroll 16
            for (int c = piece + wave; c <= last; c += JOINERS) {
                const float4 v = *reinterpret_cast<const float4*>(p.parts + (2 * (int64_t)c + (c == piece)) * p.W + col);
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
        }
        s_sum[wave][lane] = sum;
        __syncthreads();
        if (wave == 0 && col < p.W) {
            const int waves = min(JOINERS, last - piece + 1);
            for (int w = 1; w < waves; ++w) {
                const float4 v = s_sum[w][lane];
                sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            write_sum<WB, 4>(p, key, col, &sum.x);
        }
        __syncthreads();
    }
}

struct Plan {
    int shift, columns, piece, pieces;
    int64_t sorted, merged, spanning, parts, bytes;      // offsets into the workspace
};

// threads a row: a power of two, 256 at most
int row_shift(int64_t vecs)
{
    int s = 0;
    while (s < 8 && (1 << s) < vecs) ++s;
    return s;
}

Plan make_plan(int64_t T, int64_t W, bool bf16)
{
    Plan p;
    const int64_t vecs = W / (bf16 ? 8 : 4);
    p.shift = row_shift(vecs);
    p.columns = (int)((vecs + (1 << p.shift) - 1) >> p.shift);
    // pieces as long as a thread's loads that overlap, longer where there are more than about 1024 workgroups
    const int64_t work = (T * p.columns) >> (8 - p.shift);
    p.piece = 16;
    while (p.piece < 256 && work / p.piece > 1024) p.piece *= 2;
    p.pieces = (int)((T + p.piece - 1) / p.piece);
    const auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.sorted = 0;
    p.merged = up(8 * T);
    p.spanning = p.merged + (T > CHUNK ? up(8 * T) : 0);
    p.parts = p.spanning + up(4 * (1 + p.pieces));
    p.bytes = p.parts + (p.pieces > 1 ? 8 * p.pieces * W : 0);
    return p;
}

} // namespace

size_t embedding_workspace_bytes(int64_t T, int64_t W)
{
    return (size_t)std::max(make_plan(T, W, false).bytes, make_plan(T, W, true).bytes);
}

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
    const Plan p = make_plan(a.T, a.W, a.bf16 != 0);
    char* ws = static_cast<char*>(a.workspace);
    SortArgs s{};
    s.tokens = a.tokens, s.wide = a.wide, s.T = (int)a.T, s.V = (int)a.V;
    s.sorted = reinterpret_cast<int2*>(ws + p.sorted), s.merged = reinterpret_cast<int2*>(ws + p.merged);
    s.spanning = reinterpret_cast<int*>(ws + p.spanning);
    const uint32_t tables = (uint32_t)((a.T + TABLE - 1) / TABLE);
    const bool chunks = a.T > CHUNK;
    if (tables) embedding_sort_kernel<<<tables, 1024, 0, stream>>>(s);
    if (chunks) embedding_merge_kernel<<<tables, 64 * MERGERS, 0, stream>>>(s);
    SumArgs m{};
    m.list = chunks ? s.merged : s.sorted;
    m.T = s.T, m.V = s.V, m.W = (int)a.W, m.piece = p.piece, m.pieces = p.pieces, m.shift = p.shift;
    m.dout = a.dout, m.ldd = a.ldd, m.dw = a.dweight, m.scale = a.scale, m.add = a.add;
    m.parts = reinterpret_cast<float*>(ws + p.parts), m.spanning = s.spanning;
    m.columns = p.columns;
    m.summers = (p.pieces + (256 >> p.shift) - 1) / (256 >> p.shift) * p.columns;
    const int64_t grid = m.summers + (a.add ? 0 : (a.V + ZERO_ROWS - 1) / ZERO_ROWS);
    if (grid == 0) return hipSuccess;
    void (*sum)(SumArgs);
    if (p.shift >= 6)
        sum = a.bf16 ? a.weight_bf16 ? embedding_sum_kernel<true, true, true> : embedding_sum_kernel<true, false, true>
                     : a.weight_bf16 ? embedding_sum_kernel<false, true, true> : embedding_sum_kernel<false, false, true>;
    else
        sum = a.bf16 ? a.weight_bf16 ? embedding_sum_kernel<true, true, false> : embedding_sum_kernel<true, false, false>
                     : a.weight_bf16 ? embedding_sum_kernel<false, true, false> : embedding_sum_kernel<false, false, false>;
    sum<<<(uint32_t)grid, 256, 0, stream>>>(m);
    if (p.pieces > 1) {
        auto join = a.weight_bf16 ? embedding_join_kernel<true> : embedding_join_kernel<false>;
        const int64_t columns = (a.W + 255) / 256;
        join<<<dim3((uint32_t)std::min<int64_t>(p.pieces - 1, std::max<int64_t>(8, 2048 / columns)), (uint32_t)columns), 64 * JOINERS, 0, stream>>>(m);
    }
    return hipGetLastError();
}

} // namespace fgs
